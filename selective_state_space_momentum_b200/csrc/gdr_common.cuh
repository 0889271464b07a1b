// gdr_common.cuh -- what the chunked gated-delta-rule kernels share: the
// chunk records, swizzled shared-memory tiles and the warp matrix products.
#pragma once

#include "mm_common.cuh"
#include "mm_internal.h"
#include "mm_tma_host.h"

namespace mmscan {
namespace gdr {

constexpr int C = kGdrChunk;               // steps of a chunk

// Per (batch row, head, chunk) record, written by the preparing kernel:
//   T   (C, C) bf16   (I + A)^-1, A_ij = beta_i e^(c_i - c_j) k_i.k_j (j < i),
//                     c the cumulative g of the chunk
//   Pm  (C, C) bf16   scale e^(c_i - c_j) q_i.k_j (j <= i)
//   eg, tail, beta (C) fp32: e^(c_i), e^(c_last - c_i), beta_i
// and, apart from it, Tlo (C, C) bf16, what T's rounding to bf16 left over.
// The matrices are images of their shared-memory tiles (tile_off<128>), so
// that they are copied piece by piece.
constexpr int REC_T = 0, REC_P = C * C * 2, REC_F = 2 * C * C * 2;
constexpr int REC_BYTES = REC_F + 3 * C * 4;
static_assert(REC_BYTES == kGdrRecBytes, "record size");

// Tiles in shared memory: rows of 128 bytes, the 16-byte pieces of a row
// permuted by the row's number mod 8, so that the eight rows an ldmatrix
// reads at one column lie in different banks.
template <int RB>
__device__ __forceinline__ uint32_t tile_off(int row, int c16) {
    return (uint32_t)(row * RB + ((c16 ^ (row & 7)) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void stsm4t(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
                 :: "r"(a), "r"(r0), "r"(r1), "r"(r2), "r"(r3) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Operand fragments from a tile; `lane` 0..31, every index in elements of 8
// (c16) or rows.
// B (k x n) of two neighbouring n-tiles from a tile stored [n][k].
template <int RB>
__device__ __forceinline__ void load_b_nk(uint32_t tile, int n0, int kc, int lane, uint32_t (&r)[4]) {
    const int m = lane >> 3;
    ldsm4(tile + tile_off<RB>(n0 + (m >> 1) * 8 + (lane & 7), kc + (m & 1)), r);
}
// A (16 x 16) from a tile stored [m][k] / [k][m].
template <int RB>
__device__ __forceinline__ void load_a_mk(uint32_t tile, int m0, int kc, int lane, uint32_t (&r)[4]) {
    const int m = lane >> 3;
    ldsm4(tile + tile_off<RB>(m0 + (m & 1) * 8 + (lane & 7), kc + (m >> 1)), r);
}
template <int RB>
__device__ __forceinline__ void load_a_km(uint32_t tile, int k0, int mc, int lane, uint32_t (&r)[4]) {
    const int m = lane >> 3;
    ldsm4t(tile + tile_off<RB>(k0 + (m >> 1) * 8 + (lane & 7), mc + (m & 1)), r);
}

// fp32 values in two bf16 terms: hi + lo is the fp32 value to 2^-16.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16x2(x, y);
    lo = pack_bf16x2(x - bf16_lo(hi), y - bf16_hi(hi));
}
// The A operand of k-step kt from accumulators c (the product before it), in
// two terms.
template <int NT>
__device__ __forceinline__ void acc_to_a2(const float (&c)[NT][4], int kt, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
    split2(c[2 * kt][0], c[2 * kt][1], hi[0], lo[0]);
    split2(c[2 * kt][2], c[2 * kt][3], hi[1], lo[1]);
    split2(c[2 * kt + 1][0], c[2 * kt + 1][1], hi[2], lo[2]);
    split2(c[2 * kt + 1][2], c[2 * kt + 1][3], hi[3], lo[3]);
}

// Cumulative g of a chunk in 64 bits, by one warp; lane l gets the sums at
// rows 2 l and 2 l + 1 and the chunk's last.  The decays are exponentials of
// differences of these sums, and one strongly negative g would take the low
// bits of the others' differences in fp32.  Below -1e4 (-inf included) a step
// forgets everything (e^g = 0 either way): clamped, so that no difference is
// inf - inf.  `g` points at the chunk's first step, `stride` elements apart.
__device__ __forceinline__ void chunk_cumsum(const bf16* g, int64_t stride, int valid, int lane, double& s0, double& s1, double& last) {
    const int r = 2 * lane;
    s0 = s1 = 0.0;
    if (r < valid) {
        const float x = __bfloat162float(g[r * stride]);
        s0 = x < -1e4f ? -1e4f : x;
    }
    if (r + 1 < valid) {
        const float x = __bfloat162float(g[(r + 1) * stride]);
        s1 = x < -1e4f ? -1e4f : x;
    }
    s1 += s0;
    double run = s1;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, run, m);
        if (lane >= m) run += up;
    }
    s0 += run - s1;
    s1 = run;
    last = __shfl_sync(0xffffffffu, run, 31);
}

// The A operand back to a tile stored [k][m].
template <int RB>
__device__ __forceinline__ void store_a_km(uint32_t tile, int k0, int mc, int lane, const uint32_t (&r)[4]) {
    const int m = lane >> 3;
    stsm4t(tile + tile_off<RB>(k0 + (m >> 1) * 8 + (lane & 7), mc + (m & 1)), r[0], r[1], r[2], r[3]);
}

// `bytes` (a multiple of 16) of consecutive global memory into shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// `bytes` of shared memory to consecutive global memory (this thread's bulk group).
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" :: "l"(dst), "r"(src), "r"(bytes) : "memory");
}

// mbar_wait for waits on the critical path: a try may sleep in hardware for up
// to 20 us (a polling warp takes issue slots and shared-memory cycles from the
// ones that work), and the limit's clock is read only between tries.
__device__ __forceinline__ bool mbar_wait_sleep(uint32_t bar, uint32_t parity, unsigned int* err) {
    unsigned long long t0 = 0;
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}\n"
            : "=r"(ok) : "r"(bar), "r"(parity), "r"(20000u) : "memory");
        if (ok) return true;
        const unsigned long long now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) {
            atomicOr(err, kDevErrTimeout);
            return false;
        }
    }
}

// Before a role that issued copies or products leaves: wait (again with the
// limit) for the last phase of `bar`, which they complete, whether or not some
// wait gave up.  Shared memory is handed on when the CTA exits, TMEM when it is
// freed, and neither may have anything on its way to it then.
__device__ __forceinline__ void drain(uint32_t bar, int phase, unsigned int* err) { mbar_wait_sleep(bar, (uint32_t)phase & 1u, err); }

// Whole warp: 16 consecutive 32-bit columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
          "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// One product step and the commit, by the elected lane (always the same) of a
// warp that runs together: the operands stay in uniform registers (23 cycles a
// step to issue, against 52 from a single lane's branch).
__device__ __forceinline__ void umma_elect(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
                 :: "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void commit_elect(uint32_t bar) {
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n"
                 :: "r"(bar) : "memory");
}

// 4-D bf16 map of a (batch, L, heads, width) tensor, boxes of 64 steps x 64
// columns of one head, 128-byte swizzle; steps past L read as zeros.
inline cudaError_t map_steps(CUtensorMap* m, const void* base, int64_t width, int64_t heads, int64_t L, int64_t batch, int cols = 64) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)batch};
    const cuuint64_t strides[3] = {(cuuint64_t)width * 2, (cuuint64_t)(width * heads) * 2, (cuuint64_t)(width * heads * L) * 2};
    const cuuint32_t box[4] = {(cuuint32_t)cols, 1, C, 1}, estr[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// The maps that a call's kernels share.
struct CallMaps { CUtensorMap k, q, v; };                    // v: the forward's v, the backward's do
inline cudaError_t map_call(CallMaps* m, const GDRArgs& a, const void* v) {
    cudaError_t e;
    if ((e = map_steps(&m->k, a.k, a.dstate, a.ngroups, a.seqlen, a.batch)) != cudaSuccess) return e;
    if ((e = map_steps(&m->q, a.q, a.dstate, a.ngroups, a.seqlen, a.batch)) != cudaSuccess) return e;
    return map_steps(&m->v, v, a.headdim, a.nheads, a.seqlen, a.batch);
}

}  // namespace gdr

// The chains over the chunks, forward or backward (gdr_chain.cu).
cudaError_t launch_gdr_chain(const GDRArgs& a, bool backward, const gdr::CallMaps& m, cudaStream_t s);

}  // namespace mmscan
