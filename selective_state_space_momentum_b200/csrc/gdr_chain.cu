// gdr_chain.cu -- the sequential part of the gated delta rule, forward and
// backward, on sm_100a tensor cores (tcgen05 / TMEM); formulas and names as in
// gdr_fwd.cu and gdr_bwd.cu.
//
// A CTA walks the chunks of one batch row, head and tile of 64 state rows p,
// with the state (or its gradient) transposed, S^T (N x 64), in TMEM as fp32.
// k and q of a chunk are stacked into one tile of 128 rows, so that every
// product has M = 128:
//   forward, per chunk                                 epilogue between them
//     1. [k; q] S      (S in two bf16 terms)           x = beta (v - e^c S k), in two terms
//     2. [T; Pm] x     (T, x in two terms; rows 0-63)  u; tail u in two terms
//     3. S += k^T (tail u)   onto the decayed S        next chunk: S to two terms, S <- e^c_last S
//     4. [T; Pm] u     (rows 64-127)                   o = scale e^c S q + Pm u
//   backward, per chunk, in reverse
//     0. Pm^T do, 1. [k; q] dS                         x = tail (dS k) + Pm^T do
//     2. T^T x                                         r; dv = beta r; -beta e^c r
//     3. dS += [k; q]^T [-beta e^c r; scale e^c do]    next chunk: dS to bf16, dS <- e^c_last dS
// Products 1, 2, 3 of a chunk and the epilogues between them are one chain of
// dependences; 0 and 4 run beside it.
//
// Roles (10 warps): warps 0-7 the epilogues (a thread one TMEM lane and 32 of
// the 64 columns; lanes 0-63, the rows of k, carry the chain, lanes 64-127,
// those of q, finish o), warp 8 the TMA loads (no multicast) into a ring of two
// slots, warp 9 every tcgen05.mma.  Every wait is an mbarrier wait bounded by
// kWaitLimitNs; on give-up the kernel records the fact, every role leaves its
// loop, TMEM is freed and the kernel returns.
//
// Bound: the latency of the chain -- three products of at most 0.4 us and three
// passes TMEM -> registers -> shared memory a chunk -- not tensor rate or bytes.
#include <cuda.h>

#include "gdr_common.cuh"
#include "mm_tma_host.h"

namespace mmscan {

static __device__ unsigned int g_gdr_dev_err = 0;

namespace gdr {
namespace {

constexpr int PT = kGdrTile;               // state rows p of a CTA
constexpr int SLAB = 128 * 128;            // 64 columns of the stacked [k; q] tile
constexpr int NEPI = 256, NTHREADS = NEPI + 64, W_PROD = 8, W_MMA = 9;
constexpr uint32_t TM_S = 0, TM_X = 64, TM_U = 128, TM_O = 192, TM_COLS = 256;
enum { B_FULL = 0, B_EMPTY = 2, B_S = 4, B_P1 = 5, B_X = 6, B_P2 = 7, B_V = 8, B_P3 = 9, B_P4 = 10, B_OFREE = 11, B_DO = 12, NBAR = 13 };

// Shared memory: a ring of two slots (the stacked k and q, [T; Pm], T's low
// part, v or do, the decays), then the operand tiles the epilogues write.
template <int DK>
struct Smem {
    static constexpr int KQ = 0, TP = DK / 64 * SLAB, TL = TP + 16384, V = TL + 8192, F = V + 8192, SLOT = F + 1024;
    static constexpr int SH = 2 * SLOT, SL = SH + DK * 128;      // S: [n][64 p] bf16, hi and lo
    static constexpr int XH = SL + DK * 128, XL = XH + 8192;     // x, then tail u: [step][64 p], hi and lo
    static constexpr int U = XL + 8192;                          // u: [step][64 p]
    static constexpr int BAR = U + 8192, TSLOT = BAR + NBAR * 8, ABORT = TSLOT + 8;
    static constexpr int BYTES = ABORT + 8 + 1024;
    static_assert(BYTES <= 227 * 1024 && SLOT % 1024 == 0 && SH % 1024 == 0 && XH % 1024 == 0, "shared memory");
};

constexpr uint32_t ID_KM_MN = umma_idesc_bf16(128, 64, 0, 1);    // A K-major, B MN-major
constexpr uint32_t ID_MN_MN = umma_idesc_bf16(128, 64, 1, 1);

// `bytes` (a multiple of 16) of consecutive global memory into shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// 32 fp32 values to 4 (hi) or 8 (hi and lo) pieces of 16 bytes of row `row`.
__device__ __forceinline__ void put_row(unsigned char* tile, int row, int half, const uint32_t (&w)[16]) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(tile + tile_off<128>(row, 4 * half + c)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}
__device__ __forceinline__ void split_row(const uint32_t (&r)[32], uint32_t (&hi)[16], uint32_t (&lo)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) split2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]), hi[e], lo[e]);
}
__device__ __forceinline__ void round_row(const uint32_t (&r)[32], uint32_t (&hi)[16]) {
#pragma unroll
    for (int e = 0; e < 16; ++e) hi[e] = pack_bf16x2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    uint32_t a[16], b[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        a[e] = r[e];
        b[e] = r[16 + e];
    }
    tmem_st16(taddr, a);
    tmem_st16(taddr + 16, b);
}

template <int DK, bool BWD>
__global__ void __launch_bounds__(NTHREADS, 1)
gdr_chain_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                 const __grid_constant__ CUtensorMap tm_v, const GDRArgs p) {
    using L = Smem<DK>;
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (base - raw_addr);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tiles = p.headdim / PT;
    const int64_t bh = blockIdx.x / tiles;
    const int pt = (int)(blockIdx.x % tiles);
    const int64_t b = bh / p.nheads, h = bh - b * p.nheads;
    const int n = (int)p.nchunks;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::ABORT);
    auto bar = [&](int i) { return base + L::BAR + 8u * (uint32_t)i; };
    auto chunk_of = [&](int c) -> int64_t { return BWD ? n - 1 - c : c; };

    if (tid == 0) {
        for (int k = 0; k < 2; ++k) {
            mbar_init(bar(B_FULL + k), 1);
            mbar_init(bar(B_EMPTY + k), NEPI + 1);
        }
        mbar_init(bar(B_S), NEPI);
        mbar_init(bar(B_P1), 1);
        mbar_init(bar(B_X), NEPI / 2);
        mbar_init(bar(B_P2), 1);
        mbar_init(bar(B_V), NEPI / 2);
        mbar_init(bar(B_P3), 1);
        mbar_init(bar(B_P4), 1);
        mbar_init(bar(B_OFREE), NEPI / 2);
        mbar_init(bar(B_DO), NEPI / 2);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 0) tmem_alloc(base + L::TSLOT, TM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::TSLOT);
    auto wait = [&](int i, int phase) -> bool {
        if (*abort_flag) return false;
        if (!mbar_wait(bar(i), (uint32_t)phase & 1u, &g_gdr_dev_err)) {
            *abort_flag = 1;
            return false;
        }
        return true;
    };

    if (warp == W_PROD) {
        // (stall: test only, nothing staged, every other role's wait runs out)
        if (lane == 0 && !p.stall) {
            const int grp = (int)(h / (p.nheads / p.ngroups));
            for (int c = 0; c < n; ++c) {
                if (!wait(B_EMPTY + (c & 1), (c >> 1) + 1)) break;
                const uint32_t slot = base + (c & 1) * L::SLOT, fb = bar(B_FULL + (c & 1));
                const int64_t ch = chunk_of(c), rec = bh * p.nchunks + ch;
                const unsigned char* rg = static_cast<const unsigned char*>(p.rec) + rec * REC_BYTES;
                const int t0 = (int)(ch * C);
                mbar_expect_tx(fb, DK / 64 * SLAB + 2 * C * C * 2 + (BWD ? 0 : C * C * 2) + C * PT * 2 + 3 * C * 4);
#pragma unroll
                for (int s = 0; s < DK / 64; ++s) {
                    tma_load_4d(slot + L::KQ + s * SLAB, &tm_k, fb, 64 * s, grp, t0, (int)b);
                    tma_load_4d(slot + L::KQ + s * SLAB + SLAB / 2, &tm_q, fb, 64 * s, grp, t0, (int)b);
                }
                bulk_load(slot + L::TP, rg, 2 * C * C * 2, fb);
                if constexpr (!BWD) bulk_load(slot + L::TL, static_cast<const unsigned char*>(p.tlo) + rec * (C * C * 2), C * C * 2, fb);
                tma_load_4d(slot + L::V, &tm_v, fb, pt * PT, (int)h, t0, (int)b);
                bulk_load(slot + L::F, rg + REC_F, 3 * C * 4, fb);
            }
        }
    } else if (warp == W_MMA) {
        if (lane == 0) {
            // D (+)= A . B over ks steps of 16: A from `a` (K-major: 32 bytes a step
            // within a slab of 64; MN-major: 16 rows a step), B from `bt` (MN-major)
            auto prod_km = [&](uint32_t d, uint32_t a, uint32_t bt, int ks, bool acc) {
#pragma unroll
                for (int s = 0; s < ks; ++s)
                    umma_ss(tmem + d, umma_desc_sw128(a + (s >> 2) * SLAB + (s & 3) * 32, 16, 1024),
                            umma_desc_sw128(bt + s * 2048, 8192, 1024), ID_KM_MN, acc || s > 0);
            };
            auto prod_mn = [&](uint32_t d, uint32_t a, uint32_t lbo, uint32_t bt, int ks, bool acc) {
#pragma unroll
                for (int s = 0; s < ks; ++s)
                    umma_ss(tmem + d, umma_desc_sw128(a + s * 2048, lbo, 1024), umma_desc_sw128(bt + s * 2048, 8192, 1024),
                            ID_MN_MN, acc || s > 0);
            };
            // the second 64 rows of an M of 128 that has only 64: any tile will do,
            // its results go to lanes nobody reads
            const uint32_t lbo_k = DK == 128 ? SLAB : 8192;
            bool live = true;
            for (int c = 0; c < n && live; ++c) {
                const uint32_t slot = base + (c & 1) * L::SLOT;
                const uint32_t kq = slot + L::KQ, tp = slot + L::TP, tl = slot + L::TL;
                if (!(live = wait(B_FULL + (c & 1), c >> 1))) break;
                if constexpr (BWD) {                       // Pm^T do, beside the chain
                    tc_fence_after();
                    prod_mn(TM_O, tp + 8192, 8192, slot + L::V, C / 16, false);
                }
                if (!(live = wait(B_S, c))) break;
                tc_fence_after();
                prod_km(TM_X, kq, base + L::SH, DK / 16, false);
                if constexpr (!BWD) prod_km(TM_X, kq, base + L::SL, DK / 16, true);
                umma_commit(bar(B_P1));
                if (!(live = wait(B_X, c))) break;
                tc_fence_after();
                if constexpr (BWD) {
                    prod_mn(TM_U, tp, 8192, base + L::XH, C / 16, false);
                } else {
                    prod_km(TM_U, tp, base + L::XH, C / 16, false);
                    prod_km(TM_U, tl, base + L::XH, C / 16, true);
                    prod_km(TM_U, tp, base + L::XL, C / 16, true);
                }
                umma_commit(bar(B_P2));
                if (!(live = wait(B_V, c))) break;
                if constexpr (BWD) {
                    if (!(live = wait(B_DO, c))) break;
                }
                tc_fence_after();
                if constexpr (BWD) {
                    prod_mn(TM_S, kq, lbo_k, base + L::XH, 2 * C / 16, true);     // [k; q]^T . [-beta e^c r; scale e^c do]
                    umma_commit(bar(B_P3));
                } else {
                    prod_mn(TM_S, kq, lbo_k, base + L::XH, C / 16, true);
                    prod_mn(TM_S, kq, lbo_k, base + L::XL, C / 16, true);
                    umma_commit(bar(B_P3));
                    if (!(live = wait(B_OFREE, c + 1))) break;
                    tc_fence_after();
                    prod_km(TM_O, tp, base + L::U, C / 16, false);
                    umma_commit(bar(B_P4));
                }
                umma_commit(bar(B_EMPTY + (c & 1)));
            }
            // the last commit must land before the CTA may exit
            if (live && !*abort_flag) wait(B_EMPTY + ((n - 1) & 1), (n - 1) >> 1);
        }
    } else {
        const int q = warp & 3, half = warp >> 2;
        const int t = 32 * q + lane;                       // TMEM lane: state n, or row of [k; q]
        const bool krows = q < 2;                          // lanes 0-63
        const int i = t & 63;                              // step of the chunk
        const uint32_t lb = tmem + ((uint32_t)(q * 32) << 16) + 32 * half;
        const bool states = t < DK;                        // (whole warps)
        auto wwait = [&](int bi, int phase) { return __all_sync(0xffffffffu, wait(bi, phase)); };
        // (batch, H, P, N): state n = t, rows p of this thread
        const int64_t sbase = (bh * p.headdim + pt * PT + 32 * half) * DK + t;
        const float* s0 = BWD ? p.dhT : p.h0;
        uint32_t r[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) r[e] = s0 && states ? __float_as_uint(s0[sbase + (int64_t)e * DK]) : 0u;
        tmem_st32(lb + TM_S, r);
        tmem_wait_st();

        float qs[32];                                      // lanes 64-127, forward: scale e^c S q of the chunk before
        auto put_o = [&](int64_t ch) {                     // o = qs + Pm u, row i of chunk ch
            tmem_ld32(lb + TM_O, r);
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive(bar(B_OFREE));
            if (ch * C + i >= p.seqlen) return;
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
                w[e] = pack_bf16x2(qs[2 * e] + __uint_as_float(r[2 * e]), qs[2 * e + 1] + __uint_as_float(r[2 * e + 1]));
            uint4* o = reinterpret_cast<uint4*>(static_cast<bf16*>(p.o) + ((b * p.seqlen + ch * C + i) * p.nheads + h) * p.headdim + pt * PT + 32 * half);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
        };

        bool ok = true;
        for (int c = 0; c < n; ++c) {
            const unsigned char* slot = smem + (c & 1) * L::SLOT;
            const float* f = reinterpret_cast<const float*>(slot + L::F);
            const int64_t ch = chunk_of(c), rec = bh * p.nchunks + ch;
            uint32_t hi[16], lo[16];
            if (!(ok = wwait(B_FULL + (c & 1), c >> 1))) break;
            if (c > 0 && !(ok = wwait(B_P3, c - 1))) break;
            // S as operand tiles; S <- e^(c_last) S in place
            tc_fence_after();
            const float last = f[C - 1];
            tmem_ld32(lb + TM_S, r);
            tmem_wait_ld();
            if (states) {
                if constexpr (BWD) {
                    round_row(r, hi);
                } else {
                    split_row(r, hi, lo);
                    put_row(smem + L::SL, t, half, lo);
                }
                put_row(smem + L::SH, t, half, hi);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(last * __uint_as_float(r[e]));
            tmem_st32(lb + TM_S, r);
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(bar(B_S));
            // the state at the chunk's start (its end, backward), [tile][n][64 p] bf16, as the tile's image
            void* keep = BWD ? p.dstates : p.states;
            if (keep && states) put_row(static_cast<unsigned char*>(keep) + (rec * tiles + pt) * (DK * PT * 2), t, half, hi);

            if (!krows) {
                if constexpr (BWD) {
                    // scale e^c do, rows 64-127 of the stacked operand of product 3
                    // (whose previous contents product 3 of the last chunk has read)
                    const float e = p.scale * f[i];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint4 d = *reinterpret_cast<const uint4*>(slot + L::V + tile_off<128>(i, 4 * half + x));
                        *reinterpret_cast<uint4*>(smem + L::XL + tile_off<128>(i, 4 * half + x)) =
                            make_uint4(pack_bf16x2(bf16_lo(d.x) * e, bf16_hi(d.x) * e), pack_bf16x2(bf16_lo(d.y) * e, bf16_hi(d.y) * e),
                                       pack_bf16x2(bf16_lo(d.z) * e, bf16_hi(d.z) * e), pack_bf16x2(bf16_lo(d.w) * e, bf16_hi(d.w) * e));
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(bar(B_DO));
                } else {
                    if (c > 0) {
                        if (!(ok = wwait(B_P4, c - 1))) break;
                        tc_fence_after();
                        put_o(chunk_of(c - 1));
                    }
                    const float e = p.scale * f[i];
                    if (!(ok = wwait(B_P1, c))) break;
                    tc_fence_after();
                    tmem_ld32(lb + TM_X, r);
                    tmem_wait_ld();
                    tc_fence_before();
#pragma unroll
                    for (int x = 0; x < 32; ++x) qs[x] = e * __uint_as_float(r[x]);
                }
                mbar_arrive(bar(B_EMPTY + (c & 1)));
                continue;
            }
            const float eg = f[i], tail = f[C + i], beta = f[2 * C + i];
            if constexpr (!BWD) {
                uint4 vv[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) vv[x] = *reinterpret_cast<const uint4*>(slot + L::V + tile_off<128>(i, 4 * half + x));
                if (!(ok = wwait(B_P1, c))) break;
                tc_fence_after();
                tmem_ld32(lb + TM_X, r);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const uint32_t v4[4] = {vv[x].x, vv[x].y, vv[x].z, vv[x].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int k = 8 * x + 2 * e;
                        r[k] = __float_as_uint(beta * fmaf(-eg, __uint_as_float(r[k]), bf16_lo(v4[e])));
                        r[k + 1] = __float_as_uint(beta * fmaf(-eg, __uint_as_float(r[k + 1]), bf16_hi(v4[e])));
                    }
                }
                split_row(r, hi, lo);
                put_row(smem + L::XH, i, half, hi);
                put_row(smem + L::XL, i, half, lo);
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(bar(B_X));
                mbar_arrive(bar(B_EMPTY + (c & 1)));
                if (!(ok = wwait(B_P2, c))) break;
                tc_fence_after();
                tmem_ld32(lb + TM_U, r);
                tmem_wait_ld();
                uint32_t u[16];
                round_row(r, u);
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(tail * __uint_as_float(r[e]));
                split_row(r, hi, lo);
                put_row(smem + L::XH, i, half, hi);          // product 2 has read x
                put_row(smem + L::XL, i, half, lo);
                put_row(smem + L::U, i, half, u);
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(bar(B_V));
                if (p.u) put_row(static_cast<unsigned char*>(p.u) + (rec * tiles + pt) * (C * PT * 2), i, half, u);
            } else {
                if (!(ok = wwait(B_P1, c))) break;           // product 0 came before it
                tc_fence_after();
                uint32_t d[32];
                tmem_ld32(lb + TM_X, r);
                tmem_ld32(lb + TM_O, d);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(fmaf(tail, __uint_as_float(r[e]), __uint_as_float(d[e])));
                round_row(r, hi);
                put_row(smem + L::XH, i, half, hi);
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(bar(B_X));
                mbar_arrive(bar(B_EMPTY + (c & 1)));
                if (!(ok = wwait(B_P2, c))) break;
                tc_fence_after();
                tmem_ld32(lb + TM_U, r);
                tmem_wait_ld();
                const float neg = -beta * eg;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    hi[e] = pack_bf16x2(neg * __uint_as_float(r[2 * e]), neg * __uint_as_float(r[2 * e + 1]));
                put_row(smem + L::XH, i, half, hi);          // product 2 has read x
                fence_proxy_async_smem();
                tc_fence_before();
                mbar_arrive(bar(B_V));
                round_row(r, lo);                            // r, and dv = beta r
                put_row(static_cast<unsigned char*>(p.dr) + (rec * tiles + pt) * (C * PT * 2), i, half, lo);
                if (ch * C + i < p.seqlen) {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        hi[e] = pack_bf16x2(beta * __uint_as_float(r[2 * e]), beta * __uint_as_float(r[2 * e + 1]));
                    uint4* o = reinterpret_cast<uint4*>(static_cast<bf16*>(p.dv) + ((b * p.seqlen + ch * C + i) * p.nheads + h) * p.headdim + pt * PT + 32 * half);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = make_uint4(hi[4 * e], hi[4 * e + 1], hi[4 * e + 2], hi[4 * e + 3]);
                }
            }
        }
        if constexpr (!BWD) {
            if (ok && !krows && (ok = wwait(B_P4, n - 1))) {
                tc_fence_after();
                put_o(chunk_of(n - 1));
            }
        }
        float* sT = BWD ? p.dh0 : p.hT;
        if (ok && sT && states && wwait(B_P3, n - 1)) {
            tc_fence_after();
            tmem_ld32(lb + TM_S, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) sT[sbase + (int64_t)e * DK] = __uint_as_float(r[e]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, TM_COLS);
    }
}

// 4-D bf16 map of a (batch, L, heads, width) tensor, boxes of 64 steps x 64
// columns of one head, 128-byte swizzle; steps past L read as zeros.
cudaError_t map_steps(CUtensorMap* m, const void* base, int64_t width, int64_t heads, int64_t L, int64_t batch) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)batch};
    const cuuint64_t strides[3] = {(cuuint64_t)width * 2, (cuuint64_t)(width * heads) * 2, (cuuint64_t)(width * heads * L) * 2};
    const cuuint32_t box[4] = {64, 1, C, 1}, estr[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int DK, bool BWD>
cudaError_t launch(const GDRArgs& a, cudaStream_t s) {
    CUtensorMap mk, mq, mv;
    cudaError_t e;
    if ((e = map_steps(&mk, a.k, DK, a.ngroups, a.seqlen, a.batch)) != cudaSuccess) return e;
    if ((e = map_steps(&mq, a.q, DK, a.ngroups, a.seqlen, a.batch)) != cudaSuccess) return e;
    if ((e = map_steps(&mv, BWD ? a.dout : a.v, a.headdim, a.nheads, a.seqlen, a.batch)) != cudaSuccess) return e;
    constexpr int bytes = Smem<DK>::BYTES;
    if ((e = cudaFuncSetAttribute(gdr_chain_kernel<DK, BWD>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
    gdr_chain_kernel<DK, BWD><<<(unsigned)(a.batch * a.nheads * (a.headdim / PT)), NTHREADS, bytes, s>>>(mk, mq, mv, a);
    return cudaGetLastError();
}

unsigned int read_and_clear_device_error() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_gdr_dev_err, sizeof(v)) != cudaSuccess) return 0;
    if (v) cudaMemcpyToSymbol(g_gdr_dev_err, &z, sizeof(z));
    return v;
}

[[maybe_unused]] const bool g_registered = (register_error_reader(read_and_clear_device_error), true);

}  // namespace
}  // namespace gdr

cudaError_t launch_gdr_chain(const GDRArgs& a, bool backward, cudaStream_t s) {
    if (backward) return a.dstate == 64 ? gdr::launch<64, true>(a, s) : gdr::launch<128, true>(a, s);
    return a.dstate == 64 ? gdr::launch<64, false>(a, s) : gdr::launch<128, false>(a, s);
}

}  // namespace mmscan
