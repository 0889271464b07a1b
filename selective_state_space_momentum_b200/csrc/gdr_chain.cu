// gdr_chain.cu -- the sequential part of the gated delta rule, forward and
// backward, on sm_100a tensor cores (tcgen05 / TMEM); formulas and names as in
// gdr_fwd.cu and gdr_bwd.cu.
//
// A CTA walks the chunks of one batch row, head and tile of 64 (or 32) state
// rows p, with the state (or its gradient) transposed, S^T (N x 64), in TMEM as
// fp32.
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
// dependences; 0 and 4 run beside it (4 during the next chunk's first epilogue).
// Two terms of an operand B are two 64-column groups of one product with
// N = 128, whose halves the epilogue adds: a step of 16 costs some 60 cycles
// with 64 columns and 85 with 128.  With 32 rows p the two terms lie side by
// side in one group of 64.
//
// Roles (11 warps): warps 0-7 the epilogues (a thread one TMEM lane and half
// of the columns; lanes 0-63, the rows of k, carry the chain, lanes 64-127,
// those of q, finish o), then one warp for the TMA loads (no multicast) into a
// ring of two slots, one for every tcgen05.mma, and one for the stores, as bulk
// copies of tiles: a thread's own columns of a row would be 32 lines to a store
// instruction, and the queue behind it is the one the chain's shared-memory
// accesses wait in.  Every wait is an mbarrier wait bounded by kWaitLimitNs; on
// give-up the kernel records the fact and every role leaves its loop.  Before
// the CTA frees TMEM and returns, given up or not, the loads' warp has waited
// for the loads it issued, the products' warp for its products (each with the
// same limit again) and the stores' warp for its stores.
//
// Bound: the latency of the chain -- three products and three passes TMEM ->
// registers -> shared memory a chunk -- not tensor rate or bytes.  Measured, a
// chunk of 64 steps (128 states, 64 rows, 128 CTAs): 2.4 us forward, 2.0 us
// backward.  What mattered: one arrival a warp (3.2 us with one a thread),
// waits that sleep in hardware (2.8 us polling), products issued by a warp
// that runs together, its number known to be uniform (2.6 us from one lane).
#include <cuda.h>

#include "gdr_common.cuh"

namespace mmscan {

static __device__ unsigned int g_gdr_dev_err = 0;

namespace gdr {
namespace {

constexpr int SLAB = 128 * 128;            // 64 columns of the stacked [k; q] tile
constexpr int EPI_WARPS = 8, NTHREADS = 32 * EPI_WARPS + 96, W_PROD = EPI_WARPS, W_MMA = W_PROD + 1, W_STORE = W_PROD + 2;
constexpr uint32_t TM_S = 0, TM_X = 128, TM_U = 256, TM_O = 384, TM_COLS = 512;   // S, X, U: two halves of PT, forward
enum { B_FULL = 0, B_EMPTY = 2, B_S = 4, B_P1 = 5, B_X = 6, B_P2 = 7, B_V = 8, B_P3 = 9, B_P4 = 10, B_OFREE = 11, B_DO = 12, B_OUT = 13, B_SST = 14, B_OST = 15, B_UST = 16, B_END = 17, NBAR = 18 };

// Shared memory: a ring of two slots (the stacked k and q, [T; Pm], T's low
// part, v or do, the decays), then the operand tiles the epilogues write.
template <int DK>
struct Smem {
    static constexpr int KQ = 0, TP = DK / 64 * SLAB, TL = TP + 16384, V = TL + 8192, F = V + 8192, SLOT = F + 1024;
    static constexpr int SH = 2 * SLOT, SL = SH + DK * 128;      // S: [n][64 p] bf16, hi and lo
    static constexpr int XH = SL + DK * 128, XL = XH + 8192;     // x, then tail u: [step][64 p], hi and lo
    static constexpr int U = XL + 8192;                          // u (backward: r): [step][64 p]
    static constexpr int OUT = U + 8192;                         // o (backward: dv): [step][64 p]
    static constexpr int BAR = OUT + 8192, TSLOT = BAR + NBAR * 8, ABORT = TSLOT + 8;
    static constexpr int BYTES = ABORT + 8 + 1024;
    static_assert(BYTES <= 227 * 1024 && SLOT % 1024 == 0 && SH % 1024 == 0 && XH % 1024 == 0, "shared memory");
};

// This thread's CW columns from `taddr` on; the sum of the two halves of a
// product (2 CW columns apart).
template <int CW>
__device__ __forceinline__ void tmem_store(uint32_t taddr, const uint32_t (&a)[CW]) {
#pragma unroll
    for (int k = 0; k < CW; k += 16) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = a[k + e];
        tmem_st16(taddr + k, w);
    }
}
template <int CW>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&a)[CW]) {
    if constexpr (CW == 32) tmem_ld32(taddr, a);
    else tmem_ld16(taddr, a);
}
template <int NPAIR>
__device__ __forceinline__ void tmem_get(uint32_t taddr, float2 (&x)[NPAIR]) {
    uint32_t a[2 * NPAIR];
    tmem_load(taddr, a);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < NPAIR; ++e) x[e] = f2(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1]));
}
template <int NPAIR>
__device__ __forceinline__ void tmem_get_sum(uint32_t taddr, float2 (&x)[NPAIR]) {
    uint32_t a[2 * NPAIR], b[2 * NPAIR];
    tmem_load(taddr, a);
    tmem_load(taddr + 4 * NPAIR, b);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < NPAIR; ++e)
        x[e] = add2(f2(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1])), f2(__uint_as_float(b[2 * e]), __uint_as_float(b[2 * e + 1])));
}
// A thread's values to row `row` of a tile, from piece `at` of 16 bytes on.
template <int NPAIR>
__device__ __forceinline__ void put_row(unsigned char* tile, int row, int at, const uint32_t (&w)[NPAIR]) {
#pragma unroll
    for (int c = 0; c < NPAIR / 4; ++c)
        *reinterpret_cast<uint4*>(tile + tile_off<128>(row, at + c)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
}
template <int NPAIR>
__device__ __forceinline__ void split_row(const float2 (&x)[NPAIR], uint32_t (&hi)[NPAIR], uint32_t (&lo)[NPAIR]) {
#pragma unroll
    for (int e = 0; e < NPAIR; ++e) {
        hi[e] = pack_bf16x2(x[e].x, x[e].y);
        const float2 d = add2(x[e], f2(-bf16_lo(hi[e]), -bf16_hi(hi[e])));
        lo[e] = pack_bf16x2(d.x, d.y);
    }
}
template <int NPAIR>
__device__ __forceinline__ void round_row(const float2 (&x)[NPAIR], float scale, uint32_t (&hi)[NPAIR]) {
#pragma unroll
    for (int e = 0; e < NPAIR; ++e) {
        const float2 y = mul2(f2(scale, scale), x[e]);
        hi[e] = pack_bf16x2(y.x, y.y);
    }
}
template <int NPAIR>
__device__ __forceinline__ void round_row(const float2 (&x)[NPAIR], uint32_t (&hi)[NPAIR]) {
#pragma unroll
    for (int e = 0; e < NPAIR; ++e) hi[e] = pack_bf16x2(x[e].x, x[e].y);
}

template <int DK, bool BWD, int PT>
__global__ void __launch_bounds__(NTHREADS, 1)
gdr_chain_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o, const GDRArgs p) {
    using L = Smem<DK>;
    constexpr int CW = PT / 2, NPAIR = CW / 2;           // columns a thread
    constexpr int N2 = 2 * PT;                           // columns of a product with two terms
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (base - raw_addr);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
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
            mbar_init(bar(B_EMPTY + k), EPI_WARPS + 1);
        }
        mbar_init(bar(B_S), EPI_WARPS);
        mbar_init(bar(B_P1), 1);
        mbar_init(bar(B_X), EPI_WARPS / 2);
        mbar_init(bar(B_P2), 1);
        mbar_init(bar(B_V), EPI_WARPS / 2);
        mbar_init(bar(B_P3), 1);
        mbar_init(bar(B_P4), 1);
        mbar_init(bar(B_OFREE), EPI_WARPS / 2);
        mbar_init(bar(B_DO), EPI_WARPS / 2);
        mbar_init(bar(B_OUT), EPI_WARPS / 2);
        mbar_init(bar(B_SST), 1);
        mbar_init(bar(B_OST), 1);
        mbar_init(bar(B_UST), 1);
        mbar_init(bar(B_END), 1);
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
        if (!mbar_wait_sleep(bar(i), (uint32_t)phase & 1u, &g_gdr_dev_err)) {
            *abort_flag = 1;
            return false;
        }
        return true;
    };

    if (warp == W_PROD) {
        if (lane == 0) {
            const int grp = (int)(h / (p.nheads / p.ngroups));
            // (stall: test only, only its first chunks staged, every other role's wait runs out)
            const int staged = p.stall && p.stall - 1 < n ? p.stall - 1 : n;
            int c = 0;
            for (; c < staged; ++c) {
                if (!wait(B_EMPTY + (c & 1), (c >> 1) + 1)) break;
                const uint32_t slot = base + (c & 1) * L::SLOT, fb = bar(B_FULL + (c & 1));
                const int64_t ch = chunk_of(c), rec = bh * p.nchunks + ch;
                const unsigned char* rg = static_cast<const unsigned char*>(p.rec) + rec * REC_BYTES;
                const int t0 = (int)(ch * C);
                mbar_expect_tx(fb, DK / 64 * SLAB + 2 * C * C * 2 + (BWD ? 0 : C * C * 2) + C * 64 * 2 + 3 * C * 4);
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
            for (int d = c < 2 ? 0 : c - 2; d < c; ++d) drain(bar(B_FULL + (d & 1)), d >> 1, &g_gdr_dev_err);
        }
    } else if (warp == W_MMA) {
        {
            auto mwait = [&](int bi, int phase) { return __all_sync(0xffffffffu, wait(bi, phase)); };
            // D (+)= A . B over ks steps of 16: A from `a` (K-major: 32 bytes a step
            // within a slab of 64; MN-major: 16 rows a step), B from `bt` (MN-major,
            // 64-column groups `ldb` apart), N = 64 or 128; with 32 rows p, both terms are
            // one group, and a product that needs the first alone has zeros for the second
            auto prod_km = [&](uint32_t d, uint32_t a, uint32_t bt, uint32_t ldb, int N, int ks, bool acc) {
                const uint32_t id = umma_idesc_bf16(128, N, 0, 1);
                const uint64_t da = umma_desc_sw128(a, 16, 1024), db = umma_desc_sw128(bt, ldb, 1024);
#pragma unroll
                for (int s = 0; s < ks; ++s)
                    umma_elect(tmem + d, da + (((s >> 2) * SLAB + (s & 3) * 32) >> 4), db + ((s * 2048) >> 4), id, acc || s > 0);
            };
            auto prod_mn = [&](uint32_t d, uint32_t a, uint32_t lbo, uint32_t bt, int N, int ks, bool acc) {
                const uint32_t id = umma_idesc_bf16(128, N, 1, 1);
                const uint64_t da = umma_desc_sw128(a, lbo, 1024), db = umma_desc_sw128(bt, 8192, 1024);
#pragma unroll
                for (int s = 0; s < ks; ++s)
                    umma_elect(tmem + d, da + ((s * 2048) >> 4), db + ((s * 2048) >> 4), id, acc || s > 0);
            };
            // the second 64 rows of an M of 128 that has only 64: any tile will do,
            // its results go to lanes nobody reads
            const uint32_t lbo_k = DK == 128 ? SLAB : 8192;
            bool live = true;
            for (int c = 0; c < n && live; ++c) {
                const uint32_t slot = base + (c & 1) * L::SLOT;
                const uint32_t kq = slot + L::KQ, tp = slot + L::TP, tl = slot + L::TL;
                if (!(live = mwait(B_FULL + (c & 1), c >> 1))) break;
                if constexpr (BWD) {                       // Pm^T do, beside the chain
                    tc_fence_after();
                    prod_mn(TM_O, tp + 8192, 8192, slot + L::V, 64, C / 16, false);
                }
                if (!(live = mwait(B_S, c))) break;
                tc_fence_after();
                prod_km(TM_X, kq, base + L::SH, DK * 128, BWD ? 64 : N2, DK / 16, false);
                commit_elect(bar(B_P1));
                if (!(live = mwait(B_X, c))) break;
                tc_fence_after();
                if constexpr (BWD) {
                    prod_mn(TM_U, tp, 8192, base + L::XH, 64, C / 16, false);
                } else {
                    prod_km(TM_U, tp, base + L::XH, 8192, N2, C / 16, false);
                    prod_km(TM_U, tl, base + (PT == 64 ? L::XH : L::XL), 8192, 64, C / 16, true);
                }
                commit_elect(bar(B_P2));
                if (!(live = mwait(B_V, c))) break;
                if constexpr (BWD) {
                    if (!(live = mwait(B_DO, c))) break;
                }
                tc_fence_after();
                // backward: [k; q]^T . [-beta e^c r; scale e^c do]
                prod_mn(TM_S, kq, lbo_k, base + L::XH, BWD ? 64 : N2, BWD ? 2 * C / 16 : C / 16, true);
                commit_elect(bar(B_P3));
                if constexpr (!BWD) {                      // [T; Pm] u, beside the next chunk's first epilogue
                    if (!(live = mwait(B_OFREE, c + 1))) break;
                    tc_fence_after();
                    prod_km(TM_O, tp, base + L::U, 8192, 64, C / 16, false);
                    commit_elect(bar(B_P4));
                }
                commit_elect(bar(B_EMPTY + (c & 1)));
            }
            commit_elect(bar(B_END));                      // behind every product and commit before it
            drain(bar(B_END), 0, &g_gdr_dev_err);
        }
    } else if (warp == W_STORE) {
        // Per chunk: the state's tile, then o of the chunk before and u (backward:
        // dv and r); after each, that its tile may be written again (a store
        // queues behind the loads, so nobody waits for more than it needs).
        if (lane == 0) {
            unsigned char* states = static_cast<unsigned char*>(BWD ? p.dstates : p.states);
            unsigned char* rows = static_cast<unsigned char*>(BWD ? p.dr : p.u);
            const int64_t first = bh * p.nchunks;
            auto store_out = [&](int c) {
                tma_store_4d(&tm_o, base + L::OUT, pt * PT, (int)h, (int)(chunk_of(c) * C), (int)b);
                bulk_commit_group();
                bulk_wait_read_all();
                mbar_arrive(bar(B_OST));
            };
            bool live = true;
            for (int c = 0; c < n; ++c) {
                const int64_t tile = (first + chunk_of(c)) * tiles + pt;
                if (states) {
                    if (!(live = wait(B_S, c))) break;
                    bulk_store(states + tile * (DK * PT * 2), base + L::SH, DK * PT * 2);
                    bulk_commit_group();
                    bulk_wait_read_all();
                    mbar_arrive(bar(B_SST));
                }
                if (!BWD && c > 0) {
                    if (!(live = wait(B_OUT, c - 1))) break;
                    store_out(c - 1);
                }
                if (rows) {
                    if (!(live = wait(BWD ? B_OUT : B_V, c))) break;
                    bulk_store(rows + tile * (C * PT * 2), base + L::U, C * PT * 2);
                    bulk_commit_group();
                    bulk_wait_read_all();
                    mbar_arrive(bar(B_UST));
                }
                if (BWD) store_out(c);
            }
            if (!BWD && live && wait(B_OUT, n - 1)) store_out(n - 1);
            bulk_wait_all();                               // complete before the CTA exits
        }
    } else {
        const int q = warp & 3, part = warp >> 2;          // TMEM lanes 32 q .., columns CW part ..
        const int t = 32 * q + lane;                       // TMEM lane: state n, or row of [k; q]
        const bool krows = q < 2;                          // lanes 0-63
        const int i = t & 63;                              // step of the chunk
        const int at = CW / 8 * part;                      // its first piece of 16 bytes of a tile's row
        const uint32_t lb = tmem + ((uint32_t)(q * 32) << 16) + CW * part;
        const bool states = t < DK;                        // (whole warps)
        auto wwait = [&](int bi, int phase) { return __all_sync(0xffffffffu, wait(bi, phase)); };
        // One arrival a warp: arrivals on one mbarrier are taken one by one.
        auto arrive = [&](int bi) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bi));
        };
        // (batch, H, P, N): state n = t, rows p of this thread
        const int64_t sbase = (bh * p.headdim + pt * PT + CW * part) * DK + t;
        const float* s0 = BWD ? p.dhT : p.h0;
        float2 x[NPAIR];
        uint32_t hi[NPAIR], lo[NPAIR], y[CW];
#pragma unroll
        for (int e = 0; e < CW; ++e) y[e] = s0 && states ? __float_as_uint(s0[sbase + (int64_t)e * DK]) : 0u;
        tmem_store(lb + TM_S, y);
        uint32_t zeros[CW];
#pragma unroll
        for (int e = 0; e < CW; ++e) zeros[e] = 0u;
        if constexpr (!BWD) tmem_store(lb + TM_S + PT, zeros);
        if constexpr (PT == 32) {
            const uint32_t none[NPAIR] = {};
            if (krows) put_row(smem + L::XL, i, at + 4, none);
        }
        tmem_wait_st();

        float2 qs[NPAIR];                                      // lanes 64-127, forward: scale e^c S q of the chunk before
        auto put_o = [&] {                                 // o = qs + Pm u, row i
            tmem_get(lb + TM_O, x);
            tc_fence_before();
            arrive(B_OFREE);
#pragma unroll
            for (int e = 0; e < NPAIR; ++e) x[e] = add2(x[e], qs[e]);
            round_row(x, hi);
            if constexpr (PT == 64) {
                put_row(smem + L::OUT, i, at, hi);
            } else {                                       // rows of 64 bytes, pieces permuted over pairs of rows
#pragma unroll
                for (int c = 0; c < CW / 8; ++c)
                    *reinterpret_cast<uint4*>(smem + L::OUT + i * 64 + (((at + c) ^ ((i >> 1) & 3)) << 4)) =
                        make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
            }
            fence_proxy_async_smem();
            arrive(B_OUT);
        };

        const bool keeps = BWD || p.states;                // the state's and the rows' tiles are stored
        bool ok = true;
        for (int c = 0; c < n; ++c) {
            const unsigned char* slot = smem + (c & 1) * L::SLOT;
            const float* f = reinterpret_cast<const float*>(slot + L::F);
            if (!(ok = wwait(B_FULL + (c & 1), c >> 1))) break;
            const float last = f[C - 1], eg = f[i], tail = f[C + i], beta = f[2 * C + i];
            if (c > 0 && keeps && !(ok = wwait(B_SST, c - 1))) break;
            if (c > 0 && !(ok = wwait(B_P3, c - 1))) break;
            // S <- e^(c_last) S in place, and S as operand tiles
            tc_fence_after();
            if constexpr (BWD) tmem_get(lb + TM_S, x);
            else tmem_get_sum(lb + TM_S, x);
#pragma unroll
            for (int e = 0; e < NPAIR; ++e) {
                const float2 d = mul2(f2(last, last), x[e]);
                y[2 * e] = __float_as_uint(d.x);
                y[2 * e + 1] = __float_as_uint(d.y);
            }
            tmem_store(lb + TM_S, y);
            if constexpr (!BWD) tmem_store(lb + TM_S + PT, zeros);
            if (states) {
                if constexpr (BWD) {
                    round_row(x, hi);
                } else {
                    split_row(x, hi, lo);
                    put_row(smem + (PT == 64 ? L::SL : L::SH), t, PT == 64 ? at : at + 4, lo);
                }
                put_row(smem + L::SH, t, at, hi);
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            arrive(B_S);
            if (!krows) {
                if constexpr (BWD) {
                    // scale e^c do, rows 64-127 of the stacked operand of product 3
                    // (whose previous contents product 3 of the last chunk has read)
                    const float e = p.scale * eg;
#pragma unroll
                    for (int k = 0; k < CW / 8; ++k) {
                        const uint4 d = *reinterpret_cast<const uint4*>(slot + L::V + tile_off<128>(i, at + k));
                        *reinterpret_cast<uint4*>(smem + L::XL + tile_off<128>(i, at + k)) =
                            make_uint4(pack_bf16x2(bf16_lo(d.x) * e, bf16_hi(d.x) * e), pack_bf16x2(bf16_lo(d.y) * e, bf16_hi(d.y) * e),
                                       pack_bf16x2(bf16_lo(d.z) * e, bf16_hi(d.z) * e), pack_bf16x2(bf16_lo(d.w) * e, bf16_hi(d.w) * e));
                    }
                    fence_proxy_async_smem();
                    arrive(B_DO);
                    arrive(B_EMPTY + (c & 1));
                } else {
                    arrive(B_EMPTY + (c & 1));
                    if (c > 0) {
                        if (!(ok = wwait(B_P4, c - 1) && (c < 2 || wwait(B_OST, c - 2)))) break;
                        tc_fence_after();
                        put_o();
                    }
                    if (!(ok = wwait(B_P1, c))) break;
                    tc_fence_after();
                    tmem_get_sum(lb + TM_X, qs);
                    tc_fence_before();
                    const float e = p.scale * eg;
#pragma unroll
                    for (int k = 0; k < NPAIR; ++k) qs[k] = mul2(f2(e, e), qs[k]);
                }
                continue;
            }
            if constexpr (!BWD) {
                float2 bv[NPAIR];                                // beta v, before the product is there
#pragma unroll
                for (int k = 0; k < CW / 8; ++k) {
                    const uint4 d = *reinterpret_cast<const uint4*>(slot + L::V + tile_off<128>(i, at + k));
                    const uint32_t w4[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) bv[4 * k + e] = mul2(f2(beta, beta), f2(bf16_lo(w4[e]), bf16_hi(w4[e])));
                }
                const float nb = -beta * eg;
                if (!(ok = wwait(B_P1, c))) break;
                tc_fence_after();
                tmem_get_sum(lb + TM_X, x);
#pragma unroll
                for (int e = 0; e < NPAIR; ++e) x[e] = fma2(f2(nb, nb), x[e], bv[e]);
                split_row(x, hi, lo);
                put_row(smem + L::XH, i, at, hi);
                put_row(smem + (PT == 64 ? L::XL : L::XH), i, PT == 64 ? at : at + 4, lo);
                if constexpr (PT == 32) put_row(smem + L::XL, i, at, hi);   // beside zeros
                fence_proxy_async_smem();
                tc_fence_before();
                arrive(B_X);
                arrive(B_EMPTY + (c & 1));
                if (keeps && c > 0 && !(ok = wwait(B_UST, c - 1))) break;
                if (!(ok = wwait(B_P2, c))) break;
                tc_fence_after();
                tmem_get_sum(lb + TM_U, x);
                uint32_t u[NPAIR];
                round_row(x, u);
#pragma unroll
                for (int e = 0; e < NPAIR; ++e) x[e] = mul2(f2(tail, tail), x[e]);
                split_row(x, hi, lo);
                put_row(smem + L::XH, i, at, hi);          // product 2 has read x
                put_row(smem + (PT == 64 ? L::XL : L::XH), i, PT == 64 ? at : at + 4, lo);
                put_row(smem + L::U, i, at, u);
                fence_proxy_async_smem();
                tc_fence_before();
                arrive(B_V);
            } else {
                if (!(ok = wwait(B_P1, c))) break;           // product 0 came before it
                tc_fence_after();
                uint32_t a[CW], d[CW];
                tmem_ld32(lb + TM_X, a);
                tmem_ld32(lb + TM_O, d);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < NPAIR; ++e)
                    x[e] = fma2(f2(tail, tail), f2(__uint_as_float(a[2 * e]), __uint_as_float(a[2 * e + 1])),
                                f2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])));
                round_row(x, hi);
                put_row(smem + L::XH, i, at, hi);
                fence_proxy_async_smem();
                tc_fence_before();
                arrive(B_X);
                arrive(B_EMPTY + (c & 1));
                if (c > 0 && !(ok = wwait(B_UST, c - 1) && wwait(B_OST, c - 1))) break;
                if (!(ok = wwait(B_P2, c))) break;
                tc_fence_after();
                tmem_get(lb + TM_U, x);
                round_row(x, -beta * eg, hi);
                put_row(smem + L::XH, i, at, hi);          // product 2 has read x
                fence_proxy_async_smem();
                tc_fence_before();
                arrive(B_V);
                round_row(x, lo);                      // r, and dv = beta r
                put_row(smem + L::U, i, at, lo);
                round_row(x, beta, hi);
                put_row(smem + L::OUT, i, at, hi);
                fence_proxy_async_smem();
                arrive(B_OUT);
            }
        }
        if constexpr (!BWD) {
            if (ok && !krows && (ok = wwait(B_P4, n - 1) && (n < 2 || wwait(B_OST, n - 2)))) {
                tc_fence_after();
                put_o();
            }
        }
        float* sT = BWD ? p.dh0 : p.hT;
        if (ok && sT && states && wwait(B_P3, n - 1)) {
            tc_fence_after();
            if constexpr (BWD) tmem_get(lb + TM_S, x);
            else tmem_get_sum(lb + TM_S, x);
#pragma unroll
            for (int e = 0; e < NPAIR; ++e) {
                sT[sbase + (int64_t)(2 * e) * DK] = x[e].x;
                sT[sbase + (int64_t)(2 * e + 1) * DK] = x[e].y;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, TM_COLS);
    }
}

template <int DK, bool BWD, int PT>
cudaError_t launch(const GDRArgs& a, const CallMaps& m, cudaStream_t s) {
    CUtensorMap mo;
    cudaError_t e;
    if ((e = map_steps(&mo, BWD ? a.dv : a.o, a.headdim, a.nheads, a.seqlen, a.batch, PT)) != cudaSuccess) return e;
    constexpr int bytes = Smem<DK>::BYTES;
    static std::atomic<uint64_t> attr_done{0};
    if ((e = allow_dynamic_smem(reinterpret_cast<const void*>(gdr_chain_kernel<DK, BWD, PT>), bytes, attr_done)) != cudaSuccess) return e;
    gdr_chain_kernel<DK, BWD, PT><<<(unsigned)(a.batch * a.nheads * (a.headdim / PT)), NTHREADS, bytes, s>>>(m.k, m.q, m.v, mo, a);
    return cudaGetLastError();
}

template <int DK>
cudaError_t launch_fwd(const GDRArgs& a, const CallMaps& m, cudaStream_t s) {
    // Tiles of 32 rows p where they still have an SM each: 1.72 us a chunk against
    // 2.24 (one sequence of 16397 steps, 32 heads of 128 rows: 442 us on 128 CTAs
    // against 575 on 64 with tiles of 64).
    // The checkpoint's tiles are of 64 rows, and so are the CTAs that write them.
    if (!a.states && a.batch * a.nheads * (a.headdim / 32) <= 148) return launch<DK, false, 32>(a, m, s);
    return launch<DK, false, kGdrTile>(a, m, s);
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

cudaError_t launch_gdr_chain(const GDRArgs& a, bool backward, const gdr::CallMaps& m, cudaStream_t s) {
    if (backward) return a.dstate == 64 ? gdr::launch<64, true, kGdrTile>(a, m, s) : gdr::launch<128, true, kGdrTile>(a, m, s);
    return a.dstate == 64 ? gdr::launch_fwd<64>(a, m, s) : gdr::launch_fwd<128>(a, m, s);
}

}  // namespace mmscan
