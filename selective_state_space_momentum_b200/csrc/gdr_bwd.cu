// gdr_bwd.cu -- sm_100a kernels for the gradients of the gated delta rule, in
// the chunked form (gdr_fwd.cu has the forward's formulas and names).
//
// From the forward, per chunk: T, Pm (the masked, scaled q.k), the decays,
// the state S at its start and the rows u it wrote.  With dS' the gradient
// reaching the state at the chunk's end, D_ij = e^(c_i - c_j) (j <= i), and
// rows i, j of the chunk:
//     du_j  = sum_{i>=j} Pm_ij do_i + e^(c_last - c_j) dS' k_j,    r = T^T du
//     dS    = e^(c_last) dS' + sum_i scale e^(c_i) do_i q_i^T - sum_j beta_j e^(c_j) r_j k_j^T
//     dv_j  = beta_j r_j
//     pd_ij = scale D_ij do_i.u_j (j <= i),   ad_ij = -beta_i D_ij r_i.u_j (j < i)
//     dq_i  = sum_j pd_ij k_j + scale e^(c_i) S^T do_i
//     dk_j  = sum_i pd_ij q_i + sum_i (ad_ij + ad_ji) k_i + e^(c_last - c_j) dS'^T u_j
//             - beta_j e^(c_j) S^T r_j
//     dbeta_i = r_i.v_i - e^(c_i) k_i.(S^T r_i) - sum_j D_ij (k_i.k_j) r_i.u_j
//     dc_i  = sum_j W_ij - sum_j W_ji + scale e^(c_i) q_i.(S^T do_i) - beta_i e^(c_i) k_i.(S^T r_i)
//             - e^(c_last - c_i) k_i.(dS'^T u_i),    W_ij = pd_ij q_i.k_j + ad_ij k_i.k_j  (j < i)
//     dc_last += e^(c_last) <S, dS'> + sum_i e^(c_last - c_i) k_i.(dS'^T u_i)
//     dg_t  = sum_{i >= t} dc_i over the chunk
// (the diagonal of W would cancel between its row and its column).
//
// Two launches: gdr_chain_kernel (gdr_chain.cu) walks the chunks backwards and
// writes dv, r and dS' per chunk; gdr_bwd_grad_kernel, parallel over chunks,
// forms the rest.  dq and dk of a group sum over its heads inside one block:
// no atomics, the same bits in every run.
//
// Precision: every gradient leaves as bf16 (2^-9).  The operands of the
// products are rounded to bf16 once each; products, sums, dS, the row sums
// and dc are fp32 or wider.  dh0 carries the products' operand rounding.
#include <cuda.h>

#include "gdr_common.cuh"

namespace mmscan {

static __device__ unsigned int g_grad_dev_err = 0;

namespace gdr {
namespace {

// ------------------------------------------------- everything else, by chunk ----
template <int DK, int DV>
struct GradSmem {
    static constexpr int Q = 0, K = Q + C * DK * 2, DO = K + C * DK * 2, S = DO + C * DV * 2, DS = S + DV * DK * 2;
    static constexpr int U = DS + DV * DK * 2, R = U + DV * C * 2, PD = R + DV * C * 2, AD = PD + C * C * 2;
    static constexpr int F = AD + C * C * 2;           // eg, tail, beta
    static constexpr int CUM = F + 3 * C * 4;          // double c[C]
    static constexpr int ROW = CUM + C * 8;            // float [4 column groups][3 kinds][C]
    static constexpr int COL = ROW + 12 * C * 4;       // float [4 row tiles][C]
    static constexpr int RV = COL + 4 * C * 4;         // float [C]: r.v
    static constexpr int RED = RV + C * 4;             // float [16]: <S, dS'> by warp
    static constexpr int BAR = RED + 64;               // q and k; do, u, r, decays; S, dS'
    static constexpr int BYTES = BAR + 3 * 8;
};

// acc (16 rows x NTC n-tiles) += A (64 x 64 stored [m][k], or [k][m]) . B stored
// [k][n] in slabs of 64 columns.
template <int NTC, bool AKM>
__device__ __forceinline__ void product(float (&acc)[NTC][4], uint32_t at, uint32_t bt, int m0, int nc0, int k_lo, int k_hi, int lane) {
#pragma unroll
    for (int kt = 0; kt < 4; ++kt) {
        if (kt < k_lo || kt > k_hi) continue;
        uint32_t a[4];
        if constexpr (AKM) load_a_km<128>(at, 16 * kt, 2 * m0, lane, a);
        else load_a_mk<128>(at, 16 * m0, 2 * kt, lane, a);
#pragma unroll
        for (int n = 0; n < NTC; n += 2) {
            uint32_t f[4];
            load_b_kn<128>(bt + ((nc0 + n) >> 3) * (C * 128), 16 * kt, (nc0 + n) & 7, lane, f);
            mma(acc[n], a, f[0], f[1]);
            mma(acc[n + 1], a, f[2], f[3]);
        }
    }
}

// acc += A . B over the head's width: A [row][p], B [n][p], both in tiles of 64 p.
template <int NTC, int DV, int DK>
__device__ __forceinline__ void product_p(float (&acc)[NTC][4], uint32_t at, uint32_t bt, int m0, int nc0, int lane) {
#pragma unroll
    for (int kt = 0; kt < DV / 16; ++kt) {
        uint32_t a[4];
        load_a_mk<128>(at + (kt >> 2) * (C * 128), 16 * m0, 2 * (kt & 3), lane, a);
#pragma unroll
        for (int n = 0; n < NTC; n += 2) {
            uint32_t f[4];
            load_b_nk<128>(bt + (kt >> 2) * (DK * 128), 8 * (nc0 + n), 2 * (kt & 3), lane, f);
            mma(acc[n], a, f[0], f[1]);
            mma(acc[n + 1], a, f[2], f[3]);
        }
    }
}

template <int NTC>
__device__ __forceinline__ void zero(float (&a)[NTC][4]) {
#pragma unroll
    for (int n = 0; n < NTC; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[n][e] = 0.0f;
}

// Row dots of acc with rows i0 and i0 + 8 of q or k (columns of this warp).
template <int NTC>
__device__ __forceinline__ float2 row_dots(const float (&acc)[NTC][4], const unsigned char* tile, int i0, int nc0, int tq) {
    float2 d = f2(0.0f, 0.0f);
#pragma unroll
    for (int n = 0; n < NTC; ++n) {
        const unsigned char* slab = tile + ((nc0 + n) >> 3) * (C * 128) + 4 * tq;
        const uint32_t a = *reinterpret_cast<const uint32_t*>(slab + tile_off<128>(i0, (nc0 + n) & 7));
        const uint32_t b = *reinterpret_cast<const uint32_t*>(slab + tile_off<128>(i0 + 8, (nc0 + n) & 7));
        d.x = fmaf(acc[n][0], bf16_lo(a), fmaf(acc[n][1], bf16_hi(a), d.x));
        d.y = fmaf(acc[n][2], bf16_lo(b), fmaf(acc[n][3], bf16_hi(b), d.y));
    }
    return d;
}

// Sixteen warps: warp w the rows 16 (w mod 4) .. and a quarter of the columns.
template <int DK, int DV>
__global__ void __launch_bounds__(512, 1)
gdr_bwd_grad_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_do, const __grid_constant__ CUtensorMap tm_dk,
                    const __grid_constant__ CUtensorMap tm_dq, const GDRArgs p) {
    using L = GradSmem<DK, DV>;
    constexpr int RB = DK * 2, NTC = DK / 32;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, lane = tid & 31, w = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int gq = lane >> 2, tq = lane & 3;
    const int mi = w & 3, hf = w >> 2, nc0 = hf * NTC;
    const int i0 = 16 * mi + gq;
    const int64_t ch = blockIdx.x % p.nchunks, bg = blockIdx.x / p.nchunks;
    const int64_t b = bg / p.ngroups, grp = bg - b * p.ngroups;
    const int hpg = (int)(p.nheads / p.ngroups);
    const int64_t t0 = ch * C;
    const int valid = (int)(p.seqlen - t0 < C ? p.seqlen - t0 : C);
    const int64_t vstride = p.nheads * DV * 2;
    const uint32_t base = smem_u32(sm), bar = base + L::BAR;
    const uint32_t qs = base + L::Q, ks = base + L::K, dos = base + L::DO, ss = base + L::S, dss = base + L::DS, us = base + L::U,
                   rs = base + L::R, pds = base + L::PD, ads = base + L::AD;
    float* eg = reinterpret_cast<float*>(sm + L::F);
    double* cum = reinterpret_cast<double*>(sm + L::CUM);
    float* rowv = reinterpret_cast<float*>(sm + L::ROW);
    float* colv = reinterpret_cast<float*>(sm + L::COL);
    float* rvv = reinterpret_cast<float*>(sm + L::RV);
    float* red = reinterpret_cast<float*>(sm + L::RED);
    auto record = [&](int hh) { return (b * p.nheads + grp * hpg + hh) * p.nchunks + ch; };
    auto issue = [&](int hh) {                // one thread: the tiles of head hh of the group
        const int64_t rec = record(hh);
        mbar_expect_tx(bar + 8, 3 * C * DV * 2 + 3 * C * 4);
#pragma unroll
        for (int t = 0; t < DV / 64; ++t)
            tma_load_4d(dos + t * C * 128, &tm_do, bar + 8, 64 * t, (int)grp * hpg + hh, (int)t0, (int)b);
        bulk_load(us, static_cast<const unsigned char*>(p.u) + rec * DV * C * 2, DV * C * 2, bar + 8);
        bulk_load(rs, static_cast<const unsigned char*>(p.dr) + rec * DV * C * 2, DV * C * 2, bar + 8);
        bulk_load(base + L::F, static_cast<const unsigned char*>(p.rec) + rec * REC_BYTES + REC_F, 3 * C * 4, bar + 8);
        mbar_expect_tx(bar + 16, 2 * DV * RB);
        bulk_load(ss, static_cast<const unsigned char*>(p.states) + rec * DV * RB, DV * RB, bar + 16);
        bulk_load(dss, static_cast<const unsigned char*>(p.dstates) + rec * DV * RB, DV * RB, bar + 16);
    };
    // Whether the loads behind barrier k have come (the same answer to everybody).
    auto landed = [&](int k, int phase) {
        return __syncthreads_and(mbar_wait_sleep(bar + 8 * k, (uint32_t)phase & 1u, &g_grad_dev_err)) != 0;
    };
    if (tid == 0) {
        for (int k = 0; k < 3; ++k) mbar_init(bar + 8 * k, 1);
        fence_barrier_init();
        if (!p.stall) {                       // (test only: nothing staged, the waits run out)
            mbar_expect_tx(bar, 2 * C * RB);
#pragma unroll
            for (int s = 0; s < DK / 64; ++s) {
                tma_load_4d(qs + s * C * 128, &tm_q, bar, 64 * s, (int)grp, (int)t0, (int)b);
                tma_load_4d(ks + s * C * 128, &tm_k, bar, 64 * s, (int)grp, (int)t0, (int)b);
            }
            issue(0);
        }
    }
    __syncthreads();

    float dq[NTC][4], dk[NTC][4], qk[2][4], kk[2][4];
    zero(dq); zero(dk); zero(qk); zero(kk);
    for (int hh = 0; hh < hpg; ++hh) {
        const int64_t h = grp * hpg + hh;
        if (w == 15) {
            double s0, s1, last;
            chunk_cumsum(static_cast<const bf16*>(p.g) + (b * p.seqlen + t0) * p.nheads + h, p.nheads, valid, lane, s0, s1, last);
            cum[2 * lane] = s0;
            cum[2 * lane + 1] = s1;
        }
        if (hh == 0) {                        // q.k and k.k are the group's
            if (!landed(0, 0)) return;
            if (hf <= mi) {
#pragma unroll
                for (int kt = 0; kt < DK / 16; ++kt) {
                    const uint32_t slab = (kt >> 2) * C * 128;
                    uint32_t aq[4], ak[4], f[4];
                    load_a_mk<128>(qs + slab, 16 * mi, 2 * (kt & 3), lane, aq);
                    load_a_mk<128>(ks + slab, 16 * mi, 2 * (kt & 3), lane, ak);
                    load_b_nk<128>(ks + slab, 16 * hf, 2 * (kt & 3), lane, f);
                    mma(qk[0], aq, f[0], f[1]);
                    mma(qk[1], aq, f[2], f[3]);
                    mma(kk[0], ak, f[0], f[1]);
                    mma(kk[1], ak, f[2], f[3]);
                }
            }
        }
        if (!landed(1, hh)) return;
        float dp[2][4], da[2][4];
        zero(dp); zero(da);
        if (hf <= mi) {
#pragma unroll
            for (int kt = 0; kt < DV / 16; ++kt) {
                const uint32_t slab = (kt >> 2) * C * 128;
                uint32_t ao[4], ar[4], f[4];
                load_a_mk<128>(dos + slab, 16 * mi, 2 * (kt & 3), lane, ao);
                load_a_mk<128>(rs + slab, 16 * mi, 2 * (kt & 3), lane, ar);
                load_b_nk<128>(us + slab, 16 * hf, 2 * (kt & 3), lane, f);
                mma(dp[0], ao, f[0], f[1]);
                mma(dp[1], ao, f[2], f[3]);
                mma(da[0], ar, f[0], f[1]);
                mma(da[1], ar, f[2], f[3]);
            }
        }
        // rows' sums kept by this thread: [row half] of dc, of e^.. k.(dS' u), of dbeta
        float rc[2] = {0.0f, 0.0f}, rk[2] = {0.0f, 0.0f}, rb[2] = {0.0f, 0.0f};
        const double c0 = cum[i0], c1 = cum[i0 + 8];
        const float b0 = eg[2 * C + i0], b1 = eg[2 * C + i0 + 8];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            if (hf > mi) break;
            const int j = 16 * hf + 8 * n + 2 * tq;
            float cs[2] = {0.0f, 0.0f};
            float pv[4], av[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + 8 * (e >> 1), jj = j + (e & 1);
                const float d = jj <= i ? ex2_approx((float)(((e >> 1 ? c1 : c0) - cum[jj]) * kLog2e)) : 0.0f;
                pv[e] = p.scale * d * dp[n][e];
                const float x = jj < i ? -d * da[n][e] : 0.0f;
                av[e] = (e >> 1 ? b1 : b0) * x;
                const float wv = jj < i ? fmaf(pv[e], qk[n][e], av[e] * kk[n][e]) : 0.0f;
                rc[e >> 1] += wv;
                cs[e & 1] += wv;
                rb[e >> 1] = fmaf(x, kk[n][e], rb[e >> 1]);
            }
            *reinterpret_cast<uint32_t*>(sm + L::PD + tile_off<128>(i0, 2 * hf + n) + 4 * tq) = pack_bf16x2(pv[0], pv[1]);
            *reinterpret_cast<uint32_t*>(sm + L::PD + tile_off<128>(i0 + 8, 2 * hf + n) + 4 * tq) = pack_bf16x2(pv[2], pv[3]);
            *reinterpret_cast<uint32_t*>(sm + L::AD + tile_off<128>(i0, 2 * hf + n) + 4 * tq) = pack_bf16x2(av[0], av[1]);
            *reinterpret_cast<uint32_t*>(sm + L::AD + tile_off<128>(i0 + 8, 2 * hf + n) + 4 * tq) = pack_bf16x2(av[2], av[3]);
#pragma unroll
            for (int m = 4; m < 32; m <<= 1) {
                cs[0] += __shfl_xor_sync(0xffffffffu, cs[0], m);
                cs[1] += __shfl_xor_sync(0xffffffffu, cs[1], m);
            }
            if (gq == 0) *reinterpret_cast<float2*>(colv + mi * C + j) = f2(cs[0], cs[1]);
        }
        {                                     // r.v, eight threads a row
            const int i = tid >> 3, part = tid & 7;
            float d = 0.0f;
            if (i < valid) {
                const uint4* vg = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.v) + (b * p.seqlen + t0 + i) * vstride + h * DV * 2);
#pragma unroll
                for (int x = part; x < DV / 8; x += 8) {
                    const uint4 vv = vg[x];
                    const uint4 rr = *reinterpret_cast<const uint4*>(sm + L::R + (x >> 3) * (C * 128) + tile_off<128>(i, x & 7));
                    d = fmaf(bf16_lo(vv.x), bf16_lo(rr.x), fmaf(bf16_hi(vv.x), bf16_hi(rr.x), d));
                    d = fmaf(bf16_lo(vv.y), bf16_lo(rr.y), fmaf(bf16_hi(vv.y), bf16_hi(rr.y), d));
                    d = fmaf(bf16_lo(vv.z), bf16_lo(rr.z), fmaf(bf16_hi(vv.z), bf16_hi(rr.z), d));
                    d = fmaf(bf16_lo(vv.w), bf16_lo(rr.w), fmaf(bf16_hi(vv.w), bf16_hi(rr.w), d));
                }
            }
#pragma unroll
            for (int m = 1; m < 8; m <<= 1) d += __shfl_xor_sync(0xffffffffu, d, m);
            if (part == 0) rvv[i] = d;
        }
        if (!landed(2, hh)) return;           // pd, ad, S, dS' are there

        product<NTC, false>(dq, pds, ks, mi, nc0, 0, mi, lane);
        product<NTC, true>(dk, pds, qs, mi, nc0, mi, 3, lane);
        product<NTC, false>(dk, ads, ks, mi, nc0, 0, mi, lane);
        product<NTC, true>(dk, ads, ks, mi, nc0, mi, 3, lane);
        float acc[NTC][4];
        {
            zero(acc);
            product_p<NTC, DV, DK>(acc, dos, ss, mi, nc0, lane);
            const float f0 = p.scale * eg[i0], f1 = p.scale * eg[i0 + 8];
            const float2 d = row_dots<NTC>(acc, sm + L::Q, i0, nc0, tq);
            rc[0] = fmaf(f0, d.x, rc[0]);
            rc[1] = fmaf(f1, d.y, rc[1]);
#pragma unroll
            for (int n = 0; n < NTC; ++n) {
                dq[n][0] = fmaf(f0, acc[n][0], dq[n][0]);
                dq[n][1] = fmaf(f0, acc[n][1], dq[n][1]);
                dq[n][2] = fmaf(f1, acc[n][2], dq[n][2]);
                dq[n][3] = fmaf(f1, acc[n][3], dq[n][3]);
            }
        }
        {
            zero(acc);
            product_p<NTC, DV, DK>(acc, rs, ss, mi, nc0, lane);
            const float f0 = eg[i0], f1 = eg[i0 + 8];
            const float2 d = row_dots<NTC>(acc, sm + L::K, i0, nc0, tq);
            rb[0] = fmaf(-f0, d.x, rb[0]);
            rb[1] = fmaf(-f1, d.y, rb[1]);
            rc[0] = fmaf(-f0 * b0, d.x, rc[0]);
            rc[1] = fmaf(-f1 * b1, d.y, rc[1]);
#pragma unroll
            for (int n = 0; n < NTC; ++n) {
                dk[n][0] = fmaf(-f0 * b0, acc[n][0], dk[n][0]);
                dk[n][1] = fmaf(-f0 * b0, acc[n][1], dk[n][1]);
                dk[n][2] = fmaf(-f1 * b1, acc[n][2], dk[n][2]);
                dk[n][3] = fmaf(-f1 * b1, acc[n][3], dk[n][3]);
            }
        }
        {
            zero(acc);
            product_p<NTC, DV, DK>(acc, us, dss, mi, nc0, lane);
            const float f0 = eg[C + i0], f1 = eg[C + i0 + 8];
            const float2 d = row_dots<NTC>(acc, sm + L::K, i0, nc0, tq);
            rk[0] = f0 * d.x;
            rk[1] = f1 * d.y;
#pragma unroll
            for (int n = 0; n < NTC; ++n) {
                dk[n][0] = fmaf(f0, acc[n][0], dk[n][0]);
                dk[n][1] = fmaf(f0, acc[n][1], dk[n][1]);
                dk[n][2] = fmaf(f1, acc[n][2], dk[n][2]);
                dk[n][3] = fmaf(f1, acc[n][3], dk[n][3]);
            }
        }
        // <S, dS'>: both tiles have the same layout
        float sd = 0.0f;
#pragma unroll 4
        for (int i = tid; i < DV * RB / 16; i += 512) {
            const uint4 x = *reinterpret_cast<const uint4*>(sm + L::S + i * 16), y = *reinterpret_cast<const uint4*>(sm + L::DS + i * 16);
            sd = fmaf(bf16_lo(x.x), bf16_lo(y.x), fmaf(bf16_hi(x.x), bf16_hi(y.x), sd));
            sd = fmaf(bf16_lo(x.y), bf16_lo(y.y), fmaf(bf16_hi(x.y), bf16_hi(y.y), sd));
            sd = fmaf(bf16_lo(x.z), bf16_lo(y.z), fmaf(bf16_hi(x.z), bf16_hi(y.z), sd));
            sd = fmaf(bf16_lo(x.w), bf16_lo(y.w), fmaf(bf16_hi(x.w), bf16_hi(y.w), sd));
        }
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) sd += __shfl_xor_sync(0xffffffffu, sd, m);
        if (lane == 0) red[w] = sd;
#pragma unroll
        for (int m = 1; m < 4; m <<= 1)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                rc[e] += __shfl_xor_sync(0xffffffffu, rc[e], m);
                rk[e] += __shfl_xor_sync(0xffffffffu, rk[e], m);
                rb[e] += __shfl_xor_sync(0xffffffffu, rb[e], m);
            }
        if (tq == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                rowv[(hf * 3 + 0) * C + i0 + 8 * e] = rc[e];
                rowv[(hf * 3 + 1) * C + i0 + 8 * e] = rk[e];
                rowv[(hf * 3 + 2) * C + i0 + 8 * e] = rb[e];
            }
        }
        const float eg_last = eg[C - 1];
        __syncthreads();
        if (tid == 0 && hh + 1 < hpg) issue(hh + 1);       // every product has read this head's tiles
        if (w == 0) {
            float dc[2], ok[2], db[2], sums = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                float col = 0.0f;
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (m >= i / 16) col += colv[m * C + i];       // row tiles from the diagonal on were written
                ok[e] = dc[e] = db[e] = 0.0f;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    dc[e] += rowv[3 * m * C + i];
                    ok[e] += rowv[(3 * m + 1) * C + i];
                    db[e] += rowv[(3 * m + 2) * C + i];
                }
                dc[e] -= col + ok[e];
                sums += ok[e];
            }
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) sums += __shfl_xor_sync(0xffffffffu, sums, m);
            if (lane == 31) {
                float t = 0.0f;
#pragma unroll
                for (int m = 0; m < 16; ++m) t += red[m];
                dc[1] = fmaf(eg_last, t, dc[1] + sums);
            }
            // dg = the sums from each row to the chunk's end
            dc[0] += dc[1];
            float run = dc[0];
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const float dn = __shfl_down_sync(0xffffffffu, run, m);
                if (lane + m < 32) run += dn;
            }
            const float after = run - dc[0];
            const int64_t at = (b * p.seqlen + t0 + 2 * lane) * p.nheads + h;
            bf16* dg = static_cast<bf16*>(p.dg);
            bf16* dbg = static_cast<bf16*>(p.dbeta);
            if (2 * lane < valid) {
                dg[at] = __float2bfloat16_rn(run);
                dbg[at] = __float2bfloat16_rn(rvv[2 * lane] + db[0]);
            }
            if (2 * lane + 1 < valid) {
                dg[at + p.nheads] = __float2bfloat16_rn(dc[1] + after);
                dbg[at + p.nheads] = __float2bfloat16_rn(rvv[2 * lane + 1] + db[1]);
            }
        }
    }
    // dq, dk through the tiles of q and k to memory (rows past L are clipped)
#pragma unroll
    for (int n = 0; n < NTC; ++n) {
        const uint32_t slab = ((nc0 + n) >> 3) * (C * 128) + 4 * tq;
        const uint32_t o0 = slab + tile_off<128>(i0, (nc0 + n) & 7), o1 = slab + tile_off<128>(i0 + 8, (nc0 + n) & 7);
        *reinterpret_cast<uint32_t*>(sm + L::Q + o0) = pack_bf16x2(dq[n][0], dq[n][1]);
        *reinterpret_cast<uint32_t*>(sm + L::Q + o1) = pack_bf16x2(dq[n][2], dq[n][3]);
        *reinterpret_cast<uint32_t*>(sm + L::K + o0) = pack_bf16x2(dk[n][0], dk[n][1]);
        *reinterpret_cast<uint32_t*>(sm + L::K + o1) = pack_bf16x2(dk[n][2], dk[n][3]);
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int s = 0; s < DK / 64; ++s) {
            tma_store_4d(&tm_dq, qs + s * C * 128, 64 * s, (int)grp, (int)t0, (int)b);
            tma_store_4d(&tm_dk, ks + s * C * 128, 64 * s, (int)grp, (int)t0, (int)b);
        }
        bulk_commit_group();
        bulk_wait_all();                      // complete before the CTA exits
    }
}

unsigned int read_and_clear_grad_error() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_grad_dev_err, sizeof(v)) != cudaSuccess) return 0;
    if (v) cudaMemcpyToSymbol(g_grad_dev_err, &z, sizeof(z));
    return v;
}

[[maybe_unused]] const bool g_registered = (register_error_reader(read_and_clear_grad_error), true);

template <int DK, int DV>
cudaError_t launch_grad(const GDRArgs& a, cudaStream_t s) {
    constexpr int bytes = GradSmem<DK, DV>::BYTES;
    static_assert(bytes <= 227 * 1024, "shared memory");
    CUtensorMap mk, mq, mdo, mdk, mdq;
    cudaError_t e;
    if ((e = map_steps(&mk, a.k, DK, a.ngroups, a.seqlen, a.batch)) != cudaSuccess) return e;
    if ((e = map_steps(&mq, a.q, DK, a.ngroups, a.seqlen, a.batch)) != cudaSuccess) return e;
    if ((e = map_steps(&mdk, a.dk, DK, a.ngroups, a.seqlen, a.batch)) != cudaSuccess) return e;
    if ((e = map_steps(&mdq, a.dq, DK, a.ngroups, a.seqlen, a.batch)) != cudaSuccess) return e;
    if ((e = map_steps(&mdo, a.dout, DV, a.nheads, a.seqlen, a.batch)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(gdr_bwd_grad_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) != cudaSuccess) return e;
    gdr_bwd_grad_kernel<DK, DV><<<(unsigned)(a.batch * a.ngroups * a.nchunks), 512, bytes, s>>>(mk, mq, mdo, mdk, mdq, a);
    return cudaGetLastError();
}

template <int DK>
cudaError_t launch_bwd(const GDRArgs& a, cudaStream_t s) {
    cudaError_t e = launch_gdr_chain(a, true, s);
    if (e != cudaSuccess) return e;
    return a.headdim == 64 ? launch_grad<DK, 64>(a, s) : launch_grad<DK, 128>(a, s);
}

}  // namespace
}  // namespace gdr

cudaError_t launch_gdr_bwd(const GDRArgs& a, cudaStream_t s) {
    return a.dstate == 64 ? gdr::launch_bwd<64>(a, s) : gdr::launch_bwd<128>(a, s);
}

}  // namespace mmscan
