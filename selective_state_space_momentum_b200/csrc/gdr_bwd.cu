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
#include "gdr_common.cuh"

namespace mmscan {

namespace gdr {

// ------------------------------------------------- everything else, by chunk ----
template <int DK, int DV>
struct GradSmem {
    static constexpr int Q = 0, K = Q + C * DK * 2, DO = K + C * DK * 2, S = DO + C * DV * 2, DS = S + DV * DK * 2;
    static constexpr int U = DS + DV * DK * 2, R = U + DV * C * 2, PD = R + DV * C * 2, AD = PD + C * C * 2;
    static constexpr int F = AD + C * C * 2;           // eg, tail, beta
    static constexpr int CUM = F + 3 * C * 4;          // double c[C]
    static constexpr int ROW = CUM + C * 8;            // float [2 halves][3 kinds][C]
    static constexpr int COL = ROW + 6 * C * 4;        // float [4 row tiles][C]
    static constexpr int RV = COL + 4 * C * 4;         // float [C]: r.v
    static constexpr int RED = RV + C * 4;             // float [8]: <S, dS'> by warp
    static constexpr int BYTES = RED + 64;
};

// acc (16 rows x NTC n-tiles) += A (k from stored [k][m] or [m][k]) . B stored [k][n]
template <int NTC, int KT, bool AKM, int RA, int RBB>
__device__ __forceinline__ void product(float (&acc)[NTC][4], uint32_t at, uint32_t bt, int m0, int nc0, int k_lo, int k_hi, int lane) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
        if (kt < k_lo || kt > k_hi) continue;
        uint32_t a[4];
        if constexpr (AKM) load_a_km<RA>(at, 16 * kt, 2 * m0, lane, a);
        else load_a_mk<RA>(at, 16 * m0, 2 * kt, lane, a);
#pragma unroll
        for (int n = 0; n < NTC; n += 2) {
            uint32_t f[4];
            load_b_kn<RBB>(bt, 16 * kt, nc0 + n, lane, f);
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

// Row dots of acc with a tile's rows i0 and i0 + 8 (columns of this warp).
template <int NTC, int RB>
__device__ __forceinline__ float2 row_dots(const float (&acc)[NTC][4], const unsigned char* tile, int i0, int nc0, int tq) {
    float2 d = f2(0.0f, 0.0f);
#pragma unroll
    for (int n = 0; n < NTC; ++n) {
        const uint32_t a = *reinterpret_cast<const uint32_t*>(tile + tile_off<RB>(i0, nc0 + n) + 4 * tq);
        const uint32_t b = *reinterpret_cast<const uint32_t*>(tile + tile_off<RB>(i0 + 8, nc0 + n) + 4 * tq);
        d.x = fmaf(acc[n][0], bf16_lo(a), fmaf(acc[n][1], bf16_hi(a), d.x));
        d.y = fmaf(acc[n][2], bf16_lo(b), fmaf(acc[n][3], bf16_hi(b), d.y));
    }
    return d;
}

template <int DK, int DV>
__global__ void __launch_bounds__(256, 1) gdr_bwd_grad_kernel(const GDRArgs p) {
    using L = GradSmem<DK, DV>;
    constexpr int RB = DK * 2, NTC = DK / 16;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int gq = lane >> 2, tq = lane & 3;
    const int mi = w & 3, hf = w >> 2, nc0 = hf * NTC;
    const int i0 = 16 * mi + gq;
    const int64_t ch = blockIdx.x % p.nchunks, bg = blockIdx.x / p.nchunks;
    const int64_t b = bg / p.ngroups, grp = bg - b * p.ngroups;
    const int hpg = (int)(p.nheads / p.ngroups);
    const int64_t t0 = ch * C;
    const int valid = (int)(p.seqlen - t0 < C ? p.seqlen - t0 : C);
    const int64_t kstride = p.ngroups * DK * 2, vstride = p.nheads * DV * 2;
    const int64_t koff = (b * p.seqlen + t0) * kstride + grp * DK * 2;
    const uint32_t qs = smem_u32(sm + L::Q), ks = smem_u32(sm + L::K), dos = smem_u32(sm + L::DO), ss = smem_u32(sm + L::S),
                   dss = smem_u32(sm + L::DS), us = smem_u32(sm + L::U), rs = smem_u32(sm + L::R), pds = smem_u32(sm + L::PD),
                   ads = smem_u32(sm + L::AD);
    float* eg = reinterpret_cast<float*>(sm + L::F);
    double* cum = reinterpret_cast<double*>(sm + L::CUM);
    float* rowv = reinterpret_cast<float*>(sm + L::ROW);
    float* colv = reinterpret_cast<float*>(sm + L::COL);
    float* rvv = reinterpret_cast<float*>(sm + L::RV);
    float* red = reinterpret_cast<float*>(sm + L::RED);

    load_tile<RB, C>(sm + L::Q, static_cast<const unsigned char*>(p.q) + koff, kstride, valid, tid, 256);
    load_tile<RB, C>(sm + L::K, static_cast<const unsigned char*>(p.k) + koff, kstride, valid, tid, 256);
    cp_async_commit();

    float dq[NTC][4], dk[NTC][4], qk[4][4], kk[4][4];
    zero(dq); zero(dk); zero(qk); zero(kk);
    for (int hh = 0; hh < hpg; ++hh) {
        const int64_t h = grp * hpg + hh;
        const int64_t rec = (b * p.nheads + h) * p.nchunks + ch;
        const int64_t voff = (b * p.seqlen + t0) * vstride + h * DV * 2;
        const unsigned char* rg = static_cast<const unsigned char*>(p.rec) + rec * REC_BYTES;
#pragma unroll
        for (int t = 0; t < DV / 64; ++t)
            load_tile<128, C>(sm + L::DO + t * C * 128, static_cast<const unsigned char*>(p.dout) + voff + t * 128, vstride, valid, tid, 256);
        load_image(sm + L::U, static_cast<const unsigned char*>(p.u) + rec * DV * C * 2, DV * C * 2, tid, 256);
        load_image(sm + L::R, static_cast<const unsigned char*>(p.dr) + rec * DV * C * 2, DV * C * 2, tid, 256);
        if (tid < 48) cp_async_16(sm + L::F + tid * 16, rg + REC_F + tid * 16, 16);
        cp_async_commit();
        load_image(sm + L::S, static_cast<const unsigned char*>(p.states) + rec * DV * RB, DV * RB, tid, 256);
        load_image(sm + L::DS, static_cast<const unsigned char*>(p.dstates) + rec * DV * RB, DV * RB, tid, 256);
        cp_async_commit();
        if (w == 7) {
            double s0, s1, last;
            chunk_cumsum(static_cast<const bf16*>(p.g) + (b * p.seqlen + t0) * p.nheads + h, p.nheads, valid, lane, s0, s1, last);
            cum[2 * lane] = s0;
            cum[2 * lane + 1] = s1;
        }
        cp_async_wait<1>();
        __syncthreads();

        if (hh == 0) {                        // q.k and k.k are the group's
#pragma unroll
            for (int kt = 0; kt < DK / 16; ++kt) {
                uint32_t aq[4], ak[4];
                load_a_mk<RB>(qs, 16 * mi, 2 * kt, lane, aq);
                load_a_mk<RB>(ks, 16 * mi, 2 * kt, lane, ak);
#pragma unroll
                for (int n = 0; n < 4; n += 2) {
                    if (4 * hf + n > 2 * mi + 1) break;
                    uint32_t f[4];
                    load_b_nk<RB>(ks, 32 * hf + 8 * n, 2 * kt, lane, f);
                    mma(qk[n], aq, f[0], f[1]);
                    mma(qk[n + 1], aq, f[2], f[3]);
                    mma(kk[n], ak, f[0], f[1]);
                    mma(kk[n + 1], ak, f[2], f[3]);
                }
            }
        }
        float dp[4][4], da[4][4];
        zero(dp); zero(da);
#pragma unroll
        for (int kt = 0; kt < DV / 16; ++kt) {
            uint32_t ao[4], ar[4];
            load_a_mk<128>(dos + (kt >> 2) * (C * 128), 16 * mi, 2 * (kt & 3), lane, ao);
            load_a_mk<128>(rs + (kt >> 2) * (C * 128), 16 * mi, 2 * (kt & 3), lane, ar);
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
                if (4 * hf + n > 2 * mi + 1) break;
                uint32_t f[4];
                load_b_nk<128>(us + (kt >> 2) * (C * 128), 32 * hf + 8 * n, 2 * (kt & 3), lane, f);
                mma(dp[n], ao, f[0], f[1]);
                mma(dp[n + 1], ao, f[2], f[3]);
                mma(da[n], ar, f[0], f[1]);
                mma(da[n + 1], ar, f[2], f[3]);
            }
        }
        // rows' sums kept by this thread: [row half] of dc, of e^.. k.(dS' u), of dbeta
        float rc[2] = {0.0f, 0.0f}, rk[2] = {0.0f, 0.0f}, rb[2] = {0.0f, 0.0f};
        const double c0 = cum[i0], c1 = cum[i0 + 8];
        const float b0 = eg[2 * C + i0], b1 = eg[2 * C + i0 + 8];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (4 * hf + n > 2 * mi + 1) break;
            const int j = 32 * hf + 8 * n + 2 * tq;
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
            *reinterpret_cast<uint32_t*>(sm + L::PD + tile_off<128>(i0, 4 * hf + n) + 4 * tq) = pack_bf16x2(pv[0], pv[1]);
            *reinterpret_cast<uint32_t*>(sm + L::PD + tile_off<128>(i0 + 8, 4 * hf + n) + 4 * tq) = pack_bf16x2(pv[2], pv[3]);
            *reinterpret_cast<uint32_t*>(sm + L::AD + tile_off<128>(i0, 4 * hf + n) + 4 * tq) = pack_bf16x2(av[0], av[1]);
            *reinterpret_cast<uint32_t*>(sm + L::AD + tile_off<128>(i0 + 8, 4 * hf + n) + 4 * tq) = pack_bf16x2(av[2], av[3]);
#pragma unroll
            for (int m = 4; m < 32; m <<= 1) {
                cs[0] += __shfl_xor_sync(0xffffffffu, cs[0], m);
                cs[1] += __shfl_xor_sync(0xffffffffu, cs[1], m);
            }
            if (gq == 0) *reinterpret_cast<float2*>(colv + mi * C + j) = f2(cs[0], cs[1]);
        }
        {                                     // r.v, four threads a row
            const int i = tid >> 2, part = tid & 3;
            float d = 0.0f;
            if (i < valid) {
                const uint4* vg = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.v) + voff + i * vstride);
#pragma unroll
                for (int x = part * (DV / 32); x < (part + 1) * (DV / 32); ++x) {
                    const uint4 vv = vg[x];
                    const uint4 rr = *reinterpret_cast<const uint4*>(sm + L::R + (x >> 3) * (C * 128) + tile_off<128>(i, x & 7));
                    d = fmaf(bf16_lo(vv.x), bf16_lo(rr.x), fmaf(bf16_hi(vv.x), bf16_hi(rr.x), d));
                    d = fmaf(bf16_lo(vv.y), bf16_lo(rr.y), fmaf(bf16_hi(vv.y), bf16_hi(rr.y), d));
                    d = fmaf(bf16_lo(vv.z), bf16_lo(rr.z), fmaf(bf16_hi(vv.z), bf16_hi(rr.z), d));
                    d = fmaf(bf16_lo(vv.w), bf16_lo(rr.w), fmaf(bf16_hi(vv.w), bf16_hi(rr.w), d));
                }
            }
            d += __shfl_xor_sync(0xffffffffu, d, 1);
            d += __shfl_xor_sync(0xffffffffu, d, 2);
            if (part == 0) rvv[i] = d;
        }
        cp_async_wait<0>();
        __syncthreads();                      // pd, ad, S, dS' are there

        product<NTC, 4, false, 128, RB>(dq, pds, ks, mi, nc0, 0, mi, lane);
        product<NTC, 4, true, 128, RB>(dk, pds, qs, mi, nc0, mi, 3, lane);
        product<NTC, 4, false, 128, RB>(dk, ads, ks, mi, nc0, 0, mi, lane);
        product<NTC, 4, true, 128, RB>(dk, ads, ks, mi, nc0, mi, 3, lane);
        float acc[NTC][4];
        {
            zero(acc);
            product_p<NTC, DV, DK>(acc, dos, ss, mi, nc0, lane);
            const float f0 = p.scale * eg[i0], f1 = p.scale * eg[i0 + 8];
            const float2 d = row_dots<NTC, RB>(acc, sm + L::Q, i0, nc0, tq);
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
            const float2 d = row_dots<NTC, RB>(acc, sm + L::K, i0, nc0, tq);
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
            const float2 d = row_dots<NTC, RB>(acc, sm + L::K, i0, nc0, tq);
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
        for (int i = tid; i < DV * RB / 16; i += 256) {
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
        __syncthreads();
        if (w == 0) {
            float dc[2], ok[2], sums = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                float col = 0.0f;
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    if (m >= i / 16) col += colv[m * C + i];       // row tiles from the diagonal on were written
                ok[e] = rowv[C + i] + rowv[4 * C + i];
                dc[e] = rowv[i] + rowv[3 * C + i] - col - ok[e];
                sums += ok[e];
            }
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) sums += __shfl_xor_sync(0xffffffffu, sums, m);
            if (lane == 31) {
                float t = 0.0f;
#pragma unroll
                for (int m = 0; m < 8; ++m) t += red[m];
                dc[1] = fmaf(eg[C - 1], t, dc[1] + sums);
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
            bf16* db = static_cast<bf16*>(p.dbeta);
            if (2 * lane < valid) {
                dg[at] = __float2bfloat16_rn(run);
                db[at] = __float2bfloat16_rn(rvv[2 * lane] + rowv[2 * C + 2 * lane] + rowv[5 * C + 2 * lane]);
            }
            if (2 * lane + 1 < valid) {
                dg[at + p.nheads] = __float2bfloat16_rn(dc[1] + after);
                db[at + p.nheads] = __float2bfloat16_rn(rvv[2 * lane + 1] + rowv[2 * C + 2 * lane + 1] + rowv[5 * C + 2 * lane + 1]);
            }
        }
        __syncthreads();                      // the next head overwrites the tiles and the sums
    }
    // dq, dk through the tiles of q and k to memory
#pragma unroll
    for (int n = 0; n < NTC; ++n) {
        *reinterpret_cast<uint32_t*>(sm + L::Q + tile_off<RB>(i0, nc0 + n) + 4 * tq) = pack_bf16x2(dq[n][0], dq[n][1]);
        *reinterpret_cast<uint32_t*>(sm + L::Q + tile_off<RB>(i0 + 8, nc0 + n) + 4 * tq) = pack_bf16x2(dq[n][2], dq[n][3]);
        *reinterpret_cast<uint32_t*>(sm + L::K + tile_off<RB>(i0, nc0 + n) + 4 * tq) = pack_bf16x2(dk[n][0], dk[n][1]);
        *reinterpret_cast<uint32_t*>(sm + L::K + tile_off<RB>(i0 + 8, nc0 + n) + 4 * tq) = pack_bf16x2(dk[n][2], dk[n][3]);
    }
    __syncthreads();
    for (int i = tid; i < C * RB / 16; i += 256) {
        const int r = i / (RB / 16), c = i % (RB / 16);
        if (r < valid) {
            *reinterpret_cast<uint4*>(static_cast<unsigned char*>(p.dq) + koff + r * kstride + c * 16) =
                *reinterpret_cast<const uint4*>(sm + L::Q + tile_off<RB>(r, c));
            *reinterpret_cast<uint4*>(static_cast<unsigned char*>(p.dk) + koff + r * kstride + c * 16) =
                *reinterpret_cast<const uint4*>(sm + L::K + tile_off<RB>(r, c));
        }
    }
}

template <int DK, int DV>
cudaError_t launch_grad(const GDRArgs& a, cudaStream_t s) {
    constexpr int bytes = GradSmem<DK, DV>::BYTES;
    static_assert(bytes <= 227 * 1024, "shared memory");
    cudaError_t e = cudaFuncSetAttribute(gdr_bwd_grad_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    gdr_bwd_grad_kernel<DK, DV><<<(unsigned)(a.batch * a.ngroups * a.nchunks), 256, bytes, s>>>(a);
    return cudaGetLastError();
}

template <int DK>
cudaError_t launch_bwd(const GDRArgs& a, cudaStream_t s) {
    cudaError_t e = launch_gdr_chain(a, true, s);
    if (e != cudaSuccess) return e;
    return a.headdim == 64 ? launch_grad<DK, 64>(a, s) : launch_grad<DK, 128>(a, s);
}

}  // namespace gdr

cudaError_t launch_gdr_bwd(const GDRArgs& a, cudaStream_t s) {
    return a.dstate == 64 ? gdr::launch_bwd<64>(a, s) : gdr::launch_bwd<128>(a, s);
}

}  // namespace mmscan
