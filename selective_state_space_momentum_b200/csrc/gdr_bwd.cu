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
// Two launches: gdr_bwd_chain_kernel walks the chunks backwards, one warp per
// 16 rows p of dS as in the forward, and writes dv, r and dS' per chunk;
// gdr_bwd_grad_kernel, parallel over chunks, forms the rest.  dq and dk of a
// group sum over its heads inside one block: no atomics, the same bits in
// every run.
//
// Precision: every gradient leaves as bf16 (2^-9).  The operands of the
// products are rounded to bf16 once each; products, sums, dS, the row sums
// and dc are fp32 or wider.  dh0 carries the products' operand rounding.
#include "gdr_common.cuh"

namespace mmscan {

namespace gdr {

template <int DK, int NW>
struct BwdChainSmem {
    static constexpr int K = 0, Q = C * DK * 2, T = 2 * C * DK * 2, PM = T + C * C * 2;
    static constexpr int V = PM + C * C * 2, VB = 32 * NW;
    static constexpr int F = V + C * VB, STAGE = F + 1024;
    static constexpr int BYTES = 2 * STAGE;
    static_assert(VB == 128 || VB == 256, "a row of dO is a tile row");
};

template <int DK, int NW>
__global__ void __launch_bounds__(32 * NW, 1) gdr_bwd_chain_kernel(const GDRArgs p) {
    using L = BwdChainSmem<DK, NW>;
    constexpr int RB = DK * 2, VB = L::VB, NT = DK / 8, DVT = 16 * NW, NTH = 32 * NW;
    extern __shared__ __align__(1024) unsigned char sm[];
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int gq = lane >> 2, tq = lane & 3;
    const int tiles = p.headdim / DVT;
    const int64_t bh = blockIdx.x / tiles;
    const int p0 = (int)(blockIdx.x % tiles) * DVT;
    const int64_t b = bh / p.nheads, h = bh - b * p.nheads;
    const int64_t kstride = p.ngroups * DK * 2, vstride = p.nheads * p.headdim * 2;
    const unsigned char* kg = static_cast<const unsigned char*>(p.k) + b * p.seqlen * kstride + h / (p.nheads / p.ngroups) * DK * 2;
    const unsigned char* qg = static_cast<const unsigned char*>(p.q) + b * p.seqlen * kstride + h / (p.nheads / p.ngroups) * DK * 2;
    const int64_t voff = b * p.seqlen * vstride + (h * p.headdim + p0) * 2;
    const unsigned char* og = static_cast<const unsigned char*>(p.dout) + voff;

    auto issue = [&](int64_t ch) {
        unsigned char* st = sm + (ch & 1) * L::STAGE;
        const int64_t t0 = ch * C;
        const int valid = (int)(p.seqlen - t0 < C ? p.seqlen - t0 : C);
        const unsigned char* rg = static_cast<const unsigned char*>(p.rec) + (bh * p.nchunks + ch) * REC_BYTES;
        load_tile<RB, C>(st + L::K, kg + t0 * kstride, kstride, valid, tid, NTH);
        load_tile<RB, C>(st + L::Q, qg + t0 * kstride, kstride, valid, tid, NTH);
        load_tile<128, C>(st + L::T, rg + REC_T, 128, C, tid, NTH);
        load_tile<128, C>(st + L::PM, rg + REC_P, 128, C, tid, NTH);
        load_tile<VB, C>(st + L::V, og + t0 * vstride, vstride, valid, tid, NTH);
        if (tid < 48) cp_async_16(st + L::F + tid * 16, rg + REC_F + tid * 16, 16);
        cp_async_commit();
    };

    const int64_t prow = bh * p.headdim + p0 + 16 * w + gq;
    float s[NT][4];                          // dS^T of this warp's rows p
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float2 x = f2(0.0f, 0.0f), y = x;
        if (p.dhT) {
            x = *reinterpret_cast<const float2*>(p.dhT + prow * DK + 8 * n + 2 * tq);
            y = *reinterpret_cast<const float2*>(p.dhT + (prow + 8) * DK + 8 * n + 2 * tq);
        }
        s[n][0] = x.x; s[n][1] = x.y; s[n][2] = y.x; s[n][3] = y.y;
    }
    issue(p.nchunks - 1);
    for (int64_t ch = p.nchunks - 1; ch >= 0; --ch) {
        cp_async_wait<0>();
        __syncthreads();
        if (ch > 0) issue(ch - 1);
        unsigned char* st = sm + (ch & 1) * L::STAGE;
        const uint32_t ks = smem_u32(st + L::K), qs = smem_u32(st + L::Q), ts = smem_u32(st + L::T),
                       ps = smem_u32(st + L::PM), vs = smem_u32(st + L::V);
        const float* eg = reinterpret_cast<const float*>(st + L::F);
        const int64_t rec = bh * p.nchunks + ch;

        bf16* sv = static_cast<bf16*>(p.dstates) + (rec * p.headdim + p0 + 16 * w + gq) * DK + 2 * tq;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            *reinterpret_cast<uint32_t*>(sv + 8 * n) = pack_bf16x2(s[n][0], s[n][1]);
            *reinterpret_cast<uint32_t*>(sv + 8 * DK + 8 * n) = pack_bf16x2(s[n][2], s[n][3]);
        }
        // x = tail (dS' k) + do Pm
        float x[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[n][e] = 0.0f;
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt) {
            uint32_t a[4];
            acc_to_a<NT>(s, kt, a);
#pragma unroll
            for (int n = 0; n < 8; n += 2) {
                uint32_t f[4];
                load_b_nk<RB>(ks, 8 * n, 2 * kt, lane, f);
                mma(x[n], a, f[0], f[1]);
                mma(x[n + 1], a, f[2], f[3]);
            }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 t = *reinterpret_cast<const float2*>(eg + C + 8 * n + 2 * tq);
            x[n][0] *= t.x; x[n][1] *= t.y; x[n][2] *= t.x; x[n][3] *= t.y;
        }
        uint32_t dof[4][4];
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            load_a_km<VB>(vs, 16 * kt, 2 * w, lane, dof[kt]);
#pragma unroll
            for (int n = 0; n <= 2 * kt; n += 2) {
                uint32_t f[4];
                load_b_kn<128>(ps, 16 * kt, n, lane, f);
                mma(x[n], dof[kt], f[0], f[1]);
                mma(x[n + 1], dof[kt], f[2], f[3]);
            }
        }
        // r = x T
        float r[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) r[n][e] = 0.0f;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t a[4];
            acc_to_a<8>(x, kt, a);
#pragma unroll
            for (int n = 0; n <= 2 * kt; n += 2) {
                uint32_t f[4];
                load_b_kn<128>(ts, 16 * kt, n, lane, f);
                mma(r[n], a, f[0], f[1]);
                mma(r[n + 1], a, f[2], f[3]);
            }
        }
        bf16* rv = static_cast<bf16*>(p.dr) + (rec * p.headdim + p0 + 16 * w + gq) * C + 2 * tq;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            *reinterpret_cast<uint32_t*>(rv + 8 * n) = pack_bf16x2(r[n][0], r[n][1]);
            *reinterpret_cast<uint32_t*>(rv + 8 * C + 8 * n) = pack_bf16x2(r[n][2], r[n][3]);
        }
        // dS <- e^(c_last) dS' + (scale e^c do) q - (beta e^c r) k
        const float last = eg[C - 1];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] *= last;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            const float2 e0 = *reinterpret_cast<const float2*>(eg + 16 * kt + 2 * tq);
            const float2 e1 = *reinterpret_cast<const float2*>(eg + 16 * kt + 8 + 2 * tq);
            uint32_t a[4];
            a[0] = pack_bf16x2(bf16_lo(dof[kt][0]) * (e0.x * p.scale), bf16_hi(dof[kt][0]) * (e0.y * p.scale));
            a[1] = pack_bf16x2(bf16_lo(dof[kt][1]) * (e0.x * p.scale), bf16_hi(dof[kt][1]) * (e0.y * p.scale));
            a[2] = pack_bf16x2(bf16_lo(dof[kt][2]) * (e1.x * p.scale), bf16_hi(dof[kt][2]) * (e1.y * p.scale));
            a[3] = pack_bf16x2(bf16_lo(dof[kt][3]) * (e1.x * p.scale), bf16_hi(dof[kt][3]) * (e1.y * p.scale));
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t f[4];
                load_b_kn<RB>(qs, 16 * kt, n, lane, f);
                mma(s[n], a, f[0], f[1]);
                mma(s[n + 1], a, f[2], f[3]);
            }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 be = *reinterpret_cast<const float2*>(eg + 2 * C + 8 * n + 2 * tq);
            r[n][0] *= be.x; r[n][1] *= be.y; r[n][2] *= be.x; r[n][3] *= be.y;      // dv
        }
        // dv through the warp's own columns of dO's tile (read above) to memory
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
            const int m = lane >> 3;
            stsm4t(vs + tile_off<VB>(8 * n + (m >> 1) * 8 + (lane & 7), 2 * w + (m & 1)), pack_bf16x2(r[n][0], r[n][1]),
                   pack_bf16x2(r[n][2], r[n][3]), pack_bf16x2(r[n + 1][0], r[n + 1][1]), pack_bf16x2(r[n + 1][2], r[n + 1][3]));
        }
        __syncwarp();
        const int valid = (int)(p.seqlen - ch * C < C ? p.seqlen - ch * C : C);
        unsigned char* dvg = static_cast<unsigned char*>(p.dv) + voff + ch * C * vstride + 32 * w;
#pragma unroll
        for (int i = lane; i < 2 * C; i += 32) {
            const int row = i >> 1, c = i & 1;
            if (row < valid)
                *reinterpret_cast<uint4*>(dvg + row * vstride + c * 16) =
                    *reinterpret_cast<const uint4*>(st + L::V + tile_off<VB>(row, 2 * w + c));
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 e = *reinterpret_cast<const float2*>(eg + 8 * n + 2 * tq);
            r[n][0] *= -e.x; r[n][1] *= -e.y; r[n][2] *= -e.x; r[n][3] *= -e.y;
        }
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t a[4];
            acc_to_a<8>(r, kt, a);
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t f[4];
                load_b_kn<RB>(ks, 16 * kt, n, lane, f);
                mma(s[n], a, f[0], f[1]);
                mma(s[n + 1], a, f[2], f[3]);
            }
        }
    }
    if (p.dh0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            *reinterpret_cast<float2*>(p.dh0 + prow * DK + 8 * n + 2 * tq) = f2(s[n][0], s[n][1]);
            *reinterpret_cast<float2*>(p.dh0 + (prow + 8) * DK + 8 * n + 2 * tq) = f2(s[n][2], s[n][3]);
        }
    }
}

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
    constexpr int RB = DK * 2, VB = DV * 2, NTC = DK / 16;
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
        load_tile<VB, C>(sm + L::DO, static_cast<const unsigned char*>(p.dout) + voff, vstride, valid, tid, 256);
        load_tile<128, DV>(sm + L::U, static_cast<const unsigned char*>(p.u) + rec * DV * C * 2, C * 2, DV, tid, 256);
        load_tile<128, DV>(sm + L::R, static_cast<const unsigned char*>(p.dr) + rec * DV * C * 2, C * 2, DV, tid, 256);
        if (tid < 48) cp_async_16(sm + L::F + tid * 16, rg + REC_F + tid * 16, 16);
        cp_async_commit();
        load_tile<RB, DV>(sm + L::S, static_cast<const unsigned char*>(p.states) + rec * DV * RB, RB, DV, tid, 256);
        load_tile<RB, DV>(sm + L::DS, static_cast<const unsigned char*>(p.dstates) + rec * DV * RB, RB, DV, tid, 256);
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
            load_a_mk<VB>(dos, 16 * mi, 2 * kt, lane, ao);
            load_a_km<128>(rs, 16 * kt, 2 * mi, lane, ar);
#pragma unroll
            for (int n = 0; n < 4; n += 2) {
                if (4 * hf + n > 2 * mi + 1) break;
                uint32_t f[4];
                load_b_kn<128>(us, 16 * kt, 4 * hf + n, lane, f);
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
                const bf16* vg = static_cast<const bf16*>(p.v) + voff / 2 + i * (vstride / 2);
#pragma unroll 4
                for (int c = part * (DV / 4); c < (part + 1) * (DV / 4); c += 4) {
                    const float4 vv = load4(vg + c);
                    const unsigned char* rr = sm + L::R + (i & 7) * 2;
                    d = fmaf(vv.x, load1(reinterpret_cast<const bf16*>(rr + tile_off<128>(c, i >> 3))), d);
                    d = fmaf(vv.y, load1(reinterpret_cast<const bf16*>(rr + tile_off<128>(c + 1, i >> 3))), d);
                    d = fmaf(vv.z, load1(reinterpret_cast<const bf16*>(rr + tile_off<128>(c + 2, i >> 3))), d);
                    d = fmaf(vv.w, load1(reinterpret_cast<const bf16*>(rr + tile_off<128>(c + 3, i >> 3))), d);
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
            product<NTC, DV / 16, false, VB, RB>(acc, dos, ss, mi, nc0, 0, 15, lane);
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
            product<NTC, DV / 16, true, 128, RB>(acc, rs, ss, mi, nc0, 0, 15, lane);
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
            product<NTC, DV / 16, true, 128, RB>(acc, us, dss, mi, nc0, 0, 15, lane);
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

template <int DK, int NW>
cudaError_t launch_bwd_chain(const GDRArgs& a, cudaStream_t s) {
    constexpr int bytes = BwdChainSmem<DK, NW>::BYTES;
    cudaError_t e = cudaFuncSetAttribute(gdr_bwd_chain_kernel<DK, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    gdr_bwd_chain_kernel<DK, NW><<<(unsigned)(a.batch * a.nheads * (a.headdim / (16 * NW))), 32 * NW, bytes, s>>>(a);
    return cudaGetLastError();
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
    const bool wide = a.headdim == 128 && a.batch * a.nheads * 2 > 148;
    cudaError_t e = wide ? launch_bwd_chain<DK, 8>(a, s) : launch_bwd_chain<DK, 4>(a, s);
    if (e != cudaSuccess) return e;
    return a.headdim == 64 ? launch_grad<DK, 64>(a, s) : launch_grad<DK, 128>(a, s);
}

}  // namespace gdr

cudaError_t launch_gdr_bwd(const GDRArgs& a, cudaStream_t s) {
    return a.dstate == 64 ? gdr::launch_bwd<64>(a, s) : gdr::launch_bwd<128>(a, s);
}

}  // namespace mmscan
