// gdr_fwd.cu -- sm_100a kernels for the gated delta rule over a sequence, in
// the chunked form, forward.
//
// What it computes, per batch row and head, with state S (P, N):
//     S_t = e^(g_t) S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,  o_t = scale S_t q_t
// Over a chunk of 64 steps starting from S, with c the cumulative g:
//     A_ij = beta_i e^(c_i - c_j) k_i.k_j (j < i),   T = (I + A)^-1
//     u_i  = sum_j T_ij beta_j (v_j - e^(c_j) S k_j)          (the rows written)
//     o_i  = scale (e^(c_i) S q_i + sum_{j<=i} e^(c_i - c_j) (q_i.k_j) u_j)
//     S'   = e^(c_last) S + sum_j e^(c_last - c_j) u_j k_j^T
//
// Two launches.  gdr_prep_kernel, parallel over chunks, forms T and the
// masked q.k of every chunk (what does not depend on the state).
// gdr_chain_kernel walks the chunks in order, one warp per 16 rows p of the
// state: S^T lives in the warp's registers as fp32 accumulators, and since
// the columns of the accumulators of one product are the A operand of the
// next, S -> S k -> u -> S' needs no shared memory and no barrier between the
// products; the rows p never meet.
//
// Precision: the state is fp32.  Where it enters a product it is split in two
// bf16 terms (hi + lo, 2^-17), and so are v - e^c S k, T and e^c u; k, q, v are bf16
// already.  The outputs o are rounded to bf16 anyway (2^-9), so the products
// that reach only o take the hi terms alone.
#include "gdr_common.cuh"

namespace mmscan {

namespace gdr {

constexpr int PITCH = 68;                  // floats of a row of A and T in shared memory

template <int DK>
constexpr int prep_smem() { return 2 * C * DK * 2 + 2 * C * PITCH * 4 + C * 8 + C * 4; }

// c = a + b * (-1): rows [r0, r0 + n) etc. of T <- -(X . Y), used by the
// block inverse below; each of `nt` threads forms EW neighbouring outputs.
template <int DIM, int EW>
__device__ __forceinline__ void block_product(float* out, const float* X, const float* Y, float sign, int t) {
    const int r = t / (DIM / EW), c = (t % (DIM / EW)) * EW;
    float acc[EW];
#pragma unroll
    for (int e = 0; e < EW; ++e) acc[e] = 0.0f;
#pragma unroll 8
    for (int k = 0; k < DIM; ++k) {
        const float x = X[r * PITCH + k];
#pragma unroll
        for (int e = 0; e < EW; e += 4) {
            const float4 y = *reinterpret_cast<const float4*>(Y + k * PITCH + c + e);
            acc[e] = fmaf(x, y.x, acc[e]);
            acc[e + 1] = fmaf(x, y.y, acc[e + 1]);
            acc[e + 2] = fmaf(x, y.z, acc[e + 2]);
            acc[e + 3] = fmaf(x, y.w, acc[e + 3]);
        }
    }
#pragma unroll
    for (int e = 0; e < EW; e += 4)
        *reinterpret_cast<float4*>(out + r * PITCH + c + e) =
            make_float4(sign * acc[e], sign * acc[e + 1], sign * acc[e + 2], sign * acc[e + 3]);
}

template <int DK>
__global__ void __launch_bounds__(128) gdr_prep_kernel(const GDRArgs p) {
    constexpr int RB = DK * 2;
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char* Kt = sm;
    unsigned char* Qt = sm + C * RB;
    float* A = reinterpret_cast<float*>(sm + 2 * C * RB);
    float* T = A + C * PITCH;
    double* cum = reinterpret_cast<double*>(T + C * PITCH);
    float* beta = reinterpret_cast<float*>(cum + C);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int64_t rec = blockIdx.x;                        // (b, h, chunk)
    const int64_t bh = rec / p.nchunks, ch = rec - bh * p.nchunks;
    const int64_t b = bh / p.nheads, h = bh - b * p.nheads;
    const int64_t t0 = ch * C;
    const int valid = (int)(p.seqlen - t0 < C ? p.seqlen - t0 : C);
    const int64_t gk = ((b * p.seqlen + t0) * p.ngroups + h / (p.nheads / p.ngroups)) * DK;
    const int64_t kstride = p.ngroups * DK * 2;
    load_tile<RB, C>(Kt, static_cast<const bf16*>(p.k) + gk, kstride, valid, tid, 128);
    load_tile<RB, C>(Qt, static_cast<const bf16*>(p.q) + gk, kstride, valid, tid, 128);
    cp_async_commit();

    unsigned char* out = static_cast<unsigned char*>(p.rec) + rec * REC_BYTES;
    float* fout = reinterpret_cast<float*>(out + REC_F);
    const int64_t gh = (b * p.seqlen + t0) * p.nheads + h;
    if (w == 0) {
        const int r = 2 * lane;
        double s0, s1, last;
        chunk_cumsum(static_cast<const bf16*>(p.g) + gh, p.nheads, valid, lane, s0, s1, last);
        cum[r] = s0;
        cum[r + 1] = s1;
        *reinterpret_cast<float2*>(fout + r) = f2(ex2_approx((float)(s0 * kLog2e)), ex2_approx((float)(s1 * kLog2e)));
        *reinterpret_cast<float2*>(fout + C + r) =
            f2(ex2_approx((float)((last - s0) * kLog2e)), ex2_approx((float)((last - s1) * kLog2e)));
    } else if (w == 1) {
#pragma unroll
        for (int r = lane; r < C; r += 32) {
            const float x = r < valid ? __bfloat162float(static_cast<const bf16*>(p.beta)[gh + r * p.nheads]) : 0.0f;
            beta[r] = x;
            fout[2 * C + r] = x;
        }
    }
    cp_async_wait<0>();
    __syncthreads();

    // k.k and q.k: warp w the rows 16 w .. 16 w + 15, n-tiles up to the diagonal
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[n][e] = qk[n][e] = 0.0f;
    const uint32_t ks = smem_u32(Kt), qs = smem_u32(Qt);
#pragma unroll
    for (int kt = 0; kt < DK / 16; ++kt) {
        uint32_t ak[4], aq[4];
        load_a_mk<RB>(ks, 16 * w, 2 * kt, lane, ak);
        load_a_mk<RB>(qs, 16 * w, 2 * kt, lane, aq);
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
            if (n > 2 * w + 1) break;
            uint32_t bk[4];
            load_b_nk<RB>(ks, 8 * n, 2 * kt, lane, bk);
            mma(kk[n], ak, bk[0], bk[1]);
            mma(kk[n + 1], ak, bk[2], bk[3]);
            mma(qk[n], aq, bk[0], bk[1]);
            mma(qk[n + 1], aq, bk[2], bk[3]);
        }
    }
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int i = 16 * w + gq + 8 * half;
        const double ci = cum[i];
        const float bi = beta[i];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int j = 8 * n + 2 * tq;
            float pv[2], av[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float d = j + e <= i ? ex2_approx((float)((ci - cum[j + e]) * kLog2e)) : 0.0f;
                pv[e] = j + e <= i ? p.scale * qk[n][2 * half + e] * d : 0.0f;
                av[e] = j + e < i ? bi * kk[n][2 * half + e] * d : 0.0f;
            }
            *reinterpret_cast<float2*>(A + i * PITCH + j) = f2(av[0], av[1]);
            *reinterpret_cast<uint32_t*>(out + REC_P + (i * C + j) * 2) = pack_bf16x2(pv[0], pv[1]);
        }
    }
    __syncthreads();

    // T = (I + A)^-1 in fp32: the diagonal 16 x 16 blocks by substitution, a
    // lane a column, then twice the join [[Ta, 0], [-Tb A_ba Ta, Tb]].  Every
    // step is a forward substitution over blocks, as stable as the
    // substitution itself.  The upper blocks of T hold the joins' inner products.
    if (lane < 16) {
        const float* Ab = A + 16 * w * PITCH + 16 * w;
        float t[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == lane ? 1.0f : 0.0f;
#pragma unroll
            for (int m = 0; m < i; ++m) s = fmaf(-Ab[i * PITCH + m], t[m], s);
            t[i] = s;
            T[(16 * w + i) * PITCH + 16 * w + lane] = s;
        }
    }
    __syncthreads();
    {
        const int a = 32 * (tid >> 6), t = tid & 63;       // blocks (a, a) and (a + 16, a + 16)
        block_product<16, 4>(T + a * PITCH + a + 16, A + (a + 16) * PITCH + a, T + a * PITCH + a, 1.0f, t);
        __syncthreads();
        block_product<16, 4>(T + (a + 16) * PITCH + a, T + (a + 16) * PITCH + a + 16, T + a * PITCH + a + 16, -1.0f, t);
        __syncthreads();
        // the scratch blocks inside the 32 x 32 diagonal blocks back to zero
        *reinterpret_cast<float4*>(T + (a + t / 4) * PITCH + a + 16 + 4 * (t & 3)) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        __syncthreads();
        block_product<32, 8>(T + 32, A + 32 * PITCH, T, 1.0f, tid);
        __syncthreads();
        block_product<32, 8>(T + 32 * PITCH, T + 32 * PITCH + 32, T + 32, -1.0f, tid);
        __syncthreads();
    }
    // T in two bf16 terms
    unsigned char* lo_out = static_cast<unsigned char*>(p.tlo) + rec * (C * C * 2);
    const int r = tid >> 1, c0 = 32 * (tid & 1);
#pragma unroll
    for (int c = c0; c < c0 + 32; c += 8) {
        uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
        if (r >= 32 || c < 32) {                             // the block above the diagonal is scratch
            const float* s = T + r * PITCH + c;
            split2(s[0], s[1], hi.x, lo.x);
            split2(s[2], s[3], hi.y, lo.y);
            split2(s[4], s[5], hi.z, lo.z);
            split2(s[6], s[7], hi.w, lo.w);
        }
        *reinterpret_cast<uint4*>(out + REC_T + (r * C + c) * 2) = hi;
        *reinterpret_cast<uint4*>(lo_out + (r * C + c) * 2) = lo;
    }
}

// ------------------------------------------------------------- the chain ----
template <int DK, int NW>
struct ChainSmem {
    static constexpr int K = 0, Q = C * DK * 2, T = 2 * C * DK * 2, TL = T + C * C * 2, PM = TL + C * C * 2;
    static constexpr int V = PM + C * C * 2, VB = 32 * NW;            // bytes of a row of V
    static constexpr int F = V + C * (VB < 128 ? 128 : VB), STAGE = F + 1024;
    static constexpr int BYTES = 2 * STAGE + 1024;
    static_assert(VB == 128 || VB == 256, "a row of V is a tile row");
};

template <int DK, int NW, bool TRAIN>
__global__ void __launch_bounds__(32 * NW, 1) gdr_chain_kernel(const GDRArgs p) {
    using L = ChainSmem<DK, NW>;
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
    const unsigned char* vg = static_cast<const unsigned char*>(p.v) + b * p.seqlen * vstride + (h * p.headdim + p0) * 2;

    auto issue = [&](int64_t ch) {
        unsigned char* st = sm + (ch & 1) * L::STAGE;
        const int64_t t0 = ch * C;
        const int valid = (int)(p.seqlen - t0 < C ? p.seqlen - t0 : C);
        const int64_t rec = bh * p.nchunks + ch;
        const unsigned char* rg = static_cast<const unsigned char*>(p.rec) + rec * REC_BYTES;
        load_tile<RB, C>(st + L::K, kg + t0 * kstride, kstride, valid, tid, NTH);
        load_tile<RB, C>(st + L::Q, qg + t0 * kstride, kstride, valid, tid, NTH);
        load_tile<128, C>(st + L::T, rg + REC_T, 128, C, tid, NTH);
        load_tile<128, C>(st + L::TL, static_cast<const unsigned char*>(p.tlo) + rec * (C * C * 2), 128, C, tid, NTH);
        load_tile<128, C>(st + L::PM, rg + REC_P, 128, C, tid, NTH);
        load_tile<VB, C>(st + L::V, vg + t0 * vstride, vstride, valid, tid, NTH);
        if (tid < 48) cp_async_16(st + L::F + tid * 16, rg + REC_F + tid * 16, 16);
        cp_async_commit();
    };

    // S^T of this warp's rows p: accumulator tile n holds states 8 n .. 8 n + 7
    const int64_t prow = bh * p.headdim + p0 + 16 * w + gq;
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float2 x = f2(0.0f, 0.0f), y = x;
        if (p.h0) {
            x = *reinterpret_cast<const float2*>(p.h0 + prow * DK + 8 * n + 2 * tq);
            y = *reinterpret_cast<const float2*>(p.h0 + (prow + 8) * DK + 8 * n + 2 * tq);
        }
        s[n][0] = x.x; s[n][1] = x.y; s[n][2] = y.x; s[n][3] = y.y;
    }
    issue(0);
    for (int64_t ch = 0; ch < p.nchunks; ++ch) {
        cp_async_wait<0>();
        __syncthreads();                     // this chunk is there, and every warp is done with the other slot
        if (ch + 1 < p.nchunks) issue(ch + 1);
        unsigned char* st = sm + (ch & 1) * L::STAGE;
        const uint32_t ks = smem_u32(st + L::K), qs = smem_u32(st + L::Q), ts = smem_u32(st + L::T),
                       tl = smem_u32(st + L::TL), ps = smem_u32(st + L::PM), vs = smem_u32(st + L::V);
        const float* eg = reinterpret_cast<const float*>(st + L::F);
        const int64_t rec = bh * p.nchunks + ch;

        if constexpr (TRAIN) {               // the state at the chunk's start, for the backward (bf16)
            bf16* sv = static_cast<bf16*>(p.states) + (rec * p.headdim + p0 + 16 * w + gq) * DK + 2 * tq;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                *reinterpret_cast<uint32_t*>(sv + 8 * n) = pack_bf16x2(s[n][0], s[n][1]);
                *reinterpret_cast<uint32_t*>(sv + 8 * DK + 8 * n) = pack_bf16x2(s[n][2], s[n][3]);
            }
        }
        // x = S k (16 rows p x 64 steps), o = S q
        float x[8][4], o[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[n][e] = o[n][e] = 0.0f;
#pragma unroll
        for (int kt = 0; kt < DK / 16; ++kt) {
            uint32_t hi[4], lo[4];
            acc_to_a2<NT>(s, kt, hi, lo);
#pragma unroll
            for (int n = 0; n < 8; n += 2) {
                uint32_t f[4];
                load_b_nk<RB>(ks, 8 * n, 2 * kt, lane, f);
                mma(x[n], hi, f[0], f[1]);
                mma(x[n + 1], hi, f[2], f[3]);
                mma(x[n], lo, f[0], f[1]);
                mma(x[n + 1], lo, f[2], f[3]);
                load_b_nk<RB>(qs, 8 * n, 2 * kt, lane, f);
                mma(o[n], hi, f[0], f[1]);
                mma(o[n + 1], hi, f[2], f[3]);
            }
        }
        // x <- beta (v - e^c x), o <- scale e^c o
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
            uint32_t vv[4];
            const int m = lane >> 3;
            ldsm4t(vs + tile_off<VB>(8 * n + (m >> 1) * 8 + (lane & 7), 2 * w + (m & 1)), vv);
#pragma unroll
            for (int d = 0; d < 2; ++d) {
                const int j = 8 * (n + d) + 2 * tq;
                const float2 e = *reinterpret_cast<const float2*>(eg + j);
                const float2 be = *reinterpret_cast<const float2*>(eg + 2 * C + j);
                float(&xx)[4] = x[n + d];
                xx[0] = be.x * fmaf(-e.x, xx[0], bf16_lo(vv[2 * d]));
                xx[1] = be.y * fmaf(-e.y, xx[1], bf16_hi(vv[2 * d]));
                xx[2] = be.x * fmaf(-e.x, xx[2], bf16_lo(vv[2 * d + 1]));
                xx[3] = be.y * fmaf(-e.y, xx[3], bf16_hi(vv[2 * d + 1]));
                float(&oo)[4] = o[n + d];
                oo[0] *= p.scale * e.x; oo[1] *= p.scale * e.y; oo[2] *= p.scale * e.x; oo[3] *= p.scale * e.y;
            }
        }
        // u = x T^T (T lower triangular: step j reaches rows i >= j)
        float u[8][4];
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) u[n][e] = 0.0f;
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t hi[4], lo[4];
            acc_to_a2<8>(x, kt, hi, lo);
#pragma unroll
            for (int n = 2 * kt; n < 8; n += 2) {
                uint32_t f[4];
                load_b_nk<128>(ts, 8 * n, 2 * kt, lane, f);
                mma(u[n], hi, f[0], f[1]);
                mma(u[n + 1], hi, f[2], f[3]);
                mma(u[n], lo, f[0], f[1]);
                mma(u[n + 1], lo, f[2], f[3]);
                load_b_nk<128>(tl, 8 * n, 2 * kt, lane, f);
                mma(u[n], hi, f[0], f[1]);
                mma(u[n + 1], hi, f[2], f[3]);
            }
        }
        if constexpr (TRAIN) {               // u for the backward, (P, C) bf16
            bf16* uv = static_cast<bf16*>(p.u) + (rec * p.headdim + p0 + 16 * w + gq) * C + 2 * tq;
#pragma unroll
            for (int n = 0; n < 8; ++n) {
                *reinterpret_cast<uint32_t*>(uv + 8 * n) = pack_bf16x2(u[n][0], u[n][1]);
                *reinterpret_cast<uint32_t*>(uv + 8 * C + 8 * n) = pack_bf16x2(u[n][2], u[n][3]);
            }
        }
        // o += u Pm^T
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t a[4];
            acc_to_a<8>(u, kt, a);
#pragma unroll
            for (int n = 2 * kt; n < 8; n += 2) {
                uint32_t f[4];
                load_b_nk<128>(ps, 8 * n, 2 * kt, lane, f);
                mma(o[n], a, f[0], f[1]);
                mma(o[n + 1], a, f[2], f[3]);
            }
        }
        // S <- e^(c_last) S + (tail u) k
        const float last = eg[C - 1];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] *= last;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 tl2 = *reinterpret_cast<const float2*>(eg + C + 8 * n + 2 * tq);
            u[n][0] *= tl2.x; u[n][1] *= tl2.y; u[n][2] *= tl2.x; u[n][3] *= tl2.y;
        }
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
            uint32_t hi[4], lo[4];
            acc_to_a2<8>(u, kt, hi, lo);
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t f[4];
                load_b_kn<RB>(ks, 16 * kt, n, lane, f);
                mma(s[n], hi, f[0], f[1]);
                mma(s[n + 1], hi, f[2], f[3]);
                mma(s[n], lo, f[0], f[1]);
                mma(s[n + 1], lo, f[2], f[3]);
            }
        }
        // o through the warp's own columns of V's tile (read above) to memory
        __syncwarp();
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
            const int m = lane >> 3;
            stsm4t(vs + tile_off<VB>(8 * n + (m >> 1) * 8 + (lane & 7), 2 * w + (m & 1)), pack_bf16x2(o[n][0], o[n][1]),
                   pack_bf16x2(o[n][2], o[n][3]), pack_bf16x2(o[n + 1][0], o[n + 1][1]), pack_bf16x2(o[n + 1][2], o[n + 1][3]));
        }
        __syncwarp();
        const int valid = (int)(p.seqlen - ch * C < C ? p.seqlen - ch * C : C);
        unsigned char* og = static_cast<unsigned char*>(p.o) + (b * p.seqlen + ch * C) * vstride + (h * p.headdim + p0 + 16 * w) * 2;
#pragma unroll
        for (int i = lane; i < 2 * C; i += 32) {
            const int r = i >> 1, c = i & 1;
            if (r < valid)
                *reinterpret_cast<uint4*>(og + r * vstride + c * 16) =
                    *reinterpret_cast<const uint4*>(st + L::V + tile_off<VB>(r, 2 * w + c));
        }
    }
    if (p.hT) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            *reinterpret_cast<float2*>(p.hT + prow * DK + 8 * n + 2 * tq) = f2(s[n][0], s[n][1]);
            *reinterpret_cast<float2*>(p.hT + (prow + 8) * DK + 8 * n + 2 * tq) = f2(s[n][2], s[n][3]);
        }
    }
}

template <int DK, int NW, bool TRAIN>
cudaError_t launch_chain(const GDRArgs& a, cudaStream_t s) {
    constexpr int bytes = ChainSmem<DK, NW>::BYTES;
    cudaError_t e = cudaFuncSetAttribute(gdr_chain_kernel<DK, NW, TRAIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const int64_t blocks = a.batch * a.nheads * (a.headdim / (16 * NW));
    gdr_chain_kernel<DK, NW, TRAIN><<<(unsigned)blocks, 32 * NW, bytes, s>>>(a);
    return cudaGetLastError();
}

template <int DK>
cudaError_t launch_fwd(const GDRArgs& a, cudaStream_t s) {
    constexpr int bytes = prep_smem<DK>();
    cudaError_t e = cudaFuncSetAttribute(gdr_prep_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    gdr_prep_kernel<DK><<<(unsigned)(a.batch * a.nheads * a.nchunks), 128, bytes, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // A warp's products fill a quarter of its scheduler's tensor pipe time
    // alone; two warps a scheduler (NW = 8) pay once the GPU is full.
    const bool wide = a.headdim == 128 && a.batch * a.nheads * 2 > 148;
    if (a.states) return wide ? launch_chain<DK, 8, true>(a, s) : launch_chain<DK, 4, true>(a, s);
    return wide ? launch_chain<DK, 8, false>(a, s) : launch_chain<DK, 4, false>(a, s);
}

}  // namespace gdr

bool gdr_shape_supported(int64_t headdim, int64_t dstate) {
    return (headdim == 64 || headdim == 128) && (dstate == 64 || dstate == 128);
}

cudaError_t launch_gdr_fwd(const GDRArgs& a, cudaStream_t s) {
    return a.dstate == 64 ? gdr::launch_fwd<64>(a, s) : gdr::launch_fwd<128>(a, s);
}

}  // namespace mmscan
