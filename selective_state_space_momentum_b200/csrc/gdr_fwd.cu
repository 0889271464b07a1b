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
// masked q.k of every chunk (what does not depend on the state);
// gdr_chain_kernel (gdr_chain.cu) walks the chunks in order.
//
// Precision: the state is fp32.  Where it enters a product it is split in two
// bf16 terms (hi + lo, 2^-16), and so are v - e^c S k, T and e^c u; k, q, v are bf16
// already.  The outputs o are rounded to bf16 anyway (2^-8), so the products
// that reach only o take the hi terms of u alone.
#include <cuda.h>

#include "gdr_common.cuh"

namespace mmscan {

static __device__ unsigned int g_prep_dev_err = 0;

namespace gdr {
namespace {

// ---------------------------------------------- the chunks' own matrices ----
// One CTA of four warps takes a chunk of up to four heads that share q and k
// (their products are formed once); warp w holds rows 16 w .. 16 w + 15.
//
// T = (I + A)^-1, in 16 x 16 blocks: T_ww by substitution in fp32, a lane a
// column; below the diagonal T_ij = -T_ii sum_{j<=m<i} A_im T_mj, warp j its
// block column j, on the tensor cores with every operand split in two bf16
// terms.  This is forward substitution by blocks, so it is as stable as the
// substitution is, whatever the size of A (a product of powers of A would not
// be: their entries grow and cancel).
//
// Bound: latency of the dependent steps (loads, k.k, substitution, three block
// rows, the barriers between them) and instruction issue (a third to half of
// the slots), hidden by four CTAs an SM.  Measured, 128 states: 8192 chunks of
// 32 heads that share one group 72 us (2.9 TB/s of records written), 2048
// chunks with q and k of their own 37 us.  A head a CTA: 119 us for the first;
// the last head's store overlapped with the next one's A (Pm formed after it,
// its decays a second time): 78.
constexpr int MAXH = 4;                                      // heads of a CTA, at most
struct PrepSmem {
    // K and Q (2 C DK bf16 from 0 on) until the products are formed, then:
    static constexpr int AH = 0, AL = 8192, PM = 16384, TH = 24576, TL = 32768;
    static constexpr int DIAG = 40960, DP = 20;              // per warp: 16 x DP floats, column i of its diagonal block of A
    static constexpr int CUM = DIAG + 4 * 16 * DP * 4;       // per head: double c[C], then float ef, ff, beta [C]
    static constexpr int HEAD = C * 8 + 3 * C * 4;
    static constexpr int WIDE = CUM + MAXH * HEAD, BAR = WIDE + 16, BYTES = BAR + 8;
};

template <int DK>
__global__ void __launch_bounds__(128, 4) gdr_prep_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                                                       const GDRArgs p, const int nh) {
    using L = PrepSmem;
    constexpr int RB = DK * 2;
    extern __shared__ __align__(1024) unsigned char sm[];
    int* wide = reinterpret_cast<int*>(sm + L::WIDE);
    const int tid = threadIdx.x, lane = tid & 31, w = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int gq = lane >> 2, tq = lane & 3;
    const int hsets = (int)p.nheads / nh;
    const int64_t bs = blockIdx.x / p.nchunks, ch = blockIdx.x - bs * p.nchunks;
    const int64_t b = bs / hsets;
    const int h0 = (int)(bs - b * hsets) * nh;               // heads h0 .. h0 + nh - 1, of one group
    const int64_t t0 = ch * C;
    const int valid = (int)(p.seqlen - t0 < C ? p.seqlen - t0 : C);
    const uint32_t base = smem_u32(sm), qs = base + C * RB, bar = base + L::BAR;
    auto record = [&](int hh) { return (b * p.nheads + h0 + hh) * p.nchunks + ch; };
    if (tid == 0) {
        mbar_init(bar, 1);
        fence_barrier_init();
        const int grp = h0 / (int)(p.nheads / p.ngroups);
        if (p.stall != 1) {                                  // (test only: nothing staged, the wait runs out)
            mbar_expect_tx(bar, 2 * C * RB);
#pragma unroll
            for (int s = 0; s < DK / 64; ++s) {
                tma_load_4d(base + s * C * 128, &tm_k, bar, 64 * s, grp, (int)t0, (int)b);
                tma_load_4d(qs + s * C * 128, &tm_q, bar, 64 * s, grp, (int)t0, (int)b);
            }
        }
    }
    if (w < nh) {                                            // the decays of head w
        double* cum = reinterpret_cast<double*>(sm + L::CUM + w * L::HEAD);
        float* ef = reinterpret_cast<float*>(cum + C);
        float* fout = reinterpret_cast<float*>(static_cast<unsigned char*>(p.rec) + record(w) * REC_BYTES + REC_F);
        const int64_t gh = (b * p.seqlen + t0) * p.nheads + h0 + w;
        const int r = 2 * lane;
        float2 be = f2(0.0f, 0.0f);
        if (r < valid) be.x = __bfloat162float(static_cast<const bf16*>(p.beta)[gh + r * p.nheads]);
        if (r + 1 < valid) be.y = __bfloat162float(static_cast<const bf16*>(p.beta)[gh + (r + 1) * p.nheads]);
        double s0, s1, last;
        chunk_cumsum(static_cast<const bf16*>(p.g) + gh, p.nheads, valid, lane, s0, s1, last);
        cum[r] = s0;
        cum[r + 1] = s1;
        // e^(c_i - c_j) as the product of e^(c_i - mid) and e^(mid - c_j), where
        // neither can leave fp32's range (2^60 either way); else by element
        const double first = __shfl_sync(0xffffffffu, s0, 0), mid = 0.5 * (first + last);
        const double a0 = (s0 - mid) * kLog2e, a1 = (s1 - mid) * kLog2e;
        const bool far = __any_sync(0xffffffffu, !(fabs(a0) < 60.0) || !(fabs(a1) < 60.0));
        *reinterpret_cast<float2*>(ef + r) = far ? f2(1.0f, 1.0f) : f2(ex2_approx((float)a0), ex2_approx((float)a1));
        *reinterpret_cast<float2*>(ef + C + r) = far ? f2(1.0f, 1.0f) : f2(ex2_approx((float)-a0), ex2_approx((float)-a1));
        *reinterpret_cast<float2*>(ef + 2 * C + r) = be;
        if (lane == 0) wide[w] = far;
        *reinterpret_cast<float2*>(fout + r) = f2(ex2_approx((float)(s0 * kLog2e)), ex2_approx((float)(s1 * kLog2e)));
        *reinterpret_cast<float2*>(fout + C + r) =
            f2(ex2_approx((float)((last - s0) * kLog2e)), ex2_approx((float)((last - s1) * kLog2e)));
        *reinterpret_cast<float2*>(fout + 2 * C + r) = be;
    }
    __syncthreads();
    if (!__syncthreads_and(mbar_wait_sleep(bar, 0, &g_prep_dev_err))) {
        if (tid == 0 && p.stall != 1) drain(bar, 0, &g_prep_dev_err);   // (the copies, if they were issued)
        return;
    }

    // k.k and q.k, n-tiles up to the diagonal
    float kk[8][4], qk[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) kk[n][e] = qk[n][e] = 0.0f;
#pragma unroll
    for (int kt = 0; kt < DK / 16; ++kt) {
        const uint32_t slab = (kt >> 2) * C * 128;
        uint32_t ak[4], aq[4];
        load_a_mk<128>(base + slab, 16 * w, 2 * (kt & 3), lane, ak);
        load_a_mk<128>(qs + slab, 16 * w, 2 * (kt & 3), lane, aq);
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
            if (n > 2 * w + 1) break;
            uint32_t bk[4];
            load_b_nk<128>(base + slab, 8 * n, 2 * (kt & 3), lane, bk);
            mma(kk[n], ak, bk[0], bk[1]);
            mma(kk[n + 1], ak, bk[2], bk[3]);
            mma(qk[n], aq, bk[0], bk[1]);
            mma(qk[n + 1], aq, bk[2], bk[3]);
        }
    }
    __syncthreads();                                         // K and Q give way to A, Pm and T
    const int i0 = 16 * w + gq;
    float* diag = reinterpret_cast<float*>(sm + L::DIAG) + w * 16 * L::DP;
    // the tiles are stored whole; T and Pm are zero above the diagonal blocks
    for (int i = tid; i < 3 * C * 8; i += 128) {
        const int r = (i >> 3) & 63, c = i & 7;
        if (c / 2 > r / 16) *reinterpret_cast<uint4*>(sm + L::PM + (i >> 9) * 8192 + tile_off<128>(r, c)) = make_uint4(0, 0, 0, 0);
    }
#pragma unroll 1
    for (int hh = 0; hh < nh; ++hh) {
        const double* cum = reinterpret_cast<const double*>(sm + L::CUM + hh * L::HEAD);
        const float* ef = reinterpret_cast<const float*>(cum + C);
        const float be[2] = {ef[2 * C + i0], ef[2 * C + i0 + 8]};
        const float ei[2] = {ef[i0], ef[i0 + 8]};
        const bool apart = wide[hh] != 0;                    // decays by element (the factors are ones then)
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            if (n > 2 * w + 1) break;
            const int j = 8 * n + 2 * tq;
            const float2 fj = *reinterpret_cast<const float2*>(ef + C + j);
            float d[4] = {ei[0] * fj.x, ei[0] * fj.y, ei[1] * fj.x, ei[1] * fj.y};
            if (apart) {
#pragma unroll 1
                for (int e = 0; e < 4; ++e) {
                    const int i = i0 + 8 * (e >> 1), jj = j + (e & 1);
                    const float x = jj <= i ? ex2_approx((float)((cum[i] - cum[jj]) * kLog2e)) : 0.0f;
                    d[0] = e == 0 ? x : d[0];
                    d[1] = e == 1 ? x : d[1];
                    d[2] = e == 2 ? x : d[2];
                    d[3] = e == 3 ? x : d[3];
                }
            }
            float av[4], pv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = i0 + 8 * (e >> 1), jj = j + (e & 1);
                pv[e] = jj <= i ? p.scale * qk[n][e] * d[e] : 0.0f;
                av[e] = jj < i ? be[e >> 1] * kk[n][e] * d[e] : 0.0f;
            }
            const uint32_t o0 = tile_off<128>(i0, n) + 4 * tq, o1 = tile_off<128>(i0 + 8, n) + 4 * tq;
            *reinterpret_cast<uint32_t*>(sm + L::PM + o0) = pack_bf16x2(pv[0], pv[1]);
            *reinterpret_cast<uint32_t*>(sm + L::PM + o1) = pack_bf16x2(pv[2], pv[3]);
            if (n >= 2 * w) {                                // the diagonal block, by columns
#pragma unroll
                for (int e = 0; e < 4; ++e) diag[(j + (e & 1) - 16 * w) * L::DP + gq + 8 * (e >> 1)] = av[e];
            } else {
                uint32_t hi[2], lo[2];
                split2(av[0], av[1], hi[0], lo[0]);
                split2(av[2], av[3], hi[1], lo[1]);
                *reinterpret_cast<uint32_t*>(sm + L::AH + o0) = hi[0];
                *reinterpret_cast<uint32_t*>(sm + L::AH + o1) = hi[1];
                *reinterpret_cast<uint32_t*>(sm + L::AL + o0) = lo[0];
                *reinterpret_cast<uint32_t*>(sm + L::AL + o1) = lo[1];
            }
        }
        __syncwarp();
        if (lane < 16) {                                     // T_ww, column `lane`
            float t[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) t[i] = i == lane ? 1.0f : 0.0f;
#pragma unroll
            for (int i = 0; i < 15; ++i) {
                float a[16];
#pragma unroll
                for (int q = (i + 1) / 4; q < 4; ++q)
                    *reinterpret_cast<float4*>(a + 4 * q) = *reinterpret_cast<const float4*>(diag + i * L::DP + 4 * q);
#pragma unroll
                for (int r = i + 1; r < 16; ++r) t[r] = fmaf(-a[r], t[i], t[r]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bf16 hi = __float2bfloat16_rn(t[i]);
                const uint32_t off = tile_off<128>(16 * w + i, 2 * w + (lane >> 3)) + 2 * (lane & 7);
                *reinterpret_cast<bf16*>(sm + L::TH + off) = hi;
                *reinterpret_cast<bf16*>(sm + L::TL + off) = __float2bfloat16_rn(t[i] - __bfloat162float(hi));
            }
        }
        __syncthreads();
        // block column w: X = T_iw^T (16 columns w x 16 rows i) as the A operand
        if (w < 3) {
            uint32_t xh[3][4], xl[3][4];
            load_a_km<128>(base + L::TH, 16 * w, 2 * w, lane, xh[0]);
            load_a_km<128>(base + L::TL, 16 * w, 2 * w, lane, xl[0]);
#pragma unroll
            for (int d = 1; d < 4; ++d) {
                const int i = w + d;
                if (i > 3) break;
                float acc[2][4], tr[2][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[0][e] = acc[1][e] = tr[0][e] = tr[1][e] = 0.0f;
#pragma unroll
                for (int m = 0; m < d; ++m) {
                    uint32_t fh[4], fl[4];
                    load_b_nk<128>(base + L::AH, 16 * i, 2 * (w + m), lane, fh);
                    load_b_nk<128>(base + L::AL, 16 * i, 2 * (w + m), lane, fl);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        mma(acc[t], xh[m], fh[2 * t], fh[2 * t + 1]);
                        mma(acc[t], xl[m], fh[2 * t], fh[2 * t + 1]);
                        mma(acc[t], xh[m], fl[2 * t], fl[2 * t + 1]);
                    }
                }
                uint32_t sh[4], sl[4], fh[4], fl[4];
                acc_to_a2<2>(acc, 0, sh, sl);
                load_b_nk<128>(base + L::TH, 16 * i, 2 * i, lane, fh);
                load_b_nk<128>(base + L::TL, 16 * i, 2 * i, lane, fl);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    mma(tr[t], sh, fh[2 * t], fh[2 * t + 1]);
                    mma(tr[t], sl, fh[2 * t], fh[2 * t + 1]);
                    mma(tr[t], sh, fl[2 * t], fl[2 * t + 1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) tr[t][e] = -tr[t][e];
                }
                acc_to_a2<2>(tr, 0, sh, sl);
                store_a_km<128>(base + L::TH, 16 * i, 2 * w, lane, sh);
                store_a_km<128>(base + L::TL, 16 * i, 2 * w, lane, sl);
                if (d < 3)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        xh[d][e] = sh[e];
                        xl[d][e] = sl[e];
                    }
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
        if (tid == 0) {                                      // the tiles as they are, and then they may be written again
            unsigned char* out = static_cast<unsigned char*>(p.rec) + record(hh) * REC_BYTES;
            bulk_store(out + REC_T, base + L::TH, C * C * 2);
            bulk_store(out + REC_P, base + L::PM, C * C * 2);
            bulk_store(static_cast<unsigned char*>(p.tlo) + record(hh) * (C * C * 2), base + L::TL, C * C * 2);
            bulk_commit_group();
            bulk_wait_read_all();
        }
        __syncthreads();
    }
    if (tid == 0) bulk_wait_all();                           // complete before the CTA exits
}

unsigned int read_and_clear_prep_error() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_prep_dev_err, sizeof(v)) != cudaSuccess) return 0;
    if (v) cudaMemcpyToSymbol(g_prep_dev_err, &z, sizeof(z));
    return v;
}

[[maybe_unused]] const bool g_registered = (register_error_reader(read_and_clear_prep_error), true);

// Heads of a CTA: as many as share q and k, up to MAXH, while the CTAs still
// fill the GPU's four an SM twice over.
int prep_heads(const GDRArgs& a) {
    const int64_t per_group = a.nheads / a.ngroups, chunks = a.batch * a.nheads * a.nchunks;
    for (int nh = MAXH; nh > 1; nh /= 2)
        if (per_group % nh == 0 && chunks / nh >= 2 * 4 * 148) return nh;
    return 1;
}

template <int DK>
cudaError_t launch_fwd(const GDRArgs& a, cudaStream_t s) {
    CallMaps m;
    cudaError_t e;
    if ((e = map_call(&m, a, a.v)) != cudaSuccess) return e;
    constexpr int bytes = PrepSmem::BYTES;
    static std::atomic<uint64_t> attr_done{0};
    if ((e = allow_dynamic_smem(reinterpret_cast<const void*>(gdr_prep_kernel<DK>), bytes, attr_done)) != cudaSuccess) return e;
    const int nh = prep_heads(a);
    gdr_prep_kernel<DK><<<(unsigned)(a.batch * (a.nheads / nh) * a.nchunks), 128, bytes, s>>>(m.k, m.q, a, nh);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_gdr_chain(a, false, m, s);
}

}  // namespace
}  // namespace gdr

bool gdr_shape_supported(int64_t headdim, int64_t dstate) {
    return (headdim == 64 || headdim == 128) && (dstate == 64 || dstate == 128);
}

cudaError_t launch_gdr_fwd(const GDRArgs& a, cudaStream_t s) {
    return a.dstate == 64 ? gdr::launch_fwd<64>(a, s) : gdr::launch_fwd<128>(a, s);
}

}  // namespace mmscan
