// gdr_step.cu -- sm_100a kernel for one decode step of the gated delta rule.
//
// What it computes, per request b and head h (group g = h / (H / G)), on the
// cached state S (headdim P, dstate N), updated in place:
//     S <- exp(g) S,   u = beta (v - S k),   S <- S + u k^T,   o = scale S q
//
// Bound: HBM, 8 P N bytes of state a head read and written once against 6 P N
// operations; for a few requests, the latency of one pass.  A row S[p, :] is
// independent of the others, so it lives in the registers of LPR lanes for
// the step: two dot products of a row (with k and with q, the second as
// o = scale ((e^g S) q + u (k . q)), so that both are formed in one pass over
// the loaded row and one shuffle reduction serves both).  All arithmetic is
// fp32.  Eight lanes a row (16 above 128 states) and 12 blocks an SM keep 96 KB
// of states in flight.  Measured for 512 requests of 32 heads of 64 x 128: 176 us a
// step in a row (6.1 TB/s; in a graph 175), 187 to 190 with cold caches, 205 right
// behind 256 MB of other writes, which still leave L2 then; 3.2 us for one request
// of 32 heads of 128 x 128.  With 8 blocks an SM (k kept in registers) 184 against
// 175, with loads and stores that stay in the caches 194; behind the writes,
// against 202 with 12 blocks: 216 with 16 (spills), 222 with 8, 242 with 16 lanes
// a row, 294 with 32, 236 with 4.
#include "mm_common.cuh"
#include "mm_internal.h"

namespace mmscan {

namespace {

// LPR lanes hold a row of N <= 4 LPR NV states as NV vectors of four each.
template <typename IO, int LPR, int NV>
__global__ void __launch_bounds__(128, 12) gdr_step_kernel(const GDRStepArgs p) {
    const int lane = threadIdx.x % LPR;
    const int64_t rows = p.batch * p.nheads * p.headdim;
    const int64_t row0 = ((int64_t)blockIdx.x * 128 + threadIdx.x) / LPR;
    const bool active = row0 < rows;
    const int64_t row = active ? row0 : rows - 1;            // idle lanes follow along (shuffles)
    const int64_t bh = row / p.headdim;
    const int64_t b = bh / p.nheads, h = bh - b * p.nheads;
    const int N = p.dstate;
    const int64_t gk = (b * p.ngroups + h / (p.nheads / p.ngroups)) * N;
    const IO* k = static_cast<const IO*>(p.k) + gk;
    const IO* q = static_cast<const IO*>(p.q) + gk;
    float* S = p.h + row * N;

    float4 s[NV];
    float sk = 0.0f, sq = 0.0f, kq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int n = (lane + i * LPR) * 4;
        s[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (n < N) s[i] = __ldcs(reinterpret_cast<const float4*>(S + n));
    }
    const float a = ex2_approx(load1(static_cast<const IO*>(p.g) + bh) * kLog2e);
    const float beta = load1(static_cast<const IO*>(p.beta) + bh);
    const float v = load1(static_cast<const IO*>(p.v) + row);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int n = (lane + i * LPR) * 4;
        if (n >= N) continue;
        const float4 kk = load4(k + n);
        const float4 qq = load4(q + n);
        s[i].x *= a; s[i].y *= a; s[i].z *= a; s[i].w *= a;
        sk = fmaf(s[i].x, kk.x, fmaf(s[i].y, kk.y, fmaf(s[i].z, kk.z, fmaf(s[i].w, kk.w, sk))));
        sq = fmaf(s[i].x, qq.x, fmaf(s[i].y, qq.y, fmaf(s[i].z, qq.z, fmaf(s[i].w, qq.w, sq))));
        kq = fmaf(kk.x, qq.x, fmaf(kk.y, qq.y, fmaf(kk.z, qq.z, fmaf(kk.w, qq.w, kq))));
    }
#pragma unroll
    for (int m = LPR / 2; m >= 1; m >>= 1) {
        sk += __shfl_xor_sync(0xffffffffu, sk, m);
        sq += __shfl_xor_sync(0xffffffffu, sq, m);
        kq += __shfl_xor_sync(0xffffffffu, kq, m);
    }
    const float u = beta * (v - sk);
    if (!active) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int n = (lane + i * LPR) * 4;
        if (n >= N) continue;
        const float4 kk = load4(k + n);                      // (again, from L1: kept, its registers cost four blocks an SM)
        __stcs(reinterpret_cast<float4*>(S + n),
               make_float4(fmaf(u, kk.x, s[i].x), fmaf(u, kk.y, s[i].y), fmaf(u, kk.z, s[i].z),
                           fmaf(u, kk.w, s[i].w)));
    }
    if (lane == 0) store1(static_cast<IO*>(p.o) + row, p.scale * fmaf(u, kq, sq));
}

template <typename IO, int LPR, int NV>
cudaError_t launch_step(const GDRStepArgs& a, cudaStream_t s) {
    const int64_t blocks = (a.batch * a.nheads * a.headdim * LPR + 127) / 128;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    gdr_step_kernel<IO, LPR, NV><<<(unsigned)blocks, 128, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t launch_io(const GDRStepArgs& a, cudaStream_t s) {
    if (a.dstate <= 32) return launch_step<IO, 8, 1>(a, s);
    if (a.dstate <= 64) return launch_step<IO, 8, 2>(a, s);
    if (a.dstate <= 128) return launch_step<IO, 8, 4>(a, s);
    return launch_step<IO, 16, 4>(a, s);
}

}  // namespace

cudaError_t launch_gdr_step(const GDRStepArgs& a, int io, cudaStream_t s) {
    return io == 0 ? launch_io<float>(a, s) : launch_io<bf16>(a, s);
}

}  // namespace mmscan
