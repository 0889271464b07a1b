// layer_norm.cu -- sm_100a kernels for layer norm over the last dimension,
// forward and backward, with an optional gate.
//
// What it computes, per row of x (rows, cols):
//     xh = (x - mean) rstd,  rstd = 1 / sqrt(var + eps)     (rms: mean = 0)
//     n  = xh w + b,         y = n silu(z)                  (w, b, z optional)
// and, with dn = dy silu(z), d = dn w, averages over the row's columns:
//     dx = rstd (d - avg(d) - xh avg(d xh))                 (rms: no avg(d))
//     dz = dy n sig(z) (1 + z (1 - sig(z))),  dw = sum_rows dn xh,  db = sum_rows dn
//
// Bound: HBM (x, z, dy read once, y, dx, dz written once; a dozen operations
// an element).  A row is kept in the registers of TPR threads, so that the
// mean, the centred sum of squares (two passes over registers: no
// cancellation when the mean is large) and the output take one read of
// memory.  All statistics and sums are fp32.
//
// The forward gives each group of TPR threads one row (16 elements a thread)
// and lets many small blocks overlap.  The backward keeps 8 elements a thread
// and as many blocks as the SMs hold; they walk the rows in a grid-stride loop
// with the next row's loads issued before this row's sums, the weights and
// the sums of a thread's columns in registers over all its rows.
//
// The weight's gradient: every block writes one partial row to the workspace,
// and a second kernel adds the partials in block order: no atomics, so the
// result is bit-identical from run to run.
#include <type_traits>

#include "mm_common.cuh"
#include "mm_internal.h"

namespace mmscan {

namespace {


__device__ __forceinline__ float sigmoid_f32(float z) { return __fdividef(1.0f, 1.0f + ex2_approx(-z * kLog2e)); }

// VEC consecutive elements, widened to fp32 (16-byte accesses for VEC > 1).
template <typename IO, int VEC>
__device__ __forceinline__ void load_vec(const IO* p, float* v) {
    if constexpr (VEC == 1) {
        v[0] = load1(p);
    } else if constexpr (sizeof(IO) == 4) {
        const float4 q = *reinterpret_cast<const float4*>(p);
        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
        v[4] = bf16_lo(q.z); v[5] = bf16_hi(q.z); v[6] = bf16_lo(q.w); v[7] = bf16_hi(q.w);
    }
}

template <typename IO, int VEC>
__device__ __forceinline__ void store_vec(IO* p, const float* v) {
    if constexpr (VEC == 1) {
        store1(p, v[0]);
    } else if constexpr (sizeof(IO) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
}

template <int VEC>
__device__ __forceinline__ void load_param(const float* p, float* v, float none) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = none;
    if (!p) return;
    if constexpr (VEC == 1) {
        v[0] = *p;
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
            const float4 q = *reinterpret_cast<const float4*>(p + e);
            v[e] = q.x; v[e + 1] = q.y; v[e + 2] = q.z; v[e + 3] = q.w;
        }
    }
}

// Sum of (a, b) over the TPR threads of a row, in every one of them.  Rows of
// more than a warp go through `red`, one of two slots that alternate from
// call to call, so that one barrier a call is enough: a slot is written again
// only after the barrier of the call in between.
template <int TPR>
__device__ __forceinline__ float2 row_sum(float2 v, float2* red, int& slot) {
#pragma unroll
    for (int m = (TPR < 32 ? TPR : 32) / 2; m >= 1; m >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, m);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, m);
    }
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        float2* r = red + slot * W;
        slot ^= 1;
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
        __syncthreads();
        v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            v.x += r[w].x;
            v.y += r[w].y;
        }
    }
    return v;
}

constexpr int norm_block(int tpr) { return tpr < 128 ? 128 : tpr; }

// VEC elements as they are in memory (the next row's, while this one's are used).
template <typename IO, int VEC>
struct Raw {
    typename std::conditional<VEC == 1, IO, uint4>::type v;
    __device__ __forceinline__ void load(const IO* p) { v = *reinterpret_cast<const decltype(v)*>(p); }
    __device__ __forceinline__ void get(float* f) const { load_vec<IO, VEC>(reinterpret_cast<const IO*>(&v), f); }
};

template <typename IO, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(norm_block(TPR)) norm_fwd_kernel(const NormArgs p) {
    constexpr int RPB = norm_block(TPR) / TPR;
    __shared__ float2 red[2 * (TPR > 32 ? TPR / 32 : 1)];
    int slot = 0;
    const int t = threadIdx.x % TPR;
    const int64_t row0 = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
    const bool active = row0 < p.rows;
    const int64_t row = active ? row0 : p.rows - 1;        // idle groups follow along (shuffles)
    const int cols = (int)p.cols;
    const IO* x = static_cast<const IO*>(p.x) + row * cols;

    float v[NV * VEC];
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * TPR) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i * VEC + e] = 0.0f;
        if (c < cols) load_vec<IO, VEC>(x + c, v + i * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e) s.x += v[i * VEC + e];
    }
    float mean = 0.0f;
    if (!p.rms) mean = row_sum<TPR>(s, red, slot).x * p.inv_cols;
    s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool in = (t + i * TPR) * VEC < cols;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            v[i * VEC + e] -= mean;
            if (in) s.x = fmaf(v[i * VEC + e], v[i * VEC + e], s.x);
        }
    }
    const float var = row_sum<TPR>(s, red, slot).x * p.inv_cols;
    const float rstd = 1.0f / sqrtf(var + p.eps);
    if (!active) return;
    if (t == 0) {
        if (p.mean && !p.rms) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    IO* y = static_cast<IO*>(p.y) + row * cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * TPR) * VEC;
        if (c >= cols) continue;
        float w[VEC], b[VEC];
        load_param<VEC>(p.weight ? p.weight + c : nullptr, w, 1.0f);
        load_param<VEC>(p.bias ? p.bias + c : nullptr, b, 0.0f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = fmaf(v[i * VEC + e] * rstd, w[e], b[e]);
        if (p.z) {
            float z[VEC];
            load_vec<IO, VEC>(static_cast<const IO*>(p.z) + row * cols + c, z);
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] *= z[e] * sigmoid_f32(z[e]);
        }
        store_vec<IO, VEC>(y + c, w);
    }
}

// Resident blocks an SM that the backward's grid counts on: 24 warps at 8
// elements a thread in 16-byte pieces (up to 80 registers); 16 by element or
// at 16 elements (128 registers; a block of 1024 threads has 64 and spills).
constexpr int norm_bwd_resident(int bt, int elems, int vec) { return bt >= 512 ? 1 : elems > 8 || vec == 1 ? 512 / bt : 768 / bt; }

template <typename IO, int VEC, int TPR, int NV, bool GATE>
__global__ void __launch_bounds__(norm_block(TPR), norm_bwd_resident(norm_block(TPR), NV * VEC, VEC)) norm_bwd_kernel(const NormArgs p) {
    constexpr int BT = norm_block(TPR);
    constexpr int RPB = BT / TPR;
    __shared__ float2 red[2 * (TPR > 32 ? TPR / 32 : 1)];
    int slot = 0;
    const int t = threadIdx.x % TPR;
    const int grp = threadIdx.x / TPR;
    const int cols = (int)p.cols;
    float dw[NV * VEC], db[NV * VEC], w[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * TPR) * VEC;
        load_param<VEC>(p.weight && c < cols ? p.weight + c : nullptr, w + i * VEC, 1.0f);
    }
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) dw[i] = db[i] = 0.0f;

    const int64_t step = (int64_t)gridDim.x * RPB;
    Raw<IO, VEC> rx[NV], ry[NV], rz[GATE ? NV : 1];
    float mean, rstd;
    auto fetch = [&](int64_t r0) {
        const int64_t row = r0 + grp < p.rows ? r0 + grp : p.rows - 1;     // idle groups follow along (shuffles)
        mean = p.rms ? 0.0f : p.mean[row];
        rstd = p.rstd[row];
        const int64_t base = row * cols;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * TPR) * VEC;
            if (c >= cols) continue;
            rx[i].load(static_cast<const IO*>(p.x) + base + c);
            ry[i].load(static_cast<const IO*>(p.dy) + base + c);
            if constexpr (GATE) rz[i].load(static_cast<const IO*>(p.z) + base + c);
        }
    };
    int64_t r0 = (int64_t)blockIdx.x * RPB;
    constexpr bool kAhead = VEC > 1 || (NV <= 8 && TPR < 1024);   // elements one by one: as registers allow
    if (kAhead) fetch(r0);
    for (; r0 < p.rows; r0 += step) {
        if (!kAhead) fetch(r0);
        const bool active = r0 + grp < p.rows;
        const int64_t base = (r0 + grp) * cols;
        const float rs = rstd;
        float xh[NV * VEC], d[NV * VEC];
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * TPR) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) xh[i * VEC + e] = d[i * VEC + e] = 0.0f;
            if (c >= cols) continue;
            rx[i].get(xh + i * VEC);
            ry[i].get(d + i * VEC);
#pragma unroll
            for (int e = 0; e < VEC; ++e) xh[i * VEC + e] = (xh[i * VEC + e] - mean) * rs;
            if constexpr (GATE) {
                float z[VEC], b[VEC], dz[VEC];
                rz[i].get(z);
                load_param<VEC>(p.bias ? p.bias + c : nullptr, b, 0.0f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int k = i * VEC + e;
                    const float sg = sigmoid_f32(z[e]);
                    const float n = fmaf(xh[k], w[k], b[e]);
                    dz[e] = d[k] * n * sg * fmaf(z[e], 1.0f - sg, 1.0f);
                    d[k] *= z[e] * sg;
                }
                if (active && p.dz) store_vec<IO, VEC>(static_cast<IO*>(p.dz) + base + c, dz);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int k = i * VEC + e;
                if (active) {
                    dw[k] = fmaf(d[k], xh[k], dw[k]);
                    db[k] += d[k];
                }
                d[k] *= w[k];
                s.x += d[k];
                s.y = fmaf(d[k], xh[k], s.y);
            }
        }
        if (kAhead && r0 + step < p.rows) fetch(r0 + step);
        s = row_sum<TPR>(s, red, slot);
        const float a0 = p.rms ? 0.0f : s.x * p.inv_cols;
        const float a1 = s.y * p.inv_cols;
        if (active) {
            IO* dx = static_cast<IO*>(p.dx) + base;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * TPR) * VEC;
                if (c >= cols) continue;
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const int k = i * VEC + e;
                    o[e] = rs * (d[k] - a0 - xh[k] * a1);
                }
                store_vec<IO, VEC>(dx + c, o);
            }
        }
    }
    if (!p.part) return;
    // Rows of one block that share a warp: add their sums by shuffles, then
    // the block's groups in group order through shared memory.
    float* part = p.part + (int64_t)blockIdx.x * 2 * cols;
    if constexpr (TPR < 32) {
#pragma unroll
        for (int m = TPR; m < 32; m <<= 1)
#pragma unroll
            for (int i = 0; i < NV * VEC; ++i) {
                dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], m);
                db[i] += __shfl_xor_sync(0xffffffffu, db[i], m);
            }
    }
    if constexpr (RPB > 1) {
        constexpr int W = BT / 32, TW = TPR < 32 ? TPR : 32;
        __shared__ float acc[W][TW * NV * VEC];
        const int w = threadIdx.x / 32, l = threadIdx.x % 32;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (l < TW)
#pragma unroll
                for (int i = 0; i < NV * VEC; ++i) acc[w][l * NV * VEC + i] = half ? db[i] : dw[i];
            __syncthreads();
            for (int j = threadIdx.x; j < TW * NV * VEC; j += BT) {
                const int k = j % (NV * VEC);
                const int c = (j / (NV * VEC) + (k / VEC) * TPR) * VEC + k % VEC;
                float s = 0.0f;
#pragma unroll
                for (int q = 0; q < W; ++q) s += acc[q][j];
                if (c < cols) part[half * cols + c] = s;
            }
            __syncthreads();
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * TPR) * VEC;
            if (c >= cols) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                part[c + e] = dw[i * VEC + e];
                part[cols + c + e] = db[i * VEC + e];
            }
        }
    }
}

// dw, db (the two halves of a partial row) = the sums over the blocks, in a
// fixed order: thread row r adds blocks r, r + 32, ..., then the 32 sums.
__global__ void __launch_bounds__(1024) norm_param_kernel(const float* part, int nblk, int64_t cols, float* dw, float* db) {
    __shared__ float acc[32][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.0f;
    if (c < 2 * cols)
#pragma unroll 4
        for (int b = threadIdx.y; b < nblk; b += 32) s += part[(int64_t)b * 2 * cols + c];
    acc[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < 2 * cols) {
        s = 0.0f;
#pragma unroll
        for (int r = 0; r < 32; ++r) s += acc[r][threadIdx.x];
        if (c < cols) {
            if (dw) dw[c] = s;
        } else if (db) {
            db[c - cols] = s;
        }
    }
}

template <typename IO, int VEC, int TPR, int NV>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t s) {
    constexpr int BT = norm_block(TPR), RPB = BT / TPR;
    const int64_t blocks = (a.rows + RPB - 1) / RPB;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    norm_fwd_kernel<IO, VEC, TPR, NV><<<(unsigned)blocks, BT, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO, int VEC, int TPR, int NV>
cudaError_t launch_bwd(const NormArgs& a, cudaStream_t s) {
    const int blocks = norm_bwd_blocks(a.rows, a.cols, sizeof(IO) == 4 ? 0 : 1);
    if (a.z) norm_bwd_kernel<IO, VEC, TPR, NV, true><<<blocks, norm_block(TPR), 0, s>>>(a);
    else norm_bwd_kernel<IO, VEC, TPR, NV, false><<<blocks, norm_block(TPR), 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.part) return e;
    norm_param_kernel<<<(unsigned)((2 * a.cols + 31) / 32), dim3(32, 32), 0, s>>>(a.part, blocks, a.cols, a.dweight, a.dbias);
    return cudaGetLastError();
}

// Forward: threads of a row at 16 elements each (8 in rows of up to 256).
// Measured (33.5 M elements in rows of 2048, bf16): 61 us at 16 elements, 81 at
// 8, 65 at 64 (a warp a row); 84 for a grid that stays and walks the rows.
template <typename IO, int VEC>
cudaError_t launch_fwd_vec(const NormArgs& a, cudaStream_t s) {
    if (a.cols <= 8) return launch_fwd<IO, VEC, 1, 8 / VEC>(a, s);
    if (a.cols <= 16) return launch_fwd<IO, VEC, 2, 8 / VEC>(a, s);
    if (a.cols <= 32) return launch_fwd<IO, VEC, 4, 8 / VEC>(a, s);
    if (a.cols <= 64) return launch_fwd<IO, VEC, 8, 8 / VEC>(a, s);
    if constexpr (VEC == 1) {                                // rows no whole number of pieces
        if (a.cols <= 128) return launch_fwd<IO, 1, 32, 4>(a, s);
        if (a.cols > 256 && a.cols <= 512) return launch_fwd<IO, 1, 128, 4>(a, s);
    }
    if (a.cols <= 256) return launch_fwd<IO, VEC, 32, 8 / VEC>(a, s);
    if (a.cols <= 512) return launch_fwd<IO, VEC, 32, 16 / VEC>(a, s);
    if (a.cols <= 2048) return launch_fwd<IO, VEC, 128, 16 / VEC>(a, s);
    if (a.cols <= 4096) return launch_fwd<IO, VEC, 256, 16 / VEC>(a, s);
    if (a.cols <= 8192) return launch_fwd<IO, VEC, 512, 16 / VEC>(a, s);
    return launch_fwd<IO, VEC, 1024, 16 / VEC>(a, s);
}

// Backward: threads of a row at 8 elements each; at 16 past 2048 columns in
// 16-byte pieces, past 8192 by element.
int norm_bwd_tpr(int64_t cols, int vec) {
    if (cols <= 64) return cols <= 8 ? 1 : cols <= 16 ? 2 : cols <= 32 ? 4 : 8;
    if (cols <= 2048) return cols <= 256 ? 32 : cols <= 1024 ? 128 : 256;
    if (vec == 1) return cols <= 4096 ? 512 : 1024;
    return cols <= 4096 ? 256 : cols <= 8192 ? 512 : 1024;
}
int norm_bwd_elems(int64_t cols, int vec) { return cols <= (vec == 1 ? 8192 : 2048) ? 8 : 16; }

template <typename IO, int VEC>
cudaError_t launch_bwd_vec(const NormArgs& a, cudaStream_t s) {
    const bool eight = norm_bwd_elems(a.cols, VEC) == 8;
    switch (norm_bwd_tpr(a.cols, VEC)) {
        case 1: return launch_bwd<IO, VEC, 1, 8 / VEC>(a, s);
        case 2: return launch_bwd<IO, VEC, 2, 8 / VEC>(a, s);
        case 4: return launch_bwd<IO, VEC, 4, 8 / VEC>(a, s);
        case 8: return launch_bwd<IO, VEC, 8, 8 / VEC>(a, s);
        case 32:
            if constexpr (VEC == 1)
                if (a.cols <= 128) return launch_bwd<IO, 1, 32, 4>(a, s);
            return launch_bwd<IO, VEC, 32, 8 / VEC>(a, s);
        case 128:
            if constexpr (VEC == 1)
                if (a.cols <= 512) return launch_bwd<IO, 1, 128, 4>(a, s);
            return launch_bwd<IO, VEC, 128, 8 / VEC>(a, s);
        case 256:
            if (eight) return launch_bwd<IO, VEC, 256, 8 / VEC>(a, s);
            if constexpr (VEC > 1) return launch_bwd<IO, VEC, 256, 16 / VEC>(a, s);
            break;
        case 512:
            if constexpr (VEC == 1) return launch_bwd<IO, 1, 512, 8>(a, s);
            else return launch_bwd<IO, VEC, 512, 16 / VEC>(a, s);
        default:
            if constexpr (VEC == 1)
                if (eight) return launch_bwd<IO, 1, 1024, 8>(a, s);
            return launch_bwd<IO, VEC, 1024, 16 / VEC>(a, s);
    }
    return cudaErrorInvalidConfiguration;
}

}  // namespace

// Blocks of the backward: what 148 SMs hold at once, and no more than there
// are rows.
int norm_bwd_blocks(int64_t rows, int64_t cols, int io) {
    const int full = io == 0 ? 4 : 8, vec = cols % full == 0 ? full : 1;
    const int tpr = norm_bwd_tpr(cols, vec), bt = norm_block(tpr);
    const int64_t need = (rows + bt / tpr - 1) / (bt / tpr);
    const int64_t fill = 148 * norm_bwd_resident(bt, norm_bwd_elems(cols, vec), vec);
    return (int)(need < fill ? need : fill);
}

// Rows of whole 16-byte pieces move 16 bytes at a time, others by element.
cudaError_t launch_norm_fwd(const NormArgs& a, int io, cudaStream_t s) {
    if (io == 0) return a.cols % 4 == 0 ? launch_fwd_vec<float, 4>(a, s) : launch_fwd_vec<float, 1>(a, s);
    return a.cols % 8 == 0 ? launch_fwd_vec<bf16, 8>(a, s) : launch_fwd_vec<bf16, 1>(a, s);
}

cudaError_t launch_norm_bwd(const NormArgs& a, int io, cudaStream_t s) {
    if (io == 0) return a.cols % 4 == 0 ? launch_bwd_vec<float, 4>(a, s) : launch_bwd_vec<float, 1>(a, s);
    return a.cols % 8 == 0 ? launch_bwd_vec<bf16, 8>(a, s) : launch_bwd_vec<bf16, 1>(a, s);
}

}  // namespace mmscan
