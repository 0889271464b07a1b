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
// Both directions run as many blocks as the SMs hold, which walk the rows in a
// grid-stride loop, the weights and (backward) the sums of a thread's columns in
// registers over all its rows.  The next rows are on their way to shared memory
// meanwhile: HBM's latency times its rate is 40 KB an SM in flight, more than
// the registers have room for beside the row at work.  Measured against the
// copy engine (44 us for the forward's 268 MB at 32768 rows of 2048, bf16):
// forward 44 us, backward (402 MB) 72; with a row a block and no loop 61, with
// the next row in registers 89.  What comes next is instruction issue (75% of
// the slots in the forward before two fp32 operations went into one: 50 us;
// the same in the backward measured 76 against 72).  Rows of more than 4096 columns or of no whole
// number of 16-byte pieces, and calls of so few rows that no block has two,
// take a row a block in the forward; the backward prefetches to registers.
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

__device__ __forceinline__ float shfl_add(float v, int m) { return v + __shfl_xor_sync(0xffffffffu, v, m); }
__device__ __forceinline__ float2 shfl_add(float2 v, int m) { return f2(shfl_add(v.x, m), shfl_add(v.y, m)); }
__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float2 plus(float2 a, float2 b) { return add2(a, b); }

// Sum of v (one value, or two) over the TPR threads of a row, in every one of
// them.  Rows of more than a warp go through `red`, one of two slots that
// alternate from call to call, so that one barrier a call is enough: a slot is
// written again only after the barrier of the call in between.
template <int TPR, typename T>
__device__ __forceinline__ T row_sum(T v, float2* red, int& slot) {
#pragma unroll
    for (int m = (TPR < 32 ? TPR : 32) / 2; m >= 1; m >>= 1) v = shfl_add(v, m);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        T* r = reinterpret_cast<T*>(red + slot * W);
        slot ^= 1;
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
        __syncthreads();
        v = r[0];
#pragma unroll
        for (int w = 1; w < W; ++w) v = plus(v, r[w]);
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

// A thread's elements of a row, in pairs: two fp32 operations an instruction.
template <int K>
__device__ __forceinline__ float2 pair(const float (&v)[K], int k) { return f2(v[k], v[k + 1]); }
template <int K>
__device__ __forceinline__ void put_pair(float (&v)[K], int k, float2 x) {
    v[k] = x.x;
    v[k + 1] = x.y;
}

// Mean and rstd of the row that v (0 past its end) is this thread's part of; v centred.
template <int VEC, int TPR, int NV>
__device__ __forceinline__ void center(float (&v)[NV * VEC], const NormArgs& p, int t, float2* red, int& slot, float& mean, float& rstd) {
    mean = 0.0f;
    if (!p.rms) {
        float2 s = f2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < NV * VEC; k += 2) s = add2(s, pair(v, k));
        mean = row_sum<TPR>(s.x + s.y, red, slot) * p.inv_cols;
        const float2 off = f2(-mean, -mean);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((t + i * TPR) * VEC >= p.cols) continue;     // stays 0
            if constexpr (VEC == 1) v[i] -= mean;
            else
#pragma unroll
                for (int e = 0; e < VEC; e += 2) put_pair(v, i * VEC + e, add2(pair(v, i * VEC + e), off));
        }
    }
    float2 s = f2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < NV * VEC; k += 2) s = fma2(pair(v, k), pair(v, k), s);
    rstd = rsqrtf(fmaf(row_sum<TPR>(s.x + s.y, red, slot), p.inv_cols, p.eps));
}

// y of VEC of its columns: v centred, w and b and (GATE) z the columns' own.
template <int VEC, bool GATE>
__device__ __forceinline__ void norm_out(const float* v, float rstd, const float* w, const float* b, const float* z, float* o) {
    if constexpr (VEC == 1) {
        o[0] = fmaf(v[0] * rstd, w[0], b[0]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 y = fma2(mul2(f2(v[e], v[e + 1]), f2(rstd, rstd)), f2(w[e], w[e + 1]), f2(b[e], b[e + 1]));
            o[e] = y.x;
            o[e + 1] = y.y;
        }
    }
    if constexpr (GATE)
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] *= z[e] * sigmoid_f32(z[e]);
}

// Rows on their way: every thread copies its own pieces of 16 bytes of the next
// rows to slots of its own in shared memory (cp.async) and reads nobody else's,
// so that a wait for its own copies is all it takes, and what is in flight
// costs no registers.
// Rows in flight, this one's included: four (six or eight measured the same or
// slower, the L1 being smaller), as far as the SM's shared memory goes.
constexpr int ring_depth(int stage, int blocks) {
    const int d = 200 * 1024 / (stage * blocks);
    return d > 4 ? 4 : d < 2 ? 2 : d;
}
constexpr bool norm_ring(int vec, int tpr) { return vec > 1 && tpr <= 256; }

constexpr int norm_fwd_resident(int bt, int elems) { return (elems > 8 ? 768 : 1024) / bt; }
template <int BT, int NV, int VEC, bool GATE>
struct FwdRing {
    static constexpr int STAGE = BT * NV * 16 * (GATE ? 2 : 1), D = ring_depth(STAGE, norm_fwd_resident(BT, NV * VEC));
};

template <typename IO, int VEC, int TPR, int NV, bool GATE>
__global__ void __launch_bounds__(norm_block(TPR), norm_fwd_resident(norm_block(TPR), NV * VEC)) norm_fwd_ring_kernel(const NormArgs p) {
    constexpr int BT = norm_block(TPR), RPB = BT / TPR;
    constexpr int STAGE = FwdRing<BT, NV, VEC, GATE>::STAGE, D = FwdRing<BT, NV, VEC, GATE>::D;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ float2 red[2 * (TPR > 32 ? TPR / 32 : 1)];
    int slot = 0;
    const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int cols = (int)p.cols;
    unsigned char* const own = ring + threadIdx.x * 16;
    const int64_t step = (int64_t)gridDim.x * RPB;
    auto fetch = [&](int64_t r0, int stage) {
        if (r0 < p.rows) {
            const int64_t base = (r0 + grp < p.rows ? r0 + grp : p.rows - 1) * cols;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * TPR) * VEC;
                if (c >= cols) continue;
                cp_async_16(own + stage * STAGE + i * BT * 16, static_cast<const IO*>(p.x) + base + c, 16);
                if constexpr (GATE) cp_async_16(own + stage * STAGE + (NV + i) * BT * 16, static_cast<const IO*>(p.z) + base + c, 16);
            }
        }
        cp_async_commit();
    };
    int64_t r0 = (int64_t)blockIdx.x * RPB;
#pragma unroll
    for (int d = 0; d < D - 1; ++d) fetch(r0 + d * step, d);
    float w[NV * VEC], b[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * TPR) * VEC;
        load_param<VEC>(p.weight && c < cols ? p.weight + c : nullptr, w + i * VEC, 1.0f);
        load_param<VEC>(p.bias && c < cols ? p.bias + c : nullptr, b + i * VEC, 0.0f);
    }
    for (int now = 0; r0 < p.rows; r0 += step, now = now + 1 == D ? 0 : now + 1) {
        cp_async_wait<D - 2>();
        const unsigned char* mine = own + now * STAGE;
        float v[NV * VEC], mean, rstd;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i * VEC + e] = 0.0f;
            if ((t + i * TPR) * VEC < cols) load_vec<IO, VEC>(reinterpret_cast<const IO*>(mine + i * BT * 16), v + i * VEC);
        }
        center<VEC, TPR, NV>(v, p, t, red, slot, mean, rstd);
        const int64_t row = r0 + grp;
        if (row < p.rows) {
            if (t == 0) {
                if (p.mean && !p.rms) p.mean[row] = mean;
                if (p.rstd) p.rstd[row] = rstd;
            }
            IO* y = static_cast<IO*>(p.y) + row * cols;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * TPR) * VEC;
                if (c >= cols) continue;
                float o[VEC], z[VEC];
                if constexpr (GATE) load_vec<IO, VEC>(reinterpret_cast<const IO*>(mine + (NV + i) * BT * 16), z);
                norm_out<VEC, GATE>(v + i * VEC, rstd, w + i * VEC, b + i * VEC, z, o);
                store_vec<IO, VEC>(y + c, o);
            }
        }
        // into the slots of the row before this one
        fetch(r0 + (D - 1) * step, now == 0 ? D - 1 : now - 1);
    }
}

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

    float v[NV * VEC], mean, rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * TPR) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i * VEC + e] = 0.0f;
        if (c < cols) load_vec<IO, VEC>(x + c, v + i * VEC);
    }
    center<VEC, TPR, NV>(v, p, t, red, slot, mean, rstd);
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
        float w[VEC], b[VEC], z[VEC], o[VEC];
        load_param<VEC>(p.weight ? p.weight + c : nullptr, w, 1.0f);
        load_param<VEC>(p.bias ? p.bias + c : nullptr, b, 0.0f);
        if (p.z) {
            load_vec<IO, VEC>(static_cast<const IO*>(p.z) + row * cols + c, z);
            norm_out<VEC, true>(v + i * VEC, rstd, w, b, z, o);
        } else {
            norm_out<VEC, false>(v + i * VEC, rstd, w, b, z, o);
        }
        store_vec<IO, VEC>(y + c, o);
    }
}

// Resident blocks an SM that the backward's grid counts on: 24 warps at 8
// elements a thread in 16-byte pieces (up to 80 registers); 16 by element or
// at 16 elements (128 registers; a block of 1024 threads has 64 and spills).
// (28 and 20 warps spill or crowd the ring: 62 and 92 us against 56 and 72.)
constexpr int norm_bwd_resident(int bt, int elems, int vec) { return bt >= 512 ? 1 : elems > 8 || vec == 1 ? 512 / bt : 768 / bt; }

// A thread's slots of a row: x, dy (z); then the row's mean and rstd, in rows of
// a warp and more once a warp (all its lanes copying one address take turns: 136
// us against 87, 32768 rows of 2048), in narrower ones for every thread (56 us
// against 58, 524288 gated rows of 64).
template <int BT, int TPR, int NV, int VEC, bool GATE>
struct BwdRing {
    static constexpr int LANES = TPR < 32 ? 1 : 32;
    static constexpr int STATS = BT * NV * 16 * (GATE ? 3 : 2), STAGE = STATS + BT / LANES * 8;
    static constexpr int D = ring_depth(STAGE, norm_bwd_resident(BT, NV * VEC, VEC));
};

template <typename IO, int VEC, int TPR, int NV, bool GATE>
__global__ void __launch_bounds__(norm_block(TPR), norm_bwd_resident(norm_block(TPR), NV * VEC, VEC)) norm_bwd_kernel(const NormArgs p) {
    constexpr int BT = norm_block(TPR);
    constexpr int RPB = BT / TPR;
    constexpr bool RING = norm_ring(VEC, TPR);
    using R = BwdRing<BT, TPR, NV, VEC, GATE>;
    extern __shared__ __align__(16) unsigned char ring[];
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
    unsigned char* const own = ring + threadIdx.x * 16;
    unsigned char* const stats = ring + R::STATS + threadIdx.x / R::LANES * 8;
    auto copy = [&](int64_t r0, int stage) {
        if (r0 < p.rows) {
            const int64_t row = r0 + grp < p.rows ? r0 + grp : p.rows - 1, base = row * cols;
            if (threadIdx.x % R::LANES == 0) {
                if (!p.rms) cp_async_4(stats + stage * R::STAGE, p.mean + row, 4);
                cp_async_4(stats + stage * R::STAGE + 4, p.rstd + row, 4);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * TPR) * VEC;
                if (c >= cols) continue;
                unsigned char* const at = own + stage * R::STAGE + i * BT * 16;
                cp_async_16(at, static_cast<const IO*>(p.x) + base + c, 16);
                cp_async_16(at + NV * BT * 16, static_cast<const IO*>(p.dy) + base + c, 16);
                if constexpr (GATE) cp_async_16(at + 2 * NV * BT * 16, static_cast<const IO*>(p.z) + base + c, 16);
            }
        }
        cp_async_commit();
    };
    int64_t r0 = (int64_t)blockIdx.x * RPB;
    constexpr bool kAhead = !RING && (VEC > 1 || (NV <= 8 && TPR < 1024));   // elements one by one: as registers allow
    int now = 0;
    if constexpr (RING) {
#pragma unroll
        for (int d = 0; d < R::D - 1; ++d) copy(r0 + d * step, d);
    } else if constexpr (kAhead) {
        fetch(r0);
    }
    for (; r0 < p.rows; r0 += step) {
        if constexpr (RING) {
            cp_async_wait<R::D - 2>();
            __syncwarp();                                    // the statistics are another lane's copy
            const unsigned char* mine = own + now * R::STAGE;
            const float2 st = *reinterpret_cast<const float2*>(stats + now * R::STAGE);
            mean = p.rms ? 0.0f : st.x;
            rstd = st.y;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                rx[i].load(reinterpret_cast<const IO*>(mine + i * BT * 16));
                ry[i].load(reinterpret_cast<const IO*>(mine + (NV + i) * BT * 16));
                if constexpr (GATE) rz[i].load(reinterpret_cast<const IO*>(mine + (2 * NV + i) * BT * 16));
            }
        } else if constexpr (!kAhead) {
            fetch(r0);
        }
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
        if constexpr (RING) {                                // into the slots of the row before this one
            copy(r0 + (R::D - 1) * step, now == 0 ? R::D - 1 : now - 1);
            now = now + 1 == R::D ? 0 : now + 1;
        } else if constexpr (kAhead) {
            if (r0 + step < p.rows) fetch(r0 + step);
        }
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

template <typename IO, int VEC, int TPR, int NV, bool GATE>
cudaError_t launch_fwd_ring(const NormArgs& a, int blocks, cudaStream_t s) {
    using R = FwdRing<norm_block(TPR), NV, VEC, GATE>;
    static std::atomic<uint64_t> attr_done{0};
    const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(norm_fwd_ring_kernel<IO, VEC, TPR, NV, GATE>), R::D * R::STAGE, attr_done);
    if (e != cudaSuccess) return e;
    norm_fwd_ring_kernel<IO, VEC, TPR, NV, GATE><<<blocks, norm_block(TPR), R::D * R::STAGE, s>>>(a);
    return cudaGetLastError();
}

template <typename IO, int VEC, int TPR, int NV, bool GATE>
cudaError_t launch_bwd_rows(const NormArgs& a, int blocks, cudaStream_t s) {
    using R = BwdRing<norm_block(TPR), TPR, NV, VEC, GATE>;
    constexpr int bytes = norm_ring(VEC, TPR) ? R::D * R::STAGE : 0;
    static std::atomic<uint64_t> attr_done{0};
    const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(norm_bwd_kernel<IO, VEC, TPR, NV, GATE>), bytes, attr_done);
    if (e != cudaSuccess) return e;
    norm_bwd_kernel<IO, VEC, TPR, NV, GATE><<<blocks, norm_block(TPR), bytes, s>>>(a);
    return cudaGetLastError();
}

template <typename IO, int VEC, int TPR, int NV>
cudaError_t launch_fwd(const NormArgs& a, cudaStream_t s) {
    constexpr int BT = norm_block(TPR), RPB = BT / TPR;
    const int64_t blocks = (a.rows + RPB - 1) / RPB;
    if constexpr (norm_ring(VEC, TPR)) {                     // where blocks have several rows each
        constexpr int resident = norm_fwd_resident(BT, NV * VEC);
        if (blocks > 148 * resident) return a.z ? launch_fwd_ring<IO, VEC, TPR, NV, true>(a, 148 * resident, s) : launch_fwd_ring<IO, VEC, TPR, NV, false>(a, 148 * resident, s);
    }
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    norm_fwd_kernel<IO, VEC, TPR, NV><<<(unsigned)blocks, BT, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename IO, int VEC, int TPR, int NV>
cudaError_t launch_bwd(const NormArgs& a, cudaStream_t s) {
    const int blocks = norm_bwd_blocks(a.rows, a.cols, sizeof(IO) == 4 ? 0 : 1);
    const cudaError_t e = a.z ? launch_bwd_rows<IO, VEC, TPR, NV, true>(a, blocks, s) : launch_bwd_rows<IO, VEC, TPR, NV, false>(a, blocks, s);
    if (e != cudaSuccess || !a.part) return e;
    norm_param_kernel<<<(unsigned)((2 * a.cols + 31) / 32), dim3(32, 32), 0, s>>>(a.part, blocks, a.cols, a.dweight, a.dbias);
    return cudaGetLastError();
}

// Forward: threads of a row at 16 elements each (8 in rows of up to 256; a row a
// block, 32768 rows of 2048 in bf16: 61 us at 16, 81 at 8, 65 at 64).
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

// Backward: threads of a row at 8 elements each; at 16 past 1024 columns in
// 16-byte pieces (72 us against 87, 32768 rows of 2048 in bf16: fewer warps take
// part in a row's sums), past 8192 by element.
int norm_bwd_tpr(int64_t cols, int vec) {
    if (cols <= 64) return cols <= 8 ? 1 : cols <= 16 ? 2 : cols <= 32 ? 4 : 8;
    if (cols <= 2048) return cols <= 256 ? 32 : cols <= 1024 || vec > 1 ? 128 : 256;
    if (vec == 1) return cols <= 4096 ? 512 : 1024;
    return cols <= 4096 ? 256 : cols <= 8192 ? 512 : 1024;
}
int norm_bwd_elems(int64_t cols, int vec) { return cols <= (vec == 1 ? 8192 : 1024) ? 8 : 16; }

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
            if constexpr (VEC > 1)
                if (!eight) return launch_bwd<IO, VEC, 128, 16 / VEC>(a, s);
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
