// mm_layer_api.cpp -- the C ABI of the gated delta rule and layer norm
// (declared in include/mm_scan.h): host-side argument checks and launch.
// Every check runs before anything is enqueued; a rejected call touches no
// buffer.
#include <cmath>

#include "mm_checks.h"
#include "mm_internal.h"
#include "mm_scan.h"

namespace {

using mmscan::aligned16;
using mmscan::inject_launch_failure;
using mmscan::kMaxIndex;
using mmscan::kMaxSeqlen;
using mmscan::mul_ok;
using mmscan::overlap;
using mmscan::Range;
using mmscan::report;
using mmscan::report_ok;
using mmscan::rng;

constexpr int64_t kC = mmscan::kGdrChunk;

mm_status from_cuda(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return report_ok();
    return report(MM_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

// One operand of a call: its name, address and bytes.
struct Operand {
    const char* name;
    const void* ptr;
    int64_t bytes;
};

// Alignment of every given pointer; no output over an input or another
// output, except outs[same_out] on exactly ins[same_in] (in-place state).
template <int NI, int NO>
mm_status check_operands(const Operand (&ins)[NI], const Operand (&outs)[NO], int same_out = -1, int same_in = -1) {
    for (const Operand& o : ins)
        if (o.ptr && !aligned16(o.ptr)) return report(MM_ERR_ALIGN, "%s is not 16-byte aligned", o.name);
    for (const Operand& o : outs)
        if (o.ptr && !aligned16(o.ptr)) return report(MM_ERR_ALIGN, "%s is not 16-byte aligned", o.name);
    for (int i = 0; i < NO; ++i) {
        const Range a = rng(outs[i].name, outs[i].ptr, outs[i].bytes);
        for (int j = 0; j < NI; ++j) {
            if (i == same_out && j == same_in && outs[i].ptr == ins[j].ptr) continue;
            if (overlap(a, rng(ins[j].name, ins[j].ptr, ins[j].bytes)))
                return report(MM_ERR_ALIAS, "%s overlaps %s", outs[i].name, ins[j].name);
        }
        for (int j = 0; j < i; ++j)
            if (overlap(a, rng(outs[j].name, outs[j].ptr, outs[j].bytes)))
                return report(MM_ERR_ALIAS, "%s overlaps %s", outs[i].name, outs[j].name);
    }
    return MM_OK;
}

// Byte counts of the operands of a gated-delta-rule call.
struct GdrSizes {
    int64_t qk, v, gate, state;                  // (b, L, G, N), (b, L, H, P), (b, L, H) io; (b, H, P, N) fp32
    int64_t nchunks, chunks;                     // per sequence; batch * H * nchunks
    int64_t rec, tlo, states, u;                 // records, low parts of T, bf16 states, rows written
};

mm_status check_gdr(const mm_gdr_dims* d, GdrSizes* z) {
    const int64_t B = d->batch, L = d->seqlen, H = d->nheads, P = d->headdim, N = d->dstate, G = d->ngroups;
    if (B < 1 || L < 1 || H < 1 || P < 1 || N < 1 || G < 1 || H % G != 0)
        return report(MM_ERR_DIMS, "sizes must be >= 1 and ngroups must divide nheads (batch=%lld seqlen=%lld nheads=%lld "
                      "headdim=%lld dstate=%lld ngroups=%lld)", (long long)B, (long long)L, (long long)H, (long long)P,
                      (long long)N, (long long)G);
    if (d->io != MM_F32 && d->io != MM_BF16) return report(MM_ERR_DTYPE, "io=%d is not MM_F32 or MM_BF16", (int)d->io);
    if (L > kMaxSeqlen || B > kMaxIndex || H > kMaxIndex || P > kMaxIndex || N > kMaxIndex)
        return report(MM_ERR_UNSUPPORTED, "seqlen must be <= 2^30 and the other sizes < 2^31");
    const int64_t eb = d->io == MM_F32 ? 4 : 2;
    z->nchunks = (L + kC - 1) / kC;
    int64_t bl, bh, pn;
    if (!mul_ok(B, L, &bl) || !mul_ok(bl, G, &z->qk) || !mul_ok(z->qk, N * eb, &z->qk) || !mul_ok(bl, H, &z->gate) ||
        !mul_ok(z->gate, P * eb, &z->v) || !mul_ok(z->gate, eb, &z->gate) || !mul_ok(B, H, &bh) || !mul_ok(P, N, &pn) ||
        !mul_ok(bh, pn, &z->state) || !mul_ok(z->state, 4, &z->state) || !mul_ok(bh, z->nchunks, &z->chunks) ||
        !mul_ok(pn, 2, &pn) || !mul_ok(z->chunks, mmscan::kGdrRecBytes, &z->rec) || !mul_ok(z->chunks, kC * kC * 2, &z->tlo) ||
        !mul_ok(z->chunks, pn, &z->states) || !mul_ok(z->chunks, P * kC * 2, &z->u) ||
        z->rec > INT64_MAX / 4 || z->states > INT64_MAX / 4 || z->u > INT64_MAX / 4)
        return report(MM_ERR_DIMS, "sizes overflow 64-bit byte counts");
    return MM_OK;
}

// What the chunked kernels need beyond check_gdr.
mm_status check_gdr_chunked(const mm_gdr_dims* d, GdrSizes* z) {
    if (mm_status st = check_gdr(d, z)) return st;
    if (d->io != MM_BF16) return report(MM_ERR_DTYPE, "the gated delta rule over a sequence takes bf16 (MM_BF16)");
    if (!mmscan::gdr_shape_supported(d->headdim, d->dstate))
        return report(MM_ERR_UNSUPPORTED, "the gated delta rule needs headdim and dstate of 64 or 128 (got %lld, %lld)",
                      (long long)d->headdim, (long long)d->dstate);
    if (z->chunks > kMaxIndex)
        return report(MM_ERR_UNSUPPORTED, "batch * nheads * ceil(seqlen / 64) = %lld must be < 2^31", (long long)z->chunks);
    return MM_OK;
}

mm_status check_scale(float scale) {
    if (!std::isfinite(scale)) return report(MM_ERR_SCALAR, "scale=%g must be finite", (double)scale);
    return MM_OK;
}

int64_t ckpt_bytes(const GdrSizes& z) { return z.rec + z.states + z.u; }
int64_t fwd_ws_bytes(const GdrSizes& z, bool with_ckpt) { return with_ckpt ? z.tlo : z.rec + z.tlo; }
int64_t bwd_ws_bytes(const GdrSizes& z) { return z.states + z.u; }

mm_status check_workspace(const void* ws, size_t have, int64_t need) {
    if (!ws) return report(MM_ERR_NULL, "workspace is NULL");
    if (have < static_cast<uint64_t>(need))
        return report(MM_ERR_DIMS, "workspace holds %llu bytes; the call needs %lld", (unsigned long long)have, (long long)need);
    return MM_OK;
}

mmscan::GDRArgs gdr_args(const mm_gdr_dims* d, const GdrSizes& z, float scale) {
    mmscan::GDRArgs a{};
    a.batch = d->batch; a.seqlen = d->seqlen; a.nheads = d->nheads; a.ngroups = d->ngroups;
    a.stall = mmscan::inject_gdr_stall();
    a.nchunks = z.nchunks; a.headdim = (int)d->headdim; a.dstate = (int)d->dstate; a.scale = scale;
    return a;
}

void* at(void* base, int64_t bytes) { return static_cast<unsigned char*>(base) + bytes; }

mm_status check_norm(const mm_norm_dims* d, int64_t* io_bytes) {
    if (d->rows < 1 || d->cols < 1)
        return report(MM_ERR_DIMS, "sizes must be >= 1 (rows=%lld cols=%lld)", (long long)d->rows, (long long)d->cols);
    if (d->io != MM_F32 && d->io != MM_BF16) return report(MM_ERR_DTYPE, "io=%d is not MM_F32 or MM_BF16", (int)d->io);
    if (d->cols > mmscan::kNormMaxCols || d->rows > kMaxIndex)
        return report(MM_ERR_UNSUPPORTED, "rows=%lld cols=%lld: rows must be < 2^31 and cols <= %lld", (long long)d->rows,
                      (long long)d->cols, (long long)mmscan::kNormMaxCols);
    *io_bytes = d->rows * d->cols * (d->io == MM_F32 ? 4 : 2);
    return MM_OK;
}

int64_t norm_ws_bytes(const mm_norm_dims* d) { return (int64_t)mmscan::norm_bwd_blocks(d->rows, d->cols, d->io) * 2 * d->cols * 4; }

}  // namespace

extern "C" {

mm_status mm_gdr_ckpt_size(const mm_gdr_dims* dims, size_t* bytes) {
    if (!dims || !bytes) return report(MM_ERR_NULL, "dims and bytes are required");
    GdrSizes z;
    if (mm_status st = check_gdr_chunked(dims, &z)) return st;
    *bytes = static_cast<size_t>(ckpt_bytes(z));
    return report_ok();
}

mm_status mm_gdr_fwd_workspace_size(const mm_gdr_dims* dims, int with_ckpt, size_t* bytes) {
    if (!dims || !bytes) return report(MM_ERR_NULL, "dims and bytes are required");
    GdrSizes z;
    if (mm_status st = check_gdr_chunked(dims, &z)) return st;
    *bytes = static_cast<size_t>(fwd_ws_bytes(z, with_ckpt != 0));
    return report_ok();
}

mm_status mm_gdr_bwd_workspace_size(const mm_gdr_dims* dims, size_t* bytes) {
    if (!dims || !bytes) return report(MM_ERR_NULL, "dims and bytes are required");
    GdrSizes z;
    if (mm_status st = check_gdr_chunked(dims, &z)) return st;
    *bytes = static_cast<size_t>(bwd_ws_bytes(z));
    return report_ok();
}

mm_status mm_gdr_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta, const float* h0,
                     float scale, void* o, float* hT, void* ckpt, void* workspace, size_t workspace_bytes,
                     const mm_gdr_dims* dims, void* stream) {
    if (!dims) return report(MM_ERR_NULL, "dims is NULL");
    if (!q || !k || !v || !g || !beta || !o) return report(MM_ERR_NULL, "q, k, v, g, beta and o are required");
    GdrSizes z;
    if (mm_status st = check_gdr_chunked(dims, &z)) return st;
    if (mm_status st = check_scale(scale)) return st;
    const int64_t ws = fwd_ws_bytes(z, ckpt != nullptr);
    if (mm_status st = check_workspace(workspace, workspace_bytes, ws)) return st;
    const Operand ins[] = {{"q", q, z.qk}, {"k", k, z.qk}, {"v", v, z.v}, {"g", g, z.gate}, {"beta", beta, z.gate},
                           {"h0", h0, z.state}};
    const Operand outs[] = {{"o", o, z.v}, {"hT", hT, z.state}, {"ckpt", ckpt, ckpt_bytes(z)}, {"workspace", workspace, ws}};
    if (mm_status st = check_operands(ins, outs, 1, 5)) return st;
    if (inject_launch_failure()) return report(MM_ERR_CUDA, "injected launch failure (MMSCAN_FAULT_INJECT)");
    mmscan::GDRArgs a = gdr_args(dims, z, scale);
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.h0 = h0; a.o = o; a.hT = hT;
    a.tlo = workspace;
    a.rec = ckpt ? ckpt : at(workspace, z.tlo);
    if (ckpt) {
        a.states = at(ckpt, z.rec);
        a.u = at(ckpt, z.rec + z.states);
    }
    return from_cuda(mmscan::launch_gdr_fwd(a, static_cast<cudaStream_t>(stream)), "mm_gdr_fwd launch");
}

mm_status mm_gdr_bwd(const void* q, const void* k, const void* v, const void* g, const void* beta, float scale,
                     const void* ckpt, const void* dout, const float* dhT, void* dq, void* dk, void* dv, void* dg, void* dbeta,
                     float* dh0, void* workspace, size_t workspace_bytes, const mm_gdr_dims* dims, void* stream) {
    if (!dims) return report(MM_ERR_NULL, "dims is NULL");
    if (!q || !k || !v || !g || !beta || !ckpt || !dout || !dq || !dk || !dv || !dg || !dbeta)
        return report(MM_ERR_NULL, "q, k, v, g, beta, ckpt, dout, dq, dk, dv, dg and dbeta are required");
    GdrSizes z;
    if (mm_status st = check_gdr_chunked(dims, &z)) return st;
    if (mm_status st = check_scale(scale)) return st;
    const int64_t ws = bwd_ws_bytes(z);
    if (mm_status st = check_workspace(workspace, workspace_bytes, ws)) return st;
    const Operand ins[] = {{"q", q, z.qk}, {"k", k, z.qk}, {"v", v, z.v}, {"g", g, z.gate}, {"beta", beta, z.gate},
                           {"ckpt", ckpt, ckpt_bytes(z)}, {"dout", dout, z.v}, {"dhT", dhT, z.state}};
    const Operand outs[] = {{"dq", dq, z.qk}, {"dk", dk, z.qk}, {"dv", dv, z.v}, {"dg", dg, z.gate}, {"dbeta", dbeta, z.gate},
                            {"dh0", dh0, z.state}, {"workspace", workspace, ws}};
    if (mm_status st = check_operands(ins, outs)) return st;
    if (inject_launch_failure()) return report(MM_ERR_CUDA, "injected launch failure (MMSCAN_FAULT_INJECT)");
    mmscan::GDRArgs a = gdr_args(dims, z, scale);
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
    void* ck = const_cast<void*>(ckpt);          // read only by the backward's kernels
    a.rec = ck;
    a.states = at(ck, z.rec);
    a.u = at(ck, z.rec + z.states);
    a.dout = dout; a.dhT = dhT; a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dh0 = dh0;
    a.dstates = workspace;
    a.dr = at(workspace, z.states);
    return from_cuda(mmscan::launch_gdr_bwd(a, static_cast<cudaStream_t>(stream)), "mm_gdr_bwd launch");
}

mm_status mm_gdr_step(const void* q, const void* k, const void* v, const void* g, const void* beta, float* h, float scale,
                      void* o, const mm_gdr_dims* dims, void* stream) {
    if (!dims) return report(MM_ERR_NULL, "dims is NULL");
    if (!q || !k || !v || !g || !beta || !h || !o) return report(MM_ERR_NULL, "q, k, v, g, beta, h and o are required");
    if (dims->seqlen != 1) return report(MM_ERR_DIMS, "a decode step has seqlen 1 (got %lld)", (long long)dims->seqlen);
    GdrSizes z;
    if (mm_status st = check_gdr(dims, &z)) return st;
    if (dims->dstate % 4 != 0 || dims->dstate > 256)
        return report(MM_ERR_UNSUPPORTED, "the gated delta rule's step needs dstate a multiple of 4 up to 256 (got %lld)",
                      (long long)dims->dstate);
    if (mm_status st = check_scale(scale)) return st;
    int64_t rows;
    if (!mul_ok(dims->batch * dims->nheads, dims->headdim, &rows) || rows > (kMaxIndex << 3))
        return report(MM_ERR_UNSUPPORTED, "batch * nheads * headdim must be < 2^34");
    const Operand ins[] = {{"q", q, z.qk}, {"k", k, z.qk}, {"v", v, z.v}, {"g", g, z.gate}, {"beta", beta, z.gate}};
    const Operand outs[] = {{"h", h, z.state}, {"o", o, z.v}};
    if (mm_status st = check_operands(ins, outs)) return st;
    if (inject_launch_failure()) return report(MM_ERR_CUDA, "injected launch failure (MMSCAN_FAULT_INJECT)");
    mmscan::GDRStepArgs a{};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.h = h; a.o = o;
    a.batch = dims->batch; a.nheads = dims->nheads; a.ngroups = dims->ngroups;
    a.headdim = (int)dims->headdim; a.dstate = (int)dims->dstate; a.scale = scale;
    return from_cuda(mmscan::launch_gdr_step(a, dims->io, static_cast<cudaStream_t>(stream)), "mm_gdr_step launch");
}

mm_status mm_layer_norm_fwd(const void* x, const float* weight, const float* bias, const void* z, float eps, int rms, void* y,
                            float* mean, float* rstd, const mm_norm_dims* dims, void* stream) {
    if (!dims) return report(MM_ERR_NULL, "dims is NULL");
    if (!x || !y) return report(MM_ERR_NULL, "x and y are required");
    int64_t n;
    if (mm_status st = check_norm(dims, &n)) return st;
    if (!std::isfinite(eps) || eps < 0.0f) return report(MM_ERR_SCALAR, "eps=%g must be finite and >= 0", (double)eps);
    const Operand ins[] = {{"x", x, n}, {"weight", weight, dims->cols * 4}, {"bias", bias, dims->cols * 4}, {"z", z, n}};
    const Operand outs[] = {{"y", y, n}, {"mean", mean, dims->rows * 4}, {"rstd", rstd, dims->rows * 4}};
    if (mm_status st = check_operands(ins, outs)) return st;
    if (inject_launch_failure()) return report(MM_ERR_CUDA, "injected launch failure (MMSCAN_FAULT_INJECT)");
    mmscan::NormArgs a{};
    a.x = x; a.z = z; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    a.rows = dims->rows; a.cols = dims->cols; a.eps = eps; a.inv_cols = 1.0f / (float)dims->cols; a.rms = rms ? 1 : 0;
    return from_cuda(mmscan::launch_norm_fwd(a, dims->io, static_cast<cudaStream_t>(stream)), "mm_layer_norm_fwd launch");
}

mm_status mm_layer_norm_bwd_workspace_size(const mm_norm_dims* dims, size_t* bytes) {
    if (!dims || !bytes) return report(MM_ERR_NULL, "dims and bytes are required");
    int64_t n;
    if (mm_status st = check_norm(dims, &n)) return st;
    *bytes = static_cast<size_t>(norm_ws_bytes(dims));
    return report_ok();
}

mm_status mm_layer_norm_bwd(const void* x, const float* weight, const float* bias, const void* z, int rms, const float* mean,
                            const float* rstd, const void* dy, void* dx, float* dweight, float* dbias, void* dz, void* workspace,
                            size_t workspace_bytes, const mm_norm_dims* dims, void* stream) {
    if (!dims) return report(MM_ERR_NULL, "dims is NULL");
    if (!x || !rstd || !dy || !dx || (!mean && !rms))
        return report(MM_ERR_NULL, "x, mean (unless rms), rstd, dy and dx are required");
    if (dz && !z) return report(MM_ERR_NULL, "dz without the gate z");
    int64_t n;
    if (mm_status st = check_norm(dims, &n)) return st;
    const bool params = dweight || dbias;
    const int64_t ws = params ? norm_ws_bytes(dims) : 0;
    if (params)
        if (mm_status st = check_workspace(workspace, workspace_bytes, ws)) return st;
    const Operand ins[] = {{"x", x, n}, {"weight", weight, dims->cols * 4}, {"bias", bias, dims->cols * 4}, {"z", z, n},
                           {"mean", mean, dims->rows * 4}, {"rstd", rstd, dims->rows * 4}, {"dy", dy, n}};
    const Operand outs[] = {{"dx", dx, n}, {"dweight", dweight, dims->cols * 4}, {"dbias", dbias, dims->cols * 4}, {"dz", dz, n},
                            {"workspace", params ? workspace : nullptr, ws}};
    if (mm_status st = check_operands(ins, outs)) return st;
    if (inject_launch_failure()) return report(MM_ERR_CUDA, "injected launch failure (MMSCAN_FAULT_INJECT)");
    mmscan::NormArgs a{};
    a.x = x; a.z = z; a.weight = weight; a.bias = bias; a.dy = dy; a.dx = dx; a.dz = dz;
    a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
    a.dweight = dweight; a.dbias = dbias; a.part = params ? static_cast<float*>(workspace) : nullptr;
    a.rows = dims->rows; a.cols = dims->cols; a.inv_cols = 1.0f / (float)dims->cols; a.rms = rms ? 1 : 0;
    return from_cuda(mmscan::launch_norm_bwd(a, dims->io, static_cast<cudaStream_t>(stream)), "mm_layer_norm_bwd launch");
}

}  // extern "C"
