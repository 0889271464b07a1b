// layer_checks_sanitized.cpp -- the host-side checks of the gated delta rule's
// and layer norm's entry points (mm_layer_api.cpp) under AddressSanitizer and
// UndefinedBehaviorSanitizer, without CUDA: the launchers are stubs that only
// count, sizes are taken at and past every limit, and pointers are fake and
// never dereferenced.  Exit status 0 and "layer checks ok" when every call
// returns a documented status without undefined behaviour and the calls in
// range reach their launcher.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <limits>

#include "cuda_runtime.h"
#include "mm_internal.h"
#include "mm_scan.h"

const char* cudaGetErrorString(cudaError_t) { return "stub"; }
const char* cudaGetErrorName(cudaError_t) { return "stub"; }

namespace {
int g_launches = 0;
}

namespace mmscan {
mm_status report(mm_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return st;
}
mm_status report_ok() { return MM_OK; }
bool gdr_shape_supported(int64_t p, int64_t n) { return (p == 64 || p == 128) && (n == 64 || n == 128); }
cudaError_t launch_gdr_fwd(const GDRArgs&, cudaStream_t) { ++g_launches; return cudaSuccess; }
cudaError_t launch_gdr_bwd(const GDRArgs&, cudaStream_t) { ++g_launches; return cudaSuccess; }
cudaError_t launch_gdr_step(const GDRStepArgs&, int, cudaStream_t) { ++g_launches; return cudaSuccess; }
cudaError_t launch_norm_fwd(const NormArgs&, int, cudaStream_t) { ++g_launches; return cudaSuccess; }
cudaError_t launch_norm_bwd(const NormArgs&, int, cudaStream_t) { ++g_launches; return cudaSuccess; }
int norm_bwd_blocks(int64_t rows, int64_t, int) { return rows < 444 ? (int)rows : 444; }
}  // namespace mmscan

int main() {
    const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 2, 4, 63, 64, 65, 128, 256, 260, 1 << 20, 1 << 30, (int64_t(1) << 30) + 1,
                             (int64_t(1) << 31) - 1, int64_t(1) << 31, int64_t(1) << 40, int64_t(1) << 62, INT64_MAX};
    const float scalars[] = {0.0f, 0.1f, -1.0f, std::numeric_limits<float>::infinity(), std::numeric_limits<float>::quiet_NaN()};
    auto ptr = [](int k) { return reinterpret_cast<void*>(uintptr_t(k + 1) << 58); };
    auto fp = [&](int k) { return static_cast<float*>(ptr(k)); };
    int calls = 0, bad = 0;
    auto see = [&](mm_status st) {
        ++calls;
        if (st < MM_OK || st > MM_ERR_ALIAS || st == MM_ERR_CUDA) ++bad;
    };
    for (int64_t a : sizes)
        for (int64_t b : sizes)
            for (int64_t c : sizes)
                for (int io = 0; io < 3; ++io) {
                    const mm_gdr_dims forms[] = {{a, b, c, 64, 128, 1, io}, {1, a, 2, b, c, 1, io}, {a, 64, b, 64, 64, c, io}, {a, 1, b, 64, c, 1, io}};
                    for (const mm_gdr_dims& d : forms)
                        for (float s : {0.1f, scalars[(calls % 5 + 5) % 5]}) {
                            size_t n = 0;
                            see(mm_gdr_ckpt_size(&d, &n));
                            see(mm_gdr_fwd_workspace_size(&d, io, &n));
                            see(mm_gdr_bwd_workspace_size(&d, &n));
                            see(mm_gdr_fwd(ptr(0), ptr(1), ptr(2), ptr(3), ptr(4), nullptr, s, ptr(5), nullptr, nullptr, ptr(6), SIZE_MAX, &d, nullptr));
                            see(mm_gdr_bwd(ptr(0), ptr(1), ptr(2), ptr(3), ptr(4), s, ptr(5), ptr(6), nullptr, ptr(7), ptr(8), ptr(9), ptr(10), ptr(11),
                                           nullptr, ptr(12), SIZE_MAX, &d, nullptr));
                            see(mm_gdr_step(ptr(0), ptr(1), ptr(2), ptr(3), ptr(4), fp(5), s, ptr(6), &d, nullptr));
                        }
                    const mm_norm_dims nd = {a, b, io};
                    size_t n = 0;
                    see(mm_layer_norm_bwd_workspace_size(&nd, &n));
                    see(mm_layer_norm_fwd(ptr(0), fp(1), fp(2), ptr(3), scalars[calls % 5], 0, ptr(4), fp(5), fp(6), &nd, nullptr));
                    see(mm_layer_norm_bwd(ptr(0), fp(1), fp(2), ptr(3), 1, nullptr, fp(4), ptr(5), ptr(6), fp(7), fp(8), ptr(9), ptr(10), SIZE_MAX, &nd,
                                          nullptr));
                }
    const mm_gdr_dims fine = {2, 130, 4, 64, 128, 2, MM_BF16};
    const mm_gdr_dims one = {2, 1, 4, 7, 12, 2, MM_F32};
    const mm_norm_dims norm = {3, 77, MM_BF16};
    const int before = g_launches;
    bad += mm_gdr_fwd(ptr(0), ptr(1), ptr(2), ptr(3), ptr(4), fp(9), 0.1f, ptr(5), fp(9), ptr(7), ptr(6), SIZE_MAX, &fine, nullptr) != MM_OK;
    bad += mm_gdr_step(ptr(0), ptr(1), ptr(2), ptr(3), ptr(4), fp(5), 0.1f, ptr(6), &one, nullptr) != MM_OK;
    bad += mm_layer_norm_fwd(ptr(0), nullptr, nullptr, nullptr, 0.0f, 0, ptr(4), nullptr, nullptr, &norm, nullptr) != MM_OK;
    bad += mm_layer_norm_bwd(ptr(0), nullptr, nullptr, nullptr, 1, nullptr, fp(4), ptr(5), ptr(6), nullptr, nullptr, nullptr, nullptr, 0, &norm, nullptr) != MM_OK;
    bad += g_launches != before + 4;
    if (bad) printf("%d of %d calls wrong\n", bad, calls);
    else printf("layer checks ok: %d calls, %d launches\n", calls, g_launches);
    return bad != 0;
}
