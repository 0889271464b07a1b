// mm_checks.h -- the host-side argument checks the C entry points share.
#pragma once

#include <cstdint>
#include <cstdlib>
#include <cstring>

namespace mmscan {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// a * b without int64 overflow; false on overflow.
inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > INT64_MAX / a) return false;
    *out = a * b;
    return true;
}

// The kernels form time coordinates of the tiled copies, grid sizes and
// channel numbers in 32 bits; requests beyond these bounds are refused
// before launch.
constexpr int64_t kMaxSeqlen = int64_t(1) << 30;
constexpr int64_t kMaxIndex = 0x7fffffffLL;

struct Range {
    const char* name;
    uintptr_t lo, hi;   // [lo, hi)
};

inline Range rng(const char* name, const void* p, int64_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Range{name, lo, p ? lo + static_cast<uintptr_t>(bytes) : lo};
}

inline bool overlap(const Range& a, const Range& b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;   // NULL / empty
    return a.lo < b.hi && b.lo < a.hi;
}

// Fault-injection hook for the host-side error path: with
// MMSCAN_FAULT_INJECT=launch a call that passed its checks returns
// MM_ERR_CUDA without launching anything.
inline bool inject_launch_failure() {
    const char* v = std::getenv("MMSCAN_FAULT_INJECT");
    return v && std::strcmp(v, "launch") == 0;
}

// Test hook for the device-side give-up path: with MMSCAN_FAULT_INJECT=stall
// the kernels that stage their inputs through bounded waits (the two forward
// scans, the backward, the SSD kernels, the gated delta rule) are launched with their producer told
// to issue nothing.  Nothing is then in flight; every wait runs out after its
// limit, the kernel returns, and mm_device_status reports
// MM_ERR_DEVICE_TIMEOUT.  The outputs of such a call are undefined.
inline int inject_stall() {
    const char* v = std::getenv("MMSCAN_FAULT_INJECT");
    return (v && std::strcmp(v, "stall") == 0) ? 1 : 0;
}

// The same for the gated delta rule's kernels after a start:
// MMSCAN_FAULT_INJECT=stall-late stages the first two chunks (heads) of a CTA,
// so that the waits run out with copies and products issued.  GDRArgs::stall.
inline int inject_gdr_stall() {
    const char* v = std::getenv("MMSCAN_FAULT_INJECT");
    return (v && std::strcmp(v, "stall-late") == 0) ? 3 : inject_stall();
}

}  // namespace mmscan
