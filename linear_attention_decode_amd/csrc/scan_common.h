// scan_common.h -- what the two scan kernels (scan.hip: float32 matrix
// instructions; scan_mx.hip: bf16 ones) share.
#pragma once

#include "device_common.h"

namespace replay {

constexpr int kScanChunk = 64;   // segments are whole chunks of either kernel

// Where a workgroup's tokens are.
struct Span {
    int t0, n;         // first row and number of tokens of the segment
    bool run, last;    // there is such a segment; it ends its sequence
};

__device__ __forceinline__ Span find_span(const ScanArgs &a, int b, int seg) {
    const int s0 = a.cu[b], s1 = a.cu[b + 1];
    if (s0 < 0 || s1 < s0 || s1 > a.T || s1 - s0 > a.max_len) return {0, 0, false, false};
    const int n = s1 - s0, at = seg * a.seg_len;
    if (at > 0 && at >= n) return {0, 0, false, false};
    const int left = n - at;
    return {s0 + at, left < a.seg_len ? left : a.seg_len, true, left <= a.seg_len};
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// The bf16 kernel's part of launch_scan: whether it covers the shape, the
// heads it gives a workgroup, and its launch (state_only: the segments' own
// states into the workspace).
bool scan_mx_supported(int P, int N, const ScanArgs &a);
int scan_mx_heads(int P, int H, int G);
hipError_t launch_scan_mx(int P, int N, const ScanArgs &a, bool state_only, hipStream_t s);

}  // namespace replay
