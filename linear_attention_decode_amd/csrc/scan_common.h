// scan_common.h -- what the two scan kernels (scan.hip: float32 matrix
// instructions; scan_mx.hip: bf16 ones) share.
#pragma once

#include "device_common.h"
#include "prompt.h"

namespace replay {

constexpr int kScanChunk = 64;   // segments are whole chunks of either kernel

// Workgroup -> (sequence, segment, first head): the workgroups of one group's
// heads (`per` of them, HB heads each) read the same q and k, so they go to
// one XCD (workgroup i runs on XCD i mod 8) one after the other; neighbouring
// groups go to neighbouring XCDs, so that each gets a share of every sequence
// where lengths differ.  Of up to 64 sequences the longest go first (a lane
// each, ranked by 64 comparisons): the last workgroups to start are then the
// shortest.  False for the places that fill up the last round.
struct Place {
    int b, seg, h, g;
};
__device__ __forceinline__ bool find_place(const ScanArgs &a, int HB, Place *p) {
    const int per = a.H / a.G / HB, x = blockIdx.x & 7, j = blockIdx.x >> 3;
    const int64_t unit = (int64_t)(j / per) * 8 + x;
    if (unit >= (int64_t)a.B * a.nseg * a.G) return false;
    p->g = (int)(unit % a.G);
    p->seg = (int)(unit / a.G % a.nseg);
    p->b = (int)(unit / a.G / a.nseg);
    if (a.B > 1 && a.B <= 64) {
        const int lane = threadIdx.x & 63;
        const int len = lane < a.B ? (int)((uint32_t)a.cu[lane + 1] - (uint32_t)a.cu[lane]) : 0;
        int rank = 0;
        for (int o = 0; o < a.B; ++o) {
            const int other = __builtin_amdgcn_readlane(len, o);
            rank += other > len || (other == len && o < lane);
        }
        p->b = __builtin_ctzll(__ballot(lane < a.B && rank == p->b));
    }
    p->h = p->g * (a.H / a.G) + j % per * HB;
    return true;
}
inline unsigned scan_blocks(const ScanArgs &a, int HB) {
    const int64_t units = (int64_t)a.B * a.nseg * a.G;
    return (unsigned)((units + 7) / 8 * 8 * (a.H / a.G / HB));
}

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
