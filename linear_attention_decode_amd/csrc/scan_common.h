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
// CB workgroups share a head, each with its columns of v: block cb of them.
// 2^a.share XCDs share a group's workgroups.
struct Place {
    int b, seg, h, g, cb;
};
__device__ __forceinline__ bool find_place(const ScanArgs &a, int HB, Place *p, int CB = 1) {
    const int per = a.H / a.G / HB * CB, others = (1 << a.share) - 1, part = (per + others) >> a.share;
    const int x = blockIdx.x & 7, j = blockIdx.x >> 3;
    int64_t unit = (int64_t)(j / part) * 8 + x;
    const int i = ((int)unit & others) * part + j % part;   // of the group's workgroups
    unit >>= a.share;
    if (unit >= (int64_t)a.B * a.nseg * a.G || i >= per) return false;
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
    p->h = p->g * (a.H / a.G) + i / CB * HB;
    p->cb = i % CB;
    return true;
}
inline unsigned scan_blocks(const ScanArgs &a, int HB, int CB = 1) {
    const int64_t units = (int64_t)a.B * a.nseg * a.G << a.share;
    return (unsigned)((units + 7) / 8 * 8 * ((a.H / a.G / HB * CB + (1 << a.share) - 1) >> a.share));
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

// The value of the lane d before (behind) this one in its row of 16, 1 past the row's end.
template <int CTRL>
__device__ __forceinline__ float row_move(float x) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0x3f800000, (int)__float_as_uint(x), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float row_upto(float x) {
    x *= row_move<0x111>(x);
    x *= row_move<0x112>(x);
    x *= row_move<0x114>(x);
    x *= row_move<0x118>(x);
    return x;
}
__device__ __forceinline__ float row_from(float x) {
    x *= row_move<0x101>(x);
    x *= row_move<0x102>(x);
    x *= row_move<0x104>(x);
    x *= row_move<0x108>(x);
    return x;
}

// alpha_{j+1} ... alpha_i of a tile of 16, lane (i = c, j = 4 lg + r), for j <= i:
// alpha over the blocks of 4 between j's and i, times what is behind j in its own
__device__ __forceinline__ f32x4 diagonal_decays(const float *alpha, int c, int lg) {
    const f32x4 aa = *reinterpret_cast<const f32x4 *>(alpha + 4 * lg);
    const float R = row_upto(c >= 4 * (lg + 1) ? alpha[c] : 1.f);
    f32x4 D = {R, R, R, R};
    float f = 1.f;
#pragma unroll
    for (int r = 2; r >= 0; --r) {
        f = 4 * lg + r + 1 <= c ? f * aa[r + 1] : 1.f;
        D[r] *= f;
    }
    return D;
}

__device__ __forceinline__ float lane_value(float x, int lane) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), lane));
}

// x's upper bits and y's as a bf16 pair
__device__ __forceinline__ uint32_t upper_pair(float x, float y) {
    return __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
}
// what these leave of x
__device__ __forceinline__ float below_upper(float x) { return x - __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// ... of both, as a bf16 pair
__device__ __forceinline__ uint32_t lower_pair(float x, float y) { return f32x2_to_bf16_pair(below_upper(x), below_upper(y)); }

// The bf16 kernel's part of launch_scan: whether it covers the shape, the
// heads it gives a workgroup, and its launch (state_only: the segments' own
// states into the workspace).
bool scan_mx_supported(int P, int N, const ScanArgs &a);
int scan_mx_heads(int P, int H, int G);
hipError_t launch_scan_mx(int P, int N, const ScanArgs &a, bool state_only, hipStream_t s);
// The bf16 kernels' part of launch_delta_scan (delta_mx.hip): where the workspace
// holds chunks (a.window > 0).
hipError_t launch_delta_mx(int P, int N, const ScanArgs &a, hipStream_t s);

}  // namespace replay
