// delta_mx.h -- what the two forms of the bf16 gated delta scan (delta_mx.hip,
// delta_few.hip) share: the workspace's layout, operands, and the rule token by
// token for chunks with values that are no numbers.
#pragma once

#include "scan_common.h"

namespace replay {

constexpr int kQ = kScanChunk;
static_assert(kQ == 64, "two blocks of 32 tokens");

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float acc4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// A head's chunk in the workspace: T's operands (tiles of 16 tokens by steps of
// 32, three parts each), G's, g and e, and whether the chunk holds a value
// that is no number.  Operand x < 4 is tile x at the step its tokens are in,
// the two behind them are tiles 2 and 3 at step 0.
constexpr int kFrag = 1024, kFrags = 6;
constexpr int kTBytes = kFrags * 3 * kFrag, kGBytes = kTBytes;
constexpr int kImage = kTBytes + kGBytes + 2 * kQ * 4;
constexpr int kSlot = (kImage + 16 + 255) / 256 * 256;
static_assert(kImage % 16 == 0, "whole pieces");
__host__ __device__ constexpr int frag(int tile, int step) { return step == tile >> 1 ? tile : tile + 2; }
// A product of two operands in three parts: parts kA[z] and kB[z], the largest first.
// What is left out is 2^-20 of a term at most.
constexpr int kProducts = 6, kA[kProducts] = {0, 0, 1, 1, 0, 2}, kB[kProducts] = {0, 1, 0, 1, 2, 0};

__device__ __forceinline__ acc4 mma16(bf8 a, bf8 b, acc4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ acc4 mma4(float a, float b, acc4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ bool odd_pair(uint32_t w) {   // a bf16 pair with a value that is no number
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Eight (four) floats as PARTS operands that hold 8 bits each, the last one rounded.
template <int PARTS>
__device__ __forceinline__ void split(const acc4 &lo, const acc4 &hi, bf8 *out) {
    float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
    for (int z = 0; z < PARTS; ++z) {
        u32x4 w;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (z + 1 < PARTS) {
                w[r] = upper_pair(x[2 * r], x[2 * r + 1]);
                x[2 * r] = below_upper(x[2 * r]);
                x[2 * r + 1] = below_upper(x[2 * r + 1]);
            } else {
                w[r] = f32x2_to_bf16_pair(x[2 * r], x[2 * r + 1]);
            }
        }
        out[z] = __builtin_bit_cast(bf8, w);
    }
}

template <int PARTS>
__device__ __forceinline__ void split4(const acc4 &a, u32x2 *out) {
    float x[4] = {a[0], a[1], a[2], a[3]};
#pragma unroll
    for (int z = 0; z < PARTS; ++z)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            if (z + 1 < PARTS) {
                out[z][r] = upper_pair(x[2 * r], x[2 * r + 1]);
                x[2 * r] = below_upper(x[2 * r]);
                x[2 * r + 1] = below_upper(x[2 * r + 1]);
            } else {
                out[z][r] = f32x2_to_bf16_pair(x[2 * r], x[2 * r + 1]);
            }
        }
}

__device__ __forceinline__ bf8 frag16(const uint8_t *m) { return __builtin_bit_cast(bf8, *reinterpret_cast<const u32x4 *>(m)); }
// Rows of k and q in LDS: the sixteen 8-byte pieces of 128 bytes are permuted by the
// row's number, so that 16 rows' equal pieces, and 4 rows' 4 neighbouring ones, lie
// in distinct banks.
__device__ __forceinline__ int turn(int row) { return (row & 3) << 2 | (row >> 2 & 3); }
// an operand's two pieces
__device__ __forceinline__ bf8 row8(const uint8_t *first, const uint8_t *second) {
    const u32x2 lo = *reinterpret_cast<const u32x2 *>(first), hi = *reinterpret_cast<const u32x2 *>(second);
    return __builtin_bit_cast(bf8, u32x4{lo[0], lo[1], hi[0], hi[1]});
}
__device__ __forceinline__ s16x4 col4(const uint8_t *m) {
    typedef __attribute__((address_space(3))) s16x4 lds4;
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)m);
}

__device__ __forceinline__ void put_frag(uint8_t *to, bf8 x) { *reinterpret_cast<u32x4 *>(to) = __builtin_bit_cast(u32x4, x); }


// A chunk token by token, by a wavefront for 16 columns.  The state stays in
// s_out, S this lane's first place there (columns 16 t + 4 lg ..).
template <int P, int N>
__device__ __forceinline__ void by_token(const ScanArgs &s, const uint8_t *rows_k, const uint8_t *rows_q, float *S, int t0, int n, int h, int p, int lane) {
    const int lg = lane >> 4;
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
        const float al = s.a[(size_t)(t0 + t) * s.H + h], be = s.dt[(size_t)(t0 + t) * s.H + h];
        const size_t o = ((size_t)(t0 + t) * s.H + h) * P + p;
        const uint8_t *k = rows_k + t * 2 * N, *q = rows_q + t * 2 * N;
        const int f = turn(t) << 3;
        float dot = 0.f, y = 0.f;
#pragma unroll 1
        for (int i = 0; i < N / 4; ++i) dot = fmaf(S[16 * (i / 4) + i % 4], load_io1<true>(k + ((32 * (i / 4) + 8 * lg) ^ f), i % 4), dot);
        dot += __shfl_xor(dot, 16);
        dot += __shfl_xor(dot, 32);
        const float u = be * fmaf(-al, dot, load_io1<true>(s.v, o));
#pragma unroll 1
        for (int i = 0; i < N / 4; ++i) {
            const float x = fmaf(u, load_io1<true>(k + ((32 * (i / 4) + 8 * lg) ^ f), i % 4), al * S[16 * (i / 4) + i % 4]);
            S[16 * (i / 4) + i % 4] = x;
            y = fmaf(x, load_io1<true>(q + ((32 * (i / 4) + 8 * lg) ^ f), i % 4), y);
        }
        y += __shfl_xor(y, 16);
        y += __shfl_xor(y, 32);
        if (lg == 0) static_cast<uint16_t *>(s.y)[o] = (uint16_t)f32_to_bf16_bits(y);
    }
}

// From chunk to chunk of a window where heads are few (delta_few.hip).
hipError_t launch_delta_few(int P, int N, const ScanArgs &a, hipStream_t s);

}  // namespace replay
