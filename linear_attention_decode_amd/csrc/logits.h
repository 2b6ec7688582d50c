// logits.h -- rows of logits and their order, as sampling (sample.hip) and
// token scores (logprobs.hip) read them: by logit, largest first, equal ones
// by index, which is the order of the composite number (~key << 32 | index),
// key being the logit's bits made monotone.
#pragma once

#include "device_common.h"
#include "prompt.h"

namespace replay {

__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 is 0
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t composite(float x, int i) { return ((uint64_t)~key_of(x) << 32) | (uint32_t)i; }
__device__ __forceinline__ float value_at(uint64_t comp) { return value_of(~(uint32_t)(comp >> 32)); }

// A row in 16-byte blocks on 16-byte boundaries: block i holds elements
// E i - off .. E i - off + E - 1; those outside the row read as -infinity,
// which weighs nothing.
template <bool BF16>
struct Logits {
    static constexpr int E = BF16 ? 8 : 4;
    const char *base;   // of block 0
    int V, off, blocks;
    __device__ __forceinline__ Logits(const void *logits, int64_t row, int64_t stride, int V_) : V(V_) {
        const char *p = static_cast<const char *>(logits) + row * stride * (BF16 ? 2 : 4);
        const uint32_t mis = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);
        base = p - mis;
        off = mis / (BF16 ? 2 : 4);
        blocks = (off + V + E - 1) / E;
    }
    __device__ __forceinline__ int first(int i) const { return E * i - off; }
    __device__ __forceinline__ void widen(u32x4 r, float *x) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (BF16) {
                x[2 * e] = bf16_bits_to_f32(r[e] & 0xffffu);
                x[2 * e + 1] = bf16_bits_to_f32(r[e] >> 16);
            } else {
                x[e] = __uint_as_float(r[e]);
            }
        }
    }
    // block i, whichever of its elements lie in the row
    __device__ __forceinline__ u32x4 load_edge(int i) const {
        u32x4 r = none();
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int j = first(i) + e;
            if (j < 0 || j >= V) continue;
            if constexpr (BF16) {
                const uint32_t x = reinterpret_cast<const uint16_t *>(base)[(size_t)(j + off)];
                r[e / 2] = e & 1 ? (r[e / 2] & 0xffffu) | (x << 16) : (r[e / 2] & 0xffff0000u) | x;
            } else {
                r[e] = reinterpret_cast<const uint32_t *>(base)[(size_t)(j + off)];
            }
        }
        return r;
    }
    static __device__ __forceinline__ u32x4 none() {
        constexpr uint32_t x = BF16 ? 0xff80ff80u : 0xff800000u;
        return u32x4{x, x, x, x};
    }
};

}  // namespace replay
