// sample.hip -- tokens from logits by temperature, top-k, top-p and min-p
// with given random numbers, and the drafts that they reject.
//
// Weights are whole numbers, w_i = rint(2^45 exp((x_i - max) / T)): their
// sums in 64 bits are exact (V <= 2^18), so neither the order in which
// lanes, waves and atomics add nor the split of a row changes a token, and a
// draw next to a border falls on the side that the definition says.  The
// exponential is taken in float64: at 2^45 a float32 one would be off by a
// million units.
//
// Tokens are ordered by logit, largest first, ties by index: the order of
// the composite number (~key << 32 | index), key being the logit's bits made
// monotone.  Top-k and top-p keep a prefix of that order, hence all tokens
// whose composite is at most some bound.  The bound is found without
// sorting the row: a histogram over kBins steps of the distance to the
// maximum finds the step where the prefix ends, and the tokens of that step
// (with top-k: of all steps up to it) are gathered into LDS and sorted
// there; rows where more than kList would have to be (thousands of equal
// logits, or a large k) take a radix selection over the composite's digits.
//
// One workgroup a row; the row comes from HBM once, later passes from the
// caches.
#include "device_common.h"

namespace replay {

namespace {

constexpr int kNT = 1024, kWaves = kNT / 64;
constexpr int kBins = 1024;      // steps of the distance to the maximum, 1/32 of a temperature each; the last takes the rest
constexpr int kList = 4096;      // tokens sorted in LDS
constexpr int kIndexBits = 18;   // V <= 2^18
constexpr int kOneBits = 45;     // the largest logit's weight is 2^45

struct Lds {
    uint64_t list[kList];
    uint64_t mass[kBins];
    uint32_t count[kBins];
    uint64_t wave[kWaves];
    uint64_t pick[4];
    uint32_t n, flag;
};

__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 is 0
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t composite(float x, int i) { return ((uint64_t)~key_of(x) << 32) | (uint32_t)i; }
__device__ __forceinline__ float value_at(uint64_t comp) { return value_of(~(uint32_t)(comp >> 32)); }

// rint(2^45 2^t), t <= 0: 2^f by its Taylor series in f ln 2, |f| <= 1/2
// (13 terms: 2e-16 of the value), rounded to a whole number by adding 2^52.
__device__ __forceinline__ uint64_t weight_of(float x, double top, double scale) {
    const double t = ((double)x - top) * scale;
    if (!(t > -(kOneBits + 2.0))) return 0;
    const double n = rint(t), f = (t - n) * 0.69314718055994530942;
    double p = 1.0 / 479001600.0;
    p = fma(p, f, 1.0 / 39916800.0);
    p = fma(p, f, 1.0 / 3628800.0);
    p = fma(p, f, 1.0 / 362880.0);
    p = fma(p, f, 1.0 / 40320.0);
    p = fma(p, f, 1.0 / 5040.0);
    p = fma(p, f, 1.0 / 720.0);
    p = fma(p, f, 1.0 / 120.0);
    p = fma(p, f, 1.0 / 24.0);
    p = fma(p, f, 1.0 / 6.0);
    p = fma(p, f, 0.5);
    p = fma(p, f, 1.0);
    p = fma(p, f, 1.0);
    const double w = ldexp(p, (int)n + kOneBits) + 0x1p52;
    return __double_as_longlong(w) & ((1ull << 52) - 1);
}

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
    __device__ __forceinline__ bool inside(int i) const { return first(i) >= 0 && first(i) + E <= V; }
    __device__ __forceinline__ u32x4 raw(int i) const { return *reinterpret_cast<const u32x4 *>(base + (size_t)16 * i); }
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
    __device__ __forceinline__ void load(int i, float *x) const {
        if (inside(i)) {
            widen(raw(i), x);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int j = first(i) + e;
                x[e] = -__builtin_inff();
                if (j >= 0 && j < V) x[e] = load_io1<BF16>(base, (size_t)(j + off));
            }
        }
    }
    // f(x, index) for every element, in no order
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        for (int i = threadIdx.x; i < blocks; i += kNT) {
            float x[E];
            load(i, x);
#pragma unroll
            for (int e = 0; e < E; ++e) f(x[e], first(i) + e);
        }
    }
};

__device__ __forceinline__ uint64_t wave_sum(uint64_t v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor((unsigned long long)v, d);
    return v;
}
__device__ __forceinline__ uint64_t wave_upto(uint64_t v) {   // inclusive, by lane
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t o = __shfl_up((unsigned long long)v, d);
        if ((int)(threadIdx.x & 63) >= d) v += o;
    }
    return v;
}

// The sum of v over the threads before this one (and over all, in *total).
// Every thread calls; l.wave is free afterwards.
__device__ __forceinline__ uint64_t before(Lds &l, uint64_t v, uint64_t *total) {
    const int w = threadIdx.x >> 6;
    const uint64_t upto = wave_upto(v);
    if ((threadIdx.x & 63) == 63) l.wave[w] = upto;
    __syncthreads();
    uint64_t ahead = 0, all = 0;
    for (int i = 0; i < kWaves; ++i) {
        const uint64_t s = l.wave[i];
        if (i < w) ahead += s;
        all += s;
    }
    __syncthreads();
    *total = all;
    return ahead + upto - v;
}

// list[0, n) in ascending order; entries n .. the next power of two are overwritten.
__device__ void sort_list(Lds &l, int n) {
    int m = 1;
    while (m < n) m <<= 1;
    for (int i = n + threadIdx.x; i < m; i += kNT) l.list[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= m; k <<= 1)
        for (int j = k >> 1; j; j >>= 1) {
            for (int t = threadIdx.x; t < m / 2; t += kNT) {
                const int lo = 2 * t - (t & (j - 1)), hi = lo + j;
                const uint64_t a = l.list[lo], b = l.list[hi];
                if ((a > b) == ((lo & k) == 0)) {
                    l.list[lo] = b;
                    l.list[hi] = a;
                }
            }
            __syncthreads();
        }
}

// Where a prefix of the order ends.
struct Cut {
    uint64_t last;   // the composite of its last token
    uint64_t mass;   // its weight
};

// The prefix of the first `want` tokens (BY_MASS: of the fewest tokens that
// weigh at least `want`), by the composite's digits, high to low.  `want` is
// between 1 and the row's number of tokens (weight).
template <bool BF16, bool BY_MASS>
__device__ Cut radix_cut(Lds &l, const Logits<BF16> &row, double top, double scale, uint64_t want) {
    uint64_t prefix = 0, mass = 0;
    // 32 bits of key, then the index
    constexpr int kDigits = 7;
    for (int d = 0; d < kDigits; ++d) {
        const int shift = d < 4 ? 56 - 8 * d : 16 - 8 * (d - 4);
        const uint64_t above = d == 0 ? 0 : ~0ull << (d < 4 ? shift + 8 : (d == 4 ? 32 : shift + 8));
        if (threadIdx.x < 256) {
            l.mass[threadIdx.x] = 0;
            l.count[threadIdx.x] = 0;
        }
        __syncthreads();
        row.each([&](float x, int i) {
            if (i < 0 || i >= row.V) return;
            const uint64_t c = composite(x, i);
            if ((c & above) != prefix) return;
            const int digit = (int)(c >> shift) & 255;
            atomicAdd(&l.count[digit], 1u);
            const uint64_t w = weight_of(x, top, scale);
            if (w) atomicAdd((unsigned long long *)&l.mass[digit], (unsigned long long)w);
        });
        __syncthreads();
        uint64_t w = 0, c = 0, all;
        if (threadIdx.x < 256) {
            w = l.mass[threadIdx.x];
            c = l.count[threadIdx.x];
        }
        const uint64_t v = BY_MASS ? w : c;
        const uint64_t ahead = before(l, v, &all), massed = before(l, w, &all);
        if (threadIdx.x < 256 && ahead < want && want <= ahead + v) {
            l.pick[0] = threadIdx.x;
            l.pick[1] = want - ahead;
            l.pick[2] = massed;
        }
        __syncthreads();
        prefix |= l.pick[0] << shift;
        want = l.pick[1];
        mass += l.pick[2];
        __syncthreads();
    }
    // the last digit's token is one
    return {prefix, mass + weight_of(value_at(prefix), top, scale)};
}

// Step of the distance to the maximum: monotone in x.
__device__ __forceinline__ int step_of(float x, float top, float rate) {
    return (int)fminf((top - x) * rate, (float)(kBins - 1));
}

// Histogram of the row over the steps.
template <bool BF16, bool MASS>
__device__ void histogram(Lds &l, const Logits<BF16> &row, float top, float rate, double scale) {
    l.count[threadIdx.x] = 0;
    l.mass[threadIdx.x] = 0;
    __syncthreads();
    row.each([&](float x, int i) {
        if (i < 0 || i >= row.V) return;
        const int s = step_of(x, top, rate);
        atomicAdd(&l.count[s], 1u);
        if constexpr (MASS) {
            const uint64_t w = weight_of(x, (double)top, scale);
            if (w) atomicAdd((unsigned long long *)&l.mass[s], (unsigned long long)w);
        }
    });
    __syncthreads();
}

// The composites of the row's tokens in steps lo..hi, sorted.
template <bool BF16>
__device__ int gather(Lds &l, const Logits<BF16> &row, float top, float rate, int lo, int hi) {
    if (threadIdx.x == 0) l.n = 0;
    __syncthreads();
    row.each([&](float x, int i) {
        const int s = step_of(x, top, rate);
        if (s >= lo && s <= hi && i >= 0 && i < row.V) {
            const uint32_t at = atomicAdd(&l.n, 1u);
            if (at < (uint32_t)kList) l.list[at] = composite(x, i);
        }
    });
    __syncthreads();
    const int n = l.n < (uint32_t)kList ? (int)l.n : kList;
    sort_list(l, n);
    return n;
}

// floor(u mass), within 0 .. mass - 1
__device__ __forceinline__ uint64_t target_of(float u, uint64_t mass) {
    const double x = floor((double)u * (double)mass);
    const uint64_t t = x > 0.0 ? (x < (double)mass ? (uint64_t)x : mass) : 0;
    return t < mass ? t : mass - 1;
}

constexpr int kEach = kList / kNT;   // list entries a thread holds, in order

template <bool BF16>
__global__ __launch_bounds__(kNT) void sample_kernel(SampleArgs a) {
    __shared__ Lds l;
    const int r = blockIdx.x, b = r / a.W, tid = threadIdx.x;
    const Logits<BF16> row(a.logits, r, a.stride, a.V);
    const float T = a.temperature ? a.temperature[b] : 1.f, u = a.u[r];

    // the maximum and the first token that has it
    uint64_t best = ~0ull;
    bool bad = false;
    row.each([&](float x, int i) {
        bad |= !(x < __builtin_inff());   // NaN or +infinity
        const uint64_t c = composite(x, i);
        best = (i >= 0 && i < row.V && c < best) ? c : best;
    });
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)best, d);
        best = o < best ? o : best;
    }
    if (tid == 0) l.flag = 0;
    __syncthreads();
    if (bad) l.flag = 1;
    if ((tid & 63) == 0) l.wave[tid >> 6] = best;
    __syncthreads();
    bad = l.flag != 0;
    for (int i = 0; i < kWaves; ++i) best = l.wave[i] < best ? l.wave[i] : best;
    __syncthreads();
    const float top = value_at(best);
    if (bad || !(top > -__builtin_inff()) || !(T >= 0.f && T < __builtin_inff()) || u != u || T == 0.f) {
        const bool greedy = !bad && top > -__builtin_inff() && T == 0.f;
        if (tid == 0) {
            a.tokens[r] = greedy ? (int32_t)(uint32_t)best : -1;
            if (a.probs) a.probs[r] = greedy ? 1.f : 0.f;
        }
        return;
    }

    const double dtop = (double)top, scale = 1.4426950408889634074 / (double)T;
    const float rate = fminf(32.f / T, 3e38f);
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.f, mp = a.min_p ? a.min_p[b] : 0.f;
    const bool by_k = k > 0 && k < a.V, by_p = p < 1.f;
    const uint64_t least = mp > 0.f ? (uint64_t)ceil(fmin((double)mp, 1.0) * (double)(1ull << kOneBits)) : 0;
    uint64_t last = ~0ull;   // composites up to this one are kept
    // the weight that top-p asks for of one that is kept so far
    auto share = [&](uint64_t mass) {
        const double x = ceil((double)p * (double)mass);
        return x >= 1.0 ? (uint64_t)x : 1ull;
    };
    if (by_k) {
        histogram<BF16, false>(l, row, top, rate, scale);
        uint64_t all;
        const uint64_t ahead = before(l, l.count[tid], &all);
        if (ahead < (uint64_t)k && (uint64_t)k <= ahead + l.count[tid]) {
            l.pick[0] = tid;
            l.pick[1] = ahead + l.count[tid];
        }
        __syncthreads();
        if (l.pick[1] <= (uint64_t)kList) {
            // everything that can be kept is in LDS
            gather<BF16>(l, row, top, rate, 0, (int)l.pick[0]);
            uint64_t w[kEach], sum = 0, mass;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int i = tid * kEach + e;
                w[e] = i < k ? weight_of(value_at(l.list[i]), dtop, scale) : 0;
                sum += w[e];
            }
            uint64_t at = before(l, sum, &mass);
            const uint64_t want = by_p ? share(mass) : ~0ull;
            // those that are kept, by their index: (index, weight) pairs
            uint64_t kept = 0, total;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const bool in = w[e] > 0 && at < want && w[e] >= least;
                at += w[e];
                w[e] = in ? ((l.list[tid * kEach + e] & ((1ull << kIndexBits) - 1)) << (kOneBits + 1)) | w[e] : 0;
                kept += in;
            }
            const uint64_t slot = before(l, kept, &total);
            uint64_t s = slot;
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                if (w[e]) l.list[s++] = w[e];
            __syncthreads();
            sort_list(l, (int)total);
            sum = 0;
            constexpr uint64_t kWeight = (1ull << (kOneBits + 1)) - 1;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int i = tid * kEach + e;
                w[e] = i < (int)total ? l.list[i] & kWeight : 0;
                sum += w[e];
            }
            at = before(l, sum, &mass);
            const uint64_t target = target_of(u, mass);
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (at <= target && target < at + w[e]) {
                    a.tokens[r] = (int32_t)(l.list[tid * kEach + e] >> (kOneBits + 1));
                    if (a.probs) a.probs[r] = (float)((double)w[e] / (double)mass);
                }
                at += w[e];
            }
            return;
        }
        const Cut cut = radix_cut<BF16, false>(l, row, dtop, scale, (uint64_t)k);
        last = cut.last;
        if (by_p) {
            const Cut c2 = radix_cut<BF16, true>(l, row, dtop, scale, share(cut.mass));
            last = c2.last < last ? c2.last : last;
        }
    } else if (by_p) {
        histogram<BF16, true>(l, row, top, rate, scale);
        uint64_t all;
        const uint64_t m = l.mass[tid], ahead = before(l, m, &all), want = share(all);
        if (ahead < want && want <= ahead + m) {
            l.pick[0] = tid;
            l.pick[1] = ahead;
        }
        __syncthreads();
        const int s = (int)l.pick[0];
        const uint64_t passed = l.pick[1];
        if (l.count[s] <= (uint32_t)kList) {
            const int n = gather<BF16>(l, row, top, rate, s, s);
            uint64_t w[kEach], sum = 0;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int i = tid * kEach + e;
                w[e] = i < n ? weight_of(value_at(l.list[i]), dtop, scale) : 0;
                sum += w[e];
            }
            uint64_t at = passed + before(l, sum, &all);
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (at < want && want <= at + w[e]) l.pick[2] = l.list[tid * kEach + e];
                at += w[e];
            }
            __syncthreads();
            last = l.pick[2];
        } else {
            last = radix_cut<BF16, true>(l, row, dtop, scale, want).last;
        }
    }

    // the draw, in the order of the indexes: each wavefront sums a run of
    // blocks, the run that holds the target is split again, down to a block a lane
    const int w = tid >> 6, lane = tid & 63;
    auto kept = [&](float x, int i) -> uint64_t {
        if (composite(x, i) > last) return 0;
        const uint64_t v = weight_of(x, dtop, scale);
        return v >= least ? v : 0;
    };
    int lo = 0, hi = row.blocks;
    uint64_t target = 0, mass = 0;
    while (true) {
        const int run = hi - lo > 64 ? ((hi - lo + kWaves - 1) / kWaves + 63) / 64 * 64 : 64;
        const int from = lo + w * run, to = from + run < hi ? from + run : hi;
        uint64_t sum = 0;
        for (int i = from + lane; i < to; i += 64) {
            float x[Logits<BF16>::E];
            row.load(i, x);
#pragma unroll
            for (int e = 0; e < Logits<BF16>::E; ++e) sum += kept(x[e], row.first(i) + e);
        }
        const bool narrow = hi - lo <= 64;   // one block a lane of wavefront 0
        if (narrow) {
            if (w == 0) {
                if (mass == 0) {   // a row of 64 blocks or fewer
                    mass = wave_sum(sum);
                    target = target_of(u, mass);
                }
                uint64_t at = wave_upto(sum) - sum;
                if (at <= target && target < at + sum) {
                    float x[Logits<BF16>::E];
                    row.load(lo + lane, x);
#pragma unroll
                    for (int e = 0; e < Logits<BF16>::E; ++e) {
                        const uint64_t v = kept(x[e], row.first(lo + lane) + e);
                        if (at <= target && target < at + v) {
                            a.tokens[r] = row.first(lo + lane) + e;
                            if (a.probs) a.probs[r] = (float)((double)v / (double)mass);
                        }
                        at += v;
                    }
                }
            }
            return;
        }
        sum = wave_sum(sum);
        if (lane == 0) l.wave[w] = sum;
        __syncthreads();
        if (mass == 0) {
            for (int i = 0; i < kWaves; ++i) mass += l.wave[i];
            target = target_of(u, mass);
        }
        int next = 0;
        for (; next < kWaves - 1; ++next) {
            if (target < l.wave[next]) break;
            target -= l.wave[next];
        }
        __syncthreads();
        lo += next * run;
        hi = lo + run < hi ? lo + run : hi;
    }
}

// Position w of a window stays while the token drawn before it is the one
// that was fed there.
__global__ __launch_bounds__(256) void reject_kernel(const int32_t *tokens, const int32_t *fed, int32_t *n_reject, int B,
                                                     int W) {
    const int b = blockIdx.x * 256 + threadIdx.x;
    if (b >= B) return;
    int kept = 1;
    while (kept < W && tokens[(size_t)b * W + kept - 1] == fed[(size_t)b * W + kept]) ++kept;
    n_reject[b] = W - kept;
}

}  // namespace

size_t sample_workspace(int, int, int) { return 0; }

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) {
    const unsigned rows = (unsigned)((int64_t)a.B * a.W);
    if (a.bf16)
        sample_kernel<true><<<rows, kNT, 0, s>>>(a);
    else
        sample_kernel<false><<<rows, kNT, 0, s>>>(a);
    if (a.n_reject) reject_kernel<<<(a.B + 255) / 256, 256, 0, s>>>(a.tokens, a.fed, a.n_reject, a.B, a.W);
    return hipGetLastError();
}

}  // namespace replay
