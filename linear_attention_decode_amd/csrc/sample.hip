// sample.hip -- tokens from logits by temperature, top-k, top-p and min-p
// with given random numbers, and the drafts that they reject.
//
// Weights are whole numbers, w_i = rint(2^45 exp((x_i - max) / T)): their
// sums in 64 bits are exact (V <= 2^18), so neither the order in which
// lanes, waves and atomics add nor the split of a row changes a token.  The
// exponential is taken in float64, to some 6e-16 of itself: 2 or 3 in 1000 of
// the largest weights (above 2^43) are one unit off the definition's, all the
// others are its own; borders between tokens lie where these weights put them,
// a part in 2^45 of the largest weight a token from the definition's at most.
// A float32 exponential would be off by a million units.
//
// Tokens are ordered by logit, largest first, ties by index: the order of
// their composites (logits.h).  Top-k and top-p keep a prefix of that order,
// hence all tokens whose composite is at most some bound.
//
// One workgroup a row.  Where filters leave few tokens, these are gathered
// into LDS: a second pass that loads again the blocks alone whose maximum,
// kept from the first, says that they hold one.  Whom to gather is found from the
// threads' own maxima, four each: of 2048 of them, the k-th largest is no
// larger than the k-th largest logit, so that all of the top k lie within the
// step (of 1/16 of a temperature) where it does; for k = 50 that gathers some
// 60 tokens, for k = 1000 some 1400.  Rows that this does not settle (top-p
// alone, thousands of equal logits, k past 2048) take a histogram of the
// steps over all tokens and gather the step that the prefix ends in, and
// where that is too full to sort, a radix selection over the composite's
// digits.
//
// Bound by the chain of steps of a row (two passes, a dozen barriers, sorts of
// few tokens) and by the float64 exponentials, more than by reading the
// logits.  Rows of 131072 in bf16, 256 of them, all filters on: 39 us, 1.7
// TB/s of 67 MB (the copy rate would take 14 us); top-k of 50 alone 29 us, of
// 1000 35 us, of 5000 120 us; min-p of .05 25 us; greedy 31 us; top-p of .98
// alone 179 us and no filter 75 us, where every token's weight is computed and
// every token counts.  One row 22 us.  512 threads a row: 1024 leave half the
// registers, and spill.
#include "logits.h"

namespace replay {

namespace {

constexpr int kNT = kSampleNT, kWaves = kNT / 64;   // 1024 threads would have 128 registers each, 50 too few
constexpr int kBins = kNT;       // steps of the distance to the maximum, 1/16 of a temperature each; the last takes the rest
constexpr float kSteps = kBins / 32;   // steps of a temperature
constexpr int kList = 4096;      // tokens sorted in LDS
constexpr int kIndexBits = 18;   // V <= 2^18
constexpr int kOneBits = 45;     // the largest logit's weight is 2^45

constexpr int kFine = 16;        // entries of the exponential's table: one for each pair of banks, so that no two lanes wait

struct Lds {
    uint64_t list[kList], part[kList];
    double fine[kFine];          // 2^(j / 16)
    uint64_t mass[kBins];
    uint32_t count[kBins];
    uint64_t wave[kWaves];
    uint64_t pick[4];
    uint64_t k_step, k_mass;     // the step that a k past the list ends in, and what its prefix weighs in it
    uint64_t p_want;             // what top-p asks for behind such a k
    u32x4 edge[2];               // the row's first and last block, where they are not whole
    uint32_t n, listed, flag;
};

// The thread's number, hidden from the compiler's view of what a loop leaves
// unchanged: it would keep every address of every pass in a register from
// the kernel's start on, 70 more than there are.
__device__ __forceinline__ int thread() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// the bits of the least bf16 that is not below x (x no NaN)
__device__ __forceinline__ uint32_t bf16_above(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u >> 31 ? u : u + 0xffffu) >> 16;
}

// rint(2^45 exp((x - top) / T)), scale = 16 log2(e) / T.  2^(n / 16) from
// l.fine and a shift, the rest, y = f ln 2 / 16 with |f| <= 1/2, by its
// Taylor series (y^7 / 5040 < 5e-16).  The rounding to a whole number is the
// addition of 2^52, that of n the addition of 1.5 2^52, whose low word is n.
// Distances past 48 powers of two, infinite ones among them, round to nothing there.
__device__ __forceinline__ uint64_t weight_of(const double *fine, float x, double top, double scale) {
    const double t = fmax(((double)x - top) * scale, -(double)kFine * (kOneBits + 3));
    const double shifted = t + 0x1.8p52;
    const int n = (int)(uint32_t)__double_as_longlong(shifted);
    const double f = t - (shifted - 0x1.8p52);
    constexpr double c = 0.69314718055994530942 / kFine;
    double p = c * c * c * c * c * c / 720;
    p = fma(p, f, c * c * c * c * c / 120);
    p = fma(p, f, c * c * c * c / 24);
    p = fma(p, f, c * c * c / 6);
    p = fma(p, f, c * c / 2);
    p = fma(p, f, c);
    const double b = fine[n & (kFine - 1)];
    p = fma(b * f, p, b);
    const uint64_t e = (uint64_t)(uint32_t)((n >> 4) + kOneBits) << 52;
    return (uint64_t)__double_as_longlong(__longlong_as_double(__double_as_longlong(p) + e) + 0x1p52) & ((1ull << 52) - 1);
}

// The row as the threads go over it: block t kNT + tid in turn t.  Whole
// blocks come through a buffer resource over them alone; the first and the
// last, where they are not whole, from LDS.
constexpr int kTurns = 64;   // turns whose block maxima a thread keeps: 256 K bf16, 128 K float32 logits
template <bool BF16>
struct Row : Logits<BF16> {
    using L = Logits<BF16>;
    int turns, lo, hi;   // blocks lo .. hi - 1 are whole
    const u32x4 *edge;
    __amdgpu_buffer_rsrc_t whole;
    // every thread calls; the edges are there behind the next barrier
    __device__ __forceinline__ Row(Lds &l, const void *logits, int64_t row, int64_t stride, int V)
        : L(logits, row, stride, V), turns((L::blocks + kNT - 1) / kNT), lo(L::off ? 1 : 0), hi((L::off + V) / L::E),
          edge(l.edge) {
        whole = make_rsrc(L::base + 16 * lo, hi > lo ? (uint32_t)(hi - lo) * 16u : 0u);
        if (threadIdx.x < 2) l.edge[threadIdx.x] = L::load_edge(threadIdx.x ? L::blocks - 1 : 0);
    }
    // block i as far as it is whole, and what it is
    __device__ __forceinline__ u32x4 load_block(int i) const {
        return __builtin_amdgcn_raw_buffer_load_b128(whole, (uint32_t)(i - lo) * 16u, 0, 0);
    }
    __device__ __forceinline__ u32x4 mend(int i, u32x4 r) const {
        if (i < lo || i >= hi) r = i < L::blocks ? edge[i < lo ? 0 : 1] : L::none();
        return r;
    }
    // U turns from t on, all loads in flight together
    template <int U>
    __device__ __forceinline__ void load_turns(int t, u32x4 *r) const {
        const int i0 = t * kNT + thread();
#pragma unroll
        for (int v = 0; v < U; ++v) r[v] = load_block(i0 + v * kNT);
        if ((t + U) * kNT > hi || (t == 0 && lo)) {
#pragma unroll
            for (int v = 0; v < U; ++v) r[v] = mend(i0 + v * kNT, r[v]);
        }
    }
    // f(turn, the elements of a block, the first one's index) for every turn,
    // four turns' loads ahead; elements outside the row are -infinity
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        constexpr int U = 4;
        const int tid = thread();
        u32x4 r[U], ahead[U];
        load_turns<U>(0, ahead);
#pragma unroll 1
        for (int t = 0; t < turns; t += U) {
#pragma unroll
            for (int v = 0; v < U; ++v) r[v] = ahead[v];
            load_turns<U>(t + U, ahead);   // past the row: nothing is read
#pragma unroll 1
            for (int v = 0; v < U; ++v) {
                if (t + v >= turns) break;
                float x[L::E];
                L::widen(v < 2 ? (v ? r[1] : r[0]) : (v == 2 ? r[2] : r[3]), x);
                f(t + v, x, L::first((t + v) * kNT + tid));
            }
        }
    }
};

// Sums over the lanes up to this one, by moves between lanes that pass no
// memory (within rows of 16, then from row to row).  64 summands of 22 bits
// stay within 32, so a 64-bit sum goes in three parts.
__device__ __forceinline__ uint32_t lanes_upto(uint32_t v) {
    v += __builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false);
    return v;
}
__device__ __forceinline__ uint64_t wave_upto(uint64_t v) {
    constexpr uint32_t m = (1u << 22) - 1;
    const uint64_t a = lanes_upto((uint32_t)v & m), b = lanes_upto((uint32_t)(v >> 22) & m), c = lanes_upto((uint32_t)(v >> 44));
    return a + (b << 22) + (c << 44);
}
__device__ __forceinline__ uint64_t wave_sum(uint64_t v) {   // the same in every lane
    const uint64_t all = wave_upto(v);
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(all >> 32), 63) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)all, 63);
}

// The sum of v over the threads before this one (and over all, in *total).
// Every thread calls; l.wave is free afterwards.
__device__ __forceinline__ uint64_t before(Lds &l, uint64_t v, uint64_t *total) {
    const int tid = thread(), w = tid >> 6;
    const uint64_t upto = wave_upto(v);
    if ((tid & 63) == 63) l.wave[w] = upto;
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

// list[0, n), of kList places, in ascending order; entries n .. the next power of two are
// overwritten.  Exchanges over up to 64 entries stay within the 128 that a
// wavefront's own threads hold, and need no barrier of the workgroup.
__device__ void sort_list(uint64_t *list, int n) {
    const int tid = thread();
    int m = 2;
    while (m < n) m <<= 1;
    for (int i = n + tid; i < m; i += kNT) list[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= m; k <<= 1)
        for (int j = k >> 1; j; j >>= 1) {
            for (int t = tid; t < m / 2; t += kNT) {
                const int lo = 2 * t - (t & (j - 1)), hi = lo + j;
                const uint64_t a = list[lo], b = list[hi];
                if ((a > b) == ((lo & k) == 0)) {
                    list[lo] = b;
                    list[hi] = a;
                }
            }
            const int next = j > 1 ? j >> 1 : k;
            if (j > 64 || next > 64) {
                __syncthreads();
            } else {
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        }
    __syncthreads();
}

// Where a prefix of the order ends.
struct Cut {
    uint64_t last;   // the composite of its last token
    uint64_t mass;   // its weight
};

// The prefix of the first `want` tokens (by_mass: of the fewest tokens that
// weigh at least `want`), by the composite's digits, high to low.  `want` is
// between 1 and the row's number of tokens (weight).
template <class R>
__device__ Cut radix_cut(Lds &l, const R &row, bool by_mass, double top, double scale, uint64_t want) {
    uint64_t prefix = 0, mass = 0;
    constexpr int kDigits = 7;   // 32 bits of key, then the index
#pragma unroll 1
    for (int d = 0; d < kDigits; ++d) {
        const int shift = d < 4 ? 56 - 8 * d : 16 - 8 * (d - 4);
        const uint64_t above = d == 0 ? 0 : ~0ull << (d < 4 ? shift + 8 : (d == 4 ? 32 : shift + 8));
        if (threadIdx.x < 256) {
            l.mass[threadIdx.x] = 0;
            l.count[threadIdx.x] = 0;
        }
        __syncthreads();
        row.each([&](int, const float *x, int i) {
#pragma unroll 1
            for (int e = 0; e < R::E; ++e, ++i) {
                const uint64_t c = composite(x[e], i);
                if (i < 0 || i >= row.V || (c & above) != prefix) continue;
                const int digit = (int)(c >> shift) & 255;
                atomicAdd(&l.count[digit], 1u);
                const uint64_t w = weight_of(l.fine, x[e], top, scale);
                if (w) atomicAdd((unsigned long long *)&l.mass[digit], (unsigned long long)w);
            }
        });
        __syncthreads();
        uint64_t w = 0, c = 0, all;
        if (threadIdx.x < 256) {
            w = l.mass[threadIdx.x];
            c = l.count[threadIdx.x];
        }
        const uint64_t v = by_mass ? w : c;
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
    return {prefix, mass + weight_of(l.fine, value_at(prefix), top, scale)};
}

// Step of the distance to the maximum: monotone in x.
__device__ __forceinline__ int step_of(float x, float top, float rate) {
    return (int)fminf(fmaxf((top - x) * rate, 0.f), (float)(kBins - 1));
}

// Histogram of the row over the steps: of its tokens, but for the last step's
// (the caller knows how many there are), or of their weight.  Neither the last
// step's tokens nor blocks that weigh nothing are added: on a masked row, or at
// a low temperature, that is nearly all of it, and would queue for one word
// (256 rows of 131072, bf16, 99 % masked: top-p .98 155 -> 70 us, top-k of 1000
// 145 -> 52; T = .1, top-p .98 153 -> 63).
template <class R>
__device__ void histogram(Lds &l, const R &row, bool mass, float top, float rate, double scale) {
    l.count[threadIdx.x] = 0;
    l.mass[threadIdx.x] = 0;
    __syncthreads();
    if (mass) {
        row.each([&](int, const float *x, int) {
            uint64_t w[R::E], some = 0;
#pragma unroll
            for (int e = 0; e < R::E; ++e) some |= w[e] = weight_of(l.fine, x[e], (double)top, scale);
            if (!some) return;
#pragma unroll
            for (int e = 0; e < R::E; ++e)
                atomicAdd((unsigned long long *)&l.mass[step_of(x[e], top, rate)], (unsigned long long)w[e]);
        });
    } else {
        row.each([&](int, const float *x, int i) {
#pragma unroll
            for (int e = 0; e < R::E; ++e) {
                const int s = step_of(x[e], top, rate);
                if (i + e >= 0 && i + e < row.V && s < kBins - 1) atomicAdd(&l.count[s], 1u);
            }
        });
    }
    __syncthreads();
}

// Room for `mine` more entries of a counted list: where this lane's start.
// One addition a wavefront; every lane of it calls.
__device__ __forceinline__ uint32_t reserve(uint32_t *count, uint32_t mine) {
    const uint32_t upto = lanes_upto(mine), all = (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    uint32_t at = 0;
    if (all && (threadIdx.x & 63) == 0) at = atomicAdd(count, all);
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)at) + upto - mine;
}

// The composites of the row's tokens of x >= low (and, where step >= 0, of
// that step alone) into the list, unsorted; their number, or more than the
// list holds (where a float32 block's rounded maximum says so, it may be less:
// the caller then goes the way of too many).  low is above -infinity; `blocks` has a bit for each of the
// first kTurns turns whose block of this thread may hold one.  These blocks
// are listed first, so that the threads share them out evenly, and loaded again.
template <class R>
__device__ int gather(Lds &l, const R &row, uint64_t blocks, float low, int step, float top, float rate) {
    const int tid = thread();
    if (tid < 2) (tid ? l.listed : l.n) = 0;
    __syncthreads();
    uint32_t *list = reinterpret_cast<uint32_t *>(l.part);
    constexpr uint32_t kRoom = 2 * kList;
    uint32_t at = reserve(&l.listed, (uint32_t)__popcll(blocks));
    for (; blocks && at < kRoom; blocks &= blocks - 1, ++at) list[at] = __builtin_ctzll(blocks) * kNT + tid;
    __syncthreads();
    // the listed blocks and all behind those turns; all of the row where they are too many to list
    if (step < 0 && l.listed > (uint32_t)kList) return kList + 1;   // a token of each
    const uint32_t listed = l.listed > kRoom ? 0u : l.listed, from = l.listed > kRoom ? 0u : kTurns * kNT;
    const uint32_t more = (uint32_t)row.blocks > from ? (uint32_t)row.blocks - from : 0u;
    constexpr int U = 4;
#pragma unroll 1
    for (uint32_t j0 = 0; j0 < listed + more; j0 += U * kNT) {
        if (*(volatile uint32_t *)&l.n > (uint32_t)kList) break;   // too many already: how many is not asked
        int block[U];
        u32x4 r[U];
#pragma unroll
        for (int v = 0; v < U; ++v) {
            const uint32_t j = j0 + v * kNT + tid;
            block[v] = j < listed ? (int)list[j] : (j < listed + more ? (int)(j - listed + from) : row.blocks);
        }
#pragma unroll
        for (int v = 0; v < U; ++v) r[v] = row.load_block(block[v]);
#pragma unroll
        for (int v = 0; v < U; ++v) {
            float x[R::E];
            row.widen(row.mend(block[v], r[v]), x);
            uint32_t hits = 0;
#pragma unroll
            for (int e = 0; e < R::E; ++e)
                hits |= x[e] >= low && (step < 0 || step_of(x[e], top, rate) == step) ? 1u << e : 0u;
            if (__ballot(hits != 0)) {
                uint32_t to = reserve(&l.n, (uint32_t)__popc(hits));
#pragma unroll
                for (int e = 0; e < R::E; ++e) {
                    if ((hits >> e & 1u) && to < (uint32_t)kList) l.list[to] = composite(x[e], row.first(block[v]) + e);
                    to += hits >> e & 1u;
                }
            }
        }
    }
    __syncthreads();
    return (int)l.n;
}

// the weight that top-p asks for of this much
__device__ __forceinline__ uint64_t share_of(float p, uint64_t mass) {
    const double x = ceil((double)p * (double)mass);
    return x >= 1.0 ? (uint64_t)x : 1ull;
}

// top - distance, and a little less
__device__ __forceinline__ float below(float top, float distance) {
    return top - distance - (fabsf(top) + distance) * 0x1p-20f;
}

// floor(u mass), within 0 .. mass - 1
__device__ __forceinline__ uint64_t target_of(float u, uint64_t mass) {
    const double x = floor((double)u * (double)mass);
    const uint64_t t = x > 0.0 ? (x < (double)mass ? (uint64_t)x : mass) : 0;
    return t < mass ? t : mass - 1;
}

constexpr int kEach = kList / kNT;   // list entries a thread holds

// The end of the prefix of the list's order that has `want` tokens (by_mass:
// that weighs `want`, with the fewest), and its weight, from the histogram
// (l.count, l.mass) of the list's steps: the step that it ends in is sorted.
__device__ Cut list_cut(Lds &l, int n, bool by_mass, float top, float peak, float rate, double scale, uint64_t want) {
    const int tid = thread();
    const uint64_t m = l.mass[tid], c = l.count[tid], v = by_mass ? m : c;
    uint64_t all;
    const uint64_t passed = before(l, m, &all), ahead = by_mass ? passed : before(l, c, &all);
    if (tid == 0) l.n = 0;
    if (ahead < want && want <= ahead + v) {
        l.pick[0] = tid;
        l.pick[1] = want - ahead;
        l.pick[2] = passed;
    }
    __syncthreads();
    const int step = (int)l.pick[0];
    want = l.pick[1];
    const uint64_t base = l.pick[2];
    for (int i = tid; i < n; i += kNT)
        if (step_of(value_at(l.list[i]), peak, rate) == step) l.part[atomicAdd(&l.n, 1u)] = l.list[i];
    __syncthreads();
    const int members = (int)l.n;
    sort_list(l.part, members);
    uint64_t w[kEach], sum = 0;
    const int per = (members + kNT - 1) / kNT;   // entries a thread takes
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        w[e] = 0;
        if (e >= per) break;
        const int i = tid * per + e;
        w[e] = i < members ? weight_of(l.fine, value_at(l.part[i]), (double)top, scale) : 0;
        sum += w[e];
    }
    uint64_t at = before(l, sum, &all);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        if (e >= per) break;
        const uint64_t i = tid * per + e;
        if (by_mass ? at < want && want <= at + w[e] : i + 1 == want) {
            l.pick[0] = l.part[i];
            l.pick[1] = base + at + w[e];
        }
        at += w[e];
    }
    __syncthreads();
    const Cut cut = {l.pick[0], l.pick[1]};
    __syncthreads();
    return cut;
}

template <bool BF16>
__global__ __launch_bounds__(kNT) void sample_kernel(SampleArgs a) {
    __shared__ Lds l;
    using R = Row<BF16>;
    const int r = blockIdx.x, b = r / a.W, tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
    const float T = a.temperature ? a.temperature[b] : 1.f, u = a.u[r];
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.f, mp = a.min_p ? a.min_p[b] : 0.f;
    const R row(l, a.logits, r, a.stride, a.V);
    if (a.W == 1 && a.n_reject && tid == 0) a.n_reject[b] = 0;   // the one position stays
    if (tid < kFine) l.fine[tid] = exp2((double)tid / kFine);
    __syncthreads();

    // the thread's maximum and the row's; NaN or +infinity
    // a block's maximum as the least bf16 not below it
    float own[4];   // of every fourth turn
#pragma unroll
    for (int t = 0; t < 4; ++t) own[t] = -__builtin_inff();
    uint32_t block_max[kTurns / 2];
    uint32_t odd = 0;
    auto look = [&](u32x4 raw, int t) {
        float x[R::E], m = -__builtin_inff();
        row.widen(raw, x);
#pragma unroll
        for (int e = 0; e < R::E; ++e) m = fmaxf(m, x[e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (BF16) {   // the larger magnitude of each half
                typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
                odd = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, odd),
                                                                             __builtin_bit_cast(u16x2, raw[e] & 0x7fff7fffu)));
            } else {
                odd = odd > (raw[e] & 0x7fffffffu) ? odd : raw[e] & 0x7fffffffu;
            }
        }
        own[t] = fmaxf(own[t], m);
        return m;
    };
#pragma unroll
    for (int t0 = 0; t0 < kTurns; t0 += 16) {
        if (t0 >= row.turns) {
#pragma unroll
            for (int t = 0; t < 16; t += 2) block_max[(t0 + t) / 2] = 0xff80ff80u;
            continue;
        }
        u32x4 raw[16];
        row.template load_turns<16>(t0, raw);
#pragma unroll
        for (int t = 0; t < 16; t += 2)
            block_max[(t0 + t) / 2] = bf16_above(look(raw[t], t & 2)) | bf16_above(look(raw[t + 1], (t & 2) + 1)) << 16;
    }
#pragma unroll 1
    for (int t = kTurns; t < row.turns; t += 4) {
        u32x4 raw[4];
        row.template load_turns<4>(t, raw);
#pragma unroll
        for (int v = 0; v < 4; ++v) (void)look(raw[v], v);
    }
    const bool nan = BF16 ? (odd & 0xffffu) > 0x7f80u || (odd >> 16) > 0x7f80u : odd > 0x7f800000u;
    float top = fmaxf(fmaxf(own[0], own[1]), fmaxf(own[2], own[3]));
#pragma unroll
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (tid == 0) l.flag = 0;
    __syncthreads();
    if (nan) l.flag = 1;
    if (lane == 0) l.wave[w] = __float_as_uint(top);
    __syncthreads();
    const bool bad = l.flag != 0;
    for (int i = 0; i < kWaves; ++i) top = fmaxf(top, __uint_as_float((uint32_t)l.wave[i]));
    __syncthreads();
    const bool finite_top = top > -__builtin_inff() && top < __builtin_inff();
    if (bad || !finite_top || !(T > 0.f && T < __builtin_inff()) || u != u) {
        const bool greedy = !bad && finite_top && u == u && T == 0.f;
        uint32_t i = ~0u;
        if (greedy) {   // the first of the largest
            row.each([&](int, const float *x, int j) {
#pragma unroll
                for (int e = 0; e < R::E; ++e) i = x[e] == top && (uint32_t)(j + e) < i ? (uint32_t)(j + e) : i;
            });
            if (tid == 0) l.n = ~0u;
            __syncthreads();
            atomicMin(&l.n, i);
            __syncthreads();
            i = l.n;
        }
        if (tid == 0) {
            a.tokens[r] = greedy ? (int32_t)i : -1;
            if (a.probs) a.probs[r] = greedy ? 1.f : 0.f;
        }
        return;
    }

    const double dtop = (double)top, scale = kFine * 1.4426950408889634074 / (double)T;
    const float rate = fminf(kSteps / T, 3e38f);
    const bool by_k = k > 0 && k < a.V, by_p = p < 1.f;
    const uint64_t least = mp > 0.f ? (uint64_t)ceil(fmin((double)mp, 1.0) * (double)(1ull << kOneBits)) : 0;
    // how low the list goes: by the threads' maxima, or, where nothing asks
    // for the weight of more, by min-p (with a step of slack for its logarithm);
    // bounds are lowered by a part in 2^20 of top and distance, so that none
    // of the tokens they stand for is lost to a rounding
    float low = -__builtin_inff();
    if (by_k && k <= 4 * kNT) {
        l.count[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int t = 0; t < 4; ++t) atomicAdd(&l.count[step_of(own[t], top, rate)], 1u);
        __syncthreads();
        const uint64_t c = l.count[tid];
        uint64_t sum;
        const uint64_t ahead = before(l, c, &sum);
        if (ahead < (uint64_t)k && (uint64_t)k <= ahead + c) l.pick[0] = tid;
        __syncthreads();
        const int s = (int)l.pick[0];
        if (s < kBins - 1) low = below(top, (float)(s + 1) / rate);
    }
    if (mp > 0.f && !by_p) low = fmaxf(low, below(top, T * (1.f / kSteps - logf(fminf(mp, 1.f)))));
    if (a.V <= kList && (by_k || by_p)) low = fmaxf(low, -3.402823466e+38f);   // all but -infinity: those weigh nothing

    uint64_t last = ~0ull;     // composites up to this one are kept
    uint64_t want = 0;         // what the prefix of step `step` weighs in it
    int step = -1;
    bool cut_k = by_k, cut_p = by_p;   // what the list is still to be cut by
    bool k_known = false, p_known = false;   // the end of a k past the list, of top-p: found in its step
    // 0: the list as found above; 1: as a histogram of the row says; 2: top-p behind such a k; 3: the prefix is known
    for (int stage = 0; stage < 4; ++stage) {
        const int tid = thread();
        if (stage == 1 || stage == 2) {
            if (stage == 1 && !by_k && !by_p) break;
            if (stage == 2 && !(by_p && k_known)) continue;
            const bool count = stage == 1 && by_k;
            histogram(l, row, !count, top, rate, scale);
            uint64_t v = count ? l.count[tid] : l.mass[tid], all;
            const uint64_t ahead = before(l, v, &all);
            if (count && tid == kBins - 1) v = (uint64_t)row.V - ahead;
            if (stage == 2) {   // the k's whole weight
                if (tid == (int)l.k_step) l.pick[2] = ahead + l.k_mass;
                __syncthreads();
                all = l.pick[2];
            }
            want = count ? (uint64_t)k : share_of(p, all);
            if (tid == 0) l.p_want = want;
            if (ahead < want && want <= ahead + v) {
                l.pick[0] = tid;
                l.pick[1] = ahead;
            }
            __syncthreads();
            const int s = (int)l.pick[0];
            step = -1;
            if (!count || k > kList) {
                step = s;
                want -= l.pick[1];
            }
            low = s < kBins - 1 ? below(top, (float)(s + 1) / rate) : -3.402823466e+38f;
            __syncthreads();
        } else if (stage == 3) {
            if (last == ~0ull || (by_p && k_known && !p_known)) {   // too full to sort: by digits
                want = l.p_want;
                if (last == ~0ull && by_k) {
                    const Cut cut = radix_cut(l, row, false, dtop, scale, (uint64_t)k);
                    last = cut.last;
                    want = share_of(p, cut.mass);
                }
                if (by_p) {
                    if (!by_k) {   // of the whole row's weight again, without the steps before
                        uint64_t sum = 0;
                        row.each([&](int, const float *x, int) {
#pragma unroll
                            for (int e = 0; e < R::E; ++e) sum += weight_of(l.fine, x[e], dtop, scale);
                        });
                        (void)before(l, sum, &want);
                        want = share_of(p, want);
                    }
                    const uint64_t end = radix_cut(l, row, true, dtop, scale, want).last;
                    last = end < last ? end : last;
                }
            }
            low = value_at(last);
            step = -1;
            cut_k = cut_p = false;
        }
        if (!(low > -__builtin_inff())) continue;
        uint64_t blocks = 0;
#pragma unroll
        for (int t0 = 0; t0 < kTurns; t0 += 16) {
            if (t0 >= row.turns) break;
            uint32_t some = 0;
#pragma unroll
            for (int t = 0; t < 16; t += 2) {
                uint32_t two = block_max[(t0 + t) / 2];
                asm volatile("" : "+v"(two));   // unpacked here, not for good
                some |= bf16_bits_to_f32(two & 0xffffu) < low ? 0u : 1u << t;
                some |= bf16_bits_to_f32(two >> 16) < low ? 0u : 2u << t;
            }
            blocks |= (uint64_t)some << t0;
        }
        const int n = gather(l, row, blocks, low, step, top, rate);
        if (n > kList) continue;

        // steps that share out the list's range, as far as it weighs anything
        const float peak = step < 0 ? top : top - (float)step / rate;
        const float fine = fminf(fmaxf((float)(kBins - 1) / (peak - low), rate), 3e38f);
        uint64_t c[kEach], v[kEach], sum = 0, mass;
        const bool do_k = step < 0 ? cut_k && k < n : stage == 1 && by_k, do_p = step < 0 ? cut_p : !do_k;
        if (step >= 0 && do_k && want > (uint64_t)n) continue;   // it ends among -infinities, which are not gathered
        const bool cut = do_k || do_p;
        if (cut) {
            l.count[tid] = 0;
            l.mass[tid] = 0;
            __syncthreads();
        }
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = e * kNT + tid;
            c[e] = ~0ull;
            v[e] = 0;
            if (e * kNT >= n) continue;
            c[e] = i < n ? l.list[i] : ~0ull;
            v[e] = i < n ? weight_of(l.fine, value_at(c[e]), dtop, scale) : 0;
            sum += v[e];
            if (i < n && cut) {
                const int s = step_of(value_at(c[e]), peak, fine);
                atomicAdd(&l.count[s], 1u);
                atomicAdd((unsigned long long *)&l.mass[s], (unsigned long long)v[e]);
            }
        }
        if (cut) {
            (void)before(l, sum, &mass);
#pragma unroll 1
            for (int by = 0; by < 2; ++by) {
                if (by == 0 ? !do_k : !do_p) continue;
                const Cut end = list_cut(l, n, by == 1, top, peak, fine, scale,
                                         step >= 0 ? want : (by == 0 ? (uint64_t)k : share_of(p, mass)));
                last = end.last < last ? end.last : last;
                mass = end.mass;
            }
            if (step >= 0) {   // that was the prefix's end; the list is not the whole prefix
                if (do_k && tid == 0) {
                    l.k_step = (uint64_t)step;
                    l.k_mass = mass;
                }
                k_known = by_k;
                p_known = do_p;
                continue;
            }
        }
        sum = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            v[e] = c[e] <= last && v[e] >= least ? v[e] : 0;
            sum += v[e];
        }
        (void)before(l, sum, &mass);
        uint64_t target = target_of(u, mass);
        // in the order of the indexes, by three digits of 6 bits: the weight of each digit's value, and where the target falls
        uint32_t prefix = 0;
#pragma unroll 1
        for (int shift = kIndexBits - 6; shift >= 0; shift -= 6) {
            if (tid < 64) l.mass[tid] = 0;
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (e * kNT >= n) break;
                const uint32_t i = (uint32_t)c[e];
                if (v[e] && (i >> (shift + 6)) == prefix)
                    atomicAdd((unsigned long long *)&l.mass[(i >> shift) & 63], (unsigned long long)v[e]);
            }
            __syncthreads();
            const uint64_t m = l.mass[lane], upto = wave_upto(m);
            const int digit = __builtin_ctzll(__ballot(target < upto));
            target -= __shfl((unsigned long long)(upto - m), digit);
            prefix = prefix << 6 | digit;
            sum = __shfl((unsigned long long)m, digit);
            __syncthreads();
        }
        if (tid == 0) {
            a.tokens[r] = (int32_t)prefix;
            if (a.probs) a.probs[r] = (float)((double)sum / (double)mass);
        }
        return;
    }
    const float x_last = value_at(last);   // NaN where all is kept

    // the draw over the row, in the order of the indexes: a wavefront's weight
    // in each turn, then the wavefront that holds the target, lane by lane
    auto kept = [&](float x, int i) -> uint64_t {
        const uint64_t v = weight_of(l.fine, x, dtop, scale);
        const bool past = x < x_last || (x == x_last && (uint32_t)i > (uint32_t)last);   // composite(x, i) > last
        return !past && v >= least ? v : 0;
    };
    // [turn][wavefront]; 2^18 float32 logits off a 16-byte boundary have 129 turns
    static_assert(((kMaxVocab + R::E) / R::E + kNT - 1) / kNT * kWaves <= kList, "a row's parts fit the list");
    uint64_t *part = l.list;
    row.each([&](int t, const float *x, int i) {
        uint64_t sum = 0;
#pragma unroll
        for (int e = 0; e < R::E; ++e) sum += kept(x[e], i + e);
        sum = wave_sum(sum);
        if (lane == 0) part[t * kWaves + w] = sum;
    });
    __syncthreads();
    // parts in order, kEach a thread
    const int parts = (row.blocks + kNT - 1) / kNT * kWaves;
    uint64_t v[kEach], sum = 0, mass;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        v[e] = tid * kEach + e < parts ? part[tid * kEach + e] : 0;
        sum += v[e];
    }
    uint64_t at = before(l, sum, &mass);
    const uint64_t target = target_of(u, mass);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        if (at <= target && target < at + v[e]) {
            l.pick[0] = tid * kEach + e;
            l.pick[1] = at;
        }
        at += v[e];
    }
    __syncthreads();
    const int t = (int)l.pick[0] / kWaves, i = t * kNT + ((int)l.pick[0] % kWaves) * 64 + lane;
    if (w == 0) {
        float x[R::E];
        uint64_t v8[R::E], s8 = 0;
        row.widen(row.load_edge(i < row.blocks ? i : 0), x);
#pragma unroll
        for (int e = 0; e < R::E; ++e) {
            v8[e] = i < row.blocks ? kept(x[e], row.first(i) + e) : 0;
            s8 += v8[e];
        }
        uint64_t from = l.pick[1] + wave_upto(s8) - s8;
#pragma unroll
        for (int e = 0; e < R::E; ++e) {
            if (from <= target && target < from + v8[e]) {
                a.tokens[r] = row.first(i) + e;
                if (a.probs) a.probs[r] = (float)((double)v8[e] / (double)mass);
            }
            from += v8[e];
        }
    }
}

// Position w of a window stays while the token drawn before it is the one
// that was fed there; no token (-1) is none that can be fed.
__global__ __launch_bounds__(256) void reject_kernel(const int32_t *tokens, const int32_t *fed, int32_t *n_reject, int B,
                                                     int W) {
    const int b = blockIdx.x * 256 + threadIdx.x;
    if (b >= B) return;
    int kept = 1;
    for (; kept < W; ++kept) {
        const int token = tokens[(size_t)b * W + kept - 1];
        if (token < 0 || token != fed[(size_t)b * W + kept]) break;
    }
    n_reject[b] = W - kept;
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, hipStream_t s) {
    const unsigned rows = (unsigned)((int64_t)a.B * a.W);
    if (a.bf16)
        sample_kernel<true><<<rows, kNT, 0, s>>>(a);
    else
        sample_kernel<false><<<rows, kNT, 0, s>>>(a);
    if (a.n_reject && a.W > 1) reject_kernel<<<(a.B + 255) / 256, 256, 0, s>>>(a.tokens, a.fed, a.n_reject, a.B, a.W);
    return hipGetLastError();
}

}  // namespace replay
