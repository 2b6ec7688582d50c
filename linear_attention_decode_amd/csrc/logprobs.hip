// logprobs.hip -- log-probabilities of given tokens, the entropy of the
// distribution and its most likely tokens, from logits.
//
// With m the row's maximum, t_i = (m - x_i) / T >= 0 and Z = sum exp(-t_i),
//     log p_i = -t_i - log Z,     H = -sum p_i log p_i = log Z + sum exp(-t_i) t_i / Z;
// all terms of both sums are positive, so nothing cancels.  log Z is taken as
// log1p(Z - 1), Z - 1 summed without one of the elements that equal m: where
// one token holds nearly all, its log-probability is the small number that
// the others leave.
//
// A row is cut into parts, a workgroup each, that hold their logits in
// registers from one reading: the maximum first, then the sums from it, then
// the part's first n tokens.  A second launch, a workgroup a row, scales the
// parts' sums to the row's maximum, merges their first tokens and looks up
// the given ones.
//
// The first n of a part: of the largest keys of its 64 groups of threads the
// n-th (n <= 32) bounds the n-th of all from below, so that only tokens from it
// on (some n of them) are gathered and ranked, each by counting those before
// it.  Blocks of 4 or 8 logits that hold none are told by their maximum.  Where
// equal logits make them too many, the n-th token's composite is found by bisection.
// In a part of fewer groups than n the threads' own largest bound it (1280 rows of
// 300 in bf16, n = 20: 15 us, 25 with all of them ranked).
//
// Bound by the vector instructions beside the reading, a dozen a logit.  240
// rows of 50021 in float32, n = 20: 21 us for the parts, 2.3 TB/s of 48 MB, and 7 to
// join them, a chain of a dozen dependent steps a row; one row of 131072 in
// bf16, n = 5: 6 and 7.
// Sums: a block's 4 or 8 terms in float32, a thread's blocks and all beyond
// in float64; the exponential is the hardware's, within 2^-22 of a term.
#include "logits.h"

namespace replay {

namespace {

constexpr int kNT = kPartNT, kWaves = kNT / 64;
constexpr int kList = 1024;                      // tokens gathered
static_assert(kMaxVocab / kPartSmall + 1 <= kNT, "a thread of the join a part");

struct Found {
    __align__(16) uint64_t list[kList];
    __align__(16) uint32_t key[64];   // of four neighbouring threads' tokens the largest
    float top[kWaves];
    uint64_t first[kWaves];
    double sum[kWaves], spread[kWaves];
    uint32_t ones[kWaves], bad[kWaves], n, bound;
};

__device__ __forceinline__ uint64_t wave_min(uint64_t x) {
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint64_t y = (uint64_t)__shfl_xor((long long)x, d);
        x = x < y ? x : y;
    }
    return x;
}
__device__ __forceinline__ uint32_t wave_add(uint32_t x) {
#pragma unroll
    for (int d = 32; d; d >>= 1) x += (uint32_t)__shfl_xor((int)x, d);
    return x;
}
__device__ __forceinline__ double wave_add(double x) {
#pragma unroll
    for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

// 1 / T, where T scales a distribution (T = 0 takes the largest alone)
__device__ __forceinline__ bool scales(float T) { return T > 0.f && T < __builtin_inff(); }

// U blocks of 16 bytes a thread
template <bool BF16, int U>
__global__ __launch_bounds__(kNT) void logprobs_part_kernel(LogprobArgs a) {
    using L = Logits<BF16>;
    constexpr int E = L::E;
    __shared__ Found f;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    const L l(a.logits, row, a.stride, a.V);
    const float T = a.temperature ? a.temperature[row / a.W] : 1.f;

    // blocks lo .. hi - 1 of the row are whole
    const int lo = l.off ? 1 : 0, hi = (l.off + a.V) / E, i0 = part * (kNT * U) + tid;
    const auto whole = make_rsrc(l.base + 16 * lo, hi > lo ? (uint32_t)(hi - lo) * 16u : 0u);
    u32x4 r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = __builtin_amdgcn_raw_buffer_load_b128(whole, (uint32_t)(i0 + u * kNT - lo) * 16u, 0, 0);
    if ((part == 0 && lo) || (part + 1) * (kNT * U) > hi) {   // blocks that are not whole, or none
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kNT;
            const u32x4 edge = i < l.blocks && (i < lo || i >= hi) ? l.load_edge(i) : L::none();
            const bool in = i >= lo && i < hi;
#pragma unroll
            for (int e = 0; e < 4; ++e) r[u][e] = in ? r[u][e] : edge[e];
        }
    }

    // the blocks' largest, and whether a value is none of a distribution's
    float most[U], top = -__builtin_inff();
    bool bad = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float x[E];
        l.widen(r[u], x);
        most[u] = x[0];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            bad |= !(x[e] < __builtin_inff());
            if (e) most[u] = fmaxf(most[u], x[e]);
        }
        top = fmaxf(top, most[u]);
    }
    float m = top;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        m = fmaxf(m, __shfl_xor(m, d));
        if (d == 2 && !(lane & 3)) f.key[tid >> 2] = i0 < l.blocks ? key_of(m) : 0u;
    }
    const bool wave_bad = __any(bad);
    if (lane == 0) {
        f.top[wave] = m;
        f.bad[wave] = wave_bad;
    }
    if (tid == 0) f.n = 0;
    __syncthreads();
    uint32_t worse = f.bad[0];
    m = f.top[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
        m = fmaxf(m, f.top[w]);
        worse |= f.bad[w];
    }
    uint64_t *out = a.ws + (size_t)blockIdx.x * (kPartWords + (a.n > 0 ? a.n : 1));

    // the sums, from this part's maximum (nothing but -infinity weighs nothing),
    // and the first of the tokens that have it
    double sum = 0., spread = 0.;
    uint32_t ones = 0;
    uint64_t lead = ~0ull;
    // (m - x) log2(e) / T as (m p - x p) log2(e) / (T p), p a power of two: the distance of two
    // logits may be past float32's range, and so may 1 / T.  With p = 2^64 m p may be infinite:
    // logits that differ are 2^100 T apart then, and but the largest weigh nothing.
    const float p = T > 1.f ? 0.5f : T < 0x1p-60f ? 0x1p64f : 1.f, mp = m * p;
    const float c = scales(T) && m > -__builtin_inff() ? 1.44269504088896340736f / (T * p) : 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float x[E], w[E], d[E];
        l.widen(r[u], x);
        if (c != 0.f) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                d[e] = fminf(fmaf(-x[e], p, mp) * c, 200.f);   // 2^-200 is no float32: -infinity and the far ones weigh nothing
                w[e] = __builtin_amdgcn_exp2f(-d[e]);
                d[e] *= w[e];
            }
        }
        if (most[u] == m) {   // in few blocks
#pragma unroll
            for (int e = E - 1; e >= 0; --e) {
                const int i = l.first(i0 + u * kNT) + e;
                if (x[e] == m && i >= 0 && i < a.V) {
                    const uint64_t comp = composite(m, i);
                    lead = comp < lead ? comp : lead;
                    ++ones;
                    w[e] = d[e] = 0.f;
                }
            }
        }
        if (c != 0.f) {
#pragma unroll
            for (int s = E / 2; s; s >>= 1)
#pragma unroll
                for (int e = 0; e < s; ++e) {
                    w[e] += w[e + s];
                    d[e] += d[e + s];
                }
            sum += w[0];
            spread += d[0];
        }
    }
    sum = wave_add(sum);
    spread = wave_add(spread);
    ones = wave_add(ones);
    lead = wave_min(lead);
    if (lane == 0) {
        f.sum[wave] = sum;
        f.spread[wave] = spread;
        f.ones[wave] = ones;
        f.first[wave] = lead;
    }
    // the key that the n-th of the groups' largest has
    const int n = a.n;
    if (n > 1 && tid < 64) {
        const uint32_t mine = f.key[tid];
        int rank = 0;
#pragma unroll
        for (int o = 0; o < 64; o += 4) {
            const u32x4 k = *reinterpret_cast<const u32x4 *>(&f.key[o]);
#pragma unroll
            for (int e = 0; e < 4; ++e) rank += k[e] > mine || (k[e] == mine && o + e < tid);
        }
        if (rank == n - 1) f.bound = mine;
    }
    __syncthreads();
    if (tid == 0) {
        double s = 0., d = 0.;
        uint32_t o = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            s += f.sum[w];
            d += f.spread[w];
            o += f.ones[w];
            lead = f.first[w] < lead ? f.first[w] : lead;
        }
        out[0] = (uint64_t)__double_as_longlong(s);
        out[1] = (uint64_t)__double_as_longlong(d);
        out[2] = (uint64_t)worse << 32 | o;
        if (n <= 1) out[kPartWords] = lead;
    }
    if (n <= 1) return;

    // g(composite) for this part's tokens from a key on, thread by thread
    auto each = [&](uint32_t from, auto g) {
        const float least = value_of(from);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (from && !(most[u] >= least)) continue;
            float x[E];
            l.widen(r[u], x);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = l.first(i0 + u * kNT) + e;
                if (i >= 0 && i < a.V) g(composite(x[e], i));
            }
        }
    };
    uint32_t bound = f.bound;
    const int behind = l.blocks - part * (kNT * U), holders = behind < kNT ? behind : kNT;   // threads with tokens
    if (bound == 0 && holders > n) {   // groups without tokens, in a short part: the threads' largest then
        uint32_t *const keys = reinterpret_cast<uint32_t *>(f.list);
        const uint32_t mine = i0 < l.blocks ? key_of(top) : 0u;
        keys[tid] = mine;
        __syncthreads();
        int rank = 0;
        for (int o = 0; o < holders; o += 4) {   // (fewer than 4 n: of their groups fewer than n have tokens)
            const u32x4 k = *reinterpret_cast<const u32x4 *>(&keys[o]);
#pragma unroll
            for (int e = 0; e < 4; ++e) rank += k[e] > mine || (k[e] == mine && o + e < tid);
        }
        if (rank == n - 1) f.bound = mine;
        __syncthreads();
        bound = f.bound;
    }
    // (a bound of 0, of a thread without tokens, takes all there are)
    uint64_t upto = ((uint64_t)~bound << 32) | 0xffffffffu;
    auto gather = [&] {
        each(bound, [&](uint64_t comp) {
            if (comp <= upto) {
                const uint32_t k = atomicAdd(&f.n, 1u);
                if (k < kList) f.list[k] = comp;
            }
        });
        __syncthreads();
    };
    gather();
    if (f.n > kList) {
        // equal logits: the n-th composite, the least that n are not above
        uint64_t below = 0, here = upto;   // fewer than n are <= below - 1; n or more are <= here
        while (below < here) {
            const uint64_t mid = below + (here - below) / 2;
            uint32_t count = 0;
            each(bound, [&](uint64_t comp) { count += comp <= mid; });
            count = wave_add(count);
            __syncthreads();
            if (lane == 0) f.ones[wave] = count;
            __syncthreads();
            uint32_t all = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) all += f.ones[w];
            if (all >= (uint32_t)n)
                here = mid;
            else
                below = mid + 1;
        }
        upto = here;
        __syncthreads();
        if (tid == 0) f.n = 0;
        __syncthreads();
        gather();
    }
    const int found = (int)f.n;
    for (int i = tid; i < found; i += kNT) {
        const uint64_t mine = f.list[i];
        int rank = 0;
#pragma unroll 8
        for (int o = 0; o < found; ++o) rank += f.list[o] < mine;
        if (rank < n) out[kPartWords + rank] = mine;
    }
    for (int i = found + tid; i < n; i += kNT) out[kPartWords + i] = ~0ull;   // a part of fewer tokens
}

// One workgroup a row: its parts joined.
__global__ __launch_bounds__(kNT) void logprobs_join_kernel(LogprobArgs a) {
    extern __shared__ uint64_t list[];   // the parts' first tokens, [parts][n], and behind them those that are kept
    __shared__ uint64_t lead_of[kWaves];
    __shared__ double sums[kWaves], spreads[kWaves];
    __shared__ uint32_t bads[kWaves], kept;
    __shared__ uint64_t bound;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, row = blockIdx.x;
    const int n = a.n > 0 ? a.n : 1, words = kPartWords + n, parts = a.parts;
    uint64_t *const keep = list + parts * n;
    const uint64_t *ws = a.ws + (size_t)row * parts * words;
    for (int i = tid; i < parts * n; i += kNT) list[i] = ws[i / n * words + kPartWords + i % n];
    double s = 0., d = 0.;
    uint64_t head = 0, mine = ~0ull;
    if (tid < parts) {
        s = __longlong_as_double((long long)ws[tid * words]);
        d = __longlong_as_double((long long)ws[tid * words + 1]);
        head = ws[tid * words + 2];
        mine = ws[tid * words + kPartWords];
    }
    const uint64_t first = wave_min(mine);
    const bool wave_bad = __any((int)(head >> 32) != 0);
    if (lane == 0) {
        lead_of[wave] = first;
        bads[wave] = wave_bad;
    }
    if (tid == 0) kept = 0;
    __syncthreads();
    uint64_t lead = lead_of[0];
    uint32_t worse = bads[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
        lead = lead_of[w] < lead ? lead_of[w] : lead;
        worse |= bads[w];
    }
    const float T = a.temperature ? a.temperature[row / a.W] : 1.f;
    const float top = value_at(lead);
    const bool valid = !worse && top > -__builtin_inff() && (T == 0.f || scales(T));
    const double per = scales(T) ? 1. / (double)T : 0.;

    // Z - 1 and sum exp(-t) t from the row's maximum: a part's terms, w of its
    // own, weigh f w there, and its t grow by the maxima's distance
    double zs = 0., hs = 0.;
    if (tid < parts && valid && T > 0.f && mine != ~0ull) {
        const float m = value_at(mine);
        const double t = ((double)top - (double)m) * per, f = m > -__builtin_inff() ? exp(-t) : 0.;
        const double ones = (double)(uint32_t)head, all = ones + s;
        zs = f * s + (mine == lead ? ones - 1. : f * ones);
        hs = f > 0. ? f * (d * 0.69314718055994530942 + t * all) : 0.;
    }
    zs = wave_add(zs);
    hs = wave_add(hs);
    if (lane == 0) {
        sums[wave] = zs;
        spreads[wave] = hs;
    }
    // of entry q of every part the k-th: n tokens at least are not behind it
    const int q = (n + parts - 1) / parts - 1, k = (n + q) / (q + 1);
    if (tid < parts) {
        const uint64_t e = list[tid * n + q];
        int rank = 0;
        for (int o = 0; o < parts; ++o) {
            const uint64_t x = list[o * n + q];
            rank += x < e || (x == e && o < tid);
        }
        if (rank == k - 1) bound = e;
    }
    __syncthreads();
    double z = 0., h = 0.;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        z += sums[w];
        h += spreads[w];
    }
    const float nan = __builtin_nanf("");
    const double log_z = log1p(z);
    if (tid == 0 && a.entropy) a.entropy[row] = valid ? (float)(log_z + h / (1. + z)) : nan;
    // log p of a logit; T = 0: the first of the largest has all
    auto score = [&](float x, bool is_lead) {
        if (!valid) return nan;
        if (T == 0.f) return is_lead ? 0.f : -__builtin_inff();
        return (float)(((double)x - (double)top) * per - log_z);
    };
    for (int i = tid; i < a.M; i += kNT) {
        const int id = a.ids[(size_t)row * a.M + i];
        float lp = nan;
        if (id >= 0 && id < a.V) {
            const size_t at = (size_t)((int64_t)row * a.stride + id);
            const float x = a.bf16 ? load_io1<true>(a.logits, at) : load_io1<false>(a.logits, at);
            lp = score(x, id == (int)(uint32_t)lead);
        }
        a.logp[(size_t)row * a.M + i] = lp;
    }
    if (!a.n) return;
    if (!valid) {
        for (int i = tid; i < n; i += kNT) {
            a.top_ids[(size_t)row * n + i] = -1;
            a.top_logp[(size_t)row * n + i] = nan;
        }
        return;
    }
    for (int i = tid; i < parts * n; i += kNT) {
        const uint64_t e = list[i];
        if (e <= bound && e != ~0ull) keep[atomicAdd(&kept, 1u)] = e;
    }
    __syncthreads();
    const int c = (int)kept;
    for (int i = tid; i < c; i += kNT) {
        const uint64_t e = keep[i];
        int rank = 0;
#pragma unroll 8
        for (int o = 0; o < c; ++o) rank += keep[o] < e;
        if (rank < n) {
            const size_t at = (size_t)row * n + rank;
            a.top_ids[at] = (int)(uint32_t)e;
            a.top_logp[at] = score(value_at(e), e == lead);
        }
    }
}

template <bool BF16, int U>
void launch_parts(const LogprobArgs &a, hipStream_t s) {
    logprobs_part_kernel<BF16, U><<<(unsigned)((int64_t)a.B * a.W * a.parts), kNT, 0, s>>>(a);
}

}  // namespace

// Small parts where big ones would leave CUs without a few workgroups each.
int logprob_part(int64_t rows, int V, int *parts) {
    const int part = rows * (V / kPartBig + 1) < 1024 ? kPartSmall : kPartBig;
    *parts = (V + 7 + part - 1) / part;   // a row may begin up to 7 elements into its first block
    return part;
}

hipError_t launch_logprobs(const LogprobArgs &a, hipStream_t s) {
    if (a.part == kPartBig) {
        if (a.bf16) launch_parts<true, kPartBig / kNT / 8>(a, s);
        else launch_parts<false, kPartBig / kNT / 4>(a, s);
    } else {
        if (a.bf16) launch_parts<true, kPartSmall / kNT / 8>(a, s);
        else launch_parts<false, kPartSmall / kNT / 4>(a, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const size_t lds = (size_t)a.parts * (a.n > 0 ? a.n : 1) * 2 * sizeof(uint64_t);
    logprobs_join_kernel<<<(unsigned)((int64_t)a.B * a.W), kNT, lds, s>>>(a);
    return hipGetLastError();
}

}  // namespace replay
