// conv.hip -- the short causal convolution and the discretisation that turn
// a layer's projected rows into the (q, k, v, dt, a) of the recurrence, for
// packed prompts and for the tokens of a decode step or verify round.
//
// Channel c of token i of a sequence, K taps:
//     o[i][c] = act(bias_c + sum_{j<K} w[c][j] x[i - K + 1 + j][c]),
// act = SiLU or none, in float32, rounded once to the io type; and
//     dt = clamp(softplus(dt_raw + dt_bias)),  a = exp(-exp(a_log) dt).
// Rows before the sequence come from its convolution state: the last rows,
// kept by token position modulo R, so that the pointer move of a rollback
// takes the convolution back with the ring.
//
// Both kernels are bound by HBM: a handful of FMAs and one exponential per
// element against a read and a write of it.  A thread owns 16 bytes of
// channels and keeps their taps and the last K - 1 rows in registers, so
// every row is read once (plus K - 1 rows of halo per tile).
//
// Measured (bf16, K = 4, 10240 channels, 128 heads, with dt and a): a
// prompt batch of 15013 tokens 134 us, 4.75 TB/s of its 635 MB (a large copy
// reaches 4.85), 154 us out of projection rows of 18560; single tokens of 256
// sequences 9.3 us, 3.4 TB/s of 32 MB (float32: 12.8 us, 64 MB), and of one 3.7
// us, a launch and one chain of loads; windows of 5 drafts, 64 heads, 15.6 us
// (float32 20).
#include "tree_common.h"

namespace replay {

namespace {

// Prompt tokens per workgroup; their K - 1 rows of halo come from the L2.
// 15013 tokens x 10240 channels in bf16: tiles of 8, 16 and 32 take 144, 134
// and 141 us (204, 154 and 148 us out of wider projection rows).  Tiles of 8 where those of 16 would not give every CU one: 203
// tokens then take 6.0 us, not 7.9; at 1024, past that, both take 14.8.
constexpr int kTile = 16, kShortTile = 8, kCUs = 256;
constexpr int kNT = 256;      // threads of a prompt workgroup
constexpr int kStepNT = 64;   // threads of a step workgroup: one sequence's channels spread over many CUs
constexpr int kAhead = 8;     // rows a thread loads before it uses the first
// (token, head) pairs of a prompt workgroup that makes dt and a, 4 a thread:
// its exponentials and logarithms are a chain, and 32 of them (64 tokens of
// 128 heads) took 25 us, the whole time of a short prompt.
constexpr int kGates = 1024;
constexpr int kTreeGates = 256;        // (node, head) pairs of a workgroup that makes dt and a
constexpr int kManyTreeBlocks = 2048;  // workgroups of 16 nodes from which on they need not be split

// 16 bytes of io elements as floats, by one load where the row is 16-byte
// aligned and element by element otherwise.
template <bool BF16, bool AL>
struct Row {
    static constexpr int E = BF16 ? 8 : 4;
    IoVec<BF16, E> r;
    float s[AL ? 1 : E];
    __device__ __forceinline__ void load(const void *x, size_t i) {
        if constexpr (AL) {
            r.load(x, i);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) s[e] = load_io1<BF16>(x, i + e);
        }
    }
    __device__ __forceinline__ void widen(float *out) const {
        if constexpr (AL) {
            r.widen(out);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) out[e] = s[e];
        }
    }
};

template <bool BF16, int E>
__device__ __forceinline__ void store_row(void *dst, size_t i, const float *f) {
    if constexpr (BF16) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = f32x2_to_bf16_pair(f[2 * e], f[2 * e + 1]);
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(dst) + i) = w;
    } else {
        const f32x4 w = {f[0], f[1], f[2], f[3]};
        *reinterpret_cast<f32x4 *>(static_cast<float *>(dst) + i) = w;
    }
}

// SiLU.  bf16 results keep 8 bits, so the hardware exponential and
// reciprocal (each within about one part in 2^22) decide no rounding that
// float32 would have decided otherwise but in one case of some thousands;
// float32 results take the correctly rounded division.
template <bool BF16>
__device__ __forceinline__ float silu(float x) {
    if constexpr (BF16) return x * __builtin_amdgcn_rcpf(1.f + __expf(-x));
    return x / (1.f + expf(-x));
}

// The thread's channels: their taps, and where their outputs go.
template <bool BF16, int K>
struct Channels {
    static constexpr int E = BF16 ? 8 : 4;
    float w[E][K], bias[E];
    void *out;          // v, k or q
    int row, col;       // its row length and the thread's column in it
    bool act;
    __device__ __forceinline__ void init(const ConvArgs &a, int c0) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            bias[e] = a.bias ? a.bias[c0 + e] : 0.f;
#pragma unroll
            for (int j = 0; j < K; ++j) w[e][j] = a.weight[(size_t)(c0 + e) * K + j];
        }
        const int HP = a.H * a.P, GN = a.G * a.N;
        out = c0 < HP ? a.v : (c0 < HP + GN ? a.k : a.q);
        row = c0 < HP ? HP : GN;
        col = c0 < HP ? c0 : (c0 < HP + GN ? c0 - HP : c0 - HP - GN);
        act = a.silu != 0;
    }
    // hist[0] is the oldest of the K - 1 rows before x
    __device__ __forceinline__ void apply(const float (*hist)[E], const float *x, size_t t) const {
        float o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            float acc = bias[e];
#pragma unroll
            for (int j = 0; j < K - 1; ++j) acc = fmaf(w[e][j], hist[j][e], acc);
            acc = fmaf(w[e][K - 1], x[e], acc);
            o[e] = act ? silu<BF16>(acc) : acc;
        }
        store_row<BF16, E>(out, t * (size_t)row + col, o);
    }
};

template <int E, int K>
__device__ __forceinline__ void shift(float (*hist)[E], const float *x) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll
        for (int j = 0; j + 1 < K - 1; ++j) hist[j][e] = hist[j + 1][e];
        hist[K - 2][e] = x[e];
    }
}

// One (token, head): dt and a.  Accurate functions throughout: a enters
// products over whole prompts.  NaN stays NaN through the clamp.
template <bool BF16>
__device__ __forceinline__ void discretise(const ConvArgs &a, size_t t, int h) {
    float x = load_io1<BF16>(a.dt_raw, t * (size_t)a.dt_stride + h);
    if (a.dt_bias) x += a.dt_bias[h];
    float d = fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
    if (x != x) d = x;
    d = d < a.dt_min ? a.dt_min : d;
    d = d > a.dt_max ? a.dt_max : d;
    a.dt[t * (size_t)a.H + h] = d;
    a.a[t * (size_t)a.H + h] = expf(-expf(a.a_log[h]) * d);
}

// A bit per token t0 + lane that lies in a sequence with a valid range, at
// least `skip` tokens behind its start.  The search keeps cu[lo] <= t <
// cu[hi] whatever the array holds, so a bad array costs its own sequences
// only.
__device__ __forceinline__ uint64_t token_mask(const int32_t *cu, int B, int T, int t0, int skip) {
    const int t = t0 + (int)(threadIdx.x & 63);
    bool in = t < T && cu[0] <= t && t < cu[B];
    if (in) {
        int lo = 0, hi = B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t) lo = mid; else hi = mid;
        }
        const int s = cu[lo];
        in = s >= 0 && cu[hi] <= T && t - s >= skip;
    }
    return __ballot(in);
}

// Workgroups: [0, B CB) one sequence's first K - 1 tokens and its state (the
// only ones that read or write it, each thread its own channels: state_in
// and state_out may be the same buffer), then one tile of `tile` packed
// tokens each (tokens from the K - 1st of their sequence on, whose history
// is in x), then `gate` tokens' dt and a each.
template <bool BF16, bool AL, int K>
__global__ __launch_bounds__(kNT) void conv_prompt_kernel(ConvArgs a, int CB, int tiles, int tile, int gate) {
    constexpr int E = BF16 ? 8 : 4;
    int id = blockIdx.x;
    if (id < a.B * CB) {
        const int b = id / CB, c0 = ((id % CB) * kNT + (int)threadIdx.x) * E;
        const int s0 = a.cu[b], s1 = a.cu[b + 1];
        if (s0 < 0 || s1 < s0 || s1 > a.T) {
            if (id % CB == 0 && threadIdx.x == 0) raise_seq_error(a.err, b, REPLAY_SEQERR_BAD_RANGE);
            return;
        }
        if (c0 >= a.C) return;
        Channels<BF16, K> ch;
        ch.init(a, c0);
        const int pm = a.pos ? (int)((uint32_t)a.pos[b] % (uint32_t)a.R) : 0;
        const size_t st = (size_t)b * a.R * a.C + c0;
        float hist[K - 1][E];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {   // row K - 1 - j behind the next token
            int slot = pm - (K - 1 - j);
            slot += slot < 0 ? a.R : 0;
            if (a.state_in) {
                Row<BF16, true> r;
                r.load(a.state_in, st + (size_t)slot * a.C);
                r.widen(hist[j]);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) hist[j][e] = 0.f;
            }
        }
        const int n = s1 - s0;
#pragma unroll
        for (int i = 0; i < K - 1; ++i) {
            if (i < n) {
                Row<BF16, AL> r;
                r.load(a.x, (size_t)(s0 + i) * a.x_stride + c0);
                float x[E];
                r.widen(x);
                ch.apply(hist, x, s0 + i);
                shift<E, K>(hist, x);
            }
        }
        if (n > K - 1) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                Row<BF16, AL> r;
                r.load(a.x, (size_t)(s1 - (K - 1) + j) * a.x_stride + c0);
                r.widen(hist[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            int slot = pm - (K - 1 - j);
            slot += slot < 0 ? a.R : 0;
            store_row<BF16, E>(a.state_out, st + (size_t)slot * a.C, hist[j]);
        }
        return;
    }
    id -= a.B * CB;
    if (id < tiles * CB) {
        const int t0 = (id / CB) * tile, c0 = ((id % CB) * kNT + (int)threadIdx.x) * E;
        const uint64_t mask = token_mask(a.cu, a.B, a.T, t0, K - 1);
        if (c0 >= a.C || !(mask & ((1ull << tile) - 1))) return;
        Channels<BF16, K> ch;
        ch.init(a, c0);
        Row<BF16, AL> halo[K - 1], ahead[kAhead];
        float hist[K - 1][E];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int t = t0 - (K - 1) + j;
            halo[j].load(a.x, (size_t)(t < 0 ? 0 : t) * a.x_stride + c0);   // before row 0: no token of the tile uses it
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int t = t0 + i;
            ahead[i].load(a.x, (size_t)(t < a.T ? t : a.T - 1) * a.x_stride + c0);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) halo[j].widen(hist[j]);
        for (int i0 = 0; i0 < tile; i0 += kAhead) {
            Row<BF16, AL> cur[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) cur[i] = ahead[i];
            if (i0 + kAhead < tile) {
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    const int t = t0 + i0 + kAhead + i;
                    ahead[i].load(a.x, (size_t)(t < a.T ? t : a.T - 1) * a.x_stride + c0);
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                float x[E];
                cur[i].widen(x);
                if ((mask >> (i0 + i)) & 1) ch.apply(hist, x, t0 + i0 + i);
                shift<E, K>(hist, x);
            }
        }
        return;
    }
    id -= tiles * CB;
    const int t0 = id * gate;
    const uint64_t mask = token_mask(a.cu, a.B, a.T, t0, 0);
    for (int i = threadIdx.x; i < gate * a.H; i += kNT)
        if ((mask >> (i / a.H)) & 1) discretise<BF16>(a, (size_t)t0 + i / a.H, i % a.H);
}

// Where the history of a sequence's next token is: the slot of that token.
__device__ __forceinline__ int step_slot(const ConvArgs &a, int b) {
    int p = a.pos[b];
    if (a.n_reject) {   // as the rollback itself: out of range, the pointer stays
        const int r = a.n_reject[b];
        if (r >= 0 && r <= p - a.base[b]) p -= r;
    }
    return (int)((uint32_t)p % (uint32_t)a.R);
}

// The tokens of a step or round: workgroups [0, ceil(B / S) CB) take S
// sequences' channels, the rest (token, head) pairs.  The thread that reads a
// channel's history is the one that writes its new rows.  S > 1, for single
// tokens: the taps, 9 times a token's bytes (bf16), are loaded once for S of them.
template <bool BF16, bool AL, int K, int S>
__global__ __launch_bounds__(kStepNT) void conv_step_kernel(ConvArgs a, int CB) {
    constexpr int E = BF16 ? 8 : 4, U = 4;
    int id = blockIdx.x;
    const int groups = (a.B + S - 1) / S;
    if (id >= groups * CB) {
        const size_t i = (size_t)(id - groups * CB) * kStepNT + threadIdx.x;
        if (i < (size_t)a.T * a.H) discretise<BF16>(a, i / a.H, (int)(i % a.H));
        return;
    }
    const int b0 = id / CB * S, c0 = ((id % CB) * kStepNT + (int)threadIdx.x) * E;
    if (c0 >= a.C) return;
    Channels<BF16, K> ch;
    float hist[K - 1][E];
    if constexpr (S > 1) {
        Row<BF16, true> old[S][K - 1];
        Row<BF16, AL> cur[S];
        int slot[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int b = b0 + s < a.B ? b0 + s : a.B - 1;
            slot[s] = step_slot(a, b);
            cur[s].load(a.x, (size_t)b * a.x_stride + c0);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) {
                int from = slot[s] - (K - 1 - j);
                from += from < 0 ? a.R : 0;
                old[s][j].load(a.state_out, ((size_t)b * a.R + from) * a.C + c0);
            }
        }
        ch.init(a, c0);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            if (b0 + s >= a.B) break;
            float x[E];
#pragma unroll
            for (int j = 0; j < K - 1; ++j) old[s][j].widen(hist[j]);
            cur[s].widen(x);
            ch.apply(hist, x, b0 + s);
            store_row<BF16, E>(a.state_out, ((size_t)(b0 + s) * a.R + slot[s]) * a.C + c0, x);
        }
        return;
    }
    const int pm = step_slot(a, b0);
    const size_t st = (size_t)b0 * a.R * a.C + c0;
    Row<BF16, true> old[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        int slot = pm - (K - 1 - j);
        slot += slot < 0 ? a.R : 0;
        old[j].load(a.state_out, st + (size_t)slot * a.C);
    }
    const size_t t0 = (size_t)b0 * a.W;
    Row<BF16, AL> cur[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (i < a.W) cur[i].load(a.x, (t0 + i) * a.x_stride + c0);
    ch.init(a, c0);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) old[j].widen(hist[j]);
    int slot = pm;
    for (int w0 = 0; w0 < a.W; w0 += U) {
        Row<BF16, AL> nxt[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (w0 + U + i < a.W) nxt[i].load(a.x, (t0 + w0 + U + i) * a.x_stride + c0);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (w0 + i < a.W) {
                float x[E];
                cur[i].widen(x);
                ch.apply(hist, x, t0 + w0 + i);
                store_row<BF16, E>(a.state_out, st + (size_t)slot * a.C, x);
                slot = slot + 1 == a.R ? 0 : slot + 1;
                shift<E, K>(hist, x);
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) cur[i] = nxt[i];
    }
}

// The nodes of a tree: workgroups [0, B CB NB) take `per` nodes' channels of
// a sequence each, the rest 64 (node, head) pairs' dt and a a thread block.  A
// node's K rows are read where they lie, its own and its ancestors' in x and
// those before the tree in the state: neighbours in a tree find them in the
// caches, and no load waits for another.
//
// 256 sequences of 16 nodes, 6144 channels in bf16: 33 us, 3.4 TB/s of 111 MB, 77 of them
// at HBM: three wavefronts a SIMD, each of which four times over sends 16 loads and
// waits for them (its 1560 vector instructions are a ninth of its cycles); with 8 and 4
// nodes a workgroup, which read more of their ancestors again, 8 and 22 us more.  One sequence of 10240
// channels has too few workgroups of 16: 5.6 us, a launch and one chain of loads.
template <bool BF16, bool AL, int K>
__global__ __launch_bounds__(kStepNT) void conv_tree_kernel(ConvArgs a, int CB, int NB, int per, int gates) {
    constexpr int E = BF16 ? 8 : 4, U = 4;
    const int lane = threadIdx.x;
    int id = blockIdx.x;
    const bool gate = id >= a.B * CB * NB;
    if (gate) id -= a.B * CB * NB;
    const int b = gate ? id / gates : id / (CB * NB);
    Tree tree;
    tree.load(a.parent, a.n_nodes, b, a.W, lane);
    if (!tree.ok) {
        if (!gate && id % (CB * NB) == 0 && lane == 0) raise_seq_error(a.err, b, REPLAY_SEQERR_BAD_TREE);
        return;
    }
    if (gate) {
        for (int i = id % gates * kTreeGates + lane; i < (id % gates + 1) * kTreeGates && i < tree.n * a.H; i += kStepNT)
            discretise<BF16>(a, (size_t)b * a.W + i / a.H, i % a.H);
        return;
    }
    int from[K];   // lane w: where the K rows of node w are
    from[0] = lane;
#pragma unroll
    for (int d = 1; d < K; ++d) from[d] = tree.up(from[d - 1]);
    const int w0 = id % NB * per, c0 = (id / NB % CB * kStepNT + lane) * E;
    const bool in = c0 < a.C;
    Channels<BF16, K> ch;
    if (in) ch.init(a, c0);
    const int pm = (int)((uint32_t)a.pos[b] % (uint32_t)a.R);
    for (int i0 = w0; i0 < w0 + per && i0 < tree.n; i0 += U) {
        Row<BF16, AL> rows[U][K];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int w = i0 + u < tree.n ? i0 + u : tree.n - 1;
#pragma unroll
            for (int d = 0; d < K; ++d) {
                const int f = __builtin_amdgcn_readlane(from[d], w);
                int slot = pm + f;
                slot += slot < 0 ? a.R : 0;
                if (in) {
                    if (f >= 0)
                        rows[u][d].load(a.x, ((size_t)b * a.W + f) * a.x_stride + c0);
                    else
                        rows[u][d].load(a.state_out, ((size_t)b * a.R + slot) * a.C + c0);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!in || i0 + u >= tree.n || i0 + u >= w0 + per) break;
            float hist[K - 1][E], x[E];
#pragma unroll
            for (int d = 1; d < K; ++d) rows[u][d].widen(hist[K - 1 - d]);
            rows[u][0].widen(x);
            ch.apply(hist, x, (size_t)b * a.W + i0 + u);
        }
    }
}

// The rows of a tree's kept path into the state, behind its newest.  Bound by the
// copy: 256 sequences, 16 rows of 6144 channels each, 14 us for 100 MB, half of
// which the last-level cache holds.
template <bool BF16, bool AL>
__global__ __launch_bounds__(kStepNT) void conv_path_kernel(ConvArgs a, int CB) {
    constexpr int E = BF16 ? 8 : 4;
    const int b = blockIdx.x / CB, lane = threadIdx.x, c0 = (blockIdx.x % CB * kStepNT + lane) * E;
    const int n = a.n_keep[b];
    const int node = lane < a.W ? a.path[(size_t)b * a.W + lane] : 0;
    if (n < 0 || n > a.W || __any(lane < n && (node < 0 || node >= a.W))) {
        if (blockIdx.x % CB == 0 && lane == 0) raise_seq_error(a.err, b, REPLAY_SEQERR_BAD_TREE);
        return;
    }
    int slot = (int)((uint32_t)a.pos[b] % (uint32_t)a.R);
    for (int i = 0; i < n; ++i) {
        const int f = __builtin_amdgcn_readlane(node, i);
        if (i + a.R >= n && c0 < a.C) {   // no later row takes this slot
            Row<BF16, AL> r;
            float x[E];
            r.load(a.x, ((size_t)b * a.W + f) * a.x_stride + c0);
            r.widen(x);
            store_row<BF16, E>(a.state_out, ((size_t)b * a.R + slot) * a.C + c0, x);
        }
        slot = slot + 1 == a.R ? 0 : slot + 1;
    }
}

bool rows_aligned(const ConvArgs &a) {
    const size_t esz = a.io_bf16 ? 2 : 4;
    return (reinterpret_cast<uintptr_t>(a.x) & 15u) == 0 && (a.x_stride * esz) % 16 == 0;
}

// Sequences a thread of the step takes: several where one each makes more
// workgroups of single tokens than the card holds at a time (32 a CU).
constexpr int kShare = 4, kManyGroups = 2048;

template <bool BF16, bool AL, int K>
hipError_t launch_tree(const ConvArgs &a, hipStream_t s) {
    constexpr int E = BF16 ? 8 : 4;
    const int64_t cb = (a.C / E + kStepNT - 1) / kStepNT;
    const int per = (int64_t)a.B * cb * ((a.W + 15) / 16) < kManyTreeBlocks ? 4 : 16;
    const int64_t nb = (a.W + per - 1) / per;
    const int64_t gates = a.dt_raw ? ((int64_t)a.W * a.H + kTreeGates - 1) / kTreeGates : 0;
    const int64_t blocks = a.B * (cb * nb + gates);
    if (!launch_fits(blocks, kStepNT)) return hipErrorInvalidConfiguration;
    conv_tree_kernel<BF16, AL, K><<<(unsigned)blocks, kStepNT, 0, s>>>(a, (int)cb, (int)nb, per, (int)gates);
    return hipGetLastError();
}

template <bool BF16, bool AL>
hipError_t launch_tree_width(const ConvArgs &a, hipStream_t s) {
    if (a.path) {
        const int64_t cb = (a.C / (BF16 ? 8 : 4) + kStepNT - 1) / kStepNT;
        if (!launch_fits(a.B * cb, kStepNT)) return hipErrorInvalidConfiguration;
        conv_path_kernel<BF16, AL><<<(unsigned)(a.B * cb), kStepNT, 0, s>>>(a, (int)cb);
        return hipGetLastError();
    }
    if (a.K == 2) return launch_tree<BF16, AL, 2>(a, s);
    if (a.K == 3) return launch_tree<BF16, AL, 3>(a, s);
    if (a.K == 4) return launch_tree<BF16, AL, 4>(a, s);
    return hipErrorInvalidValue;
}

template <bool BF16, bool AL, int K>
hipError_t launch_one(const ConvArgs &a, bool step, hipStream_t s) {
    constexpr int E = BF16 ? 8 : 4;
    const int64_t nt = step ? kStepNT : kNT;
    const int64_t cb = (a.C / E + nt - 1) / nt;
    const int tile = ((int64_t)a.T + kTile - 1) / kTile * cb < kCUs ? kShortTile : kTile;
    const int64_t tiles = step ? 0 : ((int64_t)a.T + tile - 1) / tile;
    const int gate = kGates / a.H < 1 ? 1 : (kGates / a.H > 64 ? 64 : kGates / a.H);
    const int64_t gates = !a.dt_raw ? 0 : step ? ((int64_t)a.T * a.H + nt - 1) / nt : ((int64_t)a.T + gate - 1) / gate;
    const bool share = step && a.W == 1 && a.B * cb >= kManyGroups;
    const int64_t blocks = (share ? (a.B + kShare - 1) / kShare : a.B) * cb + tiles * cb + gates;
    if (!launch_fits(blocks, nt)) return hipErrorInvalidConfiguration;
    if (!step)
        conv_prompt_kernel<BF16, AL, K><<<(unsigned)blocks, kNT, 0, s>>>(a, (int)cb, (int)tiles, tile, gate);
    else if (share)
        conv_step_kernel<BF16, AL, K, kShare><<<(unsigned)blocks, kStepNT, 0, s>>>(a, (int)cb);
    else
        conv_step_kernel<BF16, AL, K, 1><<<(unsigned)blocks, kStepNT, 0, s>>>(a, (int)cb);
    return hipGetLastError();
}

template <bool BF16, bool AL>
hipError_t launch_width(const ConvArgs &a, bool step, hipStream_t s) {
    if (a.K == 2) return launch_one<BF16, AL, 2>(a, step, s);
    if (a.K == 3) return launch_one<BF16, AL, 3>(a, step, s);
    if (a.K == 4) return launch_one<BF16, AL, 4>(a, step, s);
    return hipErrorInvalidValue;
}

hipError_t launch_conv(const ConvArgs &a, bool step, hipStream_t s) {
    // rows off 16-byte boundaries (a view into rows of an odd length) are read element by element
    const bool al = rows_aligned(a);
    if (a.io_bf16) return al ? launch_width<true, true>(a, step, s) : launch_width<true, false>(a, step, s);
    return al ? launch_width<false, true>(a, step, s) : launch_width<false, false>(a, step, s);
}

}  // namespace

hipError_t launch_conv_prompt(const ConvArgs &a, hipStream_t s) { return launch_conv(a, false, s); }
hipError_t launch_conv_step(const ConvArgs &a, hipStream_t s) { return launch_conv(a, true, s); }

hipError_t launch_conv_tree(const ConvArgs &a, hipStream_t s) {
    const bool al = rows_aligned(a);
    if (a.io_bf16) return al ? launch_tree_width<true, true>(a, s) : launch_tree_width<true, false>(a, s);
    return al ? launch_tree_width<false, true>(a, s) : launch_tree_width<false, false>(a, s);
}

}  // namespace replay
