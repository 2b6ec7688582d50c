// tree_impl.h -- outputs of a tree of drafted tokens, against one read of
// the checkpoint; instantiated by rule and io type in tree_*.hip.
//
// A node's output is y_w = S_w q_w, S_w the state that the ring's entries and
// the nodes on the way to w leave (page "ReplaySSM: Cachear Inputs, No
// Estado", section "Paralelismo": entry j is visible to a position when it
// lies before it; in a tree, when it lies on its path).  With the entries
// (ring, then nodes) numbered j, D_wj the product of the a behind j up to w
// on w's path and g_w all of them from the checkpoint on:
//   Mamba-2  y_w = g_w S0 q_w + sum_j dt_j D_wj (k_j . q_w) v_j
//   gated delta rule: with A_ij = beta_i D_ij (k_i . k_j) (j before i on i's
//     path) and G_wj = D_wj (k_j . q_w), the weights C = G (I + A)^-1 diag(beta),
//            y_w = S0 x_w + sum_j C_wj v_j,  x_w = g_w q_w - sum_j C_wj g_j k_j,
//     which is the recurrence solved for its corrections, as over a prompt's
//     chunk, with "before" read off the tree.
//
// The system is solved in blocks of 16 entries from the last one back: C_J^T =
// T_JJ^T (G_J^T - sum_{I > J} A_IJ^T C_I^T), T_JJ the inverse of a diagonal block by
// substitution, all of them at once.  A row of A or T that is not finite (a value that
// is no number, or long keys) leaves the system, and the nodes behind it, like those
// whose weights are not finite, go through the rule token by token: T is every node's,
// and 0 times its infinity would be every node's NaN.
//
// A workgroup takes one (sequence, head), a wavefront 16 of its rows: their
// tile of S0, and the columns of v that meet it, are on their way while the
// workgroup forms the weights C (and x) in LDS; then S0 x^T and V^T C^T go into one
// accumulator, 16 nodes at a time: on v_mfma_f32_16x16x4_f32, or, where S0 (or v and
// k of the gated delta rule) holds bf16 numbers or fewer bits, on v_mfma_f32_16x16x32_bf16
// with x and C as three numbers of 8 bits each, which is exact.
//
// Bound by workgroups that load, wait and compute in turn.  Mamba-2, four of them a CU: 256
// sequences of 64 heads of 64 x 128, rings of up to 16 and trees of up to 16 nodes, 155 us
// for 678 MB, of which 286 come from HBM and the rest from the last-level cache (a copy
// in bf16 116 us for 410 MB, e4m3 102 for 276, FP4, whose blocks have a product each,
// 129 for 213).  The gated delta rule, two a CU (LDS): 96 sequences of 32 heads of 128 x 128,
// trees of up to 41 nodes against an e4m3 copy, 126 us for 190 MB; of a workgroup's 43000
// cycles 8500 wait for its loads, the dots take 8000, the inverses 4000, the solve
// 4700, the queries 6800, the outputs 5400.  The order of the loads is worth 41 and 86 us
// (S0 first kept all others waiting), the bf16 instructions 30.
#pragma once

#include "tree.h"
#include "tree_common.h"
#include "wide_mx.h"

namespace replay {

template <int P, int N>
struct TreeShape {
    static constexpr int NW = P / 16, NT = 64 * NW;
    static constexpr int MT = (kMaxRing + kMaxTree) / 16;   // tiles of entries
    static constexpr int QU = 4 * N / NT;                   // units of 4 columns of 16 queries, by thread
    static_assert(4 * N % NT == 0, "queries by thread");
    // The queries: float32, rows of XS floats; or, where S0 is of fewer bits, as the
    // bf16 numbers that they are the sum of (one for bf16 queries, else three of 8
    // bits each, which is exact), [part][row] of XB.
    static constexpr int XS = N + 4, XB = N + 8;
    template <int ST, bool IOB, bool DELTA>
    static constexpr int PARTS = !WideTile<P, N, ST>::BF ? 0 : (IOB && !DELTA ? 1 : 3);
    template <int ST, bool IOB, bool DELTA>
    static constexpr int XF = PARTS<ST, IOB, DELTA> ? PARTS<ST, IOB, DELTA> * XB / 2 : XS;
    template <bool IOB>
    static constexpr int KS = N * (IOB ? 2 : 4) / 4 + 4;    // LDS row stride of the keys, floats
    template <int ST>
    static constexpr int TILE = WideTile<P, N, ST>::COAL ? NW * 16 * WideTile<P, N, ST>::TROW : 0;
};

// LDS, in floats.  Mamba-2: weights C [WP][CS], queries (XF a row), decays D
// [WP][WP], whose place the tile of S0 takes on its way into operands (`tile`
// floats).  The gated delta rule: C, D and also A^T [ES][CS], the diagonal blocks' inverses [ES][16] (transposed) and the
// ring's own decays [LP][LP]; the queries lie in place of what is not needed any
// more when they are formed, all but C, or all (`parts`: C then goes on as
// [3][WP][CB] bf16, which lie in place of D and the ring's decays); then the keys
// [ES][KS], whose place the tile takes.
struct TreeLds {
    int WP, LP, ES, CS, CB, D, x, A, inv, rr, parts, k, total;
    __host__ __device__ TreeLds(int W, int L, bool delta, bool in_parts, int XF, int KS, int tile) {
        WP = (W + 15) / 16 * 16;
        LP = (L + 15) / 16 * 16;
        ES = LP + WP;
        CS = ES + 4;
        CB = (ES + 31) / 32 * 32 + 8;
        A = WP * CS;
        inv = A + ES * CS;
        parts = inv + ES * 16;
        const int queries = WP * XF;
        if (!delta) {
            x = A;
            k = D = rr = x + queries;
            total = k + (WP * WP > tile ? WP * WP : tile);
            return;
        }
        x = in_parts ? 0 : A;
        if (in_parts && queries > parts) parts = queries;
        D = parts;
        rr = D + WP * WP;
        k = rr + LP * LP;
        if (in_parts && parts + 3 * WP * CB / 2 > k) k = parts + 3 * WP * CB / 2;
        if (x + queries > k) k = x + queries;
        total = k + (ES * KS > tile ? ES * KS : tile);
    }
};

// The rows of k (or v) of the entries: ring entries 0 .. LP - 1 (there are
// count), then the nodes.  Loads of a row that is none read zero.
struct Entries {
    const char *ring, *nodes;
    uint32_t ring_bytes, node_bytes, row, stride;   // bytes in all, of a row, from a node to the next
    int bmod, L, count, LP;
    __device__ __forceinline__ Entries(const void *ring0, const void *node0, uint32_t row_, uint32_t stride_, int bmod_, int L_,
                                       int count_, int n, int LP_)
        : ring(static_cast<const char *>(ring0)), nodes(static_cast<const char *>(node0)), ring_bytes((uint32_t)L_ * row_),
          node_bytes((uint32_t)(n - 1) * stride_ + row_), row(row_), stride(stride_), bmod(bmod_), L(L_), count(count_), LP(LP_) {}
    // of the tile of 16 entries from e0 on (all the ring's, or all nodes)
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(int e0) const {
        return make_rsrc(e0 < LP ? ring : nodes, e0 < LP ? ring_bytes : node_bytes);
    }
    __device__ __forceinline__ uint32_t at(int e0, int i) const {
        const int e = e0 + i;
        const uint32_t in_ring = e < count ? (uint32_t)ring_slot(bmod, e, L) * row : 0x80000000u;
        return e0 < LP ? in_ring : (uint32_t)(e - LP) * stride;
    }
};
template <bool IOB>
__device__ __forceinline__ uint32_t load_raw(__amdgpu_buffer_rsrc_t rows, uint32_t o, int col) {
    if constexpr (IOB) return (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rows, o + 2 * col, 0, 0);
    return __builtin_amdgcn_raw_buffer_load_b32(rows, o + 4 * col, 0, 0);
}
template <bool IOB>
__device__ __forceinline__ float entry_value(uint32_t raw) { return IOB ? bf16_bits_to_f32(raw) : __uint_as_float(raw); }

// A lane's part of an operand of k . k or k . q: 8 of every 32 columns of a row.
template <int N, bool IOB>
struct DotRow {
    static constexpr int KB = (N + 31) / 32;
    u32x4 b[KB][IOB ? 1 : 2];
    // the row at byte o; columns past N (only where N < 32) read zero
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rows, uint32_t o, int lane) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int c = 32 * kb + 8 * (lane >> 4);
            const uint32_t at = c < N ? o + c * (IOB ? 2 : 4) : 0x80000000u;
#pragma unroll
            for (int x = 0; x < (IOB ? 1 : 2); ++x) b[kb][x] = __builtin_amdgcn_raw_buffer_load_b128(rows, at + 16 * x, 0, 0);
        }
    }
    __device__ __forceinline__ void load(const float *rows, int stride, int lane) {   // from LDS
        const char *row = reinterpret_cast<const char *>(rows + (lane & 15) * stride);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int c = 32 * kb + 8 * (lane >> 4);
#pragma unroll
            for (int x = 0; x < (IOB ? 1 : 2); ++x) {
                b[kb][x] = u32x4{0, 0, 0, 0};
                if (c < N) b[kb][x] = *reinterpret_cast<const u32x4 *>(row + c * (IOB ? 2 : 4) + 16 * x);
            }
        }
    }
    // rows of this (M) by rows of o (N): register r is (4 (lane / 16) + r, lane % 16)
    __device__ __forceinline__ f32x4 dots(const DotRow &o) const {
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            if constexpr (IOB) {
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b[kb][0]), __builtin_bit_cast(bf16x8_t, o.b[kb][0]), d, 0, 0, 0);
            } else {
#pragma unroll
                for (int t = 0; t < 8; ++t)
                    d = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(b[kb][t >> 2][t & 3]), __uint_as_float(o.b[kb][t >> 2][t & 3]), d, 0, 0, 0);
            }
        }
        return d;
    }
};

// 0, or a NaN from the first value on that is no number
__device__ __forceinline__ float none_of(f32x4 x, float none = 0.f) {
#pragma unroll
    for (int u = 0; u < 4; ++u) none = fmaf(x[u], 0.f, none);
    return none;
}

// 4 values as PARTS bf16 numbers each: 8 bits, then what is left
template <int PARTS>
__device__ __forceinline__ void split_parts(f32x4 x, u32x2 *out) {
#pragma unroll
    for (int z = 0; z < PARTS; ++z) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u[i] = __float_as_uint(z == 0 ? __builtin_canonicalizef(x[i]) : x[i]);   // a NaN stays one
            if (z + 1 < PARTS) {
                const float left = x[i] - __uint_as_float(u[i] & 0xffff0000u);
                x[i] = z > 0 || finite(x[i]) ? left : 0.f;
            }
        }
        out[z] = u32x2{u[0] >> 16 | (u[1] & 0xffff0000u), u[2] >> 16 | (u[3] & 0xffff0000u)};
    }
}
template <int PARTS>   // `part` elements apart
__device__ __forceinline__ void put_parts(uint16_t *to, int part, f32x4 x) {
    u32x2 p[PARTS];
    split_parts<PARTS>(x, p);
#pragma unroll
    for (int z = 0; z < PARTS; ++z) *reinterpret_cast<u32x2 *>(to + z * part) = p[z];
}

// An operand of 16 columns (16 nt on) of bf16 rows in LDS: column lane % 16 of rows 4 lg + u
// of the first 16 rows, then of those `second` floats on, each by one transposing read.
__device__ __forceinline__ bf16x8_t cols8(const float *rows, int second, int stride, int nt, int lane) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const int lr = lane & 15, lg = lane >> 4;
    const float *at = rows + (4 * lg + (lr >> 2)) * stride + 8 * nt + 2 * (lr & 3);
    const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)at));
    const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(at + second)));
    return __builtin_bit_cast(bf16x8_t, u32x4{a.x, a.y, b.x, b.y});
}

// S0 x^T over 16 rows and 16 queries in PARTS bf16 numbers, on v_mfma_f32_16x16x32_bf16:
// bf16, e4m3 (unscaled) and MX FP4 values are bf16 numbers, and every product is exact
// (an infinite one times a part that is 0 is a NaN).
// At 128 columns 12 products (16 cycles each) take the place of 32 of 32 cycles.
template <int PARTS, int P, int N, int ST>
__device__ __forceinline__ f32x4 dot_parts(const WideRows<P, N, ST> &rows, const uint16_t *x, int part, int stride, int lane,
                                           const uint8_t *rsc) {
    using WT = WideTile<P, N, ST>;
    const int lg = lane >> 4;
    const uint16_t *row = x + (lane & 15) * stride;
    f32x4 out = {0.f, 0.f, 0.f, 0.f};
    uint32_t sw[ST == ST_FP4 ? WT::NB : 1];   // the 4 rows' scale bytes, rr NB + st
    if constexpr (ST == ST_FP4)
#pragma unroll
        for (int i = 0; i < WT::NB; ++i) sw[i] = reinterpret_cast<const uint32_t *>(rsc)[i];
#pragma unroll
    for (int st = 0; st < WT::STEPS; ++st) {
        constexpr int HALVES = WT::CVEC / 8;
#pragma unroll
        for (int hh = 0; hh < HALVES; ++hh) {
            uint4 a;
            if constexpr (ST == ST_BF16) a = rows.at[st].v;
            else if constexpr (ST == ST_FP8) a = rows.at[st].bf16_half(hh);
            else a = rows.at[st].bf16x8();
            f32x4 acc = ST == ST_FP4 ? f32x4{0.f, 0.f, 0.f, 0.f} : out;
#pragma unroll
            for (int z = PARTS - 1; z >= 0; --z) {
                const uint4 q = *reinterpret_cast<const uint4 *>(row + z * part + (4 * st + lg) * WT::CVEC + 8 * hh);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(q), acc, 0, 0, 0);
            }
            if constexpr (ST == ST_FP4) {
#pragma unroll
                for (int rr = 0; rr < 4; ++rr) {
                    const int i = rr * WT::NB + st;
                    out[rr] += ldexpf(acc[rr], (int)((sw[i >> 2] >> (8 * (i & 3))) & 0xffu) - 127);
                }
            } else {
                out = acc;
            }
        }
    }
    return out;
}

// Nodes through the gated delta rule token by token, a wavefront the 16 rows that are
// its own, lane (row lr, columns 16 i + 4 lg + u).  Rare: it takes its arguments from
// the kernel's again and works out its place again, so that nothing stays in registers
// for it while the weights are made.
template <int P, int N, int ST, bool IOB>
__device__ __forceinline__ void run_rule(uint64_t nodes, const uint64_t *s_anc) {
    typedef const uint64_t __attribute__((address_space(4))) word;
    static_assert(sizeof(TreeArgs) % 8 == 0, "whole words");
    word *from = (word *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(from) : : "memory");
    uint64_t words[sizeof(TreeArgs) / 8];
#pragma unroll
    for (size_t i = 0; i < sizeof(TreeArgs) / 8; ++i) words[i] = from[i];
    TreeArgs t;
    __builtin_memcpy(&t, words, sizeof t);
    const RingView &r = t.r;
    const int lid = xcd_remap(blockIdx.x, gridDim.x), H = r.H, G = r.G, L = r.L, W = t.W;
    const int b = lid / H, h = lid % H, g = h / (H / G), base = r.base[b], count = r.pos[b] - base;
    const size_t bh = (size_t)b * H + h, bg = (size_t)b * G + g;
    const int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0)), lr = lane & 15, lg = lane >> 4;
    const int row = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 16 + lr;
    const float sc = ST == ST_FP8 ? static_cast<const float *>(t.scale)[bh] : 1.f;
    f32x4 S[N / 16];
    auto piece = [&](const void *rows, size_t at, int i) {   // of the row that begins at element `at`
        IoVec<IOB, 4> x;
        x.load(rows, at + 16 * i + 4 * lg);
        float f[4];
        x.widen(f);
        return f32x4{f[0], f[1], f[2], f[3]};
    };
    auto over = [&](const void *rows, size_t at) {   // S x
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < N / 16; ++i) d += S[i] * piece(rows, at, i);
        float x = d[0] + d[1] + d[2] + d[3];
        x += __shfl_xor(x, 16);
        return x + __shfl_xor(x, 32);
    };
    auto token = [&](const void *k, size_t k_at, const void *v, size_t v_at, float beta, float alpha) {
        const float add = beta * fmaf(-alpha, over(k, k_at), load_io1<IOB>(v, v_at + row));
#pragma unroll
        for (int i = 0; i < N / 16; ++i) S[i] = alpha * S[i] + add * piece(k, k_at, i);
    };
#pragma unroll 1
    for (; nodes; nodes &= nodes - 1) {
        asm volatile("" ::: "memory");
        const int w = __builtin_ctzll(nodes);
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {
            const size_t e = (bh * P + row) * N + 16 * i + 4 * lg;
            WideA<ST, false> a;
            if constexpr (ST == ST_FP4) a.load_mx(t.S, t.scale, e);
            else a.load(t.S, e);
            S[i] = sc * a.f32();
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll 1
        for (int e = 0; e < count; ++e) {
            const int slot = ring_slot(base % L, e, L);
            const size_t at = dta_index(b, bh, H, L, slot);
            token(r.k, (bg * L + slot) * N, r.v, (bh * L + slot) * P, r.dt[at], r.a[at]);
        }
#pragma unroll 1
        for (uint64_t on = s_anc[w]; on; on &= on - 1) {   // a node's ancestors come before it
            const size_t j = (size_t)b * W + __builtin_ctzll(on);
            token(t.k, (j * G + g) * N, t.v, (j * H + h) * P, t.dt[j * H + h], t.a[j * H + h]);
        }
        const size_t at = (size_t)b * W + w;
        const float y = over(t.q, (at * G + g) * N);
        if (lg == 0) t.y[(at * H + h) * P + row] = y;
    }
}

template <int P, int N, int ST, bool IOB, bool DELTA>
__global__ __launch_bounds__((TreeShape<P, N>::NT), DELTA ? (IOB ? 4 : 3) : 1) void verify_tree_kernel(TreeArgs t) {
    using Sh = TreeShape<P, N>;
    using WT = WideTile<P, N, ST>;
    constexpr int NW = Sh::NW, NT = Sh::NT, XS = Sh::XS;
    constexpr int KS = Sh::template KS<IOB>, PARTS = Sh::template PARTS<ST, IOB, DELTA>, XF = Sh::template XF<ST, IOB, DELTA>;
    constexpr bool CP = DELTA && IOB;   // C as bf16 parts
    extern __shared__ __align__(16) float lds[];
    __shared__ uint64_t s_anc[kMaxTree];            // ancestors of a node, itself among them
    // products of a: of a node's path; from the checkpoint up to and with an
    // entry; of the ring behind an entry.  An entry's dt (beta), 0 where there is none
    __shared__ __align__(16) float s_gam[kMaxRing + kMaxTree], s_dt[kMaxRing + kMaxTree];
    __shared__ __align__(16) float s_path[kMaxTree], s_R[kMaxRing];
    __shared__ uint32_t s_odd[NW];   // a wavefront's keys hold a value that is no number
    // the gated delta rule: ring entries and nodes whose row of A or T is not finite; nodes whose weights are not
    __shared__ uint32_t s_lost[3], s_redo[2];

    const RingView &r = t.r;
    const int lid = xcd_remap(blockIdx.x, gridDim.x);
    const int H = r.H, L = r.L, W = t.W;
    const int b = lid / H, h = lid % H;
    const int g = h / (H / r.G);
    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const size_t bh = (size_t)b * H + h;
    const int p0 = 16 * wave;

    const int base = r.base[b], count = r.pos[b] - base, n = t.n_nodes ? t.n_nodes[b] : W;
    Tree tree;
    auto fail = [&] {
        for (int i = tid; i < W * P; i += NT) t.y[(((size_t)b * W + i / P) * H + h) * P + i % P] = __builtin_nanf("");
        if (tid == 0 && h == 0) raise_seq_error(r.err, b, tree.ok ? REPLAY_SEQERR_TOO_FEW : REPLAY_SEQERR_BAD_TREE);
    };
    if (count < 0 || count > L || n < 0 || n > W) {   // uniform over the workgroup, as every check here
        tree.load(t.parent, t.n_nodes, b, W, lane);
        fail();
        return;
    }
    if (n == 0) return;

    // Every load that the weights wait for, then V and the tile of S0: loads
    // return in the order in which they were sent.
    const int parent = t.parent[(size_t)b * W + (lane < n ? lane : 0)];
    const int bmod = base % L, last = lane < count ? ring_slot(bmod, lane, L) : 0;
    float ra = r.a[dta_index(b, bh, H, L, last)], rdt = r.dt[dta_index(b, bh, H, L, last)];
    const size_t node = ((size_t)b * W + (lane < n ? lane : 0)) * H + h;
    float na = t.a[node], ndt = t.dt[node];
    const float sc = ST == ST_FP8 ? static_cast<const float *>(t.scale)[bh] : 1.f;

    const TreeLds at(W, L, DELTA, CP, XF, KS, Sh::template TILE<ST>);
    const int WP = at.WP, LP = at.LP, CS = at.CS;
    float *s_C = lds, *s_D = lds + at.D, *s_X = lds + at.x, *s_A = lds + at.A, *s_inv = lds + at.inv, *s_RR = lds + at.rr;
    float *s_K = lds + at.k;
    uint16_t *s_P = reinterpret_cast<uint16_t *>(lds + at.parts);   // C's parts
    const int part = WP * Sh::XB, cpart = WP * at.CB;   // elements
    auto put_query = [&](int w, int c, f32x4 x) {   // columns c .. c + 3
        if constexpr (PARTS) put_parts<PARTS>(reinterpret_cast<uint16_t *>(s_X) + w * Sh::XB + c, part, x);
        else *reinterpret_cast<f32x4 *>(&s_X[w * XS + c]) = x;
    };
    const int wt_n = (n + 15) / 16, et_n = LP / 16 + wt_n, e_end = LP + n;
    constexpr uint32_t ESZ = IOB ? 2 : 4;
    const Entries ks(static_cast<const char *>(r.k) + ((size_t)b * r.G + g) * L * N * ESZ,
                     static_cast<const char *>(t.k) + ((size_t)b * W * r.G + g) * N * ESZ, N * ESZ, (uint32_t)r.G * N * ESZ, bmod,
                     L, count, n, LP);
    const Entries vs(static_cast<const char *>(r.v) + bh * L * P * ESZ, static_cast<const char *>(t.v) + ((size_t)b * W * H + h) * P * ESZ,
                     P * ESZ, (uint32_t)H * P * ESZ, bmod, L, count, n, LP);
    const auto qs = make_rsrc(static_cast<const char *>(t.q) + ((size_t)b * W * r.G + g) * N * ESZ, (uint32_t)(n - 1) * ks.stride + N * ESZ);

    // k . q: a wavefront has one tile of queries (every ND-th, where there are more
    // of them than wavefronts) and every `ways`-th tile of entries
    constexpr int ND = DELTA && NW >= 4 ? NW - 1 : NW;   // the last one has the decays to do
    const int ways = ND > wt_n ? ND / wt_n : 1;
    const int ot0 = ways > 1 ? wave % wt_n : wave, et0 = ways > 1 ? wave / wt_n : 0;
    const bool dots = wave < ND && et0 < ways && ot0 < wt_n;
    DotRow<N, IOB> Q, K;
    Q.load(qs, dots ? (uint32_t)(16 * ot0 + lr) * ks.stride : 0x80000000u, lane);
    // the gated delta rule's keys, 64 units of 16 bytes (8 where a row has but two of 16) by wavefront and turn
    constexpr int UB = N * ESZ / 4 < 16 ? 8 : 16, UR = N * ESZ / UB, TU = 16 * UR / 64;   // turns a tile
    constexpr int KT = DELTA ? (Sh::MT * TU + NW - 1) / NW : 1;
    static_assert(16 * UR % 64 == 0, "a turn within a tile");
    u32x4 kraw[KT];
    u32x2 qraw[Sh::QU][IOB ? 1 : 2];
    auto load_queries = [&](int wt) {
#pragma unroll
        for (int i = 0; i < Sh::QU; ++i) {
            const int x = tid + i * NT, w = 16 * wt + x / (N / 4);
            const uint32_t o = (uint32_t)w * ks.stride + x % (N / 4) * 4 * ESZ;
#pragma unroll
            for (int y = 0; y < (IOB ? 1 : 2); ++y) qraw[i][y] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(qs, o + 8 * y, 0, 0));
        }
    };
    auto store_queries = [&](int wt) {
#pragma unroll
        for (int i = 0; i < Sh::QU; ++i) {
            const int x = tid + i * NT;
            const u32x2 u = qraw[i][0], v = qraw[i][IOB ? 0 : 1];
            f32x4 q;
            if constexpr (IOB) q = f32x4{bf16_bits_to_f32(u.x & 0xffffu), bf16_bits_to_f32(u.x >> 16), bf16_bits_to_f32(u.y & 0xffffu), bf16_bits_to_f32(u.y >> 16)};
            else q = f32x4{__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(v.x), __uint_as_float(v.y)};
            put_query(16 * wt + x / (N / 4), x % (N / 4) * 4, q);
        }
    };
    if constexpr (DELTA) {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int turn = i * NW + wave, e0 = turn / TU * 16, x = turn % TU * 64 + lane;
            const auto rows_k = ks.rows_of(e0);
            const uint32_t o = e0 < e_end ? ks.at(e0, x / UR) + x % UR * UB : 0x80000000u;
            if constexpr (UB == 16) {
                kraw[i] = __builtin_amdgcn_raw_buffer_load_b128(rows_k, o, 0, 0);
            } else {
                const u32x2 u = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rows_k, o, 0, 0));
                kraw[i] = u32x4{u.x, u.y, 0, 0};
            }
        }
    } else {
        const bool first = dots && et0 < et_n;
        K.load(ks.rows_of(first ? 16 * et0 : 0), first ? ks.at(16 * et0, lr) : 0x80000000u, lane);
        load_queries(0);
    }
    // column p0 + lr of v of entries 16 i + 4 lg + u
    uint32_t vc[Sh::MT][4];
#pragma unroll
    for (int i = 0; i < Sh::MT; ++i) {
#pragma unroll
        for (int u = 0; u < 4; ++u) vc[i][u] = 0;
        if (16 * i < e_end) {
            const auto rows_v = vs.rows_of(16 * i);
#pragma unroll
            for (int u = 0; u < 4; ++u) vc[i][u] = load_raw<IOB>(rows_v, vs.at(16 * i, 4 * lg + u), p0 + lr);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    WideRows<P, N, ST> rows;
    rows.load(t.S, bh * (size_t)(P * N), p0, lane, t.scale);
    __builtin_amdgcn_sched_barrier(0);

    tree.set(parent, n, lane);
    if (!tree.ok) {
        fail();
        return;
    }
    if (DELTA && tid < 5) (tid < 3 ? s_lost[tid] : s_redo[tid - 3]) = 0;
    auto lose = [&](int e) { atomicOr(&s_lost[e < LP ? 0 : 1 + (e - LP) / 32], 1u << (e < LP ? e : (e - LP) % 32)); };
    auto redo = [&](int w) { atomicOr(&s_redo[w / 32], 1u << w % 32); };

    // raw dots: C[w][e] = k_e . q_w, and A^T[j][i] = k_j . k_i of tiles i >= j
    if constexpr (DELTA) {
        if constexpr (CP) {
            bool bad = false;
#pragma unroll
            for (int i = 0; i < KT; ++i)
#pragma unroll
                for (int u = 0; u < UB / 4; ++u)
                    bad |= (kraw[i][u] & 0x7f80u) == 0x7f80u || (kraw[i][u] & 0x7f800000u) == 0x7f800000u;
            bad = __any(bad);
            if (lane == 0) s_odd[wave] = bad;
        }
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int turn = i * NW + wave, e0 = turn / TU * 16, x = turn % TU * 64 + lane;
            char *to = reinterpret_cast<char *>(s_K + (e0 + x / UR) * KS) + x % UR * UB;
            if (e0 < e_end) {
                if constexpr (UB == 16) *reinterpret_cast<u32x4 *>(to) = kraw[i];
                else *reinterpret_cast<u32x2 *>(to) = u32x2{kraw[i].x, kraw[i].y};
            }
        }
        lds_barrier();
        for (int x = ND - 1 - wave; x >= 0 && x < et_n * (et_n + 1) / 2; x += ND) {
            int ot = 0, et = x;
            while (et > ot) et -= ++ot;   // et <= ot
            DotRow<N, IOB> A, B;
            A.load(s_K + 16 * et * KS, KS, lane);
            B.load(s_K + 16 * ot * KS, KS, lane);
            const f32x4 d = A.dots(B);
#pragma unroll
            for (int rr = 0; rr < 4; ++rr) s_A[(16 * et + 4 * lg + rr) * CS + 16 * ot + lr] = d[rr];
        }
    }
    if (dots)
        for (int ot = ot0; ot < wt_n; ot += ways > 1 ? wt_n : ND) {
            if (ot != ot0) Q.load(qs, (uint32_t)(16 * ot + lr) * ks.stride, lane);
            for (int et = et0; et < et_n; et += ways) {
                if constexpr (DELTA) K.load(s_K + 16 * et * KS, KS, lane);
                else if (et != et0 || ot != ot0) K.load(ks.rows_of(16 * et), ks.at(16 * et, lr), lane);
                *reinterpret_cast<f32x4 *>(&s_C[(16 * ot + lr) * CS + 16 * et + 4 * lg]) = K.dots(Q);
            }
        }
    if constexpr (!DELTA) {
        store_queries(0);
        for (int wt = 1; wt < wt_n; ++wt) {
            load_queries(wt);
            store_queries(wt);
        }
    }
    // the decays, by the last wavefront: lane j has ring entry j and node j
    if (wave == NW - 1) {
        if (lane >= count) {
            ra = 1.f;
            rdt = 0.f;
        }
        if (lane >= n) {
            na = 1.f;
            ndt = 0.f;
        }
        float pre = ra, suf = ra;   // of the ring, up to and with j; from j on
#pragma unroll
        for (int d = 1; d < kMaxRing; d <<= 1)
            if (d < LP) {
                const float u = __shfl_up(pre, d), o = __shfl_down(suf, d);
                if (lane >= d) pre *= u;
                if (lane + d < 64) suf *= o;
            }
        const float all = __shfl(pre, LP - 1);
        suf = __shfl_down(suf, 1);
        // up from node `lane`, the nearest first, two steps a turn: D[w][j] for the
        // j on the way, and who they are
        uint64_t anc = 0;
        float path = 1.f;
        int x = lane < n ? lane : -1;
        const int up = tree.parent < 0 ? 0 : tree.parent;
        const float na2 = __shfl(na, up);
        const int up2 = __shfl(tree.parent, up);
        while (__any(x >= 0)) {
            const int at_x = x < 0 ? 0 : x;
            const float f = __shfl(na, at_x), f2 = __shfl(na2, at_x);
            const int u = __shfl(tree.parent, at_x), u2 = __shfl(up2, at_x);
            if (x >= 0) {
                s_D[lane * WP + x] = path;
                path *= f;
                anc |= 1ull << x;
                x = -1;
                if (u >= 0) {
                    s_D[lane * WP + u] = path;
                    path *= f2;
                    anc |= 1ull << u;
                    x = u2;
                }
            }
        }
        if (lane < kMaxRing) {
            s_R[lane] = suf;
            if (lane < LP) {
                s_gam[lane] = pre;
                s_dt[lane] = rdt;
            }
        }
        if (lane < WP) {
            s_anc[lane] = anc;
            s_path[lane] = path;
            s_gam[LP + lane] = path * all;
            s_dt[LP + lane] = ndt;
        }
    }
    if constexpr (DELTA)
        if (wave == ND - 1) {
            float p = 1.f;
            for (int i = 0; i < count; ++i) {   // a behind j up to and with i
                if (i > lane) p *= bcast(ra, i);
                if (lane < LP) s_RR[lane * LP + i] = p;
            }
        }
    lds_barrier();

    // v, where it is no number 0: what such a value has to reach is added at the end
    float vf[Sh::MT][4];
    bf16x8_t vp[Sh::MT / 2];   // C in parts: entries 32 i + 4 lg + u, then 32 i + 16 + 4 lg + u
    bool odd = false;
#pragma unroll
    for (int i = 0; i < Sh::MT; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            asm volatile("" : "+v"(vc[i][u]));   // its load ends here, not where it was sent
            vf[i][u] = entry_value<IOB>(vc[i][u]);
            if (!finite(vf[i][u])) {
                vf[i][u] = 0.f;
                vc[i][u] = 0;
                odd = true;
            }
        }
    if constexpr (CP) {
#pragma unroll
        for (int i = 0; i < Sh::MT / 2; ++i) {
            u32x4 x;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t two = vc[2 * i + u / 2][2 * u % 4] | vc[2 * i + u / 2][2 * u % 4 + 1] << 16;
                asm volatile("" : "+v"(two));   // one register from here on
                x[u] = two;
            }
            vp[i] = __builtin_bit_cast(bf16x8_t, x);
        }
    }
    odd = __any(odd);

    // weights: the dots of what lies on the node's path, decayed (selects, not
    // factors of 0: another branch's NaN stays there), by tiles, lane (column lr, entries or nodes 4 lg + u)
    auto on_path = [&](int w, int e) { return w < n && (e < LP ? e < count : (s_anc[w] >> (e - LP) & 1) != 0); };
    auto vec = [](const float *p) { return *reinterpret_cast<const f32x4 *>(p); };
    for (int x = wave; x < et_n * wt_n; x += NW) {
        const int e = x / wt_n * 16 + 4 * lg, w = x % wt_n * 16 + lr;
        const bool of_ring = x / wt_n * 16 < LP;   // uniform
        const uint32_t on = w >= n ? 0u : of_ring ? (uint32_t)((1ull << count) - 1) >> e : (uint32_t)(s_anc[w] >> (e - LP));
        f32x4 c = vec(s_C + w * CS + e) * (of_ring ? vec(s_R + e) * s_path[w] : vec(s_D + w * WP + e - LP));
        if constexpr (!DELTA) c *= vec(s_dt + e);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (!(on >> u & 1)) c[u] = 0.f;
        *reinterpret_cast<f32x4 *>(s_C + w * CS + e) = c;
    }
    if constexpr (DELTA) {
        // A^T, tiles i >= j; of values that are no numbers nothing, their entries are lost
        for (int x = NW - 1 - wave; x < et_n * (et_n + 1) / 2; x += NW) {
            int ot = 0, et = x;
            while (et > ot) et -= ++ot;
            const int j = 16 * et + lr, i = 16 * ot + 4 * lg;
            f32x4 d;
            uint32_t on = 0;
            if (16 * ot < LP) {
                d = vec(s_RR + j * LP + i);
                on = (uint32_t)((1ull << count) - 1) >> i;
            } else if (16 * et < LP) {
                d = vec(s_path + i - LP) * s_R[j];
                on = j < count ? 15 : 0;
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    d[u] = s_D[(i + u - LP) * WP + j - LP];
                    on |= (uint32_t)(s_anc[i + u - LP] >> (j - LP) & 1) << u;
                }
            }
            f32x4 c = d * vec(s_A + j * CS + i) * vec(s_dt + i);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (!(on >> u & 1) || i + u <= j || i + u >= e_end) c[u] = 0.f;
            if (none_of(c) != 0.f)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (!finite(c[u])) {
                        lose(i + u);
                        c[u] = 0.f;
                    }
            *reinterpret_cast<f32x4 *>(s_A + j * CS + i) = c;
        }
        if constexpr (CP) {
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < NW; ++i) bad |= s_odd[i];
            if (bad)   // the products take 0 for such values: another's weight makes its nodes NaN as it is
                for (int x = tid; x < 16 * et_n * (N / 2); x += NT) {
                    uint32_t *u = reinterpret_cast<uint32_t *>(s_K + x / (N / 2) * KS) + x % (N / 2);
                    *u &= ((*u & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) | ((*u & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
                }
        }
        lds_barrier();
        // rows of the diagonal blocks' inverses T, a lane a row: y (I + A) = e_r from the last column back
        for (int x = tid; x < 16 * et_n; x += NT) {
            const int b0 = x & ~15, row = x & 15;
            float y[16];
#pragma unroll
            for (int j = 15; j >= 0; --j) {
                y[j] = j == row ? 1.f : 0.f;
#pragma unroll
                for (int i4 = 12; i4 >= (j & ~3); i4 -= 4) {
                    const f32x4 c = *reinterpret_cast<const f32x4 *>(&s_A[(b0 + j) * CS + b0 + i4]);
#pragma unroll
                    for (int u = 3; u >= 0; --u)
                        if (i4 + u > j) y[j] = fmaf(-c[u], y[i4 + u], y[j]);
                }
                s_inv[(b0 + j) * 16 + row] = y[j];   // T^T
                __builtin_amdgcn_sched_barrier(0);
            }
            float none = 0.f;
#pragma unroll
            for (int j = 0; j < 16; j += 4) none = none_of(f32x4{y[j], y[j + 1], y[j + 2], y[j + 3]}, none);
            if (none != 0.f) {   // its zeros off the path would be NaN, and reach every node: the entry is lost
                lose(x);
                for (int j = 0; j < 16; ++j) s_inv[(b0 + j) * 16 + row] = 0.f;
            }
        }
        lds_barrier();
        // C^T by blocks, lane (node lr, entries 4 lg + u), a wavefront 16 nodes: C_J^T = T_JJ^T (what is left of
        // G_J^T), and what C_J takes from the blocks before it
        for (int wt = wave; wt < wt_n; wt += NW) {
            asm volatile("" ::: "memory");   // A and T stay in LDS
            float *row = s_C + (16 * wt + lr) * CS + 4 * lg;
            const int w = 16 * wt + lr;   // the entries on its path, from 4 lg on
            const uint64_t nodes = w < n ? s_anc[w] >> 4 * lg : 0;
            const uint32_t in_ring = w < n ? (uint32_t)((1ull << count) - 1) >> 4 * lg : 0;
            f32x4 c[Sh::MT];
#pragma unroll
            for (int J = 0; J < Sh::MT; ++J)
                c[J] = *reinterpret_cast<const f32x4 *>(row + 16 * (J < et_n ? J : 0));
#pragma unroll
            for (int J = Sh::MT - 1; J >= 0; --J)
                if (J < et_n) {
                    const f32x4 T = *reinterpret_cast<const f32x4 *>(&s_inv[(16 * J + lr) * 16 + 4 * lg]);
                    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int u = 0; u < 4; ++u) sum = __builtin_amdgcn_mfma_f32_16x16x4f32(T[u], c[J][u], sum, 0, 0, 0);
                    c[J] = sum;
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int I = J - 1; I >= 0; --I) {
                        const f32x4 m = *reinterpret_cast<const f32x4 *>(&s_A[(16 * I + lr) * CS + 16 * J + 4 * lg]);
#pragma unroll
                        for (int u = 0; u < 4; ++u) c[I] = __builtin_amdgcn_mfma_f32_16x16x4f32(-m[u], c[J][u], c[I], 0, 0, 0);
                    }
                }
            float none = 0.f;
#pragma unroll
            for (int J = 0; J < Sh::MT; ++J)
                if (J < et_n) {
                    f32x4 o;
                    const f32x4 beta = *reinterpret_cast<const f32x4 *>(&s_dt[16 * J + 4 * lg]);
                    const uint32_t on = 16 * J < LP ? in_ring >> 16 * J : (uint32_t)(nodes >> (16 * J - LP));
#pragma unroll
                    for (int u = 0; u < 4; ++u) o[u] = on >> u & 1 ? c[J][u] * beta[u] : 0.f;
                    none = none_of(o, none);
                    if constexpr (CP) put_parts<3>(s_P + w * at.CB + 16 * J + 4 * lg, cpart, o);
                    else *reinterpret_cast<f32x4 *>(row + 16 * J) = o;
                }
            if (none != 0.f) redo(w);
            if constexpr (CP)
                if (et_n & 1)   // the other half of the last 32
#pragma unroll
                    for (int z = 0; z < 3; ++z) *reinterpret_cast<u32x2 *>(s_P + z * cpart + w * at.CB + 16 * et_n + 4 * lg) = u32x2{0, 0};
        }
    }
    lds_barrier();

    if constexpr (CP) {   // the queries: a wavefront has 16 nodes and every `turns`-th 16 columns
        const int turns = NW > wt_n ? NW / wt_n : 1;
        const int first = turns > 1 ? wave / wt_n : 0;
        if (first < turns)
            for (int wt = turns > 1 ? wave % wt_n : wave; wt < wt_n; wt += turns > 1 ? wt_n : NW) {
                asm volatile("" ::: "memory");   // gamma stays in LDS
                const int w = 16 * wt + lr;
                bf16x8_t c[Sh::MT / 2][3];   // C gamma of entries 32 i + 4 lg + u and 32 i + 16 + 4 lg + u
#pragma unroll
                for (int i = 0; i < Sh::MT / 2; ++i)
                    if (32 * i < e_end) {
                        u32x2 o[2][3];
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            const int e = 32 * i + 16 * hh + 4 * lg;
                            u32x2 in[3];
#pragma unroll
                            for (int z = 0; z < 3; ++z) in[z] = *reinterpret_cast<const u32x2 *>(s_P + z * cpart + w * at.CB + e);
                            const f32x4 gam = vec(s_gam + e);
                            f32x4 x;
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                float v[3];
#pragma unroll
                                for (int z = 0; z < 3; ++z) v[z] = bf16_bits_to_f32(u & 1 ? in[z][u >> 1] >> 16 : in[z][u >> 1] & 0xffffu);
                                const float f = v[2] + v[1] + v[0];
                                x[u] = f == 0.f || 16 * (2 * i + hh) >= e_end ? 0.f : f * gam[u];
                            }
                            split_parts<3>(x, o[hh]);
                        }
#pragma unroll
                        for (int z = 0; z < 3; ++z) c[i][z] = __builtin_bit_cast(bf16x8_t, u32x4{o[0][z].x, o[0][z].y, o[1][z].x, o[1][z].y});
                    }
                const float gw = s_gam[LP + w];
                auto query = [&](int nt) {
                    return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(qs, nt < N / 16 ? (uint32_t)w * ks.stride + (16 * nt + 4 * lg) * ESZ : 0x80000000u, 0, 0));
                };
                u32x2 q = query(first);
                float none = 0.f;
                for (int nt = first; nt < N / 16; nt += turns) {
                    const u32x2 next = query(nt + turns);
                    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < Sh::MT / 2; ++i)
                        if (32 * i < e_end) {
                            const bf16x8_t k = cols8(s_K + 32 * i * KS, 32 * i + 16 < e_end ? 16 * KS : 0, KS, nt, lane);
#pragma unroll
                            for (int z = 2; z >= 0; --z) x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, c[i][z], x, 0, 0, 0);
                        }
                    f32x4 o;
#pragma unroll
                    for (int rr = 0; rr < 4; ++rr)
                        o[rr] = w < n ? fmaf(gw, bf16_bits_to_f32(rr & 1 ? q[rr >> 1] >> 16 : q[rr >> 1] & 0xffffu), -x[rr]) : 0.f;
                    none = none_of(o, none);
                    put_query(w, 16 * nt + 4 * lg, o);
                    q = next;
                }
                if (none != 0.f) redo(w);
            }
    } else if constexpr (DELTA) {
        for (int nt = wave; nt < N / 16; nt += NW) {
            u32x4 q[kMaxTree / 16];
#pragma unroll
            for (int wt = 0; wt < kMaxTree / 16; ++wt) {
                q[wt] = u32x4{0, 0, 0, 0};
                if (16 * wt < n) q[wt] = __builtin_amdgcn_raw_buffer_load_b128(qs, (uint32_t)(16 * wt + lr) * ks.stride + (16 * nt + 4 * lg) * ESZ, 0, 0);
            }
            float kc[Sh::MT][4];   // column 16 nt + lr of entries 16 i + 4 lg + u
#pragma unroll
            for (int i = 0; i < Sh::MT; ++i)
                if (16 * i < e_end)
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float k = s_K[(16 * i + 4 * lg + u) * KS + 16 * nt + lr];
                        kc[i][u] = finite(k) ? k : 0.f;   // another's weight makes its nodes NaN as it is
                    }
#pragma unroll
            for (int wt = 0; wt < kMaxTree / 16; ++wt) {
                if (16 * wt >= n) break;
                const int w = 16 * wt + lr;
                f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < Sh::MT; ++i)
                    if (16 * i < e_end) {
                        const f32x4 c = *reinterpret_cast<const f32x4 *>(&s_C[w * CS + 16 * i + 4 * lg]);
                        const f32x4 gam = *reinterpret_cast<const f32x4 *>(&s_gam[16 * i + 4 * lg]);
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            x = __builtin_amdgcn_mfma_f32_16x16x4f32(kc[i][u], c[u] == 0.f ? 0.f : c[u] * gam[u], x, 0, 0, 0);
                    }
                const float gw = s_gam[LP + w];
                f32x4 o;
#pragma unroll
                for (int rr = 0; rr < 4; ++rr) {
                    o[rr] = w < n ? fmaf(gw, __uint_as_float(q[wt][rr]), -x[rr]) : 0.f;
                }
                if (none_of(o) != 0.f) redo(w);
                put_query(w, 16 * nt + 4 * lg, o);
            }
        }
    }
    uint64_t by_rule = 0;   // nodes with a lost entry on their path, or weights that are not finite
    if constexpr (DELTA) {
        lds_barrier();
        auto word = [](uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)x); };
        by_rule = word(s_redo[0]) | (uint64_t)word(s_redo[1]) << 32;
        const uint32_t ring = word(s_lost[0]);
        const uint64_t lost = word(s_lost[1]) | (uint64_t)word(s_lost[2]) << 32;
        if (ring | lost) by_rule |= __ballot(lane < n && (ring || (s_anc[lane] & lost)));
    }

    // y^T: rows p0 + 4 lg + rr, nodes 16 wt + lr
    rows.transpose(reinterpret_cast<uint32_t (*)[WT::TROW]>(s_K + (WT::COAL ? wave * 16 * WT::TROW : 0)), lane);
    const uint8_t *rsc = static_cast<const uint8_t *>(t.scale) + (bh * P + p0 + 4 * lg) * WT::NB;   // FP4 rows
    for (int wt = 0; wt < wt_n; ++wt) {
        const int w = 16 * wt + lr;
        f32x4 y;
        if constexpr (PARTS) y = dot_parts<PARTS>(rows, reinterpret_cast<const uint16_t *>(s_X) + 16 * wt * Sh::XB, part, Sh::XB, lane, rsc);
        else y = rows.dot_f32q(reinterpret_cast<const float (*)[XS]>(s_X + 16 * wt * XS), lane, rsc);
        y *= DELTA ? sc : sc * s_gam[LP + w];
        if constexpr (CP) {
#pragma unroll
            for (int i = 0; i < Sh::MT / 2; ++i)
                if (32 * i < e_end)
#pragma unroll
                    for (int z = 2; z >= 0; --z) {
                        const uint16_t *c = s_P + z * cpart + w * at.CB + 32 * i + 4 * lg;
                        const u32x2 c0 = *reinterpret_cast<const u32x2 *>(c), c1 = *reinterpret_cast<const u32x2 *>(c + 16);
                        y = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vp[i], __builtin_bit_cast(bf16x8_t, u32x4{c0.x, c0.y, c1.x, c1.y}), y, 0, 0, 0);
                    }
        } else
#pragma unroll
        for (int i = 0; i < Sh::MT; ++i)
            if (16 * i < e_end) {
                const f32x4 c = *reinterpret_cast<const f32x4 *>(&s_C[w * CS + 16 * i + 4 * lg]);
#pragma unroll
                for (int u = 0; u < 4; ++u) y = __builtin_amdgcn_mfma_f32_16x16x4f32(vf[i][u], c[u], y, 0, 0, 0);
            }
        if (w >= n || (DELTA && by_rule >> w & 1)) continue;
        if (odd) {   // a value that is no number, for the nodes behind it alone
            for (int e = 0; e < e_end; ++e) {
                if (!on_path(w, e)) continue;
#pragma unroll
                for (int rr = 0; rr < 4; ++rr) {
                    const float v = entry_value<IOB>(load_raw<IOB>(vs.rows_of(e & ~15), vs.at(e & ~15, e & 15), p0 + 4 * lg + rr));
                    if (finite(v)) continue;
                    if constexpr (CP) y[rr] = fmaf(bf16_bits_to_f32(s_P[w * at.CB + e]), v, y[rr]);   // its sign and whether it is 0
                    else y[rr] = fmaf(s_C[w * CS + e], v, y[rr]);
                }
            }
        }
        *reinterpret_cast<f32x4 *>(&t.y[(((size_t)b * W + w) * H + h) * P + p0 + 4 * lg]) = y;
    }

    if constexpr (DELTA)
        if (by_rule) run_rule<P, N, ST, IOB>(by_rule, s_anc);
}

template <int P, int N, int ST, bool IOB, bool DELTA>
hipError_t launch_tree_one(const TreeArgs &a, hipStream_t s) {
    using Sh = TreeShape<P, N>;
    const TreeLds at(a.W, a.r.L, DELTA, DELTA && IOB, Sh::template XF<ST, IOB, DELTA>, Sh::template KS<IOB>, Sh::template TILE<ST>);
    verify_tree_kernel<P, N, ST, IOB, DELTA>
        <<<(unsigned)((int64_t)a.r.B * a.r.H), TreeShape<P, N>::NT, at.total * sizeof(float), s>>>(a);
    return hipGetLastError();
}

template <int P, int N, bool IOB, bool DELTA>
hipError_t launch_tree_st(int st, const TreeArgs &a, hipStream_t s) {
    switch (st) {
        case ST_F32: return launch_tree_one<P, N, ST_F32, IOB, DELTA>(a, s);
        case ST_BF16: return launch_tree_one<P, N, ST_BF16, IOB, DELTA>(a, s);
        case ST_FP8: return launch_tree_one<P, N, ST_FP8, IOB, DELTA>(a, s);
        case ST_FP4: return launch_tree_one<P, N, ST_FP4, IOB, DELTA>(a, s);
        default: return hipErrorInvalidValue;
    }
}

template <bool IOB, bool DELTA>
hipError_t launch_tree(int P, int N, int st, const TreeArgs &a, hipStream_t s) {
    if (P == 16 && N == 16) return launch_tree_st<16, 16, IOB, DELTA>(st, a, s);
    if (P == 64 && N == 64) return launch_tree_st<64, 64, IOB, DELTA>(st, a, s);
    if (P == 64 && N == 128) return launch_tree_st<64, 128, IOB, DELTA>(st, a, s);
    if (P == 128 && N == 128) return launch_tree_st<128, 128, IOB, DELTA>(st, a, s);
    return hipErrorInvalidValue;
}

}  // namespace replay
