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
// substitution, all of them at once.
//
// A workgroup takes one (sequence, head), a wavefront 16 of its rows: their
// tile of S0, and the columns of v that meet it, are on their way while the
// workgroup forms the weights C (and x) in LDS; then S0 x^T and V^T C^T go into one
// accumulator, both on v_mfma_f32_16x16x4_f32, 16 nodes at a time.
#pragma once

#include "tree.h"
#include "tree_common.h"
#include "wide_mx.h"

namespace replay {

template <int P, int N>
struct TreeShape {
    static constexpr int NW = P / 16, NT = 64 * NW;
    static constexpr int XS = N + 4;      // LDS row stride of the queries, floats
    static constexpr int KB = (N + 31) / 32;
    static constexpr int ME = (kMaxRing + kMaxTree) / 4;   // entries a lane of the V product holds
};

// LDS, in floats: weights C [WP][CS], decays D [WP][WP]; then the queries
// [WP][XS], which for the gated delta rule take the place of A^T [ES][CS], the diagonal
// blocks' inverses [ES][16] (transposed) and the ring's own decays [LP][LP].
struct TreeLds {
    int WP, LP, ES, CS, x, inv, rr, total;
    __host__ __device__ TreeLds(int W, int L, int N, bool delta) {
        WP = (W + 15) / 16 * 16;
        LP = (L + 15) / 16 * 16;
        ES = LP + WP;
        CS = ES + 4;
        x = WP * CS + WP * WP;
        inv = x + ES * CS;
        rr = inv + ES * 16;
        const int first = delta ? rr + LP * LP : 0, second = x + WP * (N + 4);
        total = first > second ? first : second;
    }
};

// The rows of k (or v) of the entries, in bytes: ring entries 0 .. LP - 1 (there
// are count), then the nodes.  Loads of a row that is none read zero.
struct Entries {
    __amdgpu_buffer_rsrc_t ring, nodes;
    uint32_t row, stride;   // bytes of a row; from a node to the next
    int bmod, L, count, LP;
    __device__ __forceinline__ Entries(const void *ring0, const void *node0, uint32_t row_, uint32_t stride_, int base, int L_,
                                       int count_, int n, int LP_)
        : ring(make_rsrc(ring0, (uint32_t)L_ * row_)), nodes(make_rsrc(node0, (uint32_t)(n - 1) * stride_ + row_)), row(row_),
          stride(stride_), bmod(base % L_), L(L_), count(count_), LP(LP_) {}
    __device__ __forceinline__ uint32_t ring_at(int e) const {
        return e < count ? (uint32_t)ring_slot(bmod, e, L) * row : 0x80000000u;
    }
    // element `col` of entry e, of a tile of entries that are all the ring's or all nodes
    template <bool IOB>
    __device__ __forceinline__ uint32_t value(int e, bool of_ring, int col) const {
        const uint32_t o = (of_ring ? ring_at(e) : (uint32_t)(e - LP) * stride) + col * (IOB ? 2 : 4);
        if constexpr (IOB) return of_ring ? (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(ring, o, 0, 0) : (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(nodes, o, 0, 0);
        return of_ring ? __builtin_amdgcn_raw_buffer_load_b32(ring, o, 0, 0) : __builtin_amdgcn_raw_buffer_load_b32(nodes, o, 0, 0);
    }
};
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

__device__ __forceinline__ bool tree_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

template <int P, int N, int ST, bool IOB, bool DELTA>
__global__ __launch_bounds__((TreeShape<P, N>::NT)) void verify_tree_kernel(TreeArgs t) {
    using Sh = TreeShape<P, N>;
    using WT = WideTile<P, N, ST>;
    constexpr int NW = Sh::NW, NT = Sh::NT, XS = Sh::XS;
    extern __shared__ __align__(16) float lds[];
    __shared__ __align__(16) uint32_t s_T[WT::COAL ? NW : 1][16][WT::TROW];   // per-wavefront staging
    __shared__ uint64_t s_anc[kMaxTree];            // ancestors of a node, itself among them
    // products of a: of a node's path; from the checkpoint up to and with an
    // entry; of the ring behind an entry.  An entry's dt (beta), 0 where there is none
    __shared__ float s_path[kMaxTree], s_gam[kMaxRing + kMaxTree], s_R[kMaxRing], s_dt[kMaxRing + kMaxTree];

    const RingView &r = t.r;
    const int lid = xcd_remap(blockIdx.x, gridDim.x);
    const int H = r.H, L = r.L, W = t.W;
    const int b = lid / H, h = lid % H;
    const int g = h / (H / r.G);
    const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const size_t bh = (size_t)b * H + h;
    const int p0 = 16 * wave;

    const int base = r.base[b], count = r.pos[b] - base;
    WideRows<P, N, ST> rows;
    rows.load(t.S, bh * (size_t)(P * N), p0, lane, t.scale);
    Tree tree;
    tree.load(t.parent, t.n_nodes, b, W, lane);
    if (!tree.ok || count < 0 || count > L) {   // uniform over the workgroup
        for (int i = tid; i < W * P; i += NT) t.y[(((size_t)b * W + i / P) * H + h) * P + i % P] = __builtin_nanf("");
        if (tid == 0 && h == 0) raise_seq_error(r.err, b, tree.ok ? REPLAY_SEQERR_TOO_FEW : REPLAY_SEQERR_BAD_TREE);
        return;
    }
    const int n = tree.n;
    if (n == 0) return;
    const TreeLds at(W, L, N, DELTA);
    const int WP = at.WP, LP = at.LP, ES = at.ES, CS = at.CS;
    float *s_C = lds, *s_D = lds + WP * CS, *s_X = lds + at.x, *s_A = s_X, *s_inv = lds + at.inv, *s_RR = lds + at.rr;
    const int wt_n = (n + 15) / 16, et_n = LP / 16 + wt_n, e_end = LP + n;
    constexpr uint32_t ESZ = IOB ? 2 : 4;
    const Entries ks(static_cast<const char *>(r.k) + ((size_t)b * r.G + g) * L * N * ESZ,
                     static_cast<const char *>(t.k) + ((size_t)b * W * r.G + g) * N * ESZ, N * ESZ, (uint32_t)r.G * N * ESZ, base,
                     L, count, n, LP);
    const Entries vs(static_cast<const char *>(r.v) + bh * L * P * ESZ, static_cast<const char *>(t.v) + ((size_t)b * W * H + h) * P * ESZ,
                     P * ESZ, (uint32_t)H * P * ESZ, base, L, count, n, LP);
    const auto qs = make_rsrc(static_cast<const char *>(t.q) + ((size_t)b * W * r.G + g) * N * ESZ, (uint32_t)(n - 1) * ks.stride + N * ESZ);

    // column p0 + lr of v of entries 4 s + lg
    uint32_t vc[Sh::ME];
#pragma unroll
    for (int s = 0; s < Sh::ME; ++s) {
        vc[s] = 0;
        if (4 * s < e_end) vc[s] = vs.template value<IOB>(4 * s + lg, 4 * s < LP, p0 + lr);
    }
    if constexpr (!DELTA) {   // the queries, 4 columns a thread and turn
        for (int i = tid; i < 16 * wt_n * (N / 4); i += NT) {
            const int w = i / (N / 4), c = i % (N / 4) * 4;
            f32x4 q;
            if constexpr (IOB) {
                const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(qs, (uint32_t)w * ks.stride + c * 2, 0, 0));
                q = f32x4{bf16_bits_to_f32(x[0] & 0xffffu), bf16_bits_to_f32(x[0] >> 16), bf16_bits_to_f32(x[1] & 0xffffu), bf16_bits_to_f32(x[1] >> 16)};
            } else {
                q = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(qs, (uint32_t)w * ks.stride + c * 4, 0, 0));
            }
            *reinterpret_cast<f32x4 *>(&s_X[w * XS + c]) = q;
        }
    }

    // raw dots: C[w][e] = k_e . q_w, and A^T[j][i] = k_j . k_i of tiles i >= j;
    // the next tile's rows are on their way during a product
    {
        const int cq = et_n * wt_n, total = cq + (DELTA ? et_n * (et_n + 1) / 2 : 0);
        auto place = [&](int x, int *et, int *ot) {
            if (x < cq) {
                *et = x / wt_n;
                *ot = x % wt_n;
                return;
            }
            int o = 0, left = x - cq;
            while (left > o) left -= ++o;
            *et = left;   // <= ot
            *ot = o;
        };
        auto rows_of = [&](DotRow<N, IOB> &d, int tile) {
            if (16 * tile < LP) d.load(ks.ring, ks.ring_at(16 * tile + lr), lane);
            else d.load(ks.nodes, (uint32_t)(16 * tile + lr - LP) * ks.stride, lane);
        };
        auto load = [&](int x, DotRow<N, IOB> &A, DotRow<N, IOB> &B) {
            int et, ot;
            place(x, &et, &ot);
            rows_of(A, et);
            if (x < cq) B.load(qs, (uint32_t)(16 * ot + lr) * ks.stride, lane);
            else rows_of(B, ot);
        };
        DotRow<N, IOB> A, B;
        if (wave < total) load(wave, A, B);
        for (int x = wave; x < total; x += NW) {
            DotRow<N, IOB> nextA, nextB;
            if (x + NW < total) load(x + NW, nextA, nextB);
            int et, ot;
            place(x, &et, &ot);
            const f32x4 d = A.dots(B);
            if (x < cq) {
                *reinterpret_cast<f32x4 *>(&s_C[(16 * ot + lr) * CS + 16 * et + 4 * lg]) = d;
            } else {
#pragma unroll
                for (int rr = 0; rr < 4; ++rr) s_A[(16 * et + 4 * lg + rr) * CS + 16 * ot + lr] = d[rr];
            }
            if (x + NW < total) {
                A = nextA;
                B = nextB;
            }
        }
    }
    // the decays, by the last wavefront: lane j has ring entry j and node j
    if (wave == NW - 1) {
        float ra = 1.f, rdt = 0.f, na = 1.f, ndt = 0.f;
        if (lane < count) {
            const int sl = ring_slot(base % L, lane, L);
            ra = r.a[dta_index(b, bh, H, L, sl)];
            rdt = r.dt[dta_index(b, bh, H, L, sl)];
        }
        if (lane < n) {
            na = t.a[((size_t)b * W + lane) * H + h];
            ndt = t.dt[((size_t)b * W + lane) * H + h];
        }
        float pre = ra, suf = ra;   // of the ring, up to and with j; from j on
#pragma unroll
        for (int d = 1; d < kMaxRing; d <<= 1) {
            const float u = __shfl_up(pre, d), o = __shfl_down(suf, d);
            if (lane >= d) pre *= u;
            if (lane + d < 64) suf *= o;
        }
        const float all = __shfl(pre, kMaxRing - 1);
        suf = __shfl_down(suf, 1);
        uint64_t anc = 1ull << lane;
        float path = na;
        int up = tree.parent;
#pragma unroll
        for (int d = 1; d < kMaxTree; d <<= 1) {   // what lies 2^d steps up
            const int from = up < 0 ? 0 : up;
            const uint64_t m = (uint64_t)__shfl((long long)anc, from);
            const float f = __shfl(path, from);
            const int u = __shfl(up, from);
            if (up >= 0) {
                anc |= m;
                path *= f;
                up = u;
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
        // D[w][j] for the j on w's way up, a lane a node: the nearest first
        {
            float p = 1.f;
            int x = lane < n ? lane : -1;
            while (__any(x >= 0)) {
                const int from = x < 0 ? 0 : x;
                const float f = __shfl(na, from);
                const int u = __shfl(tree.parent, from);
                if (x >= 0) {
                    s_D[lane * WP + x] = p;
                    p *= f;
                    x = u;
                }
            }
        }
        if constexpr (DELTA) {
            float p = 1.f;
            for (int i = 0; i < count; ++i) {   // a behind j up to and with i
                if (i > lane) p *= bcast(ra, i);
                if (lane < LP) s_RR[lane * LP + i] = p;
            }
        }
    }
    lds_barrier();

    // weights: the dots of what lies on the node's path, decayed (selects, not
    // factors of 0: another branch's NaN stays there)
    auto on_path = [&](int w, int e) { return w < n && (e < LP ? e < count : (s_anc[w] >> (e - LP) & 1) != 0); };
    auto decay = [&](int w, int e) { return e < LP ? s_R[e] * s_path[w] : s_D[w * WP + e - LP]; };
    for (int w = tid / 16; w < 16 * wt_n; w += NT / 16)   // 16 threads a row
        for (int e = tid % 16; e < ES; e += 16) {
            float *c = s_C + w * CS + e;
            *c = on_path(w, e) ? decay(w, e) * *c * (DELTA ? 1.f : s_dt[e]) : 0.f;
        }
    if constexpr (DELTA) {
        // A^T; of values that are no numbers nothing: what they have to reach, G, beta
        // and the decays carry
        for (int j = tid / 16; j < ES; j += NT / 16)
            for (int i = tid % 16; i < ES; i += 16) {
                float c = 0.f;
                if (i > j && i < e_end && (i < LP ? i < count : on_path(i - LP, j)))
                    c = (i < LP ? s_RR[j * LP + i] : decay(i - LP, j)) * s_A[j * CS + i] * s_dt[i];
                s_A[j * CS + i] = tree_finite(c) ? c : 0.f;
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
                for (int i4 = j & ~3; i4 < 16; i4 += 4) {
                    const f32x4 c = *reinterpret_cast<const f32x4 *>(&s_A[(b0 + j) * CS + b0 + i4]);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        if (i4 + u > j) y[j] = fmaf(-c[u], y[i4 + u], y[j]);
                }
                s_inv[(b0 + j) * 16 + row] = y[j];   // T^T
            }
        }
        lds_barrier();
        // C_J^T = T_JJ^T (G_J^T - sum A_IJ^T C_I^T), lane (node lr, entries 4 lg + u), a wavefront 16 nodes
        for (int wt = wave; wt < wt_n; wt += NW) {
            float *row = s_C + (16 * wt + lr) * CS + 4 * lg;
            for (int J = et_n - 1; J >= 0; --J) {
                f32x4 c = *reinterpret_cast<const f32x4 *>(row + 16 * J);
                f32x4 sum = {0.f, 0.f, 0.f, 0.f};
                for (int I = J + 1; I < et_n; ++I) {
                    const f32x4 m = *reinterpret_cast<const f32x4 *>(&s_A[(16 * J + lr) * CS + 16 * I + 4 * lg]);
                    const f32x4 o = *reinterpret_cast<const f32x4 *>(row + 16 * I);
#pragma unroll
                    for (int u = 0; u < 4; ++u) sum = __builtin_amdgcn_mfma_f32_16x16x4f32(m[u], o[u], sum, 0, 0, 0);
                }
                c -= sum;
                const f32x4 m = *reinterpret_cast<const f32x4 *>(&s_inv[(16 * J + lr) * 16 + 4 * lg]);
                sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int u = 0; u < 4; ++u) sum = __builtin_amdgcn_mfma_f32_16x16x4f32(m[u], c[u], sum, 0, 0, 0);
                *reinterpret_cast<f32x4 *>(row + 16 * J) = sum;
                wave_lds_sync();
            }
#pragma unroll 1
            for (int J = 0; J < et_n; ++J) {
                f32x4 c = *reinterpret_cast<const f32x4 *>(row + 16 * J);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int e = 16 * J + 4 * lg + u;
                    c[u] = on_path(16 * wt + lr, e) ? c[u] * s_dt[e] : 0.f;
                }
                *reinterpret_cast<f32x4 *>(row + 16 * J) = c;
            }
        }
    }
    lds_barrier();

    if constexpr (DELTA) {   // the queries, which take the place of A
        for (int nt = wave; nt < N / 16; nt += NW) {
            float kc[Sh::ME];   // column 16 nt + lr of entries 4 s + lg
#pragma unroll
            for (int s = 0; s < Sh::ME; ++s) {
                kc[s] = 0.f;
                if (4 * s < e_end) {
                    const float k = entry_value<IOB>(ks.template value<IOB>(4 * s + lg, 4 * s < LP, 16 * nt + lr));
                    if (tree_finite(k)) kc[s] = k;   // another's weight makes its nodes NaN as it is
                }
            }
            for (int wt = 0; wt < wt_n; ++wt) {
                const int w = 16 * wt + lr;
                f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < Sh::ME; ++s) {
                    if (4 * s >= e_end) break;
                    const int e = 4 * s + lg;
                    const float c = s_C[w * CS + e];
                    x = __builtin_amdgcn_mfma_f32_16x16x4f32(kc[s], c == 0.f ? 0.f : c * s_gam[e], x, 0, 0, 0);
                }
                float q[4] = {0.f, 0.f, 0.f, 0.f};
                if (w < n) load_io4<IOB>(t.q, (((size_t)b * W + w) * r.G + g) * N + 16 * nt + 4 * lg, q);
                const float gw = s_gam[LP + w];
                f32x4 o;
#pragma unroll
                for (int rr = 0; rr < 4; ++rr) o[rr] = w < n ? fmaf(gw, q[rr], -x[rr]) : 0.f;
                *reinterpret_cast<f32x4 *>(&s_X[w * XS + 16 * nt + 4 * lg]) = o;
            }
        }
    }
    if constexpr (DELTA) lds_barrier();

    // y^T: rows p0 + 4 lg + rr, nodes 16 wt + lr
    rows.transpose(s_T[WT::COAL ? wave : 0], lane);
    float vf[Sh::ME];
    bool odd = false;
#pragma unroll
    for (int s = 0; s < Sh::ME; ++s) {
        vf[s] = entry_value<IOB>(vc[s]);
        if (!tree_finite(vf[s])) {
            vf[s] = 0.f;
            odd = true;
        }
    }
    odd = __any(odd);
    const uint8_t *rsc = static_cast<const uint8_t *>(t.scale) + (bh * P + p0 + 4 * lg) * WT::NB;   // FP4 rows
    const float sc = ST == ST_FP8 ? static_cast<const float *>(t.scale)[bh] : 1.f;
    for (int wt = 0; wt < wt_n; ++wt) {
        const int w = 16 * wt + lr;
        f32x4 y = rows.dot_f32q(reinterpret_cast<const float (*)[XS]>(s_X + 16 * wt * XS), lane, rsc);
        y *= DELTA ? sc : sc * s_gam[LP + w];
#pragma unroll
        for (int s = 0; s < Sh::ME; ++s) {
            if (4 * s >= e_end) break;
            y = __builtin_amdgcn_mfma_f32_16x16x4f32(vf[s], s_C[w * CS + 4 * s + lg], y, 0, 0, 0);
        }
        if (w >= n) continue;
        if (odd) {   // a value that is no number, for the nodes behind it alone
            for (int e = 0; e < e_end; ++e) {
                if (!on_path(w, e)) continue;
#pragma unroll
                for (int rr = 0; rr < 4; ++rr) {
                    const float v = entry_value<IOB>(vs.template value<IOB>(e, e < LP, p0 + 4 * lg + rr));
                    if (!tree_finite(v)) y[rr] = fmaf(s_C[w * CS + e], v, y[rr]);
                }
            }
        }
        *reinterpret_cast<f32x4 *>(&t.y[(((size_t)b * W + w) * H + h) * P + p0 + 4 * lg]) = y;
    }
}

template <int P, int N, int ST, bool IOB, bool DELTA>
hipError_t launch_tree_one(const TreeArgs &a, hipStream_t s) {
    const TreeLds at(a.W, a.r.L, N, DELTA);
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
