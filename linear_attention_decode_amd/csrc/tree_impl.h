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
// A workgroup takes one (sequence, head), a wavefront 16 of its rows: their
// tile of S0 is on its way while the workgroup forms the weights C (and x) in
// LDS; then S0 x^T and V^T C^T go into one accumulator, both on
// v_mfma_f32_16x16x4_f32, 16 nodes at a time.
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

// LDS, in floats: weights C [WP][CS]; then the decays D [WP][WP] (gated delta
// rule: and A^T [ES][CS], the ring's own decays [LP][LP]), which the queries
// [WP][XS] replace.
struct TreeLds {
    int WP, LP, ES, CS, a, rr, total;
    __host__ __device__ TreeLds(int W, int L, int N, bool delta) {
        WP = (W + 15) / 16 * 16;
        LP = (L + 15) / 16 * 16;
        ES = LP + WP;
        CS = ES + 4;
        a = WP * CS + WP * WP;
        rr = a + ES * CS;
        const int first = delta ? rr + LP * LP : a, second = WP * (CS + N + 4);
        total = first > second ? first : second;
    }
};

// Entry e's row: ring entries 0 .. LP - 1 (there are count), then the nodes.
// False: there is none.
struct Entries {
    const TreeArgs &t;
    int b, g, h, bmod, count, n, LP;
    __device__ __forceinline__ bool at(int e, bool v, const void **base, size_t *row) const {
        const RingView &r = t.r;
        if (e < LP) {
            if (e >= count) return false;
            *base = v ? r.v : r.k;
            *row = (v ? (size_t)b * r.H + h : (size_t)b * r.G + g) * r.L + ring_slot(bmod, e, r.L);
            return true;
        }
        if (e - LP >= n) return false;
        *base = v ? t.v : t.k;
        const size_t token = (size_t)b * t.W + (e - LP);
        *row = v ? token * r.H + h : token * r.G + g;
        return true;
    }
};

// A lane's part of an operand of k . k or k . q: 8 of every 32 columns of a row.
template <int N, bool IOB>
struct DotRow {
    static constexpr int KB = (N + 31) / 32;
    uint4 b[IOB ? KB : 1];
    f32x4 f[IOB ? 1 : KB][2];
    __device__ __forceinline__ void load(const void *base, size_t row, bool there, int lane) {
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int c = 32 * kb + 8 * (lane >> 4);
            const bool in = there && c < N;
            if constexpr (IOB) {
                b[kb] = uint4{0u, 0u, 0u, 0u};
                if (in) b[kb] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + row * N + c);
            } else {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    f[kb][x] = f32x4{0.f, 0.f, 0.f, 0.f};
                    if (in) f[kb][x] = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(base) + row * N + c + 4 * x);
                }
            }
        }
    }
    // rows of this (M) by rows of o (N): register r is (4 (lane / 16) + r, lane % 16)
    __device__ __forceinline__ f32x4 dots(const DotRow &o) const {
        f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            if constexpr (IOB) {
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(b[kb]), as_bf16x8(o.b[kb]), d, 0, 0, 0);
            } else {
#pragma unroll
                for (int t = 0; t < 8; ++t) d = __builtin_amdgcn_mfma_f32_16x16x4f32(f[kb][t >> 2][t & 3], o.f[kb][t >> 2][t & 3], d, 0, 0, 0);
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
    float *s_C = lds, *s_D = lds + WP * CS, *s_A = lds + at.a, *s_RR = lds + at.rr, *s_X = lds + WP * CS;
    const int wt_n = (n + 15) / 16, et_n = LP / 16 + wt_n, e_end = LP + n;
    const Entries ent{t, b, g, h, base % L, count, n, LP};

    // raw dots: C[w][e] = k_e . q_w, and A^T[j][i] = k_j . k_i of tiles i >= j
    {
        const int cq = et_n * wt_n, total = cq + (DELTA ? et_n * (et_n + 1) / 2 : 0);
        for (int x = wave; x < total; x += NW) {
            int et, ot;
            const bool kk = x >= cq;
            if (!kk) {
                et = x / wt_n;
                ot = x % wt_n;
            } else {
                ot = 0;
                int left = x - cq;
                while (left > ot) left -= ++ot;
                et = left;   // et <= ot
            }
            DotRow<N, IOB> A, B;
            const void *src = nullptr;
            size_t row = 0;
            bool there = ent.at(16 * et + lr, false, &src, &row);
            A.load(src, row, there, lane);
            if (kk) {
                there = ent.at(16 * ot + lr, false, &src, &row);
            } else {
                const int w = 16 * ot + lr;
                there = w < n;
                src = t.q;
                row = ((size_t)b * W + w) * r.G + g;
            }
            B.load(src, row, there, lane);
            const f32x4 d = A.dots(B);
            if (!kk) {
                *reinterpret_cast<f32x4 *>(&s_C[(16 * ot + lr) * CS + 16 * et + 4 * lg]) = d;
            } else {
#pragma unroll
                for (int rr = 0; rr < 4; ++rr) s_A[(16 * et + 4 * lg + rr) * CS + 16 * ot + lr] = d[rr];
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
        // D[w][j], row by row: the parent's, one factor more
        float cur = 0.f;
        for (int w = 0; w < n; ++w) {
            const int pw = __builtin_amdgcn_readlane(tree.parent, w);
            const float aw = bcast(na, w);
            float prev = 0.f;
            if (pw >= 0) prev = pw == w - 1 ? cur : (lane < WP ? s_D[pw * WP + lane] : 0.f);
            cur = lane == w ? 1.f : prev * aw;
            if (lane < WP) s_D[w * WP + lane] = cur;
        }
        if constexpr (DELTA) {
            float p = 1.f;
            for (int i = 0; i < count; ++i) {   // a behind j up to and with i
                if (i > lane) p *= bcast(ra, i);
                if (lane < LP) s_RR[lane * LP + i] = p;
            }
        }
    }
    __syncthreads();

    // weights: the dots of what lies on the node's path, decayed (selects, not
    // factors of 0: another branch's NaN stays there)
    auto on_path = [&](int w, int e) { return w < n && (e < LP ? e < count : (s_anc[w] >> (e - LP) & 1) != 0); };
    auto decay = [&](int w, int e) { return e < LP ? s_R[e] * s_path[w] : s_D[w * WP + e - LP]; };
    for (int i = tid; i < 16 * wt_n * ES; i += NT) {
        const int w = i / ES, e = i % ES;
        float *c = s_C + w * CS + e;
        *c = on_path(w, e) ? decay(w, e) * *c * (DELTA ? 1.f : s_dt[e]) : 0.f;
    }
    if constexpr (DELTA) {
        for (int x = tid; x < ES * ES; x += NT) {
            const int j = x / ES, i = x % ES;
            if (i >= LP + 16 * wt_n) continue;
            float c = 0.f;
            if (i > j && (i < LP ? i < count : on_path(i - LP, j)))
                c = (i < LP ? s_RR[j * LP + i] : decay(i - LP, j)) * s_A[j * CS + i] * s_dt[i];
            s_A[j * CS + i] = c;
        }
        __syncthreads();
        // C (I + A) = G, a node's row from its last entry back: four lanes a
        // node, each a quarter of the sum
        const int part = lane & 3;
        for (int wt = wave; wt < wt_n; wt += NW) {
            float *row = s_C + (16 * wt + (lane >> 2)) * CS;
            for (int j = e_end - 2; j >= 0; --j) {
                if (j >= count && j < LP) j = count - 1;   // (count = 0: -1, none is left)
                if (j < 0) break;
                const float *col = s_A + j * CS;
                float sum = 0.f;
                for (int i = (j + 1 & ~3) + part; i < e_end; i += 4) {
                    const float c = row[i];
                    if (i > j && c != 0.f) sum = fmaf(c, col[i], sum);   // (0: not on the path, or without part in it)
                }
                sum += lane_partner(sum, 0);
                sum += lane_partner(sum, 1);
                if (part == 0 && sum != 0.f) row[j] -= sum;
                wave_lds_sync();
            }
        }
        __syncthreads();
        for (int i = tid; i < 16 * wt_n * ES; i += NT) {
            const int w = i / ES, e = i % ES;
            s_C[w * CS + e] = on_path(w, e) ? s_C[w * CS + e] * s_dt[e] : 0.f;
        }
    }
    __syncthreads();

    // the queries, which take the place of the decays
    if constexpr (!DELTA) {
        for (int i = tid; i < 16 * wt_n * (N / 4); i += NT) {
            const int w = i / (N / 4), c = i % (N / 4) * 4;
            float q[4] = {0.f, 0.f, 0.f, 0.f};
            if (w < n) load_io4<IOB>(t.q, (((size_t)b * W + w) * r.G + g) * N + c, q);
            *reinterpret_cast<f32x4 *>(&s_X[w * XS + c]) = f32x4{q[0], q[1], q[2], q[3]};
        }
    } else {
        for (int nt = wave; nt < N / 16; nt += NW) {
            float kc[Sh::ME];   // column 16 nt + lr of entries 4 s + lg
#pragma unroll
            for (int s = 0; s < Sh::ME; ++s) {
                kc[s] = 0.f;
                const int e = 4 * s + lg;
                const void *src;
                size_t row;
                if (e < e_end && ent.at(e, false, &src, &row)) {
                    const float k = load_io1<IOB>(src, row * N + 16 * nt + lr);
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
    __syncthreads();

    // y^T: rows p0 + 4 lg + rr, nodes 16 wt + lr
    rows.transpose(s_T[WT::COAL ? wave : 0], lane);
    float vc[Sh::ME];   // column p0 + lr of entries 4 s + lg
    bool odd = false;
#pragma unroll
    for (int s = 0; s < Sh::ME; ++s) {
        vc[s] = 0.f;
        const int e = 4 * s + lg;
        const void *src;
        size_t row;
        if (e < e_end && ent.at(e, true, &src, &row)) {
            const float v = load_io1<IOB>(src, row * P + p0 + lr);
            if (tree_finite(v)) vc[s] = v;
            else odd = true;
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
            y = __builtin_amdgcn_mfma_f32_16x16x4f32(vc[s], s_C[w * CS + 4 * s + lg], y, 0, 0, 0);
        }
        if (w >= n) continue;
        if (odd) {   // a value that is no number, for the nodes behind it alone
            for (int e = 0; e < e_end; ++e) {
                const void *src;
                size_t row;
                if (!ent.at(e, true, &src, &row) || (e >= LP && !(s_anc[w] >> (e - LP) & 1))) continue;
#pragma unroll
                for (int rr = 0; rr < 4; ++rr) {
                    const float v = load_io1<IOB>(src, row * P + p0 + 4 * lg + rr);
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
