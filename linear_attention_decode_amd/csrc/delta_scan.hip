// delta_scan.hip -- the gated delta rule over packed prompts, chunk by chunk,
// on the matrix cores:
//     S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   y_t = S_t q_t
// (gdn.hip has the rule's source).  What a token adds is its correction u_t =
// beta_t (v_t - alpha_t S_{t-1} k_t) along k_t.  Over a chunk that starts from
// S, with D[i][j] = alpha_{j+1} ... alpha_i and g_i = alpha_0 ... alpha_i,
//     (I + A) U = diag(beta) (V - diag(g) K S^T),   A[i][j] = beta_i D[i][j] (k_i . k_j), j < i,
//     y_i = g_i S q_i + sum_{j<=i} (q_i . k_j) D[i][j] u_j,
//     S'  = g_last S + sum_j D[last][j] u_j k_j^T:
// the corrections of a chunk are one triangular system, solved for all columns
// of v at once by the inverse of I + A, which k, alpha and beta alone decide.
//
// The inverse: 16 x 16 diagonal blocks by substitution (a lane a column), the
// block below them from their product, T10 = -T11 A10 T00.  Substitution, not
// the doubling (I - A)(I + A^2)(I + A^4) ..: powers of A grow where keys are
// alike, and cancel.
//
// Every decay is a product of consecutive alphas, as in scan.hip.
//
// A workgroup takes one (sequence, head), wavefront w columns 16 w .. 16 w +
// 15 of S^T [N][P], which stay in its accumulators for the whole sequence.
// K S^T, then U = T R, then G U and K^T U contract over the rows of what the
// product before left in accumulators, (column l % 16, rows 4 (l / 16) + r):
// neither S nor U passes through LDS.
//
// Bound by the chain of a chunk's steps, one workgroup's behind the other, and in
// it by the float32 matrix instructions: three prompts of 97 tokens in all, 4 heads
// of 64 x 128, 19 us; one of 1000 tokens, 32 heads, 241 us for 32 chunks of 17000 cycles
// (staging 3000, A and G 3100, K S^T and Q S^T 4900, the inverse 1000 more, U and y
// 2000, the state 2900).  With heads of up to 64 columns a wavefront of its own
// inverts while the others multiply (347 us where one of them does both, and A and
// G come one by one).  bf16 io with heads of 64 or 128 columns takes delta_mx.hip.
//
// A value that is no number: one of v is to reach its column alone, from its
// token on, and one of k, beta or alpha nothing before its token; but the
// products run over the whole chunk, and 0 NaN is NaN.  So a chunk ends ahead
// of a token that holds one, which begins the next.
#include "scan_common.h"

namespace replay {

namespace {

constexpr int kQ = 32;    // tokens of a chunk
constexpr int kPad = 4;

typedef float acc4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ acc4 mma(float a, float b, acc4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

template <int P, int N>
struct Shape {
    // wavefronts with 16 columns of S^T each; where there is room, one more, which
    // inverts while they multiply
    static constexpr int NW = P / 16, ALL = NW <= 4 ? NW + 1 : NW, NT = ALL * 64;
    static constexpr int NR = N + kPad, PR = P + kPad, GR = kQ + kPad;   // LDS row strides
};

template <int P, int N>
struct Tile {
    float q[kQ][Shape<P, N>::NR], k[kQ][Shape<P, N>::NR], v[kQ][Shape<P, N>::PR];
    float g[kQ][Shape<P, N>::GR];   // (q_i . k_j) D[i][j], j <= i
    float a[kQ][Shape<P, N>::GR];   // A
    float t[kQ][Shape<P, N>::GR];   // (I + A)^-1
    float alpha[kQ], beta[kQ];
    float pre[kQ], suf[kQ];         // products of alpha within a tile of 16: up to and with i; behind j
    float d0[kQ], e[kQ];            // within the chunk: up to and with i; behind j
    int cut;                        // the first token but token 0 that holds a value that is no number
};

// The next chunk's rows in registers: 4 io elements a thread and piece.
template <int P, int N, bool IOB>
struct Ahead {
    static constexpr int NT = Shape<P, N>::NT;
    static constexpr int NV = kQ * N / 4, NP = kQ * P / 4;
    static constexpr int IN = (NV + NT - 1) / NT, IP = (NP + NT - 1) / NT;
    IoVec<IOB, 4> q[IN], k[IN], v[IP];
    float a, b;
    __device__ __forceinline__ void load(const ScanArgs &s, int t0, int n, int h, int g) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            const int e = (i * NT + tid) * 4, t = e / N;
            if (e < kQ * N && t < n) {
                const size_t at = ((size_t)(t0 + t) * s.G + g) * N + e % N;
                k[i].load(s.k, at);
                q[i].load(s.q, at);
            }
        }
#pragma unroll
        for (int i = 0; i < IP; ++i) {
            const int e = (i * NT + tid) * 4, t = e / P;
            if (e < kQ * P && t < n) v[i].load(s.v, ((size_t)(t0 + t) * s.H + h) * P + e % P);
        }
        a = 1.f;
        b = 0.f;
        if (tid < kQ && tid < n) {
            a = s.a[(size_t)(t0 + tid) * s.H + h];
            b = s.dt[(size_t)(t0 + tid) * s.H + h];
        }
    }
    // rows past the chunk's n tokens are zero, their decay one, their beta zero
    __device__ __forceinline__ void store(Tile<P, N> &m, int n) const {
        const int tid = threadIdx.x;
        int bad = kQ;
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            const int e = (i * NT + tid) * 4, t = e / N;
            if (e < kQ * N) {
                float f[4] = {0.f, 0.f, 0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
                if (t < n) {
                    k[i].widen(f);
                    q[i].widen(o);
                }
                *reinterpret_cast<f32x4 *>(&m.k[t][e % N]) = f32x4{f[0], f[1], f[2], f[3]};
                *reinterpret_cast<f32x4 *>(&m.q[t][e % N]) = f32x4{o[0], o[1], o[2], o[3]};
                if (t > 0 && !(finite(f[0]) && finite(f[1]) && finite(f[2]) && finite(f[3]))) bad = t < bad ? t : bad;
            }
        }
#pragma unroll
        for (int i = 0; i < IP; ++i) {
            const int e = (i * NT + tid) * 4, t = e / P;
            if (e < kQ * P) {
                float f[4] = {0.f, 0.f, 0.f, 0.f};
                if (t < n) v[i].widen(f);
                *reinterpret_cast<f32x4 *>(&m.v[t][e % P]) = f32x4{f[0], f[1], f[2], f[3]};
                if (t > 0 && !(finite(f[0]) && finite(f[1]) && finite(f[2]) && finite(f[3]))) bad = t < bad ? t : bad;
            }
        }
        if (tid < 64) {   // one whole wavefront: lanes kQ.. hold ones
            const float al = tid < n ? a : 1.f, be = tid < n ? b : 0.f;
            float pre = al, suf = al;
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) {
                const float up = __shfl_up(pre, d, 16), down = __shfl_down(suf, d, 16);
                if ((tid & 15) >= d) pre *= up;
                if ((tid & 15) + d < 16) suf *= down;
            }
            const float total0 = __shfl(pre, 15), total1 = __shfl(pre, 31);
            suf = __shfl_down(suf, 1, 16);
            if ((tid & 15) == 15) suf = 1.f;
            if (tid < kQ) {
                m.alpha[tid] = al;
                m.beta[tid] = be;
                m.pre[tid] = pre;
                m.suf[tid] = suf;
                m.d0[tid] = tid < 16 ? pre : total0 * pre;
                m.e[tid] = tid < 16 ? suf * total1 : suf;
                if (tid > 0 && !(finite(al) && finite(be))) bad = tid < bad ? tid : bad;
            }
        }
        if (bad < kQ) atomicMin(&m.cut, bad);
    }
};

// G and A, tile (ti, tj), transposed: rows j = 4 lg + r, column i = c
template <int P, int N>
__device__ __forceinline__ void weigh(Tile<P, N> &m, int ti, int tj, int c, int lg) {
    acc4 dg = {0.f, 0.f, 0.f, 0.f}, da = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < N / 16; ++t) {
        const f32x4 kj = *reinterpret_cast<const f32x4 *>(&m.k[16 * tj + c][16 * t + 4 * lg]);
        const f32x4 qi = *reinterpret_cast<const f32x4 *>(&m.q[16 * ti + c][16 * t + 4 * lg]);
        const f32x4 ki = *reinterpret_cast<const f32x4 *>(&m.k[16 * ti + c][16 * t + 4 * lg]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            da = mma(kj[r], ki[r], da);
            dg = mma(kj[r], qi[r], dg);
        }
    }
    const int i = 16 * ti + c, j0 = 16 * tj + 4 * lg;
    const f32x4 D = ti != tj ? m.pre[i] * *reinterpret_cast<const f32x4 *>(&m.suf[j0]) : diagonal_decays(&m.alpha[16 * tj], c, lg);
    const float be = m.beta[i];
    f32x4 o, a;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        o[r] = j0 + r <= i ? dg[r] * D[r] : 0.f;
        a[r] = j0 + r < i ? be * (da[r] * D[r]) : 0.f;
    }
    *reinterpret_cast<f32x4 *>(&m.g[i][j0]) = o;
    *reinterpret_cast<f32x4 *>(&m.a[i][j0]) = a;
}

// (I + A)^-1, by one wavefront: the diagonal blocks, lane (block, column c)
// a column, then the block below.
template <int P, int N>
__device__ __forceinline__ void invert(Tile<P, N> &m, int lane) {
    const int c = lane & 15, lg = lane >> 4;
    if (lane < 32) {
        const int b0 = lane & 16;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = i == c ? 1.f : 0.f;
#pragma unroll
            for (int j4 = 0; j4 < i; j4 += 4) {
                const f32x4 a = *reinterpret_cast<const f32x4 *>(&m.a[b0 + i][b0 + j4]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (j4 + r < i) x[i] = fmaf(-a[r], x[j4 + r], x[i]);
            }
            m.t[b0 + i][b0 + c] = x[i];
            if (b0 == 0) m.t[i][16 + c] = 0.f;
        }
    }
    wave_lds_sync();
    acc4 d = {0.f, 0.f, 0.f, 0.f}, o = {0.f, 0.f, 0.f, 0.f};
    const f32x4 a10 = *reinterpret_cast<const f32x4 *>(&m.a[16 + c][4 * lg]);
#pragma unroll
    for (int r = 0; r < 4; ++r) d = mma(a10[r], m.t[4 * lg + r][c], d);
    const f32x4 t11 = *reinterpret_cast<const f32x4 *>(&m.t[16 + c][16 + 4 * lg]);
#pragma unroll
    for (int r = 0; r < 4; ++r) o = mma(t11[r], d[r], o);
#pragma unroll
    for (int r = 0; r < 4; ++r) m.t[16 + 4 * lg + r][c] = -o[r];
}

template <int P, int N, bool IOB>
__global__ __launch_bounds__((Shape<P, N>::NT)) void delta_scan_kernel(ScanArgs s) {
    using Sh = Shape<P, N>;
    constexpr int NW = Sh::NW, TN = N / 16;
    __shared__ __align__(16) Tile<P, N> m;

    Place place;
    if (!find_place(s, 1, &place)) return;
    const int h = place.h, b = place.b, g = place.g;
    const Span sp = find_span(s, b, 0);
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 15, lg = lane >> 4;
    if (h == 0 && !sp.run && tid == 0) raise_seq_error(s.err, b, REPLAY_SEQERR_BAD_RANGE);
    if (!sp.run) return;

    const size_t bh = (size_t)b * s.H + h, tile = (size_t)P * N;
    const size_t row = (size_t)(16 * w + c) * N + 4 * lg;   // this lane's 4 columns of tile 0 in S [P][N]
    acc4 S[TN];
#pragma unroll
    for (int t = 0; t < TN; ++t) {
        S[t] = acc4{0.f, 0.f, 0.f, 0.f};
        if (s.s_in && w < NW) S[t] = *reinterpret_cast<const acc4 *>(s.s_in + bh * tile + row + 16 * t);
    }

    Ahead<P, N, IOB> ahead;
    ahead.load(s, sp.t0, sp.n, h, g);
    if (tid == 0) m.cut = kQ;
    int at = 0;
    while (at < sp.n) {
        int n = sp.n - at < kQ ? sp.n - at : kQ;
        lds_barrier();   // the last chunk is read to its end
        ahead.store(m, n);
        lds_barrier();
        if (m.cut < n) {   // uniform
            n = m.cut;
            lds_barrier();
            ahead.store(m, n);
            lds_barrier();
        }
        const int next = at + n;
        if (next < sp.n) ahead.load(s, sp.t0 + next, sp.n - next, h, g);

        for (int x = w; x < 3; x += Sh::ALL) weigh(m, x == 0 ? 0 : 1, x == 2 ? 1 : 0, c, lg);
        lds_barrier();
        if (tid == 0) m.cut = kQ;   // (all have read it)
        if (w == Sh::ALL - 1) {
            __builtin_amdgcn_s_setprio(3);   // the others wait for it
            invert(m, lane);
            __builtin_amdgcn_s_setprio(0);
        }
        if (w >= NW) {
            lds_barrier();   // the inverse
            at = next;
            continue;
        }
        // K S^T and Q S^T, rows i = 16 ti + 4 lg + r, column p = c of the wavefront's 16
        acc4 ks[2], qs[2];
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
            ks[ti] = qs[ti] = acc4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < TN; ++t) {
                const f32x4 kk = *reinterpret_cast<const f32x4 *>(&m.k[16 * ti + c][16 * t + 4 * lg]);
                const f32x4 qq = *reinterpret_cast<const f32x4 *>(&m.q[16 * ti + c][16 * t + 4 * lg]);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    ks[ti] = mma(kk[r], S[t][r], ks[ti]);
                    qs[ti] = mma(qq[r], S[t][r], qs[ti]);
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * ti + 4 * lg + r;
                ks[ti][r] = m.beta[i] * fmaf(-m.d0[i], ks[ti][r], m.v[i][16 * w + c]);
                qs[ti][r] *= m.d0[i];
            }
        }
        lds_barrier();   // the inverse
        acc4 u[2];
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
            u[ti] = acc4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int tj = 0; tj <= ti; ++tj) {
                const f32x4 tt = *reinterpret_cast<const f32x4 *>(&m.t[16 * ti + c][16 * tj + 4 * lg]);
#pragma unroll
                for (int r = 0; r < 4; ++r) u[ti] = mma(tt[r], ks[tj][r], u[ti]);
            }
        }
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
            acc4 y = qs[ti];
#pragma unroll
            for (int tj = 0; tj <= ti; ++tj) {
                const f32x4 gg = *reinterpret_cast<const f32x4 *>(&m.g[16 * ti + c][16 * tj + 4 * lg]);
#pragma unroll
                for (int r = 0; r < 4; ++r) y = mma(gg[r], u[tj][r], y);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * ti + 4 * lg + r;
                if (i < n) {
                    const size_t o = ((size_t)(sp.t0 + at + i) * s.H + h) * P + 16 * w + c;
                    if constexpr (IOB)
                        static_cast<uint16_t *>(s.y)[o] = (uint16_t)f32_to_bf16_bits(y[r]);
                    else
                        static_cast<float *>(s.y)[o] = y[r];
                }
            }
        }
        // S^T <- (whole decay) S^T + K^T (e U)
        const float all = m.d0[kQ - 1];
#pragma unroll
        for (int t = 0; t < TN; ++t) S[t] *= all;
#pragma unroll
        for (int tj = 0; tj < 2; ++tj)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int j = 16 * tj + 4 * lg + r;
                const float x = u[tj][r] * m.e[j];
#pragma unroll
                for (int t = 0; t < TN; ++t) S[t] = mma(m.k[j][16 * t + c], x, S[t]);
            }
        at = next;
    }
    if (w >= NW) return;
#pragma unroll
    for (int t = 0; t < TN; ++t) *reinterpret_cast<acc4 *>(s.s_out + bh * tile + row + 16 * t) = S[t];
}

template <int P, int N, bool IOB>
hipError_t launch_one(const ScanArgs &a, hipStream_t s) {
    delta_scan_kernel<P, N, IOB><<<scan_blocks(a, 1), Shape<P, N>::NT, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_scan(int P, int N, const ScanArgs &a, hipStream_t s) {
    if (a.window > 0) return launch_delta_mx(P, N, a, s);   // bf16, but for heads of 16 columns (delta_window)
    if (P == 16 && N == 16) return a.io_bf16 ? launch_one<16, 16, true>(a, s) : launch_one<16, 16, false>(a, s);
    if (a.io_bf16) return hipErrorInvalidValue;
    if (P == 64 && N == 64) return launch_one<64, 64, false>(a, s);
    if (P == 64 && N == 128) return launch_one<64, 128, false>(a, s);
    if (P == 128 && N == 128) return launch_one<128, 128, false>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace replay
