// scan.hip -- the recurrence over packed prompts, chunk by chunk, on the
// matrix cores:
//     S_t = a_t S_{t-1} + dt_t v_t k_t^T,   y_t = S_t q_t
// (page "ReplaySSM: Cachear Inputs, No Estado", section "La solucion", eqs.
// "Forma resumen" and "Forma historia").  Over a chunk of kQ tokens that
// starts from state S, with D[i][j] = a_{j+1} ... a_i,
//     y_i = (a_0 ... a_i) S q_i + sum_{j<=i} (q_i . k_j) D[i][j] dt_j v_j,
//     S'  = (a_0 ... a_last) S + sum_j D[last][j] dt_j v_j k_j^T:
// four matrix products a chunk, and one pass over the inputs.
//
// Every decay is a product of a's, never a quotient or a difference of
// logarithms: a = 0 (a reset), values that underflow and long chunks are as
// exact as the recurrence.  D over two tiles of 16 tokens is the product of
// the later tile's prefix, the earlier one's suffix and the tiles between.
// Only a's of consecutive tokens are multiplied, and these products have to be
// finite, as they always are for |a| <= 1: one that overflows has met no state
// yet, and a state of zero or a reset behind it would make it NaN.
//
// A workgroup takes one (sequence, head, segment), wavefront w columns
// 16 w .. 16 w + 15 of S^T [N][P], which stay in its accumulators for the
// whole segment: a 16 x 16 accumulator tile (lane: column l % 16, rows
// 4 (l / 16) + r) is laid out as the operand of the product S q, whose
// contraction runs over its rows, so the state never passes through LDS.
//
// Bound by the float32 matrix instructions (a sixteenth of the bf16 rate):
// four ragged sequences of 1999 tokens in all, 32 heads of 128 x 128, in
// segments: 122 us (32 us for their states, 7 us to join them, the rest for
// the outputs), against 20 us for the bytes and some 35 us for the products
// at full rate.  16 x 16 heads, a wavefront each: 15013 tokens of 128 heads in
// bf16 196 us, against 31 us for the bytes, 16100 vector instructions a
// wavefront to 1200 matrix ones.  97 tokens of 12 (sequence, head) pairs take
// 16 us, one chunk's steps behind the other.
#include "scan_common.h"

#include <algorithm>

namespace replay {

namespace {

constexpr int kQ = 32;    // tokens of a chunk
constexpr int kPad = 4;   // floats behind an LDS row: 16 rows' 16-byte reads touch distinct banks

typedef float acc4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ acc4 mma(float a, float b, acc4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

template <int P, int N>
struct Shape {
    static constexpr int NW = P / 16, NT = NW * 64;
    static constexpr int NR = N + kPad, PR = P + kPad, GR = kQ + kPad;   // LDS row strides
};

template <int P, int N>
struct Tile {
    float q[kQ][Shape<P, N>::NR], k[kQ][Shape<P, N>::NR], v[kQ][Shape<P, N>::PR];
    float g[kQ][Shape<P, N>::GR];   // g[i][j] = (q_i . k_j) D[i][j] dt_j, j <= i
    float a[kQ], dt[kQ];
    float pre[kQ], suf[kQ];         // products of a within a tile of 16: up to and with i; behind j
    float d0[kQ], e[kQ];            // within the chunk: up to and with i; dt_j times those behind j
};

// The next chunk's rows in registers: 4 io elements a thread and piece.
template <int P, int N, bool IOB>
struct Ahead {
    static constexpr int NT = Shape<P, N>::NT;
    static constexpr int NV = kQ * N / 4, NP = kQ * P / 4;
    static constexpr int IN = (NV + NT - 1) / NT, IP = (NP + NT - 1) / NT;
    IoVec<IOB, 4> q[IN], k[IN], v[IP];
    float a, dt;
    __device__ __forceinline__ void load(const ScanArgs &s, int t0, int n, int h, int g, bool need_q) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            const int e = (i * NT + tid) * 4, t = e / N;
            if (e < kQ * N && t < n) {
                const size_t at = ((size_t)(t0 + t) * s.G + g) * N + e % N;
                k[i].load(s.k, at);
                if (need_q) q[i].load(s.q, at);
            }
        }
#pragma unroll
        for (int i = 0; i < IP; ++i) {
            const int e = (i * NT + tid) * 4, t = e / P;
            if (e < kQ * P && t < n) v[i].load(s.v, ((size_t)(t0 + t) * s.H + h) * P + e % P);
        }
        a = 1.f;
        dt = 0.f;
        if (tid < kQ && tid < n) {
            a = s.a[(size_t)(t0 + tid) * s.H + h];
            dt = s.dt[(size_t)(t0 + tid) * s.H + h];
        }
    }
    // rows past the chunk's n tokens are zero, their decay one, their step zero
    __device__ __forceinline__ void store(Tile<P, N> &m, int n, bool need_q) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            const int e = (i * NT + tid) * 4, t = e / N;
            if (e < kQ * N) {
                float f[4] = {0.f, 0.f, 0.f, 0.f};
                if (t < n) k[i].widen(f);
                *reinterpret_cast<f32x4 *>(&m.k[t][e % N]) = f32x4{f[0], f[1], f[2], f[3]};
                if (need_q) {
                    if (t < n) q[i].widen(f);
                    *reinterpret_cast<f32x4 *>(&m.q[t][e % N]) = f32x4{f[0], f[1], f[2], f[3]};
                }
            }
        }
#pragma unroll
        for (int i = 0; i < IP; ++i) {
            const int e = (i * NT + tid) * 4, t = e / P;
            if (e < kQ * P) {
                float f[4] = {0.f, 0.f, 0.f, 0.f};
                if (t < n) v[i].widen(f);
                *reinterpret_cast<f32x4 *>(&m.v[t][e % P]) = f32x4{f[0], f[1], f[2], f[3]};
            }
        }
        if (tid < 64) {   // one whole wavefront: lanes kQ.. hold ones
            float pre = a, suf = a;
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
                m.a[tid] = a;
                m.dt[tid] = dt;
                m.pre[tid] = pre;
                m.suf[tid] = suf;
                m.d0[tid] = tid < 16 ? pre : total0 * pre;
                m.e[tid] = dt * (tid < 16 ? suf * total1 : suf);
            }
        }
    }
};

// STATE_ONLY: the segment's own state from zero, and its whole decay, to the
// workspace; else outputs, from the state before the segment.
template <int P, int N, bool IOB, bool STATE_ONLY>
__global__ __launch_bounds__((Shape<P, N>::NT)) void scan_kernel(ScanArgs s) {
    using Sh = Shape<P, N>;
    constexpr int NW = Sh::NW, TN = N / 16;
    __shared__ Tile<P, N> m;

    Place place;
    if (!find_place(s, 1, &place)) return;
    const int h = place.h, seg = place.seg, b = place.b, g = place.g;
    const Span sp = find_span(s, b, seg);
    const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63, c = lane & 15, lg = lane >> 4;
    if (!STATE_ONLY && seg == 0 && h == 0 && !sp.run && tid == 0) raise_seq_error(s.err, b, REPLAY_SEQERR_BAD_RANGE);
    if (!sp.run || (STATE_ONLY && sp.last)) return;

    const size_t bh = (size_t)b * s.H + h, tile = (size_t)P * N;
    const size_t row = (size_t)(16 * w + c) * N + 4 * lg;   // this lane's 4 columns of tile 0 in S [P][N]
    acc4 S[TN];
    const float *from = STATE_ONLY ? nullptr
                        : seg > 0 ? s.ws + (bh * (s.nseg - 1) + seg - 1) * tile
                                  : (s.s_in ? s.s_in + bh * tile : nullptr);
#pragma unroll
    for (int t = 0; t < TN; ++t) {
        S[t] = acc4{0.f, 0.f, 0.f, 0.f};
        if (from) S[t] = *reinterpret_cast<const acc4 *>(from + row + 16 * t);
    }

    Ahead<P, N, IOB> ahead;
    float decay = 1.f;
    ahead.load(s, sp.t0, sp.n, h, g, !STATE_ONLY);
    for (int at = 0; at < sp.n; at += kQ) {
        const int n = sp.n - at < kQ ? sp.n - at : kQ;
        if (at > 0) __syncthreads();   // the last chunk is read to its end
        ahead.store(m, n, !STATE_ONLY);
        if (at + kQ < sp.n) ahead.load(s, sp.t0 + at + kQ, sp.n - at - kQ, h, g, !STATE_ONLY);
        __syncthreads();

        if constexpr (!STATE_ONLY) {
            // g, tile (ti, tj), transposed: rows j = 4 lg + r, column i = c
            for (int x = w; x < 3; x += NW) {
                const int ti = x == 0 ? 0 : 1, tj = x == 2 ? 1 : 0;
                acc4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int t = 0; t < TN; ++t) {
                    const f32x4 kk = *reinterpret_cast<const f32x4 *>(&m.k[16 * tj + c][16 * t + 4 * lg]);
                    const f32x4 qq = *reinterpret_cast<const f32x4 *>(&m.q[16 * ti + c][16 * t + 4 * lg]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) d = mma(kk[r], qq[r], d);
                }
                const int i = 16 * ti + c, j0 = 16 * tj + 4 * lg;
                f32x4 o;
                if (ti != tj) {
                    const float p = m.pre[i];
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[r] = d[r] * (p * m.suf[j0 + r] * m.dt[j0 + r]);
                } else {
                    // a_{j+1} ... a_i for this lane's four j, by one walk down from the tile's end
                    float p = 1.f;
                    f32x4 dec = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int jj = 15; jj >= 0; --jj) {
                        if (jj < 15) p = c > jj ? p * m.a[16 * tj + jj + 1] : 1.f;
                        if (lg == jj / 4) dec[jj & 3] = p;
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[r] = j0 + r <= i ? d[r] * (dec[r] * m.dt[j0 + r]) : 0.f;
                }
                *reinterpret_cast<f32x4 *>(&m.g[i][j0]) = o;
            }
            __syncthreads();
            // y^T, rows p = 4 lg + r of the wavefront's 16, column i = c of the token tile
#pragma unroll
            for (int ti = 0; ti < 2; ++ti) {
                const int i = 16 * ti + c;
                acc4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int t = 0; t < TN; ++t) {
                    const f32x4 qq = *reinterpret_cast<const f32x4 *>(&m.q[i][16 * t + 4 * lg]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) y = mma(S[t][r], qq[r], y);
                }
                y *= m.d0[i];
                // A weight of 0 does not hide a later token's NaN or infinity
                // in v: the product goes without them, and they are added for
                // the tokens from theirs on.
                bool odd = false;
#pragma unroll
                for (int tj = 0; tj <= ti; ++tj) {
                    const f32x4 gg = *reinterpret_cast<const f32x4 *>(&m.g[i][16 * tj + 4 * lg]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float v = m.v[16 * tj + 4 * lg + r][16 * w + c];
                        odd |= !finite(v);
                        y = mma(finite(v) ? v : 0.f, gg[r], y);
                    }
                }
                if (__any(odd))
                    for (int j = 0; j < 16 * (ti + 1); ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float v = m.v[j][16 * w + 4 * lg + r];
                            if (j <= i && !finite(v)) y[r] = fmaf(m.g[i][j], v, y[r]);
                        }
                if (i < n) {
                    const size_t o = ((size_t)(sp.t0 + at + i) * s.H + h) * P + 16 * w + 4 * lg;
                    if constexpr (IOB)
                        *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(s.y) + o) =
                            u32x2{f32x2_to_bf16_pair(y[0], y[1]), f32x2_to_bf16_pair(y[2], y[3])};
                    else
                        *reinterpret_cast<f32x4 *>(static_cast<float *>(s.y) + o) = f32x4{y[0], y[1], y[2], y[3]};
                }
            }
        }
        // S^T <- (whole decay) S^T + K^T (e V)
        const float all = m.d0[kQ - 1];
        decay *= all;
#pragma unroll
        for (int t = 0; t < TN; ++t) S[t] *= all;
#pragma unroll
        for (int st = 0; st < kQ / 4; ++st) {
            const int j = 4 * st + lg;
            const float u = m.v[j][16 * w + c] * m.e[j];
#pragma unroll
            for (int t = 0; t < TN; ++t) S[t] = mma(m.k[j][16 * t + c], u, S[t]);
        }
    }

    float *to = nullptr;
    if constexpr (STATE_ONLY) {
        to = s.ws + (bh * (s.nseg - 1) + seg) * tile;
        if (tid == 0) s.ws_decay[bh * (s.nseg - 1) + seg] = decay;
    } else if (sp.last) {
        to = s.s_out + bh * tile;
    }
    if (to) {
#pragma unroll
        for (int t = 0; t < TN; ++t) *reinterpret_cast<acc4 *>(to + row + 16 * t) = S[t];
    }
}

// The states before segments 1..: ws slot i, segment i's own state on entry,
// the state before segment i + 1 on return.
__global__ __launch_bounds__(256) void scan_join_kernel(ScanArgs s, int tile4) {
    const int per = (tile4 + 255) / 256;
    const int bh = blockIdx.x / per, e = (blockIdx.x % per) * 256 + threadIdx.x;
    if (e >= tile4) return;
    const int b = bh / s.H;
    f32x4 *ws = reinterpret_cast<f32x4 *>(s.ws) + (size_t)bh * (s.nseg - 1) * tile4 + e;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (s.s_in) x = reinterpret_cast<const f32x4 *>(s.s_in)[(size_t)bh * tile4 + e];
    if (!find_span(s, b, 0).run) return;
    const int ends = (s.cu[b + 1] - s.cu[b] - 1) / s.seg_len;   // segments that are followed by another
    const float *decay = s.ws_decay + (size_t)bh * (s.nseg - 1);
    constexpr int U = 8;   // segments whose states are loaded together
    for (int seg0 = 0; seg0 < ends; seg0 += U) {
        f32x4 own[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int seg = seg0 + u < ends ? seg0 + u : ends - 1;
            own[u] = ws[(size_t)seg * tile4];
            d[u] = decay[seg];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (seg0 + u >= ends) break;
            x = d[u] * x + own[u];
            ws[(size_t)(seg0 + u) * tile4] = x;
        }
    }
}

template <int P, int N, bool IOB>
hipError_t launch_one(const ScanArgs &a, bool state_only, hipStream_t s) {
    const unsigned blocks = scan_blocks(a, 1);
    if (state_only)
        scan_kernel<P, N, IOB, true><<<blocks, Shape<P, N>::NT, 0, s>>>(a);
    else
        scan_kernel<P, N, IOB, false><<<blocks, Shape<P, N>::NT, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_kernel(int P, int N, const ScanArgs &a, bool state_only, hipStream_t s) {
    if (scan_mx_supported(P, N, a)) return launch_scan_mx(P, N, a, state_only, s);
    if (P == 16 && N == 16) return a.io_bf16 ? launch_one<16, 16, true>(a, state_only, s) : launch_one<16, 16, false>(a, state_only, s);
    if (P == 64 && N == 64) return launch_one<64, 64, false>(a, state_only, s);
    if (P == 64 && N == 128) return launch_one<64, 128, false>(a, state_only, s);
    if (P == 128 && N == 128) return launch_one<128, 128, false>(a, state_only, s);
    return hipErrorInvalidValue;
}

}  // namespace

// Segments of a sequence, where the workgroups of whole sequences leave CUs
// without work.  A segment costs a second reading of its k and v and a state
// that is written, joined and read; what it saves is the chain of chunks, 4
// to 5 us each.  Two are never the best: both passes over a half are about as
// long as one over the whole.  So: as many as give a CU one workgroup, of a chunk
// or more, and up to two (float32, whose matrix instructions take most of its
// time and gain from evener shares: four) while segments stay long; and where
// whole chunks would make two of three, segments of one chunk (float32, up to
// 255 tokens: 224 of 24 heads of 64 x 128 whole 46 us, in two 44, in four 31;
// of 85 heads of 64 x 64 59, 54, 38).  Measured
// against segments of 256 (192) tokens or more alone: one prompt of 512 tokens,
// 24 heads of 64 x 128, bf16 41 -> 26 us, float32 82 -> 35; 2048 tokens of 8
// heads of 64 x 64, bf16 30 -> 22; four of 512 tokens, 128 heads, unsplit 45
// us, in two 75.  Below the shortest lengths here whole sequences are as fast
// (320 tokens of 128 heads, bf16: 29 us, in three segments 36).
int scan_segments(int P, int N, int B, int H, int G, bool bf16, int T, int max_len, int *seg_len) {
    const int longest = max_len < T ? max_len : T;
    const int64_t groups = (int64_t)B * H / (bf16 ? scan_mx_heads(P, H, G) : 1);
    const int64_t even = std::min<int64_t>((bf16 ? 512 : 1024) / groups, longest / (bf16 ? 256 : 192));
    const int64_t chain = std::min<int64_t>(256 / groups, longest / kScanChunk);
    int64_t n = std::max(even, chain);
    if (n < 3 || longest < (bf16 ? 384 : 192)) n = 1;
    const int64_t len = (longest + n - 1) / n;
    *seg_len = (int)((len + kScanChunk - 1) / kScanChunk * kScanChunk);
    if (n > 1 && longest <= 2 * *seg_len) *seg_len = kScanChunk;
    return (int)((longest + *seg_len - 1) / *seg_len);
}

hipError_t launch_scan(int P, int N, const ScanArgs &a, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (a.nseg > 1) {
        e = launch_kernel(P, N, a, true, s);
        if (e != hipSuccess) return e;
        const unsigned per = (P * N / 4 + 255) / 256;
        scan_join_kernel<<<(unsigned)a.B * a.H * per, 256, 0, s>>>(a, P * N / 4);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_kernel(P, N, a, false, s);
}

}  // namespace replay
