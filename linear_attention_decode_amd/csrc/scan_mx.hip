// scan_mx.hip -- the recurrence over packed prompts for bf16 inputs on the
// bf16 matrix instructions; scan.hip has the mathematics.
//
// A workgroup takes one segment of one or two heads of a group (P = 64: two,
// where the group has an even number of them), 128 (or 64) columns of v in
// all, a wavefront 32 of them.  The state stays in the wavefront's
// accumulators as S^T, N x 32, float32, for the whole segment.  Per chunk of
// kQ tokens:
//   G   the weighted scores, 16 x 16 tiles of K Q^T over the wavefronts, one
//       product for both heads, weighted for each and kept in LDS as bf16;
//   y   S Q^T decayed, plus V^T G^T, both into the y^T accumulators;
//   S   decayed, plus K^T (e V).
// What is rounded to bf16: the state and G, as operands of y, itself rounded
// to bf16 (together 1.2 times the error of that last rounding on SiLU-like
// inputs).  The state is not: e V is cut into three bf16 parts that hold its
// 24 bits exactly (8 each, by truncation), so S is what float32 products give.
//
// Layouts.  A 32 x 32 accumulator tile holds in lane (column c, half hh)
// rows 8 (r / 4) + 4 hh + r % 4; an operand of 16 steps holds in the same
// lane steps 8 hh .. 8 hh + 7.  Giving tile row rho the meaning pi(rho), pi
// swapping blocks 4..7 and 8..11 of every 16, makes accumulators 8 x .. 8 x
// + 7 of half hh the steps 16 x + 8 hh + 0..7: S^T tiles are operands as
// they are, and a lane's y^T rows are 8 consecutive p, one 16-byte store.
// LDS holds q, k, v and G in rows as they come; operands that run over
// tokens are read through the transposing read (a group of 16 lanes reads 4
// rows x 16 columns, each lane gets a column).  16-byte pieces of a row are
// permuted by its number so that 16 rows' equal pieces, and 4 rows' 64
// bytes, lie in distinct banks.
#include "scan_common.h"

namespace replay {

namespace {

constexpr int kQ = kScanChunk;

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float acc16 __attribute__((ext_vector_type(16)));
typedef float acc4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ acc16 mma32(bf8 a, bf8 b, acc16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ acc4 mma16(bf8 a, bf8 b, acc4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Byte offset of byte b of a row of RB bytes.
template <int RB>
__device__ __forceinline__ int at(int row, int b) {
    static_assert(RB == 128 || RB == 256, "rows of 128 or 256 bytes");
    const int f = RB == 256 ? ((row & 3) << 2) | ((row >> 2) & 3) : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
    return row * RB + (b ^ (f << 4));
}

__device__ __forceinline__ bf8 row8(const uint8_t *m, int off) {
    return __builtin_bit_cast(bf8, *reinterpret_cast<const u32x4 *>(m + off));
}

// Operand over tokens j0 .. j0 + 15 (lane half hh: j0 + 8 hh ..): lane c of
// 32 gets column c0 + pi(c).
template <int RB>
__device__ __forceinline__ bf8 col8(const uint8_t *m, int j0, int c0) {
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const int l = threadIdx.x & 63, c = l & 15, x = c & 3;
    const int row = j0 + 8 * (l >> 5) + (c >> 2);
    const int col = c0 + (l & 16) + 4 * (x == 1 ? 2 : (x == 2 ? 1 : x));
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(m + at<RB>(row, 2 * col)));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(m + at<RB>(row + 4, 2 * col)));
    return __builtin_bit_cast(bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// pi within 32
__device__ __forceinline__ int pi(int c) {
    const int x = (c >> 2) & 3;
    return (c & ~12) | ((x == 1 ? 2 : (x == 2 ? 1 : x)) << 2);
}

// The value of the lane d before (behind) this one in its row of 16, 1 past the row's end.
template <int CTRL>
__device__ __forceinline__ float row_move(float x) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0x3f800000, (int)__float_as_uint(x), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float row_upto(float x) {
    x *= row_move<0x111>(x);
    x *= row_move<0x112>(x);
    x *= row_move<0x114>(x);
    x *= row_move<0x118>(x);
    return x;
}
__device__ __forceinline__ float row_from(float x) {
    x *= row_move<0x101>(x);
    x *= row_move<0x102>(x);
    x *= row_move<0x104>(x);
    x *= row_move<0x108>(x);
    return x;
}

__device__ __forceinline__ float lane_value(float x, int lane) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), lane));
}

template <int P, int N, int VW>
struct Shape {
    static constexpr int NW = VW / 32, NT = 64 * NW, HB = VW / P;   // wavefronts, threads, heads
    static constexpr int QB = 2 * N, VB = 2 * VW, GB = 2 * kQ;     // bytes of a row
    static constexpr int IQ = kQ * QB / 16 / NT, IV = kQ * VB / 16 / NT;   // 16-byte pieces a thread stages
    static_assert(HB >= 1 && HB <= 2 && NW >= HB, "one or two heads");
};

struct Decays {
    float a[kQ], dt[kQ];
    float pre[kQ];   // product of the a of the token's 16-tile, up to and with it
    float sd[kQ];    // dt times the product behind it in its tile
    float d0[kQ];    // product within the chunk, up to and with it
    float e[kQ];     // dt times the product behind it in the chunk
    float tot[4];    // a 16-tile's whole product
};

template <int P, int N, int VW>
struct Tile {
    using Sh = Shape<P, N, VW>;
    __align__(16) uint8_t q[kQ * Sh::QB], k[kQ * Sh::QB], v[kQ * Sh::VB], g[Sh::HB][kQ * Sh::GB];
    Decays d[Sh::HB];
};

// The next chunk's rows on their way to LDS.
template <int P, int N, int VW, bool STATE_ONLY>
struct Ahead {
    using Sh = Shape<P, N, VW>;
    u32x4 q[STATE_ONLY ? 1 : Sh::IQ], k[Sh::IQ], v[Sh::IV];
    float a, dt;
    __device__ __forceinline__ void load(const ScanArgs &s, int t0, int n, int h, int g) {
        const int tid = threadIdx.x;
        const uint16_t *sq = static_cast<const uint16_t *>(s.q), *sk = static_cast<const uint16_t *>(s.k);
        const uint16_t *sv = static_cast<const uint16_t *>(s.v);
        // rows past the n tokens are zero
#pragma unroll
        for (int i = 0; i < Sh::IQ; ++i) {
            const int e = (i * Sh::NT + tid) * 8, t = e / N;
            k[i] = u32x4{0, 0, 0, 0};
            if constexpr (!STATE_ONLY) q[i] = u32x4{0, 0, 0, 0};
            if (t < n) {
                const size_t o = ((size_t)(t0 + t) * s.G + g) * N + e % N;
                k[i] = *reinterpret_cast<const u32x4 *>(sk + o);
                if constexpr (!STATE_ONLY) q[i] = *reinterpret_cast<const u32x4 *>(sq + o);
            }
        }
#pragma unroll
        for (int i = 0; i < Sh::IV; ++i) {
            const int e = (i * Sh::NT + tid) * 8, t = e / VW;
            v[i] = u32x4{0, 0, 0, 0};
            if (t < n) v[i] = *reinterpret_cast<const u32x4 *>(sv + ((size_t)(t0 + t) * s.H + h) * P + e % VW);
        }
        a = 1.f;
        dt = 0.f;
        const int hb = tid >> 6, t = tid & 63;
        if (hb < Sh::HB && t < n) {
            a = s.a[(size_t)(t0 + t) * s.H + h + hb];
            dt = s.dt[(size_t)(t0 + t) * s.H + h + hb];
        }
    }
    __device__ __forceinline__ void store(Tile<P, N, VW> &m) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < Sh::IQ; ++i) {
            const int b = (i * Sh::NT + tid) * 16, o = at<Sh::QB>(b / Sh::QB, b % Sh::QB);
            *reinterpret_cast<u32x4 *>(m.k + o) = k[i];
            if constexpr (!STATE_ONLY) *reinterpret_cast<u32x4 *>(m.q + o) = q[i];
        }
#pragma unroll
        for (int i = 0; i < Sh::IV; ++i) {
            const int b = (i * Sh::NT + tid) * 16;
            *reinterpret_cast<u32x4 *>(m.v + at<Sh::VB>(b / Sh::VB, b % Sh::VB)) = v[i];
        }
        const int hb = tid >> 6, t = tid & 63;
        if (hb < Sh::HB) {   // whole wavefronts, a token a lane
            const float pre = row_upto(a), suf = row_move<0x101>(row_from(a));
            const float t0 = lane_value(pre, 15), t1 = lane_value(pre, 31), t2 = lane_value(pre, 47), t3 = lane_value(pre, 63);
            const int tile = t >> 4;
            const float ahead = tile == 0 ? 1.f : (tile == 1 ? t0 : (tile == 2 ? t0 * t1 : t0 * t1 * t2));
            const float behind = tile == 3 ? 1.f : (tile == 2 ? t3 : (tile == 1 ? t2 * t3 : t1 * t2 * t3));
            Decays &d = m.d[hb];
            d.a[t] = a;
            d.dt[t] = dt;
            d.pre[t] = pre;
            d.sd[t] = dt * suf;
            d.d0[t] = ahead * pre;
            d.e[t] = dt * suf * behind;
            if (t == 0) {
                d.tot[0] = t0;
                d.tot[1] = t1;
                d.tot[2] = t2;
                d.tot[3] = t3;
            }
        }
    }
};

// x's upper bits and y's as a bf16 pair
__device__ __forceinline__ uint32_t upper_pair(float x, float y) {
    return __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
}

// Steps 16 x + 8 hh .. of S^T's tile as an operand, x = 0, 1
__device__ __forceinline__ bf8 state_operand(const acc16 &S, int x) {
    u32x4 f;
#pragma unroll
    for (int r = 0; r < 4; ++r) f[r] = f32x2_to_bf16_pair(S[8 * x + 2 * r], S[8 * x + 2 * r + 1]);
    return __builtin_bit_cast(bf8, f);
}

template <int P, int N, int VW, bool STATE_ONLY>
__global__ __launch_bounds__((Shape<P, N, VW>::NT), (VW == 128 ? 2 : 1)) void scan_mx_kernel(ScanArgs s) {
    using Sh = Shape<P, N, VW>;
    constexpr int NW = Sh::NW, HB = Sh::HB, TN = N / 32, KN = N / 16;
    __shared__ Tile<P, N, VW> m;

    const int lid = xcd_remap(blockIdx.x, gridDim.x), HP = s.H / HB;
    const int h = (lid % HP) * HB, seg = (lid / HP) % s.nseg, b = lid / HP / s.nseg;
    const int g = h / (s.H / s.G);
    const Span sp = find_span(s, b, seg);
    const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63, c = lane & 31, hh = lane >> 5;
    if (!STATE_ONLY && seg == 0 && h == 0 && !sp.run && tid == 0) raise_seq_error(s.err, b, REPLAY_SEQERR_BAD_RANGE);
    if (!sp.run || (STATE_ONLY && sp.last)) return;

    const int hb = HB == 1 ? 0 : w / (NW / HB);               // this wavefront's head
    const int p0 = 32 * w - hb * P;                           // its first column there
    const size_t bh = (size_t)b * s.H + h + hb, tile = (size_t)P * N;
    const size_t row = (size_t)(p0 + pi(c)) * N + 8 * hh;     // this lane's columns of S [P][N], 8 of every 16
    acc16 S[TN];
    const float *from = STATE_ONLY ? nullptr
                        : seg > 0 ? s.ws + (bh * (s.nseg - 1) + seg - 1) * tile
                                  : (s.s_in ? s.s_in + bh * tile : nullptr);
#pragma unroll
    for (int t = 0; t < TN; ++t) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            f32x4 f = {0.f, 0.f, 0.f, 0.f};
            if (from) f = *reinterpret_cast<const f32x4 *>(from + row + 32 * t + 16 * (x >> 1) + 4 * (x & 1));
#pragma unroll
            for (int r = 0; r < 4; ++r) S[t][4 * x + r] = f[r];
        }
    }
    if constexpr (!STATE_ONLY) {   // the tiles of G above the diagonal's are never written again
        for (int i = tid; i < HB * kQ * Sh::GB / 16; i += Sh::NT)
            *reinterpret_cast<u32x4 *>(&m.g[0][0] + 16 * i) = u32x4{0, 0, 0, 0};
    }

    Ahead<P, N, VW, STATE_ONLY> ahead;
    float decay = 1.f;
    ahead.load(s, sp.t0, sp.n, h, g);
    for (int done = 0; done < sp.n; done += kQ) {
        const int n = sp.n - done < kQ ? sp.n - done : kQ;
        __syncthreads();   // the last chunk is read to its end
        ahead.store(m);
        if (done + kQ < sp.n) ahead.load(s, sp.t0 + done + kQ, sp.n - done - kQ, h, g);
        __syncthreads();

        bf8 V[kQ / 16];
        if constexpr (!STATE_ONLY) {
            // 16 x 16 tiles (ti, tj) of K Q^T: lane (column i = l % 16, rows j = 4 (l / 16) + r)
            const int ci = lane & 15, lg = lane >> 4;
            for (int x = w; x < 10; x += NW) {
                const int ti = x < 1 ? 0 : (x < 3 ? 1 : (x < 6 ? 2 : 3)), tj = x - ti * (ti + 1) / 2;
                acc4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int st = 0; st < N / 32; ++st) {
                    const int byte = 64 * st + 16 * lg;
                    d = mma16(row8(m.k, at<Sh::QB>(16 * tj + ci, byte)), row8(m.q, at<Sh::QB>(16 * ti + ci, byte)), d);
                }
                const int i = 16 * ti + ci, j0 = 16 * tj + 4 * lg;
#pragma unroll
                for (int y = 0; y < HB; ++y) {
                    const Decays &dc = m.d[y];
                    f32x4 o;
                    if (ti != tj) {
                        float R = dc.pre[i];   // a over the tiles between and this one's, up to i
                        if (ti - tj > 1) R *= dc.tot[tj + 1];
                        if (ti - tj > 2) R *= dc.tot[tj + 2];
                        const f32x4 sd = *reinterpret_cast<const f32x4 *>(&dc.sd[j0]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[r] = d[r] * (R * sd[r]);
                    } else {
                        // blocks of 4: a over those between j's and i, times what is behind j in its block
                        const f32x4 aa = *reinterpret_cast<const f32x4 *>(&dc.a[j0]);
                        const f32x4 dt = *reinterpret_cast<const f32x4 *>(&dc.dt[j0]);
                        const float own = dc.a[i];
                        const float R = row_upto(ci >= 4 * (lg + 1) ? own : 1.f);
                        f32x4 D = {R, R, R, R};
                        float z = 1.f;
#pragma unroll
                        for (int r = 2; r >= 0; --r) {
                            z = j0 + r + 1 <= i ? z * aa[r + 1] : 1.f;
                            D[r] *= z;
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r) o[r] = j0 + r <= i ? d[r] * (D[r] * dt[r]) : 0.f;
                    }
                    *reinterpret_cast<u32x2 *>(m.g[y] + at<Sh::GB>(i, 2 * j0)) =
                        u32x2{f32x2_to_bf16_pair(o[0], o[1]), f32x2_to_bf16_pair(o[2], o[3])};
                }
            }
            // y^T = S Q^T, lane (token c of the 32, rows p)
            acc16 y[2];
#pragma unroll
            for (int I = 0; I < 2; ++I)
#pragma unroll
                for (int r = 0; r < 16; ++r) y[I][r] = 0.f;
#pragma unroll
            for (int st = 0; st < KN; ++st) {
                const bf8 sf = state_operand(S[st / 2], st & 1);
#pragma unroll
                for (int I = 0; I < 2; ++I) y[I] = mma32(sf, row8(m.q, at<Sh::QB>(32 * I + c, 32 * st + 16 * hh)), y[I]);
            }
#pragma unroll
            for (int I = 0; I < 2; ++I) y[I] *= m.d[hb].d0[32 * I + c];
            __syncthreads();
#pragma unroll
            for (int st = 0; st < kQ / 16; ++st) V[st] = col8<Sh::VB>(m.v, 16 * st, 32 * w);
            // A weight of 0 does not hide a later token's NaN or infinity in
            // v: where there is one (0 x = NaN), the product goes without
            // them, and they are added for the tokens from theirs on.
            float zero = 0.f;
#pragma unroll
            for (int st = 0; st < kQ / 16; ++st)
#pragma unroll
                for (int r = 0; r < 4; ++r) zero = dot2_bf16(__builtin_bit_cast(u32x4, V[st])[r], 0u, zero);
            const bool odd = __any(zero != zero);
            if (odd) {
#pragma unroll
                for (int st = 0; st < kQ / 16; ++st) {
                    u32x4 x = __builtin_bit_cast(u32x4, V[st]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if ((x[r] & 0x7f80u) == 0x7f80u) x[r] &= 0xffff0000u;
                        if ((x[r] & 0x7f800000u) == 0x7f800000u) x[r] &= 0xffffu;
                    }
                    V[st] = __builtin_bit_cast(bf8, x);
                }
            }
#pragma unroll
            for (int I = 0; I < 2; ++I) {
                const int i = 32 * I + c;
#pragma unroll
                for (int st = 0; st < 2 * (I + 1); ++st) y[I] = mma32(V[st], row8(m.g[hb], at<Sh::GB>(i, 32 * st + 16 * hh)), y[I]);
                if (odd)
                    for (int j = 0; j <= 32 * I + 31; ++j) {
                        const float gg = load_io1<true>(m.g[hb] + at<Sh::GB>(i, 2 * j), 0);
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const float x = load_io1<true>(m.v + at<Sh::VB>(j, 2 * (32 * w + pi(8 * (r / 4) + 4 * hh + r % 4))), 0);
                            if (j <= i && !finite(x)) y[I][r] = fmaf(gg, x, y[I][r]);
                        }
                    }
                if (i < n) {
                    uint16_t *o = static_cast<uint16_t *>(s.y) + ((size_t)(sp.t0 + done + i) * s.H + h) * P + 32 * w + 8 * hh;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        u32x4 f;
#pragma unroll
                        for (int r = 0; r < 4; ++r) f[r] = f32x2_to_bf16_pair(y[I][8 * x + 2 * r], y[I][8 * x + 2 * r + 1]);
                        *reinterpret_cast<u32x4 *>(o + 16 * x) = f;
                    }
                }
            }
            if (odd)
#pragma unroll
                for (int st = 0; st < kQ / 16; ++st) V[st] = col8<Sh::VB>(m.v, 16 * st, 32 * w);
        } else {
#pragma unroll
            for (int st = 0; st < kQ / 16; ++st) V[st] = col8<Sh::VB>(m.v, 16 * st, 32 * w);
        }
        // S^T <- (whole decay) S^T + K^T (e V), e V in three parts of 8 bits
        const float all = m.d[hb].d0[kQ - 1];
        decay *= all;
#pragma unroll
        for (int t = 0; t < TN; ++t) S[t] *= all;
#pragma unroll
        for (int st = 0; st < kQ / 16; ++st) {
            const u32x4 vv = __builtin_bit_cast(u32x4, V[st]);
            const f32x4 e0 = *reinterpret_cast<const f32x4 *>(&m.d[hb].e[16 * st + 8 * hh]);
            const f32x4 e1 = *reinterpret_cast<const f32x4 *>(&m.d[hb].e[16 * st + 8 * hh + 4]);
            u32x4 part[3];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float x[2];
                x[0] = bf16_bits_to_f32(vv[r] & 0xffffu) * (r < 2 ? e0[2 * r] : e1[2 * r - 4]);
                x[1] = __uint_as_float(vv[r] & 0xffff0000u) * (r < 2 ? e0[2 * r + 1] : e1[2 * r - 3]);
#pragma unroll
                for (int z = 0; z < 3; ++z) {
                    part[z][r] = upper_pair(x[0], x[1]);
#pragma unroll
                    for (int u = 0; u < 2; ++u) x[u] -= __uint_as_float(__float_as_uint(x[u]) & 0xffff0000u);
                }
            }
            bf8 K[TN];
#pragma unroll
            for (int t = 0; t < TN; ++t) K[t] = col8<Sh::QB>(m.k, 16 * st, 32 * t);
#pragma unroll
            for (int z = 2; z >= 0; --z)
#pragma unroll
                for (int t = 0; t < TN; ++t) S[t] = mma32(K[t], __builtin_bit_cast(bf8, part[z]), S[t]);
        }
    }

    float *to = nullptr;
    if constexpr (STATE_ONLY) {
        to = s.ws + (bh * (s.nseg - 1) + seg) * tile;
        if (p0 == 0 && lane == 0) s.ws_decay[bh * (s.nseg - 1) + seg] = decay;
    } else if (sp.last) {
        to = s.s_out + bh * tile;
    }
    if (to) {
#pragma unroll
        for (int t = 0; t < TN; ++t)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<f32x4 *>(to + row + 32 * t + 16 * (x >> 1) + 4 * (x & 1)) =
                    f32x4{S[t][4 * x], S[t][4 * x + 1], S[t][4 * x + 2], S[t][4 * x + 3]};
    }
}

template <int P, int N, int VW>
hipError_t launch_one(const ScanArgs &a, bool state_only, hipStream_t s) {
    using Sh = Shape<P, N, VW>;
    const unsigned blocks = (unsigned)((size_t)a.B * (a.H / Sh::HB) * a.nseg);
    if (state_only)
        scan_mx_kernel<P, N, VW, true><<<blocks, Sh::NT, 0, s>>>(a);
    else
        scan_mx_kernel<P, N, VW, false><<<blocks, Sh::NT, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

bool scan_mx_supported(int P, int N, const ScanArgs &a) {
    return a.io_bf16 && ((P == 64 && (N == 64 || N == 128)) || (P == 128 && N == 128));
}

// Two heads where they share their group's q and k.
int scan_mx_heads(int P, int H, int G) { return P == 64 && (H / G) % 2 == 0 ? 2 : 1; }

hipError_t launch_scan_mx(int P, int N, const ScanArgs &a, bool state_only, hipStream_t s) {
    const bool two = scan_mx_heads(P, a.H, a.G) == 2;
    if (P == 64 && N == 64) return two ? launch_one<64, 64, 128>(a, state_only, s) : launch_one<64, 64, 64>(a, state_only, s);
    if (P == 64 && N == 128) return two ? launch_one<64, 128, 128>(a, state_only, s) : launch_one<64, 128, 64>(a, state_only, s);
    if (P == 128 && N == 128) return launch_one<128, 128, 128>(a, state_only, s);
    return hipErrorInvalidValue;
}

}  // namespace replay
