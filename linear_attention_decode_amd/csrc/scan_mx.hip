// scan_mx.hip -- the recurrence over packed prompts for bf16 inputs on the
// bf16 matrix instructions; scan.hip has the mathematics.
//
// A workgroup takes one segment of one or two heads of a group (P = 64: two,
// where the group has an even number of them), 128 (or 64) columns of v in
// all, a wavefront 32 of them.  The state stays in the wavefront's
// accumulators as S^T, N x 32, float32, for the whole segment.  Per chunk of
// kQ tokens:
//   G   the weighted scores, 16 x 16 tiles of K Q^T over the wavefronts, one
//       product for both heads, weighted for each and kept in LDS;
//   y   S Q^T decayed, plus V^T G^T, both into the y^T accumulators;
//   S   decayed, plus K^T (e V).
// What bf16 operands leave out: the state and G enter y's products as two
// bf16 parts, the upper 8 bits by truncation and the rest rounded, so that a
// term lacks at most 2^-15 of itself and y is a float32 sum rounded once; the
// second parts cost 28 us of the 278 below, and without them y had 1.3 times
// the error of its own rounding.  e V is cut into three parts that hold its
// 24 bits exactly (8 each), so the state is what float32 products give.
//
// What bounds it.  One sequence of 8192 tokens (128 heads, 8 groups, 64 x
// 128): 209 us, of which 65 for the segments' states and 11 to join them, 315
// MB in all, 1.5 TB/s.  Sixteen ragged sequences of 15013 tokens from states
// (703 MB): 278 us, 2.5 TB/s.  A wavefront's chunk is 104 matrix instructions
// and 893 others, most of them cuts, roundings and decays, and two workgroups
// a CU overlap these with the loads in part.  The second and third part of e V
// cost 48 us, and would lose the state's float32; the float32 kernel takes
// 1677 us.
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

__device__ __forceinline__ bf8 row8(const uint8_t *m, uint32_t off) {
    return __builtin_bit_cast(bf8, *reinterpret_cast<const u32x4 *>(m + off));
}

// Offsets into a swizzled array: a lane's own part, with the parts that
// step through rows (multiples of 16 rows: added) and through a row's bytes
// (whole 32s or 64s: exclusive-or'd, they meet no bit of the lane's but the
// swizzle's) applied at the read.  A base made opaque once a chunk keeps
// the compiler from holding each step's offset in a register of its own.
__device__ __forceinline__ uint32_t opaque(uint32_t x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Operand over tokens j0 .. j0 + 15 (lane half hh: j0 + 8 hh ..), from
// col_base's offset for tokens from 0 and columns from a multiple of 32: lane
// c of 32 gets column pi(c) of them.
template <int RB>
__device__ __forceinline__ uint32_t col_base() {
    const int l = threadIdx.x & 63, c = l & 15, x = c & 3;
    return at<RB>(8 * (l >> 5) + (c >> 2), 2 * ((l & 16) + 4 * (x == 1 ? 2 : (x == 2 ? 1 : x))));
}
template <int RB>
__device__ __forceinline__ bf8 col8(const uint8_t *m, uint32_t off, int j0) {
    typedef __attribute__((address_space(3))) s16x4 lds4;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(m + off + j0 * RB));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(m + (off ^ 16) + (j0 + 4) * RB));
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

// STATE_ONLY needs neither q nor G.
template <int P, int N, int VW, bool STATE_ONLY>
struct Tile {
    using Sh = Shape<P, N, VW>;
    __align__(16) uint8_t k[kQ * Sh::QB], v[kQ * Sh::VB], q[STATE_ONLY ? 16 : kQ * Sh::QB];
    // G's upper parts in rows 0..63, a token each; the lower parts of tokens
    // 0..31, which weigh no more than 32, behind their upper ones, those of
    // tokens 32..63 in rows 64..95
    uint8_t g[Sh::HB][STATE_ONLY ? 16 : (kQ + 32) * Sh::GB];
    Decays d[Sh::HB];
};

// The next chunk's rows on their way to LDS.  Loads go through buffer
// resources over the chunk's own rows: those past its n tokens read zero.
template <int P, int N, int VW, bool STATE_ONLY>
struct Ahead {
    using Sh = Shape<P, N, VW>;
    u32x4 q[STATE_ONLY ? 1 : Sh::IQ], k[Sh::IQ], v[Sh::IV];
    float a, dt;
    uint32_t oqk, ov, oa;   // this thread's byte offsets in a chunk's rows
    uint32_t sqk, sv;       // bytes from one piece's row to the next piece's
    __device__ __forceinline__ void init(const ScanArgs &s) {
        const uint32_t tid = threadIdx.x, rqk = (uint32_t)s.G * Sh::QB, rv = (uint32_t)s.H * P * 2;
        oqk = tid / (Sh::QB / 16) * rqk + tid % (Sh::QB / 16) * 16;
        ov = tid / (Sh::VB / 16) * rv + tid % (Sh::VB / 16) * 16;
        oa = (tid & 63) * (uint32_t)s.H * 4 + (tid >> 6) % Sh::HB * 4;
        sqk = Sh::NT / (Sh::QB / 16) * rqk;
        sv = Sh::NT / (Sh::VB / 16) * rv;
    }
    // n <= 0: nothing is read
    __device__ __forceinline__ void load(const ScanArgs &s, int t0, int n, int h, int g) {
        const uint32_t rqk = (uint32_t)s.G * Sh::QB, rv = (uint32_t)s.H * P * 2, ra = (uint32_t)s.H * 4;
        const uint32_t more = n < kQ ? n - 1 : kQ - 1;   // rows behind the first
        const size_t bqk = (size_t)t0 * rqk + (size_t)g * Sh::QB, bv = (size_t)t0 * rv + (size_t)h * P * 2;
        const size_t ba = (size_t)t0 * ra + (size_t)h * 4;
        const auto rk = make_rsrc(static_cast<const char *>(s.k) + bqk, n > 0 ? more * rqk + Sh::QB : 0);
        const auto rq = make_rsrc(static_cast<const char *>(s.q) + bqk, n > 0 ? more * rqk + Sh::QB : 0);
        const auto rv_ = make_rsrc(static_cast<const char *>(s.v) + bv, n > 0 ? more * rv + Sh::VB : 0);
        const auto rda = make_rsrc(reinterpret_cast<const char *>(s.a) + ba, n > 0 ? more * ra + Sh::HB * 4 : 0);
        const auto rdt = make_rsrc(reinterpret_cast<const char *>(s.dt) + ba, n > 0 ? more * ra + Sh::HB * 4 : 0);
#pragma unroll
        for (int i = 0; i < Sh::IQ; ++i) {
            k[i] = __builtin_amdgcn_raw_buffer_load_b128(rk, oqk, i * sqk, 0);
            if constexpr (!STATE_ONLY) q[i] = __builtin_amdgcn_raw_buffer_load_b128(rq, oqk, i * sqk, 0);
        }
#pragma unroll
        for (int i = 0; i < Sh::IV; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b128(rv_, ov, i * sv, 0);
        a = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rda, oa, 0, 0));
        dt = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rdt, oa, 0, 0));
    }
    __device__ __forceinline__ void store(Tile<P, N, VW, STATE_ONLY> &m, int n) {
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
            a = t < n ? a : 1.f;
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
// what these leave of x
__device__ __forceinline__ float below_upper(float x) { return x - __uint_as_float(__float_as_uint(x) & 0xffff0000u); }
// ... of both, as a bf16 pair
__device__ __forceinline__ uint32_t lower_pair(float x, float y) { return f32x2_to_bf16_pair(below_upper(x), below_upper(y)); }

// G = the weighted scores, in 16 x 16 tiles (ti, tj) of K Q^T, lane (column i
// = l % 16, rows j = 4 (l / 16) + r).  A fourth of the work is the diagonal
// tile x, two below it and, for x = 0 and 2, the one beside it, zero (y's
// products run over 32 tokens); wavefront w takes x = w (of two: w, w + 2).
template <int P, int N, int VW>
__device__ __forceinline__ void weigh(Tile<P, N, VW, false> &m, int w, int lane) {
    using Sh = Shape<P, N, VW>;
    const int ci = lane & 15, lg = lane >> 4;
    const uint32_t in = opaque(at<Sh::QB>(ci, 16 * lg)), out = opaque(at<Sh::GB>(ci, 8 * lg)), lg4 = opaque(4 * lg);
#pragma unroll
    for (int step = 0; step < 4 / Sh::NW; ++step) {
        const int x = w + step * Sh::NW;
        const int ti[3] = {x, x == 0 ? 1 : (x == 1 ? 2 : 3), x == 0 ? 0 : (x == 1 ? 2 : (x == 2 ? 2 : 3))};
        const int tj[3] = {x, x == 3 ? 1 : 0, x == 0 ? 1 : (x == 1 ? 1 : (x == 2 ? 3 : 2))};
        acc4 d[3];
#pragma unroll
        for (int z = 0; z < 3; ++z) {
            const uint32_t ko = in + 16 * Sh::QB * tj[z], qo = in + 16 * Sh::QB * ti[z];
            bf8 k[N / 32], q[N / 32];
#pragma unroll
            for (int st = 0; st < N / 32; ++st) {
                k[st] = row8(m.k, ko ^ (64 * st));
                q[st] = row8(m.q, qo ^ (64 * st));
            }
            d[z] = acc4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < N / 32; ++st) d[z] = mma16(k[st], q[st], d[z]);
        }
#pragma unroll
        for (int y = 0; y < Sh::HB; ++y) {
            const Decays &dc = m.d[y];
#pragma unroll
            for (int z = 0; z < 3; ++z) {
                const int i = 16 * ti[z] + ci, j0 = 16 * tj[z] + lg4;
                f32x4 o;
                if (z == 0) {
                    // blocks of 4: a over those between j's and i, times what is behind j in its block
                    const f32x4 aa = *reinterpret_cast<const f32x4 *>(&dc.a[j0]);
                    const f32x4 dt = *reinterpret_cast<const f32x4 *>(&dc.dt[j0]);
                    const float own = dc.a[i];
                    const float R = row_upto(ci >= 4 * (lg + 1) ? own : 1.f);
                    f32x4 D = {R, R, R, R};
                    float f = 1.f;
#pragma unroll
                    for (int r = 2; r >= 0; --r) {
                        f = j0 + r + 1 <= i ? f * aa[r + 1] : 1.f;
                        D[r] *= f;
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[r] = j0 + r <= i ? d[z][r] * (D[r] * dt[r]) : 0.f;
                } else {
                    // a over i's own tile up to i and the tiles between, the nearest first (every product is one
                    // of consecutive tokens), times what is behind j in its tile
                    const float t1 = dc.tot[(tj[z] + 1) & 3], t2 = dc.tot[(tj[z] + 2) & 3];
                    const float R = dc.pre[i] * (ti[z] - tj[z] > 2 ? t2 : 1.f) * (ti[z] - tj[z] > 1 ? t1 : 1.f);
                    const f32x4 sd = *reinterpret_cast<const f32x4 *>(&dc.sd[j0]);
                    const bool below = z == 1 || (x & 1);
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[r] = below ? d[z][r] * (R * sd[r]) : 0.f;
                }
                const uint32_t upper = (out + 16 * Sh::GB * ti[z]) ^ (32 * tj[z]);
                const uint32_t lower = ti[z] < 2 ? upper ^ 64 : upper + 32 * Sh::GB;
                *reinterpret_cast<u32x2 *>(m.g[y] + upper) = u32x2{upper_pair(o[0], o[1]), upper_pair(o[2], o[3])};
                *reinterpret_cast<u32x2 *>(m.g[y] + lower) = u32x2{lower_pair(o[0], o[1]), lower_pair(o[2], o[3])};
            }
        }
    }
}

// Steps 16 x + 8 hh .. of S^T's tile as an operand, x = 0, 1, in two parts
__device__ __forceinline__ void state_operand(const acc16 &S, int x, bf8 *upper, bf8 *lower) {
    u32x4 u, l;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        u[r] = upper_pair(S[8 * x + 2 * r], S[8 * x + 2 * r + 1]);
        l[r] = lower_pair(S[8 * x + 2 * r], S[8 * x + 2 * r + 1]);
    }
    *upper = __builtin_bit_cast(bf8, u);
    *lower = __builtin_bit_cast(bf8, l);
}

template <int P, int N, int VW, bool STATE_ONLY>
__global__ __launch_bounds__((Shape<P, N, VW>::NT), (VW == 128 ? 2 : 1)) void scan_mx_kernel(ScanArgs s) {
    using Sh = Shape<P, N, VW>;
    constexpr int NW = Sh::NW, HB = Sh::HB, TN = N / 32, KN = N / 16;
    __shared__ Tile<P, N, VW, STATE_ONLY> m;

    Place place;
    if (!find_place(s, HB, &place)) return;
    const int h = place.h, seg = place.seg, b = place.b, g = place.g;
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
    Ahead<P, N, VW, STATE_ONLY> ahead;
    float decay = 1.f;
    ahead.init(s);
    ahead.load(s, sp.t0, sp.n, h, g);
    const uint32_t ry = (uint32_t)s.H * P * 2;
    const uint32_t yo = (c & 15) * ry + 64 * w + 16 * hh + 2 * (c & 16);   // this lane's place in a chunk's y
    if constexpr (!STATE_ONLY) {
        // Stores over no bytes: every turn of the loop then finds its loads
        // behind as many stores, and waits for the loads alone.
        const auto none = make_rsrc(s.y, 0);
#pragma unroll
        for (int x = 0; x < 4; ++x) __builtin_amdgcn_raw_buffer_store_b128(u32x4{0, 0, 0, 0}, none, yo, 16 * x * ry, 0);
    }
    for (int done = 0; done < sp.n; done += kQ) {
        const int n = sp.n - done < kQ ? sp.n - done : kQ;
        __syncthreads();   // the last chunk is read to its end
        ahead.store(m, n);
        __syncthreads();

        bf8 V[kQ / 16];
        ahead.load(s, sp.t0 + done + kQ, sp.n - done - kQ, h, g);
        const uint32_t vo = opaque(col_base<Sh::VB>() ^ (64 * w));
        if constexpr (!STATE_ONLY) {
            weigh<P, N, VW>(m, w, lane);
            // y^T = S Q^T, lane (token c of the 32, rows p)
            acc16 y[2];
#pragma unroll
            for (int I = 0; I < 2; ++I)
#pragma unroll
                for (int r = 0; r < 16; ++r) y[I][r] = 0.f;
            const uint32_t qo = opaque(at<Sh::QB>(c, 16 * hh));
            constexpr int U = 4;   // steps whose operands are loaded together
#pragma unroll
            for (int st0 = 0; st0 < KN; st0 += U) {
                bf8 q[2][U];
#pragma unroll
                for (int x = 0; x < U; ++x)
#pragma unroll
                    for (int I = 0; I < 2; ++I) q[I][x] = row8(m.q, (qo ^ (32 * (st0 + x))) + 32 * Sh::QB * I);
#pragma unroll
                for (int x = 0; x < U; ++x) {
                    bf8 upper, lower;
                    state_operand(S[(st0 + x) / 2], x & 1, &upper, &lower);
#pragma unroll
                    for (int I = 0; I < 2; ++I) y[I] = mma32(lower, q[I][x], y[I]);
#pragma unroll
                    for (int I = 0; I < 2; ++I) y[I] = mma32(upper, q[I][x], y[I]);
                }
            }
#pragma unroll
            for (int I = 0; I < 2; ++I) y[I] *= m.d[hb].d0[32 * I + c];
#pragma unroll
            for (int st = 0; st < kQ / 16; ++st) V[st] = col8<Sh::VB>(m.v, vo, 16 * st);
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
            __syncthreads();
            const uint32_t go = opaque(at<Sh::GB>(c, 16 * hh));
            // the first 32 tokens take 2 steps of either part, the others 4
#pragma unroll
            for (int rows = 0; rows < 3; ++rows) {
                bf8 G[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) G[x] = row8(m.g[hb], (go ^ (32 * x)) + 32 * Sh::GB * rows);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (rows == 0)
                        y[0] = mma32(V[x & 1], G[x], y[0]);
                    else
                        y[1] = mma32(V[x], G[x], y[1]);
                }
            }
            // y: after the exchange of odd and even rows of 16 lanes a store
            // writes 64 bytes of each of 16 tokens.  Through a buffer resource
            // over the chunk's tokens, so that it is not conditional: a wait
            // for the next chunk's loads then need not wait for these stores.
            {
                const auto ys = make_rsrc(static_cast<char *>(s.y) + (size_t)(sp.t0 + done) * ry + (size_t)h * P * 2,
                                          (uint32_t)(n - 1) * ry + Sh::VB);
#pragma unroll
                for (int I = 0; I < 2; ++I) {
                    u32x4 f[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int r = 0; r < 4; ++r) f[x][r] = f32x2_to_bf16_pair(y[I][8 * x + 2 * r], y[I][8 * x + 2 * r + 1]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const auto z = __builtin_amdgcn_permlane16_swap(f[0][r], f[1][r], false, false);
                        f[0][r] = z[0];
                        f[1][r] = z[1];
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x) __builtin_amdgcn_raw_buffer_store_b128(f[x], ys, yo, (32 * I + 16 * x) * ry, 0);
                }
            }
            if (odd) {
                // in the stored outputs, by the lanes that stored them, when the stores are done
                __builtin_amdgcn_s_waitcnt(0);
                const uint32_t token = opaque(c & 15), first = opaque(8 * hh + (c & 16));
#pragma unroll 1
                for (uint32_t x = 0; x < 32; ++x) {
                    const int i = 16 * (x >> 3) + token, p = first + (x & 7);
                    uint16_t *o = static_cast<uint16_t *>(s.y) + ((size_t)(sp.t0 + done + i) * s.H + h) * P + 32 * w + p;
#pragma unroll 1
                    for (int j = 0; j <= i && i < n; ++j) {
                        const float v = load_io1<true>(m.v + at<Sh::VB>(j, 2 * (32 * w + p)), 0);
                        const float gg = load_io1<true>(m.g[hb] + at<Sh::GB>(i, 2 * j), 0);
                        if (!finite(v)) *o = (uint16_t)f32_to_bf16_bits(fmaf(gg, v, bf16_bits_to_f32(*o)));
                    }
                }
#pragma unroll
                for (int st = 0; st < kQ / 16; ++st) V[st] = col8<Sh::VB>(m.v, vo, 16 * st);
            }
        }
        if constexpr (STATE_ONLY) {
#pragma unroll
            for (int st = 0; st < kQ / 16; ++st) V[st] = col8<Sh::VB>(m.v, vo, 16 * st);
        }
        // S^T <- (whole decay) S^T + K^T (e V), e V in three parts of 8 bits
        const float all = m.d[hb].d0[kQ - 1];
        decay *= all;
#pragma unroll
        for (int t = 0; t < TN; ++t) S[t] *= all;
        const uint32_t ko = opaque(col_base<Sh::QB>());
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
                    for (int u = 0; u < 2; ++u) x[u] = below_upper(x[u]);
                }
            }
            bf8 K[TN];
#pragma unroll
            for (int t = 0; t < TN; ++t) K[t] = col8<Sh::QB>(m.k, ko ^ (64 * t), 16 * st);
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
    const unsigned blocks = scan_blocks(a, Sh::HB);
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
