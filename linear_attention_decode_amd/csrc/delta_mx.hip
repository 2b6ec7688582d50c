// delta_mx.hip -- the gated delta rule over packed prompts for bf16 inputs on
// the bf16 matrix instructions; delta_scan.hip has the mathematics.
//
// What a chunk of 64 tokens needs of k, q, alpha and beta alone does not wait
// for a state, so it comes first and for all chunks at once: delta_prep_kernel
// makes T = (I + A)^-1 diag(beta) and G, and writes them to the workspace as
// operands, in the order in which lanes take them.  delta_mx_kernel then goes
// from chunk to chunk:
//   R = V - diag(g) K S^T,  U = T R,  Y = diag(g) Q S^T + G U,  S <- g_last S + (e U)^T K.
// A chain of chunks has little to spread over the card, so two wavefronts share 16
// columns: each has half of a chunk's tokens, and half of S^T's rows, which stay in
// its accumulators; where heads are fewer still, delta_few.hip has more of them.
// What bounds it: the chain of a chunk's steps, four barriers apart.  Sixteen
// ragged sequences of 15013 tokens (32 heads of 128 x 128): 89 us for T and G, 366 for
// the chunks, eight wavefronts a CU that wait for LDS, for the matrix instructions
// and for each other in turn; one of 8192 tokens 47, and 275 in delta_few.hip.
//
// What bf16 operands leave out: k and q are bf16 as they are; S, R, T, U, e U and G
// go into the products as three parts of 8 bits, which hold their 24 (of T R and G U
// the six products that weigh 2^-16 or more: what is left out is 2^-20 of a term at
// most), so U, the state and y are what float32 products give, and y is rounded once.
// With two parts in y's products one value in 160 rounds otherwise, and one long prompt
// takes 291 us instead of 302, the ragged batch below 382 instead of 427.
//
// Layouts (16 x 16 x 32 products).  An accumulator tile holds in lane (column
// c, group lg) rows 4 lg .. 4 lg + 3; an operand of 32 steps in lane (row or
// column c, group lg) eight of them, which eight is free as long as both
// operands agree: steps 4 lg .. + 3 and 16 + 4 lg .. + 3 are what two tiles of 16
// rows hold there.  So S^T, R and U are operands as they are, and what meets them
// (k, q, T, G) is read in that order, as two 8-byte pieces.  k^T comes
// through the transposing LDS read.  y is made transposed, a lane 4 neighbouring
// columns of one token.
//
// A chunk that holds a value that is no number (k, alpha, beta: noted by the
// first kernel; v: seen by the wavefront) is run token by token, by the rule
// itself.
#include "delta_mx.h"

namespace replay {

namespace {

// ---- T and G of every chunk and head ----------------------------------------

constexpr int kPrepNT = 256;

struct Decays {
    float alpha[kQ], beta[kQ];
    float pre[kQ], suf[kQ];   // products of alpha within a tile of 16: up to and with i; behind j
    float tot[4];             // a tile's whole product
};
// A, whose place T takes block by block
struct PrepTile {
    float a[kQ][kQ + 4];
    Decays d;
};

// The lower left corner of the inverse of rows and columns r0 .. r0 + 2 SIZE -
// 1, a wavefront for 16 columns j of it: T10 = -T11 (A10 T00).
template <int SIZE>
__device__ __forceinline__ void invert_corner(float (*m)[kQ + 4], int r0, int j, int lane) {
    constexpr int TL = SIZE / 16;
    const int c = lane & 15, lg = lane >> 4, c0 = r0 + 16 * j + c;
    acc4 x[TL];
#pragma unroll
    for (int i = 0; i < TL; ++i) x[i] = acc4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < TL; ++k) {
        if (k < j) continue;   // T00 is zero there
        float t[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) t[r] = m[r0 + 16 * k + 4 * lg + r][c0];
#pragma unroll
        for (int i = 0; i < TL; ++i) {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(&m[r0 + SIZE + 16 * i + c][r0 + 16 * k + 4 * lg]);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[i] = mma4(a[r], t[r], x[i]);
        }
    }
    acc4 o[TL];
#pragma unroll
    for (int i = 0; i < TL; ++i) {
        o[i] = acc4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k <= i; ++k) {
            const f32x4 t = *reinterpret_cast<const f32x4 *>(&m[r0 + SIZE + 16 * i + c][r0 + SIZE + 16 * k + 4 * lg]);
#pragma unroll
            for (int r = 0; r < 4; ++r) o[i] = mma4(t[r], x[k][r], o[i]);
        }
    }
    if constexpr (TL > 1) lds_barrier();   // A10 is read by both wavefronts
#pragma unroll
    for (int i = 0; i < TL; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) m[r0 + SIZE + 16 * i + 4 * lg + r][c0] = -o[i][r];
}

// D over tile (ti, tj) of one head, lane (column i = 16 ti + c, rows j = 16 tj
// + 4 lg + r): alpha_{j+1} ... alpha_i; nothing above the diagonal.
__device__ __forceinline__ f32x4 decays_of(const Decays &d, int ti, int tj, int c, int lg) {
    const int i = 16 * ti + c, j0 = 16 * tj + 4 * lg;
    if (ti == tj) return diagonal_decays(&d.alpha[16 * ti], c, lg);
    // the nearest first: every product is one of consecutive tokens
    float p = d.pre[i];
    p *= ti - tj > 1 ? d.tot[(ti - 1) & 3] : 1.f;
    p *= ti - tj > 2 ? d.tot[(ti - 2) & 3] : 1.f;
    return p * *reinterpret_cast<const f32x4 *>(&d.suf[j0]);
}

// A workgroup makes a chunk of HP heads of a group, which share k . k and k . q.  Bound
// by its own chain (products, decays, the inverse by blocks of 16, their products)
// and by what it writes: 8192 tokens of 32 heads 47 us, 3.3 TB/s of the 154 MB.
template <int N, int HP>
__global__ __launch_bounds__(kPrepNT) void delta_prep_kernel(ScanArgs s) {
    __shared__ __align__(16) PrepTile m[HP];
    __shared__ uint32_t odd[HP];
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h0 = blockIdx.x % (s.H / HP) * HP, slot = blockIdx.x / (s.H / HP), b = slot / s.window, g = h0 / (s.H / s.G);
    const Span sp = find_span(s, b, 0);
    const int first = (s.chunk0 + slot % s.window) * kQ;
    if (!sp.run || first >= sp.n) return;
    const int n = sp.n - first < kQ ? sp.n - first : kQ, t0 = sp.t0 + first;
    uint8_t *out = reinterpret_cast<uint8_t *>(s.ws) + ((size_t)slot * s.H + h0) * kSlot;

    // tiles (ti, tj) of K K^T and K Q^T, lane (column i = c, rows j = 4 lg + r): a
    // wavefront has one ti and the pairs of tj that make G's operands of it, so that
    // it writes them whole (written half by half they take a fourth longer).  Two of the tiles lie above the
    // diagonal, zeros of T and G.  Rows past the chunk's tokens read zero.
    const int ti = w < 2 ? w + 2 : w - 2, pairs = w < 2 ? 2 : 1;
    acc4 kk[4], qk[4];
    const uint32_t rqk = (uint32_t)s.G * N * 2;
    {
        const size_t base = (size_t)t0 * rqk + (size_t)g * N * 2;
        const uint32_t bytes = (uint32_t)(n - 1) * rqk + N * 2;
        const auto rk = make_rsrc(static_cast<const char *>(s.k) + base, bytes);
        const auto rq = make_rsrc(static_cast<const char *>(s.q) + base, bytes);
        const uint32_t o = c * rqk + 16 * lg;
        u32x4 kj[4][N / 32], ki[N / 32], qi[N / 32];
#pragma unroll
        for (int st = 0; st < N / 32; ++st) {
            ki[st] = __builtin_amdgcn_raw_buffer_load_b128(rk, o, 16 * ti * rqk + 64 * st, 0);
            qi[st] = __builtin_amdgcn_raw_buffer_load_b128(rq, o, 16 * ti * rqk + 64 * st, 0);
        }
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const auto rz = make_rsrc(static_cast<const char *>(s.k) + base, z <= ti ? bytes : 0);
#pragma unroll
            for (int st = 0; st < N / 32; ++st) kj[z][st] = __builtin_amdgcn_raw_buffer_load_b128(rz, o, 16 * z * rqk + 64 * st, 0);
        }
        if (w >= 4 - HP) {   // a head's decays, while the rows are on their way
            const int y = w - (4 - HP), h = h0 + y;
            Decays &d = m[y].d;
            float al = 1.f, be = 0.f;
            if (lane < n) {
                al = s.a[(size_t)(t0 + lane) * s.H + h];
                be = s.dt[(size_t)(t0 + lane) * s.H + h];
            }
            const float pre = row_upto(al), suf = row_move<0x101>(row_from(al));
            const float p0 = lane_value(pre, 15), p1 = lane_value(pre, 31), p2 = lane_value(pre, 47), p3 = lane_value(pre, 63);
            const int tile = lane >> 4;
            const float ahead = tile == 0 ? 1.f : (tile == 1 ? p0 : (tile == 2 ? p0 * p1 : p0 * p1 * p2));
            const float behind = tile == 3 ? 1.f : (tile == 2 ? p3 : (tile == 1 ? p2 * p3 : p1 * p2 * p3));
            d.alpha[lane] = al;
            d.beta[lane] = be;
            d.pre[lane] = pre;
            d.suf[lane] = suf;
            if (lane < 4) d.tot[lane] = lane == 0 ? p0 : (lane == 1 ? p1 : (lane == 2 ? p2 : p3));
            float *decay = reinterpret_cast<float *>(out + (size_t)y * kSlot + kTBytes + kGBytes);
            decay[lane] = ahead * pre;
            decay[kQ + lane] = suf * behind;
            const bool bad = __any(!(finite(al) && finite(be)));
            if (lane == 0) odd[y] = bad;
        }
        bool bad = false;
#pragma unroll
        for (int st = 0; st < N / 32; ++st)
#pragma unroll
            for (int r = 0; r < 4; ++r) bad |= odd_pair(ki[st][r]);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            kk[z] = qk[z] = acc4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int st = 0; st < N / 32; ++st) {
                kk[z] = mma16(__builtin_bit_cast(bf8, kj[z][st]), __builtin_bit_cast(bf8, ki[st]), kk[z]);
                qk[z] = mma16(__builtin_bit_cast(bf8, kj[z][st]), __builtin_bit_cast(bf8, qi[st]), qk[z]);
            }
        }
        bad = __any(bad);
        lds_barrier();   // the decays
        if (bad && lane < HP) odd[lane] = 1;
    }
#pragma unroll
    for (int y = 0; y < HP; ++y) {
        uint8_t *to_head = out + (size_t)y * kSlot + kTBytes;
        const int i = 16 * ti + c;
        const float be = m[y].d.beta[i];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            if (x == pairs) break;
            acc4 o[2];   // G's operand
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int z = 2 * x + half, j0 = 16 * z + 4 * lg;
                f32x4 D = {0.f, 0.f, 0.f, 0.f};
                if (z <= ti) D = decays_of(m[y].d, ti, z, c, lg);
                f32x4 a;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    a[r] = j0 + r < i ? be * (kk[z][r] * D[r]) : 0.f;
                    o[half][r] = j0 + r <= i ? qk[z][r] * D[r] : 0.f;
                }
                *reinterpret_cast<f32x4 *>(&m[y].a[i][j0]) = a;   // (zeros above the diagonal are T's too)
            }
            bf8 parts[3];
            split<3>(o[0], o[1], parts);
            uint8_t *to = to_head + frag(ti, x) * 3 * kFrag + lane * 16;
#pragma unroll
            for (int z = 0; z < 3; ++z) put_frag(to + z * kFrag, parts[z]);
        }
    }
    lds_barrier();
    if (w < HP) {
        // the diagonal blocks by substitution: lane (block lg, column c) a column
        float(*a)[kQ + 4] = m[w].a;
        const int b0 = 16 * lg;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = i == c ? 1.f : 0.f;
#pragma unroll
            for (int j4 = 0; j4 < i; j4 += 4) {
                const f32x4 r4 = *reinterpret_cast<const f32x4 *>(&a[b0 + i][b0 + j4]);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (j4 + r < i) x[i] = fmaf(-r4[r], x[j4 + r], x[i]);
            }
        }
        wave_lds_sync();
#pragma unroll
        for (int i = 0; i < 16; ++i) a[b0 + i][b0 + c] = x[i];
    }
    lds_barrier();
    if (w < 2 * HP) invert_corner<16>(m[w >> 1].a, 32 * (w & 1), 0, lane);
    lds_barrier();
    if (w < 2 * HP) {
        invert_corner<32>(m[w >> 1].a, 0, w & 1, lane);
    } else {
        lds_barrier();   // the one in there
    }
    lds_barrier();
    for (int x = tid; x < HP * kFrags * 64; x += kPrepNT) {
        const int y = x / (kFrags * 64), f = x / 64 % kFrags, tile = f < 4 ? f : f - 2, step = f < 4 ? tile >> 1 : 0;
        const int l = x & 63, i = 16 * tile + (l & 15), j0 = 32 * step + 4 * (l >> 4);
        acc4 v[2];
#pragma unroll
        for (int z = 0; z < 2; ++z)
            v[z] = *reinterpret_cast<const acc4 *>(&m[y].a[i][j0 + 16 * z]) * *reinterpret_cast<const acc4 *>(&m[y].d.beta[j0 + 16 * z]);
        bf8 parts[3];
        split<3>(v[0], v[1], parts);
        uint8_t *to = out + (size_t)y * kSlot + f * 3 * kFrag + l * 16;
#pragma unroll
        for (int z = 0; z < 3; ++z) *reinterpret_cast<u32x4 *>(to + z * kFrag) = __builtin_bit_cast(u32x4, parts[z]);
    }
    if (tid < HP) *reinterpret_cast<uint32_t *>(out + (size_t)tid * kSlot + kImage) = odd[tid];
}

// ---- from chunk to chunk ----------------------------------------------------

template <int P, int N>
struct Shape {
    static constexpr int CW = 4, NT = 128 * CW, PC = 16 * CW, CB = P / PC;   // pairs of wavefronts, threads, columns, workgroups a head
    static constexpr int QB = 2 * N, KN = N / 32, KH = KN / 2;       // bytes of a row; steps over it, a wavefront's own
    static constexpr int IQ = kQ * QB / 16 / NT;                     // 16-byte pieces of k, and of q, that a thread stages
    // T and G come through LDS too: the wavefronts' own loads of them would be 120
    // KB a chunk, and what a CU gets from its L2 is some 18 bytes a clock.
    static constexpr int IT = (kImage + 16) / 16 / NT + 1;           // pieces of the chunk's slot
    static_assert(P % PC == 0 && kQ * QB / 16 % NT == 0, "whole pieces");
};

// What the two wavefronts of 16 columns hand each other, as operands.  Once K S^T is made
// U lies in place of s: of either's tokens where the other, which reads it, has its part.
template <int KN>
struct Exchange {
    uint8_t s[KN][3][kFrag], e[2][3][kFrag], r[3][kFrag];
};
template <int P, int N>
struct Tile {
    using Sh = Shape<P, N>;
    __align__(16) uint8_t k[kQ * Sh::QB], q[kQ * Sh::QB];
    uint8_t odd[16];
    __align__(16) Exchange<Sh::KN> x[Sh::CW];
    __align__(16) uint8_t slot[kImage + 16];
};

// The next chunk's k and q on their way to LDS: rows past its n tokens read zero.
template <int P, int N>
struct Ahead {
    using Sh = Shape<P, N>;
    u32x4 q[Sh::IQ], k[Sh::IQ], slot[Sh::IT];
    // n <= 0: nothing is read (no load is conditional, here and below: a
    // wait could not tell it from those behind it)
    __device__ __forceinline__ void load(const char *kp, const char *qp, uint32_t rqk, int n, const uint8_t *from) {
        const uint32_t bytes = n > 0 ? (uint32_t)(n < kQ ? n - 1 : kQ - 1) * rqk + Sh::QB : 0, tid = threadIdx.x;
        const auto rk = make_rsrc(kp, bytes), rq = make_rsrc(qp, bytes);
        const uint32_t o = tid / (Sh::QB / 16) * rqk + tid % (Sh::QB / 16) * 16, step = Sh::NT / (Sh::QB / 16) * rqk;
#pragma unroll
        for (int i = 0; i < Sh::IQ; ++i) {
            k[i] = __builtin_amdgcn_raw_buffer_load_b128(rk, o, i * step, 0);
            q[i] = __builtin_amdgcn_raw_buffer_load_b128(rq, o, i * step, 0);
        }
        const auto rs = make_rsrc(from, n > 0 ? kImage + 16 : 0);
#pragma unroll
        for (int i = 0; i < Sh::IT; ++i) slot[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, tid * 16, i * Sh::NT * 16, 0);
    }
    __device__ __forceinline__ void store(Tile<P, N> &m) const {
        constexpr int PR = Sh::QB / 16, RS = Sh::NT / PR;   // pieces of a row; rows from one of a thread's to the next
        static_assert(RS % 8 == 0, "their permutations differ by exchanges of 16-byte pieces alone");
        const int tid = threadIdx.x, row = tid / PR, f = turn(row);
        const int o = row * Sh::QB + ((tid % PR * 16) ^ ((f & 14) << 3));
        const bool swap = f & 1;
        auto put = [&](uint8_t *to, u32x4 x) { *reinterpret_cast<u32x4 *>(to) = swap ? u32x4{x[2], x[3], x[0], x[1]} : x; };
#pragma unroll
        for (int i = 0; i < Sh::IQ; ++i) {
            const int to = (o ^ ((turn(i * RS) & 14) << 3)) + i * Sh::NT * 16;
            put(m.k + to, k[i]);
            put(m.q + to, q[i]);
        }
#pragma unroll
        for (int i = 0; i < Sh::IT; ++i)
            if ((i * Sh::NT + tid) * 16 < kImage + 16) *reinterpret_cast<u32x4 *>(m.slot + (i * Sh::NT + tid) * 16) = slot[i];
    }
};

// v: column c, tokens 32 th + 16 x + 4 lg + r of the next chunk
struct Values {
    uint32_t v[8];
    __device__ __forceinline__ void load(const char *vp, uint32_t rv, int n, uint32_t o) {
        const auto r = make_rsrc(vp, n > 0 ? (uint32_t)(n - 1) * rv + 32 : 0);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, o, (i & 3) * rv + (i >> 2) * 16 * rv, 0);
    }
};

// What a wavefront takes of a chunk's slot, from the copy in LDS: T at its own step and
// (th = 1) at step 0, g and e of the tokens of v, g of the last; for its two tiles of y,
// th and 3 - th, G of the first at step 0, of the other at step 1 and at step 0, and g.
struct Slot {
    const uint8_t *frags, *decay, *natural, *base;
    int step;
    __device__ __forceinline__ void init(const uint8_t *m, int th, int lane) {
        base = m;
        frags = m + 16 * lane;
        decay = m + kTBytes + kGBytes + (32 * th + 4 * (lane >> 4)) * 4;
        natural = m + kTBytes + kGBytes + (lane & 15) * 4;
        step = th;
    }
    __device__ __forceinline__ bf8 t(int x, int z) const { return frag16(frags + (6 * step + 3 * x + z) * kFrag); }
    __device__ __forceinline__ bf8 tx(int x, int z) const { return frag16(frags + (12 + 3 * x + z) * kFrag); }
    __device__ __forceinline__ bf8 g(int i, int z) const {
        return frag16(frags + kTBytes + (3 * (i == 0 ? frag(step, 0) : frag(3 - step, i == 1)) + z) * kFrag);
    }
    __device__ __forceinline__ f32x4 d(int x) const { return *reinterpret_cast<const f32x4 *>(decay + 64 * x); }
    __device__ __forceinline__ f32x4 e(int x) const { return *reinterpret_cast<const f32x4 *>(decay + 4 * kQ + 64 * x); }
    __device__ __forceinline__ float dn(int x) const { return *reinterpret_cast<const float *>(natural + 64 * (x ? 3 - step : step)); }
    __device__ __forceinline__ float all() const { return *reinterpret_cast<const float *>(base + kTBytes + kGBytes + 4 * (kQ - 1)); }
    __device__ __forceinline__ uint32_t odd() const { return *reinterpret_cast<const uint32_t *>(base + kImage); }
};

// Two wavefronts take 16 columns: th = 0, 1 have the chunk's tokens 32 th ..
// in R and U, the state's rows N / 2 th .. in S^T, and of y's four tiles of 16 tokens
// th and 3 - th, three products of G and U either (with 32 tokens each th = 1 has four and
// th = 0 two).  The system is lower triangular, so that th = 0 needs nothing of th = 1 for R and U.
template <int P, int N>
__global__ __launch_bounds__((Shape<P, N>::NT), 2) void delta_mx_kernel(ScanArgs s) {
    using Sh = Shape<P, N>;
    constexpr int KN = Sh::KN, KH = Sh::KH, QB = Sh::QB;
    __shared__ Tile<P, N> m;

    Place place;
    if (!find_place(s, 1, &place, Sh::CB)) return;
    const int h = place.h, b = place.b, g = place.g;
    const Span sp = find_span(s, b, 0);
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6), th = w & 1, pair = w >> 1;
    if (s.chunk0 == 0 && h == 0 && place.cb == 0 && !sp.run && tid == 0) raise_seq_error(s.err, b, REPLAY_SEQERR_BAD_RANGE);
    const int from = s.chunk0 * kQ, upto = sp.n < from + s.window * kQ ? sp.n : from + s.window * kQ;
    if (!sp.run || (from > 0 && from >= sp.n)) return;
    Exchange<KN> &ex = m.x[pair];
    uint8_t &odd_chunk = m.odd[pair];   // of the two wavefronts'

    const int p0 = Sh::PC * place.cb + 16 * pair;   // the wavefront's columns
    const size_t bh = (size_t)b * s.H + h;
    float *const state = s.s_out + (bh * P + p0 + c) * N + 4 * lg;          // columns 16 t + 4 lg ..
    const float *in = from > 0 ? s.s_out : s.s_in;
    // tile t of the wavefront's half of S^T: n = N / 2 th + 16 t + 4 lg + r
    acc4 S[2 * KH];
    auto get_state = [&](const float *from_) {
#pragma unroll
        for (int t = 0; t < 2 * KH; ++t) {
            S[t] = acc4{0.f, 0.f, 0.f, 0.f};
            if (from_) S[t] = *reinterpret_cast<const acc4 *>(from_ + N / 2 * th + 16 * t);
        }
    };
    auto put_state = [&] {
#pragma unroll
        for (int t = 0; t < 2 * KH; ++t) *reinterpret_cast<acc4 *>(state + N / 2 * th + 16 * t) = S[t];
    };
    auto hand_state = [&] {
        uint8_t *to = ex.s[KH * th][0] + 16 * lane;
#pragma unroll
        for (int i = 0; i < KH; ++i) {
            bf8 part[3];
            split<3>(S[2 * i], S[2 * i + 1], part);
#pragma unroll
            for (int z = 0; z < 3; ++z) put_frag(to + (3 * i + z) * kFrag, part[z]);
        }
    };
    get_state(in ? in + (bh * P + p0 + c) * N + 4 * lg : nullptr);
    if (upto == from) {   // no tokens: the state as it is
        put_state();
        return;
    }
    const uint32_t rv = (uint32_t)s.H * P * 2, rqk = (uint32_t)s.G * QB;
    const size_t t0 = (size_t)(sp.t0 + from);
    const char *kp = static_cast<const char *>(s.k) + t0 * rqk + (size_t)g * QB;
    const char *qp = static_cast<const char *>(s.q) + t0 * rqk + (size_t)g * QB;
    const char *vp = static_cast<const char *>(s.v) + t0 * rv + ((size_t)h * P + p0) * 2;
    char *yp = static_cast<char *>(s.y) + t0 * rv + ((size_t)h * P + p0) * 2;
    const uint8_t *slot = reinterpret_cast<const uint8_t *>(s.ws) + ((size_t)b * s.window * s.H + h) * kSlot;
    const size_t next_slot = (size_t)s.H * kSlot;
    const uint32_t vo = (32 * th + 4 * lg) * rv + 2 * c, yo = c * rv + 8 * lg;
    // places in a row's 128 bytes of the four pieces 4 i + lg, and of k^T's 4 i + c % 4
    int piece[4], col[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        piece[i] = (32 * th + c) * QB + (((4 * i + lg) ^ turn(c)) << 3);
        col[i] = (4 * lg + (c >> 2)) * QB + (((4 * i + (c & 3)) ^ turn(4 * lg + (c >> 2))) << 3);
    }
    auto operand = [&](const uint8_t *rows, int x, int st) {   // of tokens 32 th + 16 x + c, step st
        const int o = 16 * QB * x + 128 * (st >> 1), i = 2 * (st & 1);
        return row8(rows + piece[i] + o, rows + piece[i + 1] + o);
    };
    const int tile[2] = {th, 3 - th};   // of y
    const uint8_t *const xl = reinterpret_cast<const uint8_t *>(&ex) + 16 * lane;
    constexpr int kE = KN * 3 * kFrag, kR = kE + 6 * kFrag, kU = KH * 3 * kFrag;       // places in Exchange (kU: of th = 1)
    Ahead<P, N> ahead;
    Values val;
    Slot my;
    ahead.load(kp, qp, rqk, upto - from, slot);
    val.load(vp, rv, sp.n - from < kQ ? sp.n - from : kQ, vo);
    my.init(m.slot, th, lane);
    hand_state();
    if (th == 0 && lane == 0) odd_chunk = 0;
    ahead.store(m);
    for (int done = from; done < upto; done += kQ) {
        const int n = sp.n - done < kQ ? sp.n - done : kQ, left = upto - done - kQ;   // of this chunk; behind it
        lds_barrier();   // k, q and the operands of S^T
        kp += (size_t)kQ * rqk;
        qp += (size_t)kQ * rqk;
        vp += (size_t)kQ * rv;
        slot += next_slot;
        ahead.load(kp, qp, rqk, left, slot);
        // K S^T, rows token 32 th + 16 x + 4 lg + r, column c.  S Q^T, rows p = 4
        // lg + r, column token 16 tile[x] + c, comes behind U: here all wavefronts would
        // read k, q and S at once.
        acc4 ks[2], y[2];
        bf8 part[KN][3];   // S, kept for S Q^T
#pragma unroll
        for (int st = 0; st < KN; ++st) {
            bf8 k[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) k[x] = operand(m.k, x, st);
#pragma unroll
            for (int z = 2; z >= 0; --z) {
                const bf8 p = part[st][z] = frag16(xl + (3 * st + z) * kFrag);
#pragma unroll
                for (int x = 0; x < 2; ++x) ks[x] = mma16(k[x], p, st == 0 && z == 2 ? acc4{0.f, 0.f, 0.f, 0.f} : ks[x]);
            }
        }
        // (0 v is a NaN where v is no number)
        float none = my.odd() ? __builtin_nanf("") : 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const f32x4 d = my.d(x);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float v = bf16_bits_to_f32(val.v[4 * x + r]);
                none = fmaf(v, 0.f, none);
                ks[x][r] = fmaf(-d[r], ks[x][r], v);
            }
        }
        if (__any(none != none) && lane == 0) odd_chunk = 1;
        bf8 rp[3];
        split<3>(ks[0], ks[1], rp);
        if (th == 0)
#pragma unroll
            for (int z = 0; z < 3; ++z) put_frag(ex.r[z] + 16 * lane, rp[z]);
        lds_barrier();   // R of the first tokens
        const bool odd = odd_chunk != 0;
        val.load(vp, rv, left < kQ ? left : kQ, vo);
        bf8 up[3], ep[3];
        if (!odd) {
            acc4 u[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) u[x] = acc4{0.f, 0.f, 0.f, 0.f};
            if (th) {
                bf8 rx[3];
#pragma unroll
                for (int z = 0; z < 3; ++z) rx[z] = frag16(xl + kR + z * kFrag);
#pragma unroll
                for (int z = kProducts - 1; z >= 0; --z)
#pragma unroll
                    for (int x = 0; x < 2; ++x) u[x] = mma16(my.tx(x, kA[z]), rx[kB[z]], u[x]);
            }
#pragma unroll
            for (int z = kProducts - 1; z >= 0; --z)
#pragma unroll
                for (int x = 0; x < 2; ++x) u[x] = mma16(my.t(x, kA[z]), rp[kB[z]], u[x]);
            split<3>(u[0], u[1], up);
#pragma unroll
            for (int z = 0; z < 3; ++z) put_frag(ex.s[th ? 0 : KH][z] + 16 * lane, up[z]);
#pragma unroll
            for (int x = 0; x < 2; ++x) u[x] *= my.e(x);
            split<3>(u[0], u[1], ep);
#pragma unroll
            for (int z = 0; z < 3; ++z) put_frag(ex.e[th][z] + 16 * lane, ep[z]);
#pragma unroll
            for (int st = 0; st < KN; ++st) {
                bf8 q[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) q[x] = operand(m.q + (16 * tile[x] - 32 * th) * QB, 0, st);
#pragma unroll
                for (int z = 2; z >= 0; --z)
#pragma unroll
                    for (int x = 0; x < 2; ++x) y[x] = mma16(part[st][z], q[x], st == 0 && z == 2 ? acc4{0.f, 0.f, 0.f, 0.f} : y[x]);
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) y[x] *= my.dn(x);
        } else {
            put_state();
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        }
        const float all = my.all();   // (before the slot's next chunk is loaded)
        lds_barrier();   // U and e U
        if (!odd) {
            // y^T: + U^T G^T, in three accumulators, so that few products wait for each other
            bf8 ux[3];
#pragma unroll
            for (int z = 0; z < 3; ++z) ux[z] = frag16(xl + (th ? kU : 0) + z * kFrag);
            acc4 more = {0.f, 0.f, 0.f, 0.f};
            auto add = [&](const bf8 *u0, const bf8 *u1) {
#pragma unroll
                for (int z = kProducts - 1; z >= 0; --z) {
                    y[0] = mma16(u0[kA[z]], my.g(0, kB[z]), y[0]);
                    y[1] = mma16(u1[kA[z]], my.g(1, kB[z]), y[1]);
                    more = mma16(u0[kA[z]], my.g(2, kB[z]), more);
                }
            };
            if (th) add(ux, up);
            else add(up, ux);
            y[1] += more;
            const auto ys = make_rsrc(yp, (uint32_t)(n - 1) * rv + 32);
#pragma unroll
            for (int x = 0; x < 2; ++x)
                __builtin_amdgcn_raw_buffer_store_b64(
                    u32x2{f32x2_to_bf16_pair(y[x][0], y[x][1]), f32x2_to_bf16_pair(y[x][2], y[x][3])}, ys, yo, 16 * tile[x] * rv, 0);
            // S^T <- (whole decay) S^T + K^T (e U), the wavefront's own tokens first
            bf8 ox[3];
#pragma unroll
            for (int z = 0; z < 3; ++z) ox[z] = frag16(xl + kE + 3 * kFrag * (1 - th) + z * kFrag);
#pragma unroll
            for (int t = 0; t < 2 * KH; ++t) S[t] *= all;
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const uint8_t *const from_k = m.k + 32 * QB * (st ? 1 - th : th) + (KH == 2 ? 128 * th : 0);
                bf8 k[2 * KH];
#pragma unroll
                for (int t = 0; t < 2 * KH; ++t) {
                    const uint8_t *const kt = from_k + (KH == 2 ? col[t] : (th ? col[t + 2] : col[t]));
                    const s16x4 lo = col4(kt), hi = col4(kt + 16 * QB);
                    k[t] = __builtin_bit_cast(bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                }
#pragma unroll
                for (int z = 2; z >= 0; --z)
#pragma unroll
                    for (int t = 0; t < 2 * KH; ++t) S[t] = mma16(k[t], st ? ox[z] : ep[z], S[t]);
            }
            hand_state();
        } else if (th == 0) {
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
            by_token<P, N>(s, m.k, m.q, state, sp.t0 + done, n, h, p0 + c, lane);
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        }
        yp += (size_t)kQ * rv;
        lds_barrier();   // k, q and what was handed over are read to their end
        if (odd) {
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
            get_state(state);
            hand_state();
        }
        if (th == 0 && lane == 0) odd_chunk = 0;
        ahead.store(m);
    }
    put_state();
}

template <int P, int N>
hipError_t launch_chain(const ScanArgs &a, hipStream_t s) {
    using Sh = Shape<P, N>;
    delta_mx_kernel<P, N><<<scan_blocks(a, 1, Sh::CB), Sh::NT, 0, s>>>(a);
    return hipGetLastError();
}

template <int P, int N>
hipError_t launch_pn(ScanArgs a, hipStream_t s) {
    const int chunks = ((a.seg_len < a.max_len ? a.seg_len : a.max_len) + kQ - 1) / kQ;
    for (a.chunk0 = 0; a.chunk0 < chunks; a.chunk0 += a.window) {
        const int64_t units = (int64_t)a.B * a.window * a.H;
        if (a.H / a.G % 2 == 0)
            delta_prep_kernel<N, 2><<<(unsigned)(units / 2), kPrepNT, 0, s>>>(a);
        else
            delta_prep_kernel<N, 1><<<(unsigned)units, kPrepNT, 0, s>>>(a);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        // delta_few.hip's workgroups of 16 columns read k, q and T four times as often,
        // but there are four times as many to keep the card busy.  2048 tokens, 64
        // columns of a head counted as one, state of 128 columns: 128 of them 123 us there,
        // 168 here; 192: 194 and 183; state of 64: 128 of them 110 and 157, 192: 218 and 210.
        e = (int64_t)a.B * a.H * P / 64 > 128 ? launch_chain<P, N>(a, s) : launch_delta_few(P, N, a, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// More than this and the workspace is used again, window after window.
constexpr size_t kMostWorkspace = (size_t)512 << 20;

}  // namespace

int delta_window(int P, int N, int B, int H, bool bf16, int longest, size_t *bytes) {
    *bytes = 0;
    if (!bf16 || P < 64) return 0;
    const size_t each = (size_t)B * H * kSlot;   // a chunk of every sequence
    const size_t chunks = ((size_t)longest + kQ - 1) / kQ;
    size_t n = kMostWorkspace / each;
    n = n < 1 ? 1 : (n > chunks ? chunks : n);
    *bytes = n * each;
    return (int)n;
}

hipError_t launch_delta_mx(int P, int N, const ScanArgs &a, hipStream_t s) {
    if (P == 64 && N == 64) return launch_pn<64, 64>(a, s);
    if (P == 64 && N == 128) return launch_pn<64, 128>(a, s);
    if (P == 128 && N == 128) return launch_pn<128, 128>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace replay
