// delta_few.hip -- delta_mx.hip's way from chunk to chunk where heads are few:
// four or six wavefronts for 16 columns, so that each of a CU's SIMDs has one.
//
// TH of them (two or four) have the state, wavefront th the chunk's tokens 64 / TH th
// .. in R and U and the state's rows N / TH th .. of S^T.  What one of them makes
// enters the others' products as an operand of 32 steps or as half of one, through
// LDS.  Two more make y, tokens 0 .. 15 and 48 .. 63 or those between, from the
// operands of S^T and U that lie there anyway.
//
// Bound by the chain of a chunk's steps: K S^T, R = V - diag(g) K S^T, U = T R, the
// state, each with its cutting into parts of 8 bits, four barriers apart.  One
// sequence of 8192 tokens (32 heads of 128 x 128), 128 chunks: 275 us with TH = 4, some
// 5000 cycles a chunk, of which K S^T takes 750, R 400, U with its parts more than 1100, the
// state 500, handing it on 400, what comes from and goes to memory 500, the barriers
// 850.  With tokens 0 .. 31 and 32 .. 63 on the wavefronts that make y, two products of G
// and U on one and four on the other, 289.
#include "delta_mx.h"

namespace replay {

namespace {

constexpr int kFewCUs = 256;

template <int N, int TH>
struct Few {
    static constexpr int NS = 64 * TH, NT = NS + 128;                  // threads that have the state, and stage k; all
    static constexpr int QB = 2 * N, KN = N / 32;                      // bytes of a row; steps over it
    static constexpr int X = 4 / TH, KT = N / 16 / TH;                 // a wavefront's tiles of tokens, and of S^T
    __align__(16) uint8_t k[kQ * QB], q[kQ * QB];
    __align__(16) uint8_t s[KN][3][kFrag], r[2][3][kFrag], e[2][3][kFrag], u[2][3][kFrag];   // operands
    uint32_t odd;
};

// Rows of k or q on their way to LDS, by THREADS threads; those past n read zero.
template <int N, int THREADS>
struct Rows {
    static constexpr int QB = 2 * N, I = kQ * QB / 16 / THREADS, PR = QB / 16, RS = THREADS / PR;
    static_assert(kQ * QB / 16 % THREADS == 0 && RS % 8 == 0, "a thread's rows' permutations differ by exchanges of 16-byte pieces alone");
    u32x4 x[I];
    __device__ __forceinline__ void load(const char *p, uint32_t rqk, int n, int tid) {
        const auto rs = make_rsrc(p, n > 0 ? (uint32_t)(n < kQ ? n - 1 : kQ - 1) * rqk + QB : 0);
#pragma unroll
        for (int i = 0; i < I; ++i) x[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, tid / PR * rqk + tid % PR * 16, i * RS * rqk, 0);
    }
    __device__ __forceinline__ void store(uint8_t *m, int tid) const {
        const int row = tid / PR, f = turn(row), o = row * QB + ((tid % PR * 16) ^ ((f & 14) << 3));
        const bool swap = f & 1;
#pragma unroll
        for (int i = 0; i < I; ++i)
            *reinterpret_cast<u32x4 *>(m + (o ^ ((turn(i * RS) & 14) << 3)) + i * THREADS * 16) =
                swap ? u32x4{x[i][2], x[i][3], x[i][0], x[i][1]} : x[i];
    }
};

// Tiles of an operand's steps, x one tile or two neighbouring ones, as PARTS operands
// (or halves of them) from `to` on; tile: the first one's number.
template <int PARTS, int X>
__device__ __forceinline__ void put_tiles(uint8_t *to, int tile, const acc4 *x, int lane) {
    if constexpr (X == 2) {
        bf8 part[PARTS];
        split<PARTS>(x[0], x[1], part);
#pragma unroll
        for (int z = 0; z < PARTS; ++z) put_frag(to + ((tile >> 1) * PARTS + z) * kFrag + 16 * lane, part[z]);
    } else {
        u32x2 part[PARTS];
        split4<PARTS>(x[0], part);
#pragma unroll
        for (int z = 0; z < PARTS; ++z)
            *reinterpret_cast<u32x2 *>(to + ((tile >> 1) * PARTS + z) * kFrag + 16 * lane + 8 * (tile & 1)) = part[z];
    }
}

template <int P, int N, int TH>
__global__ __launch_bounds__((Few<N, TH>::NT)) void delta_few_kernel(ScanArgs s) {
    using Sh = Few<N, TH>;
    constexpr int KN = Sh::KN, KT = Sh::KT, QB = Sh::QB, X = Sh::X;
    __shared__ Sh m;

    Place place;
    if (!find_place(s, 1, &place, P / 16)) return;
    const int h = place.h, b = place.b, g = place.g;
    const Span sp = find_span(s, b, 0);
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    if (s.chunk0 == 0 && h == 0 && place.cb == 0 && !sp.run && tid == 0) raise_seq_error(s.err, b, REPLAY_SEQERR_BAD_RANGE);
    const int from = s.chunk0 * kQ, upto = sp.n < from + s.window * kQ ? sp.n : from + s.window * kQ;
    if (!sp.run || (from > 0 && from >= sp.n)) return;

    const int p0 = 16 * place.cb;
    const size_t bh = (size_t)b * s.H + h;
    const uint32_t rv = (uint32_t)s.H * P * 2, rqk = (uint32_t)s.G * QB;
    const size_t t0 = (size_t)(sp.t0 + from);
    const uint8_t *slot = reinterpret_cast<const uint8_t *>(s.ws) + ((size_t)b * s.window * s.H + h) * kSlot;
    const size_t next_slot = (size_t)s.H * kSlot;
    // an operand's two pieces in a row's 128 bytes: 4 i + lg
    auto pieces = [&](int *at, int row0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] = (row0 + c) * QB + (((4 * i + lg) ^ turn(c)) << 3);
    };
    auto operand = [&](const uint8_t *rows, const int *at, int st) {
        const int o = 128 * (st >> 1), i = 2 * (st & 1);
        return row8(rows + at[i] + o, rows + at[i + 1] + o);
    };

    if (w >= TH) {   // y; the same barriers as below
        if (upto == from) return;
        const int tile[2] = {w - TH, 3 - (w - TH)};   // of 16 tokens: three products of G and U in all for either wavefront
        const char *qp = static_cast<const char *>(s.q) + t0 * rqk + (size_t)g * QB;
        char *yp = static_cast<char *>(s.y) + t0 * rv + ((size_t)h * P + p0) * 2;
        const uint32_t yo = c * rv + 8 * lg;
        int at[4];
        pieces(at, 0);
        Rows<N, Sh::NT - Sh::NS> rows;
        bf8 G[3][3];   // tile[0] at step 0, tile[1] at step 1, and at step 0
        float gt[2];   // g of tokens 16 tile[x] + c
        auto load_slot = [&](const uint8_t *from_) {   // (null: nothing is read)
            const auto ws = make_rsrc(from_, from_ ? kSlot : 0);
            const int at_[3] = {frag(tile[0], 0), frag(tile[1], 1), frag(tile[1], 0)};
#pragma unroll
            for (int x = 0; x < 2; ++x)
                gt[x] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ws, (16 * tile[x] + c) * 4, kTBytes + kGBytes, 0));
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int z = 0; z < 3; ++z)
                    G[i][z] = __builtin_bit_cast(bf8, __builtin_amdgcn_raw_buffer_load_b128(ws, 16 * lane, kTBytes + (3 * at_[i] + z) * kFrag, 0));
        };
        rows.load(qp, rqk, upto - from, tid - Sh::NS);
        load_slot(slot);
        rows.store(m.q, tid - Sh::NS);
        for (int done = from; done < upto; done += kQ) {
            const int n = sp.n - done < kQ ? sp.n - done : kQ, left = upto - done - kQ;   // of this chunk; behind it
            lds_barrier();   // q and the operands of S^T
            qp += (size_t)kQ * rqk;
            slot += next_slot;
            rows.load(qp, rqk, left, tid - Sh::NS);
            // S Q^T, rows p = 4 lg + r, column token 16 tile[x] + c
            acc4 y[2] = {acc4{0.f, 0.f, 0.f, 0.f}, acc4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int st = 0; st < KN; ++st) {
                const bf8 q[2] = {operand(m.q + 16 * tile[0] * QB, at, st), operand(m.q + 16 * tile[1] * QB, at, st)};
#pragma unroll
                for (int z = 2; z >= 0; --z) {
                    const bf8 p = frag16(m.s[st][z] + 16 * lane);
#pragma unroll
                    for (int x = 0; x < 2; ++x) y[x] = mma16(p, q[x], y[x]);
                }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) y[x] *= gt[x];
            lds_barrier();   // (R)
            const bool odd = m.odd != 0;
            lds_barrier();   // U
            if (!odd) {   // + U^T G^T
                bf8 u[2][3];
#pragma unroll
                for (int st = 0; st < 2; ++st)
#pragma unroll
                    for (int z = 0; z < 3; ++z) u[st][z] = frag16(m.u[st][z] + 16 * lane);
                acc4 more = {0.f, 0.f, 0.f, 0.f};   // three accumulators, so that few products wait for each other
#pragma unroll
                for (int z = kProducts - 1; z >= 0; --z) {
                    y[0] = mma16(u[0][kA[z]], G[0][kB[z]], y[0]);
                    y[1] = mma16(u[1][kA[z]], G[1][kB[z]], y[1]);
                    more = mma16(u[0][kA[z]], G[2][kB[z]], more);
                }
                y[1] += more;
                const auto ys = make_rsrc(yp, (uint32_t)(n - 1) * rv + 32);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    __builtin_amdgcn_raw_buffer_store_b64(
                        u32x2{f32x2_to_bf16_pair(y[x][0], y[x][1]), f32x2_to_bf16_pair(y[x][2], y[x][3])}, ys, yo, 16 * tile[x] * rv, 0);
            }
            yp += (size_t)kQ * rv;
            load_slot(left > 0 ? slot : nullptr);
            lds_barrier();   // q and what was handed over are read to their end
            rows.store(m.q, tid - Sh::NS);
        }
        return;
    }

    const int th = w, own = X * th >> 1;   // its tokens' step of 32
    float *const state = s.s_out + (bh * P + p0 + c) * N + 4 * lg;   // columns 16 t + 4 lg ..
    const float *in = from > 0 ? s.s_out : s.s_in;
    acc4 S[KT];   // rows n = N / TH th + 16 t + 4 lg + r of S^T
    auto get_state = [&](const float *from_) {
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            S[t] = acc4{0.f, 0.f, 0.f, 0.f};
            if (from_) S[t] = *reinterpret_cast<const acc4 *>(from_ + N / TH * th + 16 * t);
        }
    };
    auto put_state = [&] {
#pragma unroll
        for (int t = 0; t < KT; ++t) *reinterpret_cast<acc4 *>(state + N / TH * th + 16 * t) = S[t];
    };
    auto hand_state = [&] {
#pragma unroll
        for (int t = 0; t < KT; t += 2) put_tiles<3, (KT > 1 ? 2 : 1)>(m.s[0][0], KT * th + t, S + t, lane);
    };
    get_state(in ? in + (bh * P + p0 + c) * N + 4 * lg : nullptr);
    if (upto == from) {   // no tokens: the state as it is
        put_state();
        return;
    }
    const char *kp = static_cast<const char *>(s.k) + t0 * rqk + (size_t)g * QB;
    const char *vp = static_cast<const char *>(s.v) + t0 * rv + ((size_t)h * P + p0) * 2;
    const uint32_t vo = (16 * X * th + 4 * lg) * rv + 2 * c;
    int at[4], col[KT];   // col: of k^T's tile t, tokens 4 lg ..
    pieces(at, 16 * X * th);
#pragma unroll
    for (int t = 0; t < KT; ++t) {
        const int tile = KT * th + t, row = 4 * lg + (c >> 2);
        col[t] = row * QB + 128 * (tile >> 2) + (((4 * (tile & 3) + (c & 3)) ^ turn(row)) << 3);
    }
    Rows<N, Sh::NS> rows;
    uint32_t val[X][4];       // v: column c, tokens 16 (X th + x) + 4 lg + r
    bf8 T[X][3], T0[X][3];    // at its own step; (where that is 1) at step 0
    f32x4 d[X], e[X];         // g and e of those tokens
    float all;                // g of the last
    uint32_t odd_k;
    auto load_values = [&](int n) {
        const auto r = make_rsrc(vp, n > 0 ? (uint32_t)(n - 1) * rv + 32 : 0);
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) val[x][i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, vo, (16 * x + i) * rv, 0);
    };
    auto load_slot = [&](const uint8_t *from_) {   // (null: nothing is read)
        const auto ws = make_rsrc(from_, from_ ? kSlot : 0), wx = make_rsrc(from_, from_ && own ? kSlot : 0);
        const uint32_t o = (16 * X * th + 4 * lg) * 4, after = kTBytes + kGBytes;
#pragma unroll
        for (int x = 0; x < X; ++x) {
            d[x] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ws, o + 64 * x, after, 0));
            e[x] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(ws, o + 4 * kQ + 64 * x, after, 0));
        }
        all = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ws, 4 * (kQ - 1), after, 0));
        odd_k = __builtin_amdgcn_raw_buffer_load_b32(ws, 2 * 4 * kQ, after, 0);
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
            for (int z = 0; z < 3; ++z) {
                T[x][z] = __builtin_bit_cast(bf8, __builtin_amdgcn_raw_buffer_load_b128(ws, 16 * lane, (3 * (X * th + x) + z) * kFrag, 0));
                T0[x][z] = __builtin_bit_cast(bf8, __builtin_amdgcn_raw_buffer_load_b128(wx, 16 * lane, (3 * (2 + X * th + x) + z) * kFrag, 0));
            }
    };
    rows.load(kp, rqk, upto - from, tid);
    load_values(sp.n - from < kQ ? sp.n - from : kQ);
    load_slot(slot);
    hand_state();
    if (tid == 0) m.odd = 0;
    rows.store(m.k, tid);
    for (int done = from; done < upto; done += kQ) {
        const int n = sp.n - done < kQ ? sp.n - done : kQ, left = upto - done - kQ;   // of this chunk; behind it
        lds_barrier();   // k and the operands of S^T
        kp += (size_t)kQ * rqk;
        vp += (size_t)kQ * rv;
        slot += next_slot;
        rows.load(kp, rqk, left, tid);
        // K S^T, rows token 16 (X th + x) + 4 lg + r, column c; a single tile in two
        // accumulators, so that its products do not wait for each other
        acc4 ks[2] = {acc4{0.f, 0.f, 0.f, 0.f}, acc4{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int st = 0; st < KN; ++st) {
            bf8 k[X];
#pragma unroll
            for (int x = 0; x < X; ++x) k[x] = operand(m.k + 16 * x * QB, at, st);
#pragma unroll
            for (int z = 2; z >= 0; --z) {
                const bf8 p = frag16(m.s[st][z] + 16 * lane);
#pragma unroll
                for (int x = 0; x < X; ++x) ks[X == 2 ? x : st & 1] = mma16(k[x], p, ks[X == 2 ? x : st & 1]);
            }
        }
        // (0 v is a NaN where v is no number)
        float none = odd_k ? __builtin_nanf("") : 0.f;
        acc4 R[X];
#pragma unroll
        for (int x = 0; x < X; ++x)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float v = bf16_bits_to_f32(val[x][r]);
                none = fmaf(v, 0.f, none);
                R[x][r] = fmaf(-d[x][r], X == 2 ? ks[x][r] : ks[0][r] + ks[1][r], v);
            }
        if (__any(none != none) && lane == 0) m.odd = 1;
        put_tiles<3, X>(m.r[0][0], X * th, R, lane);
        lds_barrier();   // R
        const bool odd = m.odd != 0;
        load_values(left < kQ ? left : kQ);
        if (!odd) {
            // U = T R
            acc4 u[X];
#pragma unroll
            for (int x = 0; x < X; ++x) u[x] = acc4{0.f, 0.f, 0.f, 0.f};
            bf8 Ro[3];
#pragma unroll
            for (int z = 0; z < 3; ++z) Ro[z] = frag16(m.r[own][z] + 16 * lane);
            if (own) {
                acc4 u0[X];
#pragma unroll
                for (int x = 0; x < X; ++x) u0[x] = acc4{0.f, 0.f, 0.f, 0.f};
                bf8 R0[3];
#pragma unroll
                for (int z = 0; z < 3; ++z) R0[z] = frag16(m.r[0][z] + 16 * lane);
#pragma unroll
                for (int z = kProducts - 1; z >= 0; --z)
#pragma unroll
                    for (int x = 0; x < X; ++x) {
                        u0[x] = mma16(T0[x][kA[z]], R0[kB[z]], u0[x]);
                        u[x] = mma16(T[x][kA[z]], Ro[kB[z]], u[x]);
                    }
#pragma unroll
                for (int x = 0; x < X; ++x) u[x] += u0[x];
            } else {
#pragma unroll
                for (int z = kProducts - 1; z >= 0; --z)
#pragma unroll
                    for (int x = 0; x < X; ++x) u[x] = mma16(T[x][kA[z]], Ro[kB[z]], u[x]);
            }
            put_tiles<3, X>(m.u[0][0], X * th, u, lane);
#pragma unroll
            for (int x = 0; x < X; ++x) u[x] *= e[x];
            put_tiles<3, X>(m.e[0][0], X * th, u, lane);
        } else {
            put_state();
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        }
        const float decay = all;
        load_slot(left > 0 ? slot : nullptr);
        lds_barrier();   // U and e U
        if (!odd) {
            // S^T <- (whole decay) S^T + K^T (e U)
#pragma unroll
            for (int t = 0; t < KT; ++t) S[t] *= decay;
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                bf8 k[KT];
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    const uint8_t *const kt = m.k + 32 * QB * st + col[t];
                    const s16x4 lo = col4(kt), hi = col4(kt + 16 * QB);
                    k[t] = __builtin_bit_cast(bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                }
#pragma unroll
                for (int z = 2; z >= 0; --z) {
                    const bf8 u = frag16(m.e[st][z] + 16 * lane);
#pragma unroll
                    for (int t = 0; t < KT; ++t) S[t] = mma16(k[t], u, S[t]);
                }
            }
            hand_state();
        } else if (th == 0) {
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
            by_token<P, N>(s, m.k, m.q, state, sp.t0 + done, n, h, p0 + c, lane);
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        }
        lds_barrier();   // k and what was handed over are read to their end
        if (odd) {
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
            get_state(state);
            hand_state();
        }
        if (tid == 0) m.odd = 0;
        rows.store(m.k, tid);
    }
    put_state();
}

template <int P, int N, int TH>
hipError_t launch_one(const ScanArgs &a, hipStream_t s) {
    delta_few_kernel<P, N, TH><<<scan_blocks(a, 1, P / 16), Few<N, TH>::NT, 0, s>>>(a);
    return hipGetLastError();
}

// Whether every workgroup has a CU of its own.  Two of TH = 4 and 128 columns of
// state on one are slower than two of TH = 2: 2048 tokens of 32 heads of 128 x 128 take
// 79 us with TH = 4 and 92 with TH = 2, of 64 heads 143 and 123.  With 64 columns of
// state, half the LDS traffic, TH = 4 is ahead in both: 64 heads of 64 x 64 73 and
// 81 us, 128 heads 110 and 115.
bool alone(int P, const ScanArgs &a) { return (int64_t)a.B * a.H * P / 16 <= kFewCUs; }

}  // namespace

hipError_t launch_delta_few(int P, int N, const ScanArgs &a, hipStream_t s) {
    if (P == 64 && N == 64) return launch_one<64, 64, 4>(a, s);
    if (P == 64 && N == 128) return alone(P, a) ? launch_one<64, 128, 4>(a, s) : launch_one<64, 128, 2>(a, s);
    if (P == 128 && N == 128) return alone(P, a) ? launch_one<128, 128, 4>(a, s) : launch_one<128, 128, 2>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace replay
