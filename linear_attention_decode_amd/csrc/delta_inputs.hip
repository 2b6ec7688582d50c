// delta_inputs.hip -- what a Gated DeltaNet layer does between its convolution
// and the gated delta rule: queries and keys to unit length, and its two
// scalars,
//     q <- q_scale q / sqrt(q . q + eps),   k <- k / sqrt(k . k + eps),
//     beta = 1 / (1 + exp(-b)),   alpha = exp(-exp(a_log) softplus(a + dt_bias)).
//
// Bound by HBM, every value read and written once: 15013 rows of 16 queries, 16 keys
// of 128 and 32 heads in bf16, 38 us for 252 MB, of which the last-level cache
// holds a part; 16 rows 2 us.  A vector of N elements
// lies in N / 8 (float32: N / 4) neighbouring lanes, 16 bytes each, and its
// length is summed over them without LDS.
#include "device_common.h"
#include "prompt.h"

namespace replay {

namespace {

constexpr int kNT = 256;

// Workgroups [0, vector_blocks): kNT 16-byte pieces of q, then of k; the
// others kNT (row, head) pairs each.
template <bool BF16, int N>
__global__ __launch_bounds__(kNT) void delta_inputs_kernel(DeltaInputsArgs a, unsigned piece_blocks) {
    constexpr int E = BF16 ? 8 : 4, LPV = N / E;   // elements and lanes
    if (blockIdx.x < 2 * piece_blocks) {
        const bool key = blockIdx.x >= piece_blocks;
        const size_t i = ((size_t)(key ? blockIdx.x - piece_blocks : blockIdx.x) * kNT + threadIdx.x) * E;
        const bool in = i < (size_t)a.T * a.G * N;   // whole vectors: the lanes of one agree
        float x[E] = {};
        if (in) {
            IoVec<BF16, E> r;
            r.load(key ? a.k_in : a.q_in, i);
            r.widen(x);
        }
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
        ss = group_sum<LPV>(ss) + a.eps;
        if (!(ss >= 0x1p-80f && ss < 0x1p126f)) {   // squares that float32 may not hold: of the vector times a power of two
            const float by = ss < 0x1p-80f ? 0x1p100f : 0x1p-70f;
            ss = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                x[e] *= by;
                ss = fmaf(x[e], x[e], ss);
            }
            ss = group_sum<LPV>(ss) + a.eps * by * by;   // the lanes of a vector are here together
        }
        if (!in) return;
        const float f = (key ? 1.f : a.q_scale) / sqrtf(ss);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] *= f;
        void *dst = key ? a.k : a.q;
        if constexpr (BF16) {
            u32x4 w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = f32x2_to_bf16_pair(x[2 * e], x[2 * e + 1]);
            *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(dst) + i) = w;
        } else {
            *reinterpret_cast<f32x4 *>(static_cast<float *>(dst) + i) = f32x4{x[0], x[1], x[2], x[3]};
        }
        return;
    }
    const size_t i = (size_t)(blockIdx.x - 2 * piece_blocks) * kNT + threadIdx.x;
    if (i >= (size_t)a.T * a.H) return;
    const size_t t = i / a.H;
    const int h = (int)(i % a.H);
    const float b = load_io1<BF16>(a.b_raw, t * (size_t)a.b_stride + h);
    float x = load_io1<BF16>(a.a_raw, t * (size_t)a.a_stride + h);
    if (a.dt_bias) x += a.dt_bias[h];
    float d = fmaxf(x, 0.f) + log1pf(expf(-fabsf(x)));
    if (x != x) d = x;
    a.beta[i] = 1.f / (1.f + expf(-b));
    a.alpha[i] = expf(-expf(a.a_log[h]) * d);
}

template <bool BF16, int N>
hipError_t launch_one(const DeltaInputsArgs &a, hipStream_t s) {
    const int64_t pieces = (int64_t)a.T * a.G * N / (BF16 ? 8 : 4);
    const int64_t pb = (pieces + kNT - 1) / kNT, blocks = 2 * pb + ((int64_t)a.T * a.H + kNT - 1) / kNT;
    if (!launch_fits(blocks, kNT)) return hipErrorInvalidConfiguration;
    delta_inputs_kernel<BF16, N><<<(unsigned)blocks, kNT, 0, s>>>(a, (unsigned)pb);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_inputs(const DeltaInputsArgs &a, hipStream_t s) {
    if (a.N == 16) return a.io_bf16 ? launch_one<true, 16>(a, s) : launch_one<false, 16>(a, s);
    if (a.N == 64) return a.io_bf16 ? launch_one<true, 64>(a, s) : launch_one<false, 64>(a, s);
    if (a.N == 128) return a.io_bf16 ? launch_one<true, 128>(a, s) : launch_one<false, 128>(a, s);
    return hipErrorInvalidValue;
}

}  // namespace replay
