// prompt.h -- private declarations of the calls around the recurrence: the
// inputs' convolution (conv.hip), prompts (scan.hip, scan_mx.hip) and
// sampling (sample.hip).
#pragma once

#include "internal.h"

namespace replay {

// A launch numbers its threads, over all workgroups, in 32 bits.
inline bool launch_fits(int64_t blocks, int64_t threads) { return blocks <= (int64_t)UINT32_MAX / threads; }

// Most values in a row of x, q, k, v or y: 64 rows, a chunk of the scan, then
// stay within 32-bit byte offsets.
constexpr int64_t kMaxRow = 1 << 24;

// The inputs of the recurrence from projected rows (conv.hip): T packed rows
// of a prompt batch, or T = B W rows of a step or round.
struct ConvArgs {
    int32_t B, H, G, P, N, C;      // C = H P + 2 G N channels, [v | k | q]
    int32_t K, R, silu, io_bf16;
    int32_t T, W;
    const int32_t *cu;             // prompts: [B + 1]
    const void *x, *dt_raw;        // rows x_stride, dt_stride elements apart; dt_raw null: no dt, a
    int64_t x_stride, dt_stride;
    const int32_t *pos, *base, *n_reject;
    const void *state_in;          // prompts: [B][R][C] or null (zeros)
    void *state_out;               // [B][R][C]; a step reads its history here too
    const float *weight, *bias, *dt_bias, *a_log;   // [C][K], [C], [H], [H]
    float dt_min, dt_max;
    void *q, *k, *v;
    float *dt, *a;
    int32_t *err;
};

// The recurrence over packed prompts (scan.hip).
struct ScanArgs {
    int32_t B, H, G, T, max_len, io_bf16;
    const int32_t *cu;             // [B + 1]
    const void *q, *k, *v;         // [T][G][N] x2, [T][H][P]
    const float *dt, *a;           // [T][H]
    const float *s_in;             // [B][H][P][N] or null (zeros)
    float *s_out;
    void *y;                       // [T][H][P], io dtype
    int32_t *err;
    int32_t nseg, seg_len;         // segments of a sequence, tokens of a segment
    float *ws;                     // nseg > 1: states [B][H][nseg - 1][P][N], then
    float *ws_decay;               // decays [B][H][nseg - 1]
};

// Sampling (sample.hip).
struct SampleArgs {
    int32_t B, W, V, bf16;
    const void *logits;            // B W rows of V, stride elements apart
    int64_t stride;
    const float *temperature, *top_p, *min_p;   // [B] each, or null
    const int32_t *top_k;
    const float *u;                // [B][W]
    int32_t *tokens;               // [B][W]
    float *probs;                  // [B][W] or null
    const int32_t *fed;            // [B][W], with
    int32_t *n_reject;             // [B]; both or neither
};
constexpr int kMaxVocab = 1 << 18;
constexpr int kSampleNT = 512;   // threads of a row, a workgroup each

// Launchers (return hipSuccess or the launch error).
hipError_t launch_sample(const SampleArgs &a, hipStream_t s);
hipError_t launch_scan(int P, int N, const ScanArgs &a, hipStream_t s);
int scan_segments(int P, int N, int B, int H, int G, bool bf16, int T, int max_len, int *seg_len);   // the number of segments, and their length
// hipErrorInvalidConfiguration: more workgroups than a launch numbers
hipError_t launch_conv_prompt(const ConvArgs &a, hipStream_t s);
hipError_t launch_conv_step(const ConvArgs &a, hipStream_t s);

}  // namespace replay
