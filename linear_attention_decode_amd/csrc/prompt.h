// prompt.h -- private declarations of the calls around the recurrence: the
// inputs' convolution (conv.hip), prompts (scan.hip, scan_mx.hip), sampling
// (sample.hip) and token scores (logprobs.hip).
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
    const int32_t *parent, *n_nodes;   // trees: [B][W], [B] or null
    const int32_t *path, *n_keep;      // a kept path into the state: [B][W], [B]
};
constexpr int kMaxTree = 64;   // nodes of a tree: a lane each

// A Gated DeltaNet layer's inputs (delta_inputs.hip): T rows.
struct DeltaInputsArgs {
    int32_t T, H, G, N, io_bf16;
    const void *q_in, *k_in;           // [T][G][N]
    void *q, *k;
    const void *b_raw, *a_raw;         // T rows of H, b_stride, a_stride elements apart
    int64_t b_stride, a_stride;
    const float *dt_bias, *a_log;      // [H]
    float q_scale, eps;
    float *beta, *alpha;               // [T][H]
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
    // the gated delta rule's bf16 kernels: chunks of a sequence in the
    // workspace at a time, and the first of them
    int32_t window, chunk0;
    int32_t share;                 // log2 of the XCDs that share a group's workgroups
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

// Scores of tokens (logprobs.hip).
struct LogprobArgs {
    int32_t B, W, V, M, n, bf16;   // M given tokens, n alternatives a row
    const void *logits;            // B W rows of V, stride elements apart
    int64_t stride;
    const float *temperature;      // [B] or null
    const int32_t *ids;            // [B][W][M]
    float *logp, *entropy;         // [B][W][M]; [B][W] or null
    int32_t *top_ids;              // [B][W][n], with
    float *top_logp;               // [B][W][n]
    uint64_t *ws;                  // [B W][parts][kPartWords + max(n, 1)]
    int32_t parts, part;           // parts of a row, elements of a part
};
constexpr int kMaxTop = 32;
constexpr int kPartWords = 3;      // a part's sums, ahead of its first tokens
constexpr int kPartNT = 256;       // threads of a part, and of a row's join
constexpr int kPartBig = 8192, kPartSmall = 2048;
int logprob_part(int64_t rows, int V, int *parts);   // elements of a part, and their number

// Launchers (return hipSuccess or the launch error).
hipError_t launch_logprobs(const LogprobArgs &a, hipStream_t s);
hipError_t launch_sample(const SampleArgs &a, hipStream_t s);
hipError_t launch_scan(int P, int N, const ScanArgs &a, hipStream_t s);
// the gated delta rule (delta_scan.hip): dt carries beta, a alpha
hipError_t launch_delta_scan(int P, int N, const ScanArgs &a, hipStream_t s);
// chunks of a sequence that the workspace holds at a time (0: it needs none), and its bytes
int delta_window(int P, int N, int B, int H, bool bf16, int longest, size_t *bytes);
int scan_segments(int P, int N, int B, int H, int G, bool bf16, int T, int max_len, int *seg_len);   // the number of segments, and their length
// hipErrorInvalidConfiguration: more workgroups than a launch numbers
hipError_t launch_conv_prompt(const ConvArgs &a, hipStream_t s);
hipError_t launch_conv_step(const ConvArgs &a, hipStream_t s);
hipError_t launch_conv_tree(const ConvArgs &a, hipStream_t s);   // with path: the kept rows into the state
hipError_t launch_delta_inputs(const DeltaInputsArgs &a, hipStream_t s);
// the path that sampled tokens confirm (tree.hip)
hipError_t launch_accept_tree(int B, int W, const int32_t *parent, const int32_t *n_nodes, const int32_t *tokens,
                              const int32_t *fed, int32_t *path, int32_t *n_keep, hipStream_t s);

}  // namespace replay
