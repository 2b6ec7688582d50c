// tree.hip -- what follows the scoring of a tree of drafted tokens: the path
// that the sampled tokens confirm, and its append to the ring.
#include "tree.h"
#include "tree_common.h"

namespace replay {

namespace {

// A wavefront a sequence, a lane a node: from node 0, which was fed the
// sequence's last token, to the child that was fed what was sampled behind
// it, while there is one (the first of equal ones).  A chain of as many steps as
// tokens are kept: 5 us for 16, whatever the batch.
__global__ __launch_bounds__(64) void accept_tree_kernel(int W, const int32_t *parent, const int32_t *n_nodes,
                                                         const int32_t *tokens, const int32_t *fed, int32_t *path,
                                                         int32_t *n_keep) {
    const int b = blockIdx.x, lane = threadIdx.x;
    Tree tree;
    tree.load(parent, n_nodes, b, W, lane);
    const size_t at = (size_t)b * W + lane;
    const int token = lane < tree.n ? tokens[at] : -1, mine = lane < tree.n ? fed[at] : -1;
    int keep = 0, out = -1, cur = 0;
    while (keep < tree.n) {
        if (lane == keep) out = cur;
        ++keep;
        const int want = __builtin_amdgcn_readlane(token, cur);
        const uint64_t next = __ballot(lane < tree.n && tree.parent == cur && mine == want && want >= 0);
        if (!next) break;
        cur = __builtin_ctzll(next);   // later than its parent: every node is taken once at most
    }
    if (lane < W) path[at] = out;
    if (lane == 0) n_keep[b] = keep;
}

// As append_kernel (ring.hip), the tokens a path's nodes.  Bound by the copy: 256
// sequences of 64 heads of 64 and 8 groups of 128, 16 nodes each, 17 us for 104 MB.
constexpr int kSlices = 8;

__global__ __launch_bounds__(256) void append_path_kernel(TreeArgs t, const int32_t *path, const int32_t *n_keep, void *ring_q,
                                                          void *ring_k, void *ring_v, float *ring_dt, float *ring_a,
                                                          int32_t *pos, int32_t *sync, int32_t P, int32_t N) {
    const RingView &r = t.r;
    const int b = blockIdx.x, sl = blockIdx.y, tid = threadIdx.x, nt = blockDim.x, lane = tid & 63;
    const int H = r.H, G = r.G, L = r.L, W = t.W;
    __shared__ int s_path[kMaxTree];
    const int p0 = pos[b], count = p0 - r.base[b], n = n_keep[b];
    const int node = lane < W ? path[(size_t)b * W + lane] : 0;
    int bad = 0;
    if (n < 0 || n > W || __any(lane < n && (node < 0 || node >= W)))
        bad = REPLAY_SEQERR_BAD_TREE;
    else if (count < 0 || count + n > L)
        bad = REPLAY_SEQERR_RING_OVERFLOW;
    else if ((long long)p0 + n > 2147483647LL)
        bad = REPLAY_SEQERR_POS_OVERFLOW;
    if (bad) {   // the same in every wavefront of every slice
        if (sl == 0 && tid == 0) raise_seq_error(r.err, b, bad);
        return;
    }
    if (tid < 64 && lane < n) s_path[lane] = node;
    __syncthreads();
    const int esz = r.io_bf16 ? 2 : 4;
    const int h0 = sl * H / kSlices, nh = (sl + 1) * H / kSlices - h0;
    const int g0 = sl * G / kSlices, ng = (sl + 1) * G / kSlices - g0;
    {
        const int pieces = P * esz / 16;
        const uint4 *src = static_cast<const uint4 *>(t.v);
        uint4 *dst = static_cast<uint4 *>(ring_v);
        for (int i = tid; i < n * nh * pieces; i += nt) {
            const int row = i / pieces, c = i % pieces, k = row / nh, h = h0 + row % nh;
            dst[(((size_t)b * H + h) * L + (p0 + k) % L) * pieces + c] = src[(((size_t)b * W + s_path[k]) * H + h) * pieces + c];
        }
    }
    {
        const int pieces = N * esz / 16;
        for (int i = tid; i < n * ng * pieces; i += nt) {
            const int row = i / pieces, c = i % pieces, k = row / ng, g = g0 + row % ng;
            const size_t to = (((size_t)b * G + g) * L + (p0 + k) % L) * pieces + c;
            const size_t from = (((size_t)b * W + s_path[k]) * G + g) * pieces + c;
            static_cast<uint4 *>(ring_q)[to] = static_cast<const uint4 *>(t.q)[from];
            static_cast<uint4 *>(ring_k)[to] = static_cast<const uint4 *>(t.k)[from];
        }
    }
    for (int i = tid; i < n * nh; i += nt) {
        const int k = i / nh, h = h0 + i % nh;
        const size_t to = dta_index(b, (size_t)b * H + h, H, L, (p0 + k) % L), from = ((size_t)b * W + s_path[k]) * H + h;
        ring_dt[to] = t.dt[from];
        ring_a[to] = t.a[from];
    }
    // every wavefront of this slice has read pos[b] before the slice arrives
    __syncthreads();
    if (tid == 0) {
        int32_t *cnt = sync + ((size_t)b * (G + 1) + G) * kSyncStride;
        if (atomicAdd(cnt, 1) == kSlices - 1) {
            atomicExch(cnt, 0);
            pos[b] = p0 + n;
        }
    }
}

}  // namespace

hipError_t launch_accept_tree(int B, int W, const int32_t *parent, const int32_t *n_nodes, const int32_t *tokens,
                              const int32_t *fed, int32_t *path, int32_t *n_keep, hipStream_t s) {
    accept_tree_kernel<<<B, 64, 0, s>>>(W, parent, n_nodes, tokens, fed, path, n_keep);
    return hipGetLastError();
}

hipError_t launch_append_path(int P, int N, const TreeArgs &t, const int32_t *path, const int32_t *n_keep, void *ring_q,
                              void *ring_k, void *ring_v, float *ring_dt, float *ring_a, int32_t *pos, int32_t *sync,
                              hipStream_t s) {
    append_path_kernel<<<dim3(t.r.B, kSlices), 256, 0, s>>>(t, path, n_keep, ring_q, ring_k, ring_v, ring_dt, ring_a, pos,
                                                            sync, P, N);
    return hipGetLastError();
}

}  // namespace replay
