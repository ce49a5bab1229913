// What a tree of drafted tokens needs around its attention: the ancestor
// masks and positions of its nodes, and, once a path of it is accepted, the
// move of that path's cache rows up behind the committed ones.
//
// A sequence's tree has n <= 64 nodes, appended at positions L - n .. L - 1
// of its context (L = context_len, the tree included); node t's parent is an
// earlier node or -1 (a child of the last committed token).
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

static __device__ unsigned g_draft_error = 0;

constexpr int kTreeMaxNodes = 64;
constexpr int kPageTokens = 16;

// mask[t] = bit t | mask[parent], position = L - n + depth, depth = bits - 1.
// One CTA per sequence, one thread per node; six doublings of the ancestor
// pointers reach 64 nodes up.  20 bytes a node: bound by the launch (256 trees of
// 16 nodes: 1.6 us in a graph).
__global__ void __launch_bounds__(kTreeMaxNodes)
tree_layout_kernel(const int32_t* __restrict__ parents, const int32_t* __restrict__ q_start,
                   int total_q, int max_q_len, const int32_t* __restrict__ context_lens,
                   unsigned long long* __restrict__ tree_mask, int64_t* __restrict__ positions) {
  griddep_wait();
  __shared__ unsigned long long mask[kTreeMaxNodes];
  __shared__ int up[kTreeMaxNodes];
  const int seq = blockIdx.x, t = threadIdx.x;
  const int qs = __ldg(q_start + seq), qe = __ldg(q_start + seq + 1);
  const int ctx = __ldg(context_lens + seq);
  const int n = qe - qs;
  if (qs < 0 || n < 0 || qe > total_q || n > max_q_len || n > ctx) {
    if (t == 0) atomicOr(&g_draft_error, kErrBadQueryRange);
    return;
  }
  int p = -1;
  if (t < n) {
    p = __ldg(parents + qs + t);
    if (p < -1 || p >= t) {
      atomicOr(&g_draft_error, kErrBadTree);
      p = -1;
    }
  }
  mask[t] = 1ull << t;
  up[t] = p;
  __syncthreads();
#pragma unroll
  for (int step = 0; step < 6; ++step) {
    const int a = up[t];
    const unsigned long long above = a >= 0 ? mask[a] : 0ull;
    const int further = a >= 0 ? up[a] : -1;
    __syncthreads();
    mask[t] |= above;
    up[t] = further;
    __syncthreads();
  }
  if (t < n) {
    tree_mask[qs + t] = mask[t];
    positions[qs + t] = int64_t(ctx - n) + __popcll(mask[t]) - 1;
  }
}

// The row at position L - n + accepted[i] moves to position L - n + i, in
// every layer's K and V pool, for i < num_accepted; accepted is increasing,
// so accepted[i] >= i.
//
// In place without a second buffer or a barrier: a thread owns one 16-byte
// column of the rows and moves it in order of i, kMoveBatch loads ahead of
// their stores.  Row i is a source only of moves j <= i, so each column is
// read before it is overwritten.  A move of a row onto itself is skipped.
// Bound by memory for a batch over all layers (64 sequences x 32 layers, FP8:
// 7.8 us in a graph, the bytes' 4.4), by the launch for few sequences (2.5 us).
constexpr int kMoveThreads = 128;
constexpr int kMoveBatch = 8;

__global__ void __launch_bounds__(kMoveThreads)
accept_rows_kernel(const AcceptArgs a) {
  griddep_wait();
  __shared__ int64_t src[kTreeMaxNodes], dst[kTreeMaxNodes];
  const int per_seq = a.col_blocks;
  const int64_t item = blockIdx.x / per_seq;
  const int cb = int(blockIdx.x - item * per_seq);
  const int layer = int(item / a.num_seqs);
  const int seq = int(item - int64_t(layer) * a.num_seqs);
  const int i = threadIdx.x;
  // the path is read beside the sizes that say how much of it counts
  const int32_t* path = a.accepted + int64_t(seq) * a.max_accepted;
  const int node = i < a.max_accepted ? __ldg(path + i) : 0;
  const int before = i > 0 && i < a.max_accepted ? __ldg(path + i - 1) : -1;
  const int qs = __ldg(a.q_start + seq), qe = __ldg(a.q_start + seq + 1);
  const int ctx = __ldg(a.context_lens + seq);
  const int count = __ldg(a.num_accepted + seq);
  const int n = qe - qs;
  const bool first = layer == 0 && cb == 0;  // this block reports for the sequence
  bool ok = n >= 0 && n <= kTreeMaxNodes && n <= ctx &&
            (int64_t(ctx) + kPageTokens - 1) / kPageTokens <= a.max_blocks_per_seq && count >= 0 &&
            count <= n && count <= a.max_accepted;
  if (ok && i < count && (node <= before || node >= n)) ok = false;
  ok = __syncthreads_and(ok);
  if (!ok) {
    if (first && threadIdx.x == 0) {
      atomicOr(&g_draft_error, kErrBadTree);
      a.new_context_lens[seq] = ctx;
    }
    return;
  }
  const int base = ctx - n;
  if (first && threadIdx.x == 0) a.new_context_lens[seq] = base + count;
  if (i < count) {
    const int32_t* table = a.block_tables + int64_t(seq) * a.max_blocks_per_seq;
    const int from = base + node, to = base + i;
    const int bf = __ldg(table + from / kPageTokens), bt = __ldg(table + to / kPageTokens);
    const bool known = bf >= 0 && bf < a.num_blocks && bt >= 0 && bt < a.num_blocks;
    if (!known && first) atomicOr(&g_draft_error, kErrBadBlockId);
    src[i] = known && from != to ? int64_t(bf) * kPageTokens + from % kPageTokens : -1;
    dst[i] = int64_t(bt) * kPageTokens + to % kPageTokens;
  }
  __syncthreads();
  int col = cb * kMoveThreads + threadIdx.x;
  if (col >= 2 * a.row_vec) return;
  uint4* pool = col < a.row_vec ? a.k_cache + int64_t(layer) * a.k_layer_vec
                                : a.v_cache + int64_t(layer) * a.v_layer_vec;
  if (col >= a.row_vec) col -= a.row_vec;
  for (int b = 0; b < count; b += kMoveBatch) {
    uint4 r[kMoveBatch];
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u)
      if (b + u < count && src[b + u] >= 0) r[u] = pool[src[b + u] * a.row_vec + col];
#pragma unroll
    for (int u = 0; u < kMoveBatch; ++u)
      if (b + u < count && src[b + u] >= 0) pool[dst[b + u] * a.row_vec + col] = r[u];
  }
}

cudaError_t draft_error_word(unsigned** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_draft_error);
}

unsigned read_draft_error(bool clear) {
  unsigned word = 0;
  if (cudaMemcpyFromSymbol(&word, g_draft_error, sizeof(word)) != cudaSuccess) return ~0u;
  if (clear) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_draft_error, &zero, sizeof(zero)) != cudaSuccess) return ~0u;
  }
  return word;
}

int tree_max_nodes() { return kTreeMaxNodes; }

cudaError_t launch_tree_layout(const int32_t* parents, const int32_t* q_start, int num_seqs,
                               int total_q, int max_q_len, const int32_t* context_lens,
                               uint64_t* tree_mask, int64_t* positions, cudaStream_t stream) {
  return launch_after_previous(tree_layout_kernel, dim3(num_seqs), dim3(kTreeMaxNodes), 0, stream,
                               parents, q_start, total_q, max_q_len, context_lens,
                               reinterpret_cast<unsigned long long*>(tree_mask), positions);
}

static int accept_col_blocks(int row_vec) {
  return (2 * row_vec + kMoveThreads - 1) / kMoveThreads;
}

int64_t accept_rows_blocks(int num_layers, int num_seqs, int row_vec) {
  return int64_t(num_layers) * num_seqs * accept_col_blocks(row_vec);
}

cudaError_t launch_accept_rows(const AcceptArgs& args, int num_layers, cudaStream_t stream) {
  AcceptArgs a = args;
  a.col_blocks = accept_col_blocks(a.row_vec);
  const int64_t blocks = accept_rows_blocks(num_layers, a.num_seqs, a.row_vec);
  return launch_after_previous(accept_rows_kernel, dim3(unsigned(blocks)), dim3(kMoveThreads), 0,
                               stream, a);
}

}  // namespace pkv
