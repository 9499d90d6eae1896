// pa_commit_tree: keep the accepted path of every sequence's drafted tree.
//
// The drafted tokens of a sequence sit in the cache rows behind its context, in
// node order; the accepted ones are a node and its ancestors, p_0 < p_1 < ... .
// Committing moves row (context + p_j) to row (context + j) in every layer, K and
// V, and sets the context's new length. Since p is increasing, p_j >= j: a row is
// written only after it has been read when the rows of one sequence move in
// order, so the move needs no scratch. Pure data movement, bit-exact; a row that
// is in its place already (the usual start of a path) is not touched.
#include <algorithm>
#include <cstdint>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kCommitThreads = 128;
constexpr int kCommitLayers = 128;  // layers per launch (their pointers are kernel arguments, 2 KB)
constexpr int kCommitMaxWords = 4;  // trees of up to 256 nodes
constexpr int kCommitFlight = 8;    // rows a thread has in flight

struct CommitPtrs {
  uint4* k[kCommitLayers];
  uint4* v[kCommitLayers];
};

struct CommitParams {
  const int32_t* block_tables;
  int max_blocks;
  const int32_t *context_lens, *query_starts;
  const int32_t* before;                // null: a sequence without a context gets length 0; may be new_context_lens
  const unsigned long long* tree_mask;  // null: drafts without branches
  int words;
  const int32_t* accepted;
  int32_t* new_context_lens;
  int num_tokens, layers, layers_per_cta;
  int G, vpr, B, nhd;                   // vpr: 16-byte vectors of one head's row
  long long num_blocks;
  unsigned* err;
};

// grid = (sequences, layer chunks, 2): one CTA moves the K (z = 0) or V rows of
// one sequence for layers_per_cta layers. The first warp turns the path into a
// list of (source, destination) rows; then each thread takes 16-byte columns and
// moves all the list's rows of a column in order, eight loads ahead of their
// stores (the stores of a batch end at row j + 7 < p_{j+8}, the next batch's
// first source).
// Bound by the chain of loads that finds the path (lengths, mask, block ids), which every
// CTA repeats, and by the moves behind it, not by bandwidth: 64 sequences x 32 layers move
// 27 MB in 14.7 us in a graph (54 MB read and written, 3.7 TB/s of 6.8); four or six rows
// in flight at up to 16 CTAs per SM are within 1%, and slower (14.3 - 15.1 us for 14.2) on
// 40-head rows.
__global__ void __launch_bounds__(kCommitThreads) commit_tree_kernel(const CommitPtrs ptrs, const CommitParams p) {
  pdl_begin();
  __shared__ long long src[64 * kCommitMaxWords], dst[64 * kCommitMaxWords];  // first vector of head 0's row
  __shared__ int moves;
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) {
    const bool lead = blockIdx.y == 0 && blockIdx.z == 0 && lane == 0;
    const int q0 = __ldg(p.query_starts + s), q1 = __ldg(p.query_starts + s + 1);
    int ctx = __ldg(p.context_lens + s);
    const int acc = __ldg(p.accepted + s);
    unsigned bad = 0;
    const long long room = (long long)p.max_blocks * p.B;
    if (ctx < 0 || ctx > room) {
      bad |= kErrContext;
      ctx = ctx < 0 ? 0 : (int)room;
    }
    int n = (int)((unsigned)q1 - (unsigned)q0);
    if (q0 < 0 || q1 < q0 || q1 > p.num_tokens || n > ctx) {
      // no drafted tokens that could be told from the context (an unserved sequence has neither)
      if (ctx > 0 || q0 < 0 || q1 < q0 || q1 > p.num_tokens) bad |= kErrQuery;
      n = 0;
    }
    int a = acc;
    if (a < -1 || a >= n) {
      if (n > 0) bad |= kErrQuery;
      a = -1;
    }
    if (p.tree_mask != nullptr && n > 64 * p.words) {
      bad |= kErrQuery;
      a = -1;
    }
    const int prefix = ctx - n;
    int kept = 0, listed = 0;
    if (a >= 0 && p.tree_mask == nullptr) kept = a + 1;  // nodes 0 .. a are in place
    if (a >= 0 && p.tree_mask != nullptr) {
      for (int w = 0; w < p.words; ++w) {
        unsigned long long bits = __ldg(p.tree_mask + (long long)(q0 + a) * p.words + w);
        const int left = n - 64 * w;  // nodes of this word
        if (left <= 0) bits = 0;
        else if (left < 64) bits &= (1ull << left) - 1;
        // lane: bits lane and lane + 32 of the word, each to its rank on the path
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int b = lane + 32 * h;
          const bool on = (bits >> b) & 1;
          const int rank = kept + __popcll(bits & ((1ull << b) - 1));
          const bool move = on && rank != 64 * w + b;
          const unsigned ballot = __ballot_sync(0xffffffffu, move);
          if (move) {
            const int from = prefix + 64 * w + b, to = prefix + rank;
            const long long fb = __ldg(p.block_tables + (long long)s * p.max_blocks + from / p.B);
            const long long tb = __ldg(p.block_tables + (long long)s * p.max_blocks + to / p.B);
            const bool ok = fb >= 0 && fb < p.num_blocks && tb >= 0 && tb < p.num_blocks;
            if (!ok) bad |= kErrBlockId;
            const int at = listed + __popc(ballot & ((1u << lane) - 1));
            const long long row = p.vpr;
            const long long fr = p.nhd ? (fb * p.B + from % p.B) * p.G * row : (fb * p.G * p.B + from % p.B) * row;
            const long long tr = p.nhd ? (tb * p.B + to % p.B) * p.G * row : (tb * p.G * p.B + to % p.B) * row;
            src[at] = ok ? fr : -1;
            dst[at] = tr;
          }
          listed += __popc(ballot);
        }
        kept += __popcll(bits);
      }
    }
    if (bad && blockIdx.y == 0 && blockIdx.z == 0) atomicOr(p.err, bad);
    // A context of 0 is how an unserved sequence comes here: it keeps the length that it had. (Only this thread reads
    // the old length, so the new one may be written over it.)
    if (lead) p.new_context_lens[s] = ctx == 0 && p.before != nullptr ? max(p.before[s], 0) : prefix + kept;
    if (lane == 0) moves = listed;
  }
  __syncthreads();
  const int n = moves;
  if (n == 0) return;
  const int l0 = blockIdx.y * p.layers_per_cta, l1 = min(p.layers, l0 + p.layers_per_cta);
  const long long head = p.nhd ? p.vpr : (long long)p.B * p.vpr;  // vectors between two heads' rows
  const int cols = p.G * p.vpr;
  for (int l = l0; l < l1; ++l) {
    uint4* pool = blockIdx.z ? ptrs.v[l] : ptrs.k[l];
    for (int c = tid; c < cols; c += kCommitThreads) {
      uint4* col = pool + (c / p.vpr) * head + c % p.vpr;
      for (int j = 0; j < n; j += kCommitFlight) {
        uint4 r[kCommitFlight];
#pragma unroll
        for (int u = 0; u < kCommitFlight; ++u)
          if (j + u < n && src[j + u] >= 0) r[u] = col[src[j + u]];
#pragma unroll
        for (int u = 0; u < kCommitFlight; ++u)
          if (j + u < n && src[j + u] >= 0) col[dst[j + u]] = r[u];
      }
    }
  }
}

// Whether a pool is given twice (its rows would move twice, at the same time). Addresses that meet in the table of bits
// are compared with all before them; the others are distinct.
bool twice(void* const* k, void* const* v, int layers) {
  uint64_t seen[64] = {0};
  auto pool = [&](int i) { return i < layers ? k[i] : v[i - layers]; };
  for (int i = 0; i < 2 * layers; ++i) {
    const uint64_t h = ((uint64_t)reinterpret_cast<uintptr_t>(pool(i)) >> 4) * 0x9E3779B97F4A7C15ull >> 52;
    if (seen[h >> 6] >> (h & 63) & 1)
      for (int j = 0; j < i; ++j)
        if (pool(j) == pool(i)) return true;
    seen[h >> 6] |= 1ull << (h & 63);
  }
  return false;
}

int esize(pa_dtype dt) { return dt == PA_F32 ? 4 : (dt == PA_FP8_E4M3 ? 1 : 2); }
bool valid_dtype(pa_dtype dt) { return dt == PA_F32 || dt == PA_F16 || dt == PA_BF16 || dt == PA_FP8_E4M3; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace pa

extern "C" pa_status pa_commit_tree(void* const* k_caches, void* const* v_caches, int num_layers,
                                    const int32_t* block_tables, int max_blocks_per_seq,
                                    const int32_t* context_lens, const int32_t* query_starts,
                                    const int64_t* tree_mask, int mask_words, const int32_t* accepted,
                                    int32_t* new_context_lens, int num_seqs, int num_tokens, int num_kv_heads,
                                    int head_dim, int block_size, pa_kv_layout layout, int64_t num_blocks,
                                    pa_dtype dtype, cudaStream_t stream) {
  return pa_commit_tree_keep(k_caches, v_caches, num_layers, block_tables, max_blocks_per_seq, context_lens, nullptr,
                             query_starts, tree_mask, mask_words, accepted, new_context_lens, num_seqs, num_tokens,
                             num_kv_heads, head_dim, block_size, layout, num_blocks, dtype, stream);
}

extern "C" pa_status pa_commit_tree_keep(void* const* k_caches, void* const* v_caches, int num_layers,
                                         const int32_t* block_tables, int max_blocks_per_seq,
                                         const int32_t* context_lens, const int32_t* context_lens_before,
                                         const int32_t* query_starts, const int64_t* tree_mask, int mask_words,
                                         const int32_t* accepted, int32_t* new_context_lens, int num_seqs,
                                         int num_tokens, int num_kv_heads, int head_dim, int block_size,
                                         pa_kv_layout layout, int64_t num_blocks, pa_dtype dtype,
                                         cudaStream_t stream) {
  using namespace pa;
  if (num_layers <= 0 || num_seqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      num_blocks <= 0 || max_blocks_per_seq <= 0 || !valid_dtype(dtype) ||
      (layout != PA_LAYOUT_HND && layout != PA_LAYOUT_NHD))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!k_caches || !v_caches || !block_tables || !context_lens || !query_starts || !accepted || !new_context_lens)
    return PA_ERR_INVALID_ARG;
  const void* words4[] = {block_tables, context_lens, context_lens_before, query_starts, accepted, new_context_lens};
  for (const void* q : words4)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return PA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(tree_mask) & 7u) || (tree_mask != nullptr && mask_words <= 0))
    return PA_ERR_INVALID_ARG;
  for (int l = 0; l < num_layers; ++l)
    if (!k_caches[l] || !v_caches[l] || !aligned16(k_caches[l]) || !aligned16(v_caches[l])) return PA_ERR_INVALID_ARG;
  if (twice(k_caches, v_caches, num_layers)) return PA_ERR_INVALID_ARG;
  // every CTA of a sequence reads its old length while one writes the new one
  const uintptr_t n0 = reinterpret_cast<uintptr_t>(new_context_lens), bytes = (uintptr_t)num_seqs * 4;
  struct Span { const void* p; uintptr_t n; };
  const Span ins[] = {{context_lens, bytes}, {accepted, bytes}, {query_starts, bytes + 4},
                      {block_tables, bytes * max_blocks_per_seq},
                      {context_lens_before, context_lens_before && context_lens_before != new_context_lens ? bytes : 0},
                      {tree_mask, tree_mask ? (uintptr_t)num_tokens * mask_words * 8 : 0}};
  for (const Span& q : ins) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(q.p);
    if (q.n && n0 < a + q.n && a < n0 + bytes) return PA_ERR_INVALID_ARG;
  }
  const int row_bytes = head_dim * esize(dtype);
  if (row_bytes % 16 || (tree_mask != nullptr && mask_words > kCommitMaxWords) ||
      (long long)max_blocks_per_seq * block_size > 0x7fffffffLL)
    return PA_ERR_UNSUPPORTED;
  CommitParams p{};
  p.block_tables = block_tables;
  p.max_blocks = max_blocks_per_seq;
  p.context_lens = context_lens;
  p.before = context_lens_before;
  p.query_starts = query_starts;
  p.tree_mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  p.words = mask_words;
  p.accepted = accepted;
  p.new_context_lens = new_context_lens;
  p.num_tokens = num_tokens;
  p.G = num_kv_heads;
  p.vpr = row_bytes / 16;
  p.B = block_size;
  p.nhd = layout == PA_LAYOUT_NHD;
  p.num_blocks = num_blocks;
  int sms = 0;
  const pa_status st = device_state(&p.err, &sms);
  if (st != PA_OK) return st;
  // drafts without branches have nothing to move: one layer's CTAs set the lengths
  const int layers = tree_mask ? num_layers : 1;
  for (int b = 0; b < layers; b += kCommitLayers) {
    const int nl = std::min(kCommitLayers, layers - b);
    CommitPtrs ptrs;
    for (int i = 0; i < kCommitLayers; ++i) {
      ptrs.k[i] = i < nl ? static_cast<uint4*>(k_caches[b + i]) : nullptr;
      ptrs.v[i] = i < nl ? static_cast<uint4*>(v_caches[b + i]) : nullptr;
    }
    // a layer per CTA up to 32 CTAs per SM (9 of them run at a time): a larger batch takes several layers per CTA and
    // finds its paths once for them (64 sequences x 32 layers, 27 CTAs per SM: 14.5 us at one layer per CTA, 15.2 at two)
    const long long all = (long long)num_seqs * nl * 2, target = (long long)sms * 16;
    p.layers = nl;
    p.layers_per_cta = (int)std::max(1LL, std::min<long long>(nl, all / target));
    const dim3 grid((unsigned)num_seqs, (unsigned)((nl + p.layers_per_cta - 1) / p.layers_per_cta), 2);
    if (launch_pdl(commit_tree_kernel, grid, dim3(kCommitThreads), 0, stream, ptrs, p) != cudaSuccess)
      return PA_ERR_CUDA;
  }
  return PA_OK;
}
