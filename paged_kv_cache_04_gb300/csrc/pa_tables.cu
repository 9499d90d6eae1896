// pa_build_tables: the metadata of one step, built on the GPU from the lengths of
// its requests -- what the block manager's on-demand allocation does on the host
// (CS349E Lecture 7 notes, §4.1: a sequence gets a new block only when its last
// one is full) for a whole batch in one launch.
//
// For sequence s with c cached tokens, h blocks in its table row and n new tokens:
//   want = ceil((c + n) / B),  need = max(0, want - h)
//   its blocks  free_blocks[f + sum_{r<s} need_r ..]      (f: the list's first free entry)
//   its tokens  query_starts[s] = sum_{r<s} n_r
//   token i     position c + i, slot table[(c + i) / B] * B + (c + i) % B
// and, with a tree's parents, the ancestors of every node as a row of bits.
//
// The work is a few bytes per token behind two prefix sums, so the call is bound
// by latency: every CTA computes both sums over the whole batch by itself (the
// lengths are a few KB, in L2 after the first CTA) instead of waiting for a
// scan kernel, then takes its share of the tokens and table entries. A batch
// entry's table row and the free list are read directly, so no CTA reads what
// another writes.
#include <algorithm>
#include <cstdint>
#include <mutex>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kBuildThreads = 512;
constexpr int kBuildMaxSeqs = 4096;   // a batch's starts, bases and lengths sit in shared memory (64 KB)
constexpr int kBuildMaxWords = 4;     // trees of up to 256 nodes
constexpr int kBuildReach = 64 * kBuildMaxWords;

struct BuildParams {
  int32_t* block_tables;
  int max_blocks;
  int32_t *table_lens_out, *context_lens_out, *query_starts;
  int64_t* slot_mapping;
  int32_t *positions, *free_first_out;
  const int32_t *table_lens, *context_lens, *new_lens, *free_blocks, *free_first;
  int num_free;
  const int32_t* parents;
  unsigned long long* tree_mask;
  int words;
  int S, max_tokens, B;
  long long num_blocks;
  unsigned* err;
};

// A batch entry's numbers, with values outside their ranges replaced by the nearest
// valid one (the caller records them).
struct BuildSeq {
  int ctx, held, fresh;
  long long want;
  int need;       // blocks to take from the list
  unsigned err;
};

__device__ __forceinline__ BuildSeq build_seq(const BuildParams& p, int s) {
  BuildSeq q;
  q.ctx = __ldg(p.context_lens + s);
  q.held = __ldg(p.table_lens + s);
  q.fresh = __ldg(p.new_lens + s);
  q.err = 0;
  if (q.ctx < 0 || q.fresh < 0 || q.held < 0 || q.held > p.max_blocks) q.err = kErrContext;
  q.ctx = max(q.ctx, 0);
  q.fresh = max(q.fresh, 0);
  q.held = min(max(q.held, 0), p.max_blocks);
  q.want = ((long long)q.ctx + q.fresh + p.B - 1) / p.B;
  q.need = 0;
  // a row too short for the sequence (or a length past 32 bits): nothing is taken for it
  if ((long long)q.ctx + q.fresh > 0x7fffffffLL) q.want = (long long)p.max_blocks + 1;
  if (q.want > p.max_blocks) q.err |= kErrContext;
  else if (q.want > q.held) q.need = (int)q.want - q.held;
  return q;
}

__device__ __forceinline__ long long warp_incl(long long x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += v;
  }
  return x;
}

// The last index i in [0, n) with a[i] <= x (a non-decreasing, a[0] <= x).
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// TPT consecutive tokens per thread: 1, or 4 where there are enough tokens to fill
// the GPU (one search then serves four tokens: 512 prompt chunks, 525k tokens, 10.7 us
// for 12.4). In a graph: 6.3 us for 256 sequences with a token each, 9.2 for 64 trees
// of 9 to 32 nodes (the walks up the parents), of which a launch is about 3.
template <int TPT>
__global__ void __launch_bounds__(kBuildThreads) build_tables_kernel(const BuildParams p) {
  pdl_begin();
  extern __shared__ int build_smem[];
  int* starts = build_smem;              // [S + 1] first token of each sequence
  int* base = starts + p.S + 1;          // [S + 1] its first free-list entry, as an offset
  int* ctxs = base + p.S + 1;            // [S]
  int* helds = ctxs + p.S;               // [S] blocks held, ~ of it where the sequence is not served
  int* par = helds + p.S;                // [kBuildReach + kBuildThreads] parents of the nodes at hand
  __shared__ long long wsum[2][kBuildThreads / 32];
  __shared__ int taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool lead = blockIdx.x == 0;

  // both exclusive sums; each thread takes a run of consecutive sequences
  const int per = (p.S + kBuildThreads - 1) / kBuildThreads;
  const int b = min(p.S, tid * per), e = min(p.S, b + per);
  const int first = __ldg(p.free_first);
  long long tok = 0, blk = 0;
  unsigned bad = 0;
  BuildSeq q;
  for (int s = b; s < e; ++s) {
    q = build_seq(p, s);
    tok += q.fresh;
    blk += q.need;
    bad |= q.err;
  }
  const bool first_ok = first >= 0 && first <= p.num_free;
  const int avail = first_ok ? p.num_free - first : 0;
  if (lead && tid == 0 && !first_ok) atomicOr(p.err, kErrNoBlocks);
  const long long ti = warp_incl(tok, lane), bi = warp_incl(blk, lane);
  if (lane == 31) {
    wsum[0][warp] = ti;
    wsum[1][warp] = bi;
  }
  if (tid == 0) taken = 0;
  __syncthreads();
  long long t0 = ti - tok, b0 = bi - blk, total = 0;
  for (int w = 0; w < kBuildThreads / 32; ++w) {
    if (w < warp) {
      t0 += wsum[0][w];
      b0 += wsum[1][w];
    }
    total += wsum[0][w];
  }
  // A sequence is served when its blocks lie in the list and its tokens in the
  // arrays. An unserved one takes nothing: no entry, slots of -1, a context of 0.
  // (Both sums count it, so what lies behind it in the list or the arrays is out of
  // reach for it and for all that follow it and need any.)
  for (int s = b; s < e; ++s) {
    if (per > 1) q = build_seq(p, s);
    const bool fits = q.fresh == 0 || t0 + q.fresh <= p.max_tokens;
    const bool blocks = q.need == 0 || b0 + q.need <= avail;
    const bool ok = fits && blocks && q.want <= p.max_blocks;
    starts[s] = (int)min(t0, (long long)p.max_tokens);
    base[s] = (int)min(b0, (long long)avail);
    ctxs[s] = q.ctx;
    helds[s] = ok ? q.held : ~q.held;
    if (!fits) bad |= kErrQuery;
    if (!blocks) bad |= kErrNoBlocks;
    if (ok && q.need > 0) atomicMax(&taken, (int)b0 + q.need);
    if (lead) {
      p.table_lens_out[s] = ok ? max(q.held, (int)q.want) : q.held;
      p.context_lens_out[s] = ok ? q.ctx + q.fresh : 0;
      p.query_starts[s] = starts[s];
    }
    t0 += q.fresh;
    b0 += q.need;
  }
  const int tokens = (int)min(total, (long long)p.max_tokens);
  if (tid == 0) starts[p.S] = tokens;
  if (lead && bad) atomicOr(p.err, bad);
  __syncthreads();
  if (lead && tid == 0) {
    p.query_starts[p.S] = tokens;
    *p.free_first_out = first_ok ? first + taken : first;
  }

  // table growth: a thread per list entry
  for (int k = (int)blockIdx.x * kBuildThreads + tid; k < taken; k += (int)gridDim.x * kBuildThreads) {
    const int s = last_at_most(base, p.S, k);
    if (helds[s] < 0) continue;
    int id = __ldg(p.free_blocks + first + k);
    if (id < 0 || id >= p.num_blocks) {
      atomicOr(p.err, kErrBlockId);
      id = -1;
    }
    p.block_tables[(long long)s * p.max_blocks + helds[s] + (k - base[s])] = id;
  }

  // tokens
  const long long step = (long long)kBuildThreads * TPT;
  for (long long c0 = (long long)blockIdx.x * step; c0 < p.max_tokens; c0 += (long long)gridDim.x * step) {
    if (TPT == 1 && p.parents != nullptr) {  // the nodes of this pass and all their possible ancestors
      __syncthreads();
      for (int k = tid; k < kBuildReach + kBuildThreads; k += kBuildThreads) {
        const long long n = c0 - kBuildReach + k;
        par[k] = n >= 0 && n < tokens ? __ldg(p.parents + n) : -1;
      }
      __syncthreads();
    }
    const long long n0 = c0 + tid * TPT;
    int s = n0 < tokens ? last_at_most(starts, p.S, (int)n0) : 0;
#pragma unroll
    for (int u = 0; u < TPT; ++u) {
      const long long n = n0 + u;
      if (n >= p.max_tokens) continue;
      if (n >= tokens) {  // behind the last sequence: padding that the cache write skips
        p.slot_mapping[n] = -1;
        p.positions[n] = 0;
        if (p.parents != nullptr)
          for (int w = 0; w < p.words; ++w) p.tree_mask[n * p.words + w] = 0;
        continue;
      }
      if (TPT > 1)
        while (n >= starts[s + 1]) ++s;
      const int i = (int)n - starts[s], held = helds[s];
      const long long pos = (long long)ctxs[s] + i;
      long long slot = -1;
      if (held >= 0) {
        const int at = pos <= 0x7fffffffLL ? (int)pos / p.B : (int)(pos / p.B);
        const int id = at < held ? __ldg(p.block_tables + (long long)s * p.max_blocks + at)
                                 : __ldg(p.free_blocks + first + base[s] + (at - held));
        if (id >= 0 && id < p.num_blocks) slot = (long long)id * p.B + (pos - (long long)at * p.B);
        else atomicOr(p.err, kErrBlockId);
      }
      p.slot_mapping[n] = slot;
      int where = (int)min(pos, 0x7fffffffLL);
      if (TPT == 1 && p.parents != nullptr) {
        unsigned long long bits[kBuildMaxWords] = {0, 0, 0, 0};
        unsigned wrong = 0;
        if (__ldg(p.new_lens + s) > 64 * p.words) {
          wrong = kErrQuery;  // more nodes than a row has bits: no bits
        } else {
          // up the parents; each is below its child, so the walk ends
          const int* mine = par + kBuildReach + tid - i;  // mine[j]: parent of node j
          int depth = 0;
          for (int j = i; j >= 0; ++depth) {
#pragma unroll
            for (int w = 0; w < kBuildMaxWords; ++w)
              if (w == (j >> 6)) bits[w] |= 1ull << (j & 63);
            int up = mine[j];
            if (up < -1 || up >= j) {
              wrong = kErrQuery;
              up = -1;
            }
            j = up;
          }
          where = (int)min((long long)ctxs[s] + depth - 1, 0x7fffffffLL);
        }
        if (wrong) atomicOr(p.err, wrong);
#pragma unroll
        for (int w = 0; w < kBuildMaxWords; ++w)
          if (w < p.words) p.tree_mask[n * p.words + w] = bits[w];
      }
      p.positions[n] = where;
    }
  }
}

// Shared memory above 48 KB (batches of more than about 2,800 sequences) is opted into once per device.
template <int TPT>
pa_status launch_build(const BuildParams& p, unsigned grid, size_t smem, cudaStream_t stream) {
  constexpr size_t most = ((size_t)4 * kBuildMaxSeqs + 2 + kBuildReach + kBuildThreads) * 4;
  static std::mutex mu;
  static bool set[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set[dev]) {
      if (cudaFuncSetAttribute(build_tables_kernel<TPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) !=
          cudaSuccess)
        return PA_ERR_CUDA;
      set[dev] = true;
    }
  }
  return launch_pdl(build_tables_kernel<TPT>, dim3(grid), dim3(kBuildThreads), smem, stream, p) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace
}  // namespace pa

extern "C" pa_status pa_build_tables(int32_t* block_tables, int max_blocks_per_seq, int32_t* table_lens_out,
                                     int32_t* context_lens_out, int32_t* query_starts, int64_t* slot_mapping,
                                     int32_t* positions, int32_t* free_first_out, const int32_t* table_lens,
                                     const int32_t* context_lens, const int32_t* new_lens,
                                     const int32_t* free_blocks, int num_free, const int32_t* free_first,
                                     const int32_t* parents, int64_t* tree_mask, int mask_words, int num_seqs,
                                     int max_tokens, int block_size, int64_t num_blocks, cudaStream_t stream) {
  using namespace pa;
  if (num_seqs < 0 || max_tokens < 0 || num_free < 0 || max_blocks_per_seq <= 0 || block_size <= 0 ||
      num_blocks <= 0)
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0) return PA_OK;
  if (!block_tables || !table_lens_out || !context_lens_out || !query_starts || !free_first_out || !table_lens ||
      !context_lens || !new_lens || !free_first || (num_free > 0 && !free_blocks) ||
      (max_tokens > 0 && (!slot_mapping || !positions)))
    return PA_ERR_INVALID_ARG;
  const void* words4[] = {block_tables, table_lens_out, context_lens_out, query_starts, positions, free_first_out,
                          table_lens,   context_lens,   new_lens,         free_blocks,  free_first, parents};
  for (const void* q : words4)
    if (reinterpret_cast<uintptr_t>(q) & 3u) return PA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(slot_mapping) & 7u) || (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
    return PA_ERR_INVALID_ARG;
  if ((parents != nullptr) != (tree_mask != nullptr) || (parents != nullptr && mask_words <= 0))
    return PA_ERR_INVALID_ARG;
  if (num_seqs > kBuildMaxSeqs || num_blocks > 0x7fffffffLL || (parents != nullptr && mask_words > kBuildMaxWords))
    return PA_ERR_UNSUPPORTED;
  // Every CTA reads all the lengths while the first one writes the new ones: no
  // output may lie on an input, or on another output.
  const size_t n4 = (size_t)num_seqs * 4;
  struct Span { const void* p; size_t n; };
  const Span outs[] = {{block_tables, n4 * max_blocks_per_seq}, {table_lens_out, n4}, {context_lens_out, n4},
                       {query_starts, n4 + 4}, {slot_mapping, (size_t)max_tokens * 8},
                       {positions, (size_t)max_tokens * 4}, {free_first_out, 4},
                       {tree_mask, parents ? (size_t)max_tokens * mask_words * 8 : 0}};
  const Span ins[] = {{table_lens, n4}, {context_lens, n4}, {new_lens, n4}, {free_blocks, (size_t)num_free * 4},
                      {free_first, 4}, {parents, parents ? (size_t)max_tokens * 4 : 0}};
  for (size_t i = 0; i < sizeof(outs) / sizeof(outs[0]); ++i) {
    if (outs[i].n == 0) continue;
    for (const Span& q : ins)
      if (q.n && overlap(outs[i].p, outs[i].n, q.p, q.n)) return PA_ERR_INVALID_ARG;
    for (size_t j = 0; j < i; ++j)
      if (outs[j].n && overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return PA_ERR_INVALID_ARG;
  }
  BuildParams p{};
  p.block_tables = block_tables;
  p.max_blocks = max_blocks_per_seq;
  p.table_lens_out = table_lens_out;
  p.context_lens_out = context_lens_out;
  p.query_starts = query_starts;
  p.slot_mapping = slot_mapping;
  p.positions = positions;
  p.free_first_out = free_first_out;
  p.table_lens = table_lens;
  p.context_lens = context_lens;
  p.new_lens = new_lens;
  p.free_blocks = free_blocks;
  p.free_first = free_first;
  p.num_free = num_free;
  p.parents = parents;
  p.tree_mask = reinterpret_cast<unsigned long long*>(tree_mask);
  p.words = mask_words;
  p.S = num_seqs;
  p.max_tokens = max_tokens;
  p.B = block_size;
  p.num_blocks = num_blocks;
  int sms = 0;
  const pa_status st = device_state(&p.err, &sms);
  if (st != PA_OK) return st;
  // One token per thread while the threads of one CTA per SM are enough (a small step is one CTA), then four.
  const bool many = parents == nullptr && (long long)max_tokens > (long long)sms * kBuildThreads;
  const long long step = (long long)kBuildThreads * (many ? 4 : 1);
  const long long want = std::max<long long>(((long long)max_tokens + step - 1) / step, 1);
  const unsigned grid = (unsigned)std::min<long long>(want, (long long)sms * 2);
  const size_t smem = ((size_t)4 * num_seqs + 2 + kBuildReach + kBuildThreads) * 4;
  return many ? launch_build<4>(p, grid, smem, stream) : launch_build<1>(p, grid, smem, stream);
}
