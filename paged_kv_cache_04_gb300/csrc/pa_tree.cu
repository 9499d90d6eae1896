// pa_decode_tree: argument checks, workspace layout and dispatch.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>
#include <mutex>

#include "pa_internal.h"
#include "pa_tree.cuh"
#include "pa_tree_tc.cuh"

namespace pa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool valid_dtype(pa_dtype dt) { return dt == PA_F32 || dt == PA_F16 || dt == PA_BF16; }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Rows of an item at most: the vector kernel takes 8 or 32. Batches of 3 to 7 rows a kv head took 18.6 us with 8 and
// 21.2 with 32 (idle rows still cost their warps' loops); above 8 rows, tiles of 8 would read the context once for each.
int vec_rows(int max_rows) { return max_rows <= 8 ? 8 : 32; }

// Rows that a call's items can have, as multiples of 8: the tensor-core kernel takes
// up to 256 (128 at head_dim 256).
int tc_rows(int max_rows, int D) { return std::min((max_rows + 7) / 8 * 8, D == 256 ? 128 : 256); }

// Workspace: the join records, then two partials per CTA.
size_t join_bytes() { return align256(kTreeMaxCtas * sizeof(TreeJoin)); }

template <typename OT, int D>
pa_status launch_join(const TreeParams& p, int grid, cudaStream_t stream) {
  const dim3 ctas(grid, (p.slot_rows + 31) / 32, D / 64);
  return launch_pdl(tree_join_kernel<OT, D>, ctas, dim3(kTreeJoinThreads), 0, stream, p) == cudaSuccess ? PA_OK
                                                                                                     : PA_ERR_CUDA;
}

template <int D, int RB>
pa_status launch_vec(TreeParams p, int sms, cudaStream_t stream) {
  auto kern = tree_vec_kernel<D, RB>;
  constexpr unsigned smem = tree_vec_smem<D, RB>();
  static std::mutex mu;
  static int per_sm[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_CUDA;
  int n;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (per_sm[dev] == 0) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
          cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, 256, smem) != cudaSuccess || n < 1)
        return PA_ERR_CUDA;
      per_sm[dev] = std::min(n, 2);
    }
    n = per_sm[dev];
  }
  p.tile_toks = RB / p.group;
  p.tile_shift = tree_vec_tokens<D>() == 64 ? 6 : 5;
  p.slot_rows = RB;
  p.item_units = 1;
  p.min_units = 1;
  const int grid = std::min(sms * n, kTreeMaxCtas);
  if (launch_pdl(kern, dim3(grid), dim3(256), smem, stream, p) != cudaSuccess) return PA_ERR_CUDA;
  return launch_join<float, D>(p, grid, stream);
}

template <typename DT, typename OT, int D, int QR>
pa_status launch_tc(TreeParams p, pa_dtype dt, int sms, cudaStream_t stream) {
  using C = TreeTc<D, QR>;
  auto kern = tree_tc_kernel<DT, OT, D, QR>;
  static std::mutex mu;
  static bool set[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!set[dev]) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::TOTAL) != cudaSuccess)
        return PA_ERR_CUDA;
      set[dev] = true;
    }
  }
  const int half_toks = QR / p.group;
  p.tile_toks = half_toks * (QR == 128 ? C::NS : 1);
  p.tile_shift = 6;
  static_assert(kTreeTile == 64, "tile_shift");
  p.slot_rows = tc_rows(p.max_tree * p.group, D);
  // An item's queries, checks and output cost about this many of its tiles (measured against 1: 128 us for 192 on 32
  // sequences x 40 kv heads of 5 rows, 118 for 132 on 64 x 8; at head_dim 256, whose tiles take longer, 53.5 for 54.1).
  p.item_units = D == 256 ? 2 : 6;
  // One sequence of 100 tokens: 12.4 us with shares of two tiles at least, 14.2 with one; no difference on long ones.
  p.min_units = 2;
  const pa_kv_layout layout = p.nhd ? PA_LAYOUT_NHD : PA_LAYOUT_HND;
  CUtensorMap km, vm, qm;
  pa_status s = make_pool_map_3d(&km, p.k_cache, dt, D, p.G, p.B, p.num_blocks, layout);
  if (s == PA_OK) s = make_pool_map_3d(&vm, p.v_cache, dt, D, p.G, p.B, p.num_blocks, layout);
  if (s == PA_OK) s = make_q_map(&qm, p.q, dt, D, p.H, p.N, p.group, half_toks);
  if (s != PA_OK) return s;
  const int grid = std::min(sms, kTreeTcCtas);
  if (launch_pdl(kern, dim3(grid), dim3(C::THREADS), C::TOTAL, stream, km, vm, qm, p) != cudaSuccess)
    return PA_ERR_CUDA;
  return launch_join<OT, D>(p, grid, stream);
}

// 16-bit caches take the tensor cores, fp32 ones the FMA units (a 16-bit product
// would lose what fp32 storage keeps).
template <typename DT, typename OT, int D>
pa_status launch_type(const TreeParams& p, pa_dtype dt, int sms, cudaStream_t stream) {
  if constexpr (sizeof(DT) == 2) {
    // Query tiles of 64 rows where every item fits: 32 x 40 kv heads of 5 rows, head_dim 128, 128.6 us for 137.6, and no
    // difference at head_dim 256. (At head_dim 64 the rings are as deep as they need to be with 128 rows.)
    if constexpr (D > 64) {
      if (p.max_tree <= 64 / p.group) return launch_tc<DT, OT, D, 64>(p, dt, sms, stream);
    }
    return launch_tc<DT, OT, D, 128>(p, dt, sms, stream);
  } else
    return vec_rows(p.max_tree * p.group) == 8 ? launch_vec<D, 8>(p, sms, stream)
                                               : launch_vec<D, 32>(p, sms, stream);
}

template <typename DT, typename OT>
pa_status launch_dim(const TreeParams& p, pa_dtype dt, int D, int sms, cudaStream_t stream) {
  switch (D) {
    case 64: return launch_type<DT, OT, 64>(p, dt, sms, stream);
    case 128: return launch_type<DT, OT, 128>(p, dt, sms, stream);
    default: return launch_type<DT, OT, 256>(p, dt, sms, stream);
  }
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_decode_tree_workspace_bytes(int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                                 int max_tree_tokens) {
  using namespace pa;
  if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || head_dim <= 0 ||
      max_tree_tokens <= 0 || max_tree_tokens > kTreeMaxTokens)
    return 0;
  const int rows = max_tree_tokens * (num_heads / num_kv_heads);
  // (the type decides which kernel runs; the size covers both)
  const size_t partials =
      std::max((size_t)kTreeMaxCtas * vec_rows(rows), (size_t)kTreeTcCtas * tc_rows(rows, head_dim)) * 2;
  return join_bytes() + align256(partials * (head_dim + 2) * 4);
}

extern "C" pa_status pa_decode_tree(void* out, const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* block_tables, int max_blocks_per_seq,
                                    const int32_t* context_lens, const int32_t* query_starts,
                                    const int64_t* tree_mask, int mask_words, int num_seqs, int num_tokens,
                                    int num_heads, int num_kv_heads, int head_dim, int block_size,
                                    pa_kv_layout layout, int64_t num_blocks, float scale, pa_dtype dtype,
                                    pa_dtype out_dtype, int max_tree_tokens, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
  using namespace pa;
  if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads ||
      head_dim <= 0 || block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || max_tree_tokens <= 0 ||
      !valid_dtype(dtype) || !valid_dtype(out_dtype) || !std::isfinite(scale) ||
      (layout != PA_LAYOUT_HND && layout != PA_LAYOUT_NHD) || (tree_mask != nullptr && mask_words <= 0))
    return PA_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_starts || !workspace)
    return PA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(workspace) ||
      (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
      (reinterpret_cast<uintptr_t>(query_starts) & 3u) || (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
    return PA_ERR_INVALID_ARG;
  const int group = num_heads / num_kv_heads;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || (block_size != 16 && block_size != 32) || group > 8 ||
      max_tree_tokens > kTreeMaxTokens || (out_dtype != dtype && out_dtype != PA_F32))
    return PA_ERR_UNSUPPORTED;
  if (tree_mask != nullptr && mask_words < (max_tree_tokens + 63) / 64) return PA_ERR_INVALID_ARG;
  // token positions, TMA row coordinates and the search for a share's first sequence are 32-bit; so are one sequence's
  // units
  if (num_seqs > kTreeMaxSeqs ||
      (long long)max_blocks_per_seq * block_size > 0x7fffffffLL - 64 ||
      (long long)num_blocks * num_kv_heads * block_size > 0x7fffffffLL ||
      (long long)num_kv_heads * max_tree_tokens * ((long long)max_blocks_per_seq * block_size / 32 + 8) > 0x7fffffffLL)
    return PA_ERR_UNSUPPORTED;
  const size_t need =
      pa_decode_tree_workspace_bytes(num_tokens, num_heads, num_kv_heads, head_dim, max_tree_tokens);
  if (need == 0 || workspace_bytes < need) return PA_ERR_INVALID_ARG;
  // rows and partials are written while other items' inputs still have to be read
  const auto esize = [](pa_dtype t) { return t == PA_F32 ? 4u : 2u; };
  const size_t elems = (size_t)num_tokens * num_heads * head_dim, out_bytes = elems * esize(out_dtype);
  const size_t pool = (size_t)num_blocks * num_kv_heads * block_size * head_dim * esize(dtype);
  struct Span { const void* p; size_t n; };
  const Span ins[] = {{q, elems * esize(dtype)}, {k_cache, pool}, {v_cache, pool},
                      {block_tables, (size_t)num_seqs * max_blocks_per_seq * 4}, {context_lens, (size_t)num_seqs * 4},
                      {query_starts, (size_t)num_seqs * 4 + 4},
                      {tree_mask, tree_mask ? (size_t)num_tokens * mask_words * 8 : 0}};
  for (const Span& x : ins)
    if (x.n && (overlap(out, out_bytes, x.p, x.n) || overlap(workspace, need, x.p, x.n))) return PA_ERR_INVALID_ARG;
  if (overlap(out, out_bytes, workspace, need)) return PA_ERR_INVALID_ARG;
  TreeParams p{};
  p.out = out;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.max_blocks = max_blocks_per_seq;
  p.context_lens = context_lens;
  p.query_starts = query_starts;
  p.mask = reinterpret_cast<const unsigned long long*>(tree_mask);
  p.words = mask_words;
  p.S = num_seqs;
  p.N = num_tokens;
  p.H = num_heads;
  p.G = num_kv_heads;
  p.group = group;
  p.B = block_size;
  p.block_shift = block_size == 32 ? 5 : 4;
  p.nhd = layout == PA_LAYOUT_NHD;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * 1.4426950408889634f;
  // Masked scores are infinities times the scale, so a scale of zero becomes the smallest number above it (2^-149): the
  // largest finite score, 2^128, times that is 2^-21, which moves no weight by more than 2^-21.
  if (p.scale_log2 == 0.f) p.scale_log2 = std::numeric_limits<float>::denorm_min();
  p.max_tree = max_tree_tokens;
  p.join = static_cast<TreeJoin*>(workspace);
  p.ws = reinterpret_cast<float*>(static_cast<char*>(workspace) + join_bytes());
  int sms = 0;
  const pa_status s = device_state(&p.err, &sms);
  if (s != PA_OK) return s;
  switch (dtype) {
    case PA_BF16:
      return out_dtype == PA_F32 ? launch_dim<__nv_bfloat16, float>(p, dtype, head_dim, sms, stream)
                                 : launch_dim<__nv_bfloat16, __nv_bfloat16>(p, dtype, head_dim, sms, stream);
    case PA_F16:
      return out_dtype == PA_F32 ? launch_dim<__half, float>(p, dtype, head_dim, sms, stream)
                                 : launch_dim<__half, __half>(p, dtype, head_dim, sms, stream);
    default: return launch_dim<float, float>(p, dtype, head_dim, sms, stream);
  }
}
