// Attention of drafted tokens (trees or chains) over the paged cache.
//
// What is computed: node i of sequence s, query head h, kv head kv = h / group,
// with c cached tokens in front of the n drafted ones,
//     out = sum_t softmax_t(scale * q . K[t]) V[t]   over t < c and t = c + j for
//                                                     the nodes j that i attends
// (the attention of decode, CS349E Lecture 7 notes §4.2, with more rows per
// sequence and a mask at the end of the context).
//
// Work: the rows of one (sequence, kv head), node x query head, share every K and
// V row, so they are taken together in tiles of up to a few hundred rows; an item
// is (sequence, kv head, row tile) over the context's token tiles. The items'
// token tiles, one behind the other, are one long line of units that is cut into
// as many equal shares as there are CTAs: every CTA streams the same number of
// bytes whatever the lengths and the batch, and at most its first and last items
// are not its alone. Those leave (max, sum, unnormalised output) of their share in
// the workspace, and a second small kernel joins them, in the order of the CTAs
// (attention over a context is the merge of attention over any split of it, CMU
// 15-779 Lecture 16 notes §3.3).
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr int kTreeMaxTokens = 256;   // drafted tokens of one sequence
constexpr int kTreeMaxSeqs = 1 << 24;
constexpr int kTreeMaxCtas = 320;     // shares of a call (workspace slots): two CTAs per SM of the vector kernel,
constexpr int kTreeTcCtas = 160;      // one of the tensor-core kernel
// What the joining kernel has to know of an item whose shares start in CTA c.
struct TreeJoin {
  int last;        // its last CTA; -1: CTA c starts no such item
  int q0;          // its first token's row in q
  int rows;        // token x query head
  int kv;
};

struct TreeParams {
  void* out;
  const void *q, *k_cache, *v_cache;
  const int32_t* block_tables;
  int max_blocks;
  const int32_t *context_lens, *query_starts;
  const unsigned long long* mask;  // null: chains
  int words;
  int S, N, H, G, group;
  int B, block_shift, nhd;
  long long num_blocks;
  float scale_log2;
  int max_tree;
  int tile_toks;    // nodes of an item at most
  int tile_shift;   // log2 of a unit's context tokens
  int item_units;   // units of an item besides its token tiles
  int min_units;    // a share's units at least (fewer CTAs work when there are fewer)
  TreeJoin* join;   // [gridDim.x]
  float* ws;        // [gridDim.x][2] partials: float2 ml[slot_rows], float4 o[D / 4][slot_rows]
  int slot_rows;
  unsigned* err;
};

struct TreeSeq {
  int q0, n, ctx, tiles, row_tiles;
};

// What the call's arrays say about sequence s.
struct TreeRaw {
  int a, b, c;
};
__device__ __forceinline__ TreeRaw tree_raw(const TreeParams& p, int s) {
  return {__ldg(p.query_starts + s), __ldg(p.query_starts + s + 1), __ldg(p.context_lens + s)};
}

// The sequence as the kernels take it; errors are recorded where `report`.
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, const TreeRaw& raw, bool report) {
  TreeSeq t;
  int c = raw.c;
  unsigned bad = 0;
  const long long room = (long long)p.max_blocks * p.B;
  if (c < 0 || c > room) {
    bad |= kErrContext;
    c = c < 0 ? 0 : (int)room;
  }
  t.q0 = raw.a;
  t.n = (int)((unsigned)raw.b - (unsigned)raw.a);
  t.ctx = c;
  // (without a context any number of nodes: an unserved prompt's rows are zeros, from items of one tile that reads nothing)
  if (raw.a < 0 || raw.b < raw.a || raw.b > p.N || (c > 0 && (t.n > p.max_tree || t.n > c))) {
    bad |= kErrQuery;
    t.n = 0;
  }
  if (report && bad) atomicOr(p.err, bad);
  t.tiles = max(1, (c + (1 << p.tile_shift) - 1) >> p.tile_shift);
  t.row_tiles = (t.n + p.tile_toks - 1) / p.tile_toks;
  return t;
}

// A CTA's share of an item: token tiles [tile0, tile1) of `tiles`.
struct TreeItem {
  int s, kv, q0, tok0, rows;  // tok0: the row tile's first node; q0: its row in q
  int ctx, prefix;            // prefix: tokens in front of the drafted ones
  int tile0, tile1, tiles;
  long long end;              // one past the item's last unit
};

// The walk over a CTA's share of the units; every warp of the CTA does the same.
struct TreeWalk {
  int s, kv, rt, w;  // sequence, kv head, row tile, unit within the item
  TreeSeq t;         // sequence s
  TreeRaw ahead;     // what is said about sequence s + 1, loaded an item or more before it is needed
  long long pos;     // absolute unit
  long long left;    // units of the share not yet walked
  long long size;    // units of a share; the first `extra` shares have one more
  int extra;

  __device__ __forceinline__ bool next(const TreeParams& p, TreeItem& it) {
    while (left > 0) {
      if (kv == p.G || t.row_tiles == 0) {
        if (++s >= p.S) return false;
        t = tree_seq(p, ahead, false);
        if (s + 1 < p.S) ahead = tree_raw(p, s + 1);
        kv = 0;
        continue;
      }
      const int per = t.tiles + p.item_units;
      const int take = (int)min((long long)(per - w), left);
      it.tile0 = max(0, w - p.item_units);
      it.tile1 = max(0, w + take - p.item_units);
      it.s = s;
      it.kv = kv;
      it.tok0 = rt * p.tile_toks;
      it.q0 = t.q0 + it.tok0;
      it.rows = min(p.tile_toks, t.n - it.tok0) * p.group;
      it.ctx = t.ctx;
      it.prefix = max(0, t.ctx - t.n);
      it.tiles = t.tiles;
      it.end = pos - w + per;
      pos += take;
      left -= take;
      w += take;
      if (w == per) {
        w = 0;
        if (++rt == t.row_tiles) {
          rt = 0;
          ++kv;
        }
      }
      if (it.tile0 != it.tile1) return true;  // (else none of the item's tiles fall into this share)
    }
    return false;
  }
  // CTA of an item's last unit
  __device__ __forceinline__ int last_cta(const TreeItem& it) const {
    const long long x = it.end - 1, longer = extra * (size + 1);
    return (int)(x < longer ? x / (size + 1) : extra + (x - longer) / size);
  }
};

// Find this CTA's share. THREADS threads take part; `scratch` holds THREADS / 32 + 3
// long longs of shared memory. Ends with a barrier.
template <int THREADS>
__device__ __forceinline__ TreeWalk tree_share(const TreeParams& p, long long* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int WARPS = THREADS / 32;
  const int per = (p.S + THREADS - 1) / THREADS;
  const int b = min(p.S, tid * per), e = min(p.S, b + per);
  auto units_of = [&](const TreeSeq& t) { return (long long)p.G * t.row_tiles * (t.tiles + p.item_units); };
  long long mine = 0;
  TreeSeq t;
  for (int s = b; s < e; ++s) {
    t = tree_seq(p, tree_raw(p, s), blockIdx.x == 0);
    mine += units_of(t);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  static_assert(WARPS <= 32, "one lane per warp");
  const long long sum = lane < WARPS ? scratch[lane] : 0;
  long long upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  const long long before = incl - mine + __shfl_sync(0xffffffffu, upto - sum, warp);
  const long long total = __shfl_sync(0xffffffffu, upto, 31);
  TreeWalk k;
  int ctas = (int)gridDim.x;
  if (total < (long long)ctas * p.min_units) ctas = (int)max(1LL, total / p.min_units);
  k.size = total <= 0xffffffffLL ? (uint32_t)total / (uint32_t)ctas : total / ctas;
  k.extra = (int)(total - k.size * ctas);
  const int c = blockIdx.x;
  const long long u0 = c < ctas ? c * k.size + min(c, k.extra) : total;
  const long long u1 = c < ctas ? u0 + k.size + (c < k.extra ? 1 : 0) : total;
  if (u0 < u1 && u0 >= before && u0 < before + mine) {  // this thread's sequences hold the share's first unit
    long long at = before;
    for (int s = b; s < e; ++s) {
      if (per > 1) t = tree_seq(p, tree_raw(p, s), false);
      if (u0 < at + units_of(t)) {
        scratch[WARPS] = s;
        scratch[WARPS + 1] = u0 - at;
        break;
      }
      at += units_of(t);
    }
  }
  __syncthreads();
  k.pos = u0;
  k.left = u1 - u0;
  k.s = k.kv = k.rt = k.w = 0;
  k.t = TreeSeq{0, 0, 0, 1, 0};
  k.ahead = TreeRaw{0, 0, 0};
  if (k.left > 0) {
    k.s = (int)scratch[WARPS];
    k.t = tree_seq(p, tree_raw(p, k.s), false);
    if (k.s + 1 < p.S) k.ahead = tree_raw(p, k.s + 1);
    const long long off = scratch[WARPS + 1];
    const int per = k.t.tiles + p.item_units;
    // (with a context the units of a sequence fit 31 bits, see the host's checks)
    const int idx = off <= 0x7fffffffLL ? (int)off / per : (int)(off / per);
    k.w = (int)(off - (long long)idx * per);
    k.kv = idx / k.t.row_tiles;
    k.rt = idx - k.kv * k.t.row_tiles;
  }
  return k;
}

// Which of the 64 tokens from offset j (relative to the first drafted token, possibly
// negative) on node `node` (row q0 + node of the batch: `row`) attends: cached
// tokens all, drafted ones by the mask. Bits past the drafted tokens are not
// cleared here (the caller knows the context's end).
__device__ __forceinline__ unsigned long long tree_window(const TreeParams& p, long long row, int node, int j) {
  if (j <= -64) return ~0ull;
  auto word = [&](int w) -> unsigned long long {  // nodes 64 w .. 64 w + 63
    if (p.mask != nullptr) return w < p.words ? __ldg(p.mask + row * p.words + w) : 0ull;
    const int last = node - 64 * w;
    return last >= 63 ? ~0ull : (last < 0 ? 0ull : (2ull << last) - 1);
  };
  if (j < 0) return (word(0) << -j) | ((1ull << -j) - 1);
  const int w = j >> 6, r = j & 63;
  return r == 0 ? word(w) : (word(w) >> r) | (word(w + 1) << (64 - r));
}

// Bring a mask row close: it is read at an item's end, where nothing else would hide a trip to memory.
__device__ __forceinline__ void tree_mask_touch(const TreeParams& p, long long row) {
  if (p.mask != nullptr) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.mask + row * p.words));
}

// A partial's place in the workspace.
template <int D>
__device__ __forceinline__ float* tree_slot(const TreeParams& p, int cta, int which) {
  return p.ws + ((long long)cta * 2 + which) * p.slot_rows * (D + 2);
}

// The element offset of token t's row (kv head kv) in block `phys`.
template <int D>
__device__ __forceinline__ long long tree_row(const TreeParams& p, long long phys, int kv, int t) {
  const int r = t & (p.B - 1);
  return p.nhd ? ((phys * p.B + r) * p.G + kv) * D : ((phys * p.G + kv) * p.B + r) * D;
}

// ---------------------------------------------------------------------------------
// The vector kernel: fp32 caches, arithmetic on the FMA units (a 16-bit product would
// lose what fp32 storage keeps).
//
// Eight warps, each with RB / 8 rows of the item: a tile of K and V (NT tokens) is
// staged in shared memory for all of them; a warp computes its rows'
// scores with lane = token, keeps the running maximum and sum of each row, and
// accumulates the output with lane = D / 32 columns. Nothing passes between the
// warps but the staged tile. 8 sequences of 33 to 1,500 tokens, 4 heads of 64, 3 to 7
// nodes (12.7 MB): 18.6 us in a graph, 12 of them this kernel (a launch, the search for
// the share, one or two tiles: latency), the rest the joining kernel.
// ---------------------------------------------------------------------------------
template <int D>
__host__ __device__ constexpr int tree_vec_tokens() { return D == 256 ? 32 : 64; }

template <int D, int RB>
__host__ __device__ constexpr unsigned tree_vec_smem() {
  constexpr int NT = tree_vec_tokens<D>();
  return (RB * D + 2 * NT * (D + 4) + 2 * NT * D + RB * NT) * 4;
}

template <int D, int RB>
__global__ void __launch_bounds__(256) tree_vec_kernel(const TreeParams p) {
  pdl_begin();
  constexpr int NT = tree_vec_tokens<D>(), RW = RB / 8, TL = NT / 32, CV = D / 32, KP = D + 4;
  extern __shared__ __align__(16) float tree_smem[];
  float* Qs = tree_smem;             // [RB][D]
  float* Ks = Qs + RB * D;           // [2][NT][KP]  (padded: lanes read one row each)
  float* Vs = Ks + 2 * NT * KP;      // [2][NT][D]
  float* Ps = Vs + 2 * NT * D;       // [RB][NT]
  __shared__ long long scratch[8 + 3];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float NEG_INF = -__int_as_float(0x7f800000);
  if (tid == 0) p.join[blockIdx.x].last = -1;
  TreeWalk walk = tree_share<256>(p, scratch);
  const float* kc = static_cast<const float*>(p.k_cache);
  const float* vc = static_cast<const float*>(p.v_cache);

  TreeItem it;
  while (walk.next(p, it)) {
    const int32_t* table = p.block_tables + (long long)it.s * p.max_blocks;
    auto block_of = [&](int t) -> long long {  // -1: past the context or outside the pool
      if (t >= it.ctx) return -1;
      const int id = __ldg(table + (t >> p.block_shift));
      return id >= 0 && id < p.num_blocks ? id : -1;
    };
    auto stage = [&](int tile, int buf) {  // K and V rows of a tile; rows that are not there are zeros
      float* kd = Ks + buf * NT * KP;
      float* vd = Vs + buf * NT * D;
      for (int i = tid; i < NT * (D / 4); i += 256) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4, t = tile * NT + r;
        const long long phys = block_of(t);
        if (c == 0 && phys < 0 && t < it.ctx) atomicOr(p.err, kErrBlockId);
        const long long at = phys >= 0 ? tree_row<D>(p, phys, it.kv, t) + c : 0;
        if (phys >= 0) {
          cp_async16(kd + r * KP + c, kc + at);
          cp_async16(vd + r * D + c, vc + at);
        } else {
          *reinterpret_cast<float4*>(kd + r * KP + c) = make_float4(0.f, 0.f, 0.f, 0.f);
          *reinterpret_cast<float4*>(vd + r * D + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      cp_async_commit();
    };
    __syncthreads();  // the last item's tiles have been read
    stage(it.tile0, 0);
    for (int i = tid; i < RB * D; i += 256) {
      const int r = i / D, c = i % D;
      float x = 0.f;
      if (r < it.rows)
        x = static_cast<const float*>(p.q)[((long long)(it.q0 + r / p.group) * p.H + it.kv * p.group + r % p.group) * D + c];
      Qs[i] = x;
    }
    float m[RW], l[RW], acc[RW][CV];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      m[r] = NEG_INF;
      l[r] = 0.f;
#pragma unroll
      for (int c = 0; c < CV; ++c) acc[r][c] = 0.f;
    }
    for (int tile = it.tile0; tile < it.tile1; ++tile) {
      const int buf = (tile - it.tile0) & 1;
      cp_async_wait_all();
      __syncthreads();  // this tile (and the queries) are staged; the last one has been read
      if (tile + 1 < it.tile1) stage(tile + 1, buf ^ 1);
      if (warp * RW < it.rows) {
        const float* kd = Ks + buf * NT * KP;
        const float* vd = Vs + buf * NT * D;
        const int t0 = tile * NT;
        // scores: this lane's tokens lane and (NT = 64) lane + 32, this warp's rows
        float z[RW][TL];
#pragma unroll
        for (int r = 0; r < RW; ++r)
#pragma unroll
          for (int u = 0; u < TL; ++u) z[r][u] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
          float4 k[TL];
#pragma unroll
          for (int u = 0; u < TL; ++u) k[u] = *reinterpret_cast<const float4*>(kd + (lane + 32 * u) * KP + c);
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const float4 q = *reinterpret_cast<const float4*>(Qs + (warp * RW + r) * D + c);
#pragma unroll
            for (int u = 0; u < TL; ++u)
              z[r][u] = fmaf(q.w, k[u].w, fmaf(q.z, k[u].z, fmaf(q.y, k[u].y, fmaf(q.x, k[u].x, z[r][u]))));
          }
        }
        const bool masked = t0 + NT > it.prefix;  // drafted tokens or the context's end lie in the tile
        bool there[TL];
#pragma unroll
        for (int u = 0; u < TL; ++u) there[u] = block_of(t0 + lane + 32 * u) >= 0;
#pragma unroll
        for (int r = 0; r < RW; ++r) {
          const int row = warp * RW + r;
          unsigned long long seen = ~0ull;
          if (masked && row < it.rows) {
            const int node = row / p.group;
            seen = tree_window(p, it.q0 + node, it.tok0 + node, t0 - it.prefix);
          }
          float mx = NEG_INF;
#pragma unroll
          for (int u = 0; u < TL; ++u) {
            const bool on = there[u] && ((seen >> (lane + 32 * u)) & 1);
            z[r][u] = on ? z[r][u] * p.scale_log2 : NEG_INF;
            mx = fmaxf(mx, z[r][u]);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float mn = fmaxf(m[r], mx);
          const float ref = mn == NEG_INF ? 0.f : mn;
          const float f = m[r] == mn ? 1.f : exp2f(m[r] - ref);
          m[r] = mn;
          l[r] *= f;
#pragma unroll
          for (int c = 0; c < CV; ++c) acc[r][c] *= f;
#pragma unroll
          for (int u = 0; u < TL; ++u) {
            const float w = exp2f(z[r][u] - ref);
            l[r] += w;
            Ps[row * NT + lane + 32 * u] = w;
          }
        }
        __syncwarp();
        // output: weight x V row, lane = CV columns. In a tile with masked tokens a
        // zero weight does not touch its row, which may hold anything.
#pragma unroll 2
        for (int t = 0; t < NT; t += 4) {
          float4 w[RW];
#pragma unroll
          for (int r = 0; r < RW; ++r) w[r] = *reinterpret_cast<const float4*>(Ps + (warp * RW + r) * NT + t);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float v[CV];
#pragma unroll
            for (int c = 0; c < CV; ++c) v[c] = vd[(t + u) * D + 32 * c + lane];
#pragma unroll
            for (int r = 0; r < RW; ++r) {
              const float wu = u == 0 ? w[r].x : (u == 1 ? w[r].y : (u == 2 ? w[r].z : w[r].w));
#pragma unroll
              for (int c = 0; c < CV; ++c)
                if (!masked || wu != 0.f) acc[r][c] = fmaf(wu, v[c], acc[r][c]);
            }
          }
        }
        __syncwarp();
      }
    }
    // the item's rows: the output, or this share's partial
    const bool whole = it.tile0 == 0 && it.tile1 == it.tiles;
    if (!whole && it.tile0 == 0 && tid == 0) p.join[blockIdx.x] = TreeJoin{walk.last_cta(it), it.q0, it.rows, it.kv};
    float* slot = tree_slot<D>(p, blockIdx.x, it.tile0 == 0 ? 1 : 0);
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const int row = warp * RW + r;
      float ls = l[r];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
      if (row >= it.rows) continue;
      if (whole) {
        const float inv = ls == 0.f ? 0.f : 1.f / ls;
        float* dst = static_cast<float*>(p.out) +
                     ((long long)(it.q0 + row / p.group) * p.H + it.kv * p.group + row % p.group) * D;
#pragma unroll
        for (int c = 0; c < CV; ++c) dst[32 * c + lane] = acc[r][c] * inv;
      } else {
        if (lane == 0) reinterpret_cast<float2*>(slot)[row] = make_float2(m[r], ls);
#pragma unroll
        for (int c = 0; c < CV; ++c) {
          const int col = 32 * c + lane;
          slot[2 * p.slot_rows + ((long long)(col >> 2) * p.slot_rows + row) * 4 + (col & 3)] = acc[r][c];
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------------
// Joining the shares of the items that more than one CTA worked on: CTA x of the
// grid takes the item that starts, unfinished, in CTA x of the attention kernel,
// rows 32 y .. 32 y + 31 and columns 64 z .. 64 z + 63. M = max_c m_c,
// w_c = 2^(m_c - M), out = sum_c w_c o_c / sum_c w_c l_c, over the item's CTAs in
// order. Lane = row, and a warp has two vectors of four columns, eight vectors apart:
// a partial lies [D / 4][rows], so a warp reads 512 bytes of it at once, with four
// partials' loads in flight. Bound by latency: a few microseconds behind the attention
// (5 us under ncu on 160 CTAs' partials). More loads in flight leave two CTAs on an SM
// (eight partials, four vectors: 18.5 us); two partials and four vectors a thread cost
// 2 us where few items are shared by many CTAs and gain nothing where many are shared
// by two or three.
// ---------------------------------------------------------------------------------
constexpr int kTreeJoinThreads = 256;

template <typename OT, int D>
__global__ void __launch_bounds__(kTreeJoinThreads) tree_join_kernel(const TreeParams p) {
  pdl_begin();
  constexpr int NV = 2, BATCH = 4;
  const int c0 = blockIdx.x;
  const TreeJoin j = p.join[c0];
  const int row = (int)blockIdx.y * 32 + (threadIdx.x & 31);
  if (j.last < 0 || row >= j.rows) return;
  const int v = (int)blockIdx.z * 8 * NV + (threadIdx.x >> 5);  // column vectors v, v + 8, ..: columns 4 v + 32 e ..
  const float NEG_INF = -__int_as_float(0x7f800000);
  float M = NEG_INF, L = 0.f;
  float4 acc[NV];
#pragma unroll
  for (int e = 0; e < NV; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = c0; c <= j.last; c += BATCH) {
    float2 ml[BATCH];
    float4 o[BATCH][NV];
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      ml[u] = make_float2(NEG_INF, 0.f);
      if (c + u > j.last) continue;
      const float* slot = tree_slot<D>(p, c + u, c + u == c0 ? 1 : 0);
      ml[u] = reinterpret_cast<const float2*>(slot)[row];
      const float4* src = reinterpret_cast<const float4*>(slot + 2 * p.slot_rows) + (long long)v * p.slot_rows + row;
#pragma unroll
      for (int e = 0; e < NV; ++e) o[u][e] = src[8LL * e * p.slot_rows];
    }
#pragma unroll
    for (int u = 0; u < BATCH; ++u) {
      if (ml[u].y == 0.f) continue;  // nothing attended in this share (a sum of NaN goes on)
      const float Mn = fmaxf(M, ml[u].x);
      const float f = M == Mn ? 1.f : exp2f(M - Mn), w = exp2f(ml[u].x - Mn);
#pragma unroll
      for (int e = 0; e < NV; ++e) {
        acc[e].x = fmaf(w, o[u][e].x, acc[e].x * f);
        acc[e].y = fmaf(w, o[u][e].y, acc[e].y * f);
        acc[e].z = fmaf(w, o[u][e].z, acc[e].z * f);
        acc[e].w = fmaf(w, o[u][e].w, acc[e].w * f);
      }
      L = fmaf(w, ml[u].y, L * f);
      M = Mn;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  OT* dst = static_cast<OT*>(p.out) +
            ((long long)(j.q0 + row / p.group) * p.H + j.kv * p.group + row % p.group) * D + 4 * v;
#pragma unroll
  for (int e = 0; e < NV; ++e) {
    alignas(16) OT x[4] = {from_f32<OT>(acc[e].x * inv), from_f32<OT>(acc[e].y * inv), from_f32<OT>(acc[e].z * inv),
                           from_f32<OT>(acc[e].w * inv)};
    if constexpr (sizeof(OT) == 2) *reinterpret_cast<uint2*>(dst + 32 * e) = *reinterpret_cast<const uint2*>(x);
    else *reinterpret_cast<uint4*>(dst + 32 * e) = *reinterpret_cast<const uint4*>(x);
  }
}

}  // namespace pa
