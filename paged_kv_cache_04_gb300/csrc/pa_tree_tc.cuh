// Attention of drafted tokens on the fifth-generation tensor cores (tcgen05,
// accumulators in tensor memory): 16-bit caches.
//
// The rows of an item (node x query head of one kv head) form the M side, 128 of
// them (padded), of
//   S = Q K^T    M = 128, N = 64 tokens, K = head_dim
//   O += P V     M = 128, N = head_dim,  K = 64 tokens
// One CTA per SM works through its share of the units (see pa_tree.cuh) with two
// streams of softmax warps, each with an accumulator O and two score buffers of
// its own. An item of more than 128 rows gives each stream one half of the rows:
// a K and V tile in shared memory then serves 256 rows, so up to that many rows
// the cache is read once. A smaller item's streams take its token tiles in turn
// and their accumulators are joined at its end, so that one stream's softmax
// always overlaps the other's products. head_dim 256 fills the tensor memory with
// one accumulator and has one stream.
//
// Warps: 4 per stream  softmax. Thread t of warp w owns row 32 w + t, in the
//                      tensor-memory lane of that number: it reads its 64 scores,
//                      keeps the running (max, sum) and writes the weights back
//                      over them in 16 bits, in two parts or one. Warps without
//                      real rows only keep the barriers going.
//        K producer    queries of each item, then the keys of each tile, 16 tokens x
//                      64 columns per TMA copy, into a ring of slots; a slot is free
//                      when the score products of its tile have completed.
//        V producer    the same for the values, freed by the output products.
//        scores        one per stream: issues its score products.
//        outputs       one per stream: issues its output products. (One warp for
//                      both streams' scores, or one for a stream's scores and
//                      outputs, was what wide items waited for: 320 and 345 us
//                      against 300 on 4 x 41k tokens, 64 q / 8 kv, 64 nodes.)
// That is fourteen warps of at most 128 registers.
// Before a tile with drafted tokens or the context's end is used, its stream's warps
// check its values: rows past the context become zeros and so do infinities and NaN
// in the drafted ones, since a weight of zero does not hide them in a product. The
// rows that do attend such a value get it added to their O.
// Scores and weights share their columns of tensor memory (a thread has read its
// 64 scores when it writes its weights): a buffer belongs to a tile from its score
// products to the end of its output products.
// A row's reference maximum moves
// only when a score passes it by kTreeRescale (log2 units); the weights stay below
// 2^kTreeRescale and numerator and denominator share the reference. fp16 has no bits
// below 2^-24, and a long flat tail under a peak is many small weights: there the
// weights are taken 2^7 times as large (below 2^15, fp16 ends at 2^16), in numerator
// and denominator alike, so what a weight may lose is 2^-32 of the reference's and a
// context of 2^17 tokens loses at most 2^-15.
//
// Weights are carried as two 16-bit parts (hi + lo, together 16 bits or more), the
// library's rule for attention, with one exception: items of more than 128 rows
// with a 16-bit output carry them as one. There the kernel is bound by the tensor
// cores and the softmax's instructions, not by memory: the second part doubles the
// output products and adds instructions for each weight (358 us against 272 on 4 x 41k
// tokens, 64 q / 8 kv, 64 nodes; at the power limit 386 against 296). One part also leaves
// registers to keep a tile's weights in, so its scores are read once: the weights are
// taken against the reference so far and kept if their sum shows that none of them is
// above 2^kTreeRescale, else the tile is read again for a new reference (a pass for
// the maximum first: 291 us against 261 on that batch, when the sum still took the
// weights before rounding). A rounded weight w (1 + e) is
// off by at most half a step of the type. Sum and products take the same rounded
// weights, so they still make an average, and to first order in e the result is off by
//   sum w e (v - out) / sum w   <=   half a step x sum w |v - out| / sum w:
// nothing where one token carries its row or the values are alike, and about the
// output's own rounding (a total of sqrt(2) times that) where they differ at random.
// With the weights summed before they are rounded, a row carried by one token would be
// off by up to half a step more; rounding first costs 268 us against 251 on that batch
// (sustained, at the power limit: 293 against 284). An fp32 output keeps both parts
// everywhere.
//
// Every wait is bounded; on a timeout all roles stop, copies and products in
// flight are waited for, and the tensor memory is released.
//
// Measured (GB300, 2,070 MHz, attention and joining kernel, in a graph): narrow items,
// 64 sequences of 512 to 4,096 tokens with trees of 9 to 32 nodes, 32 q / 8 kv, 118 us
// (615 MB once: 5.2 TB/s; 5.6 TB/s of DRAM reads inside the kernel); wide ones, 4 of
// 16k to 64k tokens with 64 nodes, 64 q / 8 kv, 268 to 272 us (1,270 TFLOP/s; call after
// call for seconds the power limit lowers the clock, 288 to 296 us). A wide item's
// tile takes about 1,900 cycles, of which its products fill 1,250: a stream's score
// products 386, set by the operands' 6 KB of shared memory for 32 cycles of
// arithmetic at N = 64, its output products 257. The rest is hand-offs: a stream's
// next scores wait for the output products of two tiles before, which wait for the
// slowest of its four softmax warps.
#pragma once

#include "pa_tcgen05.cuh"
#include "pa_tree.cuh"

namespace pa {

constexpr int kTreeTile = 64;         // tokens of a unit
constexpr int kTreeJob = 16;          // tokens of a TMA copy
constexpr float kTreeRescale = 8.f;
template <typename DT>
constexpr float kTreeLift = std::is_same<DT, __half>::value ? 7.f : 0.f;  // log2 of what all weights are multiplied by

// Shared memory (227 KB): queries, then the K and V rings. QR: rows kept of a query
// tile. A call whose items have 64 rows at most keeps no more and has room for more K
// and V slots, or, at head_dim 256, for a second query tile (without it the next
// item's keys wait until the last item's scores are done). The products always read
// 128 rows; what lies behind a tile then makes rows that nobody reads.
template <int D, int QR>
struct TreeTc {
  static constexpr int NS = D == 256 ? 1 : 2;                    // streams
  static constexpr int QB = D == 256 && QR == 128 ? 1 : 2;       // query tiles
  static constexpr int KS = D == 256 ? 2 : (D == 128 ? (QR == 64 ? 6 : 5) : 8);
  static constexpr int VS = D == 256 ? 3 : (D == 128 ? (QR == 64 ? 6 : 5) : 8);
  static constexpr int NREG = D / 64;               // 128-byte regions of a row
  static constexpr int THREADS = (6 * NS + 2) * 32;
  static constexpr unsigned Q_BYTES = QR * D * 2, TILE = kTreeTile * D * 2, REG = kTreeTile * 128;
  static constexpr unsigned K_OFF = QB * Q_BYTES, V_OFF = K_OFF + KS * TILE, BAR_OFF = V_OFF + VS * TILE;
  static constexpr int KINDS = NS == 2 ? 3 : 1;     // whom a tile is for: stream 0, stream 1, both
  static constexpr int BARS = (KINDS + 1) * (KS + QB) + (KINDS + 3) * VS + 8 * NS + 2;
  static constexpr unsigned BAD_OFF = BAR_OFF + BARS * 8;            // u64 [2][VS]
  static constexpr unsigned ML_OFF = BAD_OFF + 2 * VS * 8;           // float2 [2][128]
  static constexpr unsigned SCRATCH_OFF = ML_OFF + (NS == 2 ? 2048 : 0);
  static constexpr unsigned MISC_OFF = SCRATCH_OFF + (THREADS / 32 + 3) * 8;
  static constexpr unsigned TOTAL = MISC_OFF + 16;
  // tensor memory: O of each stream, then two score / weight buffers of each
  static constexpr uint32_t COLS = 512;
  static constexpr uint32_t SP_COL = NS * D;
  static_assert(SP_COL + NS * 2 * kTreeTile <= COLS, "tensor-memory columns");
  static_assert(TOTAL <= 227 * 1024, "shared memory");
};

// One lane of the (converged) warp, the same one every time. TMA and tcgen05
// instructions take their operands from uniform registers: behind this test the
// compiler knows that one thread runs and moves them there directly; behind
// `lane == 0` it wraps every such instruction into a loop over the active threads
// (about 200 cycles an instruction were measured).
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(on));
  return on != 0;
}

// 32 consecutive columns of this thread's lane, complete on return (one statement: nothing computed from the
// registers can move in front of the wait).
__device__ __forceinline__ void tc_ld32_done(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// 64 consecutive columns.
__device__ __forceinline__ void tc_ld32x2_done(uint32_t taddr, uint32_t (&r)[32], uint32_t (&t)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(t[0]), "=r"(t[1]), "=r"(t[2]), "=r"(t[3]), "=r"(t[4]), "=r"(t[5]), "=r"(t[6]), "=r"(t[7]), "=r"(t[8]), "=r"(t[9]), "=r"(t[10]), "=r"(t[11]), "=r"(t[12]), "=r"(t[13]), "=r"(t[14]), "=r"(t[15]), "=r"(t[16]), "=r"(t[17]), "=r"(t[18]), "=r"(t[19]), "=r"(t[20]), "=r"(t[21]), "=r"(t[22]), "=r"(t[23]), "=r"(t[24]), "=r"(t[25]), "=r"(t[26]), "=r"(t[27]), "=r"(t[28]), "=r"(t[29]), "=r"(t[30]), "=r"(t[31])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
}
// 16 columns from each of two places.
__device__ __forceinline__ void tc_ld16_pair(uint32_t ta, uint32_t tb, uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]),
        "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]), "=r"(b[0]),
        "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(b[8]), "=r"(b[9]),
        "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15])
      : "r"(ta), "r"(tb)
      : "memory");
}

// The waits of this kernel, by all lanes of a warp (the answer is the same in each): one poll inline, the rest out of
// line. Twelve warps run four different loops, and with every wait's polling, timing and abort code inlined the loops
// outgrew the instruction cache.
static __device__ __noinline__ bool tree_wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                   unsigned* err) {
  const bool ok = mbar_wait_sleep(bar, parity, abort_flag, err, kWaitLimitNs);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned* err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return tree_wait_slow(bar, parity, abort_flag, err);
}

// Two fp32 operations at a time (a register pair).
__device__ __forceinline__ uint64_t pair2(uint32_t a, uint32_t b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint64_t pair2(float a, float b) { return pair2(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ void unpair2(uint64_t d, float& a, float& b) {
  uint32_t x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(x), "=r"(y) : "l"(d));
  a = __uint_as_float(x);
  b = __uint_as_float(y);
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// tcgen05.st without its wait.
__device__ __forceinline__ void tc_st32_issue(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tc_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Bit e set: the 16-bit value at half e of a word is an infinity or NaN.
template <typename DT>
__device__ __forceinline__ unsigned nonfinite2(uint32_t w) {
  constexpr uint32_t EXP = std::is_same<DT, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
  return ((w & EXP) == EXP ? 1u : 0u) | (((w >> 16) & EXP) == EXP ? 2u : 0u);
}

// What an item runs once or twice is kept out of line, out of the loops' way in the
// instruction cache: the mask's bits for a tile,
static __device__ __noinline__ unsigned long long tree_window_call(const TreeParams& p, long long row, int node,
                                                                   int j) {
  return tree_window(p, row, node, j);
}

// the check of rows [rb, rb + span) of a V tile (drafted tokens are rows [first, end); returns the rows, from rb
// on, in which infinities or NaN were replaced by zeros),
template <typename DT, int D>
static __device__ __noinline__ unsigned tree_check_v(uint8_t* v, int rb, int span, int first, int end) {
  constexpr int NREG = D / 64, FLIGHT = 4;  // 16-byte chunks in flight per lane
  const int lane = threadIdx.x & 31;
  unsigned bad = 0;
  // rows in front of the drafted tokens, and jobs behind the context (staged as zeros), need nothing
  const int from = max(first, rb), to = min(rb + span, (max(end, 0) + kTreeJob - 1) / kTreeJob * kTreeJob);
  // (a row is NREG x 128 bytes; the swizzle moves 16-byte chunks within them)
  auto chunk = [&](int i) {
    const int k = i / (8 * NREG), c = i % (8 * NREG);
    return reinterpret_cast<uint4*>(v + (c >> 3) * (kTreeTile * 128) + k * 128 + (c & 7) * 16);
  };
#pragma unroll 1
  for (int i0 = from * 8 * NREG; i0 < to * 8 * NREG; i0 += 32 * FLIGHT) {
    uint4 x[FLIGHT];
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      const int i = i0 + 32 * u + lane;
      x[u] = i < to * 8 * NREG ? *chunk(i) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < FLIGHT; ++u) {
      const int i = i0 + 32 * u + lane;
      if (i >= to * 8 * NREG) continue;
      if (i >= end * 8 * NREG) {
        *chunk(i) = make_uint4(0u, 0u, 0u, 0u);
      } else if (nonfinite2<DT>(x[u].x) | nonfinite2<DT>(x[u].y) | nonfinite2<DT>(x[u].z) |
                 nonfinite2<DT>(x[u].w)) {  // rare
        bad |= 1u << (i / (8 * NREG) - rb);
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
          uint16_t* h = reinterpret_cast<uint16_t*>(chunk(i)) + e;
          if (nonfinite2<DT>(*h)) *h = 0;
        }
      }
    }
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  fence_proxy_async_smem();
  __syncwarp();
  return bad;
}

// and the values replaced there, from the cache, to the rows of O (at `o`, this thread's lane) that attend them: bit
// t - t0 of `seen` (0 for threads without a row) says so for token t.
template <typename DT, int D>
static __device__ __noinline__ void tree_add_bad(const TreeParams& p, const int32_t* table, int kv, int t0,
                                                 unsigned long long bad, unsigned long long seen, uint32_t o) {
  for (; bad; bad &= bad - 1) {
    const int j = __ffsll((long long)bad) - 1, t = t0 + j;
    const bool on = (seen >> j) & 1;
    const int blk = __ldg(table + (t >> p.block_shift));
    if (blk < 0 || blk >= p.num_blocks) continue;
    const DT* row = static_cast<const DT*>(p.v_cache) + tree_row<D>(p, blk, kv, t);
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      uint32_t x[32];
      tc_ld32(o + c0, x);
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const float v = to_f32(row[c0 + e]);
        if (on && !(fabsf(v) <= 3.4028235e38f)) x[e] = __float_as_uint(__uint_as_float(x[e]) + v);
      }
      tc_st32(o + c0, x);
    }
  }
}

// A row's reference maximum from the 64 scores at `sp`, where they pass the old one by more than 2^2 (64 weights of
// that size sum to 2^kTreeRescale), its sum and (with `bar`, the barrier of the products that O waits for) its O brought
// to the new one. Once or twice an item.
struct TreeRef {
  float m, l;
  bool ok;
};
template <int D>
static __device__ __noinline__ TreeRef tree_new_ref(uint32_t sp, float scale, float m, float l, uint64_t* bar,
                                                    uint32_t parity, uint32_t o, volatile int* abort_flag,
                                                    unsigned* err) {
  const float NEG_INF = -__int_as_float(0x7f800000);
  const uint64_t scale2 = pair2(scale, scale);
  float mx = NEG_INF;
#pragma unroll 1
  for (int h = 0; h < kTreeTile; h += 32) {
    uint32_t s[32];
    tc_ld32_done(sp + h, s);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float a, c;
      unpair2(mul2(pair2(s[2 * e], s[2 * e + 1]), scale2), a, c);
      mx = max3(mx, a, c);
    }
  }
  const bool move = mx > m + (kTreeRescale - 6.f) || (m == NEG_INF && mx > NEG_INF);
  if (!__any_sync(0xffffffffu, move)) return {m, l, true};
  const float m_new = move ? mx : m, c = move ? exp2f(m - m_new) : 1.f;
  if (bar != nullptr) {
    if (!tree_wait(bar, parity, abort_flag, err)) return {m, l, false};
    tc_fence_after();
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
      uint32_t x[32];
      tc_ld32_done(o + c0, x);
#pragma unroll
      for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * c);
      tc_st32(o + c0, x);
    }
  }
  return {m_new, l * c, true};
}

// The weights 2^(scale x score + neg) of a row's 64 scores at `sp`, in one 16-bit part, written over the scores'
// first 32 columns (without a wait), their sum added to `l`: of the weights as they were rounded, which are the ones
// that the output products take. With `check`, not if a sum of the warp's rows allows a weight above 2^kTreeRescale
// (then: false; tree_new_ref moves references by less, so that it does not come again).
template <typename DT>
__device__ __forceinline__ bool tree_weights(uint32_t sp, float scale, float neg, bool check, float& l) {
  const uint64_t scale2 = pair2(scale, scale), neg2 = pair2(neg, neg);
  uint64_t ls[2] = {0, 0};
  uint32_t pw[32];
  uint32_t sa[32], sb[32];
  tc_ld32x2_done(sp, sa, sb);
#pragma unroll
  for (int h = 0; h < kTreeTile; h += 32) {
    uint32_t (&s)[32] = h ? sb : sa;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float a, c;
      unpair2(fma2(pair2(s[2 * e], s[2 * e + 1]), scale2, neg2), a, c);
      a = ex2_ftz(a);
      c = ex2_ftz(c);
      const uint32_t w = Mma<DT>::pack(a, c);
      unpack2(w, (DT*)nullptr, a, c);
      ls[e & 1] = add2(ls[e & 1], pair2(a, c));
      pw[h / 2 + e] = w;
    }
  }
  float l0, l1;
  unpair2(add2(ls[0], ls[1]), l0, l1);
  l0 += l1;
  constexpr float LIMIT = std::is_same<DT, __half>::value ? 32768.f : 256.f;  // 2^(kTreeRescale + kTreeLift)
  if (check && __any_sync(0xffffffffu, l0 > LIMIT)) return false;
  tc_st32_issue(sp, pw);
  l += l0;
  return true;
}

// Matrix descriptors of the 128-byte swizzle as two words, of which only the lower one (address and leading
// offset) varies; see tc_desc.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  return (uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32 | lo;
}

template <typename DT, typename OT, int D, int QR>
__global__ void __launch_bounds__(TreeTc<D, QR>::THREADS, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ CUtensorMap qmap, const TreeParams p) {
  static_assert(sizeof(DT) == 2, "16-bit caches");
  using C = TreeTc<D, QR>;
  constexpr int NS = C::NS, QB = C::QB, KS = C::KS, VS = C::VS, NREG = C::NREG, T = kTreeTile, J = kTreeJob;
  constexpr int SW = 4 * NS;  // softmax warps; then K, V, scores of each stream, outputs of each stream
  constexpr uint32_t ID_S = tc_idesc<DT>(128, T, false), ID_PV = tc_idesc<DT>(128, D, true);

  extern __shared__ __align__(1024) uint8_t tree_tc_smem[];  // (128-byte swizzled tiles start on 1,024 bytes)
  uint8_t* smem = tree_tc_smem;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  // Landed keys, values and queries have one set of barriers for each kind of tile: whoever waits on a barrier by
  // parity must see every one of its phases, and a stream sees its own tiles and the common ones only. Values to be
  // checked are waited for by the checking warps, which see no others.
  constexpr int KINDS = C::KINDS;
  uint64_t* k_full = bars;                  // [KINDS][KS] keys landed
  uint64_t* k_empty = k_full + KINDS * KS;  // [KS] score products done
  uint64_t* v_full = k_empty + KS;          // [KINDS][VS] values landed, of tiles that need no check
  uint64_t* m_full = v_full + KINDS * VS;   // [VS] values landed, of tiles to be checked
  uint64_t* v_clean = m_full + VS;          // [VS] those checked, bad_rows written
  uint64_t* v_empty = v_clean + VS;         // [VS] output products done
  uint64_t* q_full = v_empty + VS;          // [KINDS][QB] queries landed
  uint64_t* q_free = q_full + KINDS * QB;   // [QB] the score products that read them done
  uint64_t* s_full = q_free + QB;         // [NS][2] scores written
  uint64_t* p_full = s_full + 2 * NS;     // [NS][2] weights written
  uint64_t* pv_done = p_full + 2 * NS;    // [NS][2] output products done: buffer free, O current
  uint64_t* o_free = pv_done + 2 * NS;    // O read at an item's end
  uint64_t* ml_full = o_free + 1;         // both streams' (max, sum) in shared memory
  uint64_t* fin = o_free + 2;             // [2][NS] every product done (teardown)
  // [2][VS] what the check of a slot's tile found, in two copies that its checked tiles take in turn. A warp reads the
  // word after its weights have gone off, and the slot may be filled and checked again before it has (at head_dim 256
  // by a warp three tiles on, which waits for no weights of this one's next tile). It can not be filled a second time:
  // that takes the output products of the tile in between, and so this warp's weights.
  unsigned long long* bad_rows = reinterpret_cast<unsigned long long*>(smem + C::BAD_OFF);
  float2* ml = reinterpret_cast<float2*>(smem + C::ML_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  volatile int* gaps = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 8);  // a block outside the pool was met
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid < C::BARS) {  // a thread per barrier
    uint64_t* bar = bars + tid;
    const bool each = (bar >= k_empty && bar < v_full) || (bar >= v_empty && bar < q_full) ||
                      (bar >= q_free && bar < s_full);  // one arrival from every stream
    const bool warps = bar >= p_full && bar < pv_done;  // from every warp of a stream
    const bool all = (bar >= v_clean && bar < v_empty) || bar == o_free || bar == ml_full;  // from all their warps
    mbar_init(bar, all ? SW : (warps ? 4 : (each ? NS : 1)));
    fence_barrier_init();
  }
  if (tid == 0) {
    *abort_flag = 0;
    *gaps = 0;
  }
  if (tid == 32) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&qmap);
  }
  const int half_toks = QR / p.group;         // nodes of one tile of QR rows
  const int half_rows = half_toks * p.group;
  // query rows past the box stay zeros (16-byte chunks of every query tile, region and row from half_rows on)
  for (int i = tid; i < QB * NREG * (QR - half_rows) * 8; i += C::THREADS) {
    const int region = i / ((QR - half_rows) * 8), at = half_rows * 8 + i % ((QR - half_rows) * 8);
    reinterpret_cast<uint4*>(smem + region * (QR * 128))[at] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (warp == SW + 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(C::COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_begin();  // (nothing above touches global memory)
  if (tid == 0) p.join[blockIdx.x].last = -1;
  TreeWalk walk = tree_share<C::THREADS>(p, reinterpret_cast<long long*>(smem + C::SCRATCH_OFF));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  auto both = [&](const TreeItem& it) { return NS == 2 && QR == 128 && it.rows > half_rows; };  // each stream has rows of its own
  auto one_part = [](bool two) { return sizeof(OT) == 2 && two; };  // weights in one 16-bit part
  auto masked = [&](const TreeItem& it, int tile) { return (tile + 1) * T > it.prefix; };
  auto kind_of = [](bool two, int k) { return NS == 1 ? 0 : (two ? 2 : k & 1); };  // of an item's k-th tile
  auto uniform = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
  auto wait = [&](uint64_t* bar, uint32_t parity) { return tree_wait(bar, parity, abort_flag, p.err); };
  TreeItem it;
  auto next_item = [&]() { return walk.next(p, it); };

  if (warp == SW || warp == SW + 1) {
    // ------------------------------- producers -------------------------------
    const bool is_v = warp == SW + 1;
    const int R = is_v ? VS : KS;
    uint64_t* full = is_v ? v_full : k_full;    // [KINDS][R]; m_full lies behind v_full as a further kind
    uint64_t* empty = is_v ? v_empty : k_empty;
    uint8_t* ring = smem + (is_v ? C::V_OFF : C::K_OFF);
    const CUtensorMap* map = is_v ? &vmap : &kmap;
    int n = 0, qn = 0;
    static_assert(KS <= 8 && VS <= 8 && KINDS < 4, "one bit for each kind and slot");
    uint32_t uses = 0, last = 0;  // bit 8 kind + slot: parity of its uses; 4 bits for each slot: its last tile's kind
    uint32_t quses = 0, qlast = 0;
    bool stop = false;
    while (!stop && next_item()) {
      const int32_t* table = p.block_tables + (long long)it.s * p.max_blocks;
      const int je = (it.ctx + J - 1) / J;  // the context's jobs
      // the pool map's row of job j: -kTreeJob (rows in front of the pool, read as zeros) where there is none
      auto job_row = [&](int j) {
        if (j >= je) return -J;
        const int t = j * J, id = __ldg(table + (t >> p.block_shift));
        if (id < 0 || id >= p.num_blocks) {
          if (!is_v) atomicOr(p.err, kErrBlockId);
          *gaps = 1;  // (before the copies of its tile are announced, so before its scores are read)
          return -J;
        }
        return ((p.nhd ? id : id * p.G + it.kv) << p.block_shift) + (t & (p.B - 1));
      };
      // lane l holds job wbase + l, and that of the next window
      int wbase = it.tile0 * (T / J);
      int cur = job_row(wbase + lane), nxt = job_row(wbase + 32 + lane);
      if (!is_v) {
        const int nq = both(it) ? 2 : 1;
        for (int w = 0; w < nq; ++w, ++qn) {
          const int qb = qn % QB;
          if (qn >= QB && !wait(&q_free[qb], ((qn / QB) - 1) & 1)) {
            stop = true;
            break;
          }
          const int kind = NS == 1 ? 0 : (nq == 2 ? w : 2);
          uint64_t* bar = &q_full[kind * QB + qb];
          quses ^= 1u << (8 * kind + qb);
          qlast = (qlast & ~(15u << (4 * qb))) | (uint32_t)kind << (4 * qb);
          if (elect_one()) {
            mbar_arrive_expect_tx(bar, (uint32_t)(half_rows * D * 2));
#pragma unroll
            for (int rg = 0; rg < NREG; ++rg)
              tma_load_3d(smem + qb * C::Q_BYTES + rg * (QR * 128), &qmap, rg * 64, it.kv * p.group,
                          it.q0 + w * half_toks, bar);
          }
        }
        if (stop) break;
      }
      for (int tile = it.tile0; tile < it.tile1; ++tile, ++n) {
        const int j0 = tile * (T / J);
        if (j0 >= wbase + 32) {
          wbase += 32;
          cur = nxt;
          nxt = job_row(wbase + 32 + lane);
        }
        const int slot = n % R;
        if (n >= R && !wait(&empty[slot], ((n / R) - 1) & 1)) {
          stop = true;
          break;
        }
        const int head = p.nhd ? it.kv : 0;  // the pool map's middle coordinate
        int row[T / J];
#pragma unroll
        for (int j = 0; j < T / J; ++j) row[j] = __shfl_sync(0xffffffffu, cur, j0 + j - wbase);
        const int kind = is_v && masked(it, tile) ? KINDS : kind_of(both(it), tile - it.tile0);
        uint64_t* bar = &full[kind * R + slot];
        uses ^= 1u << (8 * kind + slot);
        last = (last & ~(15u << (4 * slot))) | (uint32_t)kind << (4 * slot);
        if (elect_one()) {
          uint8_t* dst = ring + slot * C::TILE;
          mbar_arrive_expect_tx(bar, C::TILE);
#pragma unroll
          for (int i = 0; i < (T / J) * NREG; ++i)
            tma_load_3d(dst + (i % NREG) * C::REG + (i / NREG) * (J * 128), map, (i % NREG) * 64, head, row[i / NREG], bar);
        }
      }
    }
    // let the last copies land before the block can exit
    if (lane == 0) {
      for (int slot = 0; slot < min(n, R); ++slot) {
        const int kind = (last >> (4 * slot)) & 15;
        mbar_wait_bounded(&full[kind * R + slot], ((uses >> (8 * kind + slot)) & 1) ^ 1, nullptr, p.err, kDrainLimitNs);
      }
      for (int qb = 0; qb < min(qn, QB); ++qb) {
        const int kind = (qlast >> (4 * qb)) & 15;
        mbar_wait_bounded(&q_full[kind * QB + qb], ((quses >> (8 * kind + qb)) & 1) ^ 1, nullptr, p.err, kDrainLimitNs);
      }
    }
    __syncwarp();
  } else if (warp >= SW + 2 && warp < SW + 2 + NS) {
    // ------------------------------ score products ------------------------------
    // A slot or query tile that one stream alone uses gets its commits for both.
    const int w = warp - SW - 2;
    int kslot = 0, qn = 0, turn = 0;    // K slot and query tile of the walk; the stream's tiles so far
    uint32_t kuses = 0, quses = 0;      // bit 8 kind + slot: parity of the next use
    bool stop = false;
    while (!stop && next_item()) {
      const bool two = both(it);
      const int qb = (qn + (two ? w : 0)) % QB, qkind = NS == 1 ? 0 : (two ? w : 2);
      // (broadcasts tell the compiler that the operands are the same in every lane)
      const uint32_t qlo = uniform(desc_lo(smem_u32(smem + qb * C::Q_BYTES), 16));
      if (!wait(&q_full[qkind * QB + qb], (quses >> (8 * qkind + qb)) & 1)) break;
      quses ^= 1u << (8 * qkind + qb);
      for (int k = 0; k < it.tile1 - it.tile0; ++k) {
        const int slot = kslot, kind = kind_of(two, k);
        if (++kslot == KS) kslot = 0;
        if (NS == 2 && kind != 2 && kind != w) continue;
        const int b = turn & 1;
        const uint32_t klo = uniform(desc_lo(smem_u32(smem + C::K_OFF + slot * C::TILE), 16));
        const uint32_t d = uniform(tbase + C::SP_COL + (2 * w + b) * T);
        // (the buffer last: it is what the stream's next scores usually wait for)
        if (!wait(&k_full[kind * KS + slot], (kuses >> (8 * kind + slot)) & 1) ||
            (turn >= 2 && !wait(&pv_done[2 * w + b], ((turn >> 1) - 1) & 1))) {
          stop = true;
          break;
        }
        if (elect_one()) {
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            tc_mma(d, desc_of(qlo + ((ks >> 2) * (QR * 128) + (ks & 3) * 32) / 16),
                   desc_of(klo + ((ks >> 2) * C::REG + (ks & 3) * 32) / 16), ID_S, ks > 0);
          tc_commit(&s_full[2 * w + b]);
          tc_commit(&k_empty[slot]);
          if (NS == 2 && !two) tc_commit(&k_empty[slot]);
        }
        kuses ^= 1u << (8 * kind + slot);
        ++turn;
      }
      if (!stop && elect_one()) {
        tc_commit(&q_free[qb]);
        if (two) tc_commit(&q_free[qb]);
      }
      qn += two ? 2 : 1;
    }
    if (elect_one()) {  // (no products at all: the commit arrives at once)
      tc_commit(&fin[w]);
      mbar_wait_bounded(&fin[w], 0, nullptr, p.err, kDrainLimitNs);
    }
    __syncwarp();
  } else if (warp >= SW + 2 + NS) {
    // ------------------------------ output products ------------------------------
    const int w = warp - SW - 2 - NS;
    int vslot = 0, turn = 0, item = 0;
    uint32_t vuses = 0, clean = 0;  // bit 8 kind + slot: parity of the next use; of a slot's next checked tile
    bool stop = false;
    for (; !stop && next_item(); ++item) {
      const bool two = both(it);
      const uint32_t d = uniform(tbase + w * D);
      for (int k = 0; k < it.tile1 - it.tile0; ++k) {
        const int slot = vslot, kind = kind_of(two, k);
        const bool mk = masked(it, it.tile0 + k);
        const uint32_t cpar = (clean >> slot) & 1;
        if (mk) clean ^= 1u << slot;
        if (++vslot == VS) vslot = 0;
        if (NS == 2 && kind != 2 && kind != w) continue;
        const int b = turn & 1;
        const uint32_t vlo = uniform(desc_lo(smem_u32(smem + C::V_OFF + slot * C::TILE), C::REG));
        const uint32_t a = uniform(tbase + C::SP_COL + (2 * w + b) * T);
        const uint32_t add = uniform(k >= (two || NS == 1 ? 1 : 2));  // not the stream's first tile of the item
        // The values, then the weights, which usually come last; the rest behind the weights, whose arrival means
        // that the check's and the item's barriers, which this warp does not follow through the other stream's
        // tiles, are at most one phase behind. An item's first products overwrite O, so the last item's has been
        // read.
        if (!mk) {
          stop = !wait(&v_full[kind * VS + slot], (vuses >> (8 * kind + slot)) & 1);
          vuses ^= 1u << (8 * kind + slot);
        }
        if (!stop) stop = !wait(&p_full[2 * w + b], (turn >> 1) & 1);
        if (!stop && mk) stop = !wait(&v_clean[slot], cpar);
        if (!stop && !add && item > 0) stop = !wait(o_free, (item - 1) & 1);
        if (stop) break;
        if (elect_one()) {
          tc_fence_after();
          if (one_part(two)) {  // columns 8 ks .. + 7: the weights of tokens 16 ks .. + 15
#pragma unroll
            for (int ks = 0; ks < T / 16; ++ks)
              tc_mma_tmem_a(d, a + ks * 8, desc_of(vlo + ks * (2048 / 16)), ID_PV, ks > 0 ? 1u : add);
          } else {  // columns 16 ks .. + 7: their hi parts, then their lo parts
#pragma unroll
            for (int ks = 0; ks < T / 16; ++ks) {
              tc_mma_tmem_a(d, a + ks * 16, desc_of(vlo + ks * (2048 / 16)), ID_PV, ks > 0 ? 1u : add);
              tc_mma_tmem_a(d, a + ks * 16 + 8, desc_of(vlo + ks * (2048 / 16)), ID_PV, true);
            }
          }
          tc_commit(&pv_done[2 * w + b]);
          tc_commit(&v_empty[slot]);
          if (NS == 2 && !two) tc_commit(&v_empty[slot]);
        }
        ++turn;
      }
    }
    if (elect_one()) {
      tc_commit(&fin[NS + w]);
      mbar_wait_bounded(&fin[NS + w], 0, nullptr, p.err, kDrainLimitNs);
    }
    __syncwarp();
  } else {
    // -------------------------------- softmax --------------------------------
    const float NEG_INF = -__int_as_float(0x7f800000);
    const int w = NS == 2 ? warp >> 2 : 0, wq = warp & 3;  // stream; quarter of the tensor-memory lanes
    const int r = 32 * wq + lane;                          // this thread's row
    const uint32_t lanes = tbase + ((uint32_t)(32 * wq) << 16);
    int n = 0, ns = 0, joined = 0;  // tiles of the CTA and of this stream; items joined in shared memory
    uint32_t clean = 0;  // parity of each V slot's next checked tile
    bool stop = false;
    while (!stop && next_item()) {
      const bool two = both(it);
      const int row0 = two && w == 1 ? half_rows : 0;  // this stream's first row of the item
      const int rows = two ? (w == 0 ? half_rows : it.rows - half_rows) : it.rows;
      const bool warp_live = 32 * wq < rows, live = r < rows;
      const int node = (row0 + (live ? r : 0)) / p.group;
      tree_mask_touch(p, it.q0 + node);
      const int32_t* table = p.block_tables + (long long)it.s * p.max_blocks;
      float m_ref = NEG_INF, l = 0.f;
      const int step = two || NS == 1 ? 1 : 2, first = it.tile0 + (step == 2 ? w : 0);  // this stream's tiles
      const int mk0 = max(it.tile0, it.prefix / T);  // tiles from here on have drafted tokens or the context's end
      for (int tile = first; tile < it.tile1; tile += step, ++ns) {
        const int b = ns & 1, t0 = tile * T;
        const bool mk = tile >= mk0;
        int vslot = 0;
        uint32_t vpar = 0;
        unsigned long long seen = ~0ull;
        if (mk) {
          vslot = (n + tile - it.tile0) % VS;
          vpar = ((clean >> vslot) ^ ((tile - mk0) / VS)) & 1;
          if (warp_live) seen = tree_window_call(p, it.q0 + node, it.tok0 + node, t0 - it.prefix);
          // the check of V, by all warps that use the tile (8 or 16 rows each)
          if (!wait(&m_full[vslot], vpar)) {
            stop = true;
            break;
          }
          const int span = two ? 8 : 16, rb = (two ? warp : wq) * span;
          const unsigned bad = tree_check_v<DT, D>(smem + C::V_OFF + vslot * C::TILE, rb, span, it.prefix - t0,
                                                   it.ctx - t0);
          unsigned long long* word = &bad_rows[vpar * VS + vslot];
          if (NS == 1 || !two) {
            if (lane < NS) {
              reinterpret_cast<uint16_t*>(word)[wq] = (uint16_t)bad;
              mbar_arrive(&v_clean[vslot]);
            }
          } else if (lane == 0) {
            reinterpret_cast<uint8_t*>(word)[warp] = (uint8_t)bad;
            mbar_arrive(&v_clean[vslot]);
          }
        }
        if (!wait(&s_full[2 * w + b], (ns >> 1) & 1)) {
          stop = true;
          break;
        }
        tc_fence_after();
        const uint32_t sp = lanes + C::SP_COL + (2 * w + b) * T;
        if (warp_live) {
          if (mk || *gaps) {
            // masked scores become the value whose product with the scale is -infinity, in place (an item's
            // last tile or two; the softmax below stays one short piece of code)
            const int end = it.ctx - t0;
            if (end < 64) seen &= (1ull << max(end, 0)) - 1;
            if (*gaps) {  // jobs outside the pool were staged as zeros
              const int t = t0 + lane * J;
              const int id = lane < T / J && t < it.ctx ? __ldg(table + (t >> p.block_shift)) : 0;
              const unsigned there = __ballot_sync(0xffffffffu, id >= 0 && id < p.num_blocks);
              for (int j = 0; j < T / J; ++j)
                if (!((there >> j) & 1)) seen &= ~(0xffffull << (16 * j));
            }
            const uint32_t off = __float_as_uint(p.scale_log2 < 0.f ? -NEG_INF : NEG_INF);
#pragma unroll 1
            for (int c0 = 0; c0 < T; c0 += 32) {
              uint32_t x[32];
              tc_ld32_done(sp + c0, x);
              const uint32_t bits = (uint32_t)(seen >> c0);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = (bits >> e) & 1 ? x[e] : off;
              tc_st32(sp + c0, x);
            }
          }
          if (one_part(two)) {
            // The weights against the reference so far, which usually stands; their sum tells. They wait in registers
            // for it, so that a tile whose scores pass the reference can be read again. (In two parts they are too
            // many for that: narrow items, 64 sequences, 119 us became 131.)
            uint64_t* before = &pv_done[2 * w + (b ^ 1)];  // O of the tiles before is complete
            bool known = __all_sync(0xffffffffu, m_ref > NEG_INF || !live);  // (rows of no node may be NaN throughout)
            for (;;) {
              if (!known) {
                const TreeRef x = tree_new_ref<D>(sp, p.scale_log2, m_ref, l, tile != first ? before : nullptr,
                                                  ((ns - 1) >> 1) & 1, lanes + w * D, abort_flag, p.err);
                if (!x.ok) {
                  stop = true;
                  break;
                }
                m_ref = x.m;
                l = x.l;
              }
              if (tree_weights<DT>(sp, p.scale_log2, m_ref == NEG_INF ? 0.f : kTreeLift<DT> - m_ref, known, l)) break;
              known = false;
            }
            if (stop) break;
          } else {
            // The scores are read twice, 32 at a time, rather than kept: the loops' code halves, and so do the
            // registers.
            const uint64_t scale2 = pair2(p.scale_log2, p.scale_log2);
            float mx = NEG_INF;
#pragma unroll 1
            for (int h = 0; h < T; h += 32) {
              uint32_t s[32];
              tc_ld32_done(sp + h, s);
              float tm[4] = {mx, NEG_INF, NEG_INF, NEG_INF};
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float a, c;
                unpair2(mul2(pair2(s[2 * e], s[2 * e + 1]), scale2), a, c);
                tm[e & 3] = max3(tm[e & 3], a, c);
              }
              mx = max3(fmaxf(tm[0], tm[1]), tm[2], tm[3]);
            }
            const bool move = mx > m_ref + kTreeRescale || (m_ref == NEG_INF && mx > NEG_INF);
            if (__any_sync(0xffffffffu, move)) {
              const float m_new = move ? mx : m_ref;
              const float c = move ? exp2f(m_ref - m_new) : 1.f;
              l *= c;
              m_ref = m_new;
              if (tile != first) {  // O of the tiles before, to the new reference
                if (!wait(&pv_done[2 * w + (b ^ 1)], ((ns - 1) >> 1) & 1)) {
                  stop = true;
                  break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                  uint32_t o[32];
                  tc_ld32_done(lanes + w * D + c0, o);
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * c);
                  tc_st32(lanes + w * D + c0, o);
                }
              }
            }
            const float neg = m_ref == NEG_INF ? 0.f : kTreeLift<DT> - m_ref;
            const uint64_t neg2 = pair2(neg, neg);
            uint64_t ls[2] = {0, 0};
#pragma unroll 1
            for (int h = 0; h < T; h += 32) {  // 32 tokens: per 16, 8 words of hi parts, then 8 of lo parts
              uint32_t s[32], pw[32];
              tc_ld32_done(sp + h, s);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float a, c;
                unpair2(fma2(pair2(s[2 * e], s[2 * e + 1]), scale2, neg2), a, c);
                a = ex2_ftz(a);
                c = ex2_ftz(c);
                const uint64_t w2 = pair2(a, c);
                ls[e & 1] = add2(ls[e & 1], w2);
                const uint32_t hi = Mma<DT>::pack(a, c);
                float h0, h1;
                unpack2(hi, (DT*)nullptr, h0, h1);
                unpair2(sub2(w2, pair2(h0, h1)), a, c);
                const int at = (e >> 3) * 16 + (e & 7);
                pw[at] = hi;
                pw[at + 8] = Mma<DT>::pack(a, c);
              }
              tc_st32_issue(sp + h, pw);
            }
            float l0, l1;
            unpair2(add2(ls[0], ls[1]), l0, l1);
            l += l0 + l1;
          }
          tc_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * w + b]);
        if (mk && warp_live) {  // (usually the stream's last tile of the item, whose products are waited for anyway)
          if (!wait(&v_clean[vslot], vpar) || !wait(&pv_done[2 * w + b], (ns >> 1) & 1)) {
            stop = true;
            break;
          }
          const unsigned long long bad = bad_rows[vpar * VS + vslot];
          if (bad) {  // infinities and NaN of drafted tokens, to the rows that attend them
            tc_fence_after();
            tree_add_bad<DT, D>(p, table, it.kv, t0, bad, live ? seen : 0ull, lanes + w * D);
            tc_fence_before();
          }
        }
      }
      if (stop) break;
      for (int tile = mk0, slot = (n + mk0 - it.tile0) % VS; tile < it.tile1; ++tile) {
        clean ^= 1u << slot;
        if (++slot == VS) slot = 0;
      }
      n += it.tile1 - it.tile0;
      // the item's end: O is complete; join the streams; write the rows
      if (first < it.tile1 && !wait(&pv_done[2 * w + ((ns - 1) & 1)], ((ns - 1) >> 1) & 1)) break;
      tc_fence_after();
      float M = m_ref, L = l, f0 = 1.f, f1 = 0.f;
      const bool join2 = NS == 2 && !two, second = join2 && it.tile1 - it.tile0 >= 2;
      if (join2) {
        // (a stream without a tile here has nothing to say, and is ahead: the last item's values may still be read)
        if (first < it.tile1) ml[w * 128 + r] = make_float2(m_ref, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full);
        if (!wait(ml_full, joined & 1)) break;
        ++joined;
        tc_fence_after();
        const float2 a = ml[r], b = ml[128 + r];
        M = second ? fmaxf(a.x, b.x) : a.x;
        const float ref = M == NEG_INF ? 0.f : M;
        f0 = exp2f(a.x - ref);
        f1 = second ? exp2f(b.x - ref) : 0.f;
        L = second ? fmaf(a.y, f0, b.y * f1) : a.y * f0;
      }
      const bool whole = it.tile0 == 0 && it.tile1 == it.tiles;
      if (warp_live) {
        const float inv = !whole ? 1.f : (L == 0.f ? 0.f : 1.f / L);
        const uint64_t g0 = pair2(f0 * inv, f0 * inv), g1 = pair2(f1 * inv, f1 * inv);
        const int row = row0 + r;
        float* slot = tree_slot<D>(p, blockIdx.x, it.tile0 == 0 ? 1 : 0);
        OT* dst = static_cast<OT*>(p.out) +
                  ((long long)(it.q0 + node) * p.H + it.kv * p.group + row % p.group) * D;
        // a joined item's columns are shared out between the streams
        const int cb = join2 ? w * (D / 2) : 0, ce = join2 ? cb + D / 2 : D;
        // (16 columns at a time: the code runs once an item, and its length is paid in instruction-cache misses)
#pragma unroll 1
        for (int c0 = cb; c0 < ce; c0 += 16) {
          uint32_t o[16], x[16];
          tc_ld16_pair(lanes + (join2 ? 0 : w * D) + c0, lanes + (NS - 1) * D + c0, o, x);
          uint64_t y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = mul2(pair2(o[2 * e], o[2 * e + 1]), g0);
            if (second) y[e] = fma2(pair2(x[2 * e], x[2 * e + 1]), g1, y[e]);
          }
          if (!live) continue;
          float a, c;
          if (whole && sizeof(OT) == 2) {
            uint32_t z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              unpair2(y[e], a, c);
              z[e] = Mma<DT>::pack(a, c);  // (a 16-bit output has the cache's type)
            }
            uint4* to = reinterpret_cast<uint4*>(dst + c0);
            to[0] = make_uint4(z[0], z[1], z[2], z[3]);
            to[1] = make_uint4(z[4], z[5], z[6], z[7]);
          } else {
            float4* to = whole ? reinterpret_cast<float4*>(dst + c0)
                               : reinterpret_cast<float4*>(slot + 2 * p.slot_rows) + (long long)(c0 / 4) * p.slot_rows + row;
            const long long step = whole ? 1 : p.slot_rows;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float4 f;
              unpair2(y[2 * e], f.x, f.y);
              unpair2(y[2 * e + 1], f.z, f.w);
              to[e * step] = f;
            }
          }
        }
        if (!whole && live && (!join2 || w == 0)) reinterpret_cast<float2*>(slot)[row] = make_float2(M, L);
      }
      if (!whole && it.tile0 == 0 && warp == 0 && lane == 0)
        p.join[blockIdx.x] = TreeJoin{walk.last_cta(it), it.q0, it.rows, it.kv};
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
  }

  // every role has stopped: release the tensor memory
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == SW + 2)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(C::COLS) : "memory");
}

}  // namespace pa
