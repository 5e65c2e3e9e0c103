// Attention on the 5th-generation tensor cores (tcgen05), sm_103a:
//
//   S = Q.K^T  ->  P = 2^(c S - c m), l = sum P, rounded  ->  O = P.V / l
//
// the cascade (A.B).C of this library with a softmax as the step between the
// two GEMMs.  Scores and probabilities never leave the SM: S is a tcgen05
// accumulator in tensor memory (row = lane, key = column, fp32), each softmax
// thread reads its row, and the 16-bit P goes back into the same columns as
// the A operand of the second GEMM.
//
// Online softmax (c = scale * log2 e): a row keeps a reference m and
// l = sum_j 2^(c s_j - c m); O accumulates sum_j 2^(c s_j - c m) v_j in
// tensor memory.  m is the first tile's maximum and is moved only when a
// later maximum exceeds it by more than 8 in the exponent (kAttnRescale), so P
// stays below 2^8 (exact powers apart, the relative rounding of P and the
// fp32 sums do not depend on m) and O is rarely rescaled.  A masked score
// counts as -inf whatever it holds; a row that has seen no key keeps
// m = -inf, l = 0 and gives zeros.
//
// Work items.  An item is one key/value head, one block of query tokens and a
// range of 128-key tiles.  The rows of a 128-row tile are (token, head of the
// group), token-major, so that the heads that share a key/value head share
// its loads and a single token still fills several rows.  Two streams
// (softmax warpgroup, MMA-issuing thread, S and O accumulators each) run per
// CTA, so that one stream's softmax overlaps the other's MMAs:
//   pair items: stream t has rows of its own (tile t of the block), both
//               read every key tile;
//   solo items (rows for one tile only): both streams hold the same rows and
//               take the key tiles alternately; their results are joined at
//               the end.
// Long key ranges with few rows are split over items; such an item writes its
// unnormalised O with (c m, l) as one part, and attn_combine_kernel joins the
// parts in a fixed order.
//
// CTA roles (512 threads, one CTA per SM; items handed out by cluster launch
// control, so a CTA that finishes early takes the next unstarted item):
//   warps 0-3, 4-7  softmax of stream 0 and 1 (a row per thread)
//   warps 8, 9      MMA issue of stream 0 and 1
//   warp 10         TMA loads of keys, values and queries
//   warp 11         items: asks for them and decodes them ahead of the loads
//   warps 12-15     epilogue of both streams, beside the next item's softmax
// Every wait is bounded, as in the chain kernels.
//
// What bounds it (on a GB300, a call among others): long 128-wide prompts the
// tensor pipe under the power cap (8192 tokens, 32/8 heads, bf16: 352-364 us on
// several GPUs, 1.51-1.56 PFLOP/s, pipe 72 % busy); long 64-wide ones the
// softmax's chain from scores to P (12001 tokens, 16/4 heads, fp16: 276-282 us,
// 1.05-1.07 PFLOP/s); batches on a long prefix memory (32 requests on 65,521
// keys: 58 us, 5.5 TB/s; 200 requests with keys of their own: 144 us, 5.8
// TB/s); short prompts the latencies of an item (24 prompts of 1-700 tokens:
// 55 us against 26 at the measured rates).
#pragma once

#include <cuda.h>
#include <cstdint>

#include "chain_tc.cuh"
#include "ptx.cuh"

namespace b2b {

constexpr int kAttnThreads = 512;
// registers of a softmax, an epilogue and another thread: 128 of each thread at launch, shared out anew
constexpr int kAttnSoftmaxRegs = 160, kAttnEpilogueRegs = 96, kAttnOtherRegs = 96;
static_assert(256 * kAttnSoftmaxRegs + 128 * kAttnEpilogueRegs + 128 * kAttnOtherRegs <= 65536, "register file");
constexpr int kAttnTile = 128;        // query rows and keys of a tile
constexpr int kAttnItems = 3;         // item descriptors in flight
constexpr float kAttnRescale = 8.0f;  // exponent (base 2) by which a maximum may exceed its reference

// Ring of key and value tiles, and the shared-memory layout, by padded head size.
template <int DP>
struct AttnShape {
  static constexpr int kPanels = DP / 64;                    // 128-byte column panels of a tile
  static constexpr int kTileBytes = kPanels * kPanelBytes;   // one Q, K or V tile
  static constexpr int kRing = DP == 128 ? 5 : 8;
  static constexpr int kOffRing = 2 * kTileBytes;
  static constexpr int kOffBar = kOffRing + kRing * kTileBytes;
  static constexpr int kOffItems = kOffBar + 512;
  static constexpr int kOffExchange = kOffItems + kAttnItems * 64;
  static constexpr int kOffClaimed = kOffExchange + 2 * kAttnTile * 8;  // an item claimed but handed to no role
  static constexpr int kBytes = kOffClaimed + 64;
  static_assert(kBytes <= 232448, "shared memory of a CTA");
};

enum : int {  // barrier slots (8 bytes each)
  kABFull = 0,        // [8] ring tile landed
  kABEmpty = 8,       // [8] ring tile read by both streams
  kABQFull = 16,      // [2] stream's query tile landed
  kABQEmpty = 18,     // [2] stream's query tile read
  kABSFull = 20,      // [2] stream's scores computed
  kABPFull = 22,      // [2][2] halves of a stream's probabilities written (and O rescaled)
  kABOFull = 26,      // [2] stream's O complete
  kABMlFull = 45,     // [2] stream's (m, l) written
  kABMlEmpty = 47,    // [2] stream's (m, l) read
  kABOEmpty = 49,     // [2] stream's O read
  kABTurn = 54,       // [2] the stream may compute its next exponentials
  kABAsk = 40,        // an item's loads are nearly all issued
  kABTail = 51,       // [3] last value tile landed (one arrival per item)
  kABItemFull = 28,   // [3] descriptor written
  kABItemEmpty = 31,  // [3] descriptor no longer read
  kABFixed = 34,      // [3] last value tile's rows past its last key zeroed
  kABNext = 37,       // next item handed out
  kABDrain = 38,      // [2]
  kASlotNext = 42,    // 16 bytes: cluster launch control's answer
  kASlotTmem = 44,    // uint32 tensor-memory base, then the int abort flag
};

enum : int { kAttnPrompt = 0, kAttnShared = 1 };

// Division of 0 <= x < 2^31 by a number fixed at launch: floor(x mul / 2^32) >> shift
// with mul = ceil(2^(31 + bits) / d), bits = ceil(log2 d), is exact for such x.
struct FastDiv {
  uint32_t d, mul, shift;
  static FastDiv of(uint32_t d) {
    uint32_t bits = 0;
    while ((uint64_t(1) << bits) < d) ++bits;
    if (bits == 0) return {1, 0, 0};
    return {d, static_cast<uint32_t>(((uint64_t(1) << (31 + bits)) + d - 1) / d), bits - 1};
  }
  // Quotient; x becomes the remainder.
  __device__ __forceinline__ int split(int& x) const {
    if (d == 1) {
      const int q = x;
      x = 0;
      return q;
    }
    const uint32_t q = __umulhi(static_cast<uint32_t>(x), mul) >> shift;
    x -= static_cast<int>(q * d);
    return static_cast<int>(q);
  }
  __device__ __forceinline__ int quotient(int x) const { return split(x); }
};

struct AttnParams {
  int op;
  int group, kv_heads, dim;
  FastDiv by_group, by_tokens, by_kv_heads, by_block, by_splits, by_row_blocks, by_own_splits, by_own_blocks;  // (by_block: tokens of an item)
  int tile_tokens;     // query tokens of a 128-row tile: 128 / group
  int tokens;          // query rows of the packed query tensor
  int batch;           // sequences or requests
  int causal;          // prompt: causal; (own keys of shared items always are)
  // prompt
  const int* cu_q;
  const int* cu_k;
  int key_rows;
  int most_tiles;      // no sequence has more key tiles
  // shared prefix
  int fresh;           // new tokens per request
  int prefix;          // keys of the prefix
  int prefix_items, block_tokens;
  int whole;           // an item of own keys begins with the prefix's: one part, nothing to join
  const int* lengths;
  const int* table;    // pages of the requests' own keys, or null (dense)
  int table_width, page_shift, room;
  // TMA boxes: key rows of one box in the prompt/prefix and own tensors, bytes of a query box
  int box_rows, own_box_rows;
  uint32_t q_bytes, own_q_bytes;
  // outputs: final (parts == 1) or parts
  float scale_log2, scale;
  void* out;
  long long out_row, out_head;  // element strides
  float* lse;
  long long lse_row, lse_head;
  int wide_stores;     // rows of `out` on 32-byte boundaries: 32-byte stores
  int parts;
  int join_warps;      // warps that share a row's parts when they are joined (1, 2, 4 or 8)
  // Rows of the parts are numbered (key/value head, token, head of the group),
  // as the lanes of a tile hold them: a warp's stores are consecutive.
  float* part_o;       // [parts][dim / 8][rows][8]
  float2* part_ml;     // [parts][rows]: (c m, l)
  uint32_t debug;      // bit 0: arm the first ring tile but never fill it
  int* status;
  uint32_t budget_ns;
};

struct AttnItem {
  int kind;       // 0 prompt, 1 prefix, 2 own keys, -1 no more items
  int solo;
  int head;       // key/value head
  int tok0, ntok; // first query token, valid tokens of the block
  int vis0, klen; // keys the first token sees (may be negative), all keys
  int causal;     // token i sees clamp(vis0 + i, 0, klen) keys, else klen
  int krow;       // first row of the sequence's keys, or the request
  int j0, n, n0;  // first key tile, tiles of stream 1 (solo: of both), tiles of stream 0
  int last;       // keys from the first of these tiles (past the prefix's) on that any row sees
  int fix;        // rows of the last tile that hold keys (0: all of them)
  int part;
  int pre;        // tiles of the prefix in front of the request's own (items of whole requests)
};
static_assert(sizeof(AttnItem) == 64, "descriptor slot");

namespace attn {

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
template <int R>
__device__ __forceinline__ void set_max_regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_max_regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// As BoundedWait, in fewer instructions (a 32-bit clock, the status word
// written once at the kernel's end): the roles' code together has to stay in
// the instruction cache.  With BoundedWait in every wait it was 84 KB, and a
// fifth of the warps' time on short prompts went by waiting for instructions.
struct Wait {
  volatile int* abort_flag;
  uint32_t budget_ns;
  __device__ __forceinline__ static uint32_t now() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
  }
  // By one thread.
  __device__ __forceinline__ bool wait1(uint32_t bar, uint32_t parity) const {
    const uint32_t t0 = now();
    while (!ptx::mbar_try_wait(bar, parity)) {
      if (*abort_flag) return false;
      if (now() - t0 >= budget_ns) *abort_flag = 1;
    }
    return true;
  }
  // By a whole warp; every lane gets the same answer, so that no lane goes on
  // to a warp-wide instruction without the others.
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait1(bar, parity));
  }
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }
// Keys that token i of the item's block sees.
__device__ __forceinline__ int visible(const AttnItem& a, int i) {
  return a.causal ? clampi(a.vis0 + i, 0, a.klen) : a.klen;
}
// Position in the ring of key and value tile j of an item with n tiles: the
// two streams' first key tiles, then value and key tiles in turn.
__device__ __forceinline__ uint32_t key_pos(int j) { return static_cast<uint32_t>(j < 2 ? j : 2 * j - 1); }
__device__ __forceinline__ uint32_t value_pos(int j, int n) { return static_cast<uint32_t>(j + min(n, j + 2)); }

// Key and value tiles of an item in ring order.
struct RingWalk {
  int n, keys = 0, values = 0, j = 0;
  __device__ __forceinline__ explicit RingWalk(int tiles) : n(tiles) {}
  // Moves to the next position: true for key tile j, false for value tile j.
  __device__ __forceinline__ bool next() {
    const bool is_key = keys < n && (keys < 2 || keys <= values + 1);
    j = is_key ? keys++ : values++;
    return is_key;
  }
};

// A sequence's query and key rows, inside the tensors whatever the offsets say.
struct AttnSeq {
  int q0, qlen, k0, klen, blocks;
};
__device__ __forceinline__ AttnSeq load_seq(const AttnParams& p, int b) {
  AttnSeq s = {0, 0, 0, 0, 0};
  if (p.op == kAttnPrompt && b < p.batch) {
    const int q = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1), k = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
    s.q0 = clampi(q, 0, p.tokens);
    s.qlen = clampi(q1, s.q0, p.tokens) - s.q0;
    s.k0 = clampi(k, 0, p.key_rows);
    s.klen = clampi(k1, s.k0, p.key_rows) - s.k0;
    s.blocks = p.by_block.quotient(s.qlen + static_cast<int>(p.by_block.d) - 1);
  }
  return s;
}

// Where the last item of a prompt was found.  The blocks that see n key tiles
// have the numbers first .. end - 1; `before` of these belong to the sequences
// before seq0, a multiple of 32; `all` counts every block (-1: not known yet).
struct AttnCursor {
  int n = 0, first = 0, end = 0, seq0 = 0, before = 0, all = -1;
};

// Fill `a` for item number x (whole warp; every lane gets the same).  False: no such item.
// mine: the lane's sequence, load_seq(p, lane), of a prompt.
__device__ __forceinline__ bool decode_item(const AttnParams& p, int x, int lane, const AttnSeq& mine, AttnCursor& c,
                                            AttnItem& a) {
  const int block = static_cast<int>(p.by_block.d);
  const FastDiv* by_splits = &p.by_splits;
  if (p.op == kAttnPrompt) {
    int u = p.by_splits.split(x);
    a.part = x;
    x = u;
    u = p.by_kv_heads.split(x);
    a.head = x;
    // Blocks in the order of the key tiles they see, the most first: the
    // longest items are best begun first.  count(s, n) of a sequence's blocks
    // see n tiles or more, its last ones under a causal mask, where block k sees
    // klen - qlen + min((k + 1) block, qlen) keys.  The item's n is the largest
    // for which the sequences' counts together exceed u.
    auto count = [&](const AttnSeq& s, int n) -> int {
      const int keys = (n - 1) * kAttnTile + 1;  // n tiles from so many keys on
      if (n == 0) return s.blocks;
      if (s.klen < keys) return 0;
      if (!p.causal) return s.blocks;
      const int rows = max(keys - (s.klen - s.qlen), 0);  // rows of the sequence before its blocks see that many
      return s.blocks - max(p.by_block.quotient(rows + block - 1) - 1, 0);
    };
    auto counts = [&](int n) -> int {
      int sum = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < p.batch; b0 += 32) sum += count(b0 ? load_seq(p, b0 + lane) : mine, n);
      return __reduce_add_sync(0xffffffffu, sum);
    };
    // A search reads every sequence once a step, so a CTA's next item, whose
    // number is mostly a little higher, is looked for from the last one on (200
    // prompts of 20-200 tokens, 32/8 heads: 273 -> 126 us; 1000: 6,120 -> 660 us).
    if (u < c.first || u >= c.end) {
      if (c.all < 0) {
        // No block sees more tiles than the longest sequence has, which spares
        // steps of the first search, the one the kernel's start waits for (24
        // prompts of 1-700 tokens 55.6 -> 55.1 us, 1000 of 20-200 660 -> 535 us).
        int sum = 0, keys = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
          const AttnSeq s = b0 ? load_seq(p, b0 + lane) : mine;
          sum += s.blocks;
          keys = max(keys, s.klen);
        }
        c.all = __reduce_add_sync(0xffffffffu, sum);
        c.n = (__reduce_max_sync(0xffffffffu, keys) + kAttnTile - 1) / kAttnTile + 1;
      }
      if (u >= c.all) return false;
      int lo = 0, hi = c.n, more = c.end, all = c.all;  // counts(lo) = all > u >= counts(hi) = more
      if (u < c.first) {
        hi = p.most_tiles + 1;
        more = 0;
      }
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2, n = counts(mid);
        if (n > u) {
          lo = mid;
          all = n;
        } else {
          hi = mid;
          more = n;
        }
      }
      c = {lo, more, all, 0, 0, c.all};
    } else if (u < c.first + c.before) {
      c.seq0 = c.before = 0;
    }
    u -= c.first + c.before;  // among the blocks that see just that many, of the sequences from seq0 on
    AttnSeq q = mine;
    int at = 0;
#pragma unroll 1
    for (; c.seq0 < p.batch; c.seq0 += 32) {
      if (c.seq0) q = load_seq(p, c.seq0 + lane);
      const int from = count(q, c.n), here = from - count(q, c.n + 1);
      int sum = here;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, sum > u);
      if (past) {
        const int l = __ffs(past) - 1;
        at = __shfl_sync(0xffffffffu, q.blocks - from + u - (sum - here), l) * block;
        q.q0 = __shfl_sync(0xffffffffu, q.q0, l);
        q.qlen = __shfl_sync(0xffffffffu, q.qlen, l);
        q.k0 = __shfl_sync(0xffffffffu, q.k0, l);
        q.klen = __shfl_sync(0xffffffffu, q.klen, l);
        break;
      }
      const int skipped = __shfl_sync(0xffffffffu, sum, 31);
      u -= skipped;
      c.before += skipped;
    }
    a.kind = 0;
    a.tok0 = q.q0 + at;
    a.ntok = min(block, q.qlen - at);
    a.causal = p.causal;
    a.vis0 = q.klen - q.qlen + at + 1;
    a.klen = q.klen;
    a.krow = q.k0;
  } else if (x < p.prefix_items) {
    // row blocks of the same keys next to each other: they share them in L2
    int u = p.by_row_blocks.split(x);
    a.tok0 = x * p.block_tokens;
    a.head = p.by_splits.split(u);
    a.part = u;
    a.kind = 1;
    a.ntok = min(p.block_tokens, p.tokens - a.tok0);
    a.causal = 0;
    a.vis0 = 0;
    a.klen = p.prefix;
    a.krow = 0;
  } else {
    x -= p.prefix_items;
    by_splits = &p.by_own_splits;
    int u = p.by_own_splits.split(x);
    a.part = x;
    int v = p.by_kv_heads.split(u);
    a.head = u;
    const int b = p.by_own_blocks.split(v);
    const int at = v * block;
    const int len = clampi(__ldg(p.lengths + b), 0, p.room);
    a.kind = 2;
    a.tok0 = b * p.fresh + at;
    a.ntok = min(block, p.fresh - at);
    a.causal = 1;
    a.vis0 = len - p.fresh + at + 1;
    a.klen = len;
    a.krow = b;
  }
  a.solo = a.ntok <= p.tile_tokens;
  a.pre = a.kind == 2 && p.whole ? (p.prefix + kAttnTile - 1) / kAttnTile : 0;
  const int seen = visible(a, a.ntok - 1);
  const int all = (seen + kAttnTile - 1) / kAttnTile;
  const int chunk = by_splits->quotient(all + static_cast<int>(by_splits->d) - 1);
  a.j0 = a.part * chunk;
  const int n = clampi(all - a.j0, 0, chunk);
  const int all0 = (visible(a, min(a.ntok, p.tile_tokens) - 1) + kAttnTile - 1) / kAttnTile;
  a.n = a.pre + n;
  a.n0 = a.solo ? (a.n + 1) / 2 : a.pre + clampi(all0 - a.j0, 0, n);
  a.last = min(seen - a.j0 * kAttnTile, n * kAttnTile);
  // (a prefix's last tile needs no zeroing: its tensor ends there, and TMA
  // fills what lies past it with zeros)
  a.fix = n > 0 && a.kind != 1 ? a.last % kAttnTile : 0;
  if (a.kind == 2 && p.prefix_items) a.part += static_cast<int>(p.by_splits.d);
  return true;
}

// Marks the rows of parts that a CTA has claimed and may not have written (no
// healthy part has l < 0), so that they are not joined: the workspace holds
// whatever was there before, an earlier run's parts perhaps.  A call of its
// own, which leaves the code of the roles' loops as it is.
inline __device__ __noinline__ void give_up_parts(float2* part_ml, const AttnItem* items, const AttnItem* claimed,
                                                  int kv_heads, int tokens, int group) {
  for (int s = 0; s <= kAttnItems; ++s) {
    const AttnItem& a = s < kAttnItems ? items[s] : *claimed;
    if (a.kind < 0) continue;
    float2* rows = part_ml + ((static_cast<long long>(a.part) * kv_heads + a.head) * tokens + a.tok0) * group;
    for (int i = static_cast<int>(threadIdx.x); i < a.ntok * group; i += kAttnThreads) rows[i] = make_float2(0.0f, -1.0f);
  }
}

// Key tiles of stream t.
__device__ __forceinline__ int stream_tiles(const AttnItem& a, int t) {
  return t == 0 ? a.n0 : (a.solo ? a.n / 2 : a.n);
}

}  // namespace attn

// BF16: bf16 operands, else fp16.  DP: padded head size, 64 or 128 (TMA fills
// the columns past the head size with zeros).
template <bool BF16, int DP>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_q_own,
                const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ CUtensorMap tm_k_own, const __grid_constant__ CUtensorMap tm_v_own,
                const __grid_constant__ AttnParams p) {
  using namespace ptx;
  using namespace attn;
  using L = AttnShape<DP>;
  constexpr uint32_t kRing = L::kRing;
  constexpr uint32_t kFmt = BF16 ? 1u : 0u;
  constexpr uint32_t kColO = 256;  // tensor memory: S0/P0 at 0, S1/P1 at 128, then O0, O1

  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // (every byte is used: the swizzled tiles need a base on 1024 bytes, which
  // dynamic shared memory has when a kernel has no other; checked below)
  const uint32_t base = smem_u32(smem_raw);
  uint8_t* gbase = smem_raw;
  const uint32_t bar0 = base + L::kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kOffBar + 8 * kASlotTmem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  AttnItem* items = reinterpret_cast<AttnItem*>(gbase + L::kOffItems);
  AttnItem* claimed = reinterpret_cast<AttnItem*>(gbase + L::kOffClaimed);
  float2* exchange = reinterpret_cast<float2*>(gbase + L::kOffExchange);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;

  if (base & 1023u) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kTimeoutCode);
    return;
  }
  if (warp == 0) {
    if (lane < 8) {
      mbar_init(bar(kABFull + lane), 1);
      mbar_init(bar(kABEmpty + lane), 2);
    } else if (lane < 10) {
      const int t = lane - 8;
      mbar_init(bar(kABQFull + t), 1);
      mbar_init(bar(kABQEmpty + t), 1);
      mbar_init(bar(kABSFull + t), 1);
      mbar_init(bar(kABPFull + 2 * t), 4);
      mbar_init(bar(kABPFull + 2 * t + 1), 4);
      mbar_init(bar(kABOFull + t), 1);
      mbar_init(bar(kABMlFull + t), 4);
      mbar_init(bar(kABMlEmpty + t), 4);
      mbar_init(bar(kABOEmpty + t), 4);
      mbar_init(bar(kABTurn + t), 4);
      mbar_init(bar(kABDrain + t), 1);
    } else if (lane < 10 + kAttnItems) {
      const int s = lane - 10;
      mbar_init(bar(kABItemFull + s), 1);
      mbar_init(bar(kABItemEmpty + s), 15);  // 8 softmax and 4 epilogue warps, 2 MMA warps, the loader
      mbar_init(bar(kABFixed + s), 4);
      mbar_init(bar(kABTail + s), 1);
    } else if (lane == 13) {
      mbar_init(bar(kABNext), 1);
      mbar_init(bar(kABAsk), 1);
      *abort_flag = 0;
    } else if (lane < 14 + kAttnItems) {
      items[lane - 14].kind = -1;
    } else if (lane == 14 + kAttnItems) {
      claimed->kind = -1;
    }
    if (lane < 14) fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Wait bw{abort_flag, p.budget_ns};
  grid_launch_dependents();

  if (warp < 8) {
    // -------------------------------------------------------------- softmax
    set_max_regs_up<kAttnSoftmaxRegs>();
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int row_tok = row / p.group;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lane_off + 128u * static_cast<uint32_t>(t);
    const uint32_t to = tmem + lane_off + kColO + static_cast<uint32_t>(DP * t);
    const float sl2 = p.scale_log2;
    const uint64_t sl2x2 = pack2(sl2, sl2);
    uint32_t nscore = 0, nml = 0, nturn = 0;
    grid_dependency_wait();  // (the waits below are for this run's work, not for the kernel before)
    for (uint32_t it = 0;; ++it) {
      const uint32_t islot = it % kAttnItems;
      if (!bw.wait(bar(kABItemFull + islot), (it / kAttnItems) & 1u)) break;
      const AttnItem a = items[islot];
      if (a.kind < 0) break;
      const int cnt = stream_tiles(a, t);
      const int tile0 = a.solo ? 0 : t * p.tile_tokens;  // first token of this stream's tile
      // In the tiles that both streams of a pair item have (stream 0 has no
      // more than stream 1) they take turns at the exponentials, which keeps
      // them half a tile apart, one in its MMAs while the other has the
      // exponential unit: 128-wide heads, 8192 tokens: 375 -> 358 us.  64-wide
      // ones, bound by the softmax, lose by it (284 -> 297 us).
      const int common = DP < 128 || a.solo ? 0 : a.n0;
      const int vis = visible(a, tile0 + row_tok);
      const int vis_min = __shfl_sync(0xffffffffu, vis, 0);  // the warp's first row sees the fewest
      // Rows that hold no query of the item (other queries, or what lay there
      // before) have no say in when the warp's rows are rescaled.
      const bool query = row_tok < p.tile_tokens && tile0 + row_tok < a.ntok;
      float m = -INFINITY;
      uint64_t l2 = 0;
      bool ok = true;
      for (int i = 0; i < cnt; ++i) {
        const int j = a.solo ? 2 * i + t : i;
        const int key = (j < a.pre ? j : a.j0 + j - a.pre) * kAttnTile;  // the tile's first
        if (!bw.wait(bar(kABSFull + t), nscore & 1u)) {
          ok = false;
          break;
        }
        ++nscore;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32u * c, s[c]);
        tmem_wait_ld();
        const int lim_min = (j < a.pre ? p.prefix : vis_min) - key;
        if (lim_min < kAttnTile) {
          const int lim = (j < a.pre ? p.prefix : vis) - key;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c * 32 + 32 > lim_min) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (c * 32 + k >= lim) s[c][k] = 0xff800000u;  // -inf
            }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
          for (int k = 1; k < 31; k += 2)
            mx[c] = fmaxf(fmaxf(mx[c], __uint_as_float(s[c][k])), __uint_as_float(s[c][k + 1]));
          mx[c] = fmaxf(mx[c], __uint_as_float(s[c][31]));
        }
        const float tile_max = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (i == 0) {
          m = tile_max;
        } else if (__any_sync(0xffffffffu, query && (tile_max - m) * sl2 > kAttnRescale)) {
          // S complete implies the MMAs before it: O holds every earlier tile
          // and nothing writes it until this tile's P is handed over.
          const float m_new = fmaxf(m, tile_max);
          const float f = m_new == m ? 1.0f : exp2_approx((m - m_new) * sl2);
          m = m_new;
          float la, lb;
          unpack2(l2, la, lb);
          l2 = pack2(la * f, lb * f);
#pragma unroll 1
          for (int c = 0; c < DP / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(to + 16u * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st16(to + 16u * c, o);
          }
        }
        const float mc = m == -INFINITY ? 0.0f : m * sl2;
        const uint64_t mcx2 = pack2(-mc, -mc);
        if (i < common) {
          if (!(ok = bw.wait(bar(kABTurn + t), (nturn & 1u) ^ (t == 0)))) break;
          ++nturn;
        }
        // P in two halves of 64 keys, so that the second GEMM starts on the
        // first while the second is computed; the row's sum afterwards.
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float x0, x1;
            unpack2(fma2(pack2(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), sl2x2, mcx2), x0, x1);
            x0 = exp2_approx(x0);
            x1 = exp2_approx(x1);
            s[c][2 * k] = __float_as_uint(x0);
            s[c][2 * k + 1] = __float_as_uint(x1);
            w[k] = BF16 ? pack_bf16x2(s[c][2 * k], s[c][2 * k + 1]) : pack_f16x2(s[c][2 * k], s[c][2 * k + 1]);
          }
          tmem_st16(ts + 16u * c, w);
          if (c & 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(kABPFull + 2 * t + c / 2));
              if (c == 3 && i < common) mbar_arrive(bar(kABTurn + 1 - t));
            }
          }
        }
        uint64_t sums[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          sums[c] = pack2(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
          for (int k = 2; k < 32; k += 2)
            sums[c] = add2(sums[c], pack2(__uint_as_float(s[c][k]), __uint_as_float(s[c][k + 1])));
        }
        l2 = add2(l2, add2(add2(sums[0], sums[1]), add2(sums[2], sums[3])));
      }
      if (!ok) break;
      if (cnt > 0) {
        if (!bw.wait(bar(kABMlEmpty + t), (nml & 1u) ^ 1u)) break;
        ++nml;
        float la, lb;
        unpack2(l2, la, lb);
        exchange[t * kAttnTile + row] = make_float2(m, la + lb);
      }
      __syncwarp();
      if (lane == 0) {
        if (cnt > 0) mbar_arrive(bar(kABMlFull + t));
        mbar_arrive(bar(kABItemEmpty + islot));
      }
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------- epilogue
    set_max_regs_down<kAttnEpilogueRegs>();
    const int row = (warp & 3) * 32 + lane;
    const int row_tok = row / p.group;
    const int row_head = row - row_tok * p.group;
    const uint32_t to0 = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kColO;
    const float sl2 = p.scale_log2;
    const long long part_rows = static_cast<long long>(p.tokens) * (p.group * p.kv_heads);
    uint32_t nout[2] = {0, 0}, ring = 0;
    grid_dependency_wait();  // (the outputs may still be read by the kernel before)
    bool ok = true;
    for (uint32_t it = 0; ok; ++it) {
      const uint32_t islot = it % kAttnItems;
      if (!bw.wait(bar(kABItemFull + islot), (it / kAttnItems) & 1u)) break;
      const AttnItem a = items[islot];
      if (a.kind < 0) break;
      // The rows of the last value tile past its last key become zeros: another
      // sequence's values may lie there, or NaN, and 0 x NaN is not 0.
      if (!(ok = bw.wait(bar(kABTail + islot), (it / kAttnItems) & 1u))) break;
      if (a.fix) {
        const uint32_t dst =
            base + L::kOffRing + ((ring + value_pos(a.n - 1, a.n)) % kRing) * L::kTileBytes;
#pragma unroll 1
        for (int e = a.fix * 8 + static_cast<int>(threadIdx.x & 127u); e < kAttnTile * 8; e += 128)
#pragma unroll
          for (int c = 0; c < L::kPanels; ++c)
            st_shared_v4(dst + c * kPanelBytes + static_cast<uint32_t>(e) * 16u, 0, 0, 0, 0);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kABFixed + islot));
      ring += 2u * static_cast<uint32_t>(a.n);
      // (m, l) of stream t's row, once its O is complete
      auto take = [&](int t, float& m, float& l) -> bool {
        m = -INFINITY;
        l = 0.0f;
        if (stream_tiles(a, t) == 0) return true;
        if (!bw.wait(bar(kABMlFull + t), nout[t] & 1u)) return false;
        const float2 ml = exchange[t * kAttnTile + row];
        m = ml.x;
        l = ml.y;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kABMlEmpty + t));
        if (!bw.wait(bar(kABOFull + t), nout[t] & 1u)) return false;
        ++nout[t];
        tc_fence_after();
        return true;
      };
      auto drained = [&](int t) {  // this warp's rows of stream t's O are read
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && stream_tiles(a, t) > 0) mbar_arrive(bar(kABOEmpty + t));
      };
      for (int t = 0; t < (a.solo ? 1 : 2) && ok; ++t) {
        float m, l;
        ok = take(t, m, l);
        // Solo items with work in both streams: the two O of a row are joined.
        const bool join = a.solo && a.n > 1;
        float f0 = 1.0f, f1 = 0.0f;
        if (ok && join) {
          float m1, l1;
          ok = take(1, m1, l1);
          const float m_new = fmaxf(m, m1);
          f0 = m == m_new ? 1.0f : exp2_approx((m - m_new) * sl2);
          f1 = m1 == m_new ? 1.0f : exp2_approx((m1 - m_new) * sl2);
          m = m_new;
          l = l * f0 + l1 * f1;
        }
        if (!ok) break;
        const int tile0 = a.solo ? 0 : t * p.tile_tokens;
        const bool valid = row_tok < p.tile_tokens && tile0 + row_tok < a.ntok;
        const int token = a.tok0 + tile0 + row_tok;
        const int head = a.head * p.group + row_head;
        const bool some = stream_tiles(a, t) > 0;
        const bool part = p.parts > 1;
        const float inv = 1.0f / l;
        const long long prow = (static_cast<long long>(a.head) * p.tokens + token) * p.group + row_head;
        float* pdst = p.part_o + (static_cast<long long>(a.part) * (p.dim / 8) * part_rows + prow) * 8;
        uint16_t* dst = static_cast<uint16_t*>(p.out) + token * p.out_row + head * p.out_head;
        if (valid) {
          if (part)
            p.part_ml[a.part * part_rows + prow] = make_float2(m * sl2, l);
          else if (p.lse)
            p.lse[token * p.lse_row + head * p.lse_head] = l == 0.0f ? -INFINITY : m * p.scale + logf(l);
        }
        // 32 columns of the row: independent work enough for one warp, code
        // short enough for the instruction cache (16 columns at a time took
        // 2 us a tile, one instruction after the other).
        const bool none = __any_sync(0xffffffffu, l == 0.0f);
        const uint64_t invx2 = pack2(inv, inv), f0x2 = pack2(f0, f0), f1x2 = pack2(f1, f1);
        auto emit = [&](int col, uint32_t (&o)[32]) {
          if (part) {
            float* d8 = pdst + static_cast<long long>(col / 8) * part_rows * 8;
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
              uint32_t v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) v[e] = o[k + e];
              if (valid && col + k < p.dim) st_global_v8(d8 + (k / 8) * part_rows * 8, v);
            }
            return;
          }
          uint32_t v[2][8];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x, y;
            unpack2(mul2(pack2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), invx2), x, y);
            v[e / 8][e % 8] = BF16 ? pack_bf16x2(__float_as_uint(x), __float_as_uint(y))
                                   : pack_f16x2(__float_as_uint(x), __float_as_uint(y));
          }
          if (none) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e / 8][e % 8] = l == 0.0f ? 0u : v[e / 8][e % 8];
          }
          if (!valid) return;
          if (p.wide_stores) {
            if (col < p.dim) st_global_v8(dst + col, v[0]);
            if (col + 16 < p.dim) st_global_v8(dst + col + 16, v[1]);
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (col + 8 * q < p.dim)
                *reinterpret_cast<uint4*>(dst + col + 8 * q) =
                    make_uint4(v[q / 2][4 * (q % 2)], v[q / 2][4 * (q % 2) + 1], v[q / 2][4 * (q % 2) + 2], v[q / 2][4 * (q % 2) + 3]);
          }
        };
        const uint32_t to = to0 + static_cast<uint32_t>(DP * t);
        if (some || !part) {  // (a part with l = 0 is not read)
#pragma unroll 1
          for (int col = 0; col < DP; col += 32) {
            uint32_t o[32];
            tmem_ld32(to + static_cast<uint32_t>(col), o);
            if (join) {
              uint32_t o1[32];
              tmem_ld32(to + static_cast<uint32_t>(DP + col), o1);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                float x, y;
                unpack2(fma2(pack2(__uint_as_float(o1[k]), __uint_as_float(o1[k + 1])), f1x2,
                             mul2(pack2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), f0x2)), x, y);
                o[k] = __float_as_uint(x);
                o[k + 1] = __float_as_uint(y);
              }
            } else {
              tmem_wait_ld();
            }
            emit(col, o);
          }
        }
        drained(t);
        if (join) drained(1);
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(bar(kABItemEmpty + islot));
    }
  } else {
    set_max_regs_down<kAttnOtherRegs>();
    if (warp < 10) {
      // ------------------------------------------------------------ MMA issue
      // One elected thread (measured: a warp-wide walk that elects a thread for
      // each group of MMAs issues them a fifth slower).
      const int t = warp - 8;
      grid_dependency_wait();  // (as in the softmax)
      if (elect_one()) {
        const uint32_t d_s = tmem + 128u * static_cast<uint32_t>(t);
        const uint32_t d_o = tmem + kColO + static_cast<uint32_t>(DP * t);
        constexpr uint32_t idesc_qk = make_idesc(kFmt, kAttnTile, 128, false);
        constexpr uint32_t idesc_pv = make_idesc(kFmt, DP, 128, true);
        const uint64_t q_desc = desc_sw128(base + static_cast<uint32_t>(t) * L::kTileBytes, 16u, 1024u);
        const uint64_t k_desc0 = desc_sw128(base + L::kOffRing, 16u, 1024u);
        const uint64_t v_desc0 = desc_sw128(base + L::kOffRing, kPanelBytes, 1024u);
        uint32_t ring = 0, nq = 0, np = 0, no = 0;
        bool ok = true;
        for (uint32_t it = 0; ok; ++it) {
          const uint32_t islot = it % kAttnItems, iphase = (it / kAttnItems) & 1u;
          if (!bw.wait1(bar(kABItemFull + islot), iphase)) break;
          const AttnItem& a = items[islot];
          if (a.kind < 0) break;
          const int n = a.n, fix = a.fix;
          const bool solo = a.solo != 0;
          const int cnt = stream_tiles(a, t);
          // The thread that tells the epilogue's warps, which have the time to
          // zero the tail of the item's last value tile, that it has landed (it
          // reads that tile itself; a tile that needs nothing is told of at
          // once).  A barrier per item slot: a stream can be an item ahead of
          // the other.
          const bool teller = t == (solo ? (n - 1) & 1 : 1);
          if (teller && !fix) mbar_arrive(bar(kABTail + islot));
          // Every ring tile is waited for and released by both streams, in
          // order, whether they use it or not: a stream that skipped uses of
          // a slot could not tell their completions from its own by parity.
          // Each of this stream's value tiles is held until its next key tile
          // (if there is one) has landed too, so that O += P.V and the next S
          // are issued without a wait between them.
          RingWalk w(n);
          int keys = 0, vtile = -1;  // key tiles seen; value tile held
          uint32_t vslot = 0, kslot = 0;
          bool key = false;          // key tile held
          for (int pos = 0; pos < 2 * n; ++pos) {
            const bool is_key = w.next();
            const uint32_t g = ring + static_cast<uint32_t>(pos), slot = g % kRing;
            if (!(ok = bw.wait1(bar(kABFull + static_cast<int>(slot)), (g / kRing) & 1u))) break;
            if (solo ? (w.j & 1) != t : w.j >= cnt) {
              mbar_arrive(bar(kABEmpty + static_cast<int>(slot)));
              continue;
            }
            if (is_key) {
              kslot = slot;
              key = true;
              ++keys;
            } else {
              vslot = slot;
              vtile = w.j;
            }
            if (vtile < 0 ? keys != 1 : !key && keys < cnt) continue;
            if (vtile < 0) {
              if (!(ok = bw.wait1(bar(kABQFull + t), nq & 1u))) break;
              ++nq;
            } else {
              if (fix && vtile == n - 1) {
                if (teller) mbar_arrive(bar(kABTail + islot));
                if (!(ok = bw.wait1(bar(kABFixed + islot), iphase))) break;
              }
              const bool first = vtile < (solo ? 2 : 1);
              if (first) {  // the epilogue has read the item before's O
                if (!(ok = bw.wait1(bar(kABOEmpty + t), (no & 1u) ^ 1u))) break;
                ++no;
              }
              const uint64_t vd = v_desc0 + vslot * (L::kTileBytes >> 4);
#pragma unroll
              for (uint32_t half = 0; half < 2; ++half) {
                if (!(ok = bw.wait1(bar(kABPFull + 2 * t + static_cast<int>(half)), np & 1u))) break;
                tc_fence_after();
#pragma unroll
                for (uint32_t kk = 4 * half; kk < 4 * half + 4; ++kk)
                  mma_ts<false>(d_o, d_s + kk * 8u, vd + kk * (16u * 128u >> 4), idesc_pv, (kk || !first) ? 1u : 0u);
              }
              if (!ok) break;
              ++np;
              tc_commit(bar(kABEmpty + static_cast<int>(vslot)));
              if (!key) tc_commit(bar(kABOFull + t));
              vtile = -1;
            }
            if (key) {
              key = false;
              tc_fence_after();
              const uint64_t kd = k_desc0 + kslot * (L::kTileBytes >> 4);
#pragma unroll
              for (uint32_t kk = 0; kk < DP / 16; ++kk) {
                const uint32_t off = (kk / 4) * (kPanelBytes >> 4) + (kk % 4) * 2;
                mma_ss<false>(d_s, q_desc + off, kd + off, idesc_qk, kk ? 1u : 0u);
              }
              tc_commit(bar(kABSFull + t));
              tc_commit(bar(kABEmpty + static_cast<int>(kslot)));
              if (keys == cnt) tc_commit(bar(kABQEmpty + t));
            }
          }
          if (!ok) break;
          ring += 2u * static_cast<uint32_t>(n);
          mbar_arrive(bar(kABItemEmpty + islot));
        }
        // every MMA issued must be complete before tensor memory is freed
        tc_commit(bar(kABDrain + t));
        drain_wait(bar(kABDrain + t), 0, p.budget_ns);
      }
    } else if (warp == 10) {
      // ------------------------------------------------------------ TMA loads
      if (lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        if (p.op == kAttnShared) {
          prefetch_tmap(&tm_q_own);
          prefetch_tmap(&tm_k_own);
          prefetch_tmap(&tm_v_own);
        }
      }
      grid_dependency_wait();
      uint32_t ring = 0, issued = 0;
      uint32_t nq = 0, used = 0;  // bit t: parity of stream t's query loads, whether it had any
      bool ok = true;
      const int panel = lane & (L::kPanels - 1), box_at = lane / L::kPanels;  // a lane's share of a tile's boxes
      for (uint32_t it = 0; ok; ++it) {
        const uint32_t islot = it % kAttnItems;
        if (!bw.wait(bar(kABItemFull + islot), (it / kAttnItems) & 1u)) break;
        const AttnItem& a = items[islot];
        if (a.kind < 0) break;
        const int n = a.n, head = a.head, last = a.last, krow = a.krow;
        const bool own = a.kind == 2;
        const bool paged = p.table != nullptr;
        const int pre = a.pre, j0 = a.j0;
        RingWalk w(n);
        for (int pos = 0; pos < 2 * n; ++pos) {
          if (pos == 1) {  // the query tiles, behind the first key tile
            const CUtensorMap* qm = own ? &tm_q_own : &tm_q;
#pragma unroll 1
            for (int t = 0; t < 2 && ok; ++t) {
              if (stream_tiles(a, t) == 0) continue;
              if (!(ok = bw.wait(bar(kABQEmpty + t), ((nq >> t) & 1u) ^ 1u))) break;
              nq ^= 1u << t;
              used |= 1u << t;
              if (lane == 0) mbar_arrive_expect_tx(bar(kABQFull + t), own ? p.own_q_bytes : p.q_bytes);
              __syncwarp();
              if (box_at == 0)
                tma_load_4d(base + static_cast<uint32_t>(t) * L::kTileBytes + panel * kPanelBytes, qm, bar(kABQFull + t),
                            panel * 64, 0, head, a.tok0 + (a.solo ? 0 : t * p.tile_tokens));
            }
            if (!ok) break;
          }
          // Near the end of the item's loads warp 11 asks for the next one.
          if (pos == max(2 * n - 4, 0) && lane == 0) mbar_arrive(bar(kABAsk));
          const bool is_k = w.next();
          const uint32_t g = ring + static_cast<uint32_t>(pos), slot = g % kRing;
          if (!(ok = bw.wait(bar(kABEmpty + static_cast<int>(slot)), ((g / kRing) & 1u) ^ 1u))) break;
          const bool from_own = own && w.j >= pre;  // a tile of the requests' own tensors
          const int box = from_own ? p.own_box_rows : p.box_rows;
          // keys of this tile that are seen, and this lane's first
          const int rows = min(kAttnTile, w.j < pre ? p.prefix - w.j * kAttnTile : last - (w.j - pre) * kAttnTile);
          const int key = (w.j < pre ? w.j : j0 + w.j - pre) * kAttnTile + box_at * box;
          const bool mine = box_at * box < rows;
          const uint32_t fb = bar(kABFull + static_cast<int>(slot));
          int r = key, b = krow;
          if (!from_own) {
            r = own ? key : krow + key;
            b = 0;
          } else if (paged && mine) {
            b = __ldg(p.table + static_cast<long long>(krow) * p.table_width + (key >> p.page_shift));
            r = key & ((1 << p.page_shift) - 1);
          }
          if (lane == 0)
            mbar_arrive_expect_tx(fb, static_cast<uint32_t>((rows + box - 1) & ~(box - 1)) * 128u * L::kPanels);
          issued = g + 1;
          __syncwarp();
          // test support: the very first ring tile is armed but never filled
          if (mine && !((p.debug & 1u) && g == 0))
            tma_load_4d(base + L::kOffRing + slot * L::kTileBytes + panel * kPanelBytes +
                            static_cast<uint32_t>(box_at * box) * 128u,
                        from_own ? (is_k ? &tm_k_own : &tm_v_own) : (is_k ? &tm_k : &tm_v), fb, panel * 64, head, r, b);
        }
        if (!ok) break;
        ring += 2u * static_cast<uint32_t>(n);
        __syncwarp();
        if (lane == 0) {
          if (n == 0) mbar_arrive(bar(kABAsk));
          mbar_arrive(bar(kABItemEmpty + islot));
        }
      }
      __syncwarp();
      // copies still in flight must land before the CTA exits
      for (int t = 0; t < 2; ++t)
        if ((used >> t) & 1u) drain_wait(bar(kABQFull + t), ((nq >> t) & 1u) ^ 1u, p.budget_ns);
      for (uint32_t k = 1; k <= kRing && k <= issued; ++k)
        drain_wait(bar(kABFull + static_cast<int>((issued - k) % kRing)), ((issued - k) / kRing) & 1u, p.budget_ns);
    } else {
      // ---------------------------------------------------------------- items
      grid_dependency_wait();
      const uint32_t next_slot = bar0 + 8u * kASlotNext;
      int x = static_cast<int>(blockIdx.x);
      const AttnSeq mine = load_seq(p, lane);
      AttnCursor cursor;
      uint32_t it = 0, nnext = 0;
      while (true) {
        AttnItem a;
        const bool some = decode_item(p, x, lane, mine, cursor, a);
        if (some) {
          const uint32_t islot = it % kAttnItems;
          if (!bw.wait(bar(kABItemEmpty + islot), ((it / kAttnItems) & 1u) ^ 1u)) {
            if (lane == 0) *claimed = a;
            break;
          }
          if (lane == 0) {
            items[islot] = a;
            mbar_arrive(bar(kABItemFull + islot));
          }
          // The next item is asked for when this one's loads are nearly all
          // issued: asked for earlier it would wait here while other CTAs run
          // out of work (measured: the first CTA done 30 us before the last
          // instead of the length of an item).
          if (!bw.wait(bar(kABAsk), it & 1u)) break;
          ++it;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(kABNext), 16);
          asm volatile(
              "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                  next_slot),
              "r"(bar(kABNext))
              : "memory");
        }
        __syncwarp();
        // (waited for even on an abort: the answer is written to shared memory)
        drain_wait(bar(kABNext), nnext & 1u, p.budget_ns);
        ++nnext;
        uint32_t got, nx;
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
            "ld.shared.b128 h, [%2];\n\t"
            "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t"
            "mov.u32 %1, 0;\n\t"
            "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
            : "=r"(got), "=r"(nx)
            : "r"(next_slot)
            : "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (!got) {
          const uint32_t islot = it % kAttnItems;
          if (bw.wait(bar(kABItemEmpty + islot), ((it / kAttnItems) & 1u) ^ 1u) && lane == 0) {
            items[islot].kind = -1;
            mbar_arrive(bar(kABItemFull + islot));
          }
          break;
        }
        x = static_cast<int>(nx);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
  if (*abort_flag) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0, kTimeoutCode);
    if (p.parts > 1) give_up_parts(p.part_ml, items, claimed, p.kv_heads, p.tokens, p.group);
  }
}

// Joins the parts of every row: with M = max over parts of c m_p,
// o = sum_p 2^(c m_p - M) o_p / sum_p 2^(c m_p - M) l_p.
// A block takes 32 rows and eight of their columns for each group of
// join_warps warps.  Each warp of a group reads every join_warps-th part, four
// of them in flight (one thread walking all parts of a row took 16 us for 17
// parts: a memory latency for each), and the group's results are joined
// through shared memory.  The order is fixed, so the result does not depend
// on timing.  A row with a part that was given up (l < 0) is not written.
constexpr int kJoinWarps = 8;

struct AttnPart {
  float m, l, o[8];  // (m = -inf, l = 0, o = 0: nothing yet)
  __device__ __forceinline__ void add(float pm, float pl, const float* po) {
    if (pl == 0.0f) return;  // (a part without keys; its o was not written)
    const float big = fmaxf(m, pm);
    const float f = m == big ? 1.0f : exp2f(m - big), g = pm == big ? 1.0f : exp2f(pm - big);
    m = big;
    l = l * f + pl * g;
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = o[k] * f + po[k] * g;
  }
};

template <bool BF16>
__global__ void __launch_bounds__(32 * kJoinWarps) attn_combine_kernel(const __grid_constant__ AttnParams p) {
  using namespace ptx;
  using namespace attn;
  __shared__ float joined[kJoinWarps][10][32];
  grid_launch_dependents();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long rows = static_cast<long long>(p.tokens) * (p.group * p.kv_heads);
  const int across = p.join_warps, first = warp & ~(across - 1);
  const int col8 = static_cast<int>(blockIdx.y) * (kJoinWarps / across) + warp / across;
  const int row = static_cast<int>(blockIdx.x) * 32 + lane;
  const bool valid = row < rows && col8 < p.dim / 8;
  AttnPart a = {-INFINITY, 0.0f, {0, 0, 0, 0, 0, 0, 0, 0}};
  bool lost = false;
  if (valid) {
    constexpr int kBatch = 4;
    for (int s0 = warp - first; s0 < p.parts; s0 += kBatch * across) {
      float2 ml[kBatch];
      float4 u[kBatch], v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int s = s0 + b * across;
        ml[b] = make_float2(0.0f, 0.0f);
        if (s < p.parts) {
          const float4* src =
              reinterpret_cast<const float4*>(p.part_o + ((static_cast<long long>(s) * (p.dim / 8) + col8) * rows + row) * 8);
          ml[b] = p.part_ml[s * rows + row];
          u[b] = src[0];
          v[b] = src[1];
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (s0 + b * across >= p.parts) break;
        const float po[8] = {u[b].x, u[b].y, u[b].z, u[b].w, v[b].x, v[b].y, v[b].z, v[b].w};
        lost = lost || ml[b].y < 0.0f;
        a.add(ml[b].x, ml[b].y, po);
      }
    }
  }
  joined[warp][8][lane] = a.m;
  joined[warp][9][lane] = lost ? -1.0f : a.l;
#pragma unroll
  for (int k = 0; k < 8; ++k) joined[warp][k][lane] = a.o[k];
  __syncthreads();
  if (warp != first || !valid) return;
  for (int w = first + 1; w < first + across; ++w) {
    float po[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) po[k] = joined[w][k][lane];
    lost = lost || joined[w][9][lane] < 0.0f;
    a.add(joined[w][8][lane], joined[w][9][lane], po);
  }
  if (lost) return;
  int head = row, token;
  token = p.by_group.split(head);  // head: of the group
  head += p.by_tokens.split(token) * p.group;
  if (p.op == kAttnPrompt) {
    // rows that belong to no sequence are left alone
    if (token < __ldg(p.cu_q) || token >= __ldg(p.cu_q + p.batch)) return;
  }
  const float inv = 1.0f / a.l;
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float x = a.l == 0.0f ? 0.0f : a.o[2 * k] * inv, y = a.l == 0.0f ? 0.0f : a.o[2 * k + 1] * inv;
    w[k] = BF16 ? pack_bf16x2(__float_as_uint(x), __float_as_uint(y)) : pack_f16x2(__float_as_uint(x), __float_as_uint(y));
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + token * p.out_row + head * p.out_head + col8 * 8) =
      make_uint4(w[0], w[1], w[2], w[3]);
  if (col8 == 0 && p.lse)
    p.lse[token * p.lse_row + head * p.lse_head] =
        a.l == 0.0f ? -INFINITY : static_cast<float>((a.m + log2f(a.l)) * 0.6931471805599453);
}

}  // namespace b2b
