// C entry points of the attention operators (include/b2b.h): prompts and
// batches that share a prefix.  Host side only: argument checks, tensor maps,
// how far key ranges are split over CTAs, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "attention_registry.h"
#include "b2b.h"
#include "host.h"

using namespace b2b;

struct b2b_attn_plan_s {
  b2b_dtype_t dtype;
  int device, sms;
  int q_heads, kv_heads, dim, group, tile_tokens;
  float scale;
  AttnKernels k;
  int dp;  // 0: padded head size 64, 1: 128
  int* d_status;
  uint64_t budget_ns;
  uint32_t debug;
};

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;
// The registers of the warp roles (setmaxnreg) are drawn from what the kernel
// is launched with: a kernel compiled to fewer would wait for them.
constexpr int kRegsNeeded = 256 * kAttnSoftmaxRegs + 128 * kAttnEpilogueRegs + 128 * kAttnOtherRegs;

float times_log2e(float scale) { return static_cast<float>(static_cast<double>(scale) * 1.4426950408889634); }

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Strides of a tensor of `rows` x `heads` (x `blocks`) rows of `dim` elements:
// positive multiples of 16 bytes where the extent is above one.
b2b_status_t check_rows(const b2b_attn_rows_t& t, int64_t rows, int64_t heads, int64_t blocks) {
  if (rows == 0 || blocks == 0) return B2B_OK;
  if (!t.data) return B2B_ERR_INVALID_ARG;
  if (!aligned16(t.data)) return B2B_ERR_ALIGNMENT;
  const int64_t extent[3] = {rows, heads, blocks}, stride[3] = {t.row_stride, t.head_stride, t.block_stride};
  for (int i = 0; i < 3; ++i) {
    if (extent[i] == 1) continue;
    if (stride[i] <= 0 || stride[i] >= (int64_t(1) << 38)) return B2B_ERR_INVALID_ARG;
    if (stride[i] % 8) return B2B_ERR_ALIGNMENT;
  }
  return B2B_OK;
}

size_t span_bytes(const b2b_attn_rows_t& t, int64_t rows, int64_t heads, int64_t blocks, int64_t dim) {
  if (rows == 0 || blocks == 0) return 0;
  return 2 * static_cast<size_t>((rows - 1) * t.row_stride + (heads - 1) * t.head_stride +
                                 (blocks - 1) * t.block_stride + dim);
}

// Whether the output's rows share bytes with an input's.  Tensors whose rows
// alternate, as column ranges of one buffer do, have overlapping spans but no
// byte in common: with rows an equal stride apart, and each in a window no
// wider than it, the windows repeat with that stride and have to be disjoint
// in one period.  Other strides are judged by the spans.
bool rows_overlap(const b2b_attn_rows_t& out, int64_t out_rows, int64_t out_heads, const b2b_attn_rows_t& in, int64_t rows,
                  int64_t heads, int64_t blocks, int64_t dim) {
  if (!overlaps(out.data, span_bytes(out, out_rows, out_heads, 1, dim), in.data, span_bytes(in, rows, heads, blocks, dim)))
    return false;
  if (blocks != 1 || out_rows == 1 || rows == 1 || out.row_stride != in.row_stride) return true;
  const int64_t period = 2 * out.row_stride;
  const int64_t a = static_cast<int64_t>(span_bytes(out, 1, out_heads, 1, dim)), b = static_cast<int64_t>(span_bytes(in, 1, heads, 1, dim));
  int64_t apart = (reinterpret_cast<intptr_t>(in.data) - reinterpret_cast<intptr_t>(out.data)) % period;
  if (apart < 0) apart += period;
  return apart < a || apart + b > period;  // (a window wider than the period is caught by one or the other)
}

// 4-D map with boxes of 64 columns (128 bytes, swizzled) by box1 x 1 x box3 or
// 1 x box2 rows; extents of one take a stride of one dense row.
b2b_status_t encode(CUtensorMap* map, const b2b_attn_plan_s* p, const void* data, const int64_t (&ext)[3],
                    const int64_t (&stride)[3], const uint32_t (&box)[3]) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return B2B_ERR_CUDA;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(p->dim), 0, 0, 0}, strides[3];
  cuuint32_t boxes[4] = {64, box[0], box[1], box[2]};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  for (int i = 0; i < 3; ++i) {
    dims[i + 1] = static_cast<cuuint64_t>(ext[i]);
    strides[i] = static_cast<cuuint64_t>(2 * (ext[i] == 1 ? p->dim : stride[i]));
  }
  const CUresult r =
      fn(map, p->dtype == B2B_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
         const_cast<void*>(data), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? B2B_OK : B2B_ERR_CUDA;
}

// Queries [tokens][kv_heads][group]: one box is `tokens_box` tokens of one key/value head's group.
b2b_status_t encode_q(CUtensorMap* map, const b2b_attn_plan_s* p, const b2b_attn_rows_t& t, int64_t tokens,
                      uint32_t tokens_box) {
  return encode(map, p, t.data, {p->group, p->kv_heads, tokens},
                {t.head_stride, t.head_stride * p->group, t.row_stride},
                {static_cast<uint32_t>(p->group), 1, tokens_box});
}
// Keys or values [blocks][rows][kv_heads]: one box is `box` rows of one head.
b2b_status_t encode_kv(CUtensorMap* map, const b2b_attn_plan_s* p, const b2b_attn_rows_t& t, int64_t rows,
                       int64_t blocks, uint32_t box) {
  return encode(map, p, t.data, {p->kv_heads, rows, blocks}, {t.head_stride, t.row_stride, t.block_stride}, {1, box, 1});
}

// ---------------------------------------------------------------- shapes
// How work is cut into items is chosen by a model of the time, in units of a
// key tile of a pair item (about 1.45 us for 128-wide heads; 64-wide ones, whose
// tiles take some 1.2 us, are counted in the same units): a tile of a solo item
// takes 0.55, an item's beginning and end 1.2 more (traces of both).
constexpr double kSoloTile = 0.55, kItemCost = 1.2;

// Joining parts: a second launch and memory latencies, some 4.5 us, and the
// parts' traffic, written and read once in fp32 at some 4 TB/s.  (Nine requests
// on 1,222 shared keys, which parts make quicker: 12.3 us a call counted as 8
// us, 9.3 as 4.5; three of five tokens on 207, whole either way: 7.9, in parts 11.4.)
double join_cost(const b2b_attn_plan_s* p, double tokens, int parts) {
  return parts <= 1 ? 0.0 : 3.0 + parts * tokens * p->q_heads * p->dim * 8.0 / 5.8e6;
}

struct PromptShape {
  int tiles;   // query tiles of an item: 2 (pair) or 1 (solo)
  int splits;  // parts of the key range
  int64_t blocks;  // at most so many blocks of queries
};
// Few rows over many keys are cut along the keys, and blocks that would fill
// the GPU's SMs a little more than a whole number of times are halved (six
// pieces of 200-256 tokens over 1000-6000 keys, 28/4 heads of 128: 172 items
// of two tiles 76 us, 320 of one tile 66 us; 24 prompts of 1-700 tokens keep
// two, 55 us against 61).  Between two and four rounds of the SMs the model
// counts whole ones, which short items of different lengths do not take: 16
// passages of 100-512 tokens, 12 heads of 96, get one tile (22.6 us) and would
// be quicker with two (21.5 us).
PromptShape prompt_shape(const b2b_attn_plan_s* p, int64_t batch, int64_t tokens, int64_t key_rows, bool causal) {
  PromptShape best = {2, 1, 0};
  double best_t = 1e300;
  const double b = static_cast<double>(std::max<int64_t>(1, std::min(batch, tokens)));
  const double most = static_cast<double>(key_rows) / b / kAttnTile;  // key tiles of a sequence
  const double seen = std::max(causal ? most - 0.5 * tokens / b / kAttnTile : most, 0.0);
  for (int tiles = 1; tiles <= 2; ++tiles) {
    const int64_t block = tiles * p->tile_tokens;
    const double tile = tiles == 2 ? 1.0 : kSoloTile;
    // (a sequence's last block is half empty on average)
    const double blocks = batch == 1 ? static_cast<double>((tokens + block - 1) / block) : static_cast<double>(tokens) / block + 0.5 * b;
    for (int s = 1; s <= 64 && (s == 1 || most >= 4.0 * s); ++s) {
      // (rows of parts are numbered in 31 bits)
      if (s > 1 && tokens * p->q_heads > kMaxRows) break;
      const double items = std::max(blocks, b) * p->kv_heads * s, rounds = items / p->sms;
      const double item = std::ceil(seen / s + 0.5) * tile + kItemCost, longest = (most / s + 0.5) * tile + kItemCost;
      const double t = std::max((rounds < 4.0 ? std::ceil(rounds) : rounds + 0.5) * item, longest) +
                       join_cost(p, static_cast<double>(tokens), s);
      if (t < best_t * 0.999) {
        best_t = t;
        best = {tiles, s, 0};
      }
    }
  }
  const int64_t block = best.tiles * p->tile_tokens;
  best.blocks = batch == 1 ? (tokens + block - 1) / block : tokens / block + std::min(batch, tokens);
  return best;
}

struct SharedShape {
  int64_t row_blocks, block_tokens, own_blocks, prefix_items, own_items;
  int splits, own_splits;
  bool whole;  // items of whole requests, prefix and own keys: nothing is shared, and nothing to join
};
SharedShape shared_shape(const b2b_attn_plan_s* p, int64_t batch, int64_t fresh, int64_t prefix, int64_t room) {
  SharedShape s = {};
  const int64_t tokens = batch * fresh, block = 2 * p->tile_tokens;
  s.block_tokens = tokens <= p->tile_tokens ? p->tile_tokens : block;
  s.row_blocks = (tokens + s.block_tokens - 1) / s.block_tokens;
  s.own_blocks = (fresh + block - 1) / block;
  // lengths are known to the device only: half the room on average
  const double pre_tiles = static_cast<double>((prefix + kAttnTile - 1) / kAttnTile);
  const double own_tiles = std::ceil(0.5 * static_cast<double>(room) / kAttnTile);
  const double pre_tile = s.block_tokens == block ? 1.0 : kSoloTile, own_tile = fresh > p->tile_tokens ? 1.0 : kSoloTile;
  const double pre = static_cast<double>(s.row_blocks * p->kv_heads), own = static_cast<double>(batch * s.own_blocks * p->kv_heads);
  double best_t = 1e300;
  s.splits = prefix ? 1 : 0;
  s.own_splits = 1;
  for (int so = 1; so <= 64 && (so == 1 || (own * so <= 2.0 * p->sms && own_tiles >= 2.0 * so)); ++so) {
    for (int sp = prefix ? 1 : 0; sp <= 64 && (sp <= 1 || pre_tiles >= 2.0 * sp); ++sp) {
      const double pre_item = sp ? std::ceil(pre_tiles / sp) * pre_tile + kItemCost : 0.0;
      const double own_item = std::ceil(own_tiles / so) * own_tile + kItemCost;
      // prefix items are begun first, own ones fill the gaps they leave
      const double total = (pre * sp * pre_item + own * so * own_item) / p->sms;
      const double t = std::max(total, std::max(pre_item, own_item)) + (pre * sp + own * so > p->sms ? 0.5 * own_item : 0.0) +
                       join_cost(p, static_cast<double>(tokens), sp + so);
      if (t < best_t * 0.999) {
        best_t = t;
        s.splits = sp;
        s.own_splits = so;
      }
      if (!prefix) break;
    }
  }
  // Small batches on short prefixes: every request reads the prefix itself (from
  // L2, at some 8 TB/s), which saves the join (four requests, 133 shared keys:
  // 10.1 us a call with two parts, 7.0 us whole).
  if (prefix) {
    const double item = (pre_tiles + own_tiles) * own_tile + kItemCost, rounds = own / p->sms;
    const double t = std::max((rounds < 4.0 ? std::ceil(rounds) : rounds + 0.5) * item,
                              own * static_cast<double>(prefix) * p->dim * 4.0 / 11.6e6);
    s.whole = t < best_t;
    if (s.whole) {
      s.splits = 0;
      s.own_splits = 1;
    }
  }
  s.prefix_items = s.splits * s.row_blocks * p->kv_heads;
  s.own_items = s.own_splits * batch * s.own_blocks * p->kv_heads;
  return s;
}

size_t part_bytes(const b2b_attn_plan_s* p, int64_t tokens, int64_t parts) {
  if (parts <= 1) return 0;
  return static_cast<size_t>(parts * tokens * p->q_heads) * (static_cast<size_t>(p->dim) * 4 + 8);
}

b2b_status_t check_current_device(const b2b_attn_plan_s* p) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return B2B_ERR_CUDA;
  }
  return dev == p->device ? B2B_OK : B2B_ERR_DEVICE;
}

// Some waits last as long as an item does (the epilogue's for its last tile,
// the item warp's for its loads), and the first of all as long as the search
// for an item, which reads `searched` sequences once for every halving of the
// tiles.  A budget counts as no less than these take with some ten times to
// spare: 20 us a tile of the longest item, 0.3 us a sequence and step.
uint64_t wait_budget(const b2b_attn_plan_s* p, int64_t tiles, int64_t searched) {
  uint64_t steps = 4;
  while ((int64_t(1) << (steps - 4)) < tiles) ++steps;
  return std::max(p->budget_ns, 20000 * static_cast<uint64_t>(tiles) + 300 * steps * static_cast<uint64_t>(searched));
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

AttnParams common_params(const b2b_attn_plan_s* p, int64_t tokens, int64_t batch, const b2b_attn_rows_t& out, float* lse,
                         void* workspace, int parts, uint64_t budget_ns) {
  AttnParams a;
  std::memset(&a, 0, sizeof(a));
  a.group = p->group;
  a.kv_heads = p->kv_heads;
  a.dim = p->dim;
  a.tile_tokens = p->tile_tokens;
  a.by_group = FastDiv::of(static_cast<uint32_t>(p->group));
  a.by_tokens = FastDiv::of(static_cast<uint32_t>(tokens));
  a.by_kv_heads = FastDiv::of(static_cast<uint32_t>(p->kv_heads));
  a.by_block = FastDiv::of(static_cast<uint32_t>(2 * p->tile_tokens));
  a.tokens = static_cast<int>(tokens);
  a.batch = static_cast<int>(batch);
  a.scale = p->scale;
  a.scale_log2 = times_log2e(p->scale);
  a.out = out.data;
  a.out_row = out.row_stride;
  a.out_head = out.head_stride;
  a.lse = lse;
  a.lse_row = p->q_heads;
  a.lse_head = 1;
  a.wide_stores = p->dim % 16 == 0 && reinterpret_cast<uintptr_t>(out.data) % 32 == 0 && out.row_stride % 16 == 0 &&
                  out.head_stride % 16 == 0;
  a.parts = parts;
  a.join_warps = 1;
  while (a.join_warps < kJoinWarps && a.join_warps < parts) a.join_warps *= 2;
  if (parts > 1) {
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<int64_t>(parts) * tokens * p->q_heads * p->dim);
  }
  a.q_bytes = static_cast<uint32_t>(p->group * p->tile_tokens) * 128u * (p->dp ? 2u : 1u);
  a.debug = p->debug;
  a.status = p->d_status;
  a.budget_ns = static_cast<uint32_t>(std::min<uint64_t>(budget_ns, 4000000000ull));  // (a 32-bit clock in the kernel)
  return a;
}

b2b_status_t launch(const b2b_attn_plan_s* p, CUtensorMap (&maps)[6], AttnParams& a, int64_t items, cudaStream_t stream) {
  void* args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &maps[4], &maps[5], &a};
  cudaError_t e = launch_pdl(p->k.main[p->dp], dim3(static_cast<unsigned>(items)), dim3(kAttnThreads), args,
                             p->k.smem[p->dp], stream);
  if (e == cudaSuccess && a.parts > 1) {
    const int64_t rows = static_cast<int64_t>(a.tokens) * p->q_heads;
    const int columns = kJoinWarps / a.join_warps;
    void* cargs[] = {&a};
    e = launch_pdl(p->k.combine, dim3(static_cast<unsigned>((rows + 31) / 32), static_cast<unsigned>((p->dim / 8 + columns - 1) / columns)),
                   dim3(32 * kJoinWarps), cargs, 0, stream);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return B2B_ERR_CUDA;
  }
  return B2B_OK;
}

}  // namespace

extern "C" {

b2b_status_t b2b_attn_plan_create(b2b_attn_plan_t* out, b2b_dtype_t dtype, int64_t q_heads, int64_t kv_heads,
                                  int64_t head_dim, float scale) {
  if (!out) return B2B_ERR_INVALID_ARG;
  *out = nullptr;
  if (dtype < B2B_F16_F32OUT || dtype > B2B_TF32_BF16) return B2B_ERR_INVALID_ARG;
  if (q_heads < 1 || kv_heads < 1 || head_dim < 1 || q_heads % kv_heads) return B2B_ERR_INVALID_ARG;
  if (!(scale >= 0.0f) || std::isinf(times_log2e(scale))) return B2B_ERR_INVALID_ARG;
  if (dtype != B2B_F16 && dtype != B2B_BF16) return B2B_ERR_UNSUPPORTED;
  if (head_dim % 8 || head_dim > 128 || q_heads > 65536 || q_heads / kv_heads > kAttnTile) return B2B_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  b2b_status_t st = check_device(&dev, &sms);
  if (st != B2B_OK) return st;
  b2b_attn_plan_s* p = new (std::nothrow) b2b_attn_plan_s();
  if (!p) return B2B_ERR_CUDA;
  p->dtype = dtype;
  p->device = dev;
  p->sms = sms;
  p->q_heads = static_cast<int>(q_heads);
  p->kv_heads = static_cast<int>(kv_heads);
  p->dim = static_cast<int>(head_dim);
  p->group = p->q_heads / p->kv_heads;
  p->tile_tokens = kAttnTile / p->group;
  p->scale = scale > 0.0f ? scale : static_cast<float>(1.0 / std::sqrt(static_cast<double>(head_dim)));
  p->k = dtype == B2B_F16 ? attn_kernels_f16() : attn_kernels_bf16();
  p->dp = head_dim > 64;
  p->budget_ns = kDefaultBudgetNs;
  cudaFuncAttributes fa;
  if (cudaFuncSetAttribute(p->k.main[p->dp], cudaFuncAttributeMaxDynamicSharedMemorySize, p->k.smem[p->dp]) !=
          cudaSuccess ||
      cudaFuncGetAttributes(&fa, p->k.main[p->dp]) != cudaSuccess || fa.numRegs * kAttnThreads < kRegsNeeded ||
      cudaMalloc(&p->d_status, sizeof(int)) != cudaSuccess) {
    cudaGetLastError();
    delete p;
    return B2B_ERR_CUDA;
  }
  if (cudaMemset(p->d_status, 0, sizeof(int)) != cudaSuccess) {
    cudaGetLastError();
    cudaFree(p->d_status);
    delete p;
    return B2B_ERR_CUDA;
  }
  *out = p;
  return B2B_OK;
}

b2b_status_t b2b_attn_plan_destroy(b2b_attn_plan_t p) {
  if (!p) return B2B_OK;
  cudaFree(p->d_status);
  delete p;
  return B2B_OK;
}

b2b_status_t b2b_attn_plan_device_status(b2b_attn_plan_t p, b2b_stream_t stream) {
  if (!p) return B2B_ERR_INVALID_ARG;
  int v = 0;
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess ||
      cudaMemcpy(&v, p->d_status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess ||
      cudaMemset(p->d_status, 0, sizeof(int)) != cudaSuccess) {
    cudaGetLastError();
    return B2B_ERR_CUDA;
  }
  return static_cast<b2b_status_t>(v);
}

b2b_status_t b2b_attn_plan_set_wait_budget(b2b_attn_plan_t p, uint64_t budget_ns) {
  if (!p) return B2B_ERR_INVALID_ARG;
  p->budget_ns = budget_ns ? std::max<uint64_t>(budget_ns, kMinBudgetNs) : kDefaultBudgetNs;
  return B2B_OK;
}

b2b_status_t b2b_attn_plan_set_debug(b2b_attn_plan_t p, uint32_t flags) {
  if (!p) return B2B_ERR_INVALID_ARG;
  if (flags & ~B2B_DEBUG_DROP_FIRST_LOAD) return B2B_ERR_INVALID_ARG;
  p->debug = flags;
  return B2B_OK;
}

b2b_status_t b2b_prompt_attention_workspace(b2b_attn_plan_t p, int64_t batch, int64_t tokens, int64_t key_rows,
                                            int64_t causal, size_t* bytes) {
  if (!p || !bytes || batch < 0 || tokens < 0 || key_rows < 0) return B2B_ERR_INVALID_ARG;
  if (tokens > kMaxRows || key_rows > kMaxRows || batch > kMaxRows) return B2B_ERR_UNSUPPORTED;
  *bytes = 0;
  if (batch == 0 || tokens == 0) return B2B_OK;
  *bytes = part_bytes(p, tokens, prompt_shape(p, batch, tokens, key_rows, causal != 0).splits);
  return B2B_OK;
}

b2b_status_t b2b_prompt_attention_run(b2b_attn_plan_t p, const b2b_prompt_attention_t* r, b2b_stream_t stream) {
  if (!p || !r || r->batch < 0 || r->tokens < 0 || r->key_rows < 0) return B2B_ERR_INVALID_ARG;
  if (r->tokens > kMaxRows || r->key_rows > kMaxRows || r->batch > kMaxRows) return B2B_ERR_UNSUPPORTED;
  if (r->tokens == 0 || r->batch == 0) return B2B_OK;
  if (!r->cu_q || !r->cu_k) return B2B_ERR_INVALID_ARG;
  if (!aligned4(r->cu_q) || !aligned4(r->cu_k) || !aligned4(r->lse)) return B2B_ERR_ALIGNMENT;
  const int64_t hq = p->q_heads, hk = p->kv_heads, d = p->dim;
  b2b_status_t st = check_rows(r->q, r->tokens, hq, 1);
  if (st == B2B_OK) st = check_rows(r->k, r->key_rows, hk, 1);
  if (st == B2B_OK) st = check_rows(r->v, r->key_rows, hk, 1);
  if (st == B2B_OK) st = check_rows(r->out, r->tokens, hq, 1);
  if (st != B2B_OK) return st;
  if (rows_overlap(r->out, r->tokens, hq, r->q, r->tokens, hq, 1, d) || rows_overlap(r->out, r->tokens, hq, r->k, r->key_rows, hk, 1, d) ||
      rows_overlap(r->out, r->tokens, hq, r->v, r->key_rows, hk, 1, d))
    return B2B_ERR_ALIAS;
  const PromptShape shape = prompt_shape(p, r->batch, r->tokens, r->key_rows, r->causal != 0);
  const int splits = shape.splits;
  const size_t need = part_bytes(p, r->tokens, splits);
  if (need && (!r->workspace || r->workspace_bytes < need)) return B2B_ERR_INVALID_ARG;
  if (need && reinterpret_cast<uintptr_t>(r->workspace) % 32) return B2B_ERR_ALIGNMENT;
  const int64_t items = shape.blocks * hk * splits;
  if (items > kMaxRows) return B2B_ERR_UNSUPPORTED;
  st = check_current_device(p);
  if (st != B2B_OK) return st;

  const int64_t most_tiles = ceil_div(r->key_rows, kAttnTile);
  AttnParams a = common_params(p, r->tokens, r->batch, r->out, r->lse, r->workspace, splits,
                               wait_budget(p, ceil_div(most_tiles, splits), r->batch));
  a.op = kAttnPrompt;
  a.causal = r->causal != 0;
  a.cu_q = r->cu_q;
  a.cu_k = r->cu_k;
  a.key_rows = static_cast<int>(r->key_rows);
  a.by_splits = FastDiv::of(static_cast<uint32_t>(splits));
  a.by_block = FastDiv::of(static_cast<uint32_t>(shape.tiles * p->tile_tokens));
  a.most_tiles = static_cast<int>(most_tiles);
  a.box_rows = kAttnTile;
  CUtensorMap maps[6];
  st = encode_q(&maps[0], p, r->q, r->tokens, static_cast<uint32_t>(p->tile_tokens));
  // (without keys nothing is loaded through the key and value maps)
  maps[2] = maps[3] = maps[0];
  if (st == B2B_OK && r->key_rows) st = encode_kv(&maps[2], p, r->k, r->key_rows, 1, kAttnTile);
  if (st == B2B_OK && r->key_rows) st = encode_kv(&maps[3], p, r->v, r->key_rows, 1, kAttnTile);
  maps[1] = maps[0];
  maps[4] = maps[2];
  maps[5] = maps[3];
  return st == B2B_OK ? launch(p, maps, a, items, reinterpret_cast<cudaStream_t>(stream)) : st;
}

b2b_status_t b2b_shared_attention_workspace(b2b_attn_plan_t p, int64_t batch, int64_t fresh, int64_t prefix, int64_t room,
                                            size_t* bytes) {
  if (!p || !bytes || batch < 0 || fresh < 0 || prefix < 0 || room < 0) return B2B_ERR_INVALID_ARG;
  if (batch > kMaxRows || fresh > kMaxRows || batch * fresh > kMaxRows || prefix > kMaxRows || room > kMaxRows)
    return B2B_ERR_UNSUPPORTED;
  *bytes = 0;
  if (batch * fresh == 0) return B2B_OK;
  const SharedShape s = shared_shape(p, batch, fresh, prefix, room);
  *bytes = part_bytes(p, batch * fresh, s.splits + s.own_splits);
  return B2B_OK;
}

b2b_status_t b2b_shared_attention_run(b2b_attn_plan_t p, const b2b_shared_attention_t* r, b2b_stream_t stream) {
  if (!p || !r || r->batch < 0 || r->fresh < 0 || r->prefix < 0 || r->cache_rows < 0 || r->cache_blocks < 0 ||
      r->table_width < 0)
    return B2B_ERR_INVALID_ARG;
  const bool paged = r->page_table != nullptr;
  if (r->batch > kMaxRows || r->fresh > kMaxRows || r->batch * r->fresh > kMaxRows || r->prefix > kMaxRows ||
      r->cache_rows > kMaxRows || r->cache_blocks > kMaxRows || r->table_width > kMaxRows)
    return B2B_ERR_UNSUPPORTED;
  const int64_t tokens = r->batch * r->fresh;
  if (tokens == 0) return B2B_OK;
  if (!r->lengths) return B2B_ERR_INVALID_ARG;
  if (!aligned4(r->lengths) || !aligned4(r->page_table) || !aligned4(r->lse)) return B2B_ERR_ALIGNMENT;
  if (!paged && r->cache_blocks != r->batch) return B2B_ERR_INVALID_ARG;
  int page_shift = 0;
  if (paged) {
    // pages of 16, 32, 64, .. rows: whole boxes of a tile, whole groups of eight swizzled rows
    if (r->cache_rows < 16 || (r->cache_rows & (r->cache_rows - 1))) return B2B_ERR_UNSUPPORTED;
    while ((int64_t(1) << page_shift) < r->cache_rows) ++page_shift;
  }
  const int64_t room = paged ? (r->cache_blocks ? r->table_width * r->cache_rows : 0) : r->cache_rows;
  if (room > kMaxRows) return B2B_ERR_UNSUPPORTED;
  const int64_t hq = p->q_heads, hk = p->kv_heads, d = p->dim;
  b2b_status_t st = check_rows(r->q, tokens, hq, 1);
  if (st == B2B_OK) st = check_rows(r->prefix_k, r->prefix, hk, 1);
  if (st == B2B_OK) st = check_rows(r->prefix_v, r->prefix, hk, 1);
  if (st == B2B_OK) st = check_rows(r->cache_k, r->cache_rows, hk, r->cache_blocks);
  if (st == B2B_OK) st = check_rows(r->cache_v, r->cache_rows, hk, r->cache_blocks);
  if (st == B2B_OK) st = check_rows(r->out, tokens, hq, 1);
  if (st != B2B_OK) return st;
  if (rows_overlap(r->out, tokens, hq, r->q, tokens, hq, 1, d) || rows_overlap(r->out, tokens, hq, r->prefix_k, r->prefix, hk, 1, d) ||
      rows_overlap(r->out, tokens, hq, r->prefix_v, r->prefix, hk, 1, d) ||
      rows_overlap(r->out, tokens, hq, r->cache_k, r->cache_rows, hk, r->cache_blocks, d) ||
      rows_overlap(r->out, tokens, hq, r->cache_v, r->cache_rows, hk, r->cache_blocks, d))
    return B2B_ERR_ALIAS;
  const SharedShape s = shared_shape(p, r->batch, r->fresh, r->prefix, room);
  const int parts = s.splits + s.own_splits;
  const size_t need = part_bytes(p, tokens, parts);
  if (need && (!r->workspace || r->workspace_bytes < need)) return B2B_ERR_INVALID_ARG;
  if (need && reinterpret_cast<uintptr_t>(r->workspace) % 32) return B2B_ERR_ALIGNMENT;
  if (s.prefix_items + s.own_items > kMaxRows || tokens * hq > kMaxRows) return B2B_ERR_UNSUPPORTED;
  st = check_current_device(p);
  if (st != B2B_OK) return st;

  const int64_t pre_tiles = ceil_div(r->prefix, kAttnTile), own_tiles = ceil_div(ceil_div(room, kAttnTile), s.own_splits);
  const int64_t item_tiles = std::max(s.splits ? ceil_div(pre_tiles, s.splits) : 0, own_tiles + (s.whole ? pre_tiles : 0));
  AttnParams a = common_params(p, tokens, r->batch, r->out, r->lse, r->workspace, parts, wait_budget(p, item_tiles, 0));
  a.op = kAttnShared;
  a.causal = 1;
  a.by_splits = FastDiv::of(static_cast<uint32_t>(std::max(s.splits, 1)));
  a.fresh = static_cast<int>(r->fresh);
  a.prefix = static_cast<int>(r->prefix);
  a.prefix_items = static_cast<int>(s.prefix_items);
  a.by_row_blocks = FastDiv::of(static_cast<uint32_t>(s.row_blocks));
  a.block_tokens = static_cast<int>(s.block_tokens);
  a.whole = s.whole;
  a.by_own_splits = FastDiv::of(static_cast<uint32_t>(s.own_splits));
  a.by_own_blocks = FastDiv::of(static_cast<uint32_t>(s.own_blocks));
  a.lengths = r->lengths;
  a.table = r->page_table;
  a.table_width = static_cast<int>(r->table_width);
  a.page_shift = page_shift;
  a.room = static_cast<int>(room);
  a.box_rows = kAttnTile;
  // Own keys in boxes of a page, or of 32 rows, so that little past a
  // request's length is read.
  a.own_box_rows = paged ? static_cast<int>(std::min<int64_t>(r->cache_rows, kAttnTile)) : 32;
  const uint32_t own_tokens = static_cast<uint32_t>(std::min<int64_t>(r->fresh, p->tile_tokens));
  a.own_q_bytes = static_cast<uint32_t>(p->group) * own_tokens * 128u * (p->dp ? 2u : 1u);
  CUtensorMap maps[6];
  // (maps that no item uses are copies)
  st = encode_q(&maps[1], p, r->q, tokens, own_tokens);
  maps[0] = maps[2] = maps[3] = maps[4] = maps[5] = maps[1];
  if (st == B2B_OK && s.prefix_items && own_tokens != static_cast<uint32_t>(p->tile_tokens))
    st = encode_q(&maps[0], p, r->q, tokens, static_cast<uint32_t>(p->tile_tokens));
  if (st == B2B_OK && r->prefix) st = encode_kv(&maps[2], p, r->prefix_k, r->prefix, 1, kAttnTile);
  if (st == B2B_OK && r->prefix) st = encode_kv(&maps[3], p, r->prefix_v, r->prefix, 1, kAttnTile);
  if (room) {
    const uint32_t box = static_cast<uint32_t>(a.own_box_rows);
    if (st == B2B_OK) st = encode_kv(&maps[4], p, r->cache_k, r->cache_rows, r->cache_blocks, box);
    if (st == B2B_OK) st = encode_kv(&maps[5], p, r->cache_v, r->cache_rows, r->cache_blocks, box);
  }
  return st == B2B_OK ? launch(p, maps, a, s.prefix_items + s.own_items, reinterpret_cast<cudaStream_t>(stream)) : st;
}

}  // extern "C"
