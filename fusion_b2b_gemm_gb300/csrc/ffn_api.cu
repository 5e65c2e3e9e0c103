// C entry points of the feed-forward operators (include/b2b.h).  Host side
// only: argument checks, tensor maps, how tiles are cut into units, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>

#include "b2b.h"
#include "ffn_registry.h"
#include "host.h"

using namespace b2b;

enum FfnKind { kFfn, kScaledFfn, kScaledGemm };

struct b2b_ffn_plan_s {
  FfnKind kind;
  b2b_dtype_t dtype;
  int device, sms;
  int64_t width, hidden, out_width;  // (a product: k, -, n)
  int act;
  FfnKernels k;
  ScaledKernels s;
  int* d_status;
  uint64_t budget_ns;
  uint32_t debug;
};

namespace {

constexpr int64_t kMaxExtent = int64_t(1) << 20, kMaxRows = int64_t(1) << 30, kMaxTiles = int64_t(1) << 28;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t rounded(size_t bytes) { return (bytes + 255) & ~size_t(255); }
bool is16(b2b_dtype_t t) { return t == B2B_F16 || t == B2B_BF16; }
bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// ---------------------------------------------------------------- checks
struct Matrix {
  const b2b_matrix_t* m;
  int64_t rows, cols;
  int esz;
  size_t row_bytes() const { return static_cast<size_t>(cols * esz); }
  size_t stride_bytes() const { return rows > 1 ? static_cast<size_t>(m->row_stride * esz) : row_bytes(); }
  size_t span() const { return rows ? static_cast<size_t>(rows - 1) * stride_bytes() + row_bytes() : 0; }
};

b2b_status_t check(const Matrix& t, uintptr_t to = 16) {
  if (t.rows == 0) return B2B_OK;
  if (!t.m->data) return B2B_ERR_INVALID_ARG;
  if (!aligned(t.m->data, to)) return B2B_ERR_ALIGNMENT;
  if (t.rows > 1) {
    if (t.m->row_stride < t.cols || t.m->row_stride >= (int64_t(1) << 36)) return B2B_ERR_INVALID_ARG;
    if (t.stride_bytes() % to) return B2B_ERR_ALIGNMENT;
  }
  return B2B_OK;
}

b2b_status_t check(const b2b_scales_t& s, int64_t rows) {
  if (rows == 0) return B2B_OK;
  if (!s.data) return B2B_ERR_INVALID_ARG;
  if (!aligned(s.data, 4)) return B2B_ERR_ALIGNMENT;
  const int64_t most = int64_t(1) << 36;
  return s.row_stride < 0 || s.block_stride < 0 || s.row_stride >= most || s.block_stride >= most ? B2B_ERR_INVALID_ARG : B2B_OK;
}

// Whether two matrices share bytes.  Column ranges of one buffer have spans that
// overlap and rows that do not: with equal strides the rows' windows are compared
// in one period.
bool share(const Matrix& a, const Matrix& b) {
  if (!overlaps(a.m->data, a.span(), b.m->data, b.span())) return false;
  if (a.rows == 1 || b.rows == 1 || a.stride_bytes() != b.stride_bytes()) return true;
  const intptr_t period = static_cast<intptr_t>(a.stride_bytes());
  intptr_t apart = (reinterpret_cast<intptr_t>(b.m->data) - reinterpret_cast<intptr_t>(a.m->data)) % period;
  if (apart < 0) apart += period;
  return apart < static_cast<intptr_t>(a.row_bytes()) || apart + static_cast<intptr_t>(b.row_bytes()) > period;
}
bool overlaps_scales(const Matrix& a, const b2b_scales_t& s, int64_t rows, int64_t blocks) {
  return rows && blocks &&
         overlaps(a.m->data, a.span(), s.data, 4 * static_cast<size_t>((rows - 1) * s.row_stride + (blocks - 1) * s.block_stride + 1));
}

// Checks inputs and outputs (those with data), and that no output shares bytes with another matrix.
template <int I, int O>
b2b_status_t check_all(const Matrix (&in)[I], const Matrix (&out)[O]) {
  for (const Matrix& t : in) {
    const b2b_status_t st = check(t);
    if (st != B2B_OK) return st;
  }
  for (const Matrix& t : out) {
    const b2b_status_t st = t.m->data ? check(t) : B2B_OK;
    if (st != B2B_OK) return st;
  }
  for (int o = 0; o < O; ++o) {
    for (const Matrix& t : in)
      if (share(out[o], t)) return B2B_ERR_ALIAS;
    for (int e = 0; e < o; ++e)
      if (share(out[o], out[e])) return B2B_ERR_ALIAS;
  }
  return B2B_OK;
}

b2b_status_t check_current_device(const b2b_ffn_plan_s* p) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return B2B_ERR_CUDA;
  }
  return dev == p->device ? B2B_OK : B2B_ERR_DEVICE;
}

// Memory of at least `need` bytes: a workspace, or what a forward pass kept.
b2b_status_t check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need && (!workspace || bytes < need)) return B2B_ERR_INVALID_ARG;
  return need && !aligned(workspace, 256) ? B2B_ERR_ALIGNMENT : B2B_OK;
}

// ---------------------------------------------------------------- units
struct Shape {
  int64_t tiles, whole;
  int splits;
  double time;  // in K panels of a unit
  size_t part_bytes() const { return static_cast<size_t>(tiles - whole) * splits * kGemmPartFloats * sizeof(float) * (splits > 1); }
};

// How many units the tiles that do not fill the SMs a whole number of times are
// cut into.  Times in K panels of a unit (about 0.35 us, bound by the MMAs or by
// the weights' bytes alike): those of the SMs with most of them, where tiles are cut
// 9 more for the second launch, and the parts' traffic at some 4 TB/s.  A unit's own
// beginning and end count nothing; the constants that few_shape() sets this time
// against (SkinnyCost) were fitted to it as it is.
Shape cut(int64_t tiles, int64_t kpan, int clusters) {
  const int64_t rounds = tiles / clusters, rest = tiles - rounds * clusters;
  Shape best = {tiles, tiles, 1, static_cast<double>((rounds + (rest > 0)) * kpan)};
  if (rest == 0) return best;
  for (int s = 2; s <= 32 && kpan >= 4 * s; ++s) {
    const double t = static_cast<double>(rounds * kpan + ceil_div(rest * s, clusters) * ceil_div(kpan, s)) + 9.0 +
                     static_cast<double>(rest * s) * kGemmPartFloats * 8.0 / 1.4e6;
    if (t < best.time) best = {tiles, rounds * clusters, s, t};
  }
  return best;
}

void add_problem(GemmParams& p, int64_t m, int64_t n, bool gate) {
  GemmProblem& q = p.prob[p.problems++];
  q.first = p.tiles;
  q.M = static_cast<int>(m);
  q.N = static_cast<int>(n);
  q.m_tiles = static_cast<int>(ceil_div(m, kGemmTile));
  q.n_tiles = static_cast<int>(ceil_div(n, gate ? 128 : kGemmTile));
  p.tiles += q.m_tiles * q.n_tiles;
}
void set_units(GemmParams& p, int kpan, int clusters) {
  const Shape s = cut(p.tiles, kpan, clusters);
  p.kpan = kpan;
  p.whole = static_cast<int>(s.whole);
  p.splits = s.splits;
  p.units = static_cast<int>(s.whole + (s.tiles - s.whole) * s.splits);
  p.group = 8;
}

int panels(int64_t k, bool e4m3 = false) { return static_cast<int>(ceil_div(k, e4m3 ? 128 : 64)); }
int64_t tile_count(int64_t m, int64_t n, bool gate) { return ceil_div(m, kGemmTile) * ceil_div(n, gate ? 128 : kGemmTile); }

// --------------------------------------------------------------- launches
b2b_status_t encode(CUtensorMap* map, CUtensorMapDataType type, const Matrix& t, uint32_t box_cols, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return B2B_ERR_CUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(t.cols), static_cast<cuuint64_t>(t.rows)};
  const cuuint64_t strides[1] = {(t.stride_bytes() + 15) & ~cuuint64_t(15)};
  const cuuint32_t box[2] = {box_cols, box_rows}, estr[2] = {1, 1};
  const CUresult r = fn(map, type, 2, t.m->data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? B2B_OK : B2B_ERR_CUDA;
}
CUtensorMapDataType type16(const b2b_ffn_plan_s* p) {
  return p->dtype == B2B_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// One launch in the making: tensor maps, parameters, what went wrong.
struct Launch {
  const b2b_ffn_plan_s* plan;
  GemmMaps maps;
  GemmParams p;
  b2b_status_t st = B2B_OK;
  bool gate, e4m3;

  Launch(const b2b_ffn_plan_s* plan_, bool gate_, bool e4m3_) : plan(plan_), gate(gate_), e4m3(e4m3_) {
    std::memset(&maps, 0, sizeof(maps));
    std::memset(&p, 0, sizeof(p));
    p.kseg = 1 << 30;
    p.act = plan->act;
    p.debug = plan->debug;
    p.status = plan->d_status;
  }
  CUtensorMapDataType operand() const { return e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type16(plan); }
  void map(CUtensorMap* m, CUtensorMapDataType type, const Matrix& t, uint32_t cols, uint32_t rows) {
    if (st == B2B_OK) st = encode(m, type, t, cols, rows);
  }
  // K-major operands: boxes of 128 bytes of k by 128 rows (A's: fewer where it has fewer)
  void a_rows(int i, const Matrix& t) {
    p.a_box_rows = static_cast<int>(std::min<int64_t>(128, (t.rows + 7) & ~int64_t(7)));
    map(&maps.a[i], operand(), t, e4m3 ? 128 : 64, static_cast<uint32_t>(p.a_box_rows));
  }
  void b_rows(int i, const Matrix& t) { map(&maps.b[i], operand(), t, e4m3 ? 128 : 64, 128); }
  // MN-major operands, [k][m] or [k][n]: boxes of 64 by 64
  void a_cols(int i, const Matrix& t) { map(&maps.a[i], operand(), t, 64, 64); }
  void b_cols(int i, const Matrix& t) { map(&maps.b[i], operand(), t, 64, 64); }
  // output i, in boxes of a warp's 32 rows of 128 bytes
  void out(int i, const Matrix& t) {
    map(&maps.out[i], t.esz == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : type16(plan), t, t.esz == 4 ? 32 : 64, 32);
    p.out[i] = t.m->data;
    p.out_ld[i] = t.m->row_stride;
  }
  void problem(int64_t m, int64_t n) { add_problem(p, m, n, gate); }
  b2b_status_t run(const GemmKernel& kernel, int kpan, void* parts, cudaStream_t stream) {
    if (st != B2B_OK) return st;
    const int clusters = plan->sms / 2;
    set_units(p, kpan, clusters);
    p.part = static_cast<float*>(parts);
    p.budget_ns = static_cast<uint32_t>(std::min<uint64_t>(std::max<uint64_t>(plan->budget_ns, 5000ull * kpan), 4000000000ull));
    void* args[] = {&maps, &p};
    cudaError_t e = launch_pdl(kernel.main, dim3(2 * static_cast<unsigned>(std::min(p.units, clusters))), dim3(gemm_threads(e4m3)), args,
                               kGemmSmem, stream, 2);
    if (e == cudaSuccess && p.whole < p.tiles) {
      void* cargs[] = {&p};
      e = launch_pdl(kernel.combine, dim3(static_cast<unsigned>((p.tiles - p.whole) * 8), gate ? 1 : 2), dim3(512), cargs, 0, stream);
    }
    if (e != cudaSuccess) {
      cudaGetLastError();
      return B2B_ERR_CUDA;
    }
    return B2B_OK;
  }
};

// How the kernel for few rows takes a product: tiles of 16 << size rows, a slice's
// k cut in 1 << split_bits; size -1: the pair kernel is quicker.  Of `products`
// over k each.  What it compares are not times where the weights' bytes bound a
// launch, as they have no term here: the e4m3 gate of 16 tokens on 8192/28672 counts
// as 15 us, and reading its weights takes 69.  Rows of 16-bit operands that do not lie on 128 bytes cost a box two
// lines for each of its rows (309 tokens on 1408/5376/2304 28 us, on 1400/5416/2280
// 44 us here, 36 and 41 us by the pair kernel).
struct FewShape {
  int size, row_tiles, split_bits;
};
FewShape few_shape(const b2b_ffn_plan_s* p, const SkinnyKernels& k, int64_t rows, int64_t n, int64_t depth, int products = 1) {
  const bool e4m3 = k.depth == 128;
  const int kpan = products * panels(depth, e4m3);
  const double lines = e4m3 ? 1.0 : 1.0 + 0.25 * (depth % 64 != 0) + 0.25 * ((k.k_major ? depth : n) % 64 != 0);
  const int64_t room = 2 * p->sms;  // CTAs resident at once
  double best = k.cost.pair + k.cost.pair_panel * cut(tile_count(rows, n, k.gate), kpan, p->sms / 2).time;
  FewShape shape = {-1, 0, 0};
  if (p->debug & B2B_DEBUG_PAIR_KERNEL) return shape;
  for (int size = 0; size < k.sizes; ++size) {
    const int64_t row_tiles = ceil_div(rows, 16 << size), tiles = row_tiles * ceil_div(n, k.columns);
    // k cut while all CTAs are resident at once, with two slots each at least: 16 bits as
    // often as that goes (fewer cuts where this model prefers them were no quicker on
    // average), e4m3, whose slots' sums take more of an SM, where the model says so (33 x
    // 2048 x 1368 5.7 -> 4.9 us, the block of 33 tokens on 4096/2816/4096 20.4 -> 18.0).
    int most = 0;
    while ((2 << most) <= kSkinnyMaxSplits && (tiles << (most + 1)) <= room && kpan >= (4 << most)) ++most;
    for (int bits = e4m3 ? 0 : most; bits <= most; ++bits) {
      const double second = (tiles << bits) > p->sms ? 1.0 + k.cost.second : 1.0;
      const double t = static_cast<double>(ceil_div(tiles << bits, room)) * second *
                           (1.2 + static_cast<double>(ceil_div(kpan, 1 << bits)) * lines * (k.cost.slot + k.cost.slot_row * (16 << size))) +
                       0.14 * ((1 << bits) - 1);
      if (t < best) {
        best = t;
        shape = {size, static_cast<int>(row_tiles), bits};
      }
    }
    if (row_tiles == 1) break;  // (a larger tile would be emptier)
  }
  return shape;
}

// A product for few rows in the making.
struct FewRows {
  const b2b_ffn_plan_s* plan;
  const SkinnyKernels& k;
  FewShape shape;
  bool e4m3;
  SkinnyMaps maps;
  SkinnyParams p;
  b2b_status_t st = B2B_OK;

  FewRows(const b2b_ffn_plan_s* plan_, const SkinnyKernels& k_, const FewShape& shape_, bool e4m3_, const Matrix& x)
      : plan(plan_), k(k_), shape(shape_), e4m3(e4m3_) {
    std::memset(&p, 0, sizeof(p));
    p.rows = static_cast<int>(x.rows);
    p.row_tiles = shape.row_tiles;
    p.split_bits = shape.split_bits;
    p.splits = 1 << p.split_bits;
    p.x_box_rows = static_cast<int>(std::min<int64_t>(16 << shape.size, (x.rows + 7) & ~int64_t(7)));
    p.segment = 1 << 30;
    p.act = plan->act;
    p.debug = plan->debug;
    p.status = plan->d_status;
    rows(0, x);
    maps.x[1] = maps.x[0];
  }
  void rows(int i, const Matrix& x) {
    p.slots += static_cast<int>(ceil_div(x.cols, k.depth));
    if (st == B2B_OK)
      st = encode(&maps.x[i], e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type16(plan), x, e4m3 ? 128 : 64, static_cast<uint32_t>(p.x_box_rows));
  }
  // A product to add: rows and, set by weight(1, ..), their weight.
  void more(const Matrix& x) {
    p.segment = p.slots;
    rows(1, x);
  }
  void weight(int i, const Matrix& w) {
    if (st != B2B_OK) return;
    p.N = static_cast<int>(k.k_major ? w.rows : w.cols);
    st = encode(&maps.w[i], e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : type16(plan), w, e4m3 ? 128 : 64, k.k_major ? 128 : 64);
  }
  b2b_status_t run(cudaStream_t stream) {
    if (st != B2B_OK) return st;
    const int64_t ctas = ceil_div(p.N, k.columns) * p.row_tiles * p.splits;
    p.budget_ns = static_cast<uint32_t>(std::min<uint64_t>(std::max<uint64_t>(plan->budget_ns, 5000ull * p.slots), 4000000000ull));
    void* args[] = {&maps, &p};
    if (launch_pdl(k.main[shape.size], dim3(static_cast<unsigned>(ctas)), dim3(static_cast<unsigned>(k.threads[shape.size])), args, k.smem[shape.size], stream, p.splits) !=
        cudaSuccess) {
      cudaGetLastError();
      return B2B_ERR_CUDA;
    }
    return B2B_OK;
  }
};

size_t part_bytes(const b2b_ffn_plan_s* p, int64_t tiles, int kpan) { return cut(tiles, kpan, p->sms / 2).part_bytes(); }

// Workspace of a run, its pieces one after the other.
struct Pieces {
  size_t hidden = 0;       // H; or dG; or (e4m3) H's values
  size_t second = 0;       // dU; or (e4m3) X's values
  size_t x_scale = 0, h_scale = 0;
  size_t parts = 0;
  size_t total() const { return rounded(hidden) + rounded(second) + rounded(x_scale) + rounded(h_scale) + parts; }
};

// What a forward pass keeps: G and U, then H.
struct Kept {
  int64_t blocks;     // of 32 columns
  size_t each;        // bytes of G, of U
  size_t total;
  Kept(const b2b_ffn_plan_s* p, int64_t tokens) {
    blocks = ceil_div(p->hidden, 32);
    each = static_cast<size_t>(ceil_div(tokens, 32)) * static_cast<size_t>(blocks) * 4096;
    total = 2 * each + rounded(static_cast<size_t>(tokens) * p->hidden * 2);
  }
  template <class P>
  void set(P& p, const void* kept) const {
    p.kept_gate = static_cast<float*>(const_cast<void*>(kept));
    p.kept_up = p.kept_gate + each / 4;
    p.kept_blocks = static_cast<int>(blocks);
  }
  void* hidden(const void* kept) const { return static_cast<uint8_t*>(const_cast<void*>(kept)) + 2 * each; }
};

const SkinnyKernels& product_few(const b2b_ffn_plan_s* p) { return p->s.product_few[p->dtype == B2B_BF16]; }

Pieces pieces(const b2b_ffn_plan_s* p, int64_t rows, int pass) {
  Pieces w;
  const int64_t d = p->width, f = p->hidden, o = p->out_width;
  const size_t t = static_cast<size_t>(rows);
  auto part = [&](int64_t tiles, int kpan) { w.parts = std::max(w.parts, part_bytes(p, tiles, kpan)); };
  auto product = [&](const SkinnyKernels& k, int64_t n, int64_t depth, int products = 1) {
    if (few_shape(p, k, rows, n, depth, products).size < 0) part(tile_count(rows, n, k.gate), products * panels(depth, k.depth == 128));
  };
  if (p->kind == kScaledGemm) {
    product(product_few(p), o, d);
  } else if (p->kind == kScaledFfn) {
    w.hidden = t * f;
    w.second = t * d;
    w.x_scale = 4 * t * ceil_div(d, 128);
    w.h_scale = 4 * t * ceil_div(f, 128);
    product(p->s.gate_few, f, d);
    product(product_few(p), o, f);
  } else if (pass == B2B_FFN_BACKWARD) {
    w.hidden = w.second = 2 * t * f;
    product(p->k.gate_grad_few, f, o);
    product(p->k.dx_few, d, f, 2);
    // (any of the weights' gradients may be left out)
    for (int g = 0; g <= 2; ++g)
      for (int e = 0; e <= 1; ++e)
        if (g + e) part(g * tile_count(d, f, false) + e * tile_count(f, o, false), panels(rows));
  } else {
    w.hidden = pass == B2B_FFN_TRAINING ? 0 : 2 * t * f;
    product(p->k.gate_few, f, d);
    product(p->k.down_few, o, f);
  }
  return w;
}

b2b_status_t create(b2b_ffn_plan_t* out, FfnKind kind, b2b_dtype_t dtype, int64_t width, int64_t hidden, int64_t out_width, int act) {
  if (!out) return B2B_ERR_INVALID_ARG;
  *out = nullptr;
  if (dtype < B2B_F16_F32OUT || dtype > B2B_TF32_BF16) return B2B_ERR_INVALID_ARG;
  if (width < 1 || hidden < 1 || out_width < 1 || (act != B2B_SILU && act != B2B_GELU_TANH)) return B2B_ERR_INVALID_ARG;
  const int64_t k_unit = kind == kFfn ? 8 : 16, n_unit = kind == kScaledGemm ? 8 : k_unit;
  if (!is16(dtype) || width % k_unit || hidden % k_unit || out_width % n_unit || width > kMaxExtent || hidden > kMaxExtent ||
      out_width > kMaxExtent)
    return B2B_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  const b2b_status_t st = check_device(&dev, &sms);
  if (st != B2B_OK) return st;
  b2b_ffn_plan_s* p = new (std::nothrow) b2b_ffn_plan_s();
  if (!p) return B2B_ERR_CUDA;
  p->kind = kind;
  p->dtype = dtype;
  p->device = dev;
  p->sms = sms;
  p->width = width;
  p->hidden = hidden;
  p->out_width = out_width;
  p->act = act;
  p->k = dtype == B2B_F16 ? ffn_kernels_f16() : ffn_kernels_bf16();
  p->s = scaled_kernels();
  p->budget_ns = kDefaultBudgetNs;
  // Shared memory of the kernels that this kind of plan launches.
  bool ok = true;
  auto use = [&](const GemmKernel& k) {
    ok = ok && cudaFuncSetAttribute(k.main, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem) == cudaSuccess;
  };
  auto use_few = [&](const SkinnyKernels& k) {
    for (int i = 0; i < k.sizes; ++i)
      ok = ok && cudaFuncSetAttribute(k.main[i], cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem[i]) == cudaSuccess;
  };
  // The registers of the e4m3 kernels' roles (setmaxnreg) are drawn from what
  // the kernel is launched with: compiled to fewer, it would wait for them.
  auto use_e4m3 = [&](const GemmKernel& k) {
    use(k);
    cudaFuncAttributes fa;
    ok = ok && cudaFuncGetAttributes(&fa, k.main) == cudaSuccess &&
         fa.numRegs * gemm_threads(true) >= 512 * kGemmEpilogueRegs + 128 * kGemmOtherRegs;
  };
  if (kind == kFfn) {
    for (const GemmKernel& k : {p->k.gate, p->k.down, p->k.gate_grad, p->k.dx, p->k.dw, p->k.dw_add}) use(k);
    use_few(p->k.gate_few);
    use_few(p->k.down_few);
    use_few(p->k.gate_grad_few);
    use_few(p->k.dx_few);
  } else {
    use_e4m3(p->s.product[dtype == B2B_BF16]);
    use_few(product_few(p));
    if (kind == kScaledFfn) {
      use_e4m3(p->s.gate);
      use_few(p->s.gate_few);
    }
  }
  ok = ok && cudaMalloc(&p->d_status, sizeof(int)) == cudaSuccess;
  if (ok && cudaMemset(p->d_status, 0, sizeof(int)) != cudaSuccess) {
    cudaFree(p->d_status);
    ok = false;
  }
  if (!ok) {
    cudaGetLastError();
    delete p;
    return B2B_ERR_CUDA;
  }
  *out = p;
  return B2B_OK;
}

b2b_status_t scaled_few(const b2b_ffn_plan_s* p, const FewShape& shape, const Matrix& a, const b2b_scales_t& a_scale, const Matrix& b,
                        const b2b_scales_t& b_scale, const Matrix& out, cudaStream_t stream) {
  FewRows l(p, product_few(p), shape, true, a);
  l.weight(0, b);
  l.p.out = out.m->data;
  l.p.out_ld = out.m->row_stride;
  l.p.a_scale = a_scale.data;
  l.p.a_scale_row = a_scale.row_stride;
  l.p.a_scale_k = a_scale.block_stride;
  l.p.b_scale[0] = b_scale.data;
  l.p.b_scale_row[0] = b_scale.row_stride;
  l.p.b_scale_k[0] = b_scale.block_stride;
  return l.run(stream);
}

// The 16-bit quantiser's launch.
b2b_status_t quantize(const FfnKernels& k, int64_t rows, int64_t cols, int block_rows, const b2b_matrix_t& x, const b2b_matrix_t& q,
                      const b2b_scales_t& scale, cudaStream_t stream) {
  QuantParams p;
  p.rows = rows;
  p.cols = cols;
  p.x = x.data;
  p.x_ld = x.row_stride;
  p.q = static_cast<uint8_t*>(q.data);
  p.q_ld = q.row_stride;
  p.scale = scale.data;
  p.scale_row = scale.row_stride;
  p.scale_k = scale.block_stride;
  void* args[] = {&p};
  const int64_t per = block_rows == 1 ? kQuantThreads / 16 : 128;
  const dim3 grid(static_cast<unsigned>(ceil_div(rows, per)),
                  static_cast<unsigned>(std::min<int64_t>(ceil_div(cols, block_rows == 1 ? 128 * kQuantBlocks : 128), 65535)));
  if (launch_pdl(block_rows == 1 ? k.quantize_rows : k.quantize_tiles, grid, dim3(kQuantThreads), args, 0, stream) != cudaSuccess) {
    cudaGetLastError();
    return B2B_ERR_CUDA;
  }
  return B2B_OK;
}

b2b_status_t check_tiles(const b2b_ffn_plan_s* p, int64_t rows) {
  if (rows > kMaxRows) return B2B_ERR_UNSUPPORTED;
  const int64_t most = std::max(std::max(p->hidden, p->out_width), p->width);
  return tile_count(rows, most, true) > kMaxTiles || 2 * tile_count(p->hidden, most, false) > kMaxTiles ? B2B_ERR_UNSUPPORTED : B2B_OK;
}

}  // namespace

extern "C" {

b2b_status_t b2b_ffn_plan_create(b2b_ffn_plan_t* out, b2b_dtype_t dtype, int64_t width, int64_t hidden, int64_t out_width,
                                 b2b_activation_t activation) {
  return create(out, kFfn, dtype, width, hidden, out_width, activation);
}

b2b_status_t b2b_scaled_ffn_plan_create(b2b_ffn_plan_t* out, b2b_dtype_t dtype, int64_t width, int64_t hidden, int64_t out_width,
                                        b2b_activation_t activation) {
  return create(out, kScaledFfn, dtype, width, hidden, out_width, activation);
}

b2b_status_t b2b_scaled_gemm_plan_create(b2b_ffn_plan_t* out, b2b_dtype_t dtype, int64_t k, int64_t n) {
  return create(out, kScaledGemm, dtype, k, 16, n, B2B_SILU);
}

b2b_status_t b2b_ffn_plan_destroy(b2b_ffn_plan_t p) {
  if (!p) return B2B_OK;
  cudaFree(p->d_status);
  delete p;
  return B2B_OK;
}

b2b_status_t b2b_ffn_plan_device_status(b2b_ffn_plan_t p, b2b_stream_t stream) {
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

b2b_status_t b2b_ffn_plan_set_wait_budget(b2b_ffn_plan_t p, uint64_t budget_ns) {
  if (!p) return B2B_ERR_INVALID_ARG;
  p->budget_ns = budget_ns ? std::max<uint64_t>(budget_ns, kMinBudgetNs) : kDefaultBudgetNs;
  return B2B_OK;
}

b2b_status_t b2b_ffn_plan_set_debug(b2b_ffn_plan_t p, uint32_t flags) {
  if (!p) return B2B_ERR_INVALID_ARG;
  if (flags & ~(B2B_DEBUG_DROP_FIRST_LOAD | B2B_DEBUG_PAIR_KERNEL)) return B2B_ERR_INVALID_ARG;
  p->debug = flags;
  return B2B_OK;
}

b2b_status_t b2b_ffn_workspace(b2b_ffn_plan_t p, int64_t rows, int pass, size_t* bytes) {
  if (!p || !bytes || rows < 0 || pass < B2B_FFN_INFERENCE || pass > B2B_FFN_BACKWARD) return B2B_ERR_INVALID_ARG;
  if (p->kind != kFfn && pass != B2B_FFN_INFERENCE) return B2B_ERR_INVALID_ARG;
  const b2b_status_t st = check_tiles(p, rows);
  if (st != B2B_OK) return st;
  *bytes = rows ? pieces(p, rows, pass).total() : 0;
  return B2B_OK;
}

b2b_status_t b2b_ffn_kept_bytes(b2b_ffn_plan_t p, int64_t tokens, size_t* bytes) {
  if (!p || !bytes || tokens < 0 || p->kind != kFfn) return B2B_ERR_INVALID_ARG;
  const b2b_status_t st = check_tiles(p, tokens);
  if (st != B2B_OK) return st;
  *bytes = tokens ? Kept(p, tokens).total : 0;
  return B2B_OK;
}

b2b_status_t b2b_ffn_forward(b2b_ffn_plan_t p, const b2b_ffn_forward_t* r, b2b_stream_t stream_) {
  if (!p || !r || p->kind != kFfn || r->tokens < 0) return B2B_ERR_INVALID_ARG;
  const int64_t t = r->tokens, d = p->width, f = p->hidden, o = p->out_width;
  b2b_status_t st = check_tiles(p, t);
  if (st != B2B_OK || t == 0) return st;
  if (!r->out.data) return B2B_ERR_INVALID_ARG;
  const bool keep = r->kept != nullptr;
  const Kept kept(p, t);
  const int64_t kept_row = keep ? static_cast<int64_t>(kept.total) : 0;
  const b2b_matrix_t kept_bytes = {r->kept, kept_row};
  const Matrix in[] = {{&r->x, t, d, 2}, {&r->w_gate, d, f, 2}, {&r->w_up, d, f, 2}, {&r->w_down, f, o, 2}};
  const Matrix out[] = {{&r->out, t, o, 2}, {&kept_bytes, 1, kept_row, 1}};
  if (keep) st = check_workspace(r->kept, r->kept_bytes, kept.total);
  if (st == B2B_OK) st = check_all(in, out);
  const Pieces w = pieces(p, t, keep ? B2B_FFN_TRAINING : B2B_FFN_INFERENCE);
  if (st == B2B_OK) st = check_workspace(r->workspace, r->workspace_bytes, w.total());
  if (st == B2B_OK) st = check_current_device(p);
  if (st != B2B_OK) return st;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  uint8_t* ws = static_cast<uint8_t*>(r->workspace);
  const b2b_matrix_t h_rows = {keep ? kept.hidden(r->kept) : ws, f};
  void* parts = ws + rounded(w.hidden);
  const Matrix h = {&h_rows, t, f, 2};
  const FewShape up_few = few_shape(p, p->k.gate_few, t, f, d), down_few = few_shape(p, p->k.down_few, t, o, f);
  if (up_few.size >= 0) {
    FewRows l(p, p->k.gate_few, up_few, false, in[0]);
    l.weight(0, in[1]);
    l.weight(1, in[2]);
    l.p.out = h_rows.data;
    l.p.out_ld = f;
    if (keep) kept.set(l.p, r->kept);
    st = l.run(stream);
  } else {
    Launch l(p, true, false);
    l.a_rows(0, in[0]);
    l.b_cols(0, in[1]);
    l.b_cols(1, in[2]);
    l.out(0, h);
    if (keep) kept.set(l.p, r->kept);
    l.problem(t, f);
    st = l.run(p->k.gate, panels(d), parts, stream);
  }
  if (st != B2B_OK) return st;
  if (down_few.size >= 0) {
    FewRows l(p, p->k.down_few, down_few, false, h);
    l.weight(0, in[3]);
    l.p.out = r->out.data;
    l.p.out_ld = r->out.row_stride;
    return l.run(stream);
  }
  Launch l(p, false, false);
  l.a_rows(0, h);
  l.b_cols(0, in[3]);
  l.out(0, out[0]);
  l.problem(t, o);
  return l.run(p->k.down, panels(f), parts, stream);
}

b2b_status_t b2b_ffn_backward(b2b_ffn_plan_t p, const b2b_ffn_backward_t* r, b2b_stream_t stream_) {
  if (!p || !r || p->kind != kFfn || r->tokens < 0) return B2B_ERR_INVALID_ARG;
  const int64_t t = r->tokens, d = p->width, f = p->hidden, o = p->out_width;
  b2b_status_t st = check_tiles(p, t);
  if (st != B2B_OK) return st;
  const int gsz = r->accumulate ? 4 : 2;
  const Kept kept(p, t);
  const int64_t kept_row = t ? static_cast<int64_t>(kept.total) : 0;
  const b2b_matrix_t kept_bytes = {const_cast<void*>(r->kept), kept_row}, h_rows = {kept.hidden(r->kept), f};
  const Matrix in[] = {{&r->dy, t, o, 2},   {&r->x, t, d, 2},      {&r->w_gate, d, f, 2},
                       {&r->w_up, d, f, 2}, {&r->w_down, f, o, 2}, {&kept_bytes, t ? 1 : 0, kept_row, 1}};
  const Matrix h = {&h_rows, t, f, 2};
  const Matrix out[] = {{&r->dx, t, d, 2}, {&r->dw_gate, d, f, gsz}, {&r->dw_up, d, f, gsz}, {&r->dw_down, f, o, gsz}};
  if (t) st = check_workspace(r->kept, r->kept_bytes, kept.total);
  if (st == B2B_OK) st = check_all(in, out);
  const Pieces w = pieces(p, t, B2B_FFN_BACKWARD);
  if (st == B2B_OK) st = check_workspace(r->workspace, r->workspace_bytes, t ? w.total() : 0);
  if (st == B2B_OK) st = check_current_device(p);
  if (st != B2B_OK) return st;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (t == 0) {
    // no token: gradients of weights are zero
    for (int i = 1; i < 4 && !r->accumulate; ++i)
      if (out[i].m->data && cudaMemset2DAsync(out[i].m->data, out[i].stride_bytes(), 0, out[i].row_bytes(),
                                              static_cast<size_t>(out[i].rows), stream) != cudaSuccess) {
        cudaGetLastError();
        return B2B_ERR_CUDA;
      }
    return B2B_OK;
  }
  uint8_t* ws = static_cast<uint8_t*>(r->workspace);
  const b2b_matrix_t dg_rows = {ws, f}, du_rows = {ws + rounded(w.hidden), f};
  void* parts = ws + rounded(w.hidden) + rounded(w.second);
  const Matrix dg = {&dg_rows, t, f, 2}, du = {&du_rows, t, f, 2};
  const FewShape grad_few = few_shape(p, p->k.gate_grad_few, t, f, o), dx_few = few_shape(p, p->k.dx_few, t, d, f, 2);
  if (r->dx.data || r->dw_gate.data || r->dw_up.data) {
    if (grad_few.size >= 0) {
      FewRows l(p, p->k.gate_grad_few, grad_few, false, in[0]);
      l.weight(0, in[4]);
      l.p.out = dg_rows.data;
      l.p.out2 = du_rows.data;
      l.p.out_ld = f;
      kept.set(l.p, r->kept);
      st = l.run(stream);
    } else {
      Launch l(p, false, false);
      l.a_rows(0, in[0]);
      l.b_rows(0, in[4]);
      l.out(0, dg);
      l.out(1, du);
      kept.set(l.p, r->kept);
      l.problem(t, f);
      st = l.run(p->k.gate_grad, panels(o), parts, stream);
    }
  }
  if (st == B2B_OK && r->dx.data) {
    if (dx_few.size >= 0) {
      FewRows l(p, p->k.dx_few, dx_few, false, dg);
      l.weight(0, in[2]);
      l.more(du);
      l.weight(1, in[3]);
      l.p.out = r->dx.data;
      l.p.out_ld = r->dx.row_stride;
      st = l.run(stream);
    } else {
      Launch l(p, false, false);
      l.a_rows(0, dg);
      l.a_rows(1, du);
      l.b_rows(0, in[2]);
      l.b_rows(1, in[3]);
      l.out(0, out[0]);
      l.p.kseg = panels(f);
      l.problem(t, d);
      st = l.run(p->k.dx, 2 * panels(f), parts, stream);
    }
  }
  if (st == B2B_OK && (r->dw_gate.data || r->dw_up.data || r->dw_down.data)) {
    Launch l(p, false, false);
    auto add = [&](const Matrix& a, const Matrix& b, const Matrix& c) {
      if (!c.m->data) return;
      l.a_cols(l.p.problems, a);
      l.b_cols(l.p.problems, b);
      l.out(l.p.problems, c);
      l.problem(c.rows, c.cols);
    };
    add(in[1], dg, out[1]);
    add(in[1], du, out[2]);
    add(h, in[0], out[3]);
    st = l.run(r->accumulate ? p->k.dw_add : p->k.dw, panels(t), parts, stream);
  }
  return st;
}

b2b_status_t b2b_scaled_ffn_run(b2b_ffn_plan_t p, const b2b_scaled_ffn_t* r, b2b_stream_t stream_) {
  if (!p || !r || p->kind != kScaledFfn || r->tokens < 0) return B2B_ERR_INVALID_ARG;
  const int64_t t = r->tokens, d = p->width, f = p->hidden, o = p->out_width;
  b2b_status_t st = check_tiles(p, t);
  if (st != B2B_OK || t == 0) return st;
  if (!r->out.data) return B2B_ERR_INVALID_ARG;
  const int64_t db = ceil_div(d, 128), fb = ceil_div(f, 128), ob = ceil_div(o, 128);
  const Matrix in[] = {{&r->x, t, d, 2}, {&r->w_gate, f, d, 1}, {&r->w_up, f, d, 1}, {&r->w_down, o, f, 1}};
  const Matrix out[] = {{&r->out, t, o, 2}};
  st = check_all(in, out);
  const b2b_scales_t* scales[] = {&r->gate_scale, &r->up_scale, &r->down_scale};
  const int64_t scale_rows[] = {fb, fb, ob}, scale_blocks[] = {db, db, fb};
  for (int i = 0; i < 3; ++i) {
    if (st == B2B_OK) st = check(*scales[i], scale_rows[i]);
    if (st == B2B_OK && overlaps_scales(out[0], *scales[i], scale_rows[i], scale_blocks[i])) st = B2B_ERR_ALIAS;
  }
  const Pieces w = pieces(p, t, B2B_FFN_INFERENCE);
  if (st == B2B_OK) st = check_workspace(r->workspace, r->workspace_bytes, w.total());
  if (st == B2B_OK) st = check_current_device(p);
  if (st != B2B_OK) return st;
  const cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  uint8_t* ws = static_cast<uint8_t*>(r->workspace);
  const b2b_matrix_t hq = {ws, f}, xq = {ws + rounded(w.hidden), d};
  // scales of rows, one block's after the other's
  float* xs = reinterpret_cast<float*>(ws + rounded(w.hidden) + rounded(w.second));
  float* hs = xs + rounded(w.x_scale) / 4;
  void* parts = hs + rounded(w.h_scale) / 4;
  st = quantize(p->k, t, d, 1, r->x, xq, {xs, 1, t}, stream);
  if (st != B2B_OK) return st;
  const FewShape up_few = few_shape(p, p->s.gate_few, t, f, d), down_few = few_shape(p, product_few(p), t, o, f);
  if (up_few.size >= 0) {
    FewRows l(p, p->s.gate_few, up_few, true, {&xq, t, d, 1});
    l.weight(0, in[1]);
    l.weight(1, in[2]);
    l.p.out = ws;
    l.p.out_ld = f;
    l.p.a_scale = xs;
    l.p.a_scale_row = 1;
    l.p.a_scale_k = t;
    for (int i = 0; i < 2; ++i) {
      l.p.b_scale[i] = scales[i]->data;
      l.p.b_scale_row[i] = scales[i]->row_stride;
      l.p.b_scale_k[i] = scales[i]->block_stride;
    }
    l.p.q_scale = hs;
    l.p.q_scale_ld = t;
    st = l.run(stream);
  } else {
    Launch l(p, true, true);
    l.a_rows(0, {&xq, t, d, 1});
    l.b_rows(0, in[1]);
    l.b_rows(1, in[2]);
    l.p.a_scale = xs;
    l.p.a_scale_row = 1;
    l.p.a_scale_k = t;
    for (int i = 0; i < 2; ++i) {
      l.p.b_scale[i] = scales[i]->data;
      l.p.b_scale_row[i] = scales[i]->row_stride;
      l.p.b_scale_k[i] = scales[i]->block_stride;
    }
    l.p.q = ws;
    l.p.q_ld = f;
    l.p.q_scale = hs;
    l.p.q_scale_ld = t;
    l.problem(t, f);
    st = l.run(p->s.gate, panels(d, true), parts, stream);
  }
  if (st != B2B_OK) return st;
  if (down_few.size >= 0) return scaled_few(p, down_few, {&hq, t, f, 1}, {hs, 1, t}, in[3], r->down_scale, out[0], stream);
  Launch l(p, false, true);
  l.a_rows(0, {&hq, t, f, 1});
  l.b_rows(0, in[3]);
  l.out(0, out[0]);
  l.p.a_scale = hs;
  l.p.a_scale_row = 1;
  l.p.a_scale_k = t;
  l.p.b_scale[0] = r->down_scale.data;
  l.p.b_scale_row[0] = r->down_scale.row_stride;
  l.p.b_scale_k[0] = r->down_scale.block_stride;
  l.problem(t, o);
  return l.run(p->s.product[p->dtype == B2B_BF16], panels(f, true), parts, stream);
}

b2b_status_t b2b_scaled_gemm_run(b2b_ffn_plan_t p, const b2b_scaled_gemm_t* r, b2b_stream_t stream_) {
  if (!p || !r || p->kind != kScaledGemm || r->rows < 0) return B2B_ERR_INVALID_ARG;
  const int64_t m = r->rows, k = p->width, n = p->out_width;
  b2b_status_t st = check_tiles(p, m);
  if (st != B2B_OK || m == 0) return st;
  if (!r->out.data) return B2B_ERR_INVALID_ARG;
  const int64_t kb = ceil_div(k, 128), nb = ceil_div(n, 128);
  const Matrix in[] = {{&r->a, m, k, 1}, {&r->b, n, k, 1}};
  const Matrix out[] = {{&r->out, m, n, 2}};
  st = check_all(in, out);
  if (st == B2B_OK) st = check(r->a_scale, m);
  if (st == B2B_OK) st = check(r->b_scale, nb);
  if (st == B2B_OK && (overlaps_scales(out[0], r->a_scale, m, kb) || overlaps_scales(out[0], r->b_scale, nb, kb))) st = B2B_ERR_ALIAS;
  const Pieces w = pieces(p, m, B2B_FFN_INFERENCE);
  if (st == B2B_OK) st = check_workspace(r->workspace, r->workspace_bytes, w.total());
  if (st == B2B_OK) st = check_current_device(p);
  if (st != B2B_OK) return st;
  const FewShape few = few_shape(p, product_few(p), m, n, k);
  if (few.size >= 0)
    return scaled_few(p, few, in[0], r->a_scale, in[1], r->b_scale, out[0], reinterpret_cast<cudaStream_t>(stream_));
  Launch l(p, false, true);
  l.a_rows(0, in[0]);
  l.b_rows(0, in[1]);
  l.out(0, out[0]);
  l.p.a_scale = r->a_scale.data;
  l.p.a_scale_row = r->a_scale.row_stride;
  l.p.a_scale_k = r->a_scale.block_stride;
  l.p.b_scale[0] = r->b_scale.data;
  l.p.b_scale_row[0] = r->b_scale.row_stride;
  l.p.b_scale_k[0] = r->b_scale.block_stride;
  l.problem(m, n);
  return l.run(p->s.product[p->dtype == B2B_BF16], panels(k, true), r->workspace, reinterpret_cast<cudaStream_t>(stream_));
}

b2b_status_t b2b_ffn_units(int problems, const int64_t* sizes, int gate, int64_t kpan, int clusters, int64_t* out, int nout) {
  if (!sizes || !out || problems < 1 || problems > kGemmMaxProblems || kpan < 1 || kpan > kMaxRows || clusters < 1) return B2B_ERR_INVALID_ARG;
  GemmParams p;
  std::memset(&p, 0, sizeof(p));
  for (int i = 0; i < problems; ++i) {
    const int64_t m = sizes[2 * i], n = sizes[2 * i + 1];
    if (m < 1 || n < 1 || m > kMaxRows || n > kMaxExtent || tile_count(m, n, gate) > kMaxTiles) return B2B_ERR_INVALID_ARG;
    add_problem(p, m, n, gate);
  }
  set_units(p, static_cast<int>(kpan), clusters);
  if (nout < 1 + 6 * p.units) return B2B_ERR_INVALID_ARG;
  *out++ = p.units;
  for (int u = 0; u < p.units; ++u) {
    const GemmUnit c = gemm_unit(p, u);
    for (const int v : {c.prob, c.mt, c.nt, c.k0, c.k1, c.part}) *out++ = v;
  }
  return B2B_OK;
}

b2b_status_t b2b_quantize_blocks(b2b_dtype_t dtype, int64_t rows, int64_t cols, int block_rows, const b2b_matrix_t* x,
                                 const b2b_matrix_t* q, const b2b_scales_t* scale, b2b_stream_t stream) {
  if (dtype < B2B_F16_F32OUT || dtype > B2B_TF32_BF16 || rows < 0 || cols < 0 || !x || !q || !scale) return B2B_ERR_INVALID_ARG;
  if (block_rows != 1 && block_rows != 128) return B2B_ERR_INVALID_ARG;
  if (!is16(dtype) || cols % 8 || rows > kMaxRows || cols > kMaxRows) return B2B_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return B2B_OK;
  const Matrix xm = {x, rows, cols, 2}, qm = {q, rows, cols, 1};
  b2b_status_t st = check(xm);
  if (st == B2B_OK) st = check(qm, 8);
  const int64_t scale_rows = ceil_div(rows, block_rows), blocks = ceil_div(cols, 128);
  if (st == B2B_OK) st = check(*scale, scale_rows);
  // (scales are written: one direction's stride steps over the other's whole extent, so that blocks share none)
  const double by_row = static_cast<double>(scale->row_stride), by_block = static_cast<double>(scale->block_stride);
  const bool apart = scale_rows == 1 ? blocks == 1 || by_block > 0
                                     : by_row > 0 && (blocks == 1 || (by_block > 0 && (by_row > static_cast<double>(blocks - 1) * by_block ||
                                                                                       by_block > static_cast<double>(scale_rows - 1) * by_row)));
  if (st == B2B_OK && !apart) st = B2B_ERR_INVALID_ARG;
  if (st == B2B_OK && (share(xm, qm) || overlaps_scales(xm, *scale, scale_rows, blocks) || overlaps_scales(qm, *scale, scale_rows, blocks)))
    st = B2B_ERR_ALIAS;
  if (st == B2B_OK) st = check_device(nullptr, nullptr);
  if (st != B2B_OK) return st;
  return quantize(dtype == B2B_F16 ? ffn_kernels_f16() : ffn_kernels_bf16(), rows, cols, block_rows, *x, *q, *scale,
                  reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
