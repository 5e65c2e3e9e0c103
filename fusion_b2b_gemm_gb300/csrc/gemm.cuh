// GEMMs of the feed-forward operators on pairs of SMs (tcgen05, cta_group::2,
// sm_103a), each with the step that follows it in its epilogue:
//
//   kEpiStore      D = A.B
//   kEpiAdd        D += A.B                       (fp32 D)
//   kEpiGate       H = act(A.Bg) * (A.Bu)         (and, kept for the backward pass, G = A.Bg and U = A.Bu)
//   kEpiGateGrad   dU = (A.B) act(G), dG = (A.B) U act'(G)
//   kEpiGateQuant  as kEpiGate, brought to e4m3 with a scale for each 128 of a row
//
// act(g) = g s(u(g)), s(u) = 1 / (1 + e^-u), u = g (silu) or 2 sqrt(2/pi) (g +
// 0.044715 g^3) (gelu, tanh form: (1 + tanh z) / 2 = s(2 z)), and act'(g) =
// s + g s (1 - s) u'(g).
//
// G and U are kept in fp32: with both rounded to 16 bits the gradients that come
// of them were 1.8 times as far off as their own two roundings make them.  They
// are kept in blocks of 32 rows by 32 columns, four columns of every row together
// (gemm_kept_at), so that a warp of the epilogue, a row to a lane, writes and
// reads 512 consecutive bytes.
//
// A pair of CTAs computes a tile of 256 rows by 256 columns: each CTA holds 128
// rows of A and of the accumulator, and half of B's columns.  In kEpiGate the
// even CTA's half are 128 columns of Bg, the odd CTA's the same columns of Bu,
// so one accumulator row has the gate in its first 128 columns and the other
// projection in its last 128: both products with one read of A, and the epilogue
// finds a pair of values in one thread.  16-bit operands are read as stored,
// K-major or MN-major (AMN, BMN); 64 of them, or 128 e4m3 values, are a 128-byte
// K panel, the ring's unit.  Tensor memory holds two accumulators, so that a
// tile's epilogue runs beside the next tile's MMAs.
//
// e4m3 operands carry a scale for each 128 of k: every K panel's product is an
// accumulator of its own, which the epilogue's warps multiply by its scales and
// add up in registers in fp32 while the next panel's MMAs run.  A warp's wait for
// a panel, its loads and its release are some 500 cycles of latencies, as long
// as the MMAs take, so that sixteen warps of 64 columns share the work, 16 columns
// at a time, which also keeps the sums in registers: 8192 x 4096 x 14336 takes 385 us;
// with eight warps of 128 columns 450, with 32 columns at a time, where three
// values are spilled, 491 us; without the additions 283 us.  Two more warps hand
// the epilogue its scales, four panels ahead (each warp's own loads, one panel
// ahead: 505 us); the barrier that announces a panel's product announces these too.
//
// Work units.  A unit is a tile, or, of the last tiles, which would fill the
// SMs a fraction of a time only, a range of the tile's K panels: such a unit
// writes its accumulator as one part in fp32, and gemm_combine_kernel adds
// the parts of a tile in a fixed order and takes the epilogue's step.
//
// Roles (384 threads, one CTA per SM, persistent over units):
//   warp 0      TMA loads of this CTA's half of each panel
//   warp 1      the even CTA's elected thread issues the MMAs
//   warp 2      tensor-memory allocation
//   warps 2, 3  e4m3: scales of 64 rows each, and of the columns, for every panel
//   warps 4-11  epilogue, two warps for each quadrant of 32 rows: columns [0, 128)
//               and [128, 256), or the halves of the gate's and the other projection's 128
//   warps 4-19  the same for e4m3, four warps for each quadrant, a quarter each
// Every wait is bounded, as in the chain kernels.
#pragma once

#include <cuda.h>
#include <cstdint>

#include "chain_tc.cuh"
#include "ptx.cuh"

namespace b2b {

// epilogue warps and threads of a CTA
__host__ __device__ constexpr int gemm_warps(bool e4m3) { return e4m3 ? 16 : 8; }
__host__ __device__ constexpr int gemm_threads(bool e4m3) { return 128 + 32 * gemm_warps(e4m3); }
// panels in its ring: one less where the epilogue takes twice the room (two boxes for a warp, or twice the warps)
__host__ __device__ constexpr int gemm_ring(bool wide) { return wide ? 5 : 6; }
constexpr int kGemmTile = 256;     // rows and columns of a pair's tile
constexpr int kGemmSlot = 2 * kPanelBytes;  // a panel of A and one of B, 128 rows or columns of 128 bytes each
constexpr int kGemmStage = 4096;   // output box of a warp: 32 rows of 128 bytes
__host__ __device__ constexpr int gemm_off_stage(bool wide) { return gemm_ring(wide) * kGemmSlot; }
constexpr int kGemmOffScales = 6 * kGemmSlot + 8 * kGemmStage;  // e4m3: [3][128] scales of rows, [3][2] of columns
static_assert(gemm_off_stage(false) + 8 * kGemmStage == kGemmOffScales && gemm_off_stage(true) + 16 * kGemmStage == kGemmOffScales, "");
constexpr int kGemmOffBar = kGemmOffScales + 1536 + 32;
constexpr int kGemmSmem = kGemmOffBar + 256 + 1024;  // (the ring begins on a 1024-byte boundary)
static_assert(kGemmSmem <= 232448, "shared memory of a CTA");
// e4m3: registers of an epilogue thread and of another; 96 of each thread at launch, shared out anew
constexpr int kGemmEpilogueRegs = 104, kGemmOtherRegs = 64;
static_assert(512 * kGemmEpilogueRegs + 128 * kGemmOtherRegs <= 96 * gemm_threads(true), "register file");
constexpr int kGemmPartFloats = 2 * 128 * kGemmTile;  // a unit's part, both CTAs
constexpr int kGemmMaxProblems = 3;

enum : int { kGemmF16 = 0, kGemmBF16 = 1, kGemmE4M3 = 2 };  // operands (outputs: the first two)
enum : int { kEpiStore = 0, kEpiAdd = 1, kEpiGate = 2, kEpiGateGrad = 3, kEpiGateQuant = 4 };

enum : int {  // barrier slots (8 bytes each)
  kGBFull = 0,       // [8] panel landed in both CTAs (even CTA's)
  kGBEmpty = 8,      // [8] panel read
  kGBAccFull = 16,   // [2] accumulator complete
  kGBAccEmpty = 18,  // [2] accumulator read in both CTAs (even CTA's)
  kGBDrain = 20,
  kGBTop = 21,       // [4] the warps of a quadrant have written their rows' largest magnitudes
  kGSlotTmem = 25,   // uint32 tensor-memory base, then the int abort flag
  kGSlotEnd = 26,    // nothing, then the uint32 where the ring's loader stopped
};

// One product of a launch: D [M][N].  Tiles are numbered problem after problem.
struct GemmProblem {
  int first;             // first tile
  int m_tiles, n_tiles;  // of 256 rows; of 256 columns (gate: of 128)
  int M, N;
};

struct GemmParams {
  GemmProblem prob[kGemmMaxProblems];
  int problems;
  int tiles, whole;   // in all; computed as one unit each
  int splits;         // units of each of the others
  int units;
  int kpan;           // K panels of a product (all segments)
  int kseg;           // K panels of the first segment (then A and B go on in the second maps)
  int a_box_rows;     // rows of A's boxes (fewer than 128 for few rows: the others are never looked at)
  int group;          // 256-row tiles that share a pass over the columns
  int act;            // activation: 0 silu, 1 gelu
  // G and U, of kept_blocks blocks of 32 columns (kEpiGate: null, or written; kEpiGateGrad: read)
  float* kept_gate;
  float* kept_up;
  int kept_blocks;
  // e4m3: scales of A's rows and of B's blocks of 128 columns ([0]; [1]: the other projection's)
  const float* a_scale;
  long long a_scale_row, a_scale_k;
  const float* b_scale[2];
  long long b_scale_row[2], b_scale_k[2];
  // kEpiGateQuant: values and scales (scale of row r and block b at q_scale[b * q_scale_ld + r])
  uint8_t* q;
  long long q_ld;
  float* q_scale;
  long long q_scale_ld;
  // parts, and the outputs as gemm_combine_kernel writes them
  float* part;
  void* out[kGemmMaxProblems];
  long long out_ld[kGemmMaxProblems];
  uint32_t debug;     // bit 0: arm the first panel but never fill it
  int* status;
  uint32_t budget_ns;
};

struct GemmMaps {
  CUtensorMap a[kGemmMaxProblems], b[kGemmMaxProblems], out[kGemmMaxProblems];
};

struct GemmUnit {
  int prob, mt, nt;
  int k0, k1;   // K panels
  int part;     // number of its part, or -1
};

// Rows of the tiles go fastest within groups of p.group row tiles, so that the
// units that run side by side share few panels of A and of B.
__host__ __device__ __forceinline__ void gemm_tile(const GemmParams& p, int t, GemmUnit& c) {
  c.prob = 0;
  while (c.prob + 1 < p.problems && t >= p.prob[c.prob + 1].first) ++c.prob;
  const GemmProblem& q = p.prob[c.prob];
  t -= q.first;
  const int per_group = p.group * q.n_tiles;
  const int g = t / per_group, rem = t - g * per_group;
  const int left = q.m_tiles - g * p.group, rows = left < p.group ? left : p.group;
  c.nt = rem / rows;
  c.mt = g * p.group + rem - c.nt * rows;
}
__host__ __device__ __forceinline__ GemmUnit gemm_unit(const GemmParams& p, int u) {
  GemmUnit c;
  c.k0 = 0;
  c.k1 = p.kpan;
  c.part = -1;
  int t = u;
  if (u >= p.whole) {
    c.part = u - p.whole;
    const int i = c.part / p.splits, j = c.part - i * p.splits;
    t = p.whole + i;
    c.k0 = static_cast<int>(static_cast<long long>(p.kpan) * j / p.splits);
    c.k1 = static_cast<int>(static_cast<long long>(p.kpan) * (j + 1) / p.splits);
  }
  gemm_tile(p, t, c);
  return c;
}
// Element (row of the pair's tile, column) of a part: groups of four columns,
// then rows, so that the 32 rows of a warp are consecutive.
__host__ __device__ __forceinline__ long long gemm_part_at(int part, int row, int col4) {
  return ((static_cast<long long>(part) * 2 + (row >> 7)) * (kGemmTile / 4) + col4) * 512 + (row & 127) * 4;
}

// Float of a kept matrix of `blocks` blocks of 32 columns.
__host__ __device__ __forceinline__ long long gemm_kept_at(int row, int col, int blocks) {
  return (static_cast<long long>(row >> 5) * blocks + (col >> 5)) * 1024 + ((col & 31) >> 2) * 128 + (row & 31) * 4 + (col & 3);
}

namespace gemm {

// As ptx::BoundedWait with a 32-bit clock; the status word is written once at the end.
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
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint32_t t0 = now();
    while (!ptx::mbar_try_wait(bar, parity)) {
      if (*abort_flag) return false;
      if (now() - t0 >= budget_ns) *abort_flag = 1;
    }
    return true;
  }
  // By a whole warp: every lane gets the same answer.
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, wait1(bar, parity));
  }
};

// Loads of what an earlier kernel may have written while this one had already
// started: not through the non-coherent path.
__device__ __forceinline__ float load(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 load(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ float sigmoid(float u) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + e));  // (e infinite: 0)
  return s;
}
constexpr float kGelu = 1.5957691216057308f, kGelu3 = 0.044715f;  // 2 sqrt(2 / pi)

template <int V>
struct Constant {
  static constexpr int value = V;
};

// ACT 0: silu, 1: gelu
template <int ACT>
__device__ __forceinline__ float activation(float g) {
  return g * sigmoid(ACT ? kGelu * (g + kGelu3 * g * g * g) : g);
}
__device__ __forceinline__ float activation(int act, float g) { return act ? activation<1>(g) : activation<0>(g); }
// act(g) and its slope.  Far out s (1 - s) is 0, times a slope of u that has to stay finite.
template <int ACT>
__device__ __forceinline__ void activation_slope(float g, float& a, float& slope) {
  const float s = sigmoid(ACT ? kGelu * (g + kGelu3 * g * g * g) : g);
  a = g * s;
  const float t = fmaf(-a, s, a);  // a (1 - s)
  slope = ACT ? fmaf(t, kGelu * (1.0f + 3.0f * kGelu3 * fminf(g * g, 1e30f)), s) : s + t;
}
// f with the activation as a constant: a branch for a whole tile, not for each value.
template <class F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  if (act)
    f(Constant<1>{});
  else
    f(Constant<0>{});
}

template <int T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  return T == kGemmF16 ? ptx::pack_f16x2(__float_as_uint(lo), __float_as_uint(hi))
                       : ptx::pack_bf16x2(__float_as_uint(lo), __float_as_uint(hi));
}
template <int T>
__device__ __forceinline__ void unpack16(uint32_t w, float& lo, float& hi) {
  if constexpr (T == kGemmF16) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(w));
  } else {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
  }
}

// Scale of a block whose largest magnitude has the bits `top`, and its inverse:
// the smallest power of two that leaves nothing above 448 = 1.75 * 2^8, at least
// 2^-126.  A power of two, so that scaling rounds nothing.  A block that holds an
// infinity or a NaN gets NaN as its scale, and with it as each of its values.
__device__ __forceinline__ float block_scale(uint32_t top, float& inverse) {
  if (top >= 0x7f800000u) {
    inverse = __uint_as_float(0x7fffffffu);
    return inverse;
  }
  int e = static_cast<int>(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, 1);
  inverse = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  return __uint_as_float(static_cast<uint32_t>(e) << 23);
}
// Four values to e4m3, round to nearest even, the first in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

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

// One warp's boxes on their way out: 32 rows of 128 bytes, swizzled.
struct Stage {
  uint32_t addr;
  int lane;
  // The box before has been read.
  __device__ __forceinline__ void ready() const {
    if (lane == 0) ptx::bulk_wait_read<0>();
    __syncwarp();
  }
  __device__ __forceinline__ void store(const CUtensorMap* m, int col, int row, bool inside) const {
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && inside) {
      ptx::tma_store_2d(m, addr, col, row);
      ptx::bulk_commit();
    }
  }
  __device__ __forceinline__ void add(const CUtensorMap* m, int col, int row, bool inside) const {
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && inside) {
      ptx::tma_add_2d(m, addr, col, row);
      ptx::bulk_commit();
    }
  }
  // 32 packed 16-bit pairs: the row's 64 columns
  __device__ __forceinline__ void put(const uint32_t (&w)[32]) const {
    const uint32_t sw = static_cast<uint32_t>(lane & 7), row = addr + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
    for (uint32_t u = 0; u < 8; ++u)
      ptx::st_shared_v4(row + ((u ^ sw) << 4), w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
  }
};

}  // namespace gemm

template <int IN, bool AMN, bool BMN, int EPI, int OUT>
__global__ void __launch_bounds__(gemm_threads(IN == kGemmE4M3), 1)
    gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmParams p) {
  using namespace ptx;
  constexpr bool F8 = IN == kGemmE4M3;
  constexpr bool GATE = EPI == kEpiGate || EPI == kEpiGateQuant;
  constexpr int CK = F8 ? 128 : 64;  // K elements of a panel
  constexpr bool kWide = F8 || EPI == kEpiGateGrad;
  constexpr int kRing = gemm_ring(kWide), kWarps = gemm_warps(F8);
  static_assert(!F8 || (!AMN && !BMN && (EPI == kEpiStore || EPI == kEpiGateQuant)), "e4m3 operands are K-major");
  static_assert(F8 || (EPI != kEpiGateQuant && OUT == IN), "16-bit operands and outputs have one type");

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bar0 = base + kGemmOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + kGemmOffBar + 8 * kGSlotTmem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = rank == 0;
  const int cid = static_cast<int>(blockIdx.x >> 1), ncl = static_cast<int>(gridDim.x >> 1);

  if (warp == 0) {
    if (lane < 8) {
      mbar_init(bar(kGBFull + lane), 1);
      mbar_init(bar(kGBEmpty + lane), 1);
    } else if (lane < 10) {
      mbar_init(bar(kGBAccFull + lane - 8), F8 ? 3 : 1);  // (e4m3: and the scales, by two warps)
      mbar_init(bar(kGBAccEmpty + lane - 8), 2 * kWarps);  // epilogue warps of both CTAs
    } else if (lane == 10) {
      mbar_init(bar(kGBDrain), 1);
      *abort_flag = 0;
    } else if (lane < 15) {
      mbar_init(bar(kGBTop + lane - 11), 4);
    }
    fence_barrier_init();
  } else if (warp == 2) {
    tmem_alloc<2>(smem_u32(tmem_slot), 512);
    tmem_relinquish<2>();
  } else if (warp == 3 && lane == 0) {
    prefetch_tmap(&maps.a[0]);
    prefetch_tmap(&maps.b[0]);
    if (EPI != kEpiGateQuant) prefetch_tmap(&maps.out[0]);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_launch_dependents();
  grid_dependency_wait();

  const gemm::Wait bw{abort_flag, p.budget_ns};

  if (warp < 4) {
    if constexpr (F8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGemmOtherRegs));
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ loads
      uint32_t slot = 0, phase = 0;
      unsigned long long issued = 0;
      bool ok = true;
      const uint32_t a_bytes = AMN ? kPanelBytes : static_cast<uint32_t>(p.a_box_rows) * 128u;
      for (int u = cid; u < p.units && ok; u += ncl) {
        const GemmUnit c = gemm_unit(p, u);
        const GemmProblem& q = p.prob[c.prob];
        const int m0 = c.mt * kGemmTile + rank * 128;
        const int n0 = GATE ? c.nt * 128 : c.nt * kGemmTile + rank * 128;
        // halves past the last row or column are not loaded: what the MMAs make of
        // the panel's old contents is never looked at
        const bool a_odd = c.mt * kGemmTile + 128 < q.M, b_odd = GATE || c.nt * kGemmTile + 128 < q.N;
        const bool has_a = leader || a_odd, has_b = leader || b_odd;
        const uint32_t bytes = a_bytes * (a_odd ? 2u : 1u) + static_cast<uint32_t>(kPanelBytes) * (b_odd ? 2u : 1u);
        for (int k = c.k0; k < c.k1; ++k) {
          ok = bw.wait1(bar(kGBEmpty + slot), phase ^ 1u);
          if (!ok) break;
          const uint32_t full = mapa_shared(bar(kGBFull + slot), 0);
          // The even CTA arms its barrier for both CTAs' copies; the odd CTA's
          // may land first (the count then dips below zero, which is allowed).
          if (leader) mbar_arrive_expect_tx(bar(kGBFull + slot), bytes);
          const int seg = k >= p.kseg ? 1 : 0, kc = (k - (seg ? p.kseg : 0)) * CK;
          const CUtensorMap* ma = &maps.a[c.prob + seg];
          const CUtensorMap* mb = &maps.b[c.prob + seg + (GATE ? rank : 0)];
          const uint32_t sa = base + slot * static_cast<uint32_t>(kGemmSlot), sb = sa + kPanelBytes;
          if (!((p.debug & 1u) && issued == 0)) {  // (test support: the first panel is armed but never filled)
            if (has_a) {
              if constexpr (AMN) {
                tma_load_2d_pair(sa, ma, full, m0, kc);
                tma_load_2d_pair(sa + kPanelBytes / 2, ma, full, m0 + 64, kc);
              } else {
                tma_load_2d_pair(sa, ma, full, kc, m0);
              }
            }
            if (has_b) {
              if constexpr (BMN) {
                tma_load_2d_pair(sb, mb, full, n0, kc);
                tma_load_2d_pair(sb + kPanelBytes / 2, mb, full, n0 + 64, kc);
              } else {
                tma_load_2d_pair(sb, mb, full, kc, n0);
              }
            }
          }
          ++issued;
          if (++slot == kRing) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      tmem_slot[3] = slot | phase << 8;
      // Copies in flight land before exit (the even CTA's barriers count both CTAs').
      const unsigned long long tail = !leader ? 0 : (issued < kRing ? issued : kRing);
      for (unsigned long long j = 0; j < tail; ++j) {
        const unsigned long long idx = issued - 1 - j;
        drain_wait(bar(kGBFull + static_cast<int>(idx % kRing)), static_cast<uint32_t>((idx / kRing) & 1u),
                   p.budget_ns);
      }
    } else if (warp == 1 && leader) {
      // ------------------------------------------------------------- MMAs
      if (elect_one()) {
        constexpr uint32_t kFmt = IN == kGemmBF16 ? 1u : 0u;  // (0: f16, or e4m3 of the 8-bit kind)
        constexpr uint32_t idesc = make_idesc(kFmt, 256, 256, BMN) | (AMN ? 1u << 15 : 0u);
        // a K step (16 elements, 32 bytes) along a row, or 16 rows of 128 bytes
        constexpr uint32_t a_step = AMN ? 128 : 2, b_step = BMN ? 128 : 2;
        const uint64_t a0 = desc_sw128(base, AMN ? kPanelBytes / 2 : 16u, 1024u);
        const uint64_t b0 = desc_sw128(base + kPanelBytes, BMN ? kPanelBytes / 2 : 16u, 1024u);
        uint32_t slot = 0, phase = 0, acc = 0, acc_phase = 0;
        bool ok = true;
        for (int u = cid; u < p.units && ok; u += ncl) {
          const GemmUnit c = gemm_unit(p, u);
          for (int k = c.k0; k < c.k1; ++k) {
            // (e4m3: the accumulator is what there is to wait for)
            if (F8) ok = bw.wait1(bar(kGBFull + slot), phase);
            if (ok && (F8 || k == c.k0)) ok = bw.wait1(bar(kGBAccEmpty + acc), acc_phase ^ 1u);
            if (!F8 && ok) ok = bw.wait1(bar(kGBFull + slot), phase);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem_base + acc * 256u;
            const uint64_t a = a0 + slot * (kGemmSlot / 16), b = b0 + slot * (kGemmSlot / 16);
#pragma unroll
            for (uint32_t s = 0; s < 4; ++s) {
              const uint32_t more = s || (!F8 && k != c.k0) ? 1u : 0u;
              if constexpr (F8)
                mma_ss_f8_pair(d, a + s * a_step, b + s * b_step, idesc, more);
              else
                mma_ss<false, 2>(d, a + s * a_step, b + s * b_step, idesc, more);
            }
            if (F8 || k + 1 == c.k1) {
              tc_commit<2>(bar(kGBAccFull + acc));
              acc ^= 1u;
              if (acc == 0) acc_phase ^= 1u;
            }
            tc_commit<2>(bar(kGBEmpty + slot));
            if (++slot == kRing) {
              slot = 0;
              phase ^= 1u;
            }
          }
        }
        tc_commit<2>(bar(kGBDrain));
        drain_wait(bar(kGBDrain), 0, p.budget_ns);
      }
    } else if (F8 && warp >= 2) {
      // ----------------------------------------------------------- scales
      // Panel n's go into place n % 3 once panel n - 1's product is complete: its
      // MMAs began when panel n - 3 had been read.
      float* rows = reinterpret_cast<float*>(gbase + kGemmOffScales);
      float* cols = rows + 3 * 128;
      uint32_t place = 0, n = 0;
      bool ok = true;
      for (int u = cid; u < p.units && ok; u += ncl) {
        const GemmUnit c = gemm_unit(p, u);
        const GemmProblem& q = p.prob[c.prob];
        const int m0 = c.mt * kGemmTile + rank * 128 + (warp - 2) * 64 + lane;  // and m0 + 32
        const float* a0 = p.a_scale + (m0 < q.M ? m0 : 0) * p.a_scale_row + c.k0 * p.a_scale_k;
        const float* a1 = p.a_scale + (m0 + 32 < q.M ? m0 + 32 : 0) * p.a_scale_row + c.k0 * p.a_scale_k;
        // of the columns: warp 2 of the first 128 (or the gate's), warp 3 of the others
        const int w = warp - 2, nb = GATE ? c.nt : 2 * c.nt + w;
        const float* b0 = p.b_scale[GATE ? w : 0] + (nb * 128 < q.N ? nb : 0) * p.b_scale_row[GATE ? w : 0] + c.k0 * p.b_scale_k[GATE ? w : 0];
        // Asked for four panels ahead: one panel's time is less than a load's.
        float x0[4], x1[4], y[4];
        int next = c.k0;
        auto fetch = [&](int j) {
          if (next < c.k1) {
            x0[j] = gemm::load(a0);
            x1[j] = gemm::load(a1);
            y[j] = gemm::load(b0);
          }
          ++next;
          a0 += p.a_scale_k;
          a1 += p.a_scale_k;
          b0 += p.b_scale_k[GATE ? w : 0];
        };
#pragma unroll
        for (int j = 0; j < 4; ++j) fetch(j);
        for (int k = c.k0; k < c.k1 && ok; k += 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (k + j < c.k1 && ok) {
              if (n > 0) ok = bw.wait(bar(kGBAccFull + ((n - 1) & 1u)), ((n - 1) >> 1) & 1u);
              if (ok) {
                rows[place * 128 + w * 64 + lane] = x0[j];
                rows[place * 128 + w * 64 + 32 + lane] = x1[j];
                if (lane == 0) cols[place * 2 + w] = y[j];
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kGBAccFull + (n & 1u)));
                ++n;
                if (++place == 3) place = 0;
                fetch(j);
              }
            }
          }
        }
      }
    }
  } else {
    // ---------------------------------------------------------- epilogue
    if constexpr (F8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGemmEpilogueRegs));
    const int quad = warp & 3, half = (warp - 4) >> 2;  // (e4m3: of four quarters)
    const int row = quad * 32 + lane;  // of this CTA's 128
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const gemm::Stage stage{base + gemm_off_stage(kWide) + static_cast<uint32_t>(warp - 4) * (EPI == kEpiGateGrad ? 2 * kGemmStage : kGemmStage), lane};
    const uint32_t empty0 = mapa_shared(bar(kGBAccEmpty), 0);
    auto release = [&](uint32_t acc) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(empty0 + 8u * acc);
    };
    // first column, in the accumulator, of this warp's 32-column chunk i of four (e4m3: of two)
    auto column = [&](int i) -> int {
      if constexpr (F8) return GATE ? i * 128 + half * 32 : half * 64 + i * 32;
      return GATE ? (i >> 1) * 128 + half * 64 + (i & 1) * 32 : half * 128 + i * 32;
    };
    // kEpiGateGrad: G and U of 16 columns of this lane's row
    uint4 next_gate[4], next_up[4];
    auto fetch_kept = [&](int at_row, int col, int limit) {
      if (col < limit) {
        const long long at = gemm_kept_at(at_row + lane, col, p.kept_blocks);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          next_gate[e] = gemm::load(reinterpret_cast<const uint4*>(p.kept_gate + at + e * 128));
          next_up[e] = gemm::load(reinterpret_cast<const uint4*>(p.kept_up + at + e * 128));
        }
      }
    };
    uint32_t acc = 0, acc_phase = 0, tops = 0, place = 0;
    bool ok = true;
    for (int u = cid; u < p.units && ok; u += ncl) {
      const GemmUnit c = gemm_unit(p, u);
      const GemmProblem& q = p.prob[c.prob];
      const int m0 = c.mt * kGemmTile + rank * 128;
      const int mw = m0 + quad * 32;  // this warp's first row
      const bool rows = mw < q.M;     // it has some
      float* part = c.part < 0 ? nullptr : p.part + gemm_part_at(c.part, rank * 128 + row, 0);
      const bool mine = m0 + row < q.M;
      if constexpr (F8) {
        const float* scales = reinterpret_cast<const float*>(gbase + kGemmOffScales);
        uint64_t sum[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) sum[i] = 0;
        for (int k = c.k0; k < c.k1; ++k) {
          ok = bw.wait(bar(kGBAccFull + acc), acc_phase);
          if (!ok) break;
          tc_fence_after();
          if (rows) {
            uint64_t g2, u2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t v[16];
              tmem_ld16(lanes + acc * 256u + static_cast<uint32_t>(column(i >> 1) + (i & 1) * 16), v);
              if (i == 0) {
                const float fr = scales[place * 128 + row];
                const float2 fc = *reinterpret_cast<const float2*>(scales + 3 * 128 + place * 2);
                const float f0 = fr * (GATE || !(half & 2) ? fc.x : fc.y), f1 = GATE ? fr * fc.y : f0;
                g2 = gemm::pack2(f0, f0);
                u2 = GATE ? gemm::pack2(f1, f1) : g2;
              }
              tmem_wait_ld(v);
              if (i == 3) release(acc);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                sum[i * 8 + e] = gemm::fma2(gemm::pack2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), i < 2 ? g2 : u2, sum[i * 8 + e]);
            }
          } else {
            release(acc);
          }
          acc ^= 1u;
          if (acc == 0) acc_phase ^= 1u;
          if (++place == 3) place = 0;
        }
        if (!ok) break;
        if (part) {
          if (mine) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float4 v;
                gemm::unpack2(sum[i * 16 + 2 * e], v.x, v.y);
                gemm::unpack2(sum[i * 16 + 2 * e + 1], v.z, v.w);
                *reinterpret_cast<float4*>(part + (column(i) / 4 + e) * 512) = v;
              }
          }
        } else if constexpr (EPI == kEpiStore) {
          if (rows) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float x, y;
              gemm::unpack2(sum[e], x, y);
              w[e] = gemm::pack16<OUT>(x, y);
            }
            stage.ready();
            stage.put(w);
            const int col = c.nt * kGemmTile + half * 64;
            stage.store(&maps.out[0], col, mw, col < q.N);
          }
        } else {
          // h of 32 columns, the row's largest magnitude over the four warps' quarters, values and scale
          float h[32];
          uint32_t top = 0;
          gemm::with_activation(p.act, [&](auto act) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float g0, g1, u0, u1;
              gemm::unpack2(sum[e], g0, g1);
              gemm::unpack2(sum[16 + e], u0, u1);
              h[2 * e] = gemm::activation<act.value>(g0) * u0;
              h[2 * e + 1] = gemm::activation<act.value>(g1) * u1;
            }
          });
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            top = max(top, max(__float_as_uint(h[2 * e]) & 0x7fffffffu, __float_as_uint(h[2 * e + 1]) & 0x7fffffffu));
          }
          // (two sets in turn: a warp is at most one tile ahead of the others)
          volatile uint32_t* all = reinterpret_cast<volatile uint32_t*>(gbase + gemm_off_stage(true)) + (tops & 1u) * 512u + row;
          all[half * 128] = top;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kGBTop + quad));
          ok = bw.wait(bar(kGBTop + quad), tops & 1u);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) top = max(top, all[i * 128]);
          ++tops;
          float inv;
          const float scale = gemm::block_scale(top, inv);
          if (mine) {
            const int col = c.nt * 128 + half * 32;
            uint8_t* dst = p.q + (m0 + row) * p.q_ld + col;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint4 w;
              w.x = gemm::pack_e4m3(h[16 * e] * inv, h[16 * e + 1] * inv, h[16 * e + 2] * inv, h[16 * e + 3] * inv);
              w.y = gemm::pack_e4m3(h[16 * e + 4] * inv, h[16 * e + 5] * inv, h[16 * e + 6] * inv, h[16 * e + 7] * inv);
              w.z = gemm::pack_e4m3(h[16 * e + 8] * inv, h[16 * e + 9] * inv, h[16 * e + 10] * inv, h[16 * e + 11] * inv);
              w.w = gemm::pack_e4m3(h[16 * e + 12] * inv, h[16 * e + 13] * inv, h[16 * e + 14] * inv, h[16 * e + 15] * inv);
              if (col + 16 * e < q.N) *reinterpret_cast<uint4*>(dst + 16 * e) = w;
            }
            if (half == 0) p.q_scale[c.nt * p.q_scale_ld + m0 + row] = scale;
          }
        }
      } else {
        if (EPI == kEpiGateGrad && rows && !part) fetch_kept(mw, c.nt * kGemmTile + half * 128, q.N);
        ok = bw.wait(bar(kGBAccFull + acc), acc_phase);
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = lanes + acc * 256u;
        if (!rows) {
          release(acc);
        } else if (part) {
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            uint32_t v[32];
            tmem_ld32(src + static_cast<uint32_t>(column(i)), v);
            tmem_wait_ld(v);
            if (i == 3) release(acc);
            if (mine) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4*>(part + (column(i) / 4 + e) * 512) =
                    make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
          }
        } else if constexpr (EPI == kEpiStore) {
#pragma unroll 1
          for (int b = 0; b < 2; ++b) {
            uint32_t v0[32], v1[32];
            tmem_ld32(src + static_cast<uint32_t>(half * 128 + b * 64), v0);
            tmem_ld32(src + static_cast<uint32_t>(half * 128 + b * 64 + 32), v1);
            tmem_wait_ld(v0);
            tmem_wait_ld(v1);
            if (b == 1) release(acc);
            stage.ready();
            store_output_row<OUT == kGemmF16 ? kOutF16 : kOutBF16>(stage.addr, lane, 0, v0);
            store_output_row<OUT == kGemmF16 ? kOutF16 : kOutBF16>(stage.addr, lane, 32, v1);
            const int col = c.nt * kGemmTile + half * 128 + b * 64;
            stage.store(&maps.out[c.prob], col, mw, col < q.N);
          }
        } else if constexpr (EPI == kEpiAdd) {
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            uint32_t v[32];
            tmem_ld32(src + static_cast<uint32_t>(column(i)), v);
            tmem_wait_ld(v);
            if (i == 3) release(acc);
            stage.ready();
            store_output_row<kOutF32>(stage.addr, lane, 0, v);
            const int col = c.nt * kGemmTile + column(i);
            stage.add(&maps.out[c.prob], col, mw, col < q.N);
          }
        } else if constexpr (EPI == kEpiGate) {
          const int col = c.nt * 128 + half * 64;
          uint32_t w[32];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t g[32], v[32];
            tmem_ld32(src + static_cast<uint32_t>(column(i)), g);
            tmem_ld32(src + static_cast<uint32_t>(column(i + 2)), v);
            tmem_wait_ld(g);
            tmem_wait_ld(v);
            if (i == 1) release(acc);
            if (p.kept_gate && col + i * 32 < q.N) {
              const long long at = gemm_kept_at(mw + lane, col + i * 32, p.kept_blocks);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                *reinterpret_cast<uint4*>(p.kept_gate + at + e * 128) = make_uint4(g[4 * e], g[4 * e + 1], g[4 * e + 2], g[4 * e + 3]);
                *reinterpret_cast<uint4*>(p.kept_up + at + e * 128) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
              }
            }
            gemm::with_activation(p.act, [&](auto act) {
#pragma unroll
              for (int e = 0; e < 16; ++e)
                w[i * 16 + e] = gemm::pack16<OUT>(gemm::activation<act.value>(__uint_as_float(g[2 * e])) * __uint_as_float(v[2 * e]),
                                                  gemm::activation<act.value>(__uint_as_float(g[2 * e + 1])) * __uint_as_float(v[2 * e + 1]));
            });
          }
          stage.ready();
          stage.put(w);
          stage.store(&maps.out[0], col, mw, col < q.N);
        } else {
          // 16 columns at a time, G and U of the next ones on their way (of the first ones, since before
          // the wait); dG and dU to two boxes.
          const gemm::Stage second{stage.addr + kGemmStage, lane};
          const uint32_t sw = static_cast<uint32_t>(lane & 7), at = stage.addr + static_cast<uint32_t>(lane) * 128u;
          stage.ready();
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            uint32_t v[16];
            tmem_ld16(src + static_cast<uint32_t>(half * 128 + i * 16), v);
            uint4 g[4], u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              g[e] = next_gate[e];
              u[e] = next_up[e];
            }
            fetch_kept(mw, c.nt * kGemmTile + half * 128 + (i + 1) * 16, i < 7 ? q.N : 0);
            tmem_wait_ld(v);
            if (i == 7) release(acc);
            gemm::with_activation(p.act, [&](auto act) {
#pragma unroll
              for (uint32_t h = 0; h < 2; ++h) {
                uint32_t dg[4], du[4];
#pragma unroll
                for (uint32_t w = 0; w < 4; ++w) {
                  float a0, a1, s0, s1;
                  const uint4 &gw = g[2 * h + w / 2], &uw = u[2 * h + w / 2];
                  gemm::activation_slope<act.value>(__uint_as_float(w & 1 ? gw.z : gw.x), a0, s0);
                  gemm::activation_slope<act.value>(__uint_as_float(w & 1 ? gw.w : gw.y), a1, s1);
                  const float d0 = __uint_as_float(v[8 * h + 2 * w]), d1 = __uint_as_float(v[8 * h + 2 * w + 1]);
                  dg[w] = gemm::pack16<OUT>(d0 * __uint_as_float(w & 1 ? uw.z : uw.x) * s0, d1 * __uint_as_float(w & 1 ? uw.w : uw.y) * s1);
                  du[w] = gemm::pack16<OUT>(d0 * a0, d1 * a1);
                }
                const uint32_t unit = at + (((static_cast<uint32_t>(i & 3) * 2u + h) ^ sw) << 4);
                st_shared_v4(unit, dg[0], dg[1], dg[2], dg[3]);
                st_shared_v4(unit + kGemmStage, du[0], du[1], du[2], du[3]);
              }
            });
            if ((i & 3) == 3) {
              const int col = c.nt * kGemmTile + half * 128 + (i >> 2) * 64;
              stage.store(&maps.out[0], col, mw, col < q.N);
              second.store(&maps.out[1], col, mw, col < q.N);
              if (i == 3) stage.ready();
            }
          }
        }
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  __syncthreads();
  // Neither CTA leaves, or frees tensor memory, while the other may still
  // arrive on its barriers or the even CTA's MMAs may still write it: what the
  // MMAs' commits have to deliver has arrived in either.
  if (warp == 0) pair_exit(bar(kGBEmpty), kRing, bar(kGBDrain), bar(kGSlotTmem), p.budget_ns);
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc<2>(tmem_base, 512);
  }
  if (threadIdx.x == 0 && *abort_flag && p.status) atomicCAS(p.status, 0, kTimeoutCode);
}

// Adds the parts of the tiles that were cut along k, in order, and takes the
// epilogue's step.  blockIdx.x: 32 rows of such a tile; a warp takes 8 columns
// (of both projections for the gate), a row to a lane.
template <int EPI, int OUT>
__global__ void __launch_bounds__(512) gemm_combine_kernel(const __grid_constant__ GemmParams p) {
  constexpr bool GATE = EPI == kEpiGate || EPI == kEpiGateQuant;
  __shared__ uint32_t tops[16][32];
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x >> 3, row = (blockIdx.x & 7) * 32 + lane;
  GemmUnit c;
  gemm_tile(p, p.whole + t, c);
  const GemmProblem& q = p.prob[c.prob];
  const int m = c.mt * kGemmTile + row;
  if (c.mt * kGemmTile + (blockIdx.x & 7) * 32 >= q.M) return;
  const bool mine = m < q.M;
  // columns [8 col8, +8) of the tile, of both halves of it for the gate
  const int col8 = GATE ? warp : blockIdx.y * 16 + warp;
  float v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = 0.0f;
  if (mine) {
    for (int j = 0; j < p.splits; ++j) {
#pragma unroll
      for (int h = 0; h < (GATE ? 4 : 2); ++h) {
        const int col4 = 2 * col8 + (h & 1) + (h >> 1) * 32;
        const float4 x = *reinterpret_cast<const float4*>(p.part + gemm_part_at(t * p.splits + j, row, col4));
        v[4 * h] += x.x;
        v[4 * h + 1] += x.y;
        v[4 * h + 2] += x.z;
        v[4 * h + 3] += x.w;
      }
    }
  }
  const int col = c.nt * (GATE ? 128 : kGemmTile) + 8 * col8;
  const bool in = mine && col < q.N;
  auto store16 = [&](int o, const float* x) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out[o]) + m * p.out_ld[o] + col) =
        make_uint4(gemm::pack16<OUT>(x[0], x[1]), gemm::pack16<OUT>(x[2], x[3]), gemm::pack16<OUT>(x[4], x[5]),
                   gemm::pack16<OUT>(x[6], x[7]));
  };
  if constexpr (EPI == kEpiStore) {
    if (in) store16(c.prob, v);
  } else if constexpr (EPI == kEpiAdd) {
    if (in) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out[c.prob]) + m * p.out_ld[c.prob] + col);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float4 x = dst[h];
        x.x += v[4 * h];
        x.y += v[4 * h + 1];
        x.z += v[4 * h + 2];
        x.w += v[4 * h + 3];
        dst[h] = x;
      }
    }
  } else if constexpr (EPI == kEpiGateGrad) {
    if (in) {
      const long long at = gemm_kept_at(m, col, p.kept_blocks);
      float dg[8], du[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 gw = gemm::load(reinterpret_cast<const uint4*>(p.kept_gate + at + h * 128));
        const uint4 uw = gemm::load(reinterpret_cast<const uint4*>(p.kept_up + at + h * 128));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float g = __uint_as_float((&gw.x)[k]);
          float a, s;
          if (p.act)
            gemm::activation_slope<1>(g, a, s);
          else
            gemm::activation_slope<0>(g, a, s);
          dg[4 * h + k] = v[4 * h + k] * __uint_as_float((&uw.x)[k]) * s;
          du[4 * h + k] = v[4 * h + k] * a;
        }
      }
      store16(0, dg);
      store16(1, du);
    }
  } else {
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = gemm::activation(p.act, v[e]) * v[8 + e];
    if constexpr (EPI == kEpiGate) {
      if (in) {
        store16(0, h);
        if (p.kept_gate) {
          const long long at = gemm_kept_at(m, col, p.kept_blocks);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            *reinterpret_cast<float4*>(p.kept_gate + at + e * 128) = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            *reinterpret_cast<float4*>(p.kept_up + at + e * 128) = make_float4(v[8 + 4 * e], v[9 + 4 * e], v[10 + 4 * e], v[11 + 4 * e]);
          }
        }
      }
    } else {
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(h[e]) & 0x7fffffffu);
      tops[warp][lane] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 16; ++w) top = max(top, tops[w][lane]);
      float inv;
      const float scale = gemm::block_scale(top, inv);
      if (in)
        *reinterpret_cast<uint2*>(p.q + m * p.q_ld + col) =
            make_uint2(gemm::pack_e4m3(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv),
                       gemm::pack_e4m3(h[4] * inv, h[5] * inv, h[6] * inv, h[7] * inv));
      if (warp == 0 && mine) p.q_scale[c.nt * p.q_scale_ld + m] = scale;
    }
  }
}

}  // namespace b2b
