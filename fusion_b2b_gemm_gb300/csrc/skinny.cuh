// The feed-forward operators' products for few rows: the weights' bytes are what
// they cost, so every weight is read by many CTAs at a time, and nothing is
// written but the result.
//
// The product is taken transposed: the weights' columns are the 128 rows of
// tcgen05.mma's A, the tokens the N columns of its B, so that a token more costs
// 1/128 of the tile and not a tile's row of 256.  (The same with mma.sync, the
// operands zipped in registers, was as quick up to 16 tokens, but its rate on
// this GPU bounds it from there on: a block of 4096/14336/4096, bf16, 59, 77 and
// 111 us for 16, 32 and 64 tokens, against 56, 58 and 61 us; the pair kernel,
// whose tile of 256 rows is mostly empty, takes 72 us for one token, this one 54.)
//
// More rows make several tiles of 16, 32, 64 or (16 bits) 128, side by side on one
// slice of the columns, so that its weights come from memory once.  That is quicker
// than the pair kernel as long as its tiles of 256 x 256 leave most SMs idle: an
// e4m3 product of 128 rows by 2000 k by 1368 columns takes 6.3 us, 12.5 there, of
// 128 rows by 14336 by 4096 23 and 25 us; a training step of 192 tokens on
// 1024/2816/1024 41 and 55 us.  It reads an operand's panel for 1/4 to 1/16 of the
// work, and loses where many tiles run one after the other: 500 tokens on
// 4096/14336/4096 149 us, 110 there.  few_shape() weighs them.
//
// A CTA takes a slice of the columns and, where slices alone are too few to keep
// the memory busy, a range of k; the CTAs of a slice are a cluster and add their
// sums up through each other's shared memory in a fixed order, so there is no
// second launch and no workspace.  Up to 32 tokens each CTA writes its sums into
// the CTA that adds them up, as soon as it has them; for more, that would cost a slot
// of the ring, and the sums lie in the ring's place and are read from there (a block of
// 1024/2816/1024 for one token: 7.9 us written, 8.8 read; of 2048/5632/2048 for 33: 20.3
// read, 20.8 written into the ring's place, 21.5 written beside a shorter ring).
//
// TMA brings panels of the weight(s) and of the rows into a ring; two CTAs share an
// SM, some 160 KB in flight.
//
//   16 bits: weights as stored, [k][column] (an MN-major A) or, in the backward
//            pass, [column][k] (K-major), 128 columns by 64 k a slot; the gate takes
//            64 columns of either weight as the two halves of one A.  The sums stay in
//            tensor memory to the end.
//   e4m3:    weights [column][k], 128 columns (whole blocks of scales) by 128 k, of
//            both weights for the gate.  Each slot's product is an accumulator of
//            its own, multiplied by its scales and added up in registers.
//
// Warp 0 loads, warp 1 multiplies (one elected thread), warps 2-5 (or 2-9) read
// tensor memory.  Every wait is bounded.
#pragma once

#include "gemm.cuh"

namespace b2b {

constexpr int kSkinnyMaxSplits = 8;  // CTAs of a cluster

struct SkinnyParams {
  int rows, N;
  int slots;          // panels of the whole of k
  int segment;        // panels of the first product (then x and the weight go on in the second maps)
  int splits, split_bits;  // CTAs of a slice, a power of two
  int row_tiles;           // of NT rows
  int x_box_rows;
  int act;
  void* out;          // h (or, e4m3 gate, its values), or the product
  long long out_ld;
  void* out2;         // kEpiGateGrad: dU (out: dG)
  float* kept_gate;   // as GemmParams
  float* kept_up;
  int kept_blocks;
  const float* a_scale;
  long long a_scale_row, a_scale_k;
  const float* b_scale[2];
  long long b_scale_row[2], b_scale_k[2];
  float* q_scale;
  long long q_scale_ld;
  uint32_t debug;
  int* status;
  uint32_t budget_ns;
};

struct SkinnyMaps {
  CUtensorMap x[2], w[2];
};

enum : int {  // barrier slots (8 bytes each)
  kSBFull = 0,       // [8] slot landed
  kSBEmpty = 8,      // [8] slot read
  kSBAccFull = 16,   // [2] accumulator complete (16 bits: [0], all of k)
  kSBAccEmpty = 18,  // [2] accumulator read
  kSBDrain = 20,
  kSSlotTmem = 21,   // uint32 tensor-memory base, then the int abort flag
};

// Weights, in us, for the choice between this kernel and the pair kernel, and of its tile
// (fitted to 1..1024 rows on widths of 512 to 65536, aligned and not: what they choose
// is on average 1-2 % slower than the quickest choice): a slot of this one, the same
// for each of its rows, what a second CTA on the SM adds, relatively, and the pair
// kernel's start beyond this one's and its K panel.  They put the choices in order; the
// sums are a launch's time only where its weights lie in L2 or its MMAs bound it.
struct SkinnyCost {
  float slot, slot_row, second, pair, pair_panel;
};

template <bool F8, bool GATE, int NT>
struct SkinnyShape {
  // km: K-major weights
  static constexpr SkinnyCost cost(bool km) {
    return F8   ? GATE ? SkinnyCost{0.055f, 0.009f, 0.065f, 1.6f, 0.28f} : SkinnyCost{0.23f, 0.0033f, 0.55f, 5.7f, 0.37f}
           : km ? SkinnyCost{0.17f, 0.0024f, 0.14f, 1.6f, 0.31f}
                : SkinnyCost{0.12f, 0.003f, 0.15f, 1.6f, 0.31f};
  }
  static constexpr int kColumns = F8 || !GATE ? 128 : 64;  // of a slice
  static constexpr int kDepth = F8 ? 128 : 64;             // k of a slot
  static constexpr int kWeight = F8 && GATE ? 32768 : 16384;
  static constexpr int kSlot = kWeight + NT * 128;
  static constexpr int kSumLd = GATE ? 2 * kColumns : kColumns;
  // Warps that read tensor memory, and what a thread adds up of a column: both weights'
  // rows, or half of them, or (kByWeight) one weight's.  Eight where four have too much to
  // hold or to add (64 rows on 4096/14336/4096 46.5 -> 43.8 us, where the gate spilled
  // registers; the product of 64 x 4096 x 14336 18.0 -> 17.1); four for the product of
  // 32 rows (64 x 14336 x 4096 17.2 us, with eight 17.5).
  static constexpr int kWarps = F8 && NT >= (GATE ? 32 : 64) ? 8 : 4;
  static constexpr bool kByWeight = GATE && kWarps == 8 && NT == 64;
  static constexpr int kThreads = 64 + 32 * kWarps;
  static constexpr int kTake = kByWeight ? NT : NT / (kWarps / 4);
  // Sums of the CTAs of a slice: apart from the ring, written there by the CTA that has
  // them while another may still multiply, or in the ring's place, its CTA's own.
  static constexpr bool kApart = NT <= 32 && !(F8 && GATE);  // (one accumulator's)
  static constexpr int kSumBytes = NT * kSumLd * 4;
  static constexpr int kRing = (105 * 1024 - (kApart ? kSumBytes : 0)) / kSlot;
  static constexpr int kOffSums = kApart ? kRing * kSlot : 0;
  static constexpr int kOffScales = kRing * kSlot + (kApart ? kSumBytes : 0);  // e4m3: [warp][weights][kTake]
  static constexpr int kOffBar = kOffScales + (F8 ? 4 * 2 * NT * 4 : 0);
  static constexpr int kBytes = kOffBar + 256 + 1024;
  // columns of tensor memory: an accumulator, or two (of both weights)
  static constexpr int kTmemCols = F8 ? 2 * NT * (GATE ? 2 : 1) : (NT < 32 ? 32 : NT);
  static_assert(kRing <= 8 && kRing >= 2 && kSumBytes <= kRing * kSlot, "the sums take the ring's place");
  static_assert(2 * (kBytes + 1024) <= 233472 && 2 * kTmemCols <= 512, "two CTAs on an SM");
};

namespace skinny {

// four consecutive floats of a CTA of the cluster
__device__ __forceinline__ void add_remote(float (&sum)[4], uint32_t addr) {
  float x, y, z, w;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x), "=f"(y), "=f"(z), "=f"(w) : "r"(addr));
  sum[0] += x;
  sum[1] += y;
  sum[2] += z;
  sum[3] += w;
}
__device__ __forceinline__ void store_remote(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// C columns of this warp's lanes, C = 16 or 32
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&v)[C]) {
  if constexpr (C == 16)
    ptx::tmem_ld16(addr, v);
  else
    ptx::tmem_ld32(addr, v);
}

}  // namespace skinny

// IN: operands; OUT: 16-bit type of the result (not of kEpiGateQuant's); EPI: of gemm.cuh's, what follows the product;
// KM: K-major weights; NT: rows of a tile, 16, 32, 64 or 128.
template <int IN, int OUT, int EPI, bool KM, int NT>
__global__ void __launch_bounds__(SkinnyShape<IN == kGemmE4M3, EPI == kEpiGate || EPI == kEpiGateQuant, NT>::kThreads, 2)
    skinny_kernel(const __grid_constant__ SkinnyMaps maps, const __grid_constant__ SkinnyParams p) {
  using namespace ptx;
  constexpr bool F8 = IN == kGemmE4M3, GATE = EPI == kEpiGate || EPI == kEpiGateQuant;
  static_assert(F8 ? KM && (EPI == kEpiStore || EPI == kEpiGateQuant) : !(KM && GATE), "weights' order");
  using L = SkinnyShape<F8, GATE, NT>;
  constexpr int W = F8 && GATE ? 2 : 1;      // accumulators of a slot
  constexpr int WT = L::kByWeight ? 1 : W;   // of them a thread takes
  constexpr int T = L::kTake, C = T < 32 || L::kWarps == 8 ? 16 : 32;  // columns read at a time
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bar0 = base + L::kOffBar;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::kOffBar + 8 * kSSlotTmem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = static_cast<int>(blockIdx.x) & (p.splits - 1), tile = static_cast<int>(blockIdx.x) >> p.split_bits;
  const int col0 = tile / p.row_tiles * L::kColumns, row0 = tile % p.row_tiles * NT;
  const int rows = min(NT, p.rows - row0);
  const int s0 = static_cast<int>(static_cast<long long>(p.slots) * part / p.splits);
  const int s1 = static_cast<int>(static_cast<long long>(p.slots) * (part + 1) / p.splits);
  // MN-major: two blocks of 64 columns a slot; K-major: 128 bytes of k of 128 columns
  auto weights = [&](int s, auto&& each) {
    if constexpr (F8 && GATE) {
      each(0, &maps.w[0], s * 128, col0);
      each(16384, &maps.w[1], s * 128, col0);
    } else if constexpr (KM) {
      const int seg = s >= p.segment ? 1 : 0;
      each(0, &maps.w[seg], (s - (seg ? p.segment : 0)) * L::kDepth, col0);
    } else {
      each(0, &maps.w[0], col0, s * 64);
      each(8192, &maps.w[GATE ? 1 : 0], GATE ? col0 : col0 + 64, s * 64);
    }
  };
  // (before anything is waited for: the others may then write to this CTA's sums)
  if (L::kApart && p.splits > 1) cluster_arrive();
  if (warp == 0) {
    if (elect_one()) {
      // The first slots into L2, before anything is waited for (a prefetch reads no value).
      for (int s = s0; s < s1 && s < s0 + L::kRing; ++s)
        weights(s, [&](int, const CUtensorMap* m, int x, int y) { tma_prefetch_l2_2d(m, x, y); });
    }
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), L::kTmemCols);
    tmem_relinquish();
  } else if (warp == 2) {
    if (lane < L::kRing) {
      mbar_init(bar(kSBFull + lane), 1);
      mbar_init(bar(kSBEmpty + lane), 1);
    } else if (lane < 10 && lane >= 8) {
      mbar_init(bar(kSBAccFull + lane - 8), 1);
      mbar_init(bar(kSBAccEmpty + lane - 8), L::kWarps);
    } else if (lane == 10) {
      mbar_init(bar(kSBDrain), 1);
      *abort_flag = 0;
    }
    fence_barrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // (after the allocation: a kernel that starts behind this one waits for it with
  // tensor memory in hand, and must not hold what a CTA of this one still asks for)
  grid_launch_dependents();
  grid_dependency_wait();
  const gemm::Wait bw{abort_flag, p.budget_ns};
  float acc_sum[WT][T];  // of an epilogue thread: its column's sums, of rows [first, first + T)
  const int half = L::kWarps > 4 ? (warp - 2) / 4 : 0, first = L::kByWeight ? 0 : half * T, w0 = L::kByWeight ? half : 0;
  float* sum = reinterpret_cast<float*>(gbase + L::kOffSums);

  if (warp == 0) {
    if (elect_one()) {
      uint32_t slot = 0, phase = 0;
      int issued = 0;
      const uint32_t bytes = L::kWeight + static_cast<uint32_t>(p.x_box_rows) * 128u;
      for (int s = s0; s < s1; ++s) {
        if (!bw.wait1(bar(kSBEmpty + slot), phase ^ 1u)) break;
        const uint32_t full = bar(kSBFull + slot), dst = base + slot * static_cast<uint32_t>(L::kSlot);
        mbar_arrive_expect_tx(full, bytes);
        if (!((p.debug & 1u) && issued == 0)) {  // (test support: the first slot is armed but never filled)
          weights(s, [&](int off, const CUtensorMap* m, int x, int y) { tma_load_2d(dst + off, m, full, x, y); });
          const int seg = s >= p.segment ? 1 : 0;
          tma_load_2d(dst + L::kWeight, &maps.x[seg], full, (s - (seg ? p.segment : 0)) * L::kDepth, row0);
        }
        ++issued;
        if (++slot == L::kRing) {
          slot = 0;
          phase ^= 1u;
        }
      }
      // copies in flight land before exit
      for (int j = 0; j < issued && j < L::kRing; ++j) {
        const int i = issued - 1 - j;
        drain_wait(bar(kSBFull + i % L::kRing), static_cast<uint32_t>(i / L::kRing) & 1u, p.budget_ns);
      }
    }
  } else if (warp == 1) {
    if (elect_one()) {
      constexpr uint32_t kFmt = IN == kGemmBF16 ? 1u : 0u;
      constexpr uint32_t idesc = make_idesc(kFmt, NT, 128, false) | (KM ? 0u : 1u << 15);
      constexpr uint32_t a_step = KM ? 2 : 128;
      uint32_t slot = 0, phase = 0, acc = 0, acc_phase = 0;
      for (int s = s0; s < s1; ++s) {
        if (F8 && !bw.wait1(bar(kSBAccEmpty + acc), acc_phase ^ 1u)) break;
        if (!bw.wait1(bar(kSBFull + slot), phase)) break;
        tc_fence_after();
        const uint32_t src = base + slot * static_cast<uint32_t>(L::kSlot);
        const uint64_t b = desc_sw128(src + L::kWeight, 16u, 1024u);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const uint64_t a = desc_sw128(src + w * 16384u, KM ? 16u : 8192u, 1024u);
          const uint32_t d = tmem_base + (F8 ? (acc * W + w) * NT : 0u);
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) {
            if constexpr (F8)
              mma_ss_f8(d, a + i * a_step, b + i * 2u, idesc, i ? 1u : 0u);
            else
              mma_ss<false>(d, a + i * a_step, b + i * 2u, idesc, i || s != s0 ? 1u : 0u);
          }
        }
        tc_commit(bar(kSBEmpty + slot));
        if (++slot == L::kRing) {
          slot = 0;
          phase ^= 1u;
        }
        if (F8 || s + 1 == s1) {
          tc_commit(bar(kSBAccFull + acc));
          acc ^= 1u;
          if (acc == 0) acc_phase ^= 1u;
        }
      }
      tc_commit(bar(kSBDrain));
      drain_wait(bar(kSBDrain), 0, p.budget_ns);
    }
  } else {
    const int quad = warp & 3;
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    const int column = quad * 32 + lane;  // of A's 128: of the slice, or of both weights' 64
    bool ok = true;
    if constexpr (!F8) {
      ok = bw.wait(bar(kSBAccFull), 0);
      tc_fence_after();
      if (ok) {
#pragma unroll
        for (int c = 0; c < T; c += C) {
          if (c < rows) {
            uint32_t v[C];
            skinny::tmem_ld<C>(lanes + static_cast<uint32_t>(c), v);
            tmem_wait_ld(v);
#pragma unroll
            for (int e = 0; e < C; ++e) {
              acc_sum[0][c + e] = __uint_as_float(v[e]);
              if (!L::kApart) sum[(c + e) * L::kSumLd + column] = acc_sum[0][c + e];
            }
          }
        }
      }
    } else {
#pragma unroll
      for (auto& a : acc_sum)
#pragma unroll
        for (float& x : a) x = 0.0f;
      // Scales of the tokens times that of the weights' block, a slot ahead of their use.
      constexpr int R = T < 32 ? 1 : T / 32;
      float next[WT][R];
      const int nb = col0 / 128;
      auto fetch = [&](int s) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int r = first + i * 32 + lane;
          const float a = r < rows ? gemm::load(p.a_scale + (row0 + r) * p.a_scale_row + s * p.a_scale_k) : 0.0f;
#pragma unroll
          for (int w = 0; w < WT; ++w) next[w][i] = a * gemm::load(p.b_scale[w0 + w] + nb * p.b_scale_row[w0 + w] + s * p.b_scale_k[w0 + w]);
        }
      };
      float* scales = reinterpret_cast<float*>(gbase + L::kOffScales) + (warp - 2) * WT * T;
      if (s0 < s1) fetch(s0);
      uint32_t acc = 0, acc_phase = 0;
      for (int s = s0; s < s1; ++s) {
        __syncwarp();
#pragma unroll
        for (int w = 0; w < WT; ++w)
#pragma unroll
          for (int i = 0; i < R; ++i)
            if (i * 32 + lane < T) scales[w * T + i * 32 + lane] = next[w][i];
        __syncwarp();
        if (s + 1 < s1) fetch(s + 1);
        ok = bw.wait(bar(kSBAccFull + acc), acc_phase);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int w = 0; w < WT; ++w)
#pragma unroll
          for (int c = 0; c < T; c += C) {
            uint32_t v[C];
            skinny::tmem_ld<C>(lanes + (acc * W + static_cast<uint32_t>(w0 + w)) * NT + static_cast<uint32_t>(first + c), v);
            tmem_wait_ld(v);
#pragma unroll
            for (int e = 0; e < C; e += 4) {
              const float4 f = *reinterpret_cast<const float4*>(scales + w * T + c + e);
              acc_sum[w][c + e] += __uint_as_float(v[e]) * f.x;
              acc_sum[w][c + e + 1] += __uint_as_float(v[e + 1]) * f.y;
              acc_sum[w][c + e + 2] += __uint_as_float(v[e + 2]) * f.z;
              acc_sum[w][c + e + 3] += __uint_as_float(v[e + 3]) * f.w;
            }
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSBAccEmpty + acc));
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
      // every copy into the ring has been waited for by the MMAs that these sums came from
      if (ok && !L::kApart) {
#pragma unroll
        for (int w = 0; w < WT; ++w)
#pragma unroll
          for (int e = 0; e < T; ++e) sum[(first + e) * L::kSumLd + (w0 + w) * 128 + column] = acc_sum[w][e];
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // (before the cluster's CTAs wait for each other: one of them may still wait for
  // tensor memory that a CTA of another kernel holds, and that for this one's)
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, L::kTmemCols);
  }
  // Sums of token r are added up by CTA r % splits.  Apart: there, [CTA they come
  // from][r / splits][column], once the others have begun; else, already, here, [r][column].
  const int share = (rows + p.splits - 1) >> p.split_bits;
  if constexpr (L::kApart) {
    if (p.splits > 1) cluster_wait();
    if (warp >= 2) {
      const uint32_t mine = base + L::kOffSums + static_cast<uint32_t>(part * share * L::kSumLd + (warp & 3) * 32 + lane) * 4u;
#pragma unroll
      for (int e = 0; e < T; ++e) {
        const int r = first + e;
        if (r < rows)
          skinny::store_remote(mapa_shared(mine + static_cast<uint32_t>((r >> p.split_bits) * L::kSumLd) * 4u,
                                           static_cast<uint32_t>(r & (p.splits - 1))),
                               acc_sum[0][e]);
      }
    }
  }
  if (p.splits > 1)
    cluster_sync();
  else if (L::kApart)
    __syncthreads();

  // A warp to a row (the 16-bit gate's 64 columns: to two), four columns to a lane.
  if (!*abort_flag) {
    constexpr int V = 4, kLanes = L::kColumns / V, kRows = 32 / kLanes;
    const int at_col = lane % kLanes * V, col = col0 + at_col;
    const uint32_t sums = base + L::kOffSums + static_cast<uint32_t>(at_col) * 4u;
    for (int r = part + ((warp * kRows + lane / kLanes) << p.split_bits); r < rows; r += (L::kThreads / 32 * kRows) << p.split_bits) {
      float v[GATE ? 2 : 1][V];
#pragma unroll
      for (auto& a : v)
#pragma unroll
        for (float& b : a) b = 0.0f;
      uint32_t from = sums + static_cast<uint32_t>((L::kApart ? r >> p.split_bits : r) * L::kSumLd) * 4u;
#pragma unroll 4
      for (int c = 0; c < p.splits; ++c) {
        const uint32_t at = L::kApart ? from : mapa_shared(from, static_cast<uint32_t>(c));
        skinny::add_remote(v[0], at);
        if constexpr (GATE) skinny::add_remote(v[GATE ? 1 : 0], at + L::kColumns * 4u);
        if (L::kApart) from += static_cast<uint32_t>(share * L::kSumLd) * 4u;
      }
      const bool in = col < p.N;  // (N is a multiple of V)
      if constexpr (EPI == kEpiGateGrad) {
        if (in) {
          const long long kept = gemm_kept_at(row0 + r, col, p.kept_blocks);
          const uint4 gw = gemm::load(reinterpret_cast<const uint4*>(p.kept_gate + kept)), uw = gemm::load(reinterpret_cast<const uint4*>(p.kept_up + kept));
          float dg[V], du[V];
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float g = __uint_as_float((&gw.x)[e]);
            float a, s;
            if (p.act)
              gemm::activation_slope<1>(g, a, s);
            else
              gemm::activation_slope<0>(g, a, s);
            dg[e] = v[0][e] * __uint_as_float((&uw.x)[e]) * s;
            du[e] = v[0][e] * a;
          }
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (row0 + r) * p.out_ld + col) =
              make_uint2(gemm::pack16<OUT>(dg[0], dg[1]), gemm::pack16<OUT>(dg[2], dg[3]));
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out2) + (row0 + r) * p.out_ld + col) =
              make_uint2(gemm::pack16<OUT>(du[0], du[1]), gemm::pack16<OUT>(du[2], du[3]));
        }
      } else if constexpr (!GATE) {
        if (in)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (row0 + r) * p.out_ld + col) =
              make_uint2(gemm::pack16<OUT>(v[0][0], v[0][1]), gemm::pack16<OUT>(v[0][2], v[0][3]));
      } else {
        float h[V];
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = gemm::activation(p.act, v[0][e]) * v[1][e];
        if constexpr (F8) {
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < V; ++e) top = max(top, __float_as_uint(h[e]) & 0x7fffffffu);
          top = __reduce_max_sync(0xffffffffu, top);
          float inv;
          const float scale = gemm::block_scale(top, inv);
          if (in)
            *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + (row0 + r) * p.out_ld + col) =
                gemm::pack_e4m3(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
          if (lane == 0) p.q_scale[col0 / 128 * p.q_scale_ld + row0 + r] = scale;
        } else if (in) {
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (row0 + r) * p.out_ld + col) =
              make_uint2(gemm::pack16<OUT>(h[0], h[1]), gemm::pack16<OUT>(h[2], h[3]));
          if (p.kept_gate) {
            const long long kept = gemm_kept_at(row0 + r, col, p.kept_blocks);
            *reinterpret_cast<float4*>(p.kept_gate + kept) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
            *reinterpret_cast<float4*>(p.kept_up + kept) = make_float4(v[1][0], v[1][1], v[1][2], v[1][3]);
          }
        }
      }
    }
  }
  if (threadIdx.x == 0 && *abort_flag && p.status) atomicCAS(p.status, 0, kTimeoutCode);
  if (!L::kApart && p.splits > 1) cluster_sync();  // (the sums have been read)
}

}  // namespace b2b
