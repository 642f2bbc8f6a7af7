#pragma once

// Grouped products on block-scaled FP8 operands (E4M3 codes, one fp32 scale
// per 128 values along K) for gfx950.
//
//   C[t][n] = sum_b sa[b][t] sb[.][b] * sum_{k in block b} a[t][k] w[n][k]
//
// The operands are widened to bf16, which holds every E4M3 value: four
// v_mfma_f32_16x16x32_bf16 cover a whole scale block of a 16 x 16 output tile
// and sum it from zero in fp32 (fp8_sums: one v_mfma_f32_16x16x128_f8f6f4 on the
// codes as they are), and the vector ALU adds it, scaled, to the fp32
// accumulators: 4 fused multiply-adds (16 cycles) behind 64 (32) cycles of MFMA,
// which the SIMD's other wave hides.  The weight operand sits on the MFMA's rows
// and the tokens on its columns, so a lane holds one token's outputs: the token's
// scale is one register per column tile and the 128 x 128 weight scale is uniform.
//
// Work decomposition
//   * Workgroup: 8 waves (two per SIMD), tile 128 tokens (fp8_sums: 256) x
//     256 weight rows, wave (wn, wt) = 128 weight rows x a quarter of the
//     tokens (8 x 2 or 8 x 4 MFMA tiles); fewer tokens where tiles are few
//     (JMAX).  A group's last tile runs with the fewest 64s of tokens that hold
//     its rows.
//   * Operands go from HBM straight into LDS (buffer loads with the LDS
//     destination), two stages of one scale block (128 bytes of every row)
//     each; their scales ride along.  16-byte chunk c of a row is stored at
//     c ^ swizzle(row), which spreads the 16 rows of an operand read over all
//     banks.
//   * MFMA row m of weight tile i is weight row 32 (i / 2) + 8 (m / 4) +
//     4 (i % 2) + m % 4 (bf16 output) or 16 i + m (fp32), so that a lane's
//     outputs of two tiles, or of one, are 16 consecutive bytes of its token;
//     they leave through LDS as whole rows.
//   * Persistent workgroups walk the tiles of all experts, whose sizes are
//     read from device memory.
//
// Precision: the FP8 MFMAs add eight neighbouring products aligned to the
// largest of them and keep 13 bits below it (seen with two products 2^-14
// apart, in all four FP8 forms; products of different eights add exactly in
// fp32).  On activations that is 2e-5 to 4e-5 of the result, and moves a bf16
// output by a step where it lies that near the border of two.  The bf16 MFMAs
// lose nothing of that kind (sums exact to 1e-8), at half the peak rate and 16
// conversions per 32 codes of a lane, so sums are theirs unless the caller asks
// for the FP8 ones.
//
// The weight gradient is the same product with the routed rows as K: both
// operands transposed copies with one scale per row and block, so its
// accumulation multiplies by two scales.
//
// Bound by the vector instructions beside the MFMAs: a SIMD issues two beside a
// 16-cycle MFMA for nothing, each further one costs 4 cycles (measured with two
// waves).  The product has 3.5 (2.5 to widen, 1 to scale) and its MFMAs are busy
// for half of the time: eight experts, 16384 rows x 4096 x 14336, 1690 us, 1.14
// PFLOP/s; 89 experts of 736 rows on average x 5760 x 2880, 2350 us, 920 TFLOP/s.
// The weight gradient has 4.7 (2 to scale), and its MFMAs are busy for a quarter
// to a third of the time: 32 experts of 7168 x 2048 from 16384 rows (4.5 steps a
// tile), fp32, 845 us, of which 690 without the stores, 300 the stores (1.88 GB)
// alone.
// With fp8_sums the first product takes 795 us (2.42 PFLOP/s; a product with one
// scale for all, from a library: 2.71) and the second 1210, bound by power: the
// clock falls to 1.5 .. 1.7 GHz while the MFMAs run, and a loop of nothing but
// these MFMAs and their scaled sums makes 3.47 PFLOP/s.  (All of a running
// program, over 1000 calls; the first ten after an idle while take a fifth longer.)
#include <type_traits>
#include <utility>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kFp8Threads = 512;
constexpr int kFp8Waves = kFp8Threads / kWave;
constexpr int kFp8BN = 256;            // weight rows of a tile
constexpr int kFp8Blk = MOE_FP8_BLOCK; // K values (bytes) of a stage

typedef __attribute__((address_space(3))) void fp8_lds_t;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int fp8_u32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp8OutOfRange = 0x7fffffff;   // buffer offset past any record

MOE_DEV __amdgpu_buffer_rsrc_t fp8_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0),
                                           static_cast<int>(bytes), 0x00020000);
}
MOE_DEV void fp8_dma16(__amdgpu_buffer_rsrc_t r, void* lds, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (fp8_lds_t*)lds, 16, voff, soff, 0, 0);
}
MOE_DEV void fp8_dma4(__amdgpu_buffer_rsrc_t r, void* lds, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (fp8_lds_t*)lds, 4, voff, soff, 0, 0);
}
constexpr int fp8_wait_vm(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0F70; }

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));

// One lane's operand of a 16 x 128 block: its 32 codes, or (WIDE) these
// widened to bf16, which holds every E4M3 value.
template <bool WIDE>
struct Fp8Frag;
template <>
struct Fp8Frag<false> {
  i32x8 v;
  MOE_DEV void set(i32x4 x, i32x4 y) { v = __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7); }
};
template <>
struct Fp8Frag<true> {
  bf16x8_t v[4];
  MOE_DEV static bf16x8_t widen(int a, int b) {
    const bf16x2_v r0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false);
    const bf16x2_v r1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true);
    const bf16x2_v r2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false);
    const bf16x2_v r3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true);
    return bf16x8_t{r0[0], r0[1], r1[0], r1[1], r2[0], r2[1], r3[0], r3[1]};
  }
  MOE_DEV void set(i32x4 x, i32x4 y) {
    v[0] = widen(x[0], x[1]);
    v[1] = widen(x[2], x[3]);
    v[2] = widen(y[0], y[1]);
    v[3] = widen(y[2], y[3]);
  }
};

// D = A . B over one scale block, summed from zero.
MOE_DEV f32x4 fp8_block_mfma(const Fp8Frag<false>& a, const Fp8Frag<false>& b) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, zero, 0, 0, 0, 0, 0, 0);
}
MOE_DEV f32x4 fp8_block_mfma(const Fp8Frag<true>& a, const Fp8Frag<true>& b) {
  f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], d, 0, 0, 0);
  return d;
}

// Compile-time loop, so that indices into register arrays are constants.
template <typename F, int... Is>
MOE_DEV void fp8_for_impl(F&& f, std::integer_sequence<int, Is...>) {
  (f(std::integral_constant<int, Is>{}), ...);
}
template <int N, typename F>
MOE_DEV void fp8_for(F&& f) {
  fp8_for_impl(f, std::make_integer_sequence<int, N>{});
}

// Chunk swizzles of the LDS images.  A lane's operand is chunks g and g + 4 of
// its row (g = lane / 16; which K values these are does not matter as long as
// both operands agree).  A 16-byte read serves lanes of two neighbouring g in
// one LDS cycle (lanes 0 .. 3 go with 20 .. 23); with chunk c of the m-th row
// of 16 at c ^ (m / 2) they fall on different banks (chunks 2 g and 2 g + 1
// instead cost 3.5 conflict cycles a read).  Tokens, and weights for an fp32
// output, are 16 consecutive rows; for a bf16 one they are rows 8 x + y, x < 4,
// y in a run of 4.
MOE_DEV int fp8_swz_t(int row) { return (row >> 1) & 7; }
template <bool F32>
MOE_DEV int fp8_swz_w(int row) {
  return F32 ? (row >> 1) & 7 : ((row >> 1) & 1) | ((row >> 2) & 6);
}

// A group's rows as the kernels see them: cut to what lies between its start,
// the next start and the buffer's end.
template <typename A>
MOE_DEV int fp8_group_rows(const A& g, int e, bool aligned, bool& bad) {
  const int64_t n = g.split[e], p0 = g.padded[e], p1 = g.padded[e + 1];
  const int64_t cap = g.M_cap, end = p1 < cap ? p1 : cap;
  const int64_t span = aligned ? (n + kFp8Blk - 1) / kFp8Blk * kFp8Blk : n;
  bad = n < 0 || p0 < 0 || p0 + span > end || (aligned && n > 0 && p0 % kFp8Blk != 0);
  if (!bad) return static_cast<int>(n);
  if (n < 0 || p0 < 0 || p0 >= end || (aligned && (p0 % kFp8Blk != 0))) return 0;
  if (aligned) return static_cast<int>((end - p0) / kFp8Blk * kFp8Blk);
  return static_cast<int>(end - p0);
}

// One operand tile of R rows x 128 bytes per stage: this wave's share of the
// R / 8 one-kilobyte loads (8 rows each).
template <int R, bool W, bool F32>
struct Fp8Loader {
  static constexpr int kInstr = R / 8 / kFp8Waves;   // 1, 2 or 4
  // First row of load j in its LDS array, the wave's loads side by side, and
  // in the tile.  Of the weights, loads 0 and 1 fill the array of tiles 0 .. 3
  // (tile rows 0 .. 63 and 128 .. 191), loads 2 and 3 that of tiles 4 .. 7.
  MOE_DEV static constexpr int lds_row(int wave, int j) {
    return W ? (2 * wave + j % 2) * 8 : (wave * kInstr + j) * 8;
  }
  MOE_DEV static constexpr int tile_row(int wave, int j) {
    const int r = lds_row(wave, j);
    return W ? r % 64 + r / 64 * 128 + j / 2 * 64 : r;
  }
  __amdgpu_buffer_rsrc_t rsrc;
  int voff[kInstr];
  // K bytes of the lane's chunk: the swizzle depends on load j through j % 2
  int kbyte[2];
  MOE_DEV static constexpr int which(int j) { return j % 2; }

  // base: the tile's first row at the group's first K value; ld: bytes
  // between rows; rows: rows that exist; k: K values that exist
  MOE_DEV void init(const uint8_t* base, int rows, int64_t ld, int k, int wave, int lane) {
    const int64_t bytes = rows > 0 ? (rows < R ? rows - 1 : R - 1) * ld + k : 0;
    rsrc = fp8_rsrc(base, static_cast<uint32_t>(bytes));
#pragma unroll
    for (int j = 0; j < kInstr; ++j) {
      const int row = tile_row(wave, j) + (lane >> 3);
      const int c = 16 * ((lane & 7) ^ (W ? fp8_swz_w<F32>(row) : fp8_swz_t(row)));
      kbyte[which(j)] = c;
      voff[j] = row < rows ? static_cast<int>(row * ld) + c : kFp8OutOfRange;
    }
  }
  // Loads j0 .. j1 - 1 of stage kt; chunks at or past K value k read as zeros.
  template <int j0 = 0, int j1 = kInstr>
  MOE_DEV void issue(uint8_t* stage, int kt, int wave_s, int k) {
    const int left = k - kt * kFp8Blk;
#pragma unroll
    for (int j = j0; j < j1; ++j)
      fp8_dma16(rsrc, stage + lds_row(wave_s, j) * kFp8Blk,
                kbyte[which(j)] < left ? voff[j] : kFp8OutOfRange, left > 0 ? kt * kFp8Blk : 0);
  }
};

// The tiles of all experts in their order, from the sizes on the device.
struct Fp8Tables {
  int start[kMaxExperts + 1];   // an expert's first tile
  int rows[kMaxExperts], at[kMaxExperts];   // its rows and the first of them
  int tmp[kFp8Waves];
};
template <int BT, bool WG>
MOE_DEV int fp8_tile_prefix(const Fp8Args& g, Fp8Tables& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tiles_n = (g.N + kFp8BN - 1) / kFp8BN;
  auto tiles_of = [&](int rows) { return (WG ? (g.P + BT - 1) / BT : (rows + BT - 1) / BT) * tiles_n; };
  const int per = (g.E + kFp8Threads - 1) / kFp8Threads;   // 1 or 2
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e < g.E) {
      bool bad;
      const int n = fp8_group_rows(g, e, WG, bad);
      if (bad && blockIdx.x == 0) set_err(g.err, MOE_DEVERR_BAD_OFFSETS);
      s.rows[e] = n;
      s.at[e] = g.padded[e];
      mine += tiles_of(n);
    }
  }
  int inc = mine;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int v = __shfl_up(inc, o, kWave);
    if (lane >= o) inc += v;
  }
  if (lane == 63) s.tmp[wave] = inc;
  __syncthreads();
  int run = inc - mine, total = 0;
  for (int w = 0; w < kFp8Waves; ++w) {
    if (w < wave) run += s.tmp[w];
    total += s.tmp[w];
  }
  for (int i = 0; i < per; ++i) {
    const int e = tid * per + i;
    if (e < g.E) {
      s.start[e] = run;
      run += tiles_of(s.rows[e]);
    }
  }
  if (tid == 0) s.start[g.E] = total;
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(total);
}

struct Fp8Tile {
  int e, n_e, start;   // the expert, its rows and the first of them
  int rows_t, t0, n0;  // token rows of the expert; the tile's first token and weight row
};
template <int BT, bool WG>
MOE_DEV Fp8Tile fp8_tile_at(const Fp8Args& g, const Fp8Tables& s, int id) {
  // the last expert that starts at id or before: 64 a comparison
  int lo = -1;
  for (int e0 = 0; e0 < g.E; e0 += kWave) {
    const int e = e0 + (threadIdx.x & (kWave - 1));
    lo += __popcll(__ballot(e < g.E && s.start[e < g.E ? e : 0] <= id));
  }
  Fp8Tile t;
  t.e = __builtin_amdgcn_readfirstlane(lo);
  const int in_e = __builtin_amdgcn_readfirstlane(id - s.start[lo]);
  t.n_e = __builtin_amdgcn_readfirstlane(s.rows[lo]);
  t.start = __builtin_amdgcn_readfirstlane(s.at[lo]);
  t.rows_t = WG ? g.P : t.n_e;
  // bands of group_m token tiles, all weight tiles of a band in turn
  const int tiles_n = (g.N + kFp8BN - 1) / kFp8BN;
  const int tiles_t = (t.rows_t + BT - 1) / BT;
  const int band = in_e / (g.group_m * tiles_n), in_b = in_e - band * g.group_m * tiles_n;
  const int gm = tiles_t - band * g.group_m < g.group_m ? tiles_t - band * g.group_m : g.group_m;
  t.t0 = (band * g.group_m + in_b % gm) * BT;
  t.n0 = in_b / gm * kFp8BN;
  return t;
}
// 64-token groups a tile with this many rows left runs with.
template <int JMAX>
MOE_DEV int fp8_tile_groups(int rows) {
  const int n = (rows + 63) / 64;
  return n < JMAX ? n : JMAX;
}
// Parts that K is cut into.  A step takes a tile 1.5 us; a part's sums, 256 KB,
// cost 0.09 us of the device's time to write and read again, and the second
// launch about 9 us.  So the best number is near sqrt(16 steps / tiles) (of
// four steps each at least, and as many workgroups as there are), and it has
// to save more steps than it costs.  2 groups of 100 rows, N=112 K=4736: 49 us
// uncut, 22 cut into 9 (fp8_sums, half the time a step: 24 and 19); 2 of 200, N=512
// K=8192: 80 and 30 (40 and 24); E=4 N=656 K=1168 (31 tiles, 10 steps): 23 us
// uncut, 41 cut into 2.
MOE_DEV int fp8_parts(const Fp8Args& g, int total, int workgroups) {
  if (!g.part || total < 1) return 1;
  const int steps = (g.K + kFp8Blk - 1) / kFp8Blk;
  const int room = workgroups / total;
  int n = steps / 4 < room ? steps / 4 : room;
  while (n > 1 && static_cast<int64_t>(n) * n * total > 16 * static_cast<int64_t>(steps)) --n;
  return n > 1 && steps - steps / n >= 6 + total * n / 16 ? n : 1;
}
// Place of a workgroup in the order of tiles: contiguous runs for each XCD
// (workgroup ids go round the XCDs).
MOE_DEV int fp8_workgroup(const Fp8Args& g) {
  const int G = g.grid;
  if (G % kNumXcd != 0) return blockIdx.x;
  return (blockIdx.x % kNumXcd) * (G / kNumXcd) + blockIdx.x / kNumXcd;
}
// Column of weight tile i's MFMA row 0 in its 64 columns.
template <bool F32>
MOE_DEV constexpr int fp8_w_off(int i) {
  return F32 ? 16 * (i % 4) : 32 * (i % 4 / 2) + 4 * (i % 2);
}

// JMAX: MFMA token tiles per wave; WG: the weight gradient; F32: fp32 output;
// WIDE: summed in fp32 from widened operands.
template <int JMAX, bool WG, bool F32, bool WIDE>
__global__ __launch_bounds__(kFp8Threads) __attribute__((amdgpu_waves_per_eu(2, 2))) void fp8_gemm_kernel(
    const Fp8Args g) {
  static_assert(WIDE || !F32, "an fp32 output is worth fp32 sums");
  constexpr int BT = 64 * JMAX;   // tokens of a tile
  __shared__ __attribute__((aligned(1024))) uint8_t sT0[BT * kFp8Blk], sT1[BT * kFp8Blk];
  // weights: the rows of tiles 0 .. 3 (a) and 4 .. 7 (b) of both wave columns;
  // behind the latter the stage's scales: tokens at 0, weights at 256 (WG:
  // one per row, else the tile's two 128-row blocks).  The compiler waits for
  // every load in flight into an array before it reads from it, and tells
  // six arrays apart but not eight: hence what shares one.
  constexpr int kHalfW = kFp8BN * kFp8Blk / 2;
  __shared__ __attribute__((aligned(1024))) uint8_t sWa0[kHalfW], sWa1[kHalfW];
  __shared__ __attribute__((aligned(1024))) uint8_t sWb0[kHalfW + 2048], sWb1[kHalfW + 2048];
  auto scales = [](auto* sWb) {
    using F = std::conditional_t<std::is_const_v<std::remove_pointer_t<decltype(sWb)>>, const float, float>;
    return reinterpret_cast<F*>(sWb + kHalfW);
  };
  __shared__ Fp8Tables s_tab;

  const int tid = threadIdx.x, wave = tid >> 6;
  const int wave_s = __builtin_amdgcn_readfirstlane(wave);
  const int wn = wave & 1, wt = wave >> 1;
  const int total = fp8_tile_prefix<BT, WG>(g, s_tab);
  const int parts = WG ? 1 : fp8_parts(g, total, g.grid);

  for (int item = fp8_workgroup(g); item < total * parts; item += g.grid) {
    const Fp8Tile tile = fp8_tile_at<BT, WG>(g, s_tab, item / parts);
    const int e = tile.e, n_e = tile.n_e, start = tile.start, rows_t = tile.rows_t, t0 = tile.t0, n0 = tile.n0;
    if (WG && g.accumulate && n_e == 0) continue;   // nothing to add: C stays as it is
    // the steps [k0, k1) of this part
    const int all_K = WG ? (n_e + kFp8Blk - 1) / kFp8Blk * kFp8Blk : g.K;
    const int all_steps = (all_K + kFp8Blk - 1) / kFp8Blk;
    const int part = item % parts;
    const int k0 = parts > 1 ? static_cast<int>(static_cast<int64_t>(all_steps) * part / parts) : 0;
    const int k1 = parts > 1 ? static_cast<int>(static_cast<int64_t>(all_steps) * (part + 1) / parts) : all_steps;

    // The tile with 64 JT tokens, JT the least that covers its rows: the last
    // rows of a group cost what they are, not a whole tile.
    auto run = [&](auto jt) {
      constexpr int J = decltype(jt)::value, BT = 64 * J;
      // opaque, so that the variants' addresses are made here and not held in
      // registers (and spilled, and read back behind the stores) over all tiles
      int lane = tid & 63;
      asm volatile("" : "+v"(lane));
      // operand reads: the lane's rows; their swizzles are unchanged by + 16 j
      // and + w_off(i)
      const int l16 = lane & 15, g4 = lane >> 4;
      const int t_row = 16 * J * wt + l16, w_row = 64 * wn + (F32 ? l16 : 8 * (l16 >> 2) + (l16 & 3));
      auto w_off = [](int i) { return fp8_w_off<F32>(i); };
      const int t_sw = fp8_swz_t(l16), w_sw = fp8_swz_w<F32>(w_row);
      const int steps = k1 - k0, K = (k1 < all_steps ? k1 * kFp8Blk : all_K) - k0 * kFp8Blk;
      const int rows_a = rows_t - t0, rows_b = g.N - n0;
      Fp8Loader<BT, false, F32> lt;
      Fp8Loader<kFp8BN, true, F32> lw;
      const uint8_t* b_e = static_cast<const uint8_t*>(g.b) + (WG ? start : e * g.b_stride) + k0 * kFp8Blk;
      lt.init(g.a + (WG ? static_cast<int64_t>(t0) * g.M_cap + start
                        : static_cast<int64_t>(start + t0) * g.K) + k0 * kFp8Blk,
              rows_a, WG ? g.M_cap : g.K, K, wave_s, lane);
      const int64_t ld_b = WG ? g.M_cap : g.K;
      lw.init(b_e + n0 * ld_b, rows_b, ld_b, K, wave_s, lane);
      // this wave's 64 scales of a stage: waves 0 .. 3 tokens, 4 .. 7 weights
      const bool s_tok = wave_s < 4;
      const int s_i = (wave_s & 3) * 64 + lane;
      const float* s_base;
      int64_t s_step;
      int s_voff = kFp8OutOfRange;
      if (s_tok) {
        s_base = WG ? g.a_s + static_cast<int64_t>(start / kFp8Blk) * g.P + t0 : g.a_s + start + t0;
        s_step = WG ? g.P : g.M_cap;
        if (s_i < BT && s_i < rows_a) s_voff = 4 * s_i;
      } else if constexpr (WG) {
        s_base = g.b_s + static_cast<int64_t>(start / kFp8Blk) * g.N + n0;
        s_step = g.N;
        if (s_i < rows_b) s_voff = 4 * s_i;
      } else {
        s_base = g.b_s + e * g.b_s_stride + static_cast<int64_t>(n0 / kFp8Blk) * all_steps;
        s_step = 1;
        if (s_i < 2 && s_i * kFp8Blk < rows_b) s_voff = 4 * s_i * all_steps;
      }
      s_base += k0 * s_step;
      // A stage's loads in the order they go out: the tokens and the weights of
      // tiles 0 .. 3 (early: their room is free half a step before the rest's),
      // the other weights, the scales.  Each is issued by itself between two
      // MFMAs: a wave that issues several in a row waits for the memory pipe,
      // 16 cycles a load and eight waves at it, with its MFMAs behind.
      constexpr int kTok = Fp8Loader<BT, false, F32>::kInstr, kEarly = kTok + 2;
      auto issue_early = [&](auto l, uint8_t* sT, uint8_t* sWa, int kt) {
        const int k_left = kt < steps ? K : 0;   // past the end: zeros
        if constexpr (l < kTok) lt.template issue<l, l + 1>(sT, kt, wave_s, k_left);
        else lw.template issue<l - kTok, l - kTok + 1>(sWa, kt, wave_s, k_left);
      };
      auto issue_late = [&](auto l, uint8_t* sWb, int kt) {
        lw.template issue<2 + l, 3 + l>(sWb, kt, wave_s, kt < steps ? K : 0);
      };
      auto issue_scales = [&](uint8_t* sWb, int kt) {
        fp8_dma4(fp8_rsrc(s_base + (kt < steps ? kt : 0) * s_step, 0x7ffffffeu), scales(sWb) + wave_s * 64,
                 kt < steps ? s_voff : kFp8OutOfRange, 0);
      };

      f32x4 acc[8][J];
  #pragma unroll
      for (int i = 0; i < 8; ++i)
  #pragma unroll
        for (int j = 0; j < J; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

      // Registers of the pipeline: the weight tile in use and the next one, the
      // step's tokens, and their scales for this step and the next.
      struct Raw {
        i32x4 x, y;
      };
      Raw wr[2], tr[J];
      float fr[2][J];
      f32x4 wf[2];
      auto read_w = [&](auto i, const uint8_t* sW, const float* sS) {   // sW: the half with tile i
        const uint8_t* r = sW + (w_row + w_off(i)) * kFp8Blk;
        wr[i & 1].x = *reinterpret_cast<const i32x4*>(r + 16 * (g4 ^ w_sw));
        wr[i & 1].y = *reinterpret_cast<const i32x4*>(r + 16 * ((g4 + 4) ^ w_sw));
        if constexpr (WG)
          wf[i & 1] = *reinterpret_cast<const f32x4*>(sS + 256 + 128 * wn + 64 * (i / 4) + w_off(i) +
                                                      (F32 ? 4 : 8) * g4);
      };
      auto read_t = [&](auto par, auto j, const uint8_t* sT, const float* sS) {
        const uint8_t* r = sT + (t_row + 16 * j) * kFp8Blk;
        tr[j].x = *reinterpret_cast<const i32x4*>(r + 16 * (g4 ^ t_sw));
        tr[j].y = *reinterpret_cast<const i32x4*>(r + 16 * ((g4 + 4) ^ t_sw));
        fr[par][j] = sS[t_row + 16 * j];
        if constexpr (!WG) fr[par][j] *= sS[256 + wn];
      };
      // One step on the stage in (sT, sWa, sWb), par: which registers hold its
      // token scales.  Weight tile i + 1 is read while tile i's MFMAs run, and an
      // MFMA's sums are added three MFMAs later, when they are there (held in that
      // order, else the compiler adds them at once, behind wait states).  Half way every wave is done with
      // the stage's tokens and the first half of its weights (a barrier), so the
      // loads of stage kt + 2 into that room go out; before the last weight tile
      // all of the stage is read and the next one has landed (the other
      // barrier), so the other weights go out (the scales follow in the next
      // step), and the next step's tokens are read into the registers that the
      // last MFMAs leave.
      auto step = [&](auto par, uint8_t* sT, uint8_t* sWa, uint8_t* sWb,
                      const uint8_t* nT, const uint8_t* nWa, uint8_t* nWb, int kt) {
        const float* sS = scales(sWb);
        const float* nS = scales(nWb);
        constexpr int P = decltype(par)::value;
        Fp8Frag<WIDE> t[J];
  #pragma unroll
        for (int j = 0; j < J; ++j) t[j].set(tr[j].x, tr[j].y);
        constexpr int kLag = 3, kRing = 4;
        f32x4 p[kRing];
        constexpr int kW = J >= kLag ? 2 : 4;   // weight tiles whose sums are outstanding
        f32x4 wfm[kW];
        auto add = [&](auto m) {   // the sums of MFMA m
          constexpr int i = m / J, j = m % J;
  #pragma unroll
          for (int r4 = 0; r4 < 4; ++r4) {
            const float s = WG ? fr[P][j] * wfm[i % kW][r4] : fr[P][j];
            acc[i][j][r4] = __builtin_fmaf(p[m % kRing][r4], s, acc[i][j][r4]);
          }
        };
        fp8_for<8>([&](auto i) {
          if constexpr (i == 4) {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
          }
          if constexpr (i < 7) {
            read_w(std::integral_constant<int, i + 1>{}, i < 3 ? sWa : sWb, sS);
          } else {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(fp8_wait_vm(kEarly) & 0xC07F);   // and lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            read_w(std::integral_constant<int, 0>{}, nWa, nS);
          }
          Fp8Frag<WIDE> w;
          w.set(wr[i & 1].x, wr[i & 1].y);
          if constexpr (WG) wfm[i % kW] = wf[i & 1];
          fp8_for<J>([&](auto j) {
            constexpr int m = i * J + j;
            p[m % kRing] = fp8_block_mfma(w, t[j]);
            if constexpr (m >= kLag) add(std::integral_constant<int, m - kLag>{});
            if constexpr (i == 7) read_t(std::integral_constant<int, 1 - P>{}, j, nT, nS);
            if constexpr (i == 0 && j == J - 1) issue_scales(nWb, kt + 1);
            if constexpr (i == 7)
              fp8_for<2>([&](auto l) {
                if constexpr (j == (J == 4 ? 1 + 2 * l : J - 1)) issue_late(l, sWb, kt + 2);
              });
            fp8_for<kEarly>([&](auto l) {   // two for each of tiles 4, 5 and 6
              if constexpr (i == 4 + l / 2 && j == (l % 2 ? J - 1 : J / 2 - (J == 4))) issue_early(l, sT, sWa, kt + 2);
            });
            __builtin_amdgcn_sched_barrier(0);
          });
        });
        fp8_for<kLag>([&](auto l) { add(std::integral_constant<int, 8 * J - kLag + l>{}); });
      };

      if (steps > 0) {
        fp8_for<kEarly>([&](auto l) { issue_early(l, sT0, sWa0, 0); });
        fp8_for<2>([&](auto l) { issue_late(l, sWb0, 0); });
        issue_scales(sWb0, 0);
        fp8_for<kEarly>([&](auto l) { issue_early(l, sT1, sWa1, 1); });
        fp8_for<2>([&](auto l) { issue_late(l, sWb1, 1); });
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(fp8_wait_vm(kEarly + 2));   // stage 0 landed
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        fp8_for<J>([&](auto j) { read_t(std::integral_constant<int, 0>{}, j, sT0, scales(sWb0)); });
        read_w(std::integral_constant<int, 0>{}, sWa0, scales(sWb0));
        // (a loop with its exit in the middle would make the compiler wait for
        // loads that only that way out leaves in flight)
        int kt = 0;
        for (; kt + 1 < steps; kt += 2) {
          step(std::integral_constant<int, 0>{}, sT0, sWa0, sWb0, sT1, sWa1, sWb1, kt);
          step(std::integral_constant<int, 1>{}, sT1, sWa1, sWb1, sT0, sWa0, sWb0, kt + 1);
        }
        if (kt < steps) step(std::integral_constant<int, 0>{}, sT0, sWa0, sWb0, sT1, sWa1, sWb1, kt);
        // the zero fills past the end, and reads of the stage behind the last
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0070);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }

      if constexpr (!WG) {
        if (parts > 1) {   // the accumulators as they are, for fp8_join_kernel
          f32x4* out = g.part + static_cast<int64_t>(item) * kFp8PartFloats / 4 + tid;
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) out[(i * J + j) * kFp8Threads] = acc[i][j];
          return;
        }
      }

      // ---- store ----
      // Straight from the accumulators a store would cover 64 bytes of 16 rows.
      // Instead each wave passes its outputs, 16 tokens (4 or 8 KB) at a time,
      // through LDS of its own (the stages are drained) and stores whole rows of
      // its 128 columns: 235 -> 179 us where an output of 755 MB is all there is
      // to do.  16-byte chunk c of row r lies at c ^ r, so that writes (16 rows,
      // one chunk) and reads (one row) fall on different banks.  Large outputs
      // (g.stream) pass the caches by, which then hold more of the operands: fp32
      // weight gradients of 1.88 GB 870 -> 856 us, 89 experts' outputs of 755 MB
      // (fp8_sums) 1217 -> 1200.  Rows that are no whole 128-byte lines or outputs that fit in
      // the last-level cache were slower so (59 MB in rows of 2592 bytes: 28.5 ->
      // 31.3 us).
      constexpr int kOut = F32 ? 4 : 2, kRow = 128 * kOut, kChunks = kRow / 16;
      // token groups that have room at once: all (a bf16 tile, up to 128 KB), or one
      constexpr int kAtOnce = F32 ? 1 : J, kOwn = kAtOnce * 16 * kRow;
      static_assert(kOwn <= (JMAX == 4 ? 16384 : 8192), "a wave's room");
      uint8_t* own = JMAX == 4 ? (wave < 2   ? sT0 + (wave & 1) * kOwn
                               : wave < 4 ? sT1 + (wave & 1) * kOwn
                               : wave < 6 ? (wave & 1 ? sWa1 : sWa0)
                                          : (wave & 1 ? sWb1 : sWb0))
                            : (wave < 4 ? (wave < 2 ? sWa0 : sWa1) : (wave < 6 ? sWb0 : sWb1)) + (wave & 1) * 8192;
      const int64_t c_row0 = WG ? static_cast<int64_t>(e) * g.P + t0 : static_cast<int64_t>(start) + t0;
      // opaque, so that no address here is held in registers over the K loop
      int ln = lane;
      asm volatile("" : "+v"(ln));
      const int r16 = ln & 15, q4 = ln >> 4;
      const int chunk = ln % kChunks, n = 128 * wn + chunk * (16 / kOut);
      char* c_tile = static_cast<char*>(g.c) + (c_row0 * g.ldc + n0 + n) * kOut;
  #pragma unroll
      for (int j0 = 0; j0 < J; j0 += kAtOnce) {
  #pragma unroll
        for (int jj = 0; jj < kAtOnce; ++jj) {
          const int j = j0 + jj;
  #pragma unroll
          for (int i = 0; i < 8; i += F32 ? 1 : 2) {
            const int cw = (64 * (i / 4) + w_off(i)) * kOut / 16 + q4;
            fp8_u32x4 w;
            if constexpr (F32) {
              w = __builtin_bit_cast(fp8_u32x4, acc[i][j]);
            } else {
              const f32x4 &x = acc[i][j], &y = acc[i + 1][j];
              w = fp8_u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(y[0], y[1]),
                            pack_bf16x2(y[2], y[3])};
            }
            *reinterpret_cast<fp8_u32x4*>(own + (16 * jj + r16) * kRow + 16 * (cw ^ r16)) = w;
          }
        }
        // LDS operations of one wave complete in order
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
        auto rows_out = [&](auto stream) {   // (a branch at each store would part them)
  #pragma unroll
          for (int q = 0; q < kAtOnce * 16 * kChunks / kWave; ++q) {
            const int r = ln / kChunks + q * (kWave / kChunks), tok = 16 * J * wt + 16 * j0 + r;
            fp8_u32x4 w = *reinterpret_cast<const fp8_u32x4*>(own + r * kRow + 16 * (chunk ^ (r & 15)));
            if (tok < rows_a && n < rows_b) {   // N % 16 == 0: the 16 bytes are inside or outside
              auto* c = reinterpret_cast<fp8_u32x4*>(c_tile + static_cast<int64_t>(tok) * g.ldc * kOut);
              if (F32 && WG && g.accumulate)
                w = __builtin_bit_cast(fp8_u32x4, __builtin_bit_cast(f32x4, *c) + __builtin_bit_cast(f32x4, w));
              if constexpr (decltype(stream)::value) __builtin_nontemporal_store(w, c);
              else *c = w;
            }
          }
        };
        if (g.stream) rows_out(std::true_type{});
        else rows_out(std::false_type{});
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
      }
      // every wave has read its rows: the next tile's loads may come
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    const int groups = fp8_tile_groups<JMAX>(rows_t - t0);
    if constexpr (JMAX == 4) {
      if (groups == 4) run(std::integral_constant<int, 4>{});
      else if (groups == 3) run(std::integral_constant<int, 3>{});
    }
    if constexpr (JMAX >= 2) {
      if (groups == 2) run(std::integral_constant<int, 2>{});
    }
    if (groups == 1) run(std::integral_constant<int, 1>{});
  }
}

// Second launch where fp8_gemm_kernel may have cut K: adds a tile's parts in
// their order and stores it.  Workgroup q of a tile takes every parts-th
// accumulator (bf16: pair of weight tiles, whose outputs are neighbours).
template <int JMAX, bool F32>
__global__ __launch_bounds__(kFp8Threads) void fp8_join_kernel(const Fp8Args g) {
  constexpr int BT = 64 * JMAX, kStep = F32 ? 1 : 2;
  __shared__ Fp8Tables s_tab;
  const int total = fp8_tile_prefix<BT, false>(g, s_tab);
  const int parts = fp8_parts(g, total, g.grid);
  const int item = blockIdx.x;
  if (parts == 1 || item >= total * parts) return;
  const Fp8Tile tile = fp8_tile_at<BT, false>(g, s_tab, item / parts);
  const int J = fp8_tile_groups<JMAX>(tile.rows_t - tile.t0);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave & 1, wt = wave >> 1, l16 = lane & 15, g4 = lane >> 4;
  const f32x4* in = g.part + static_cast<int64_t>(item / parts) * parts * (kFp8PartFloats / 4) + tid;
  for (int f = item % parts; f < 8 / kStep * J; f += parts) {
    const int i = f / J * kStep, j = f % J;
    const int tok = 16 * J * wt + 16 * j + l16;
    const int n = tile.n0 + 128 * wn + 64 * (i / 4) + fp8_w_off<F32>(i) + (F32 ? 4 : 8) * g4;
    f32x4 v[kStep];
#pragma unroll
    for (int u = 0; u < kStep; ++u) v[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = 0; p < parts; ++p) {
#pragma unroll
      for (int u = 0; u < kStep; ++u)
        v[u] += in[static_cast<int64_t>(p) * (kFp8PartFloats / 4) + ((i + u) * J + j) * kFp8Threads];
    }
    if (tile.t0 + tok >= tile.rows_t || n >= g.N) continue;
    const int64_t at = (static_cast<int64_t>(tile.start) + tile.t0 + tok) * g.ldc + n;
    if constexpr (F32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(g.c) + at) = v[0];
    } else {
      *reinterpret_cast<fp8_u32x4*>(static_cast<uint16_t*>(g.c) + at) =
          fp8_u32x4{pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]),
                    pack_bf16x2(v[1][0], v[1][1]), pack_bf16x2(v[1][2], v[1][3])};
    }
  }
}

}  // namespace
}  // namespace moe
