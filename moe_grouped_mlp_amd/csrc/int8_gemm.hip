// Grouped product of 8-bit integer rows with a scale for each token and each
// weight row, for gfx950.
//
//   C[t][n] = a_s[t] b_s[n] sum_k a[t][k] w[n][k]
//
// Bound by power: the MFMAs are busy for 67% of the cycles at 1.8 GHz.
// With v_mfma_i32_32x32x32_i8, which reads its operands half as often, the same
// took 6% fewer cycles at a clock 12% lower.
//
// The sums of v_mfma_i32_16x16x64_i8 are exact in 32 bits, so the accumulators
// run through all of K and the scales come in once, as the tile is stored: the
// K loop is loads and MFMAs alone.
//
// Tiles, stages and their order are the FP8 product's (fp8_gemm_kernel.h): 8
// waves, up to 256 tokens x 256 weight rows, 128 bytes of K a stage, two stages
// in LDS, fewer tokens where tiles are few, K cut where tiles leave CUs idle (the
// parts are integers: their order does not matter).
#include "int8_gemm.h"

namespace moe {
namespace {

// The last round of tiles, which leaves workgroups idle, is cut along K: its
// tiles from `whole` on have `parts` parts, one for a workgroup.  Each costs its
// sums' way out and back (256 KB, 0.09 us of the device's time), all of them the
// second launch, so the best number is near sqrt(16 steps / tiles) (of four
// steps each at least), and it has to save more steps than it costs.  16384 rows
// over 8 experts x 4096 x 14336, 1104 tiles on 256 CUs: 800 us uncut, 767 with the
// last 80 in 3 parts (754 .. 796 over runs, 2.42 .. 2.55 PFLOP/s; a library's product
// of 16384 x 4096 x 14336 and one scale for all: 2.52).
struct Int8Cut {
  int whole, parts;
};
MOE_DEV Int8Cut int8_cut(const Int8Args& g, int total) {
  const int tail = total % g.grid;
  if (!g.part || tail == 0) return {total, 1};
  const int steps = (g.K + kInt8Blk - 1) / kInt8Blk, room = g.grid / tail;
  int n = steps / 4 < room ? steps / 4 : room;
  while (n > 1 && static_cast<int64_t>(n) * n * tail > 16 * static_cast<int64_t>(steps)) --n;
  if (n > 1 && steps - steps / n >= 6 + tail * n / 16) return {total - tail, n};
  return {total, 1};
}

template <int JMAX, bool F32>
__global__ __launch_bounds__(kFp8Threads) __attribute__((amdgpu_waves_per_eu(2, 2))) void int8_gemm_kernel(const Int8Args g) {
  constexpr int BT = 64 * JMAX;   // tokens of a tile
  constexpr int kHalfW = kFp8BN * kInt8Blk / 2;
  __shared__ __attribute__((aligned(1024))) uint8_t sT0[BT * kInt8Blk], sT1[BT * kInt8Blk];
  // weights: the rows of tiles 0 .. 3 (a) and 4 .. 7 (b) of both wave columns
  __shared__ __attribute__((aligned(1024))) uint8_t sWa0[kHalfW], sWa1[kHalfW], sWb0[kHalfW], sWb1[kHalfW];
  __shared__ Fp8Tables s_tab;

  const int tid = threadIdx.x, wave = tid >> 6;
  const int wave_s = __builtin_amdgcn_readfirstlane(wave);
  const int wn = wave & 1, wt = wave >> 1;
  const int total = fp8_tile_prefix<BT, false>(g, s_tab);
  const Int8Cut cut = int8_cut(g, total);
  const int items = cut.whole + (total - cut.whole) * cut.parts;

  for (int item = fp8_workgroup(g); item < items; item += g.grid) {
    const int q = item - cut.whole, parts = q < 0 ? 1 : cut.parts;
    const Fp8Tile tile = fp8_tile_at<BT, false>(g, s_tab, q < 0 ? item : cut.whole + q / parts);
    const int e = tile.e, start = tile.start, rows_t = tile.rows_t, t0 = tile.t0, n0 = tile.n0;
    // the steps [k0, k1) of this part
    const int all_steps = (g.K + kInt8Blk - 1) / kInt8Blk;
    const int part = q < 0 ? 0 : q % parts;
    const int k0 = parts > 1 ? static_cast<int>(static_cast<int64_t>(all_steps) * part / parts) : 0;
    const int k1 = parts > 1 ? static_cast<int>(static_cast<int64_t>(all_steps) * (part + 1) / parts) : all_steps;

    // The tile with 64 J tokens, J the least that covers its rows.
    auto run = [&](auto jt) {
      constexpr int J = decltype(jt)::value, BT = 64 * J;
      // opaque, so that the variants' addresses are made here and not held in
      // registers over all tiles
      int lane = tid & 63;
      asm volatile("" : "+v"(lane));
      const int l16 = lane & 15, g4 = lane >> 4;
      const int t_row = 16 * J * wt + l16, w_row = 64 * wn + (F32 ? l16 : 8 * (l16 >> 2) + (l16 & 3));
      auto w_off = [](int i) { return fp8_w_off<F32>(i); };
      const int t_sw = fp8_swz_t(l16), w_sw = fp8_swz_w<F32>(w_row);
      const int steps = k1 - k0, K = (k1 < all_steps ? k1 * kInt8Blk : g.K) - k0 * kInt8Blk;
      const int rows_a = rows_t - t0, rows_b = g.N - n0;
      Fp8Loader<BT, false, F32> lt;
      Fp8Loader<kFp8BN, true, F32> lw;
      lt.init(g.a + static_cast<int64_t>(start + t0) * g.K + k0 * kInt8Blk, rows_a, g.K, K, wave_s, lane);
      lw.init(g.b + e * g.b_stride + static_cast<int64_t>(n0) * g.K + k0 * kInt8Blk, rows_b, g.K, K, wave_s, lane);
      // A stage's loads in the order they go out: the tokens and the weights of
      // tiles 0 .. 3 (early: their room is free half a step before the rest's),
      // then the other weights; each by itself between two MFMAs.
      constexpr int kTok = Fp8Loader<BT, false, F32>::kInstr, kEarly = kTok + 2;
      auto issue_early = [&](auto l, uint8_t* sT, uint8_t* sWa, int kt) {
        const int k_left = kt < steps ? K : 0;   // past the end: zeros
        if constexpr (l < kTok) lt.template issue<l, l + 1>(sT, kt, wave_s, k_left);
        else lw.template issue<l - kTok, l - kTok + 1>(sWa, kt, wave_s, k_left);
      };
      auto issue_late = [&](auto l, uint8_t* sWb, int kt) {
        lw.template issue<2 + l, 3 + l>(sWb, kt, wave_s, kt < steps ? K : 0);
      };

      i32x4 acc[8][J];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < J; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

      // Registers of the pipeline: the weight tile in use and the next one, and
      // the step's tokens.
      struct Raw {
        i32x4 v[2];
      };
      Raw wr[2], tr[J];
      auto read_w = [&](auto i, const uint8_t* sW) {   // sW: the half with tile i
        const uint8_t* r = sW + (w_row + w_off(i)) * kInt8Blk;
        wr[i & 1].v[0] = *reinterpret_cast<const i32x4*>(r + 16 * (g4 ^ w_sw));
        wr[i & 1].v[1] = *reinterpret_cast<const i32x4*>(r + 16 * ((g4 + 4) ^ w_sw));
      };
      auto read_t = [&](auto j, const uint8_t* sT) {
        const uint8_t* r = sT + (t_row + 16 * j) * kInt8Blk;
        tr[j].v[0] = *reinterpret_cast<const i32x4*>(r + 16 * (g4 ^ t_sw));
        tr[j].v[1] = *reinterpret_cast<const i32x4*>(r + 16 * ((g4 + 4) ^ t_sw));
      };
      // One step on the stage in (sT, sWa, sWb): weight tile i + 1 is read while
      // tile i's MFMAs run.  Half way every wave is done with the stage's tokens
      // and the first half of its weights (a barrier), so the loads of stage
      // kt + 2 into that room go out; before the last weight tile all of the stage
      // is read and the next one has landed (the other barrier), so the other
      // weights go out, and the next step's tokens are read into the registers
      // that the last MFMAs leave.
      auto step = [&](uint8_t* sT, uint8_t* sWa, uint8_t* sWb, const uint8_t* nT, const uint8_t* nWa, int kt) {
        fp8_for<8>([&](auto i) {
          if constexpr (i == 4) {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
          }
          if constexpr (i < 7) {
            read_w(std::integral_constant<int, i + 1>{}, i < 3 ? sWa : sWb);
          } else {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(fp8_wait_vm(kEarly) & 0xC07F);   // and lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            read_w(std::integral_constant<int, 0>{}, nWa);
          }
          const Raw w = wr[i & 1];
          fp8_for<2 * J>([&](auto m) {   // the first half of the piece for every token tile, then the second
            constexpr int h = m / J, j = m % J;
            acc[i][j] = int8_mfma(w.v[h], tr[j].v[h], acc[i][j]);
            if constexpr (i == 7 && h == 1) read_t(std::integral_constant<int, j>{}, nT);
            if constexpr (i == 7)
              fp8_for<2>([&](auto l) {
                if constexpr (m == (l + 1) * J - 1) issue_late(l, sWb, kt + 2);
              });
            fp8_for<kEarly>([&](auto l) {   // two for each of tiles 4, 5 and 6
              if constexpr (i == 4 + l / 2 && m == (l % 2 + 1) * J - 1) issue_early(l, sT, sWa, kt + 2);
            });
            __builtin_amdgcn_sched_barrier(0);
          });
        });
      };

      if (steps > 0) {
        fp8_for<kEarly>([&](auto l) { issue_early(l, sT0, sWa0, 0); });
        fp8_for<2>([&](auto l) { issue_late(l, sWb0, 0); });
        fp8_for<kEarly>([&](auto l) { issue_early(l, sT1, sWa1, 1); });
        fp8_for<2>([&](auto l) { issue_late(l, sWb1, 1); });
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(fp8_wait_vm(kEarly + 2));   // stage 0 landed
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        fp8_for<J>([&](auto j) { read_t(j, sT0); });
        read_w(std::integral_constant<int, 0>{}, sWa0);
        int kt = 0;
        for (; kt + 1 < steps; kt += 2) {
          step(sT0, sWa0, sWb0, sT1, sWa1, kt);
          step(sT1, sWa1, sWb1, sT0, sWa0, kt + 1);
        }
        if (kt < steps) step(sT0, sWa0, sWb0, sT1, sWa1, kt);
        // the zero fills past the end, and reads of the stage behind the last
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0070);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
      }

      if (parts > 1) {   // the accumulators as they are, for int8_join_kernel
        i32x4* out = reinterpret_cast<i32x4*>(g.part) + static_cast<int64_t>(q) * kFp8PartFloats / 4 + tid;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < J; ++j) out[(i * J + j) * kFp8Threads] = acc[i][j];
        return;
      }

      // ---- store: scaled, then as in the FP8 product: 16 tokens of the wave's
      // 128 columns at a time through LDS of its own, and out as whole rows ----
      constexpr int kOut = F32 ? 4 : 2, kRow = 128 * kOut, kChunks = kRow / 16;
      constexpr int kAtOnce = F32 ? 1 : J, kOwn = kAtOnce * 16 * kRow;
      static_assert(kOwn <= (JMAX == 4 ? 16384 : 8192), "a wave's room");
      uint8_t* own = JMAX == 4 ? (wave < 2   ? sT0 + (wave & 1) * kOwn
                               : wave < 4 ? sT1 + (wave & 1) * kOwn
                               : wave < 6 ? (wave & 1 ? sWa1 : sWa0)
                                          : (wave & 1 ? sWb1 : sWb0))
                            : (wave < 4 ? (wave < 2 ? sWa0 : sWa1) : (wave < 6 ? sWb0 : sWb1)) + (wave & 1) * 8192;
      int ln = lane;
      asm volatile("" : "+v"(ln));
      const int r16 = ln & 15, q4 = ln >> 4;
      const int chunk = ln % kChunks, n = 128 * wn + chunk * (16 / kOut);
      const int64_t c_row0 = static_cast<int64_t>(start) + t0;
      char* c_tile = static_cast<char*>(g.c) + (c_row0 * g.ldc + n0 + n) * kOut;
      // the lane's scales: of its J tokens, and of 4 weight rows of every tile
      // (rows past the end have any: they are not stored)
      const float* bs = g.b_s + e * g.b_s_stride + n0;
      f32x4 ws[8];
      float ts[J];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = 128 * wn + 64 * (i / 4) + w_off(i) + (F32 ? 4 : 8) * q4;
        const float* b = bs + (at < rows_b ? at : 0);   // (b_s need not be 16-byte aligned)
#pragma unroll
        for (int r = 0; r < 4; ++r) ws[i][r] = b[r];
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int tok = 16 * J * wt + 16 * j + r16;
        ts[j] = g.a_s[c_row0 + (tok < rows_a ? tok : 0)];
      }
#pragma unroll
      for (int j0 = 0; j0 < J; j0 += kAtOnce) {
#pragma unroll
        for (int jj = 0; jj < kAtOnce; ++jj) {
          const int j = j0 + jj;
#pragma unroll
          for (int i = 0; i < 8; i += F32 ? 1 : 2) {
            const int cw = (64 * (i / 4) + w_off(i)) * kOut / 16 + q4;
            auto scaled = [&](int ii) {
              f32x4 v;
#pragma unroll
              for (int r = 0; r < 4; ++r) v[r] = int8_scaled(acc[ii][j][r], ts[j], ws[ii][r]);
              return v;
            };
            fp8_u32x4 w;
            const f32x4 x = scaled(i);
            if constexpr (F32) {
              w = __builtin_bit_cast(fp8_u32x4, x);
            } else {
              const f32x4 y = scaled(i + 1);
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
            const fp8_u32x4 w = *reinterpret_cast<const fp8_u32x4*>(own + r * kRow + 16 * (chunk ^ (r & 15)));
            if (tok < rows_a && n < rows_b) {   // N % 16 == 0: the 16 bytes are inside or outside
              auto* c = reinterpret_cast<fp8_u32x4*>(c_tile + static_cast<int64_t>(tok) * g.ldc * kOut);
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

// Second launch where K may have been cut: adds a tile's parts, scales and
// stores them.  Workgroup q of a tile takes every parts-th accumulator (bf16:
// pair of weight tiles, whose outputs are neighbours).
template <int JMAX, bool F32>
__global__ __launch_bounds__(kFp8Threads) void int8_join_kernel(const Int8Args g) {
  constexpr int BT = 64 * JMAX, kStep = F32 ? 1 : 2;
  __shared__ Fp8Tables s_tab;
  const int total = fp8_tile_prefix<BT, false>(g, s_tab);
  const Int8Cut cut = int8_cut(g, total);
  const int parts = cut.parts, item = blockIdx.x;
  if (parts == 1 || item >= (total - cut.whole) * parts) return;
  const Fp8Tile tile = fp8_tile_at<BT, false>(g, s_tab, cut.whole + item / parts);
  const int J = fp8_tile_groups<JMAX>(tile.rows_t - tile.t0);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wn = wave & 1, wt = wave >> 1, l16 = lane & 15, g4 = lane >> 4;
  const i32x4* in = reinterpret_cast<const i32x4*>(g.part) + static_cast<int64_t>(item / parts) * parts * (kFp8PartFloats / 4) + tid;
  for (int f = item % parts; f < 8 / kStep * J; f += parts) {
    const int i = f / J * kStep, j = f % J;
    const int tok = 16 * J * wt + 16 * j + l16;
    const int n = tile.n0 + 128 * wn + 64 * (i / 4) + fp8_w_off<F32>(i) + (F32 ? 4 : 8) * g4;
    if (tile.t0 + tok >= tile.rows_t || n >= g.N) continue;
    i32x4 v[kStep];
#pragma unroll
    for (int u = 0; u < kStep; ++u) v[u] = i32x4{0, 0, 0, 0};
    for (int p = 0; p < parts; ++p) {
#pragma unroll
      for (int u = 0; u < kStep; ++u)
        v[u] += in[static_cast<int64_t>(p) * (kFp8PartFloats / 4) + ((i + u) * J + j) * kFp8Threads];
    }
    const int64_t row = static_cast<int64_t>(tile.start) + tile.t0 + tok;
    const float as = g.a_s[row];
    const float* bs = g.b_s + tile.e * g.b_s_stride + n;
    f32x4 o[kStep];
#pragma unroll
    for (int u = 0; u < kStep; ++u)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[u][r] = int8_scaled(v[u][r], as, bs[4 * u + r]);
    const int64_t at = row * g.ldc + n;
    if constexpr (F32) {
      *reinterpret_cast<f32x4*>(static_cast<float*>(g.c) + at) = o[0];
    } else {
      *reinterpret_cast<fp8_u32x4*>(static_cast<uint16_t*>(g.c) + at) =
          fp8_u32x4{pack_bf16x2(o[0][0], o[0][1]), pack_bf16x2(o[0][2], o[0][3]),
                    pack_bf16x2(o[1][0], o[1][1]), pack_bf16x2(o[1][2], o[1][3])};
    }
  }
}

template <int JMAX, bool F32>
hipError_t launch(const Int8Args& g, hipStream_t s) {
  int8_gemm_kernel<JMAX, F32><<<g.grid, kFp8Threads, 0, s>>>(g);
  if (hipError_t e = hipGetLastError()) return e;
  if (g.part) int8_join_kernel<JMAX, F32><<<g.grid, kFp8Threads, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int8_gemm(const Int8Args& g, bool f32, int groups, hipStream_t s) {
  if (f32) return groups == 1 ? launch<1, true>(g, s) : groups == 2 ? launch<2, true>(g, s) : launch<4, true>(g, s);
  return groups == 1 ? launch<1, false>(g, s) : groups == 2 ? launch<2, false>(g, s) : launch<4, false>(g, s);
}

}  // namespace moe
