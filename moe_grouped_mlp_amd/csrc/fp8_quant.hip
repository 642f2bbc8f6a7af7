// bf16 -> block-scaled FP8 (E4M3 codes, one fp32 scale per 128 values of a
// row, or per 128 x 128 tile).
//
//   m = max(max|v|, 2^-100);  s = m / 448, r = 448 / m   (or s = 2^c, r = 1/s)
//   code = E4M3(v * r)
//
// Bound by HBM: 2 bytes read and 1 byte written per element and copy.  Row
// copies alone are made by quant_rows_kernel: 16 lanes hold a block, 8
// values each.  Everything else works on 128 x 128 tiles: a thread holds 8
// consecutive rows of 8 consecutive columns (8 loads of 16 bytes, all in
// flight), row maxima are taken over the 16 lanes of a row, column maxima
// over the 16 threads of a column (two lane exchanges, then the four waves
// through LDS), and the transposed codes leave through an LDS tile so that
// their stores are whole 128-byte lines.
//
// 17408 x 14336, both copies: 187 us, 5.4 TB/s of reads and writes; 128 weights
// of 2880 x 2880, both tile copies: 818 us, 5.2 TB/s, where a large copy reaches
// 4.8.  16 rows of 4096: 3 us, the launch.
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = MOE_FP8_BLOCK;
static_assert(kBlock == 128, "16 lanes of 8 values");

// Scale of a block with largest magnitude m, and the factor of its codes.
// Both divisions are correctly rounded (hipcc's default), so the codes do
// not depend on who computes them.
struct Scale {
  float s, r;
};
template <bool POW2>
MOE_DEV Scale block_scale(float m) {
  m = fmaxf(m, 0x1p-100f);
  const float s = m / 448.0f;
  if constexpr (POW2) {
    // up to the next power of two: m has 8 significant bits and 448 = 7 * 64,
    // so the rounded quotient is a power of two only if the exact one is.
    // An infinite m keeps an infinite scale (and the factor 0).
    const uint32_t u = __float_as_uint(s);
    if (u >= 0x7f800000u) return {s, 0.0f};
    const uint32_t e = (u + 0x007fffffu) & 0x7f800000u;
    return {__uint_as_float(e), __uint_as_float(0x7f000000u - e)};   // 2^c, 2^-c
  } else {
    return {s, 448.0f / m};
  }
}

// STREAM: nontemporal stores, and loads of what row copies are made of.  Both
// copies of 17408 x 14336 in 187 us (stores alone 191, neither 197), 128 weights'
// tile copies in 818 (loads too 827, neither 871), rows alone of 17408 x 14336 in
// 121 (neither 138).  For operands that the last-level cache does not hold, in
// rows of whole 64 bytes: 6224 x 8816, whose transposed rows are not, takes 102
// us so and 50 without.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <bool STREAM>
MOE_DEV uint4 load16(const void* p) {
  const u32x4* v = static_cast<const u32x4*>(p);
  if constexpr (STREAM) return __builtin_bit_cast(uint4, __builtin_nontemporal_load(v));
  else return __builtin_bit_cast(uint4, *v);
}
template <bool STREAM, typename T>
MOE_DEV void store(void* p, const T& v) {
  using V = std::conditional_t<sizeof(T) == 8, u32x2, u32x4>;
  if constexpr (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(V, v), static_cast<V*>(p));
  else *static_cast<T*>(p) = v;
}

MOE_DEV float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
MOE_DEV float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Four values -> four E4M3 codes (round to nearest even).
MOE_DEV uint32_t codes4(float a, float b, float c, float d) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return static_cast<uint32_t>(w);
}

MOE_DEV uint2 codes8(const uint4& v, float r) {
  return {codes4(lo_of(v.x) * r, hi_of(v.x) * r, lo_of(v.y) * r, hi_of(v.y) * r),
          codes4(lo_of(v.z) * r, hi_of(v.z) * r, lo_of(v.w) * r, hi_of(v.w) * r)};
}

// fmaxf: a NaN does not count.
MOE_DEV float amax8(const uint4& v) {
  const float a = fmaxf(fmaxf(fabsf(lo_of(v.x)), fabsf(hi_of(v.x))),
                        fmaxf(fabsf(lo_of(v.y)), fabsf(hi_of(v.y))));
  const float b = fmaxf(fmaxf(fabsf(lo_of(v.z)), fabsf(hi_of(v.z))),
                        fmaxf(fabsf(lo_of(v.w)), fabsf(hi_of(v.w))));
  return fmaxf(a, b);
}

// Maximum over the 16 lanes of a row of lanes, by DPP (no LDS round trip).
MOE_DEV float max16(float v) {
  auto step = [&](auto ctrl) {
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(
                     0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, false)));
  };
  step(std::integral_constant<int, 0xB1>{});    // quad_perm: lane ^ 1
  step(std::integral_constant<int, 0x4E>{});    // quad_perm: lane ^ 2
  step(std::integral_constant<int, 0x141>{});   // row_half_mirror: the other quad of 8
  step(std::integral_constant<int, 0x140>{});   // row_mirror: the other 8
  return v;
}

struct Q {
  const uint16_t* x;
  uint8_t* q;
  float* s;
  uint8_t* qT;
  float* sT;
  const int32_t* live;
  const int32_t* row_end;
  int rows, cols, n_rb, n_cb;   // 128-blocks along rows and columns
  int64_t x_stride;
};

MOE_DEV int rows_used(const Q& a) {
  if (!a.row_end) return a.rows;
  const int e = *a.row_end;
  return e < 0 ? 0 : e < a.rows ? e : a.rows;
}

// Row copies.  A workgroup takes 16 rows and kU column blocks (kU loads in
// flight for each thread): 256-byte runs in, 128-byte runs out, the 16
// scales of a column block side by side.
template <int kU, bool POW2, bool STREAM>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(const Q a, uint32_t units_c) {
  const int b = blockIdx.y;
  if (a.live && a.live[b] == 0) return;
  const uint32_t unit = blockIdx.x, ru = unit / units_c;
  const int cb0 = static_cast<int>(unit - ru * units_c) * kU;
  const int64_t row = static_cast<int64_t>(ru) * 16 + threadIdx.x / 16;
  const int c8 = (threadIdx.x & 15) * 8;
  if (row >= rows_used(a)) return;   // whole 16-lane rows leave
  const uint16_t* x = a.x + b * a.x_stride + row * a.cols;
  const int64_t n = static_cast<int64_t>(a.rows) * a.cols;
  uint8_t* q = a.q + b * n + row * a.cols;
  float* s = a.s + static_cast<int64_t>(b) * a.n_cb * a.rows + row;
  uint4 v[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int c = (cb0 + u) * kBlock + c8;
    v[u] = uint4{0, 0, 0, 0};
    if (c < a.cols) v[u] = load16<STREAM>(x + c);
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int cb = cb0 + u, c = cb * kBlock + c8;
    const Scale sc = block_scale<POW2>(max16(amax8(v[u])));
    if (c < a.cols) store<STREAM>(q + c, codes8(v[u], sc.r));
    if (c8 == 0 && cb < a.n_cb) s[static_cast<int64_t>(cb) * a.rows] = sc.s;
  }
}

// One 128 x 128 tile: row copies (ROW), transposed row copies (COL), or the
// tile's copy (TILE) and its transpose (TILE with COL).
template <bool ROW, bool COL, bool TILE, bool POW2, bool STREAM>
__global__ __launch_bounds__(kThreads) void quant_tile_kernel(const Q a) {
  // LDS image of the transposed tile: a column's 128 codes in 8-byte chunks,
  // chunk r of column c at r ^ 2 (c / 8 % 8).  With rows 144 bytes apart a
  // wave's 8-byte writes (16 columns 8 apart, 4 row groups) then fall on every
  // bank pair twice, the least there is; pairs of chunks stay together for
  // the 16-byte reads.
  constexpr int kLd = kBlock + 16;
  __shared__ __attribute__((aligned(16))) uint8_t s_t[COL ? kBlock * kLd : 16];
  __shared__ float s_m[4][kBlock];
  const int b = blockIdx.y;
  if (a.live && a.live[b] == 0) return;
  const int used = rows_used(a);
  const int cb = blockIdx.x % a.n_cb, rb = blockIdx.x / a.n_cb;
  const int64_t row0 = static_cast<int64_t>(rb) * kBlock;
  const int col0 = cb * kBlock;
  if (row0 >= used) return;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  const int c8 = (tid & 15) * 8, r8 = (tid >> 4) * 8;   // first column and row of the thread's 8 x 8
  const bool col_ok = col0 + c8 < a.cols;
  const int64_t n = static_cast<int64_t>(a.rows) * a.cols;
  const uint16_t* x = a.x + b * a.x_stride;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = uint4{0, 0, 0, 0};
    if (col_ok && row0 + r8 + i < used)
      v[i] = load16<STREAM && !TILE>(x + (row0 + r8 + i) * a.cols + col0 + c8);
  }
  float tile_r = 0.0f;
  if constexpr (TILE) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, amax8(v[i]));
    m = wave_max(m);
    if (lane == 0) s_m[0][wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(s_m[0][0], s_m[0][1]), fmaxf(s_m[0][2], s_m[0][3]));
    const Scale sc = block_scale<POW2>(m);
    tile_r = sc.r;
    if (tid == 0) {
      const int64_t nt = static_cast<int64_t>(b) * a.n_rb * a.n_cb;
      a.s[nt + static_cast<int64_t>(rb) * a.n_cb + cb] = sc.s;
      if constexpr (COL) a.sT[nt + static_cast<int64_t>(cb) * a.n_rb + rb] = sc.s;
    }
  }
  if constexpr (ROW || TILE) {
    uint8_t* q = a.q + b * n;
    float* s = a.s + (static_cast<int64_t>(b) * a.n_cb + cb) * a.rows;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = row0 + r8 + i;
      float r = tile_r;
      if constexpr (ROW) {
        const Scale sc = block_scale<POW2>(max16(amax8(v[i])));
        r = sc.r;
        if (c8 == 0 && row < used) s[row] = sc.s;
      }
      if (col_ok && row < used)
        store<STREAM>(q + row * a.cols + col0 + c8, codes8(v[i], r));
    }
  }
  if constexpr (COL) {
    // words of the thread's columns 2 j, 2 j + 1 of its row i
    auto word = [&](int i, int j) { return j == 0 ? v[i].x : j == 1 ? v[i].y : j == 2 ? v[i].z : v[i].w; };
    float cr[8];
    if constexpr (TILE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) cr[j] = tile_r;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m0 = fmaxf(m0, fabsf(lo_of(word(i, j))));
          m1 = fmaxf(m1, fabsf(hi_of(word(i, j))));
        }
        cr[2 * j] = m0;
        cr[2 * j + 1] = m1;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {   // the wave's four row groups: lanes ^ 16, ^ 32
        cr[j] = fmaxf(cr[j], __shfl_xor(cr[j], 16, kWave));
        cr[j] = fmaxf(cr[j], __shfl_xor(cr[j], 32, kWave));
      }
      if (lane < 16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s_m[wave][c8 + j] = cr[j];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Scale sc = block_scale<POW2>(fmaxf(fmaxf(s_m[0][c8 + j], s_m[1][c8 + j]),
                                                 fmaxf(s_m[2][c8 + j], s_m[3][c8 + j])));
        cr[j] = sc.r;
        if (r8 == 0 && col_ok)
          a.sT[(static_cast<int64_t>(b) * a.n_rb + rb) * a.cols + col0 + c8 + j] = sc.s;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint2 lo, hi;
      const float r0 = cr[2 * j], r1 = cr[2 * j + 1];
      lo.x = codes4(lo_of(word(0, j)) * r0, lo_of(word(1, j)) * r0, lo_of(word(2, j)) * r0,
                    lo_of(word(3, j)) * r0);
      lo.y = codes4(lo_of(word(4, j)) * r0, lo_of(word(5, j)) * r0, lo_of(word(6, j)) * r0,
                    lo_of(word(7, j)) * r0);
      hi.x = codes4(hi_of(word(0, j)) * r1, hi_of(word(1, j)) * r1, hi_of(word(2, j)) * r1,
                    hi_of(word(3, j)) * r1);
      hi.y = codes4(hi_of(word(4, j)) * r1, hi_of(word(5, j)) * r1, hi_of(word(6, j)) * r1,
                    hi_of(word(7, j)) * r1);
      const int at = 8 * ((tid >> 4) ^ (2 * (tid & 7)));
      *reinterpret_cast<uint2*>(s_t + (c8 + 2 * j) * kLd + at) = lo;
      *reinterpret_cast<uint2*>(s_t + (c8 + 2 * j + 1) * kLd + at) = hi;
    }
    __syncthreads();
    // the transposed matrix has a.rows columns; a 16-byte chunk of a line is
    // inside it or outside, since rows % 16 == 0
    uint8_t* qT = a.qT + b * n;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int col = p * 32 + tid / 8, r = (tid & 7) * 16;
      if (col0 + col < a.cols && row0 + r < a.rows)
        store<STREAM>(qT + static_cast<int64_t>(col0 + col) * a.rows + row0 + r,
                      *reinterpret_cast<const uint4*>(s_t + col * kLd + 8 * ((r / 8) ^ (2 * ((col >> 3) & 7)))));
    }
  }
}

template <bool POW2>
void launch(const moe_quant_fp8_args& m, const Q& a, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(m.batch) * a.rows * a.cols;
  const bool large = 2 * n > kStreamBytes && a.cols % 64 == 0;
  if (m.mode == MOE_QUANT_ROW) {
    const int64_t row_units = (static_cast<int64_t>(a.rows) + 15) / 16;
    const uint32_t uc = (a.n_cb + 7) / 8;
    auto rows = [&](auto kernel, uint32_t units_c) {
      kernel<<<dim3(static_cast<uint32_t>(row_units * units_c), m.batch), kThreads, 0, s>>>(a, units_c);
    };
    // eight blocks a thread in flight where that still leaves four
    // workgroups a CU, else one block each
    if (row_units * uc * m.batch < 1024) rows(quant_rows_kernel<1, POW2, false>, a.n_cb);
    else if (large) rows(quant_rows_kernel<8, POW2, true>, uc);
    else rows(quant_rows_kernel<8, POW2, false>, uc);
    return;
  }
  const dim3 grid(static_cast<uint32_t>(a.n_rb * a.n_cb), m.batch);
  auto tiles = [&](auto stream) {
    constexpr bool kS = decltype(stream)::value;
    if (m.mode == MOE_QUANT_BOTH)
      quant_tile_kernel<true, true, false, POW2, kS><<<grid, kThreads, 0, s>>>(a);
    else if (m.mode == MOE_QUANT_COL)
      quant_tile_kernel<false, true, false, POW2, kS><<<grid, kThreads, 0, s>>>(a);
    else if (a.qT)
      quant_tile_kernel<false, true, true, POW2, kS><<<grid, kThreads, 0, s>>>(a);
    else
      quant_tile_kernel<false, false, true, POW2, kS><<<grid, kThreads, 0, s>>>(a);
  };
  if (large && a.rows % 64 == 0) tiles(std::true_type{});
  else tiles(std::false_type{});
}

}  // namespace

hipError_t launch_quantize_fp8(const moe_quant_fp8_args& m, hipStream_t s) {
  Q a{};
  a.x = static_cast<const uint16_t*>(m.x);
  a.q = m.q;
  a.s = m.s;
  a.qT = m.qT;
  a.sT = m.sT;
  if (m.mode == MOE_QUANT_COL) {   // the kernel's transposed copy is the only one
    a.qT = m.q;
    a.sT = m.s;
  }
  a.live = m.live;
  a.row_end = m.row_end;
  a.rows = m.rows;
  a.cols = m.cols;
  a.n_rb = (m.rows + kBlock - 1) / kBlock;
  a.n_cb = (m.cols + kBlock - 1) / kBlock;
  a.x_stride = m.x_stride;
  if (m.pow2) launch<true>(m, a, s); else launch<false>(m, a, s);
  return hipGetLastError();
}

}  // namespace moe
