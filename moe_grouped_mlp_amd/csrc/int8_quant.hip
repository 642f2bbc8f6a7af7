// bf16 rows to 8-bit integers with one fp32 scale a row.
//
//   m = max(max|v|, 2^-100);  s = m / 127;  code = round(v * (127 / m))
//
// Bound by HBM: 2 bytes read and 1 written per value.  A row is held in the
// registers of a wave or of a workgroup between its maximum and its codes, so
// it is read once.  Magnitudes of bf16 values have the order of their bits, so
// the maximum is an integer one and shows infinities and NaN by itself.
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
constexpr int kThreads = 256;

struct Q {
  const uint16_t* x;
  int8_t* q;
  float* s;
  const int32_t* row_end;
  int64_t x_stride;
  int rows, cols;
};

MOE_DEV u16x2 max4(u16x2 m, u32x4 w) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
  return m;
}

// Two values -> their codes in the low byte of two words.  Adding 1.5 * 2^23
// rounds a product of at most 127.5 to an integer, ties to even.
MOE_DEV uint32_t code_of(float v, float r) {
#pragma clang fp contract(off)
  const float p = v * r;
  return __float_as_uint(p + 12582912.0f);
}
MOE_DEV uint32_t codes4(uint32_t a, uint32_t b, float r) {
  const uint32_t c0 = code_of(__uint_as_float(a << 16), r), c1 = code_of(__uint_as_float(a & 0xffff0000u), r);
  const uint32_t c2 = code_of(__uint_as_float(b << 16), r), c3 = code_of(__uint_as_float(b & 0xffff0000u), r);
  const uint32_t lo = __builtin_amdgcn_perm(c1, c0, 0x0c0c0400u), hi = __builtin_amdgcn_perm(c3, c2, 0x04000c0cu);
  return lo | hi;
}

// TPR threads a row, each with U groups of 8 values at a time.  LOOP: rows of
// more than these hold, read a second time for their codes.  STREAM: loads and
// stores past the caches, for rows that these do not hold (17408 x 14336 119 us, 6.3
// TB/s: 117 on one input again and again, 124 on three in turn; through the caches 136).
template <int TPR, int U, bool LOOP, bool STREAM>
__global__ __launch_bounds__(kThreads) void int8_quant_kernel(const Q a) {
  __shared__ uint32_t s_max[kThreads / kWave];
  const int tl = threadIdx.x & (TPR - 1);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  const int64_t end = a.row_end && *a.row_end < a.rows ? *a.row_end : a.rows;
  if (row >= end) return;   // all threads of the row (and with TPR = 256 of the workgroup)
  const uint16_t* x = a.x + row * a.x_stride;
  u32x4 v[U];
  u16x2 m = {0, 0};
  auto load = [&](int c0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + (u * TPR + tl) * 8;
      const u32x4* at = reinterpret_cast<const u32x4*>(x + (c < a.cols ? c : 0));   // (not behind a condition)
      v[u] = STREAM && !LOOP ? __builtin_nontemporal_load(at) : *at;
    }
  };
  for (int c0 = 0; c0 < a.cols; c0 += TPR * U * 8) {
    load(c0);
#pragma unroll
    for (int u = 0; u < U; ++u) m = max4(m, v[u]);   // (the row's first values twice)
    if (!LOOP) break;
  }
  uint32_t top = m[0] > m[1] ? m[0] : m[1];
#pragma unroll
  for (int o = (TPR < kWave ? TPR : kWave) / 2; o > 0; o >>= 1) {
    const uint32_t t = __shfl_xor(top, o, kWave);
    top = t > top ? t : top;
  }
  if constexpr (TPR == kThreads) {
    if ((threadIdx.x & (kWave - 1)) == 0) s_max[threadIdx.x / kWave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) top = s_max[w] > top ? s_max[w] : top;
  }
  const bool bad = top >= 0x7f80u;
  const float mm = fmaxf(__uint_as_float(top << 16), 0x1p-100f);
  const float r = bad ? 0.0f : 127.0f / mm;   // (both divisions correctly rounded)
  if (tl == 0) a.s[row] = bad ? __uint_as_float(0x7fc00000u) : mm / 127.0f;
  int8_t* q = a.q + row * a.cols;
  for (int c0 = 0; c0 < a.cols; c0 += TPR * U * 8) {
    if (LOOP) load(c0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + (u * TPR + tl) * 8;
      if (c < a.cols) {
        u32x2 w = {codes4(v[u][0], v[u][1], r), codes4(v[u][2], v[u][3], r)};
        if (bad) w = u32x2{0, 0};
        if constexpr (STREAM) __builtin_nontemporal_store(w, reinterpret_cast<u32x2*>(q + c));
        else *reinterpret_cast<u32x2*>(q + c) = w;
      }
    }
    if (!LOOP) break;
  }
}

}  // namespace

hipError_t launch_quantize_int8(const moe_quant_int8_args& a, hipStream_t s) {
  const Q q{static_cast<const uint16_t*>(a.x), a.q, a.s, a.row_end, a.x_stride ? a.x_stride : a.cols, a.rows, a.cols};
  const bool stream = 3 * static_cast<int64_t>(a.rows) * a.cols > kStreamBytes;
  auto go = [&](auto tpr, auto u, auto loop) {
    constexpr int TPR = decltype(tpr)::value, U = decltype(u)::value;
    constexpr bool LOOP = decltype(loop)::value;
    const int blocks = (a.rows + kThreads / TPR - 1) / (kThreads / TPR);
    if (stream) int8_quant_kernel<TPR, U, LOOP, true><<<blocks, kThreads, 0, s>>>(q);
    else int8_quant_kernel<TPR, U, LOOP, false><<<blocks, kThreads, 0, s>>>(q);
  };
  auto with_u = [&](auto tpr, int need) {
    using No = std::false_type;
    if (need <= 1) go(tpr, std::integral_constant<int, 1>{}, No{});
    else if (need <= 2) go(tpr, std::integral_constant<int, 2>{}, No{});
    else if (need <= 4) go(tpr, std::integral_constant<int, 4>{}, No{});
    else if (need <= 8) go(tpr, std::integral_constant<int, 8>{}, No{});
    else go(tpr, std::integral_constant<int, 8>{}, std::true_type{});
  };
  const int groups = (a.cols + 7) / 8;
  // many rows: 16 threads for up to 512 values (32768 x 256 4.7 us, with a wave 8.2; x
  // 512 8.6 and 9.8),
  // a wave for up to 4096
  if (a.rows >= 1024 && groups <= 16 * 4) with_u(std::integral_constant<int, 16>{}, (groups + 15) / 16);
  else if (a.rows >= 1024 && groups <= 64 * 8) with_u(std::integral_constant<int, 64>{}, (groups + 63) / 64);
  else with_u(std::integral_constant<int, kThreads>{}, (groups + kThreads - 1) / kThreads);
  return hipGetLastError();
}

}  // namespace moe
