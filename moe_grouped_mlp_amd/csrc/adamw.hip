// One AdamW step over a list of tensors, states in fp32 or in 8 bits.
//
//   d = g f;  m = b1 m + (1 - b1) d;  v = b2 v + (1 - b2) d^2
//   w = w - lr wd w - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps),  c = 1 - b^step
//
// As the clipping of grad.hip: the list goes to the kernel by value, cut into
// chunks that the workgroups take with a fixed stride.  A thread takes 8
// consecutive elements at a time, so 16 lanes hold a block of an 8-bit state
// and its new scale is a maximum over them.  The clipping factor is applied to
// the gradients as they are read.
#include <type_traits>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kPer = 8;   // consecutive elements of a thread
static_assert(MOE_FP8_BLOCK == 16 * kPer, "16 lanes hold a block");
static_assert(kAdamChunk % (kThreads * kPer) == 0, "whole passes");

// 8 elements at p + i, those at n and behind as zeros.
MOE_DEV void load8(const float* p, int64_t i, int64_t n, bool vec, float (&v)[kPer]) {
  if (vec && i + kPer <= n) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(p + i), b = *reinterpret_cast<const u32x4*>(p + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = __uint_as_float(a[j]);
      v[4 + j] = __uint_as_float(b[j]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) v[j] = i + j < n ? p[i + j] : 0.0f;
}
MOE_DEV void load8(const bf16_t* p, int64_t i, int64_t n, bool vec, float (&v)[kPer]) {
  if (vec && i + kPer <= n) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(p + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(a[j] << 16);
      v[2 * j + 1] = __uint_as_float(a[j] & 0xffff0000u);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) v[j] = i + j < n ? bf16_to_f32(p[i + j]) : 0.0f;
}
MOE_DEV void store8(float* p, int64_t i, int64_t n, bool vec, const float (&v)[kPer]) {
  if (vec && i + kPer <= n) {
    u32x4 a, b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = __float_as_uint(v[j]);
      b[j] = __float_as_uint(v[4 + j]);
    }
    *reinterpret_cast<u32x4*>(p + i) = a;
    *reinterpret_cast<u32x4*>(p + i + 4) = b;
    return;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (i + j < n) p[i + j] = v[j];
}
MOE_DEV void store8(bf16_t* p, int64_t i, int64_t n, bool vec, const float (&v)[kPer]) {
  if (vec && i + kPer <= n) {
    u32x4 a;
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<u32x4*>(p + i) = a;
    return;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (i + j < n) p[i + j] = static_cast<bf16_t>(pack_bf16x2(v[j], 0.0f));
}

// 8 codes and the values they stand for.
MOE_DEV u32x2 load_codes(const uint8_t* p, int64_t i, int64_t n, bool vec) {
  if (vec && i + kPer <= n) return *reinterpret_cast<const u32x2*>(p + i);
  u32x2 w = {0, 0};
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (i + j < n) w[j / 4] |= static_cast<uint32_t>(p[i + j]) << (8 * (j % 4));
  return w;
}
MOE_DEV void store_codes(uint8_t* p, int64_t i, int64_t n, bool vec, u32x2 w) {
  if (vec && i + kPer <= n) {
    *reinterpret_cast<u32x2*>(p + i) = w;
    return;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (i + j < n) p[i + j] = static_cast<uint8_t>(w[j / 4] >> (8 * (j % 4)));
}
MOE_DEV void decode8(u32x2 w, float scale, float (&v)[kPer]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[j]), false);
    const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[j]), true);
    v[4 * j] = a[0] * scale;
    v[4 * j + 1] = a[1] * scale;
    v[4 * j + 2] = b[0] * scale;
    v[4 * j + 3] = b[1] * scale;
  }
}
MOE_DEV u32x2 encode8(const float (&v)[kPer]) {
  u32x2 w;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    int c = 0;
    c = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j], v[4 * j + 1], c, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * j + 2], v[4 * j + 3], c, true);
    w[j] = static_cast<uint32_t>(c);
  }
  return w;
}

// Largest magnitude of a block: over a thread's values (a NaN does not count),
// then over the 16 lanes of a row by DPP.
MOE_DEV float block_max(const float (&v)[kPer]) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) m = fmaxf(m, fabsf(v[j]));
  auto step = [&](auto ctrl) {
    m = fmaxf(m, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(m), decltype(ctrl)::value, 0xF, 0xF, false)));
  };
  step(std::integral_constant<int, 0xB1>{});    // quad_perm: lane ^ 1
  step(std::integral_constant<int, 0x4E>{});    // quad_perm: lane ^ 2
  step(std::integral_constant<int, 0x141>{});   // row_half_mirror: the other quad of 8
  step(std::integral_constant<int, 0x140>{});   // row_mirror: the other 8
  return fmaxf(m, 0x1p-100f);
}

// 32 bits to 32 bits: two multiplications and three shifts (C. Wellons'
// lowbias32).
__host__ __device__ inline uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x7feb352du;
  x = (x ^ (x >> 15)) * 0x846ca68bu;
  return x ^ (x >> 16);
}

// y >= 0 (at most 448) to the E4M3 value below it, or with the probability of
// what that loses, r / 2^16, to the one above.  Below 2^-6, where E4M3's step
// stays 2^-9, it works on y + 2^-6, which has that step.
MOE_DEV float round_up_by(float y, uint32_t r) {
  const bool low = y < 0x1p-6f;
  const float z = low ? y + 0x1p-6f : y;
  const float c = __uint_as_float((__float_as_uint(z) + (r << 4)) & 0xfff00000u);
  return fminf(low ? c - 0x1p-6f : c, 448.0f);
}

struct Consts {
  float f, lr, lr_c1, rs_c2, b1, a1, b2, a2, eps;
};

// EXACT: each product and sum of the states rounded by itself and a correctly
// rounded root, so that codes, which one bit can move by a step, do not depend
// on who computes them.
template <bool EXACT>
MOE_DEV void update8(const Consts& c, float wd_lr, const float (&g)[kPer], float (&m)[kPer], float (&v)[kPer], float (&r)[kPer],
                     float (&w)[kPer]) {
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if constexpr (EXACT) {
#pragma clang fp contract(off)
      const float d = g[j] * c.f;
      m[j] = c.b1 * m[j] + c.a1 * d;
      v[j] = c.b2 * v[j] + c.a2 * d * d;
      r[j] = sqrtf(v[j]);
    } else {
      const float d = g[j] * c.f;
      m[j] = c.b1 * m[j] + c.a1 * d;
      v[j] = c.b2 * v[j] + c.a2 * d * d;
      r[j] = __builtin_amdgcn_sqrtf(v[j]);
    }
    // (v_sqrt and v_rcp are off by an ulp, of a term that is about lr of w)
    const float step = m[j] * __builtin_amdgcn_rcpf(__builtin_fmaf(r[j], c.rs_c2, c.eps));
    w[j] = __builtin_fmaf(-c.lr_c1, step, __builtin_fmaf(-wd_lr, w[j], w[j]));
  }
}

template <bool FP8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamList l) {
  Consts c{1.0f, l.lr, l.lr_c1, l.rs_c2, l.b1, l.a1, l.b2, l.a2, l.eps};
  if (l.lr_dev || l.step_dev) {
    if (l.lr_dev) c.lr = *l.lr_dev;
    double c1 = l.c1;
    int step = l.step;
    if (l.step_dev) {
      step = *l.step_dev;
      c1 = 1.0 - pow(l.b1_64, step);
      c.rs_c2 = static_cast<float>(1.0 / sqrt(1.0 - pow(l.b2_64, step)));
    }
    c.lr_c1 = static_cast<float>(static_cast<double>(c.lr) / c1);
  }
  if (l.sumsq) {
    const double norm = sqrt(*l.sumsq);
    if (!(norm <= 1.7976931348623157e308)) {   // infinite or NaN: no step
      if (blockIdx.x == 0 && threadIdx.x == 0) set_err(l.err, MOE_DEVERR_NONFINITE);
      return;
    }
    const double f = static_cast<double>(l.max_norm) / (norm + 1e-6);
    c.f = f < 1.0 ? static_cast<float>(f) : 1.0f;
  }
  const uint32_t step_u = l.step_dev ? static_cast<uint32_t>(*l.step_dev) : static_cast<uint32_t>(l.step);
  const uint32_t key0 = mix32(l.seed + step_u * 0x9e3779b9u);
  for (int64_t ch = blockIdx.x; ch < l.chunks; ch += gridDim.x) {
    int lo = 0, hi = l.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (l.t[mid].first <= ch) lo = mid; else hi = mid - 1;
    }
    const AdamEntry& t = l.t[lo];
    const int64_t n = t.numel, base = (ch - t.first) * kAdamChunk;
    const bool vec = t.flags & kAdamVec, p16 = t.flags & kAdamParam16, g16 = t.flags & kAdamGrad16;
    const float wd_lr = t.weight_decay * c.lr;
    const uint32_t key = mix32(key0 + t.index);
    // (the 16 lanes of a block stay together: those past the end hold zeros)
    for (int64_t i = base + threadIdx.x * kPer; i < base + kAdamChunk && i / MOE_FP8_BLOCK * MOE_FP8_BLOCK < n; i += kThreads * kPer) {
      float g[kPer], w[kPer], m[kPer], v[kPer], r[kPer];
      if (g16) load8(static_cast<const bf16_t*>(t.grad), i, n, vec, g);
      else load8(static_cast<const float*>(t.grad), i, n, vec, g);
      if (t.master) load8(t.master, i, n, vec, w);
      else if (p16) load8(static_cast<const bf16_t*>(t.param), i, n, vec, w);
      else load8(static_cast<const float*>(t.param), i, n, vec, w);
      const int64_t blk = i / MOE_FP8_BLOCK;
      if constexpr (FP8) {
        decode8(load_codes(static_cast<const uint8_t*>(t.m), i, n, vec), t.m_scale[blk], m);
        decode8(load_codes(static_cast<const uint8_t*>(t.v), i, n, vec), t.v_scale[blk], v);
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] *= v[j];
      } else {
        load8(static_cast<const float*>(t.m), i, n, vec, m);
        load8(static_cast<const float*>(t.v), i, n, vec, v);
      }
      update8<FP8>(c, wd_lr, g, m, v, r, w);
      if (t.master) store8(t.master, i, n, vec, w);
      if (p16) store8(static_cast<bf16_t*>(t.param), i, n, vec, w);
      else store8(static_cast<float*>(t.param), i, n, vec, w);
      if constexpr (FP8) {
        const float mm = block_max(m), mr = block_max(r);
        const float fm = 448.0f / mm, fr = 448.0f / mr;
        if ((threadIdx.x & 15) == 0) {
          t.m_scale[blk] = mm / 448.0f;
          t.v_scale[blk] = mr / 448.0f;
        }
        float y[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) y[j] = m[j] * fm;
        store_codes(static_cast<uint8_t*>(t.m), i, n, vec, encode8(y));
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const float z = r[j] * fr;
          y[j] = z;
          if (l.stochastic) {
            const uint32_t h = mix32(key + static_cast<uint32_t>((i + j) >> 1));
            if (z == z) y[j] = round_up_by(z, j & 1 ? h >> 16 : h & 0xffffu);   // (a NaN keeps its code)
          }
          // to nearest, 2^-10 and less would become zero
          if (z > 0.0f) y[j] = fmaxf(y[j], 0x1p-9f);
        }
        store_codes(static_cast<uint8_t*>(t.v), i, n, vec, encode8(y));
      } else {
        store8(static_cast<float*>(t.m), i, n, vec, m);
        store8(static_cast<float*>(t.v), i, n, vec, v);
      }
    }
  }
}

}  // namespace

hipError_t launch_adamw(const AdamList& l, bool fp8, hipStream_t s) {
  const int grid = static_cast<int>(l.chunks < kAdamBlocks ? l.chunks : kAdamBlocks);
  if (fp8) adamw_kernel<true><<<grid, kThreads, 0, s>>>(l);
  else adamw_kernel<false><<<grid, kThreads, 0, s>>>(l);
  return hipGetLastError();
}

}  // namespace moe
