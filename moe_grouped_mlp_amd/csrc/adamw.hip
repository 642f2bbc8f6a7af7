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
//
// Bound by HBM: an element of a bf16 weight with an fp32 master, gradient and
// states moves 30 bytes, one with 8-bit states and a bf16 gradient 10.1.  705 M
// elements take 3.73 ms (5.7 TB/s) and 1.23 ms (5.8; roots, codes and random bits
// keep the vector units busy for all of that time too); a copy of as much reaches
// 5.5 .. 5.8, one that reads 4 arrays and writes 3 5.5.  12 small tensors take 8 us,
// 6 of them the kernel's.
#include <type_traits>

#include "common.h"
#include "kernels.h"
#include "root.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kPer = 8;   // consecutive elements of a thread
static_assert(MOE_FP8_BLOCK == 16 * kPer, "16 lanes hold a block");
static_assert(kAdamChunk % (kThreads * kPer) == 0, "whole passes");

// 8 elements at p + i, those at n and behind as zeros.  (Each from where there is
// one: a load behind a condition would be waited for before the next.)
template <typename T>
MOE_DEV void load8(const T* p, int64_t i, int64_t n, float (&v)[kPer]) {
  T w[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) w[j] = p[i + j < n ? i + j : n - 1];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if constexpr (sizeof(T) == 2) v[j] = bf16_to_f32(w[j]);
    else v[j] = w[j];
    v[j] = i + j < n ? v[j] : 0.0f;
  }
}
template <typename T>
MOE_DEV void store8(T* p, int64_t i, int64_t n, const float (&v)[kPer]) {
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (i + j >= n) continue;
    if constexpr (sizeof(T) == 2) p[i + j] = static_cast<bf16_t>(pack_bf16x2(v[j], 0.0f));
    else p[i + j] = v[j];
  }
}

// 8 codes and the values they stand for.
MOE_DEV u32x2 load_codes(const uint8_t* p, int64_t i, int64_t n) {
  uint8_t c[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) c[j] = p[i + j < n ? i + j : n - 1];
  u32x2 w = {0, 0};
#pragma unroll
  for (int j = 0; j < kPer; ++j) w[j / 4] |= i + j < n ? static_cast<uint32_t>(c[j]) << (8 * (j % 4)) : 0;
  return w;
}
MOE_DEV void store_codes(uint8_t* p, int64_t i, int64_t n, u32x2 w) {
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

struct Consts {
  float f, lr, lr_c1, rs_c2, b1, a1, b2, a2, eps;
};

// The states' part of a step.  EXACT: each product and sum rounded by itself, so
// that codes, which one bit can move by a step, do not depend on who computes
// them.
template <bool EXACT>
MOE_DEV void moments(const Consts& c, float g, float& m, float& v) {
  if constexpr (EXACT) {
#pragma clang fp contract(off)
    const float d = g * c.f;
    m = c.b1 * m + c.a1 * d;
    v = c.b2 * v + c.a2 * d * d;
  } else {
    const float d = g * c.f;
    m = c.b1 * m + c.a1 * d;
    v = c.b2 * v + c.a2 * d * d;
  }
}
// (v_rcp is off by an ulp, as v_sqrt is, of a term that is about lr of w)
MOE_DEV float stepped(const Consts& c, float wd_lr, float m, float r, float w) {
  const float step = m * __builtin_amdgcn_rcpf(__builtin_fmaf(r, c.rs_c2, c.eps));
  return __builtin_fmaf(-c.lr_c1, step, __builtin_fmaf(-wd_lr, w, w));
}

// The hardware's root, off by an ulp.  It takes values below 2^-126 for zero: SMALL
// scales small ones before and after, for an eps that their roots are not lost beside.
// (Always, 705 M elements take 3.78 ms, else 3.73.)
template <bool SMALL>
MOE_DEV float root_ulp(float v) {
  if constexpr (!SMALL) return __builtin_amdgcn_sqrtf(v);
  const bool small = v < 0x1p-96f;
  return __builtin_amdgcn_sqrtf(small ? v * 0x1p64f : v) * (small ? 0x1p-32f : 1.0f);
}

// Correctly rounded roots: of values in [2^-96, inf) from the hardware's reciprocal
// root, which is off by an ulp at most.  Others (zeros, mostly) take the library's.
MOE_DEV void roots(const float (&v)[kPer], float (&r)[kPer]) {
  constexpr uint32_t kLo = 0x0f800000u, kSpan = 0x7f800000u - kLo;
  uint32_t out = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t t = __float_as_uint(v[j]) - kLo;
    out = t > out ? t : out;
    r[j] = root_from(v[j], __builtin_amdgcn_rsqf(v[j]));
  }
  if (out >= kSpan) {
    asm volatile("");   // (a branch)
#pragma unroll
    for (int j = 0; j < kPer; ++j) r[j] = sqrtf(v[j]);
  }
}

// A block's scale factors, by all of its 16 lanes.
struct Coding {
  float m, r;
};
MOE_DEV Coding coding_of(const AdamEntry& t, int64_t blk, const float (&m)[kPer], const float (&r)[kPer]) {
  const float mm = block_max(m), mr = block_max(r);
  if ((threadIdx.x & 15) == 0) {
    t.m_scale[blk] = mm / 448.0f;
    t.v_scale[blk] = mr / 448.0f;
  }
  return {448.0f / mm, 448.0f / mr};
}
MOE_DEV u32x2 encode_m(const Coding& k, const float (&m)[kPer]) {
  float y[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) y[j] = m[j] * k.m;
  return encode8(y);
}
// Roots: to nearest, or up with the probability of what rounding down would
// lose.  Times 2^-120 a value's upper bits are its code (E4M3's exponents,
// subnormal ones too, are fp32's then) and the 20 below it the part to decide by,
// so 16 random bits are added there.  (That power comes after the scale factor:
// both in one would leave fp32's normal range for roots from 2.9e4 on.)  i: of the
// first value (even).
template <bool STOCHASTIC>
MOE_DEV u32x2 encode_r(const Coding& k, uint32_t key, int64_t i, const float (&r)[kPer]) {
  // (a block with an infinity has the factor 0, and codes of zero: NaN all of it)
  const uint32_t least = k.r > 0.0f ? 0x00100000u : 0;   // the code above zero's
  if constexpr (!STOCHASTIC) {
    float y[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      y[j] = r[j] * k.r;
      if (r[j] > 0.0f && least) y[j] = fmaxf(y[j], 0x1p-9f);   // (2^-10 and less would become zero)
    }
    return encode8(y);
  } else {
    u32x2 w = {0, 0};
    bool nan = false;
#pragma unroll
    for (int j = 0; j < kPer; j += 2) {
      const uint32_t h = mix32(key + static_cast<uint32_t>(i >> 1) + j / 2);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float y = r[j + n] * k.r;
        nan |= y != y;
        uint32_t u = __float_as_uint(y * 0x1p-120f) + ((n ? h >> 16 : h & 0xffffu) << 4);
        u = u < 0x07efffffu ? u : 0x07efffffu;                 // 448
        const uint32_t some = __float_as_uint(r[j + n]) < least ? __float_as_uint(r[j + n]) : least;
        u = u > some ? u : some;                               // not zero
        w[j / 4] |= (u >> 20) << (8 * ((j + n) % 4));
      }
    }
    if (nan) {
      asm volatile("");
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const float y = r[j] * k.r;
        if (y != y) w[j / 4] |= 0x7fu << (8 * (j % 4));
      }
    }
    return w;
  }
}

// ---- aligned buffers: every load of a chunk in flight ----
// end: of the elements in whole groups (fp32 states) or blocks; FULL: the chunk
// has no others, else loads past them are made from the last ones.
// STREAM: past the caches, for lists that these do not hold.
template <bool STREAM, typename V>
MOE_DEV V load_vec(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const V*>(p));
  else return *static_cast<const V*>(p);
}
template <bool STREAM, typename V>
MOE_DEV void store_vec(void* p, V v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, static_cast<V*>(p));
  else *static_cast<V*>(p) = v;
}
MOE_DEV float lo16(uint32_t w) { return __uint_as_float(w << 16); }
MOE_DEV float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// fp32 states: 4 consecutive elements a thread, kGroups times.
template <bool FULL, bool STREAM, bool P16, bool MASTER, bool G16, bool SMALL>
MOE_DEV void chunk_f32(const AdamEntry& t, const Consts& c, float wd_lr, int64_t base, int64_t end) {
  constexpr int kGroups = kAdamChunk / (4 * kThreads);
  typedef std::conditional_t<G16, u32x2, u32x4> RawG;
  typedef std::conditional_t<P16 && !MASTER, u32x2, u32x4> RawW;
  RawG g[kGroups];
  RawW w[kGroups];
  u32x4 m[kGroups], v[kGroups];
  char* wp = static_cast<char*>(MASTER ? static_cast<void*>(t.master) : t.param);
  const int64_t i0 = base + threadIdx.x * 4;
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    int64_t i = i0 + u * 4 * kThreads;
    if (!FULL && i >= end) i = end - 4;
    g[u] = load_vec<STREAM, RawG>(static_cast<const char*>(t.grad) + i * (G16 ? 2 : 4));
    w[u] = load_vec<STREAM, RawW>(wp + i * static_cast<int64_t>(sizeof(RawW) / 4));
    m[u] = load_vec<STREAM, u32x4>(static_cast<const float*>(t.m) + i);
    v[u] = load_vec<STREAM, u32x4>(static_cast<const float*>(t.v) + i);
  }
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    const int64_t i = i0 + u * 4 * kThreads;
    if (!FULL && i >= end) break;
    float wf[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float gf, mf = __uint_as_float(m[u][j]), vf = __uint_as_float(v[u][j]);
      if constexpr (G16) gf = j % 2 ? hi16(g[u][j / 2]) : lo16(g[u][j / 2]);
      else gf = __uint_as_float(g[u][j]);
      if constexpr (P16 && !MASTER) wf[j] = j % 2 ? hi16(w[u][j / 2]) : lo16(w[u][j / 2]);
      else wf[j] = __uint_as_float(w[u][j]);
      moments<false>(c, gf, mf, vf);
      wf[j] = stepped(c, wd_lr, mf, root_ulp<SMALL>(vf), wf[j]);
      m[u][j] = __float_as_uint(mf);
      v[u][j] = __float_as_uint(vf);
    }
    const u32x4 whole = {__float_as_uint(wf[0]), __float_as_uint(wf[1]), __float_as_uint(wf[2]), __float_as_uint(wf[3])};
    const u32x2 half = {pack_bf16x2(wf[0], wf[1]), pack_bf16x2(wf[2], wf[3])};
    if constexpr (MASTER) store_vec<STREAM>(t.master + i, whole);
    if constexpr (P16) store_vec<STREAM>(static_cast<bf16_t*>(t.param) + i, half);
    else store_vec<STREAM>(static_cast<float*>(t.param) + i, whole);
    store_vec<STREAM>(static_cast<float*>(t.m) + i, m[u]);
    store_vec<STREAM>(static_cast<float*>(t.v) + i, v[u]);
  }
}

// 8-bit states: 8 consecutive elements a thread, kGroups times.
template <bool FULL, bool STREAM, bool P16, bool MASTER, bool G16, bool STOCHASTIC>
MOE_DEV void chunk_fp8(const AdamEntry& t, const Consts& c, float wd_lr, int64_t base, int64_t end, uint32_t key) {
  constexpr int kGroups = kAdamChunk / (8 * kThreads);
  constexpr int kG = G16 ? 1 : 2, kW = P16 && !MASTER ? 1 : 2;   // 16-byte loads
  u32x4 g[kGroups][kG], w[kGroups][kW];
  u32x2 mc[kGroups], rc[kGroups];
  float ms[kGroups], rs[kGroups];
  char* wp = static_cast<char*>(MASTER ? static_cast<void*>(t.master) : t.param);
  const int64_t i0 = base + threadIdx.x * 8;
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    int64_t i = i0 + u * 8 * kThreads;
    if (!FULL && i >= end) i = end - 8;
#pragma unroll
    for (int n = 0; n < kG; ++n) g[u][n] = load_vec<STREAM, u32x4>(static_cast<const char*>(t.grad) + i * (2 * kG) + 16 * n);
#pragma unroll
    for (int n = 0; n < kW; ++n) w[u][n] = load_vec<STREAM, u32x4>(wp + i * (2 * kW) + 16 * n);
    mc[u] = load_vec<STREAM, u32x2>(static_cast<const uint8_t*>(t.m) + i);
    rc[u] = load_vec<STREAM, u32x2>(static_cast<const uint8_t*>(t.v) + i);
    ms[u] = t.m_scale[i / MOE_FP8_BLOCK];
    rs[u] = t.v_scale[i / MOE_FP8_BLOCK];
  }
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    const int64_t i = i0 + u * 8 * kThreads;
    if (!FULL && i >= end) break;   // (blocks leave as a whole)
    float m[kPer], v[kPer], r[kPer], wf[kPer];
    decode8(mc[u], ms[u], m);
    decode8(rc[u], rs[u], v);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      float gf;
      if constexpr (G16) gf = j % 2 ? hi16(g[u][0][j / 2]) : lo16(g[u][0][j / 2]);
      else gf = __uint_as_float(g[u][j / 4][j % 4]);
      v[j] *= v[j];
      moments<true>(c, gf, m[j], v[j]);
    }
    roots(v, r);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if constexpr (kW == 1) wf[j] = j % 2 ? hi16(w[u][0][j / 2]) : lo16(w[u][0][j / 2]);
      else wf[j] = __uint_as_float(w[u][j / 4][j % 4]);
      wf[j] = stepped(c, wd_lr, m[j], r[j], wf[j]);
    }
    if constexpr (kW == 2) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
        store_vec<STREAM>(wp + i * 4 + 16 * n, u32x4{__float_as_uint(wf[4 * n]), __float_as_uint(wf[4 * n + 1]), __float_as_uint(wf[4 * n + 2]),
                                                     __float_as_uint(wf[4 * n + 3])});
    }
    if constexpr (P16)
      store_vec<STREAM>(static_cast<bf16_t*>(t.param) + i, u32x4{pack_bf16x2(wf[0], wf[1]), pack_bf16x2(wf[2], wf[3]), pack_bf16x2(wf[4], wf[5]),
                                                                 pack_bf16x2(wf[6], wf[7])});
    const Coding k = coding_of(t, i / MOE_FP8_BLOCK, m, r);
    store_vec<STREAM>(static_cast<uint8_t*>(t.m) + i, encode_m(k, m));
    store_vec<STREAM>(static_cast<uint8_t*>(t.v) + i, encode_r<STOCHASTIC>(k, key, i, r));
  }
}

// ---- element by element: buffers that are not aligned, and what a tensor's end
// leaves of a group (fp32 states) or a block (8-bit ones) ----
template <bool FP8, bool SPECIAL>
MOE_DEV void chunk_any(const AdamEntry& t, const Consts& c, float wd_lr, int64_t base, int64_t end, uint32_t key) {
  const int64_t n = t.numel;
  const bool p16 = t.flags & kAdamParam16, g16 = t.flags & kAdamGrad16;
  // (the 16 lanes of a block stay together: those past the end hold zeros)
  for (int64_t i = base + threadIdx.x * kPer; i < end && (FP8 ? i / MOE_FP8_BLOCK * MOE_FP8_BLOCK : i) < n; i += kThreads * kPer) {
    float g[kPer], w[kPer], m[kPer], v[kPer], r[kPer];
    if (g16) load8(static_cast<const bf16_t*>(t.grad), i, n, g);
    else load8(static_cast<const float*>(t.grad), i, n, g);
    if (t.master) load8(t.master, i, n, w);
    else if (p16) load8(static_cast<const bf16_t*>(t.param), i, n, w);
    else load8(static_cast<const float*>(t.param), i, n, w);
    const int64_t blk = i / MOE_FP8_BLOCK;
    if constexpr (FP8) {
      decode8(load_codes(static_cast<const uint8_t*>(t.m), i, n), t.m_scale[blk], m);
      decode8(load_codes(static_cast<const uint8_t*>(t.v), i, n), t.v_scale[blk], v);
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] *= v[j];
    } else {
      load8(static_cast<const float*>(t.m), i, n, m);
      load8(static_cast<const float*>(t.v), i, n, v);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) moments<FP8>(c, g[j], m[j], v[j]);
    if constexpr (FP8) roots(v, r);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if constexpr (!FP8) r[j] = root_ulp<SPECIAL>(v[j]);
      w[j] = stepped(c, wd_lr, m[j], r[j], w[j]);
    }
    if (t.master) store8(t.master, i, n, w);
    if (p16) store8(static_cast<bf16_t*>(t.param), i, n, w);
    else store8(static_cast<float*>(t.param), i, n, w);
    if constexpr (FP8) {
      const Coding k = coding_of(t, blk, m, r);
      store_codes(static_cast<uint8_t*>(t.m), i, n, encode_m(k, m));
      store_codes(static_cast<uint8_t*>(t.v), i, n, encode_r<SPECIAL>(k, key, i, r));
    } else {
      store8(static_cast<float*>(t.m), i, n, m);
      store8(static_cast<float*>(t.v), i, n, v);
    }
  }
}

// SPECIAL: roots rounded stochastically (8-bit states), those of small values scaled
// (fp32 states).
template <bool FP8, bool STREAM, bool SPECIAL>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamList l) {
  Consts c{1.0f, l.lr, l.lr_c1, l.rs_c2, l.b1, l.a1, l.b2, l.a2, l.eps};
  uint32_t step = static_cast<uint32_t>(l.step);
  if (l.lr_dev || l.step_dev) {
    if (l.lr_dev) c.lr = *l.lr_dev;
    double c1 = l.c1;
    if (l.step_dev) {
      const int n = *l.step_dev > 1 ? *l.step_dev : 1;
      step = static_cast<uint32_t>(n);
      c1 = 1.0 - pow(l.b1_64, static_cast<double>(n));
      c.rs_c2 = static_cast<float>(1.0 / sqrt(1.0 - pow(l.b2_64, static_cast<double>(n))));
    }
    c.lr_c1 = static_cast<float>(static_cast<double>(c.lr) / c1);
  }
  if (l.sumsq) {
    const double norm = sqrt(*l.sumsq);
    if (!(norm <= 1.7976931348623157e308)) {   // infinite or NaN: no step
      if (blockIdx.x == 0 && threadIdx.x == 0) set_err(l.err, MOE_DEVERR_NONFINITE);
      return;
    }
    const double f = l.max_norm / (norm + 1e-6);
    c.f = f < 1.0 ? static_cast<float>(f) : 1.0f;
  }
  constexpr bool STOCHASTIC = FP8 && SPECIAL;
  const uint32_t key0 = STOCHASTIC ? mix32(l.seed + step * 0x9e3779b9u) : 0;
  for (int64_t ch = blockIdx.x; ch < l.chunks; ch += gridDim.x) {
    int lo = 0, hi = l.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (l.t[mid].first <= ch) lo = mid; else hi = mid - 1;
    }
    const AdamEntry& t = l.t[lo];
    const int64_t base = (ch - t.first) * kAdamChunk;
    const float wd_lr = t.weight_decay * c.lr;
    const uint32_t key = STOCHASTIC ? mix32(key0 + t.index) : 0;
    if (!(t.flags & kAdamVec)) {
      chunk_any<FP8, SPECIAL>(t, c, wd_lr, base, base + kAdamChunk, key);
      continue;
    }
    const bool full = base + kAdamChunk <= t.numel;
    int64_t end = base + kAdamChunk;
    if (!full) {
      constexpr int kWhole = FP8 ? MOE_FP8_BLOCK : 4;
      end = t.numel / kWhole * kWhole;
      if (end < t.numel) chunk_any<FP8, SPECIAL>(t, c, wd_lr, end, end + kAdamChunk, key);
      if (end <= base) continue;
    }
    const bool p16 = t.flags & kAdamParam16, g16 = t.flags & kAdamGrad16;
    auto with = [&](auto whole, auto p, auto master, auto grad) {
      constexpr bool F = decltype(whole)::value, P = decltype(p)::value, M = decltype(master)::value, G = decltype(grad)::value;
      if constexpr (FP8) chunk_fp8<F, STREAM, P, M, G, STOCHASTIC>(t, c, wd_lr, base, end, key);
      else chunk_f32<F, STREAM, P, M, G, SPECIAL>(t, c, wd_lr, base, end);
    };
    auto go = [&](auto p, auto master, auto grad) {
      if (full) with(std::true_type{}, p, master, grad);
      else with(std::false_type{}, p, master, grad);
    };
    using Y = std::true_type;
    using N = std::false_type;
    if (t.master) g16 ? go(Y{}, Y{}, Y{}) : go(Y{}, Y{}, N{});
    else if (p16) g16 ? go(Y{}, N{}, Y{}) : go(Y{}, N{}, N{});
    else g16 ? go(N{}, N{}, Y{}) : go(N{}, N{}, N{});
  }
}

}  // namespace

hipError_t launch_adamw(const AdamList& l, bool fp8, hipStream_t s) {
  // a workgroup for every chunk (705 M elements, fp32 states, 30 bytes each: 3.73
  // ms; 2048 workgroups that stride over the chunks 4.15); where the step is counted
  // on the device every workgroup makes the constants, so fewer (4.19 ms, 8-bit states
  // 1.57 against 1.23)
  const int64_t most = l.step_dev ? 4096 : kAdamBlocks;
  const int grid = static_cast<int>(l.chunks < most ? l.chunks : most);
  int64_t bytes = 0;
  for (int i = 0; i < l.n; ++i) bytes += l.t[i].numel * (fp8 ? 6 : 16);
  auto go = [&](auto kernel) { kernel<<<grid, kThreads, 0, s>>>(l); };
  const bool stream = bytes > kStreamBytes;
  if (!fp8 && l.small_roots) stream ? go(adamw_kernel<false, true, true>) : go(adamw_kernel<false, false, true>);
  else if (!fp8) stream ? go(adamw_kernel<false, true, false>) : go(adamw_kernel<false, false, false>);
  else if (l.stochastic) stream ? go(adamw_kernel<true, true, true>) : go(adamw_kernel<true, false, true>);
  else stream ? go(adamw_kernel<true, true, false>) : go(adamw_kernel<true, false, false>);
  return hipGetLastError();
}

}  // namespace moe
