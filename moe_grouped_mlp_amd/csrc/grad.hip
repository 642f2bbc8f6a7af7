// Global gradient norm and clipping over a list of tensors.
//
//   S = sum g^2;  f = min(1, max_norm / (sqrt(S) + 1e-6));  out = g f
//
// Both passes are bound by HBM: the norm reads every gradient once, the
// clipping reads it again and writes it.  Squares are summed in fp64 (the
// square of an fp32 value is exact to 2^-53 and cannot overflow, and the
// fp64 rate of MI355X keeps up with the loads).  The list goes to the kernels by value, up to
// kGradList tensors a launch, so a call copies nothing to the device and can
// be captured in a graph.  Every tensor is cut into chunks of kChunk elements
// from its first 16-byte boundary on; a workgroup takes chunks with a fixed
// stride, and its fp64 sum goes to its own slot, so the order of the sum
// depends on the list alone.  Two bf16 gradients, 2.8 GB: 456 us for the norm
// (6.2 TB/s), 1021 for the clipping (5.5 TB/s of reads and writes); sixty small
// ones: 5.2, 1.6 and 6.2 us in three launches.
#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kThreads = 256;
constexpr int kVecs = 8;   // 16-byte loads a thread has in flight

template <typename T>
struct Vec;   // a 16-byte group of elements
template <>
struct Vec<bf16_t> {
  static constexpr int n = 8;
  MOE_DEV static void unpack(const uint4& w, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  MOE_DEV static uint4 pack(const float (&v)[8]) {
    return uint4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                 pack_bf16x2(v[6], v[7])};
  }
  MOE_DEV static float get(bf16_t b) { return bf16_to_f32(b); }
  MOE_DEV static bf16_t put(float f) { return static_cast<bf16_t>(pack_bf16x2(f, 0.0f)); }
};
template <>
struct Vec<float> {
  static constexpr int n = 4;
  MOE_DEV static void unpack(const uint4& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
  }
  MOE_DEV static uint4 pack(const float (&v)[4]) {
    return uint4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                 __float_as_uint(v[3])};
  }
  MOE_DEV static float get(float b) { return b; }
  MOE_DEV static float put(float f) { return f; }
};

// Elements before p's first 16-byte boundary.
template <typename T>
MOE_DEV int64_t head_of(const void* p) {
  return ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
}

// The chunk's elements [lo, hi) that lie in whole 16-byte groups, and the
// rest: [edge0, lo) and [hi, edge1).
struct Span {
  int64_t edge0, lo, hi, edge1;
};
template <typename T>
MOE_DEV Span span_of(const GradEntry& t, int64_t chunk, int64_t chunks) {
  const int64_t head = head_of<T>(t.data);
  Span s;
  s.lo = head + chunk * kGradChunk;
  s.hi = chunk + 1 == chunks ? t.numel : s.lo + kGradChunk;
  if (s.hi > t.numel) s.hi = t.numel;
  if (s.lo > s.hi) s.lo = s.hi;
  s.edge0 = chunk == 0 ? 0 : s.lo;
  s.edge1 = s.hi;
  s.hi = s.lo + (s.hi - s.lo) / Vec<T>::n * Vec<T>::n;
  return s;
}

// Loads past a chunk's end are made from its last group and dropped: one
// behind a condition would be waited for before the next.
MOE_DEV int64_t clamped(int64_t i, int64_t n) { return i < n ? i : n - 1; }

template <typename T>
MOE_DEV double chunk_sumsq(const GradEntry& t, int64_t chunk, int64_t chunks) {
  const T* p = static_cast<const T*>(t.data);
  const Span s = span_of<T>(t, chunk, chunks);
  double sum = 0.0;
  const int64_t vecs = (s.hi - s.lo) / Vec<T>::n;
  const uint4* v = reinterpret_cast<const uint4*>(p + s.lo);
  for (int64_t i = threadIdx.x; i < vecs; i += kThreads * kVecs) {
    uint4 w[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) w[j] = v[clamped(i + j * kThreads, vecs)];
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (i + j * kThreads >= vecs) w[j] = uint4{0, 0, 0, 0};
      float f[Vec<T>::n];
      Vec<T>::unpack(w[j], f);
#pragma unroll
      for (int k = 0; k < Vec<T>::n; ++k) {
        const double d = f[k];
        sum = __builtin_fma(d, d, sum);
      }
    }
  }
  const int64_t before = s.lo - s.edge0, rest = before + (s.edge1 - s.hi);
  for (int64_t i = threadIdx.x; i < rest; i += kThreads) {
    const double d = Vec<T>::get(p[i < before ? s.edge0 + i : s.hi + (i - before)]);
    sum = __builtin_fma(d, d, sum);
  }
  return sum;
}

// F: float, or double for a factor below fp32's normal range.
template <bool STREAM, typename T, typename F>
MOE_DEV void chunk_scale(const GradEntry& t, int64_t chunk, int64_t chunks, F f) {
  const T* p = static_cast<const T*>(t.data);
  T* o = static_cast<T*>(t.out);
  Span s = span_of<T>(t, chunk, chunks);
  // an output with another alignment than its input goes element by element
  if ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) s.hi = s.lo;
  const int64_t vecs = (s.hi - s.lo) / Vec<T>::n;
  // STREAM: neither what is read for the last time nor what is written stays in
  // the caches (2.8 GB with the norm: 1483 us; stores alone 1517, neither 1549;
  // 45 MB, which they hold: 20.4 us, 19.2 without)
  const u32x4* v = reinterpret_cast<const u32x4*>(p + s.lo);
  u32x4* w = reinterpret_cast<u32x4*>(o + s.lo);
  for (int64_t i = threadIdx.x; i < vecs; i += kThreads * kVecs) {
    uint4 u[kVecs];
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      u[j] = __builtin_bit_cast(uint4, STREAM ? __builtin_nontemporal_load(v + clamped(i + j * kThreads, vecs))
                                              : v[clamped(i + j * kThreads, vecs)]);
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      if (i + j * kThreads < vecs) {
        float g[Vec<T>::n];
        Vec<T>::unpack(u[j], g);
#pragma unroll
        for (int k = 0; k < Vec<T>::n; ++k) g[k] = static_cast<float>(g[k] * f);
        const u32x4 o4 = __builtin_bit_cast(u32x4, Vec<T>::pack(g));
        if constexpr (STREAM) __builtin_nontemporal_store(o4, w + i + j * kThreads);
        else w[i + j * kThreads] = o4;
      }
    }
  }
  const int64_t before = s.lo - s.edge0, rest = before + (s.edge1 - s.hi);
  for (int64_t i = threadIdx.x; i < rest; i += kThreads) {
    const int64_t e = i < before ? s.edge0 + i : s.hi + (i - before);
    o[e] = Vec<T>::put(static_cast<float>(Vec<T>::get(p[e]) * f));
  }
}

// The list entry that chunk c belongs to (first[] ascending; entries with no
// elements have no chunk and are never found).
MOE_DEV int entry_of(const GradList& l, int64_t c) {
  int lo = 0, hi = l.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.t[mid].first <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

MOE_DEV double block_sum(double v) {
  __shared__ double s_wave[kThreads / kWave];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  if (threadIdx.x % kWave == 0) s_wave[threadIdx.x / kWave] = v;
  __syncthreads();
  double r = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / kWave; ++i) r += s_wave[i];
  return r;
}

__global__ __launch_bounds__(kThreads) void grad_sumsq_kernel(const GradList l, double* partial) {
  double sum = 0.0;
  for (int64_t c = blockIdx.x; c < l.chunks; c += gridDim.x) {
    const int e = entry_of(l, c);
    const GradEntry& t = l.t[e];
    const int64_t n = (e + 1 < l.n ? l.t[e + 1].first : l.chunks) - t.first;
    sum += t.type == MOE_TYPE_BF16 ? chunk_sumsq<bf16_t>(t, c - t.first, n)
                                   : chunk_sumsq<float>(t, c - t.first, n);
  }
  const double r = block_sum(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = r;
}

__global__ __launch_bounds__(kThreads) void grad_sum_kernel(const double* partial, int n,
                                                            double* sumsq) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) sum += partial[i];
  const double r = block_sum(sum);
  if (threadIdx.x == 0) *sumsq = r;
}

template <bool STREAM>
__global__ __launch_bounds__(kThreads) void grad_scale_kernel(const GradList l, const double* sumsq,
                                                              float max_norm, float* norm_out,
                                                              int32_t* err) {
  const double norm = sqrt(*sumsq);
  const bool finite = norm <= 1.7976931348623157e308;   // false for NaN too
  const double f64 = static_cast<double>(max_norm) / (norm + 1e-6);
  const float f = finite && f64 < 1.0 ? static_cast<float>(f64) : 1.0f;
  // a norm far past max_norm: g f64 may still be a normal number
  const bool wide = f < 1.17549435e-38f && f64 > 0.0;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (norm_out) *norm_out = static_cast<float>(norm);
    if (!finite) set_err(err, MOE_DEVERR_NONFINITE);
  }
  // from the list's end, whose chunks the norm's pass read last: they are
  // the ones that the 256 MB of last-level cache still hold
  for (int64_t i = blockIdx.x; i < l.chunks; i += gridDim.x) {
    const int64_t c = l.chunks - 1 - i;
    const int e = entry_of(l, c);
    const GradEntry& t = l.t[e];
    if (f == 1.0f && t.out == t.data) continue;
    const int64_t n = (e + 1 < l.n ? l.t[e + 1].first : l.chunks) - t.first;
    if (wide) {
      if (t.type == MOE_TYPE_BF16) chunk_scale<STREAM, bf16_t, double>(t, c - t.first, n, f64);
      else chunk_scale<STREAM, float, double>(t, c - t.first, n, f64);
    } else {
      if (t.type == MOE_TYPE_BF16) chunk_scale<STREAM, bf16_t, float>(t, c - t.first, n, f);
      else chunk_scale<STREAM, float, float>(t, c - t.first, n, f);
    }
  }
}

}  // namespace

int grad_blocks(int64_t chunks) {
  return static_cast<int>(chunks < kGradBlocks ? chunks : kGradBlocks);
}

hipError_t launch_grad_sumsq(const GradList& l, double* partial, hipStream_t s) {
  grad_sumsq_kernel<<<grad_blocks(l.chunks), kThreads, 0, s>>>(l, partial);
  return hipGetLastError();
}

hipError_t launch_grad_sum(const double* partial, int n, double* sumsq, hipStream_t s) {
  grad_sum_kernel<<<1, kThreads, 0, s>>>(partial, n, sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradList& l, const double* sumsq, float max_norm, float* norm,
                             int32_t* err, hipStream_t s) {
  const int g = grad_blocks(l.chunks);
  int64_t bytes = 0;
  for (int i = 0; i < l.n; ++i) bytes += l.t[i].numel * (l.t[i].type == MOE_TYPE_BF16 ? 2 : 4);
  auto go = [&](auto kernel) { kernel<<<g < 1 ? 1 : g, kThreads, 0, s>>>(l, sumsq, max_norm, norm, err); };
  if (bytes > kStreamBytes) go(grad_scale_kernel<true>);
  else go(grad_scale_kernel<false>);
  return hipGetLastError();
}

}  // namespace moe
