// C ABI of the operators around the expert products of a training step:
// block-scaled FP8 (quantization, grouped product, weight gradient), the
// router's losses and gradient, and the gradient norm and clipping.  As in
// api.cpp every call checks its arguments, then only enqueues kernels.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "../../include/moe_gmlp.h"
#include "kernels.h"

namespace {

using moe::kMaxExperts;
using moe::kMaxTopK;

constexpr int kBlk = MOE_FP8_BLOCK;
constexpr int kTileN = 256;              // weight rows of a product's tile
constexpr int64_t kMaxGridX = 1 << 24;   // workgroups of 256 threads in x

moe_status launched(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool type_ok(int t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F32; }
int64_t type_bytes(int t) { return t == MOE_TYPE_BF16 ? 2 : 4; }

// Workgroups of a persistent product over at most `tiles` tiles.
int tile_grid(int cu, int margin, int64_t tiles) {
  int g = cu - margin;
  if (g >= 8) g -= g % 8;
  if (tiles < g) g = static_cast<int>(tiles);
  return g < 1 ? 1 : g;
}

// 64-token groups of a tile: as many as there may be, but half where that still
// leaves a CU for every tile, as the wider tile takes longer (2 groups of 372 rows,
// N=1824 K=1088: 23 us with 128 tokens, 19 with 64, by fp8_sums 20 with 256 and 13
// with 64; where tiles are more than CUs, narrow ones read the weights more often:
// 22 groups of 196 rows, N=7632 K=1296, 165 us with 128, 210 with 64, by fp8_sums
// 90 with 256, 162 with 64).  `tiles`: how many tiles of 64 g tokens.
template <typename F>
int tile_groups(bool wide, int cu, F&& tiles) {
  int g = moe::fp8_most_groups(wide);
  while (g > 1 && tiles(g / 2) <= cu) g /= 2;
  return g;
}

// Whether an output of `rows` rows of `row` bytes is stored past the caches: more
// than they hold, in whole 128-byte lines.
int streams(int64_t rows, int64_t row) { return rows * row > moe::kStreamBytes && row % 128 == 0; }

// Whether the product may cut K: rows that take the tiled kernel, 24 scale
// blocks at least, and a row buffer (less a group's padding each) that cannot
// fill the device with tiles.  The second launch costs 7 us also where nothing
// was cut (E=22 N=352 K=2080, 34 tiles of few rows, by fp8_sums: 14 us without it,
// 21 with).  Groups packed without padding hold more rows than the estimate, and
// may pay for that launch in vain: 64 of 128 rows, N=4096 K=4096, by fp8_sums 272
// us against 268.
int64_t rows_estimate(int E, int64_t M_cap) {
  return std::max<int64_t>(1, M_cap - static_cast<int64_t>(E) * (MOE_GROUP_ALIGN - 1));
}
bool cuts_k(int E, int N, int K, int64_t M_cap, int64_t most_rows, int cu) {
  const int64_t rows = rows_estimate(E, M_cap);
  return most_rows > 32 && K > 23 * kBlk && ceil_div(rows, 256) * ceil_div(N, kTileN) < cu;
}

struct Range {
  uintptr_t lo, hi;
  bool write;
};

// Whether a range that is written overlaps another one.
bool overlap(Range* r, int64_t n) {
  std::sort(r, r + n, [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t w = 0, any = 0;   // furthest end of the written ranges and of all
  for (int64_t i = 0; i < n; ++i) {
    if (r[i].lo < (r[i].write ? any : w)) return true;
    any = std::max(any, r[i].hi);
    if (r[i].write) w = std::max(w, r[i].hi);
  }
  return false;
}

// Checks of the tensor list that both calls share.
moe_status list_check(const moe_grad_args* a) {
  if (!a || a->n_tensors < 0 || (a->n_tensors > 0 && !a->tensors) || !a->sumsq ||
      (reinterpret_cast<uintptr_t>(a->sumsq) & 7))
    return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < a->n_tensors; ++i) {
    const moe_tensor& t = a->tensors[i];
    if (!type_ok(t.type) || t.numel < 0 || t.numel > (int64_t(1) << 46) ||
        (t.numel > 0 && !t.data))
      return MOE_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(t.data) | reinterpret_cast<uintptr_t>(t.out)) %
        type_bytes(t.type))
      return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

// Runs f(list) for the tensors kGradList at a time.
template <typename F>
moe_status for_lists(const moe_grad_args* a, F&& f) {
  int i = 0;
  do {
    moe::GradList l{};
    for (; i < a->n_tensors && l.n < moe::kGradList; ++i) {
      const moe_tensor& t = a->tensors[i];
      if (t.numel == 0) continue;
      l.t[l.n++] = moe::GradEntry{t.data, t.out ? t.out : t.data, t.numel, l.chunks, t.type};
      l.chunks += ceil_div(t.numel, moe::kGradChunk);
    }
    if (moe_status st = f(l)) return st;
  } while (i < a->n_tensors);
  return MOE_OK;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------- block FP8 ------
moe_status moe_quantize_fp8(const moe_quant_fp8_args* a, void* stream) {
  if (!a || a->mode < MOE_QUANT_ROW || a->mode > MOE_QUANT_TILE || a->batch < 0 || a->rows < 0 ||
      a->cols < 16 || a->cols % 16 != 0 || (a->mode != MOE_QUANT_ROW && a->rows % 16 != 0) ||
      !aligned16(a->x) || !aligned16(a->q) || !aligned16(a->qT))
    return MOE_ERR_INVALID_ARG;
  const int64_t n = static_cast<int64_t>(a->rows) * a->cols;
  if (a->x_stride != 0 && (a->x_stride < n || a->x_stride % 8 != 0)) return MOE_ERR_INVALID_ARG;
  const bool nothing = a->batch == 0 || a->rows == 0;   // empty tensors may have no address
  if (!nothing && (!a->x || !a->q || !a->s || (a->mode == MOE_QUANT_BOTH && (!a->qT || !a->sT)) ||
                   (a->mode == MOE_QUANT_TILE && (a->qT != nullptr) != (a->sT != nullptr))))
    return MOE_ERR_INVALID_ARG;
  const int64_t cb = ceil_div(a->cols, kBlk);
  const int64_t units = a->mode == MOE_QUANT_ROW ? ceil_div(a->rows, 16) * ceil_div(cb, 8)
                                                 : ceil_div(a->rows, kBlk) * cb;
  if (a->batch > 65535 || units >= kMaxGridX) return MOE_ERR_UNSUPPORTED;
  int cu = 0;
  if (moe_status st = moe::current_device(&cu)) return st;
  if (nothing) return MOE_OK;
  moe_quant_fp8_args b = *a;
  if (b.x_stride == 0) b.x_stride = n;
  return launched(moe::launch_quantize_fp8(b, static_cast<hipStream_t>(stream)));
}

// One tile's fp32 sums for every workgroup of a full grid; nothing where K is
// too short to be cut or the kernel for few rows runs, which needs none.
size_t moe_grouped_gemm_fp8_workspace_size(int E, int N, int K, int64_t M_cap, int max_rows) {
  if (E < 1 || N < 1 || K < 1 || M_cap < 1 || max_rows < 0) return 0;
  int cu = 0;
  if (moe::current_device(&cu) != MOE_OK) cu = 256;
  if (!cuts_k(E, N, K, M_cap, max_rows ? std::min<int64_t>(max_rows, M_cap) : M_cap, cu)) return 0;
  return static_cast<size_t>(cu) * moe::kFp8PartFloats * sizeof(float);
}

moe_status moe_grouped_gemm_fp8(const moe_gemm_fp8_args* a, void* stream) {
  if (!a || a->E < 1 || a->E > kMaxExperts || a->N < 16 || a->N % 16 != 0 || a->K < 16 ||
      a->K % 16 != 0 || a->K > (1 << 22) || a->M_cap < 1 || a->M_cap > INT32_MAX ||
      !a->split_sizes || !a->padded_offsets || !a->a || !a->a_s || !a->b || !a->b_s || !a->c ||
      !type_ok(a->c_type) || (a->fp8_sums && a->c_type != MOE_TYPE_BF16) || !aligned16(a->workspace) || a->max_rows < 0 || a->cu_margin < 0 || !aligned16(a->a) ||
      !aligned16(a->b) || !aligned16(a->c))
    return MOE_ERR_INVALID_ARG;
  const int64_t nk = static_cast<int64_t>(a->N) * a->K;
  const int64_t ns = ceil_div(a->N, kBlk) * ceil_div(a->K, kBlk);
  if ((a->b_stride != 0 && (a->b_stride < nk || a->b_stride % 16 != 0)) ||
      (a->b_s_stride != 0 && a->b_s_stride < ns) ||
      (a->ldc != 0 && (a->ldc < a->N || a->ldc % 8 != 0)))
    return MOE_ERR_INVALID_ARG;
  const int64_t most = a->max_rows ? std::min<int64_t>(a->max_rows, a->M_cap) : a->M_cap;
  const bool f32 = a->c_type == MOE_TYPE_F32, wide = !a->fp8_sums;
  const int64_t rows = rows_estimate(a->E, a->M_cap), tiles_n = ceil_div(a->N, kTileN);
  auto at_most = [&](int g) { return (ceil_div(a->M_cap, 64 * g) + a->E) * tiles_n; };
  if (at_most(moe::fp8_most_groups(wide)) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  int cu = 0;
  if (moe_status st = moe::current_device(&cu)) return st;
  // half a tile of every group is filled on average
  const int groups = tile_groups(wide, cu - a->cu_margin, [&](int g) { return (ceil_div(rows, 64 * g) + a->E / 2) * tiles_n; });
  const int64_t tiles = at_most(groups);
  if (a->cu_margin >= cu) return MOE_ERR_INVALID_ARG;
  moe::Fp8Args g{};
  g.E = a->E;
  g.N = a->N;
  g.K = a->K;
  g.M_cap = a->M_cap;
  g.split = a->split_sizes;
  g.padded = a->padded_offsets;
  g.a = a->a;
  g.a_s = a->a_s;
  g.b = a->b;
  g.b_s = a->b_s;
  g.b_stride = a->b_stride ? a->b_stride : nk;
  g.b_s_stride = a->b_s_stride ? a->b_s_stride : ns;
  g.c = a->c;
  g.ldc = a->ldc ? a->ldc : a->N;
  g.stream = a->M_cap <= (int64_t(1) << 62) / 4 / g.ldc && streams(a->M_cap, g.ldc * type_bytes(a->c_type));
  g.group_m = 4;
  g.err = a->err_flag;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  // (the kernel for few rows has many workgroups a CU and spreads over all of
  // them: with CUs to be left free the tiled one runs, one workgroup a CU; 2 rows
  // for each of 8 experts of 28672 x 4096: 177 us, with a margin of 32 CUs 211)
  if (most <= 32 && a->cu_margin == 0 && a->N / 32 < kMaxGridX - 1) return launched(moe::launch_fp8_rows(g, most <= 16 ? 16 : 32, f32, wide, s));
  // K may be cut where there is room for its parts; the grid is a full one
  // then, since the tiles' number is known on the device only
  const int full = tile_grid(cu, a->cu_margin, INT32_MAX);
  const bool cut = cuts_k(a->E, a->N, a->K, a->M_cap, most, cu) && a->workspace &&
                   a->workspace_bytes >= static_cast<size_t>(full) * moe::kFp8PartFloats * sizeof(float);
  if (cut) g.part = static_cast<moe::fp8_f32x4*>(a->workspace);
  g.grid = cut ? full : tile_grid(cu, a->cu_margin, tiles);
  return launched(moe::launch_fp8_gemm(g, f32, wide, groups, s));
}

moe_status moe_grouped_wgrad_fp8(const moe_wgrad_fp8_args* a, void* stream) {
  if (!a || a->E < 1 || a->E > kMaxExperts || a->P < 16 || a->P % 16 != 0 || a->Q < 16 ||
      a->Q % 16 != 0 || a->M_cap < 128 || a->M_cap % 128 != 0 || a->M_cap > 4194304 ||
      !a->split_sizes || !a->padded_offsets || !a->a || !a->a_s || !a->b || !a->b_s || !a->c ||
      !type_ok(a->c_type) || (a->accumulate && a->c_type != MOE_TYPE_F32) ||
      (a->fp8_sums && a->c_type != MOE_TYPE_BF16) || a->cu_margin < 0 ||
      !aligned16(a->a) || !aligned16(a->b) || !aligned16(a->c))
    return MOE_ERR_INVALID_ARG;
  const bool f32 = a->c_type == MOE_TYPE_F32, wide = !a->fp8_sums;
  auto count = [&](int g) { return a->E * ceil_div(a->P, 64 * g) * ceil_div(a->Q, kTileN); };
  if (count(moe::fp8_most_groups(wide)) > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  int cu = 0;
  if (moe_status st = moe::current_device(&cu)) return st;
  const int groups = tile_groups(wide, cu - a->cu_margin, count);
  const int64_t tiles = count(groups);
  if (a->cu_margin >= cu) return MOE_ERR_INVALID_ARG;
  moe::Fp8Args g{};
  g.E = a->E;
  g.N = a->Q;
  g.P = a->P;
  g.M_cap = a->M_cap;
  g.split = a->split_sizes;
  g.padded = a->padded_offsets;
  g.a = a->a;
  g.a_s = a->a_s;
  g.b = a->b;
  g.b_s = a->b_s;
  g.c = a->c;
  g.ldc = a->Q;
  g.accumulate = a->accumulate != 0;
  g.stream = streams(static_cast<int64_t>(a->E) * a->P, static_cast<int64_t>(a->Q) * type_bytes(a->c_type));
  g.group_m = 4;
  g.err = a->err_flag;
  g.grid = tile_grid(cu, a->cu_margin, tiles);
  return launched(moe::launch_fp8_wgrad(g, f32, wide, groups, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------------- router losses ------
size_t moe_router_loss_workspace_size(int T, int E) {
  if (T < 0 || E < 1 || E > kMaxExperts) return 0;
  return moe::router_loss_workspace_bytes(T, E);
}

moe_status moe_router_loss(const moe_router_loss_args* a, void* stream) {
  if (!a || a->T < 0 || a->E < 1 || a->E > kMaxExperts || a->k < 1 ||
      a->k > std::min(a->E, kMaxTopK) || static_cast<int64_t>(a->T) * a->k > INT32_MAX ||
      (a->T > 0 && (!a->logits || !a->expert_idx)) || !std::isfinite(a->balance_coef) ||
      !std::isfinite(a->z_coef) || !a->counts || !a->n_tokens || !a->prob_mean || !a->loss)
    return MOE_ERR_INVALID_ARG;
  if (!a->workspace || a->workspace_bytes < moe_router_loss_workspace_size(a->T, a->E) ||
      (reinterpret_cast<uintptr_t>(a->workspace) & 7))
    return MOE_ERR_WORKSPACE;
  int cu = 0;
  if (moe_status st = moe::current_device(&cu)) return st;
  return launched(moe::launch_router_loss(*a, static_cast<hipStream_t>(stream)));
}

moe_status moe_router_bwd(const moe_router_bwd_args* a, void* stream) {
  if (!a || a->T < 0 || a->E < 1 || a->E > kMaxExperts || a->k < 1 ||
      a->k > std::min(a->E, kMaxTopK) || static_cast<int64_t>(a->T) * a->k > INT32_MAX ||
      (a->T > 0 && (!a->logits || !a->expert_idx || !a->dlogits)) ||
      !std::isfinite(a->balance_coef) || !std::isfinite(a->z_coef) ||
      ((a->balance_coef != 0.0f || a->z_coef != 0.0f) && (!a->counts || !a->n_tokens)))
    return MOE_ERR_INVALID_ARG;
  int cu = 0;
  if (moe_status st = moe::current_device(&cu)) return st;
  if (a->T == 0) return MOE_OK;
  return launched(moe::launch_router_bwd(*a, static_cast<hipStream_t>(stream)));
}

// ------------------------------------------------ gradient norm, clipping ---
size_t moe_grad_workspace_size(int n_tensors) {
  if (n_tensors < 0) return 0;
  const int64_t lists = std::max<int64_t>(1, ceil_div(n_tensors, moe::kGradList));
  return static_cast<size_t>(lists) * moe::kGradBlocks * sizeof(double);
}

moe_status moe_grad_sumsq(const moe_grad_args* a, void* stream) {
  if (moe_status st = list_check(a)) return st;
  if (!a->workspace || a->workspace_bytes < moe_grad_workspace_size(a->n_tensors) ||
      (reinterpret_cast<uintptr_t>(a->workspace) & 7))
    return MOE_ERR_WORKSPACE;
  int cu = 0;
  if (moe_status st = moe::current_device(&cu)) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  double* partial = static_cast<double*>(a->workspace);
  int n = 0;   // partial sums so far; at most kGradBlocks per list
  if (moe_status st = for_lists(a, [&](const moe::GradList& l) {
        if (l.chunks == 0) return MOE_OK;
        const hipError_t e = moe::launch_grad_sumsq(l, partial + n, s);
        n += moe::grad_blocks(l.chunks);
        return launched(e);
      }))
    return st;
  return launched(moe::launch_grad_sum(partial, n, a->sumsq, s));
}

moe_status moe_grad_clip(const moe_grad_args* a, void* stream) {
  if (moe_status st = list_check(a)) return st;
  if (!(a->max_norm >= 0.0f)) return MOE_ERR_INVALID_ARG;
  // no tensor that is written may overlap another range of the list; a
  // tensor scaled in place is one range
  {
    Range few[2 * moe::kGradList];
    Range* r = few;
    if (a->n_tensors > moe::kGradList) {
      r = new (std::nothrow) Range[2 * static_cast<size_t>(a->n_tensors)];
      if (!r) return MOE_ERR_UNSUPPORTED;
    }
    int64_t n = 0;
    for (int i = 0; i < a->n_tensors; ++i) {
      const moe_tensor& t = a->tensors[i];
      if (t.numel == 0) continue;
      const uintptr_t bytes = static_cast<uintptr_t>(t.numel) * type_bytes(t.type);
      const uintptr_t in = reinterpret_cast<uintptr_t>(t.data);
      const uintptr_t out = t.out ? reinterpret_cast<uintptr_t>(t.out) : in;
      if (out != in) r[n++] = Range{in, in + bytes, false};
      r[n++] = Range{out, out + bytes, true};
    }
    const bool bad = overlap(r, n);
    if (r != few) delete[] r;
    if (bad) return MOE_ERR_INVALID_ARG;
  }
  int cu = 0;
  if (moe_status st = moe::current_device(&cu)) return st;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return for_lists(a, [&](const moe::GradList& l) {
    return launched(moe::launch_grad_scale(l, a->sumsq, a->max_norm, a->norm, a->err_flag, s));
  });
}

}  // extern "C"
