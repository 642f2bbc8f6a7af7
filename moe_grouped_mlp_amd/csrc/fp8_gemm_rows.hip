// The block-scaled FP8 product for groups of few rows (decoding): bound by
// the weights' bytes, which are read once, straight into registers.
//
// A workgroup takes 32 weight rows of one expert; its four waves take scale
// blocks 4 u + w of K, so one row's 512 consecutive bytes are in flight over
// the workgroup, and kUnroll of those per wave.  Per block: two sums by MFMAs
// (weights on the rows, 16 tokens on the columns) from zero, then the scaled
// sum in fp32; the waves' sums are added in a fixed order through LDS.
// MFMA row m of weight tile i is weight row 8 (m / 4) + 4 i + m % 4, so a
// lane stores 8 consecutive outputs of its token.  Two rows for each of 8
// experts of 28672 x 4096: 159 us, 5.9 TB/s (the tiled kernel, which waits at
// two barriers a step, is for more).
#include "fp8_gemm_kernel.h"

namespace moe {
namespace {

constexpr int kRowsThreads = 256;
constexpr int kRowsBN = 32;

MOE_DEV i32x4 load16(__amdgpu_buffer_rsrc_t r, int voff, int soff) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

// 100 bytes: arguments past about 104 cost a launch 0.6 us of the host's time,
// a tenth of a small decoding call.
struct RowsArgs {
  const int32_t *split, *padded;
  const uint8_t* a;
  const float* a_s;
  const void* b;
  const float* b_s;
  int64_t b_stride, b_s_stride;
  void* c;
  int64_t ldc;
  int32_t* err;
  int N, K, M_cap;
};

template <int J, bool F32, bool WIDE>
__global__ __launch_bounds__(kRowsThreads) void fp8_rows_kernel(const RowsArgs g) {
  constexpr int kUnroll = J == 1 ? 4 : 2;
  __shared__ __attribute__((aligned(16))) f32x4 s_red[4][2 * J][kWave];
  const int e = blockIdx.y;
  bool bad;
  const int n_e = fp8_group_rows(g, e, false, bad);
  if (bad && blockIdx.x == 0 && threadIdx.x == 0) set_err(g.err, MOE_DEVERR_BAD_OFFSETS);
  if (n_e == 0) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, g4 = lane >> 4;
  const int64_t start = g.padded[e];
  const int n0 = blockIdx.x * kRowsBN;
  const int K = g.K, blocks = (K + kFp8Blk - 1) / kFp8Blk;
  const int rows_w = g.N - n0 < kRowsBN ? g.N - n0 : kRowsBN;
  const auto rw = fp8_rsrc(static_cast<const uint8_t*>(g.b) + e * g.b_stride + static_cast<int64_t>(n0) * K,
                           static_cast<uint32_t>(rows_w * K));
  const float* bs = g.b_s + e * g.b_s_stride + static_cast<int64_t>(n0 / kFp8Blk) * blocks;
  int voff_w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 8 * (l16 >> 2) + 4 * i + (l16 & 3);
    voff_w[i] = row < rows_w ? row * K + 32 * g4 : kFp8OutOfRange;
  }
  for (int r0 = 0; r0 < n_e; r0 += 16 * J) {
    const int rows_t = n_e - r0 < 16 * J ? n_e - r0 : 16 * J;
    const auto rt = fp8_rsrc(g.a + (start + r0) * K, static_cast<uint32_t>(rows_t * K));
    const float* as = g.a_s + start + r0;
    int voff_t[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
      voff_t[j] = 16 * j + l16 < rows_t ? (16 * j + l16) * K + 32 * g4 : kFp8OutOfRange;
    f32x4 acc[2][J];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int b0 = wave; b0 < blocks; b0 += 4 * kUnroll) {
      i32x4 w[kUnroll][2][2], t[kUnroll][J][2];   // raw codes
      float f[kUnroll][J], ws[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int b = b0 + 4 * u;
        const int k = b * kFp8Blk;
        const int soff = k < K ? k : 0;   // never past the records: they bound what is left of it
        // the lane's two chunks of the block (the last block may end inside)
        const bool ok0 = k + 32 * g4 < K, ok1 = k + 32 * g4 + 16 < K;
        auto load = [&](i32x4 (&d)[2], __amdgpu_buffer_rsrc_t r, int v) {
          d[0] = load16(r, ok0 ? v : kFp8OutOfRange, soff);
          d[1] = load16(r, ok1 && v != kFp8OutOfRange ? v + 16 : kFp8OutOfRange, soff);
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) load(w[u][i], rw, voff_w[i]);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          load(t[u][j], rt, voff_t[j]);
          f[u][j] = b < blocks && voff_t[j] != kFp8OutOfRange ? as[static_cast<int64_t>(b) * g.M_cap + 16 * j + l16] : 0.0f;
        }
        ws[u] = b < blocks ? bs[b] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        Fp8Frag<WIDE> ft[J];
#pragma unroll
        for (int j = 0; j < J; ++j) ft[j].set(t[u][j][0], t[u][j][1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          Fp8Frag<WIDE> fw;
          fw.set(w[u][i][0], w[u][i][1]);
#pragma unroll
          for (int j = 0; j < J; ++j) {
            const f32x4 p = fp8_block_mfma(fw, ft[j]);
            const float s = f[u][j] * ws[u];
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(p[r], s, acc[i][j][r]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j) s_red[wave][i * J + j][lane] = acc[i][j];
    __syncthreads();
    if (wave < J) {   // wave j adds and stores token tile j
      const int n = n0 + 8 * g4, tok = 16 * wave + l16;
      f32x4 v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[i] = s_red[0][i * J + wave][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) v[i] += s_red[w][i * J + wave][lane];
      }
      if (tok < rows_t && n < g.N) {
        const int64_t at = (start + r0 + tok) * g.ldc + n;
        if constexpr (F32) {
          f32x4* c = reinterpret_cast<f32x4*>(static_cast<float*>(g.c) + at);
          c[0] = v[0];
          c[1] = v[1];
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.c) + at) =
              uint4{pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]),
                    pack_bf16x2(v[1][0], v[1][1]), pack_bf16x2(v[1][2], v[1][3])};
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_fp8_rows(const Fp8Args& g, int tile_rows, bool f32, bool wide, hipStream_t s) {
  const dim3 grid((g.N + kRowsBN - 1) / kRowsBN, g.E);
  const RowsArgs r{g.split, g.padded, g.a, g.a_s, g.b, g.b_s, g.b_stride, g.b_s_stride, g.c, g.ldc, g.err,
                   g.N, g.K, static_cast<int>(g.M_cap)};
  auto go = [&](auto kernel) { kernel<<<grid, kRowsThreads, 0, s>>>(r); };
  if (tile_rows == 16) f32 ? go(fp8_rows_kernel<1, true, true>) : wide ? go(fp8_rows_kernel<1, false, true>) : go(fp8_rows_kernel<1, false, false>);
  else f32 ? go(fp8_rows_kernel<2, true, true>) : wide ? go(fp8_rows_kernel<2, false, true>) : go(fp8_rows_kernel<2, false, false>);
  return hipGetLastError();
}

}  // namespace moe
