// Query up-projection in 8-bit integers for gfx950: Q[t, n] = xs[t] ws[n]
// sum_k X[t, k] W[n, k] (+ bias), RoPE, bf16 or MXFP8 in BHSD. Sums are exact in
// 32 bits. Many tokens go to the tiled kernel of the fused forward; the one here
// is for few, where reading W once (K N bytes) is what bounds it.
//
// A lane holds 32 consecutive k of one weight row in two 16-byte loads, so a
// wave reads whole 128-byte lines. The MFMA's k slots are a sum's terms and
// their order is free: in step j lane group c = lane / 16 supplies k = 32 c + 16
// j .. + 15 of a 128-wide chunk for both operands.
#include <algorithm>

#include "device_common.h"
#include "internal.h"
#include "internal_layer.h"
#include "qup_finish.h"

namespace mla {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// A workgroup makes MT tiles of 16 tokens by NT of 16 weight rows; its waves take
// the 128-wide chunks of K in turn and add up in LDS.
template <int MT, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void qup_i8_kernel(I8Params p) {
  constexpr int PITCH = 16 * NT + 4;
  __shared__ int red[WAVES][MT * 16][PITCH];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, c4 = lane >> 4;
  const int n0 = blockIdx.x * (16 * NT);
  const int chunks = (p.K + 127) / 128;
  for (int64_t t0 = (int64_t)blockIdx.y * (MT * 16); t0 < p.T; t0 += (int64_t)gridDim.y * (MT * 16)) {
    i32x4_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = i32x4_t{0, 0, 0, 0};
    const auto load = [&](i32x4_t(&w)[NT][2], i32x4_t(&x)[MT][2], int c) {
      const int k = c * 128 + 32 * c4;
      const bool in = k < p.K;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int64_t row = n0 + 16 * n + l16;
        const i32x4_t* src = reinterpret_cast<const i32x4_t*>(p.w + row * p.K + k);
        w[n][0] = w[n][1] = i32x4_t{0, 0, 0, 0};
        if (in && row < p.N) w[n][0] = src[0], w[n][1] = src[1];
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const i32x4_t* src = reinterpret_cast<const i32x4_t*>(p.x + min(t0 + 16 * m + l16, p.T - 1) * p.K + k);
        x[m][0] = x[m][1] = i32x4_t{0, 0, 0, 0};
        if (in) x[m][0] = src[0], x[m][1] = src[1];
      }
    };
    i32x4_t w[NT][2], x[MT][2];
    if (wave < chunks) load(w, x, wave);
    for (int c = wave; c < chunks; c += WAVES) {
      i32x4_t w2[NT][2], x2[MT][2];
      if (c + WAVES < chunks) load(w2, x2, c + WAVES);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[m][n] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[m][j], w[n][j], acc[m][n], 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int n = 0; n < NT; ++n) w[n][j] = w2[n][j];
#pragma unroll
        for (int m = 0; m < MT; ++m) x[m][j] = x2[m][j];
      }
    }
    __syncthreads();  // the previous tokens' sums are read
    // acc[m][n][i]: token 16 m + 4 c4 + i, weight row 16 n + l16
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave][16 * m + 4 * c4 + i][16 * n + l16] = acc[m][n][i];
    __syncthreads();
    // Four consecutive threads own 32 columns (an MX block of the output, all of
    // one head) of a token, eight each.
    const TokenMap tm{p.fmt, p.B, p.S, p.cu, p.nseq};
    for (int i = threadIdx.x; i < MT * 16 * 2 * NT; i += 64 * WAVES) {
      const int tl = i / (2 * NT), g = i - tl * (2 * NT);  // token, group of eight columns
      const int64_t t = t0 + tl;
      const int n = n0 + 8 * g;
      const bool live = t < p.T && n < p.N;
      float v[8];
      const float xs = live ? p.xs[t] : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        int s = 0;
#pragma unroll
        for (int q = 0; q < WAVES; ++q) s += red[q][tl][8 * g + k];
        v[k] = live ? (float)s * xs * p.ws[n + k] : 0.0f;
      }
      finish8(p, tm, t, n, live, (g & 3) == 0, v);
    }
  }
}

template <int MT, int NT, int WAVES>
void launch_few(const I8Params& p, hipStream_t stream) {
  const int64_t blocks = (p.T + 16 * MT - 1) / (16 * MT);
  const dim3 grid((unsigned)((p.N + 16 * NT - 1) / (16 * NT)), (unsigned)std::min<int64_t>(blocks, 4096));
  hipLaunchKernelGGL((qup_i8_kernel<MT, NT, WAVES>), grid, dim3(64 * WAVES), 0, stream, p);
}

}  // namespace

hipError_t launch_qup_i8(const I8Params& p, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  if (p.T > 64) {
    FwdParams f{};
    f.x = p.x;
    f.w = p.w;
    f.x_row_scales = p.xs;
    f.w_row_scales = p.ws;
    f.positions = p.positions;
    f.bias = p.bias;
    f.T = p.T;
    f.K = p.K;
    f.N = p.N;
    f.H = p.H;
    f.D = p.D;
    f.d_nope = p.d_nope;
    f.d_rope = p.d_rope;
    f.fmt = p.fmt;
    f.B = p.B;
    f.S = p.S;
    f.cu = p.cu;
    f.nseq = p.nseq;
    f.cos = p.cos;
    f.sin = p.sin;
    f.rope_rows = p.rope_rows;
    f.rope_pairs = p.rope_pairs;
    f.out_mx = p.out_mx;
    f.out = p.out;
    f.out_scales = p.out_scales;
    f.k_splits = 1;
    return launch_qup_fwd_i8(f, stream);
  }
  if (p.T <= 16) launch_few<1, 2, 4>(p, stream);
  else if (p.T <= 32) launch_few<2, 2, 4>(p, stream);
  else launch_few<4, 2, 4>(p, stream);
  return hipGetLastError();
}

}  // namespace mla
