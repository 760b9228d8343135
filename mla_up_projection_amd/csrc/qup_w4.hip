// Query up-projection of a few tokens with MXFP4 weights for gfx950: the
// decode form of the fused forward. Q = X deq(W)^T (+ bias), RoPE, bf16 or
// MXFP8 in BHSD.
//
// Bound by one pass over W: K N / 2 bytes of codes and K N / 32 of scales. The
// scaled convert expands an E2M1 pair times its E8M0 scale to bf16 exactly (one
// instruction for two weights), so the products go to the bf16 MFMA, 16
// tokens by 16 weight rows by 32 of K, with nothing left to scale afterwards.
//
// A lane holds 32 consecutive k of one weight row, one MX block: one 16-byte
// load and one scale byte. The MFMA's k slots are a sum's terms, so their order
// is free: in step j lane group c = lane / 16 supplies k = 32 c + 8 j .. + 7 of
// a 128-wide chunk for both operands.
#include <algorithm>

#include "device_common.h"
#include "internal_decode.h"

namespace mla {
namespace {

constexpr int W4_COLS = 32;   // weight rows (output columns) per workgroup: an MX block of the output
constexpr int W4_WAVES = 4;   // each takes every fourth 128-wide chunk of K
constexpr int W4_PITCH = 36;  // floats per token row of a wave's partial sums

// Two E2M1 codes (byte SEL of the dword) times scale, in bf16.
template <int SEL>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}

__device__ __forceinline__ bf16x8_t e2m1x8(uint32_t w, float scale) {
  const u32x4_t v = {e2m1_pair<0>(w, scale), e2m1_pair<1>(w, scale), e2m1_pair<2>(w, scale), e2m1_pair<3>(w, scale)};
  return __builtin_bit_cast(bf16x8_t, v);
}

// MT tiles of 16 tokens, CB chunks loaded before the first product.
template <int MT, int CB>
__global__ __launch_bounds__(256) void qup_w4_kernel(W4Params p) {
  __shared__ float red[W4_WAVES][MT * 16][W4_PITCH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, c4 = lane >> 4;
  const int n0 = blockIdx.x * W4_COLS;
  const int chunks = (p.K + 127) / 128;
  for (int64_t t0 = (int64_t)blockIdx.y * (MT * 16); t0 < p.T; t0 += (int64_t)gridDim.y * (MT * 16)) {
    f32x4_t acc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = f32x4_t{0, 0, 0, 0};
    uint32_t bad[2] = {0, 0};  // a scale byte of 0xFF: the weight row has a NaN block
    for (int c0 = wave; c0 < chunks; c0 += W4_WAVES * CB) {
      u32x4_t w[CB][2], x[CB][MT][4];
      uint32_t s[CB][2];
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const int k = (c0 + W4_WAVES * b) * 128 + 32 * c4;
        const bool live = k < p.K;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int64_t row = n0 + 16 * n + l16;
          w[b][n] = u32x4_t{0, 0, 0, 0};
          s[b][n] = 127;
          if (live) {
            w[b][n] = *reinterpret_cast<const u32x4_t*>(p.w + row * (p.K / 2) + k / 2);
            s[b][n] = p.ws[row * (p.K / 32) + k / 32];
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int64_t t = t0 + 16 * m + l16;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[b][m][j] = u32x4_t{0, 0, 0, 0};
            if (live && t < p.T) x[b][m][j] = *reinterpret_cast<const u32x4_t*>(p.x + t * p.K + k + 8 * j);
          }
        }
      }
#pragma unroll
      for (int b = 0; b < CB; ++b)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          bad[n] |= s[b][n] == 0xFF;
          const float scale = __uint_as_float(s[b][n] ? s[b][n] << 23 : 0x00400000u);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8_t wv = e2m1x8(w[b][n][j], scale);
#pragma unroll
            for (int m = 0; m < MT; ++m)
              acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x[b][m][j]), wv,
                                                                  acc[m][n], 0, 0, 0);
          }
        }
    }
    __syncthreads();  // the previous tokens' partial sums are read
    // acc[m][n][i]: token 16 m + 4 c4 + i, weight row 16 n + l16
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      bad[n] |= (uint32_t)__shfl_xor((int)bad[n], 16);
      bad[n] |= (uint32_t)__shfl_xor((int)bad[n], 32);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[wave][16 * m + 4 * c4 + i][16 * n + l16] = bad[n] ? __builtin_nanf("") : acc[m][n][i];
    }
    __syncthreads();
    // Four consecutive threads own a token's 32 columns, eight each.
    const int h = n0 / p.D, d_tile = n0 - h * p.D;
    const TokenMap tm{p.fmt, p.B, p.S, p.cu, p.nseq};
    for (int i = threadIdx.x; i < MT * 16 * 4; i += 256) {
      const int tl = i >> 2, g = i & 3;
      const int64_t t = t0 + tl;
      const bool live = t < p.T;
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0;
#pragma unroll
      for (int w = 0; w < W4_WAVES; ++w)
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
          const f32x4_t r = *reinterpret_cast<const f32x4_t*>(&red[w][tl][8 * g + k]);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[k + q] += r[q];
        }
      int pos = 0, bb = 0, ss = 0;
      if (live) {
        token_coords(tm, t, pos, bb, ss);
        if (p.positions) pos = p.positions[t];
      }
      const int d0 = d_tile + 8 * g;
      if (p.bias)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += bf16_bits_to_f32(p.bias[n0 + 8 * g + k]);
#pragma unroll
      for (int k = 0; k < 8; k += 2)
        if (d0 + k >= p.d_nope && live) {
          const bool ok = pos >= 0 && pos < p.rope_rows;
          const int64_t ti = (int64_t)(ok ? pos : 0) * p.rope_pairs + (d0 + k - p.d_nope) / 2;
          const float cs = ok ? p.cos[ti] : __builtin_nanf(""), sn = ok ? p.sin[ti] : __builtin_nanf("");
          const float a = v[k], b = v[k + 1];
          v[k] = a * cs - b * sn;
          v[k + 1] = a * sn + b * cs;
        }
      const int64_t o = (((int64_t)bb * p.H + h) * p.S + ss) * p.D + d0;
      if (!p.out_mx) {
        if (live)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + o) =
              make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      } else {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) m = max(m, abs_bits(v[k]));
        m = max(m, (uint32_t)__shfl_xor((int)m, 1));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2));
        uint32_t c0 = 0x7F7F7F7Fu, c1 = 0x7F7F7F7Fu, sc = 0xFF;
        if (m < 0x7F800000u) {
          const int E = mx_block_exp(m);
          c0 = e4m3_pack4(v[0], v[1], v[2], v[3], E);
          c1 = e4m3_pack4(v[4], v[5], v[6], v[7], E);
          sc = (uint32_t)(E + 127);
        }
        if (live) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + o) = make_uint2(c0, c1);
          if (g == 0) p.out_scales[o / 32] = (uint8_t)sc;
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_qup_w4(const W4Params& p, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  const unsigned nx = (unsigned)(p.N / W4_COLS);
  const int mt = p.T <= 16 ? 1 : p.T <= 32 ? 2 : 4;
  const int64_t blocks = (p.T + 16 * mt - 1) / (16 * mt);
  const dim3 grid(nx, (unsigned)std::min<int64_t>(blocks, 4096));  // the kernel strides over the rest
  if (mt == 1) hipLaunchKernelGGL((qup_w4_kernel<1, 3>), grid, dim3(256), 0, stream, p);
  else if (mt == 2) hipLaunchKernelGGL((qup_w4_kernel<2, 2>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((qup_w4_kernel<4, 1>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace mla
