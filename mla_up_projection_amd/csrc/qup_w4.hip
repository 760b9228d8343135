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
#include "qup_finish.h"

namespace mla {
namespace {

// Two E2M1 codes (byte SEL of the dword) times scale, in bf16.
template <int SEL>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}

__device__ __forceinline__ bf16x8_t e2m1x8(uint32_t w, float scale) {
  const u32x4_t v = {e2m1_pair<0>(w, scale), e2m1_pair<1>(w, scale), e2m1_pair<2>(w, scale), e2m1_pair<3>(w, scale)};
  return __builtin_bit_cast(bf16x8_t, v);
}

// 16 bytes per lane to LDS bytes [lds_addr + 16 lane, + 16).
__device__ __forceinline__ void dma16_any(const void* p, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds_addr)), "v"(p)
               : "memory", "m0");
}

// A workgroup makes MT tiles of 16 tokens by NT of 16 weight rows; its waves take
// the 128-wide chunks of K in turn and add up in LDS. X comes by
// direct loads into LDS, whole rows at a time: loaded as fragments (16 rows by 64
// bytes to an instruction) 16 tokens of the 128-head shape (K 1536) took 11.9 us,
// 32 took 16.5 and 52 took 27 (one weight tile pair); so they take 9.4, 11.4 and
// 22. One token takes 8.8 either way: 2.3 TB/s of weights.
template <int MT, int NT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void qup_w4_kernel(W4Params p) {
  constexpr int PITCH = 16 * NT + 4;   // floats per token row of a wave's partial sums
  constexpr int X_LDS = MT * 16 * 256;  // a wave's chunk of X
  constexpr int LDS = WAVES * std::max(X_LDS, MT * 16 * PITCH * 4);
  __shared__ __attribute__((aligned(1024))) uint8_t lds[LDS];
  float(*red)[MT * 16][PITCH] = reinterpret_cast<float(*)[MT * 16][PITCH]>(lds);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, c4 = lane >> 4;
  uint8_t* xs = lds + wave * X_LDS;
  const int n0 = blockIdx.x * (16 * NT);
  const int chunks = (p.K + 127) / 128;
  for (int64_t t0 = (int64_t)blockIdx.y * (MT * 16); t0 < p.T; t0 += (int64_t)gridDim.y * (MT * 16)) {
    f32x4_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[m][n] = f32x4_t{0, 0, 0, 0};
    __syncthreads();  // the previous tokens' partial sums are read
    for (int c = wave; c < chunks; c += WAVES) {
      u32x4_t w[NT], x[MT][4];
      uint32_t s[NT];
      const int k = c * 128 + 32 * c4;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int64_t row = n0 + 16 * n + l16;
        w[n] = u32x4_t{0, 0, 0, 0};
        s[n] = 127;
        if (k < p.K && row < p.N) {
          w[n] = *reinterpret_cast<const u32x4_t*>(p.w + row * (p.K / 2) + k / 2);
          s[n] = p.ws[row * (p.K / 32) + k / 32];
        }
      }
      // X: rows of 256 bytes, four to an instruction; 16-byte piece q of row r at
      // place q ^ (r & 15), so that the 16 rows of a fragment meet no bank twice.
      // Rows behind T repeat the last (their products are not stored), pieces
      // behind K are zeros.
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the previous chunk is read
#pragma unroll
      for (int g = 0; g < MT * 4; ++g) {
        const int r = 4 * g + c4, kx = c * 128 + 8 * (l16 ^ (r & 15));
        const int64_t t = min(t0 + r, p.T - 1);
        if (kx < p.K) dma16_any(p.x + t * p.K + kx, lds_u32(xs) + g * 1024);
        else *reinterpret_cast<u32x4_t*>(xs + g * 1024 + lane * 16) = u32x4_t{0, 0, 0, 0};
      }
      vm_wait<0>();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[m][j] = *reinterpret_cast<const u32x4_t*>(xs + (16 * m + l16) * 256 + (((4 * c4 + j) ^ l16) << 4));
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // the convert reads the scale's exponent field, 0 meaning 2^-127 and
        // 255 NaN, as E8M0 does
        const float scale = __uint_as_float(s[n] << 23);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8_t wv = e2m1x8(w[n][j], scale);
#pragma unroll
          for (int m = 0; m < MT; ++m)
            acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, x[m][j]), wv, acc[m][n], 0, 0, 0);
        }
      }
    }
    __syncthreads();  // the chunks of X are read
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
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0;
#pragma unroll
      for (int w = 0; w < WAVES; ++w)
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
          const f32x4_t r = *reinterpret_cast<const f32x4_t*>(&red[w][tl][8 * g + k]);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[k + q] += r[q];
        }
      finish8(p, tm, t, n, live, (g & 3) == 0, v);
    }
  }
}

template <int MT, int NT, int WAVES>
void launch_w4(const W4Params& p, hipStream_t stream) {
  const int64_t blocks = (p.T + 16 * MT - 1) / (16 * MT);  // the kernel strides over those past the grid
  const dim3 grid((unsigned)((p.N + 16 * NT - 1) / (16 * NT)), (unsigned)std::min<int64_t>(blocks, 4096));
  hipLaunchKernelGGL((qup_w4_kernel<MT, NT, WAVES>), grid, dim3(64 * WAVES), 0, stream, p);
}

}  // namespace

hipError_t launch_qup_w4(const W4Params& p, hipStream_t stream) {
  if (p.T == 0) return hipSuccess;
  // X is read once per workgroup, so many tokens want many weight rows, as long
  // as a workgroup per CU is left: 52 tokens of 128 heads (N 24576) take 16.6 us
  // with NT = 4 and 21.9 with 2, 64 tokens of 32 heads (N 6144) 13.5 and 10.7.
  // Eight waves share the chunks of K where workgroups are few and K has more
  // than four: one token, K 7168, N 12288 29.6 -> 22.3 us, 16 tokens, K 4096, 16
  // heads of 192 13.5 -> 10.0; but N 24576, K 1536 8.9 -> 11.1, K 512 3.7 -> 4.1.
  const bool few = p.N < 64 * 256, eight = few && p.K > 512;
  if (p.T <= 16) eight ? launch_w4<1, 2, 8>(p, stream) : launch_w4<1, 2, 4>(p, stream);
  else if (p.T <= 32) eight ? launch_w4<2, 2, 8>(p, stream) : launch_w4<2, 2, 4>(p, stream);
  else if (!few) launch_w4<4, 4, 4>(p, stream);
  else eight ? launch_w4<4, 2, 8>(p, stream) : launch_w4<4, 2, 4>(p, stream);
  return hipGetLastError();
}

}  // namespace mla
