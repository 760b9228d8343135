// MXFP4 quantization of a row-major matrix along its rows (OCP Microscaling
// Formats v1.0: E2M1 elements, one E8M0 scale per 32): weights of
// mla_qup_fwd_w4, laid out once. HBM-bound: reads 2 or 4 bytes an element and
// writes half a byte (24576 x 1536 bf16: 32 us, 3.0 TB/s; done once per weight).
// Four consecutive lanes own a block, eight elements each.
#include "device_common.h"
#include "internal_decode.h"

namespace mla {
namespace {

// E2M1 code of x * 2^-E, round to nearest even, saturating: the magnitudes are
// 0, .5, 1, 1.5, 2, 3, 4, 6 for codes 0..7, so the code counts the rounding
// borders .25, .75, 1.25, 1.75, 2.5, 3.5, 5 passed. A tie goes to the even code:
// the borders below an odd code (.25, 1.25, 2.5, 5) have to be passed, the
// others are passed when met. Comparing |x| against border * 2^E, which is
// exact, avoids scaling x.
__device__ __forceinline__ uint32_t e2m1_code(float x, float unit) {
  const float a = __uint_as_float(abs_bits(x));
  const uint32_t code = (a > 0.25f * unit) + (a >= 0.75f * unit) + (a > 1.25f * unit) + (a >= 1.75f * unit) +
                        (a > 2.5f * unit) + (a >= 3.5f * unit) + (a > 5.0f * unit);
  return code | (__float_as_uint(x) >> 31 << 3);
}

template <bool FP32>
__global__ __launch_bounds__(256) void mxfp4_quant_kernel(const void* __restrict__ x, int64_t groups, int64_t gpr,
                                                          int64_t ld, uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  constexpr int EB = FP32 ? 4 : 2;
  for (int64_t g0 = (int64_t)blockIdx.x * 256; g0 < groups; g0 += (int64_t)gridDim.x * 256) {
    const int64_t g = g0 + threadIdx.x;
    const int64_t gl = g < groups ? g : groups - 1;  // recomputes a valid group; stored only if live
    const int64_t row = gl / gpr;
    const u32x4_t* src = reinterpret_cast<const u32x4_t*>(static_cast<const uint8_t*>(x) + (row * ld + (gl - row * gpr) * 8) * EB);
    u32x4_t raw[2];
    raw[0] = src[0];
    if (FP32) raw[1] = src[1];
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (FP32) {
        v[i] = __uint_as_float(raw[0][i]);
        v[4 + i] = __uint_as_float(raw[1][i]);
      } else {
        v[2 * i] = bf16_bits_to_f32(raw[0][i] & 0xFFFFu);
        v[2 * i + 1] = bf16_bits_to_f32(raw[0][i] >> 16);
      }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
    m = max(m, (uint32_t)__shfl_xor((int)m, 1));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2));
    uint32_t c = 0x77777777u, sc = 0xFF;
    if (m < 0x7F800000u) {
      const int E = max((int)(m >> 23) - 127 - 2, -127);
      const float unit = __uint_as_float(E > -127 ? (uint32_t)(E + 127) << 23 : 0x00400000u);
      c = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) c |= e2m1_code(v[i], unit) << (4 * i);
      sc = (uint32_t)(E + 127);
    }
    if (g < groups) {
      *reinterpret_cast<uint32_t*>(codes + g * 4) = c;
      if ((g & 3) == 0) scales[g >> 2] = (uint8_t)sc;
    }
  }
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, int x_fp32, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                                 uint8_t* scales, hipStream_t stream) {
  const int64_t gpr = cols / 8, groups = rows * gpr;
  // at most 2^20 workgroups, which stride over the rest
  const int64_t blocks = (groups + 255) / 256;
  const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)));
  if (x_fp32)
    hipLaunchKernelGGL(mxfp4_quant_kernel<true>, grid, dim3(256), 0, stream, x, groups, gpr, ld, codes, scales);
  else
    hipLaunchKernelGGL(mxfp4_quant_kernel<false>, grid, dim3(256), 0, stream, x, groups, gpr, ld, codes, scales);
  return hipGetLastError();
}

}  // namespace mla
