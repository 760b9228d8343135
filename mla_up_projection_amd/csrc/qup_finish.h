// The end of an up-projection of few tokens: bias, rotation, quantization and
// store of eight columns of a token.
#pragma once

#include "device_common.h"

namespace mla {

// What eight columns n .. n + 7 of token t need besides their sums. It can be loaded
// ahead of them.
struct Finish8 {
  int64_t o;       // the columns' place in the output
  int d0;          // and in their head
  float cs[4], sn[4], bias[8];
};
template <class P>
__device__ __forceinline__ Finish8 finish8_begin(const P& p, const TokenMap& tm, int64_t t, int n, bool live) {
  Finish8 f{};
  int pos = 0, bb = 0, ss = 0;
  const int h = n / p.D;
  f.d0 = n - h * p.D;
  if (live) {
    token_coords(tm, t, pos, bb, ss);
    if (p.positions) pos = p.positions[t];
    if (p.bias)
#pragma unroll
      for (int k = 0; k < 8; ++k) f.bias[k] = bf16_bits_to_f32(p.bias[n + k]);
#pragma unroll
    for (int k = 0; k < 8; k += 2)
      if (f.d0 + k >= p.d_nope) {
        const bool ok = pos >= 0 && pos < p.rope_rows;
        const int64_t ti = (int64_t)(ok ? pos : 0) * p.rope_pairs + (f.d0 + k - p.d_nope) / 2;
        f.cs[k / 2] = ok ? p.cos[ti] : __builtin_nanf("");
        f.sn[k / 2] = ok ? p.sin[ti] : __builtin_nanf("");
      }
  }
  f.o = (((int64_t)bb * p.H + h) * p.S + ss) * p.D + f.d0;
  return f;
}

// v: the columns' sums. Four consecutive lanes hold 32 columns of one head and come
// here together; `first` marks the one that stores their scale. live: there are such
// a token and column.
template <class P>
__device__ __forceinline__ void finish8_end(const P& p, const Finish8& f, bool live, bool first, float (&v)[8]) {
  if (live) {
    if (p.bias)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += f.bias[k];
#pragma unroll
    for (int k = 0; k < 8; k += 2)
      if (f.d0 + k >= p.d_nope) {
        const float cs = f.cs[k / 2], sn = f.sn[k / 2], a = v[k], b = v[k + 1];
        v[k] = a * cs - b * sn;
        v[k + 1] = a * sn + b * cs;
      }
  }
  const int64_t o = f.o;
  if (!p.out_mx) {
    if (live)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + o) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                     pack_bf16x2(v[6], v[7]));
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
      if (first) p.out_scales[o / 32] = (uint8_t)sc;
    }
  }
}

template <class P>
__device__ __forceinline__ void finish8(const P& p, const TokenMap& tm, int64_t t, int n, bool live, bool first,
                                        float (&v)[8]) {
  finish8_end(p, finish8_begin(p, tm, t, n, live), live, first, v);
}

}  // namespace mla
