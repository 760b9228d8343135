// Host-side argument checks shared by the entry points of the C ABI (api.hip,
// api_decode.hip). Nothing here dereferences a device pointer or makes a HIP
// call.
#pragma once

#include <stdint.h>

#include <vector>

#include "internal.h"

namespace {

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

Range rng(const void* p, size_t bytes) {
  uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + bytes};
}

// Outputs must be disjoint from inputs and from each other.
bool overlaps(const std::vector<Range>& outs, const std::vector<Range>& ins) {
  for (size_t i = 0; i < outs.size(); ++i) {
    const Range& o = outs[i];
    if (o.hi <= o.lo) continue;
    for (const Range& r : ins)
      if (r.hi > r.lo && o.lo < r.hi && r.lo < o.hi) return true;
    for (size_t j = i + 1; j < outs.size(); ++j) {
      const Range& r = outs[j];
      if (r.hi > r.lo && o.lo < r.hi && r.lo < o.hi) return true;
    }
  }
  return false;
}

mla_status launched(hipError_t e) { return e == hipSuccess ? MLA_OK : MLA_EDEVICE; }

// Shape checks common to forward and backward.
mla_status check_head_shape(int32_t K, int32_t H, int32_t d_nope, int32_t d_rope) {
  if (K <= 0 || K % 32 != 0 || H <= 0) return MLA_EINVAL;
  if (d_nope < 0 || d_rope < 0 || (d_nope & 1) || (d_rope & 1)) return MLA_EINVAL;
  int64_t D = (int64_t)d_nope + d_rope;
  if (D <= 0 || D % 32 != 0) return MLA_EINVAL;
  if ((int64_t)H * D > (int64_t)INT32_MAX / 2) return MLA_EINVAL;
  return MLA_OK;
}

// Token format checks; max_pos receives the largest possible position.
mla_status check_tokens(const mla_tokens& tk, int64_t* max_pos) {
  if (tk.T < 0 || tk.T > (int64_t)INT32_MAX) return MLA_EINVAL;
  if (tk.fmt == MLA_FMT_BSHD || tk.fmt == MLA_FMT_SBHD) {
    if (tk.B < 1 || tk.S < 1) return MLA_EINVAL;
    if ((int64_t)tk.B * tk.S != tk.T) return MLA_EINVAL;
    *max_pos = tk.S - 1;
    return MLA_OK;
  }
  if (tk.fmt == MLA_FMT_THD) {
    if (tk.nseq < 1 || tk.max_seqlen < 1) return MLA_EINVAL;
    if (tk.T > 0 && tk.cu_seqlens == nullptr) return MLA_EINVAL;
    if (!aligned(tk.cu_seqlens, 4)) return MLA_EINVAL;
    *max_pos = tk.max_seqlen - 1;
    return MLA_OK;
  }
  return MLA_EINVAL;
}

// The cos/sin width guard: the table must hold d_rope/2 pairs per row and a
// row for every position (the out-of-bounds cos/sin read that the Megatron
// page's Problem section names as a NaN source).
mla_status check_rope(const mla_rope& r, int32_t d_rope, int64_t max_pos) {
  if (d_rope == 0) return MLA_OK;
  if (r.cos == nullptr || r.sin == nullptr) return MLA_EINVAL;
  // the inverse-RoPE kernel reads four table pairs with one 16-byte load and
  // the forward epilogue two with one 8-byte load (when pairs % 4 == 0)
  if (!aligned(r.cos, 16) || !aligned(r.sin, 16)) return MLA_EINVAL;
  if (r.pairs < d_rope / 2) return MLA_EROPE_TABLE;
  if ((int64_t)r.rows < max_pos + 1 || r.rows < 1) return MLA_EROPE_TABLE;
  return MLA_OK;
}

size_t rope_bytes(const mla_rope& r, int32_t d_rope) {
  return d_rope ? (size_t)r.rows * (size_t)r.pairs * sizeof(float) : 0;
}

void fill_token_map(const mla_tokens& tk, int& fmt, int& B, int& S, const int32_t*& cu, int& nseq) {
  fmt = tk.fmt;
  if (tk.fmt == MLA_FMT_THD) {
    B = 1;
    S = (int)tk.T;
    cu = tk.cu_seqlens;
    nseq = tk.nseq;
  } else {
    B = tk.B;
    S = tk.S;
    cu = nullptr;
    nseq = 0;
  }
}

}  // namespace
