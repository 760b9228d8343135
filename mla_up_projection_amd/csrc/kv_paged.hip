// Key and value rows of new tokens into the pages of the decode cache, for
// gfx950: mla_kv_rope with a paged destination. Per token and head
//   key = [k_nope | rotate(k_pe)], value = v,
// bf16 or MXFP8 (one E8M0 scale per 32 elements, as mla_kv_rope). Each element
// is read once and written once, so HBM (or, for a handful of tokens, the
// launch) bounds it.
//
// A workgroup takes `tok` tokens x up to PG_HEADS heads: it finds the tokens'
// sequences and pages and rotates their shared k_pe slices once into LDS, then
// each thread takes one block of 32 elements (MXFP8) or 8 elements (bf16) of a
// (token, head) row of [key | value]. 1890 tokens x 128 heads x (192 | 128):
// MXFP8 54 us (204 MB, 3.8 TB/s; 79 with 8 elements to a thread: four times the
// address arithmetic for a quarter of a scale), bf16 73 us (279 MB, 3.8 TB/s; 83
// with 32, whose stores are 64 bytes apart).
#include <algorithm>

#include "device_common.h"
#include "internal_decode.h"

namespace mla {
namespace {

constexpr int PG_TOK = 16;        // tokens per workgroup, at most
constexpr int PG_HEADS = 64;      // heads per workgroup, at most
constexpr int PG_MAX_ROPE = 256;  // widest rope slice
constexpr int PG_PITCH = PG_MAX_ROPE + 4;

template <int EPT>
__global__ __launch_bounds__(256) void kv_paged_kernel(KvPagedParams p, int tok) {
  constexpr int NG = EPT / 8;
  __shared__ float rot[PG_TOK * PG_PITCH];
  __shared__ int64_t drow[PG_TOK];  // cache row page * page_size + r, or -1
  __shared__ int spos[PG_TOK], sseq[PG_TOK];  // position, index in seqs
  const int Dk = p.d_nope + p.d_rope;
  const int row_in = p.d_nope + p.d_v;
  const int upr = (Dk + p.d_v) / EPT;
  const int hgroups = (p.H + PG_HEADS - 1) / PG_HEADS;
  const int64_t chunks = (p.T + tok - 1) / tok * hgroups;
  const int tid = threadIdx.x;
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int ck = (int)(c / hgroups);
    const int h0 = (int)(c - (int64_t)ck * hgroups) * PG_HEADS;
    const int nh = min(PG_HEADS, p.H - h0);
    const int64_t t0 = (int64_t)ck * tok;
    const int nt = (int)min((int64_t)tok, p.T - t0);
    __syncthreads();  // the previous chunk's readers are done
    if (tid < nt) {
      const int t = (int)t0 + tid;
      int64_t row = -1;
      int pos = -1, lo = 0;
      if (p.nseq > 0 && t >= p.cu[0] && t < p.cu[p.nseq]) {
        int hi = p.nseq;  // largest j with cu[j] <= t
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (p.cu[mid] <= t) lo = mid; else hi = mid;
        }
        const int seq = p.seqs[lo];
        if (seq >= 0 && seq < p.pool.max_seqs) {
          const int64_t at = (int64_t)p.pool.lens[seq] + (t - p.cu[lo]);
          const int64_t k = at / p.pool.page_size;
          pos = (int)min(at, (int64_t)0x7FFFFFFF);
          if (at >= 0 && k < min(p.pool.held[seq], p.pool.max_pages) && t - p.cu[lo] < p.max_q) {
            const int page = p.pool.table[(int64_t)seq * p.pool.max_pages + k];
            if (page >= 0 && page < p.pool.num_pages)
              row = (int64_t)page * p.pool.page_size + (at - k * p.pool.page_size);
          }
        }
        if (p.positions) pos = p.positions[t];
      }
      drow[tid] = row;
      spos[tid] = pos;
      sseq[tid] = lo;
    }
    __syncthreads();
    // tokens of a sequence that stands in seqs before are dropped (a race of
    // threads that store the same -1)
    for (int tl = 0; tl < nt; ++tl)
      for (int j = tid; j < sseq[tl]; j += 256)
        if (p.seqs[j] == p.seqs[sseq[tl]]) drow[tl] = -1;
    const int pairs = p.d_rope / 2;
    for (int i = tid; i < nt * pairs; i += 256) {
      const int tl = i / pairs, k = i - tl * pairs;
      const uint32_t ab = *reinterpret_cast<const uint32_t*>(p.pe + (t0 + tl) * p.d_rope + 2 * k);
      const float a = bf16_bits_to_f32(ab & 0xFFFFu), b = bf16_bits_to_f32(ab >> 16);
      const int pos = spos[tl];
      const bool ok = pos >= 0 && pos < p.rope_rows;
      const float nan = __builtin_nanf("");
      const int64_t ti = (int64_t)(ok ? pos : 0) * p.rope_pairs + k;
      const float cs = ok ? p.cos[ti] : nan, sn = ok ? p.sin[ti] : nan;
      rot[tl * PG_PITCH + 2 * k] = a * cs - b * sn;
      rot[tl * PG_PITCH + 2 * k + 1] = a * sn + b * cs;
    }
    __syncthreads();  // rot and drow are complete
    const int n = nh * nt * upr;
    for (int i = tid; i < n; i += 256) {
      const int tl = i / (nh * upr);
      const int64_t dr = drow[tl];
      if (dr < 0) continue;
      const int rem = i - tl * (nh * upr);
      const int h = h0 + rem / upr;
      const int e0 = (rem - (h - h0) * upr) * EPT;
      const bool is_key = e0 < Dk;
      const int d0 = is_key ? e0 : e0 - Dk;
      const uint16_t* src = p.kv + ((t0 + tl) * p.H + h) * row_in + (is_key ? 0 : p.d_nope);
      uint4 raw[NG];
#pragma unroll
      for (int q = 0; q < NG; ++q)
        if (!(is_key && d0 + 8 * q >= p.d_nope)) raw[q] = *reinterpret_cast<const uint4*>(src + d0 + 8 * q);
      float v[EPT];
#pragma unroll
      for (int q = 0; q < NG; ++q) {
        const int d = d0 + 8 * q;
        if (is_key && d >= p.d_nope) {
          const float* r = rot + tl * PG_PITCH + (d - p.d_nope);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[8 * q + k] = r[k];
        } else {
          const uint32_t w[4] = {raw[q].x, raw[q].y, raw[q].z, raw[q].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[8 * q + 2 * k] = bf16_bits_to_f32(w[k] & 0xFFFFu);
            v[8 * q + 2 * k + 1] = bf16_bits_to_f32(w[k] >> 16);
          }
        }
      }
      const int D = is_key ? Dk : p.d_v;
      const int64_t orow = dr * p.H + h;
      if (!p.mx) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(p.pool.buf[is_key ? 0 : 1]) + orow * D + d0;
#pragma unroll
        for (int q = 0; q < NG; ++q)
          reinterpret_cast<uint4*>(dst)[q] =
              make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                         pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
      } else if (EPT == 32) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < EPT; ++k) m = max(m, abs_bits(v[k]));
        uint32_t code[8], sc;
        if (m >= 0x7F800000u) {
#pragma unroll
          for (int k = 0; k < 8; ++k) code[k] = 0x7F7F7F7Fu;
          sc = 0xFF;
        } else {
          const int E = mx_block_exp(m);
#pragma unroll
          for (int k = 0; k < 8; ++k) code[k] = e4m3_pack4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3], E);
          sc = (uint32_t)(E + 127);
        }
        uint8_t* dst = p.pool.buf[is_key ? 0 : 2] + orow * D + d0;
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(code[0], code[1], code[2], code[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(code[4], code[5], code[6], code[7]);
        p.pool.buf[is_key ? 1 : 3][orow * (D / 32) + d0 / 32] = (uint8_t)sc;
      }
    }
  }
}

}  // namespace

hipError_t launch_kv_rope_paged(const KvPagedParams& p, hipStream_t stream) {
  if (p.T == 0 || p.nseq == 0) return hipSuccess;
  const int upr = (p.d_nope + p.d_rope + p.d_v) / (p.mx ? 32 : 8);
  const int hgroups = (p.H + PG_HEADS - 1) / PG_HEADS;
  // about 512 units for a workgroup's 256 threads, fewer tokens when there are
  // not enough to give every CU a workgroup
  int64_t tok = std::max<int64_t>(1, 512 / ((int64_t)std::min(p.H, PG_HEADS) * upr));
  tok = std::min<int64_t>(std::min<int64_t>(tok, PG_TOK), std::max<int64_t>(1, p.T * hgroups / 256));
  const int64_t chunks = (p.T + tok - 1) / tok * hgroups;
  const dim3 grid((unsigned)std::min<int64_t>(chunks, 65535));
  if (p.mx)
    hipLaunchKernelGGL(kv_paged_kernel<32>, grid, dim3(256), 0, stream, p, (int)tok);
  else
    hipLaunchKernelGGL(kv_paged_kernel<8>, grid, dim3(256), 0, stream, p, (int)tok);
  return hipGetLastError();
}

}  // namespace mla
