// Internal launch interface of the decode-side operators (paged cache,
// attention of drafted tokens, 4-bit up-projection). Every launcher assumes
// that api_decode.hip has validated its arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mla_qup.h"

namespace mla {

// The pool as the kernels see it.
struct PoolParams {
  int num_pages, page_size, max_seqs, max_pages;
  int32_t* refs;
  int32_t* table;
  int32_t* lens;
  int32_t* held;
  int nbuf;
  uint8_t* buf[4];
  int64_t page_bytes[4];
};

// Workspace of the page operators, in int32 words: a header of PW_HEAD words,
// then two lists of num_pages words.
//   reserve: word 0 unused; triples (src, dst, rows) of entry i at PW_PAIRS + 3 i;
//            list A: the pages taken, in order.
//   compact: word 0 = pages that move, word 1 = pages in use; list A: source
//            pages, list B: target of each source page, indexed by page.
constexpr int PW_PAIRS = 16;
constexpr int PW_HEAD = PW_PAIRS + 3 * MLA_MAX_SEQS + 16;
inline size_t pages_workspace_bytes(int num_pages) { return (size_t)4 * (PW_HEAD + 2 * (size_t)num_pages); }

hipError_t launch_pages_copy(const PoolParams& src, const PoolParams& dst, bool same, const int32_t* src_ids,
                             const int32_t* dst_ids, int n, hipStream_t stream);
hipError_t launch_pages_reserve(const PoolParams& p, const int32_t* seqs, const int32_t* new_tokens, int n,
                                int32_t* status, int32_t* ws, hipStream_t stream);
hipError_t launch_pages_fork(const PoolParams& p, const int32_t* src, const int32_t* dst, int n, hipStream_t stream);
hipError_t launch_pages_free(const PoolParams& p, const int32_t* seqs, const int32_t* keep, int n, hipStream_t stream);
hipError_t launch_pages_compact(const PoolParams& p, int32_t* used, int32_t* ws, hipStream_t stream);
hipError_t launch_draft_accept(const PoolParams& p, const int32_t* seqs, const int32_t* path, const int32_t* n_acc,
                               int n, int max_path, hipStream_t stream);

struct KvPagedParams {
  const uint16_t* kv;
  const uint16_t* pe;
  int64_t T;
  int H, d_nope, d_rope, d_v;
  const int32_t* seqs;
  const int32_t* cu;
  int nseq, max_q;
  const int32_t* positions;
  const float* cos;
  const float* sin;
  int rope_rows, rope_pairs;
  int mx;
  PoolParams pool;
};
hipError_t launch_kv_rope_paged(const KvPagedParams& p, hipStream_t stream);

struct W4Params {
  const uint16_t* x;
  const uint8_t* w;
  const uint8_t* ws;
  const uint16_t* bias;
  int64_t T;
  int K, N, H, D, d_nope, d_rope;
  int fmt, B, S;
  const int32_t* cu;
  int nseq;
  const int32_t* positions;
  const float* cos;
  const float* sin;
  int rope_rows, rope_pairs;
  int out_mx;
  void* out;
  uint8_t* out_scales;
};
hipError_t launch_qup_w4(const W4Params& p, hipStream_t stream);

hipError_t launch_mxfp4_quantize(const void* x, int x_fp32, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                                 uint8_t* scales, hipStream_t stream);

// How mla_tree_attention splits a call: row tiles of 32 * waves query rows
// (row = draft * group + head of the group) and chunks of `chunk` cache rows.
struct AttnPlan {
  int waves;       // waves of a workgroup, 32 query rows each
  int row_tiles;   // per (sequence, key head)
  int chunk;       // cache rows per workgroup, a multiple of the tile
  int chunks;      // per sequence, at most
  int groups;      // > 0: the even plan of the widest shape, with at most that many workgroups (chunk: rows whose
                   // pages the kernel lists at a time)
  size_t part_o, part_ml, sums, total;  // workspace: offsets of the partial outputs, of (max, sum) and of the even
                                        // plan's sums; bytes in all
};

// Longest sequence that the attention takes: positions of the tiles that it asks
// for ahead and the next part of a long one (65536 rows) stay within 31 bits.
constexpr int32_t kLongestSeq = INT32_MAX - (1 << 17);

struct AttnParams {
  const uint16_t* q;
  int64_t q_t, q_h;
  uint16_t* out;
  int64_t o_t, o_h;
  float* lse;
  int64_t T;
  int H, H_kv, group, d_k, d_v;
  float scale_log2;  // scale * log2(e)
  const int32_t* seqs;
  const int32_t* cu;
  int nseq, max_q, max_len;
  const uint32_t* mask;
  int mask_words;
  int mx;
  PoolParams pool;
  uint32_t page_magic;  // ceil(2^32 / page_size): quotient of small rows by a high product
  float* part_o;
  float* part_ml;
  int64_t* sums;  // even plan: how units are shared (each, more), quantum, units before each sequence
  AttnPlan plan;
};
bool attn_shape_supported(int d_k, int d_v, bool shared);
AttnPlan plan_attn(int nseq, int H, int H_kv, int d_v, int max_q, int max_len, int page_size);
hipError_t launch_tree_attn(const AttnParams& p, hipStream_t stream);

}  // namespace mla
