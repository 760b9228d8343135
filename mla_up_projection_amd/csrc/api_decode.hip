// C ABI of the decode-side operators: host-side validation, the plan of the
// attention, then the launches. Argument meanings, layouts and error behaviour
// are stated in include/mla_qup.h. As in api.hip, validation dereferences no
// device pointer, so every error path runs without a GPU (the attention's plan
// asks for the device's compute units and takes 256 where there is none);
// nothing here allocates.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <cmath>

#include "api_checks.h"
#include "internal_decode.h"

namespace {

// The ranges of one call: outputs must be disjoint from inputs and from each
// other.
struct Ranges {
  Range in[16], out[16];
  int nin = 0, nout = 0;
  void input(const void* p, size_t bytes) {
    if (p && bytes) in[nin++] = rng(p, bytes);
  }
  void output(const void* p, size_t bytes) {
    if (p && bytes) out[nout++] = rng(p, bytes);
  }
  static bool meet(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }
  bool overlap() const {
    for (int i = 0; i < nout; ++i) {
      for (int j = 0; j < nin; ++j)
        if (meet(out[i], in[j])) return true;
      for (int j = i + 1; j < nout; ++j)
        if (meet(out[i], out[j])) return true;
    }
    return false;
  }
};

mla_status check_pool(const mla_pool* p) {
  if (p == nullptr) return MLA_EINVAL;
  if (p->num_pages < 1 || p->num_pages > MLA_MAX_PAGES || p->page_size < 1 || p->page_size > MLA_MAX_PAGE_SIZE)
    return MLA_EINVAL;
  if (p->max_seqs < 1 || p->max_pages < 1) return MLA_EINVAL;
  if ((int64_t)p->max_pages * p->page_size > (int64_t)INT32_MAX) return MLA_EINVAL;
  if (!p->refs || !p->table || !p->lens || !p->held) return MLA_EINVAL;
  if (!aligned(p->refs, 4) || !aligned(p->table, 4) || !aligned(p->lens, 4) || !aligned(p->held, 4)) return MLA_EINVAL;
  if (p->nbuf < 1 || p->nbuf > 4) return MLA_EINVAL;
  for (int b = 0; b < p->nbuf; ++b) {
    if (!p->buf[b] || !aligned(p->buf[b], 16)) return MLA_EINVAL;
    if (p->page_bytes[b] < 1 || p->page_bytes[b] > ((int64_t)1 << 40) || p->page_bytes[b] % p->page_size)
      return MLA_EINVAL;
  }
  return MLA_OK;
}

size_t table_bytes(const mla_pool* p) { return (size_t)p->max_seqs * (size_t)p->max_pages * 4; }

// Ranges of a pool: its arrays, and its buffers as outputs or inputs.
void pool_arrays(Ranges& r, const mla_pool* p, bool out) {
  auto add = [&](const void* q, size_t n) { out ? r.output(q, n) : r.input(q, n); };
  add(p->refs, (size_t)p->num_pages * 4);
  add(p->table, table_bytes(p));
  add(p->lens, (size_t)p->max_seqs * 4);
  add(p->held, (size_t)p->max_seqs * 4);
}
void pool_buffers(Ranges& r, const mla_pool* p, bool out) {
  for (int b = 0; b < p->nbuf; ++b) {
    const size_t n = (size_t)p->num_pages * (size_t)p->page_bytes[b];
    out ? r.output(p->buf[b], n) : r.input(p->buf[b], n);
  }
}

mla::PoolParams pool_params(const mla_pool* p) {
  mla::PoolParams q{};
  q.num_pages = p->num_pages;
  q.page_size = p->page_size;
  q.max_seqs = p->max_seqs;
  q.max_pages = p->max_pages;
  q.refs = p->refs;
  q.table = p->table;
  q.lens = p->lens;
  q.held = p->held;
  q.nbuf = p->nbuf;
  for (int b = 0; b < p->nbuf; ++b) {
    q.buf[b] = static_cast<uint8_t*>(p->buf[b]);
    q.page_bytes[b] = p->page_bytes[b];
  }
  return q;
}

// A list of n table rows (or of values per listed row).
mla_status check_list(const void* list, int32_t n) {
  if (n < 0 || n > MLA_MAX_SEQS) return MLA_EINVAL;
  if (n > 0 && (list == nullptr || !aligned(list, 4))) return MLA_EINVAL;
  return MLA_OK;
}

// The buffers of a cache of H key heads with these widths.
mla_status check_cache(const mla_pool* p, int32_t dtype, int64_t H, int64_t d_k, int64_t d_v) {
  const int per = dtype == MLA_DTYPE_MXFP8 ? 2 : 1;
  const int want = per * ((d_k ? 1 : 0) + (d_v ? 1 : 0));
  if (p->nbuf != want) return MLA_EINVAL;
  int b = 0;
  for (int64_t d : {d_k, d_v}) {
    if (!d) continue;
    if (dtype == MLA_DTYPE_MXFP8) {
      if (p->page_bytes[b] != p->page_size * H * d || p->page_bytes[b + 1] != p->page_size * H * (d / 32))
        return MLA_EINVAL;
      b += 2;
    } else {
      if (p->page_bytes[b] != p->page_size * H * d * 2) return MLA_EINVAL;
      b += 1;
    }
  }
  return MLA_OK;
}

mla_status check_workspace(const void* ws, size_t have, size_t need, uintptr_t align) {
  if (need == 0) return MLA_OK;
  if (ws == nullptr || have < need) return MLA_EWORKSPACE;
  return aligned(ws, align) ? MLA_OK : MLA_EINVAL;
}

}  // namespace

extern "C" {

mla_status mxfp4_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ld, uint8_t* codes,
                          uint8_t* scales, void* stream) {
  if (x_dtype != MLA_DTYPE_BF16 && x_dtype != MLA_DTYPE_FP32) return MLA_EINVAL;
  if (rows < 0 || cols <= 0 || cols % 32 != 0 || ld < cols) return MLA_EINVAL;
  if (rows == 0) return MLA_OK;
  if (x == nullptr || codes == nullptr || scales == nullptr) return MLA_EINVAL;
  const size_t es = x_dtype == MLA_DTYPE_FP32 ? 4 : 2;
  if (ld > ((int64_t)1 << 40)) return MLA_EINVAL;
  if (!aligned(x, 16) || ((size_t)ld * es) % 16 != 0 || !aligned(codes, 4)) return MLA_EINVAL;
  if (rows > ((int64_t)1 << 36) / cols) return MLA_EINVAL;
  if (ld != cols && rows > ((int64_t)1 << 60) / ld) return MLA_EINVAL;
  Ranges r;
  r.output(codes, (size_t)rows * cols / 2);
  r.output(scales, (size_t)rows * cols / 32);
  r.input(x, ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * es);
  if (r.overlap()) return MLA_EALIAS;
  return launched(mla::launch_mxfp4_quantize(x, x_dtype == MLA_DTYPE_FP32, rows, cols, ld, codes, scales,
                                             (hipStream_t)stream));
}

mla_status mla_qup_fwd_w4(const mla_qup_w4_args* a, void* stream) {
  if (a == nullptr) return MLA_EINVAL;
  mla_status st = check_head_shape(a->K, a->H, a->d_nope, a->d_rope);
  if (st) return st;
  int64_t max_pos = 0;
  if ((st = check_tokens(a->tokens, &max_pos))) return st;
  if ((st = check_rope(a->rope, a->d_rope, a->positions ? 0 : max_pos))) return st;
  if (a->out_dtype != MLA_DTYPE_BF16 && a->out_dtype != MLA_DTYPE_MXFP8) return MLA_EINVAL;
  const int64_t T = a->tokens.T;
  if (T == 0) return MLA_OK;
  const int D = a->d_nope + a->d_rope;
  const int64_t N = (int64_t)a->H * D;
  if (N >= (int64_t)1 << 29) return MLA_EUNSUPPORTED;  // 8 work-items a column, 2^32 in a grid's dimension
  if (!a->x || !a->w || !a->w_scales || !a->out) return MLA_EINVAL;
  const bool mx = a->out_dtype == MLA_DTYPE_MXFP8;
  if (mx && !a->out_scales) return MLA_EINVAL;
  if (!aligned(a->x, 16) || !aligned(a->w, 16) || !aligned(a->out, 16) || !aligned(a->bias, 2) ||
      !aligned(a->positions, 4))
    return MLA_EINVAL;
  Ranges r;
  r.input(a->x, (size_t)T * a->K * 2);
  r.input(a->w, (size_t)N * a->K / 2);
  r.input(a->w_scales, (size_t)N * a->K / 32);
  r.input(a->bias, (size_t)N * 2);
  r.input(a->positions, (size_t)T * 4);
  if (a->d_rope) {
    r.input(a->rope.cos, rope_bytes(a->rope, a->d_rope));
    r.input(a->rope.sin, rope_bytes(a->rope, a->d_rope));
  }
  if (a->tokens.fmt == MLA_FMT_THD) r.input(a->tokens.cu_seqlens, ((size_t)a->tokens.nseq + 1) * 4);
  r.output(a->out, (size_t)T * N * (mx ? 1 : 2));
  if (mx) r.output(a->out_scales, (size_t)T * N / 32);
  if (r.overlap()) return MLA_EALIAS;
  mla::W4Params p{};
  p.x = (const uint16_t*)a->x;
  p.w = a->w;
  p.ws = a->w_scales;
  p.bias = (const uint16_t*)a->bias;
  p.T = T;
  p.K = a->K;
  p.N = (int)N;
  p.H = a->H;
  p.D = D;
  p.d_nope = a->d_nope;
  p.d_rope = a->d_rope;
  fill_token_map(a->tokens, p.fmt, p.B, p.S, p.cu, p.nseq);
  p.positions = a->positions;
  p.cos = a->rope.cos;
  p.sin = a->rope.sin;
  p.rope_rows = a->rope.rows;
  p.rope_pairs = a->rope.pairs;
  p.out_mx = mx;
  p.out = a->out;
  p.out_scales = a->out_scales;
  return launched(mla::launch_qup_w4(p, (hipStream_t)stream));
}

size_t mla_pages_workspace_size(const mla_pool* pool) {
  return check_pool(pool) ? 0 : mla::pages_workspace_bytes(pool->num_pages);
}

mla_status mla_pages_copy(const mla_pool* src, const mla_pool* dst, const int32_t* src_ids, const int32_t* dst_ids,
                          int32_t n, void* stream) {
  mla_status st;
  if ((st = check_pool(src)) || (st = check_pool(dst))) return st;
  if (n < 0 || n > 65536) return MLA_EINVAL;
  if (n > 0 && (!src_ids || !dst_ids || !aligned(src_ids, 4) || !aligned(dst_ids, 4))) return MLA_EINVAL;
  if (src->page_size != dst->page_size || src->nbuf != dst->nbuf) return MLA_EINVAL;
  int same = 0;
  for (int b = 0; b < src->nbuf; ++b) {
    if (src->page_bytes[b] != dst->page_bytes[b]) return MLA_EINVAL;
    same += src->buf[b] == dst->buf[b];
  }
  Ranges r;
  r.input(src_ids, (size_t)n * 4);
  r.input(dst_ids, (size_t)n * 4);
  pool_buffers(r, dst, true);
  if (same != src->nbuf || src->num_pages != dst->num_pages) {
    if (same) return MLA_EALIAS;
    pool_buffers(r, src, false);
  }
  if (r.overlap()) return MLA_EALIAS;
  return launched(mla::launch_pages_copy(pool_params(src), pool_params(dst), same != 0, src_ids, dst_ids, n,
                                         (hipStream_t)stream));
}

mla_status mla_pages_reserve(const mla_pool* pool, const int32_t* seqs, const int32_t* new_tokens, int32_t n,
                             int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  mla_status st;
  if ((st = check_pool(pool)) || (st = check_list(seqs, n)) || (st = check_list(new_tokens, n))) return st;
  if (!status || !aligned(status, 4)) return MLA_EINVAL;
  const size_t need = mla::pages_workspace_bytes(pool->num_pages);
  if ((st = check_workspace(workspace, workspace_bytes, need, 16))) return st;
  Ranges r;
  r.input(seqs, (size_t)n * 4);
  r.input(new_tokens, (size_t)n * 4);
  pool_arrays(r, pool, true);
  pool_buffers(r, pool, true);
  r.output(status, 4);
  r.output(workspace, need);
  if (r.overlap()) return MLA_EALIAS;
  return launched(mla::launch_pages_reserve(pool_params(pool), seqs, new_tokens, n, status, (int32_t*)workspace,
                                            (hipStream_t)stream));
}

mla_status mla_pages_fork(const mla_pool* pool, const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
  mla_status st;
  if ((st = check_pool(pool)) || (st = check_list(src, n)) || (st = check_list(dst, n))) return st;
  Ranges r;
  r.input(src, (size_t)n * 4);
  r.input(dst, (size_t)n * 4);
  pool_arrays(r, pool, true);
  if (r.overlap()) return MLA_EALIAS;
  return launched(mla::launch_pages_fork(pool_params(pool), src, dst, n, (hipStream_t)stream));
}

mla_status mla_pages_free(const mla_pool* pool, const int32_t* seqs, const int32_t* keep, int32_t n, void* stream) {
  mla_status st;
  if ((st = check_pool(pool)) || (st = check_list(seqs, n))) return st;
  if (!aligned(keep, 4)) return MLA_EINVAL;
  Ranges r;
  r.input(seqs, (size_t)n * 4);
  r.input(keep, (size_t)n * 4);
  pool_arrays(r, pool, true);
  if (r.overlap()) return MLA_EALIAS;
  return launched(mla::launch_pages_free(pool_params(pool), seqs, keep, n, (hipStream_t)stream));
}

mla_status mla_pages_compact(const mla_pool* pool, int32_t* used, void* workspace, size_t workspace_bytes,
                             void* stream) {
  mla_status st;
  if ((st = check_pool(pool))) return st;
  if (!used || !aligned(used, 4)) return MLA_EINVAL;
  const size_t need = mla::pages_workspace_bytes(pool->num_pages);
  if ((st = check_workspace(workspace, workspace_bytes, need, 16))) return st;
  Ranges r;
  pool_arrays(r, pool, true);
  pool_buffers(r, pool, true);
  r.output(used, 4);
  r.output(workspace, need);
  if (r.overlap()) return MLA_EALIAS;
  return launched(mla::launch_pages_compact(pool_params(pool), used, (int32_t*)workspace, (hipStream_t)stream));
}

mla_status mla_draft_accept(const mla_pool* pool, const int32_t* seqs, const int32_t* path, const int32_t* n_acc,
                            int32_t n, int32_t max_path, void* stream) {
  mla_status st;
  if ((st = check_pool(pool)) || (st = check_list(seqs, n)) || (st = check_list(path, n)) || (st = check_list(n_acc, n)))
    return st;
  if (max_path < 1) return MLA_EINVAL;
  Ranges r;
  r.input(seqs, (size_t)n * 4);
  r.input(path, (size_t)n * max_path * 4);
  r.input(n_acc, (size_t)n * 4);
  pool_arrays(r, pool, true);
  pool_buffers(r, pool, true);
  if (r.overlap()) return MLA_EALIAS;
  return launched(mla::launch_draft_accept(pool_params(pool), seqs, path, n_acc, n, max_path, (hipStream_t)stream));
}

mla_status mla_kv_rope_paged(const mla_kv_paged_args* a, void* stream) {
  if (a == nullptr) return MLA_EINVAL;
  mla_status st = check_pool(a->pool);
  if (st) return st;
  if (a->H < 1 || a->d_nope < 0 || a->d_rope < 0 || a->d_v < 0) return MLA_EINVAL;
  if (a->d_nope % 8 || a->d_rope % 8 || a->d_v % 8 || a->d_rope > 256) return MLA_EINVAL;
  const int64_t Dk = (int64_t)a->d_nope + a->d_rope, Dv = a->d_v;
  if (Dk + Dv <= 0 || Dk + Dv > (1 << 20) || (int64_t)a->H * (Dk + Dv) > ((int64_t)1 << 30)) return MLA_EINVAL;
  if (a->cache_dtype != MLA_DTYPE_BF16 && a->cache_dtype != MLA_DTYPE_MXFP8) return MLA_EINVAL;
  const bool mx = a->cache_dtype == MLA_DTYPE_MXFP8;
  if (mx && (Dk % 32 || Dv % 32)) return MLA_EINVAL;
  if (Dk == 0) return MLA_EINVAL;
  if (a->T < 0 || a->T > (int64_t)INT32_MAX || a->max_q < 1) return MLA_EINVAL;
  if ((st = check_list(a->seqs, a->nseq))) return st;
  if (a->nseq > 0 && (!a->cu_q || !aligned(a->cu_q, 4))) return MLA_EINVAL;
  if (!aligned(a->positions, 4)) return MLA_EINVAL;
  if ((st = check_rope(a->rope, a->d_rope, 0))) return st;
  if ((st = check_cache(a->pool, a->cache_dtype, a->H, Dk, Dv))) return st;
  if (a->T == 0 || a->nseq == 0) return MLA_OK;
  const int64_t row_in = (int64_t)a->d_nope + a->d_v;
  if ((row_in && !a->kv) || (a->d_rope && !a->k_pe)) return MLA_EINVAL;
  if (!aligned(a->kv, 16) || !aligned(a->k_pe, 16)) return MLA_EINVAL;
  Ranges r;
  r.input(a->kv, (size_t)a->T * a->H * row_in * 2);
  r.input(a->k_pe, (size_t)a->T * a->d_rope * 2);
  r.input(a->seqs, (size_t)a->nseq * 4);
  r.input(a->cu_q, ((size_t)a->nseq + 1) * 4);
  r.input(a->positions, (size_t)a->T * 4);
  if (a->d_rope) {
    r.input(a->rope.cos, rope_bytes(a->rope, a->d_rope));
    r.input(a->rope.sin, rope_bytes(a->rope, a->d_rope));
  }
  pool_arrays(r, a->pool, false);
  pool_buffers(r, a->pool, true);
  if (r.overlap()) return MLA_EALIAS;
  mla::KvPagedParams p{};
  p.kv = (const uint16_t*)a->kv;
  p.pe = (const uint16_t*)a->k_pe;
  p.T = a->T;
  p.H = a->H;
  p.d_nope = a->d_nope;
  p.d_rope = a->d_rope;
  p.d_v = a->d_v;
  p.seqs = a->seqs;
  p.cu = a->cu_q;
  p.nseq = a->nseq;
  p.max_q = a->max_q;
  p.positions = a->positions;
  p.cos = a->rope.cos;
  p.sin = a->rope.sin;
  p.rope_rows = a->rope.rows;
  p.rope_pairs = a->rope.pairs;
  p.mx = mx;
  p.pool = pool_params(a->pool);
  return launched(mla::launch_kv_rope_paged(p, (hipStream_t)stream));
}

}  // extern "C"

namespace mla {

int device_cu_count();

bool attn_shape_supported(int d_k, int d_v, bool shared) {
  if (shared) return (d_k == 576 && d_v == 512) || (d_k == 96 && d_v == 64);
  return (d_k == 192 && d_v == 128) || (d_k == 128 && d_v == 128) || (d_k == 64 && d_v == 64);
}

AttnPlan plan_attn(int nseq, int H, int H_kv, int d_v, int max_q, int max_len, int page_size) {
  AttnPlan pl{};
  const int64_t rows = (int64_t)max_q * (H / H_kv);
  // the pages of a chunk fit the kernel's list (with one more at each end)
  const int64_t most = std::max<int64_t>(32, std::min<int64_t>(65536, (int64_t)1000 * page_size / 32 * 32));
  if (d_v > 256) {
    // the widest shape fills a CU with one workgroup; the kernel divides the
    // steps that there are by the rule that bounds their number here
    pl.waves = 4;
    const int64_t tiles = (rows + 127) / 128;
    pl.row_tiles = (int)std::min<int64_t>(tiles, INT32_MAX);
    pl.chunk = (int)most;
    pl.chunks = 1;
    const double steps = std::max(1.0, (double)nseq * H_kv * (double)tiles * ((max_len - 1) / 32 + 1));
    pl.groups = (int)std::min({(double)device_cu_count(), steps, std::floor(std::sqrt(17.0 * steps + 84.0 * nseq * H_kv * (double)tiles)) + 1});
    if (pl.groups > 1 && max_len > 32) {  // (an item of one step has no parts)
      const size_t slots = (size_t)2 * pl.groups * pl.waves;
      pl.part_o = 0;
      pl.part_ml = slots * 32 * (size_t)d_v * 4;
      pl.sums = pl.part_ml + slots * 32 * 8;
      pl.total = pl.sums + ((size_t)nseq + 3) * 8;
    }
    return pl;
  }
  pl.waves = rows <= 32 ? 1 : rows <= 64 ? 2 : 4;
  const int64_t tiles = (rows + 32 * pl.waves - 1) / (32 * pl.waves);
  pl.row_tiles = (int)std::min<int64_t>(tiles, INT32_MAX);
  const int64_t units = std::max<int64_t>(1, (int64_t)nseq * H_kv * tiles);
  // workgroups to fill the chip twice over with the waves that fit
  const int64_t want = std::max<int64_t>(1, 2 * 256 * 4 / pl.waves / units);
  const int64_t n = std::min<int64_t>(want, (max_len - 1) / 128 + 1);  // four tiles at least
  const int64_t chunk = std::min((((int64_t)max_len + n - 1) / n + 31) / 32 * 32, most);
  pl.chunk = (int)std::max<int64_t>(chunk, 32);
  pl.chunks = (max_len - 1) / pl.chunk + 1;
  if (pl.chunks > 1) {
    const size_t slots = (size_t)units * pl.chunks * pl.waves;
    pl.part_o = 0;
    pl.part_ml = slots * 32 * (size_t)d_v * 4;
    pl.total = pl.part_ml + slots * 32 * 8;
  }
  return pl;
}

}  // namespace mla

namespace {

// The factor that makes scores powers of two.
float scale_log2(const mla_tree_attn_args* a) { return (float)((double)a->scale * 1.4426950408889634); }

mla_status check_attn(const mla_tree_attn_args* a, mla::AttnPlan* plan) {
  if (a == nullptr) return MLA_EINVAL;
  mla_status st = check_pool(a->pool);
  if (st) return st;
  if (a->T < 0 || a->T > (int64_t)INT32_MAX || a->H < 1 || a->H_kv < 1 || a->H % a->H_kv) return MLA_EINVAL;
  if (a->nseq < 0 || a->nseq > 65535 || a->max_q < 1 || a->max_len < 1) return MLA_EINVAL;
  if (!isfinite(scale_log2(a))) return MLA_EINVAL;
  if (a->cache_dtype != MLA_DTYPE_BF16 && a->cache_dtype != MLA_DTYPE_MXFP8) return MLA_EINVAL;
  if (a->d_k < 1 || a->d_v < 1 || a->d_k > 65536 || a->d_v > 65536) return MLA_EINVAL;
  const bool shared = a->pool->nbuf == (a->cache_dtype == MLA_DTYPE_MXFP8 ? 2 : 1);
  if (!mla::attn_shape_supported(a->d_k, a->d_v, shared)) return MLA_EUNSUPPORTED;
  if ((st = check_cache(a->pool, a->cache_dtype, a->H_kv, a->d_k, shared ? 0 : a->d_v))) return st;
  // scale rows of 18 bytes are read in aligned words: none may reach behind the buffer
  if (a->cache_dtype == MLA_DTYPE_MXFP8 && a->d_k == 576 && a->pool->num_pages * a->pool->page_bytes[1] % 4)
    return MLA_EINVAL;
  if ((int64_t)a->max_q * (a->H / a->H_kv) > INT32_MAX / 2) return MLA_EINVAL;
  *plan = mla::plan_attn(a->nseq, a->H, a->H_kv, a->d_v, a->max_q, a->max_len, a->pool->page_size);
  // every grid stays below 2^31 work-items, and the even plan's sums within their bits
  const double tiles = (double)a->nseq * a->H_kv * plan->row_tiles;
  if (tiles * plan->chunks >= (double)(1 << 23) || tiles * plan->waves >= (double)(1 << 21)) return MLA_EINVAL;
  if (plan->groups > 0 && tiles * ((a->max_len - 1) / 32 + 1) >= (double)((int64_t)1 << 42)) return MLA_EINVAL;
  return MLA_OK;
}

}  // namespace

extern "C" {

size_t mla_tree_attention_workspace_size(const mla_tree_attn_args* a) {
  mla::AttnPlan plan;
  return check_attn(a, &plan) ? 0 : plan.total;
}

mla_status mla_tree_attention(const mla_tree_attn_args* a, void* stream) {
  mla::AttnPlan plan;
  mla_status st = check_attn(a, &plan);
  if (st) return st;
  if (a->T == 0 || a->nseq == 0) return MLA_OK;
  if (!a->q || !a->out || !a->seqs || !a->cu_q) return MLA_EINVAL;
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->lse, 4) || !aligned(a->seqs, 4) ||
      !aligned(a->cu_q, 4) || !aligned(a->mask, 4))
    return MLA_EINVAL;
  for (int64_t s : {a->q_stride_t, a->q_stride_h, a->out_stride_t, a->out_stride_h})
    if (s < 0 || s % 8 || s > ((int64_t)1 << 40)) return MLA_EINVAL;
  if (a->mask && (a->mask_words < 1 || (int64_t)a->mask_words * 32 < a->max_q)) return MLA_EINVAL;
  // output rows must not meet: heads within a token or tokens within a head
  {
    const int64_t in = std::min(a->out_stride_t, a->out_stride_h), outer = std::max(a->out_stride_t, a->out_stride_h);
    const int64_t n_in = a->out_stride_t < a->out_stride_h ? a->T : a->H;
    const int64_t n_out = a->out_stride_t < a->out_stride_h ? a->H : a->T;
    if ((n_in > 1 && in < a->d_v) || (n_out > 1 && outer < (n_in - 1) * in + a->d_v)) return MLA_EINVAL;
  }
  if ((st = check_workspace(a->workspace, a->workspace_bytes, plan.total, 256))) return st;
  Ranges r;
  r.input(a->q, ((size_t)(a->T - 1) * a->q_stride_t + (size_t)(a->H - 1) * a->q_stride_h + a->d_k) * 2);
  r.input(a->seqs, (size_t)a->nseq * 4);
  r.input(a->cu_q, ((size_t)a->nseq + 1) * 4);
  r.input(a->mask, (size_t)a->T * a->mask_words * 4);
  pool_arrays(r, a->pool, false);
  pool_buffers(r, a->pool, false);
  r.output(a->out, ((size_t)(a->T - 1) * a->out_stride_t + (size_t)(a->H - 1) * a->out_stride_h + a->d_v) * 2);
  r.output(a->lse, (size_t)a->T * a->H * 4);
  r.output(a->workspace, plan.total);
  if (r.overlap()) return MLA_EALIAS;
  mla::AttnParams p{};
  p.q = (const uint16_t*)a->q;
  p.q_t = a->q_stride_t;
  p.q_h = a->q_stride_h;
  p.out = (uint16_t*)a->out;
  p.o_t = a->out_stride_t;
  p.o_h = a->out_stride_h;
  p.lse = a->lse;
  p.T = a->T;
  p.H = a->H;
  p.H_kv = a->H_kv;
  p.group = a->H / a->H_kv;
  p.d_k = a->d_k;
  p.d_v = a->d_v;
  p.scale_log2 = scale_log2(a);
  p.seqs = a->seqs;
  p.cu = a->cu_q;
  p.nseq = a->nseq;
  p.max_q = a->max_q;
  p.max_len = std::min(a->max_len, mla::kLongestSeq);
  p.mask = a->mask;
  p.mask_words = a->mask ? a->mask_words : 0;
  p.mx = a->cache_dtype == MLA_DTYPE_MXFP8;
  p.pool = pool_params(a->pool);
  const uint32_t ps = (uint32_t)a->pool->page_size;
  p.page_magic = ps == 1 ? 0 : (uint32_t)((((uint64_t)1 << 32) + ps - 1) / ps);
  p.plan = plan;
  p.part_o = (float*)((uint8_t*)a->workspace + plan.part_o);
  p.part_ml = (float*)((uint8_t*)a->workspace + plan.part_ml);
  p.sums = (int64_t*)((uint8_t*)a->workspace + plan.sums);
  return launched(mla::launch_tree_attn(p, (hipStream_t)stream));
}

}  // extern "C"
