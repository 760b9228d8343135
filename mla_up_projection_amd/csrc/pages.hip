// Pages of the decode cache for gfx950: reserve (with copy on write), fork,
// free, compact, copy, and the acceptance of a drafted path. The bookkeeping is
// a few kilobytes of integers, so these calls cost their launches and the page
// bytes that they move; one workgroup plans (reserve, compact) and a wide grid
// copies. All results are integers and copies that do not depend on the order
// in which workgroups run: references change by integer atomics, pages are
// taken in ascending order of their ids by prefix sums.
//
// Measured: a batch of 64 conversations forked four ways, 9 rows of room each and
// acceptance, 8192 pages: free 4, fork 5, reserve 11 + 6 (its copies), accept 9
// us. Packing 8192 latent pages of 64 rows, about 290 of which move: plan 12,
// move 9 (43 MB, 4.7 TB/s). Copying 1024 such pages 22 us (7.0 TB/s of reads and writes, partly from the
// last-level cache), 4 pages 4.2. Reading the reference counts ahead of the
// lists, and keeping the pages found in LDS, changed the plan's time by nothing:
// it is a chain of dependent loads and barriers in one workgroup.
#include <algorithm>

#include "device_common.h"
#include "internal_decode.h"

namespace mla {
namespace {

constexpr int PT = 1024;    // planning workgroup
constexpr int HASH = 2048;  // slots of its hash tables, twice the longest list

// Sum over the workgroup's earlier threads of v, and the total (PT threads).
__device__ __forceinline__ int block_exclusive_sum(int v, int* total, int* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int inc = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  __syncthreads();  // the previous use of lds is over
  if (lane == 63) lds[wave] = inc;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < PT / 64; ++w) {
    const int s = lds[w];
    before += w < wave ? s : 0;
    all += s;
  }
  *total = all;
  return before + inc - v;
}

// Slot of `key` in an open-addressed table (keys start at -1).
__device__ __forceinline__ int hash_slot(int* keys, int key) {
  uint32_t h = ((uint32_t)key * 2654435761u) >> 21;  // 11 bits
  while (true) {
    const int old = atomicCAS(&keys[h], -1, key);
    if (old == -1 || old == key) return (int)h;
    h = (h + 1) & (HASH - 1);
  }
}

// Copy `bytes` from src to dst with the workgroup's threads, in the widest
// units that both addresses allow; the last bytes one by one. Several loads are
// in flight per thread before the first store.
template <typename U>
__device__ __forceinline__ void copy_units(const uint8_t* src, uint8_t* dst, int64_t bytes, int64_t first, int64_t step) {
  const int64_t n = bytes / (int64_t)sizeof(U);
  const U* s = reinterpret_cast<const U*>(src);
  U* d = reinterpret_cast<U*>(dst);
  int64_t i = first;
  for (; i + 3 * step < n; i += 4 * step) {
    const U a = s[i], b = s[i + step], c = s[i + 2 * step], e = s[i + 3 * step];
    d[i] = a;
    d[i + step] = b;
    d[i + 2 * step] = c;
    d[i + 3 * step] = e;
  }
  for (; i < n; i += step) d[i] = s[i];
  for (int64_t k = n * (int64_t)sizeof(U) + first; k < bytes; k += step) dst[k] = src[k];
}

__device__ __forceinline__ void copy_bytes(const uint8_t* src, uint8_t* dst, int64_t bytes, int64_t first, int64_t step) {
  const uint64_t a = reinterpret_cast<uint64_t>(src) | reinterpret_cast<uint64_t>(dst);
  if ((a & 15) == 0) copy_units<u32x4_t>(src, dst, bytes, first, step);
  else if ((a & 3) == 0) copy_units<uint32_t>(src, dst, bytes, first, step);
  else copy_units<uint8_t>(src, dst, bytes, first, step);
}

// ---------------------------------------------------------------- reserve --
// One workgroup, one thread per listed sequence. Two hash tables in LDS answer
// what depends on the whole list: whether a sequence was listed before, and
// how many of the list share a partly filled page (who is last keeps it when
// nobody outside the list names it). Then prefix sums over the pages needed,
// a scan of refs for that many free pages (16 per thread and step), and, only
// if there are enough, the changes.
__global__ __launch_bounds__(PT) void reserve_plan_kernel(PoolParams p, const int32_t* __restrict__ seqs,
                                                          const int32_t* __restrict__ new_tokens, int n,
                                                          int32_t* __restrict__ status, int32_t* __restrict__ ws) {
  __shared__ int seq_key[HASH], seq_first[HASH], page_key[HASH], page_count[HASH], page_last[HASH];
  __shared__ int sums[PT / 64], bad, nwide;
  __shared__ unsigned long long wanted;
  __shared__ int w_seq[PT], w_held[PT], w_at[PT], w_add[PT];
  const int tid = threadIdx.x;
  for (int k = tid; k < HASH; k += PT) {
    seq_key[k] = page_key[k] = page_last[k] = -1;
    seq_first[k] = 0x7FFFFFFF;
    page_count[k] = 0;
  }
  if (tid == 0) {
    bad = nwide = 0;
    wanted = 0;
  }
  __syncthreads();
  int seq = -1, len = 0, held = 0, add = 0, need = 0, slot = 0, page = -1, copy = 0, fresh = 0;
  if (tid < n) {
    seq = seqs[tid];
    fresh = new_tokens[tid];
    if (seq < 0 || seq >= p.max_seqs) seq = -1;
  }
  if (seq >= 0) {
    slot = hash_slot(seq_key, seq);
    atomicMin(&seq_first[slot], tid);
  }
  __syncthreads();
  if (seq >= 0 && seq_first[slot] != tid) seq = -1;
  if (seq >= 0) {
    len = p.lens[seq];
    held = p.held[seq];
    const int64_t rows = (int64_t)len + fresh;
    if (len < 0 || fresh < 0 || held < 0 || rows > (int64_t)p.max_pages * p.page_size) {
      bad = 1;
    } else {
      // (the clamp keeps the sum over 1024 sequences within 32 bits; more than there are is refused)
      need = max(0, (int)((rows + p.page_size - 1) / p.page_size) - held);
      add = min(need, p.num_pages + 1);
      const int k = len / p.page_size;
      if (fresh > 0 && len % p.page_size != 0 && k < held) {
        page = p.table[(int64_t)seq * p.max_pages + k];
        if (page < 0 || page >= p.num_pages || p.refs[page] <= 1) page = -1;
      }
      if (page >= 0) {
        slot = hash_slot(page_key, page);
        atomicAdd(&page_count[slot], 1);
        atomicMax(&page_last[slot], tid);
      }
    }
  }
  __syncthreads();
  if (page >= 0) copy = !(page_count[slot] >= p.refs[page] && page_last[slot] == tid);
  int total;
  const int at = block_exclusive_sum(add + copy, &total, sums);
  if (bad) {  // (set before the barriers of the sum)
    if (tid == 0) status[0] = -1;
    if (tid < n) ws[PW_PAIRS + 3 * tid + 1] = -1;
    return;
  }
  // the first `total` free pages, ascending
  int32_t* taken = ws + PW_HEAD;
  int found = 0;
  for (int64_t base = 0; base < p.num_pages && found < total; base += 16 * PT) {
    const int64_t first = base + 16 * tid;
    uint32_t free_bits = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (first + k < p.num_pages && p.refs[first + k] == 0) free_bits |= 1u << k;
    int all;
    int r = found + block_exclusive_sum(__popc(free_bits), &all, sums);
    for (; free_bits; free_bits &= free_bits - 1, ++r)
      if (r < total) taken[r] = (int)(first + __builtin_ctz(free_bits));
    found += all;
  }
  __syncthreads();  // `taken` is written
  const bool enough = found >= total;
  if (!enough && seq >= 0) atomicAdd(&wanted, (unsigned long long)need + copy);
  if (tid < n) {
    const bool moves = enough && seq >= 0 && copy;
    ws[PW_PAIRS + 3 * tid] = page;
    ws[PW_PAIRS + 3 * tid + 1] = moves ? taken[at] : -1;
    ws[PW_PAIRS + 3 * tid + 2] = moves ? len % p.page_size : 0;
  }
  if (!enough) {  // `found` is all that is free
    __syncthreads();
    if (tid == 0) status[0] = (int)min(wanted - found, (unsigned long long)0x7FFFFFFF);
    return;
  }
  if (tid == 0) status[0] = 0;
  if (seq >= 0) {
    if (copy) {
      p.table[(int64_t)seq * p.max_pages + len / p.page_size] = taken[at];
      atomicSub(&p.refs[page], 1);
    }
    if (add) p.held[seq] = held + add;
    // a few added pages: by the sequence's own thread; many: below, by all
    if (add <= 4)
      for (int k = 0; k < add; ++k) p.table[(int64_t)seq * p.max_pages + held + k] = taken[at + copy + k];
  }
  for (int f = tid; f < total; f += PT) p.refs[taken[f]] = 1;
  // sequences that add many pages: their rows of the table, a wave each
  if (seq >= 0 && add > 4) {
    const int k = atomicAdd(&nwide, 1);
    w_seq[k] = seq;
    w_held[k] = held;
    w_at[k] = at + copy;
    w_add[k] = add;
  }
  __syncthreads();
  const int lane = tid & 63;
  for (int k = tid >> 6; k < nwide; k += PT / 64)
    for (int a = lane; a < w_add[k]; a += 64)
      p.table[(int64_t)w_seq[k] * p.max_pages + w_held[k] + a] = taken[w_at[k] + a];
}

// The committed rows of the pages copied on write: entry blockIdx.x, slice blockIdx.y.
__global__ __launch_bounds__(256) void reserve_copy_kernel(PoolParams p, const int32_t* __restrict__ ws) {
  const int32_t* e = ws + PW_PAIRS + 3 * blockIdx.x;
  const int dst = e[1];
  if (dst < 0) return;
  const int src = e[0], rows = e[2];
  for (int b = 0; b < p.nbuf; ++b)
    copy_bytes(p.buf[b] + src * p.page_bytes[b], p.buf[b] + dst * p.page_bytes[b],
               p.page_bytes[b] / p.page_size * rows, blockIdx.y * 256 + threadIdx.x, gridDim.y * 256);
}

// ------------------------------------------------------------ fork, free --
// Whether `seq` stands in list[0, n).
__device__ __forceinline__ bool listed(const int32_t* __restrict__ list, int n, int seq) {
  int hit = 0;
  for (int j = threadIdx.x; j < n; j += blockDim.x) hit |= list[j] == seq;
  return __syncthreads_or(hit);
}

// One workgroup per entry. A destination is written by its first entry alone
// and is the source of none, so entries are independent of each other.
__global__ __launch_bounds__(256) void fork_kernel(PoolParams p, const int32_t* __restrict__ src,
                                                   const int32_t* __restrict__ dst, int n) {
  const int i = blockIdx.x;
  const int s = src[i], d = dst[i];
  if (s < 0 || s >= p.max_seqs || d < 0 || d >= p.max_seqs) return;
  if (listed(dst, i, d) || listed(dst, n, s)) return;
  const int held_d = p.held[d], len = p.lens[s];
  if (held_d > 0) return;
  if (len < 0) return;
  const int pages = max(0, min((int)(((int64_t)len + p.page_size - 1) / p.page_size), min(p.held[s], p.max_pages)));
  for (int k = threadIdx.x; k < pages; k += 256) {
    const int page = p.table[(int64_t)s * p.max_pages + k];
    p.table[(int64_t)d * p.max_pages + k] = page;
    if (page >= 0 && page < p.num_pages) atomicAdd(&p.refs[page], 1);
  }
  __syncthreads();  // held_d is read by all before it changes
  if (threadIdx.x == 0) {
    p.held[d] = pages;
    p.lens[d] = len;
  }
}

__global__ __launch_bounds__(256) void free_kernel(PoolParams p, const int32_t* __restrict__ seqs,
                                                   const int32_t* __restrict__ keep, int n) {
  const int i = blockIdx.x;
  const int s = seqs[i];
  if (s < 0 || s >= p.max_seqs) return;
  if (listed(seqs, i, s)) return;
  const int len = p.lens[s], held = min(p.held[s], p.max_pages);
  const int left = keep ? max(0, min(keep[i], len)) : 0;
  const int first = max(0, min((int)(((int64_t)left + p.page_size - 1) / p.page_size), held));
  for (int k = first + threadIdx.x; k < held; k += 256) {
    int32_t* e = p.table + (int64_t)s * p.max_pages + k;
    const int page = *e;
    *e = -1;
    if (page >= 0 && page < p.num_pages) atomicSub(&p.refs[page], 1);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    p.held[s] = first;
    p.lens[s] = left;
  }
}

// ---------------------------------------------------------------- compact --
// Pages in use U, then the used ids >= U (sources) paired in order with the
// free ids < U (targets): there are equally many of both.
__global__ __launch_bounds__(PT) void compact_plan_kernel(PoolParams p, int32_t* __restrict__ used, int32_t* __restrict__ ws) {
  __shared__ int sums[PT / 64];
  const int tid = threadIdx.x;
  int mine = 0;
  for (int64_t base = 0; base < p.num_pages; base += 16 * PT)
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int64_t id = base + 16 * tid + k;
      mine += id < p.num_pages && p.refs[id] > 0;
    }
  int U;
  block_exclusive_sum(mine, &U, sums);
  int32_t* sources = ws + PW_HEAD;
  int32_t* target = sources + p.num_pages;  // first the targets in order, then by source page
  int ns = 0, nt = 0;
  for (int64_t base = 0; base < p.num_pages; base += 16 * PT) {
    const int64_t first = base + 16 * tid;
    uint32_t src = 0, dst = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (first + k < p.num_pages) {
        const bool u = p.refs[first + k] > 0;
        if (u && first + k >= U) src |= 1u << k;
        if (!u && first + k < U) dst |= 1u << k;
      }
    int all_s, all_t;
    int rs = ns + block_exclusive_sum(__popc(src), &all_s, sums);
    int rt = nt + block_exclusive_sum(__popc(dst), &all_t, sums);
    for (; src; src &= src - 1) sources[rs++] = (int)(first + __builtin_ctz(src));
    for (; dst; dst &= dst - 1) target[rt++] = (int)(first + __builtin_ctz(dst));  // rt < U
    ns += all_s;
    nt += all_t;
  }
  __syncthreads();
  // targets in order fill target[0, ns), ns <= min(U, num_pages - U); by page
  // they go to target[source], source >= U: the two ranges are apart
  for (int r = tid; r < ns; r += PT) {
    const int s = sources[r], d = target[r];
    target[s] = d;
    p.refs[d] = p.refs[s];
    p.refs[s] = 0;
  }
  if (tid == 0) {
    ws[0] = ns;
    ws[1] = U;
    used[0] = U;
  }
}

// Tables (the first `table_blocks` workgroups) and page contents (the others).
__global__ __launch_bounds__(256) void compact_move_kernel(PoolParams p, const int32_t* __restrict__ ws, int table_blocks) {
  const int ns = ws[0], U = ws[1];
  const int32_t* sources = ws + PW_HEAD;
  const int32_t* target = sources + p.num_pages;
  if (ns == 0) return;
  if ((int)blockIdx.x < table_blocks) {
    for (int s = blockIdx.x; s < p.max_seqs; s += table_blocks) {
      const int held = min(p.held[s], p.max_pages);
      for (int k = threadIdx.x; k < held; k += 256) {
        int32_t* e = p.table + (int64_t)s * p.max_pages + k;
        const int page = *e;
        if (page >= U && page < p.num_pages) *e = target[page];
      }
    }
    return;
  }
  for (int r = blockIdx.x - table_blocks; r < ns; r += gridDim.x - table_blocks) {
    const int64_t s = sources[r], d = target[s];
    for (int b = 0; b < p.nbuf; ++b)
      copy_bytes(p.buf[b] + s * p.page_bytes[b], p.buf[b] + d * p.page_bytes[b], p.page_bytes[b], threadIdx.x, 256);
  }
}

// ------------------------------------------------------------------- copy --
__global__ __launch_bounds__(256) void copy_kernel(PoolParams src, PoolParams dst, int same,
                                                   const int32_t* __restrict__ src_ids,
                                                   const int32_t* __restrict__ dst_ids, int n) {
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int s = src_ids[i], d = dst_ids[i];
    if (s < 0 || s >= src.num_pages || d < 0 || d >= dst.num_pages) continue;
    if (listed(dst_ids, i, d)) continue;
    if (same && listed(src_ids, n, d)) continue;
    for (int b = 0; b < src.nbuf; ++b)
      copy_bytes(src.buf[b] + s * src.page_bytes[b], dst.buf[b] + d * dst.page_bytes[b], src.page_bytes[b],
                 threadIdx.x, 256);
  }
}

// ----------------------------------------------------------------- accept --
// Entry blockIdx.x, columns blockIdx.y of its row bytes. A thread owns its
// columns for the whole path and takes the rows in ascending order, ACC of
// them loaded before the first store: row a's source lies at path[a] >= a, so
// no store of rows < a can have changed it.
constexpr int ACC = 8;

template <typename U>
__device__ __forceinline__ void accept_rows(const PoolParams& p, int b, const int32_t* __restrict__ row,
                                            const int32_t* __restrict__ path, int len, int count) {
  const int64_t row_bytes = p.page_bytes[b] / p.page_size;
  const int64_t units = row_bytes / (int64_t)sizeof(U);
  const int step = gridDim.y * blockDim.x;
  for (int64_t u = blockIdx.y * blockDim.x + threadIdx.x; u < units; u += step) {
    for (int a0 = 0; a0 < count; a0 += ACC) {
      U v[ACC];
#pragma unroll
      for (int k = 0; k < ACC; ++k)
        if (a0 + k < count) {
          const int r = len + path[a0 + k];
          v[k] = reinterpret_cast<const U*>(p.buf[b] + row[r / p.page_size] * p.page_bytes[b] +
                                            r % p.page_size * row_bytes)[u];
        }
#pragma unroll
      for (int k = 0; k < ACC; ++k)
        if (a0 + k < count) {
          const int r = len + a0 + k;
          reinterpret_cast<U*>(p.buf[b] + row[r / p.page_size] * p.page_bytes[b] + r % p.page_size * row_bytes)[u] = v[k];
        }
    }
  }
}

__device__ __forceinline__ bool accept_ok(const PoolParams& p, const int32_t* __restrict__ seqs,
                                          const int32_t* __restrict__ path, const int32_t* __restrict__ n_acc,
                                          int i, int max_path, int& s, int& count) {
  s = seqs[i];
  count = n_acc[i];
  if (s < 0 || s >= p.max_seqs || count <= 0 || count > max_path || p.lens[s] < 0) return false;
  if (listed(seqs, i, s)) return false;
  const int64_t room = (int64_t)min(p.held[s], p.max_pages) * p.page_size - p.lens[s];
  int wrong = 0;
  for (int a = threadIdx.x; a < count; a += blockDim.x) {
    const int at = path[a];
    const int k = (int)min((int64_t)p.max_pages - 1, ((int64_t)p.lens[s] + max(at, 0)) / p.page_size);
    wrong |= at <= (a ? path[a - 1] : -1) || at >= room;
    const int page = p.table[(int64_t)s * p.max_pages + k];
    const int to = p.table[(int64_t)s * p.max_pages + min((int64_t)p.max_pages - 1, ((int64_t)p.lens[s] + a) / p.page_size)];
    wrong |= page < 0 || page >= p.num_pages || to < 0 || to >= p.num_pages;
  }
  return !__syncthreads_or(wrong);
}

__global__ __launch_bounds__(256) void accept_kernel(PoolParams p, const int32_t* __restrict__ seqs,
                                                     const int32_t* __restrict__ path,
                                                     const int32_t* __restrict__ n_acc, int max_path, int lens_too) {
  const int i = blockIdx.x;
  int s, count;
  path += (int64_t)i * max_path;
  if (!accept_ok(p, seqs, path, n_acc, i, max_path, s, count)) return;
  const int len = p.lens[s];
  const int32_t* row = p.table + (int64_t)s * p.max_pages;
  for (int b = 0; b < p.nbuf; ++b) {
    const int64_t row_bytes = p.page_bytes[b] / p.page_size;
    if (((row_bytes | p.page_bytes[b]) & 15) == 0) accept_rows<u32x4_t>(p, b, row, path, len, count);
    else if (((row_bytes | p.page_bytes[b]) & 1) == 0) accept_rows<uint16_t>(p, b, row, path, len, count);
    else accept_rows<uint8_t>(p, b, row, path, len, count);
  }
  if (lens_too) {  // the only workgroup of this entry
    __syncthreads();
    if (threadIdx.x == 0) p.lens[s] = len + count;
  }
}

// Lengths of entries whose rows several workgroups moved.
__global__ __launch_bounds__(256) void accept_lens_kernel(PoolParams p, const int32_t* __restrict__ seqs,
                                                          const int32_t* __restrict__ path,
                                                          const int32_t* __restrict__ n_acc, int max_path) {
  int s, count;
  path += (int64_t)blockIdx.x * max_path;
  if (!accept_ok(p, seqs, path, n_acc, blockIdx.x, max_path, s, count)) return;
  __syncthreads();
  if (threadIdx.x == 0) p.lens[s] += count;
}

}  // namespace

hipError_t launch_pages_copy(const PoolParams& src, const PoolParams& dst, bool same, const int32_t* src_ids,
                             const int32_t* dst_ids, int n, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(copy_kernel, dim3(n), dim3(256), 0, stream, src, dst, same ? 1 : 0, src_ids, dst_ids, n);
  return hipGetLastError();
}

hipError_t launch_pages_reserve(const PoolParams& p, const int32_t* seqs, const int32_t* new_tokens, int n,
                                int32_t* status, int32_t* ws, hipStream_t stream) {
  hipLaunchKernelGGL(reserve_plan_kernel, dim3(1), dim3(PT), 0, stream, p, seqs, new_tokens, n, status, ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || n == 0) return e;
  int64_t bytes = 0;
  for (int b = 0; b < p.nbuf; ++b) bytes = std::max(bytes, p.page_bytes[b]);
  // slices of 64 KB (16 units of 16 bytes a thread), at most 64 of them
  const int slices = (int)std::min<int64_t>(64, (bytes + 65535) / 65536);
  hipLaunchKernelGGL(reserve_copy_kernel, dim3(n, slices), dim3(256), 0, stream, p, ws);
  return hipGetLastError();
}

hipError_t launch_pages_fork(const PoolParams& p, const int32_t* src, const int32_t* dst, int n, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(fork_kernel, dim3(n), dim3(256), 0, stream, p, src, dst, n);
  return hipGetLastError();
}

hipError_t launch_pages_free(const PoolParams& p, const int32_t* seqs, const int32_t* keep, int n, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(free_kernel, dim3(n), dim3(256), 0, stream, p, seqs, keep, n);
  return hipGetLastError();
}

hipError_t launch_pages_compact(const PoolParams& p, int32_t* used, int32_t* ws, hipStream_t stream) {
  hipLaunchKernelGGL(compact_plan_kernel, dim3(1), dim3(PT), 0, stream, p, used, ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int table_blocks = std::min(p.max_seqs, 256);
  const int movers = std::min(std::max(1, p.num_pages / 2), 2048);
  hipLaunchKernelGGL(compact_move_kernel, dim3(table_blocks + movers), dim3(256), 0, stream, p, ws, table_blocks);
  return hipGetLastError();
}

hipError_t launch_draft_accept(const PoolParams& p, const int32_t* seqs, const int32_t* path, const int32_t* n_acc,
                               int n, int max_path, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  int64_t row = 0;
  for (int b = 0; b < p.nbuf; ++b) row = std::max(row, p.page_bytes[b] / p.page_size);
  // a workgroup's 256 threads cover 4 KB of a row in 16-byte units; up to twice
  // that, one workgroup also moves the length, which saves the second launch
  const int slices = (int)std::min<int64_t>(64, row <= 8192 ? 1 : (row + 4095) / 4096);
  hipLaunchKernelGGL(accept_kernel, dim3(n, slices), dim3(256), 0, stream, p, seqs, path, n_acc, max_path,
                     slices == 1 ? 1 : 0);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || slices == 1) return e;
  hipLaunchKernelGGL(accept_lens_kernel, dim3(n), dim3(256), 0, stream, p, seqs, path, n_acc, max_path);
  return hipGetLastError();
}

}  // namespace mla
