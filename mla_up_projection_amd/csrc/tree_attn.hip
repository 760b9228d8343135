// Attention of drafted tokens over the paged decode cache for gfx950.
//
// Per sequence and key head the query rows are (draft, head of the group)
// pairs; one pass over the cache rows with the running maximum m and sum l of
// a softmax in base 2:
//   s = scale log2(e) q.k,  p = 2^(s - m),  l = sum p,  O = sum p v.
// A wave owns 32 query rows. Both products are computed transposed,
//   S^T = K Q^T and O^T += V^T P^T  (32x32x16 bf16 MFMA),
// so that a lane holds one query row: its softmax needs one exchange between
// the halves of the wave, the scale factors are per lane, and the S^T result
// registers are P^T's operand registers as they are (the MFMA's k slots are the
// terms of a sum, so V^T is simply read in the order S^T comes in). Q stays in
// registers; the cache tile (32 rows) is in LDS, shared by the workgroup's
// waves, V^T fragments by the transposing LDS read.
//
// The cache of a sequence is cut into parts that different workgroups take;
// their (m, l, O) are joined by a second kernel in the order of the parts. A
// sequence of one part is finished at once.
//
// What bounds it (rates on the same card: a large copy 4.9 TB/s, a large bf16
// product 1365 TFLOP/s): per-head caches HBM (4 sequences of 300 to 1500 rows, 128
// heads of 192 + 128: 62 us and 7 for the join, 4.3 TB/s); the shared 576-wide
// cache the matrix units, at 2 flops for each of 128 heads and draft to a byte (32
// sequences of 4096 rows, 16 drafts, 128 heads: 560 to 580 us, 1010 to 1045
// TFLOP/s; MXFP8 650 to 665); a single token the way through the kernel (one
// sequence of 517 rows: 18 us, of which the products are 4, and 7 for the join).
#include <algorithm>

#include "device_common.h"
#include "internal_decode.h"
#include "tree_attn_wide.h"

namespace mla {
namespace {

constexpr int TILE = 32;         // cache rows per step
constexpr int BLK = TILE * 128;  // LDS bytes of a 64-column block of a tile
constexpr int MAX_CHUNK_PAGES = 1024;
constexpr float LAZY = 64.0f;    // how many powers of two a score may lie above its row's reference
constexpr float NEG_INF = -__builtin_huge_valf();

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// Position of 16-byte chunk c of cache row t within the row's 128 bytes. A row
// spans half the 64 banks, so rows t, t + 2, .. would share theirs; moving
// chunks by the bits of t above the lowest spreads the column reads of K (8
// consecutive rows, one chunk each) and the transposing reads of V (4 rows, 64
// bytes each) over all banks.
__device__ __forceinline__ int swz(int t) { return ((t >> 1) & 1) << 2 | ((t >> 2) & 1) << 1 | ((t >> 3) & 1); }

// v, in a way that lets nothing that follows from it be worked out ahead of its
// use, where it would occupy registers in between. In the widest kernel addresses
// of the path for strange values and of the page list, worked out early, went to
// scratch memory and back on every call's way in: 19.0 us instead of 17.3 for one
// token.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// n < 2^bits_of(n)
__device__ __forceinline__ int bits_of(int n) { return 32 - __builtin_clz(n); }

// max(x, |a|, |b|), NaN if one of them is.
__device__ __forceinline__ float widest(float x, float a, float b) {
  asm("v_maximum3_f32 %0, |%1|, |%2|, %0" : "+v"(x) : "v"(a), "v"(b));
  return x;
}

// The kernel's arguments (the first of every kernel here), read again: for the paths
// that hardly run, so that nothing of theirs is worked out ahead and kept. With the
// others' copy a call of one step took 17.1 us, not 17.0, and 27 short sequences
// with 22 drafts 104, not 100.
__device__ __forceinline__ const AttnParams& arguments() {
  auto* p = (const __attribute__((address_space(4))) AttnParams*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttnParams*)p;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// A row tile of a sequence and key head, or a part of its cache rows.
struct Item {
  int j, kvh, rt;
  int t0, n, rows;      // first query token, drafts, query rows (n * group)
  int len, total, seq;  // committed rows, with drafts
  bool broken;          // it outgrew the plan or its entry is invalid: NaN
  bool whole;           // all of the sequence's cache rows are taken: the result is final
  int64_t slot;         // else the place of its partial result
};

// Sequence j of the call. Any lane may ask for any j. Committed rows behind the
// held pages are nowhere, and every token sees them, so the sequence is broken at
// once: a length that means nothing must not be worked through.
__device__ __forceinline__ void load_seq(const AttnParams& p, int j, Item& it) {
  const int T = (int)p.T;
  it.j = j;
  it.t0 = min(max(p.cu[j], 0), T);
  it.n = min(max(p.cu[j + 1], it.t0), T) - it.t0;
  it.rows = it.n * p.group;
  it.seq = p.seqs[j];
  it.broken = it.seq < 0 || it.seq >= p.pool.max_seqs || it.n > p.max_q;
  it.len = it.broken ? 0 : p.pool.lens[it.seq];
  const int held = it.broken ? 0 : p.pool.held[it.seq];
  it.broken |= it.len < 0 || it.len > p.max_len - it.n ||
               it.len > (int64_t)max(min(held, p.pool.max_pages), 0) * p.pool.page_size;
  it.total = it.len + it.n;
}
// What all lanes agree on goes to scalar registers.
__device__ __forceinline__ void uniform(const AttnParams& p, Item& it) {
  it.j = __builtin_amdgcn_readfirstlane(it.j);
  it.t0 = __builtin_amdgcn_readfirstlane(it.t0);
  it.n = __builtin_amdgcn_readfirstlane(it.n);
  it.rows = it.n * p.group;
  it.seq = __builtin_amdgcn_readfirstlane(it.seq);
  it.len = __builtin_amdgcn_readfirstlane(it.len);
  it.broken = __builtin_amdgcn_readfirstlane(it.broken);
  it.total = it.len + it.n;
}
__device__ __forceinline__ void load_seq_uniform(const AttnParams& p, int j, Item& it) {
  load_seq(p, j, it);
  uniform(p, it);
}

// Chunked plan: item number -> item and its chunk; false if there is none.
__device__ __forceinline__ bool find_item(const AttnParams& p, int64_t item, Item& it, int& chunk) {
  it.slot = item;
  it.rt = (int)(item % p.plan.row_tiles);
  item /= p.plan.row_tiles;
  chunk = (int)(item % p.plan.chunks);
  item /= p.plan.chunks;
  it.kvh = (int)(item % p.H_kv);
  const int j = (int)(item / p.H_kv);
  if (j >= p.nseq) return false;
  load_seq_uniform(p, j, it);
  it.whole = it.total <= p.plan.chunk;
  return it.n > 0;
}

// Even plan (the widest shape). A step is one cache tile of one row tile; the
// call has W of them in `items` row tiles. Two ways to divide them over
// workgroups, chosen by each from the lengths on the device:
//  - many workgroups per item: an item is cut into parts of at most `quantum`
//    steps, a workgroup takes one part (a second item would cost it another 10 us
//    for queries, pages and the first tiles);
//  - few: the steps are numbered through, and workgroup b of G takes the steps
//    [b W / G, (b + 1) W / G), so that all end at the same time; but an item of at
//    most SHORT steps is not cut: who has its first step takes it all (64
//    sequences of 100 to 400 rows, 4 drafts, 128 heads: 71 us instead of 93, 27
//    short ones with 22 drafts each 165 instead of 226; with a limit of 8 steps 93
//    and 164).
// Units below are parts (quantum > 0, one per workgroup) or steps.
constexpr int WIDE_ROWS = 128, SHORT = 16;
__device__ __forceinline__ int row_tiles_of(const Item& it) { return (it.rows + WIDE_ROWS - 1) / WIDE_ROWS; }
__device__ __forceinline__ int tiles_of(const Item& it) { return (it.total + TILE - 1) / TILE; }
__device__ __forceinline__ int units_of_item(const Item& it, int quantum) {
  return quantum ? (tiles_of(it) + quantum - 1) / quantum : tiles_of(it);
}
__device__ __forceinline__ int64_t units_of(const AttnParams& p, const Item& it, int quantum) {
  return it.broken || it.n == 0 ? 0 : (int64_t)p.H_kv * row_tiles_of(it) * units_of_item(it, quantum);
}
// a / b for a >= 0, b > 0. The 64-bit division is some hundred instructions, and
// in a kernel that runs them once their fetch costs more than they do.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (__builtin_expect(((a | b) >> 32) == 0, 1)) return (uint32_t)a / (uint32_t)b;
  return a / b;
}
// G workgroups share `units`: the first `more` take each + 1 of them, the others `each`.
struct Share {
  int64_t each, more;
  __device__ __forceinline__ int64_t first(int b) const { return each * b + min((int64_t)b, more); }
  __device__ __forceinline__ int of(int64_t unit) const {  // the workgroup that has it
    const int64_t behind = more * (each + 1);
    return (int)(unit < behind ? divide(unit, each + 1) : more + divide(unit - behind, each));
  }
};
// More workgroups shorten the longest but write more partial results: a step
// takes 2 us, a partial result (256 KB out and in again) 0.12 us of all
// workgroups' time and 0.2 us more in the join of its item (a single sequence of
// 65000 rows: 150 parts 44 + 26 us, 113 parts 48 + 21, 101 parts 51 + 19).
// An item's way in and out takes 10 us. (W 2 + items 10) / G + (0.12 + 0.2 / items) G
// is least at the square root below.
__device__ __forceinline__ int workgroups_for(const AttnParams& p, int64_t W, int64_t items) {
  const float part = 0.12f + 0.2f * __builtin_amdgcn_rcpf((float)max(items, (int64_t)1));
  const float best = __builtin_amdgcn_sqrtf((2.0f * (float)W + 10.0f * (float)items) * __builtin_amdgcn_rcpf(part));
  return (int)min((int64_t)p.plan.groups, min(W, (int64_t)max(1.0f, best)));
}
// sum over items of ceil(steps / quantum) <= W / quantum + items <= G
__device__ __forceinline__ int quantum_for(int64_t W, int64_t items, int G) {
  return 4 * items <= G ? (int)divide(W + (G - items) - 1, G - items) : 0;
}

// Every row of a broken sequence, by one workgroup.
__device__ void write_nan(const AttnParams& p, const Item& it) {
  for (int r = threadIdx.x; r < it.rows; r += blockDim.x) {
    const int i = r / p.group, h = it.kvh * p.group + r % p.group;
    uint32_t* o = reinterpret_cast<uint32_t*>(p.out + (it.t0 + i) * p.o_t + h * p.o_h);
    for (int d = 0; d < p.d_v / 2; ++d) o[d] = 0x7FC07FC0u;
    if (p.lse) p.lse[(int64_t)(it.t0 + i) * p.H + h] = __builtin_nanf("");
  }
}

// Which of the cache rows [tk, tk + 32) query draft `i` (token t) sees, as bits.
__device__ __forceinline__ uint32_t visible(const AttnParams& p, const Item& it, int64_t t, int i, int tk) {
  const int d = tk - it.len;  // draft index of bit 0 (negative: committed rows come first)
  if (d <= -32) return 0xFFFFFFFFu;
  uint32_t bits;
  if (p.mask) {
    const uint32_t* w = p.mask + t * p.mask_words;
    const int k = d >> 5, sh = d & 31;  // floor division
    const uint32_t lo = k >= 0 ? (k < p.mask_words ? w[k] : 0) : 0xFFFFFFFFu;
    const uint32_t hi = sh && k + 1 < p.mask_words ? w[k + 1] : 0;
    bits = sh ? (lo >> sh) | (hi << (32 - sh)) : lo;
  } else {
    const int last = i - d;  // bits 0 .. last
    bits = last < 0 ? 0 : last >= 31 ? 0xFFFFFFFFu : (2u << last) - 1;
  }
  const int left = it.n - d;  // rows of the sequence from bit 0 on
  return left >= 32 ? bits : left <= 0 ? 0 : bits & ((1u << left) - 1);
}

// The maximum of three pairs in fp16: a bf16 that is infinite or NaN is a NaN there
// (the exponent's upper five bits are all of fp16's, the others lie in its mantissa),
// which stays whatever the others are.
__device__ __forceinline__ uint32_t widest_pairs(uint32_t x, uint32_t a, uint32_t b) {
  asm("v_pk_maximum3_f16 %0, %1, %2, %0" : "+v"(x) : "v"(a), "v"(b));
  return x;
}

// Whether one of two bf16 is infinite or NaN.
__device__ __forceinline__ bool not_finite_pair(uint32_t v) {
  return (v & 0x7F80u) == 0x7F80u || (v & 0x7F800000u) == 0x7F800000u;
}

// Sizes of a kernel variant. A workgroup has WAVES waves of 32 query rows each
// and a ring of STAGES tiles in LDS. The widest shape always has four waves, one
// to a SIMD: waves without rows only help to load (with one wave of rows a CU
// still takes a tile in less time than HBM delivers it). The others: four waves
// keep three tiles (MXFP8 two), two waves two and one wave one, so that several
// workgroups share a CU and hide each other's loads.
template <int DK, int DV, bool SHARED, bool MX, int WAVES>
struct Shape {
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int NBK = (DK + 63) / 64, NBV = SHARED ? 0 : (DV + 63) / 64;
  static constexpr int NB = NBK + NBV;       // 64-column blocks of a tile: keys, then values
  static constexpr int KK = DK / 16, NT = DV / 32;
  static constexpr int TILE_LDS = NB * BLK;
  static constexpr bool WIDE = DK == 576 && DV == 512;  // the products are written out (tree_attn_wide.h)
  static constexpr int STAGES = WIDE ? (MX ? 3 : 4) : MX ? (WAVES == 1 ? 1 : 2) : WAVES == 4 ? 3 : WAVES;
  // WIDE MXFP8, two places each: codes of a tile, 4.5 blocks of 128 bytes a row, and scales, five words a row
  static constexpr int RAW_LDS = 5 * BLK, SCALE_LDS = TILE * 20;
  static constexpr int LDS = STAGES * TILE_LDS + (WIDE && MX ? 2 * (RAW_LDS + SCALE_LDS) : 0);
  static constexpr int RPT = TILE / (8 * WAVES);  // rows of a tile that a thread stages (16 bytes of each block)
  static constexpr int LOADS = RPT * NB;          // its loads per tile
};

__device__ __forceinline__ f32x16_t mfma(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// 16 bytes per lane from any address to LDS bytes [lds_addr + 16 lane, + 16).
__device__ __forceinline__ void dma16_far(const void* p, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" :
               : "s"(__builtin_amdgcn_readfirstlane(lds_addr)), "v"(p)
               : "memory", "m0");
}

// The same with 4 bytes per lane.
__device__ __forceinline__ void dma4_far(const void* p, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds_addr)), "v"(p)
               : "memory", "m0");
}

// Barrier after this wave's LDS reads have returned (a loading instruction may
// overwrite what they read once all waves have passed).
__device__ __forceinline__ void barrier_reads_done() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int DK, int DV, bool SHARED, bool MX, int WAVES>
struct Worker {
  using S = Shape<DK, DV, SHARED, MX, WAVES>;
  const AttnParams& p;
  const Item& it;
  uint8_t* lds;
  const int* s_page;
  int page0, tk_begin, tk_end;
  bool odd;  // a value that is not finite lies in a tile that some rows do not see whole
  // the lane's query row
  bf16x8_t q[S::KK];
  f32x16_t o[S::NT];
  float m, top, l;  // reference, largest score, sum of weights
  // LDS offsets of the first fragments. A tile starts at a multiple of 128
  // bytes, so the others differ in single bits.
  uint32_t koff0, voff0;
  int tid, wave;
  // MXFP8: the next tile's codes and scales, on their way to LDS as bf16
  static constexpr int HELD = MX && S::RPT == 1 && !S::WIDE ? S::NB : 1;
  uint2 code[HELD];
  uint32_t sc[HELD];

  __device__ __forceinline__ Worker(const AttnParams& p_, const Item& it_) : p(p_), it(it_) {}

  __device__ __forceinline__ int thread() const { return opaque(tid); }

  // The lane's query row: draft qi, token qt, head h.
  struct Row {
    int l32, half, qi, h;
    int64_t qt;
    bool live;
  };
  __device__ __forceinline__ Row row() const {
    const int lane = thread() & 63;
    Row r;
    r.l32 = lane & 31;
    r.half = lane >> 5;
    const int at = (it.rt * WAVES + wave) * 32 + r.l32;
    r.live = at < it.rows;
    r.qi = r.live ? at / p.group : 0;
    r.qt = it.t0 + r.qi;
    r.h = it.kvh * p.group + (r.live ? at - r.qi * p.group : 0);
    return r;
  }

  // K: chunk 2 c + half of a block's rows. V: rows 8 e + 4 half + .., columns
  // 32 c + .. of a block.
  __device__ __forceinline__ uint32_t k_at(uint32_t tile, int c) const { return (tile + koff0) ^ (32 * c); }
  __device__ __forceinline__ uint32_t v_at(uint32_t tile, int e, int c) const {
    return ((tile + voff0) ^ (16 * e + 64 * c)) + 1024 * e;
  }

  typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
  typedef __attribute__((address_space(3))) const bf16x8_t lds_bf16x8;

  // Row (of width d) of cache row tok; rows behind the chunk read its last one.
  __device__ __forceinline__ int64_t cache_row(int tok) const {
    const uint32_t rel = (uint32_t)(min(tok, tk_end - 1) - page0 * p.pool.page_size);
    const uint32_t pk = p.page_magic ? __umulhi(rel, p.page_magic) : rel;
    const int64_t page = max(s_page[pk], 0);
    return (page * p.pool.page_size + (rel - pk * p.pool.page_size)) * p.H_kv + it.kvh;
  }

  // The 16-byte chunk of block b that this thread stages of row r goes to LDS
  // place tid % 8 of the row, so it is the chunk that belongs there.
  __device__ __forceinline__ int chunk_of(int r, int b) const {
    int c = (tid & 7) ^ swz(r);
    if (DK % 64 && b == S::NBK - 1) c &= (DK % 64) / 8 - 1;  // half a block: its other places are not read
    return c;
  }

  __device__ __forceinline__ void load_bf16(int tk, int slot) const {
#pragma unroll
    for (int g = 0; g < S::RPT; ++g) {
      const int r = g * (8 * WAVES) + (tid >> 3);
      const int64_t row = cache_row(tk + r);
      const uint32_t to = lds_u32(lds) + slot * S::TILE_LDS + g * (8 * WAVES) * 128 + wave * 1024;
#pragma unroll
      for (int b = 0; b < S::NB; ++b) {
        const bool k = b < S::NBK;
        const uint8_t* src = p.pool.buf[k ? 0 : 1] + (row * (k ? DK : DV) + (k ? b : b - S::NBK) * 64 + 8 * chunk_of(r, b)) * 2;
        dma16_far(src, to + b * BLK);
      }
    }
  }

  // The loads of a later tile that step_ahead issues between its MFMAs: in a
  // burst in front of them they kept the matrix units waiting.
  struct Next {
    const uint8_t* src = nullptr;
    uint32_t to = 0;
    uint64_t live = 0;  // lanes that load
  };
  __device__ __forceinline__ Next next_loads(int tk, int slot) const {
    const int tid = thread(), r = tid >> 3;
    const int64_t row = cache_row(tk + r);
    const uint8_t* src;
    uint32_t to = lds_u32(lds) + wave * 1024;
    if constexpr (MX) {
      src = p.pool.buf[0] + row * DK + 16 * (tid & 7);
      to += S::STAGES * S::TILE_LDS + slot * S::RAW_LDS;
    } else {
      src = p.pool.buf[0] + (row * DK + 8 * ((tid & 7) ^ swz(r))) * 2;
      to += slot * S::TILE_LDS;
    }
    return Next{src, (uint32_t)__builtin_amdgcn_readfirstlane(to), ~(uint64_t)0};
  }

  // Such loads in a burst: `blocks` of 128 bytes, and half a block more.
  __device__ __forceinline__ static void load_now(const Next& n, int blocks, bool half_more) {
    for (int b = 0; b < blocks; ++b) dma16_far(n.src + 128 * b, n.to + b * BLK);
    if (half_more && (threadIdx.x & 7) < 4) dma16_far(n.src + 128 * blocks, n.to + blocks * BLK);
  }
  // next_loads() outside the loop and for waves without rows
  __device__ __forceinline__ void load_now(const Next& n) const {
    if (n.live) load_now(n, MX ? 4 : S::NB, MX);
    else vm_wait<0>();
  }

  // Query rows 32 g .. + 31 of the row tile, as a tile of the ring: 128 bytes of a
  // row at a time instead of the 32 that a fragment's lanes would ask for
  // (7 drafts x 8 sequences of 1000, 32 heads: 11 of 43 us less). Rows that there
  // are not repeat the last.
  __device__ __forceinline__ void load_queries(int g, int slot) const {
    const int tid = thread(), r = tid >> 3;
    const int row = min((it.rt * WAVES + g) * 32 + r, it.rows - 1), i = row / p.group;
    const uint16_t* src = p.q + (it.t0 + i) * p.q_t + (it.kvh * p.group + row - i * p.group) * p.q_h + 8 * ((tid & 7) ^ swz(r));
    load_now(Next{reinterpret_cast<const uint8_t*>(src), lds_u32(lds) + slot * S::TILE_LDS + wave * 1024, 1}, S::NBK, false);
  }
  // All queries. LDS must be free (four tiles of it; of an MXFP8 ring the fourth
  // lies where codes come in); it is again for those who meet at the next barrier
  // after take_queries().
  __device__ __forceinline__ void ask_queries() const {
    static_assert(S::LDS >= 4 * S::TILE_LDS, "room for four tiles");
    for (int g = 0; g < 4; ++g)
      if ((it.rt * WAVES + g) * 32 < it.rows) load_queries(g, g);
  }
  __device__ __forceinline__ void take_queries() {
    vm_wait<0>();
    barrier_reads_done();
#pragma unroll
    for (int kk = 0; kk < S::KK; ++kk)
      q[kk] = *(lds_bf16x8*)(uintptr_t)(k_at(lds_u32(lds) + wave * S::TILE_LDS, kk & 3) + (kk >> 2) * BLK);
  }

  // WIDE MXFP8: a row's 18 scale bytes, in the five aligned words that hold
  // them, to LDS: thread 5 r + k takes word k of row r.
  __device__ __forceinline__ void load_scales(int tk, int slot) const {
    const int tid = thread();
    if (tid >= 5 * TILE) return;
    const int r = tid / 5;
    const uint8_t* src = p.pool.buf[1] + (cache_row(tk + r) * 18 & ~(int64_t)3) + 4 * (tid - 5 * r);
    dma4_far(src, lds_u32(lds) + S::STAGES * S::TILE_LDS + 2 * S::RAW_LDS + slot * S::SCALE_LDS + wave * 256);
  }

  // A tile's codes to bf16. E4M3 times 2^(byte - 127) is exact in bf16 down to
  // its subnormals; the convert reads the scale's exponent field, 0 meaning
  // 2^-127 and 255 NaN, as E8M0 does.
  __device__ __forceinline__ void convert(int tk, int raw, int slot) const {
    const int tid = thread(), r = tid >> 3, c = (tid & 7) ^ swz(r);
    const uint8_t* from = lds + S::STAGES * S::TILE_LDS + raw * S::RAW_LDS + r * 128 + c * 8;
    const uint32_t* sw = reinterpret_cast<const uint32_t*>(lds + S::STAGES * S::TILE_LDS + 2 * S::RAW_LDS + raw * S::SCALE_LDS) + 5 * r;
    // first byte wanted of the row's words: rows start at even bytes, odd rows
    // in the middle of a word
    const uint32_t sh = 2 * ((uint32_t)cache_row(tk + r) & 1) + (c >> 2);
    uint32_t w[5];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = __builtin_amdgcn_alignbyte(sw[k + 1], sw[k], sh);
    w[4] = sw[4] >> (8 * sh);
#pragma unroll
    for (int b = 0; b < S::NBK; ++b) {
      const uint2 cd = *reinterpret_cast<const uint2*>(from + (b >> 1) * BLK + (b & 1) * 64);
      const float f = __uint_as_float((b & 1 ? w[b / 2] << 7 : w[b / 2] << 23) & 0x7F800000u);
      const u32x4_t v = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(cd.x, f, false)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(cd.x, f, true)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(cd.y, f, false)),
                         __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(cd.y, f, true))};
      *reinterpret_cast<u32x4_t*>(lds + slot * S::TILE_LDS + b * BLK + r * 128 + ((tid & 7) << 4)) = v;
    }
  }

  __device__ __forceinline__ void load_mx(int64_t row, int r, uint2* cd, uint32_t* sb) const {
#pragma unroll
    for (int b = 0; b < S::NB; ++b) {
      const bool k = b < S::NBK;
      const int d = k ? DK : DV, at = (k ? b : b - S::NBK) * 64 + 8 * chunk_of(r, b);
      cd[b] = *reinterpret_cast<const uint2*>(p.pool.buf[k ? 0 : 2] + row * d + at);
      sb[b] = p.pool.buf[k ? 1 : 3][row * (d / 32) + at / 32];
    }
  }
  __device__ __forceinline__ void store_mx(int r, int slot, const uint2* cd, const uint32_t* sb) const {
#pragma unroll
    for (int b = 0; b < S::NB; ++b) {
      const float f = __uint_as_float(sb[b] << 23);  // (see convert)
      const u32x4_t v = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(cd[b].x, f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(cd[b].x, f, true)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(cd[b].y, f, false)),
                   __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(cd[b].y, f, true))};
      *reinterpret_cast<u32x4_t*>(lds + slot * S::TILE_LDS + b * BLK + r * 128 + ((tid & 7) << 4)) = v;
    }
  }

  // V^T fragment of value columns 32 n .. + 31 and the tile's 16-row step c
  __device__ __forceinline__ u32x4_t v_frag(const uint8_t* tile, int n, int c) const {
    const uint32_t at = lds_u32(tile) + (SHARED ? 0 : S::NBK * BLK), off = (n >> 1) * BLK + c * 16 * 128;
    const uint2 a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(v_at(at, 0, n & 1) + off)));
    const uint2 b = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t)(v_at(at, 1, n & 1) + off)));
    return u32x4_t{a.x, a.y, b.x, b.y};
  }

  // S^T times the scale: element i is cache row 8 (i / 4) + 4 half + i % 4,
  // column the lane's query
  __device__ __forceinline__ f32x16_t scores(const uint8_t* tile) const {
    f32x16_t s;
    if constexpr (S::WIDE) {
      const uint32_t k = lds_u32(tile);
      asm volatile(WIDE_SCORES
                   : [s] "=&v"(s)
                   : [k0] "v"(k_at(k, 0)), [k1] "v"(k_at(k, 1)), [k2] "v"(k_at(k, 2)), [k3] "v"(k_at(k, 3)),
                     [q0] "v"(q[0]), [q1] "v"(q[1]), [q2] "v"(q[2]), [q3] "v"(q[3]), [q4] "v"(q[4]), [q5] "v"(q[5]),
                     [q6] "v"(q[6]), [q7] "v"(q[7]), [q8] "v"(q[8]), [q9] "v"(q[9]), [q10] "v"(q[10]),
                     [q11] "v"(q[11]), [q12] "v"(q[12]), [q13] "v"(q[13]), [q14] "v"(q[14]), [q15] "v"(q[15]),
                     [q16] "v"(q[16]), [q17] "v"(q[17]), [q18] "v"(q[18]), [q19] "v"(q[19]), [q20] "v"(q[20]),
                     [q21] "v"(q[21]), [q22] "v"(q[22]), [q23] "v"(q[23]), [q24] "v"(q[24]), [q25] "v"(q[25]),
                     [q26] "v"(q[26]), [q27] "v"(q[27]), [q28] "v"(q[28]), [q29] "v"(q[29]), [q30] "v"(q[30]),
                     [q31] "v"(q[31]), [q32] "v"(q[32]), [q33] "v"(q[33]), [q34] "v"(q[34]), [q35] "v"(q[35])
                   : "memory", WIDE_CLOBBERS);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 0;
#pragma unroll
      for (int kk = 0; kk < S::KK; ++kk)
        s = mfma(*(lds_bf16x8*)(uintptr_t)(k_at(lds_u32(tile), kk & 3) + (kk >> 2) * BLK), q[kk], s);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) s[k] *= p.scale_log2;
    return s;
  }

  // Scores (in powers of two) to weights 2^(s - m). m is the largest score of the
  // row's first tile with a row it sees. Weights above 1 cost nothing: fp32 and
  // bf16 both reach 2^127, and a row's weights keep their precision relative to
  // each other. So O is never rescaled on the way; a row whose scores rise more
  // than 2^LAZY above m (top says so at the end) is done again with m = top. With
  // values so large that O leaves fp32's range all the same: out_of_range().
  __device__ __forceinline__ void weights(f32x16_t& s) {
    float t = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) t = fmaxf(t, s[i]);
    const u32x2_t x = swap_halves(__float_as_uint(t), __float_as_uint(t));
    t = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
    top = fmaxf(top, t);
    m = m == NEG_INF ? t : m;
    const float mu = m == NEG_INF ? 0.0f : m;
    float sum = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = exp2_hw(s[i] - mu);
      sum += s[i];
    }
    l += sum;  // of this half's rows; the halves are added at the end
  }

  // P^T operands of the two 16-row steps: weights rounded to bf16 (each by half
  // a unit of 2^-8 at most, independently, so the error of their sum averages out)
  __device__ __forceinline__ static bf16x8_t p_frag(const f32x16_t& s, int c) {
    const u32x4_t v = {pack_bf16x2(s[8 * c], s[8 * c + 1]), pack_bf16x2(s[8 * c + 2], s[8 * c + 3]),
                       pack_bf16x2(s[8 * c + 4], s[8 * c + 5]), pack_bf16x2(s[8 * c + 6], s[8 * c + 7])};
    return __builtin_bit_cast(bf16x8_t, v);
  }

  // A tile that ends the sequence or the chunk or holds drafts. Scores of rows
  // that the lane's query does not see become -infinity.
  __device__ __forceinline__ void mask(f32x16_t& s, int tk) const {
    const Row r = row();
    uint32_t vis = visible(p, it, r.qt, r.qi, tk);
    if (tk_end - tk < TILE) vis &= (1u << (tk_end - tk)) - 1;
    vis >>= 4 * r.half;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = vis & (1u << (8 * (i / 4) + i % 4)) ? s[i] : NEG_INF;
  }
  // Values that some rows do not see may be anything, and the product would make
  // NaN of 0 times infinity, so this thread's share of the tile's values is
  // looked over: if one of a draft, or of the last row (which the places behind it
  // repeat), is not finite, slow_rows() takes over. Committed rows are seen by all.
  __device__ __forceinline__ void look_over(const uint8_t* tile, int tk) {
    const int tid = thread(), first = min(it.len, tk_end - 1) - tk;
    const uint8_t* vals = tile + (SHARED ? 0 : S::NBK * BLK);
    constexpr bool ONE_ROW = S::THREADS == 8 * TILE;  // a thread's pieces are all of one row
    if (ONE_ROW && (tid >> 3) < first) return;
#pragma unroll 1
    for (int i = tid; i < DV * TILE / 8; i += S::THREADS) {  // 16 bytes each, in any order
      if (!ONE_ROW && (i >> 3) % TILE < first) continue;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(vals + 16 * i);
#pragma unroll
      for (int k = 0; k < 4; ++k) odd |= not_finite_pair(v[k]);
    }
  }

  // O^T += V^T P^T for a tile at `tile` with weights s
  __device__ __forceinline__ void values(const uint8_t* tile, const f32x16_t& s) {
    const bf16x8_t p0 = p_frag(s, 0), p1 = p_frag(s, 1);
#pragma unroll
    for (int n = 0; n < S::NT; ++n) {
      o[n] = mfma(__builtin_bit_cast(bf16x8_t, v_frag(tile, n, 0)), p0, o[n]);
      o[n] = mfma(__builtin_bit_cast(bf16x8_t, v_frag(tile, n, 1)), p1, o[n]);
    }
  }

  // Tile i at `tile` by itself: scores, weights, O^T += V^T P^T.
  __device__ __forceinline__ void step(uint8_t* tile, int i, int full) {
    f32x16_t s = scores(tile);
    if (__builtin_expect(i >= full, 0)) {
      mask(s, tk_begin + i * TILE);
      look_over(tile, tk_begin + i * TILE);
    }
    weights(s);
    values(tile, s);
  }

  // Softmax and value products of the tile at `tile` (scores s), scores of the
  // one at `ahead` into s, and the loads of a later one.
  __device__ __forceinline__ void step_ahead(const uint8_t* tile, const uint8_t* ahead, f32x16_t& s, const Next& next) {
    const uint32_t k = lds_u32(ahead), v = lds_u32(tile);
    float t0, t1;
    if constexpr (MX) {
      asm volatile(WIDE_STEP_MX
                   : [s] "+{v[192:207]}"(s), [m] "+v"(m), [top] "+v"(top), [l] "+v"(l), [t0] "=&v"(t0), [t1] "=&v"(t1),
                     [o0] "+a"(o[0]), [o1] "+a"(o[1]), [o2] "+a"(o[2]), [o3] "+a"(o[3]), [o4] "+a"(o[4]),
                     [o5] "+a"(o[5]), [o6] "+a"(o[6]), [o7] "+a"(o[7]), [o8] "+a"(o[8]), [o9] "+a"(o[9]),
                     [o10] "+a"(o[10]), [o11] "+a"(o[11]), [o12] "+a"(o[12]), [o13] "+a"(o[13]), [o14] "+a"(o[14]),
                     [o15] "+a"(o[15])
                   : [k0] "v"(k_at(k, 0)), [k1] "v"(k_at(k, 1)), [k2] "v"(k_at(k, 2)), [k3] "v"(k_at(k, 3)),
                     [v00] "v"(v_at(v, 0, 0)), [v01] "v"(v_at(v, 0, 1)), [v10] "v"(v_at(v, 1, 0)),
                     [v11] "v"(v_at(v, 1, 1)), [c] "s"(p.scale_log2), [src] "v"(next.src), [to] "s"(next.to), [live] "s"(next.live),
                     [half] "s"(next.live & 0x0F0F0F0F0F0F0F0Full),
                     [q0] "v"(q[0]), [q1] "v"(q[1]), [q2] "v"(q[2]), [q3] "v"(q[3]), [q4] "v"(q[4]), [q5] "v"(q[5]),
                     [q6] "v"(q[6]), [q7] "v"(q[7]), [q8] "v"(q[8]), [q9] "v"(q[9]), [q10] "v"(q[10]),
                     [q11] "v"(q[11]), [q12] "v"(q[12]), [q13] "v"(q[13]), [q14] "v"(q[14]), [q15] "v"(q[15]),
                     [q16] "v"(q[16]), [q17] "v"(q[17]), [q18] "v"(q[18]), [q19] "v"(q[19]), [q20] "v"(q[20]),
                     [q21] "v"(q[21]), [q22] "v"(q[22]), [q23] "v"(q[23]), [q24] "v"(q[24]), [q25] "v"(q[25]),
                     [q26] "v"(q[26]), [q27] "v"(q[27]), [q28] "v"(q[28]), [q29] "v"(q[29]), [q30] "v"(q[30]),
                     [q31] "v"(q[31]), [q32] "v"(q[32]), [q33] "v"(q[33]), [q34] "v"(q[34]), [q35] "v"(q[35])
                   : "memory", "vcc", "scc", "m0", "v184", "v185", "v186", "v187", "v188", "v189", "v190", "v191", WIDE_CLOBBERS);
    } else {
      asm volatile(WIDE_STEP
                   : [s] "+{v[192:207]}"(s), [m] "+v"(m), [top] "+v"(top), [l] "+v"(l), [t0] "=&v"(t0), [t1] "=&v"(t1),
                     [o0] "+a"(o[0]), [o1] "+a"(o[1]), [o2] "+a"(o[2]), [o3] "+a"(o[3]), [o4] "+a"(o[4]),
                     [o5] "+a"(o[5]), [o6] "+a"(o[6]), [o7] "+a"(o[7]), [o8] "+a"(o[8]), [o9] "+a"(o[9]),
                     [o10] "+a"(o[10]), [o11] "+a"(o[11]), [o12] "+a"(o[12]), [o13] "+a"(o[13]), [o14] "+a"(o[14]),
                     [o15] "+a"(o[15])
                   : [k0] "v"(k_at(k, 0)), [k1] "v"(k_at(k, 1)), [k2] "v"(k_at(k, 2)), [k3] "v"(k_at(k, 3)),
                     [v00] "v"(v_at(v, 0, 0)), [v01] "v"(v_at(v, 0, 1)), [v10] "v"(v_at(v, 1, 0)),
                     [v11] "v"(v_at(v, 1, 1)), [c] "s"(p.scale_log2), [src] "v"(next.src), [to] "s"(next.to), [live] "s"(next.live),
                     [q0] "v"(q[0]), [q1] "v"(q[1]), [q2] "v"(q[2]), [q3] "v"(q[3]), [q4] "v"(q[4]), [q5] "v"(q[5]),
                     [q6] "v"(q[6]), [q7] "v"(q[7]), [q8] "v"(q[8]), [q9] "v"(q[9]), [q10] "v"(q[10]),
                     [q11] "v"(q[11]), [q12] "v"(q[12]), [q13] "v"(q[13]), [q14] "v"(q[14]), [q15] "v"(q[15]),
                     [q16] "v"(q[16]), [q17] "v"(q[17]), [q18] "v"(q[18]), [q19] "v"(q[19]), [q20] "v"(q[20]),
                     [q21] "v"(q[21]), [q22] "v"(q[22]), [q23] "v"(q[23]), [q24] "v"(q[24]), [q25] "v"(q[25]),
                     [q26] "v"(q[26]), [q27] "v"(q[27]), [q28] "v"(q[28]), [q29] "v"(q[29]), [q30] "v"(q[30]),
                     [q31] "v"(q[31]), [q32] "v"(q[32]), [q33] "v"(q[33]), [q34] "v"(q[34]), [q35] "v"(q[35])
                   : "memory", "vcc", "scc", "m0", "v184", "v185", "v186", "v187", "v188", "v189", "v190", "v191", WIDE_CLOBBERS);
    }
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < S::NT; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[n][i] = 0;
    top = NEG_INF;
    l = 0;
    odd = false;
  }

  // All tiles of the chunk.
  __device__ __forceinline__ void pass(int tiles, int full) {
    if constexpr (S::WIDE) pass_wide(tiles, full);
    else pass_any(tiles, full);
  }

  // Step i works on tiles i and i + 1, which are in LDS as bf16.
  __device__ __forceinline__ void pass_wide(int tiles, int full) {
    const bool active = it.rt * 32 * WAVES + wave * 32 < it.rows;
    f32x16_t s;
    if constexpr (!MX) {
      // Tile i + 2 is under way and i + 3 asked for during step i, into the
      // place of i - 1, which all have left when they meet at the barrier.
      for (int i = 0; i < min(3, tiles); ++i) load_now(next_loads(tk_begin + i * TILE, i));
      if (tiles > 2) vm_wait<2 * S::LOADS>();
      else vm_wait<0>();
      barrier_reads_done();
    } else {
      // During step i the codes of tile i + 2 are converted (before the
      // products) and those of i + 3 asked for.
      load_now(next_loads(tk_begin, 0));
      load_now(next_loads(tk_begin + TILE, 1));
      load_scales(tk_begin, 0);
      load_scales(tk_begin + TILE, 1);
      vm_wait<0>();
      barrier_reads_done();
      convert(tk_begin, 0, 0);
      convert(tk_begin + TILE, 1, 1);
      barrier_reads_done();
      load_now(next_loads(tk_begin + 2 * TILE, 0));
      load_scales(tk_begin + 2 * TILE, 0);
    }
    if (active) s = scores(lds);
    int slot = 0, third = MX ? 2 : 3;  // ring places of tile i and of the one that comes in
    for (int i = 0; i < tiles; ++i) {
      const int after = slot + 1 == S::STAGES ? 0 : slot + 1;
      Next loads;
      if constexpr (!MX) {
        if (i + 2 < tiles) vm_wait<S::LOADS>();
        else vm_wait<0>();  // nothing younger than tile i + 1 is under way
        barrier_reads_done();
        if (i + 3 < tiles) loads = next_loads(tk_begin + (i + 3) * TILE, third);
      } else {
        vm_wait<0>();
        barrier_reads_done();
        if (i + 2 < tiles) convert(tk_begin + (i + 2) * TILE, i & 1, third);
        if (i + 3 < tiles) {
          loads = next_loads(tk_begin + (i + 3) * TILE, (i + 1) & 1);
          load_scales(tk_begin + (i + 3) * TILE, (i + 1) & 1);
        }
      }
      if (__builtin_expect(i >= full, 0)) {
        if (active) mask(s, tk_begin + i * TILE);
        look_over(lds + slot * S::TILE_LDS, tk_begin + i * TILE);
      }
      // (behind the last tile the scores of what lies there are not used)
      if (active) step_ahead(lds + slot * S::TILE_LDS, lds + after * S::TILE_LDS, s, loads);
      else load_now(loads);
      slot = after;
      third = third + 1 == S::STAGES ? 0 : third + 1;
    }
#pragma unroll
    for (int n = 0; n < S::NT; ++n) asm volatile("" : "+a"(o[n]));  // O stays where it is up to here
  }

  __device__ __forceinline__ void pass_any(int tiles, int full) {
    if constexpr (!MX) {
      constexpr int AHEAD = S::STAGES - 1;
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (i < tiles) load_bf16(tk_begin + i * TILE, i);
      int slot = 0, next = AHEAD;  // ring places of tile i and of tile i + AHEAD
      for (int i = 0; i < tiles; ++i) {
        if constexpr (AHEAD == 0) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the previous tile is read
          load_bf16(tk_begin + i * TILE, 0);
          vm_wait<0>();
        } else {
          // tile i has landed when only the AHEAD - 1 younger ones are under way;
          // near the end there are fewer, so wait for all
          if (i + AHEAD <= tiles) vm_wait<(AHEAD - 1) * S::LOADS>();
          else vm_wait<0>();
          barrier_reads_done();
          if (i + AHEAD < tiles) load_bf16(tk_begin + (i + AHEAD) * TILE, next);
        }
        step(lds + slot * S::TILE_LDS, i, full);
        slot = slot + 1 == S::STAGES ? 0 : slot + 1;
        next = next + 1 == S::STAGES ? 0 : next + 1;
      }
    } else {
      int slot = 0;
      const int r = tid >> 3;
      if constexpr (S::RPT == 1) load_mx(cache_row(tk_begin + r), r, code, sc);
      for (int i = 0; i < tiles; ++i) {
        if constexpr (S::RPT == 1) {
          store_mx(r, slot, code, sc);
          barrier_reads_done();  // (two slots: the one written next was read before this barrier)
          if (i + 1 < tiles) load_mx(cache_row(tk_begin + (i + 1) * TILE + r), r, code, sc);
        } else {
          if constexpr (S::STAGES == 1) __syncthreads();
#pragma unroll
          for (int g = 0; g < S::RPT; ++g) {
            const int rr = g * (8 * WAVES) + r;
            uint2 cd[S::NB];
            uint32_t sb[S::NB];
            load_mx(cache_row(tk_begin + i * TILE + rr), rr, cd, sb);
            store_mx(rr, slot, cd, sb);
          }
          __syncthreads();
        }
        step(lds + slot * S::TILE_LDS, i, full);
        slot = slot + 1 == S::STAGES ? 0 : slot + 1;
      }
    }
  }
};

// Eight elements of a cache row, c .. c + 7, as bf16 pairs.
template <bool MX>
__device__ __forceinline__ u32x4_t cache_eight(const PoolParams& pool, int b, int64_t row, int d, int c) {
  if constexpr (!MX) return *reinterpret_cast<const u32x4_t*>(reinterpret_cast<const uint16_t*>(pool.buf[b]) + row * d + c);
  const uint2 code = *reinterpret_cast<const uint2*>(pool.buf[2 * b] + row * d + c);
  const float f = __uint_as_float((uint32_t)pool.buf[2 * b + 1][row * (d / 32) + c / 32] << 23);
  return u32x4_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code.x, f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code.x, f, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code.y, f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code.y, f, true))};
}

// sum + the products of eight bf16 and eight others.
__device__ __forceinline__ float dot8(u32x4_t a, u32x4_t b, float sum) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    sum = __builtin_fmaf(bf16_bits_to_f32(a[k] & 0xFFFFu), bf16_bits_to_f32(b[k] & 0xFFFFu), sum);
    sum = __builtin_fmaf(bf16_bits_to_f32(a[k] >> 16), bf16_bits_to_f32(b[k] >> 16), sum);
  }
  return sum;
}

// Cache row of token `tok` of a sequence that holds `held` pages; `bad` if its
// page lies outside the pool.
__device__ __forceinline__ int64_t find_row(const AttnParams& p, const Item& it, int held, uint32_t tok, bool& bad) {
  const uint32_t ps = (uint32_t)p.pool.page_size, pk = tok / ps;
  const int page = (int)pk < held ? p.pool.table[(int64_t)it.seq * p.pool.max_pages + pk] : -1;
  bad = page < 0 || page >= p.pool.num_pages;
  return ((bad ? 0 : (int64_t)page) * ps + (tok - pk * ps)) * p.H_kv + it.kvh;
}

// Cache rows [tk_begin, tk_end) for one query row by one wave, without the matrix
// units: for what those cannot do, an infinite or NaN value that some rows must
// not see (no weight keeps it out of a product) and a page id outside the pool (the
// row's result is NaN). Of 64 cache rows, eight lanes take a row's scores, then LANES
// lanes a row's values, eight columns each, all loads of 16 bytes with several in
// flight. A row that is not seen adds nothing. o: the lane's columns, 8 (lane %
// LANES) on; the reference lies so far above the largest score that the weights'
// sum stays below 1 and finite values give finite sums. All of a workgroup's rows come here, so it costs: one stray NaN among 8
// sequences of 2000 rows, 4 drafts, 16 heads makes 1.4 ms of 35 us (5.5 with a lane
// for every 64th column and one cache row at a time).
// The columns may also be some eights of them, first + step (lane % LANES). DK 0: any
// width, in few registers.
template <int DK, bool MX, int LANES>
__device__ __forceinline__ void slow_row(const AttnParams& p, const Item& it, int row, int tk_begin, int tk_end,
                                         float (&o)[8], float& m, float& l, int first = 0, int step = 1) {
  constexpr int CHUNKS = (DK + 63) / 64;  // 16-byte chunks of a key to a lane
  constexpr int PASS = 64 / LANES, AHEAD = LANES == 64 ? 8 : LANES == 1 ? 1 : 2;  // rows to a load, loads in flight
  const int lane = opaque((int)threadIdx.x) & 63, part = lane & 7, of8 = lane >> 3;
  const bool shared = p.pool.nbuf == (MX ? 2 : 1);
  const int dk = DK ? DK : p.d_k;
  const float above = (float)bits_of(tk_end - tk_begin);
  const int vb = shared ? 0 : 1, vd = shared ? p.d_k : p.d_v;
  const int held = min(p.pool.held[it.seq], p.pool.max_pages);
  const int qi = row / p.group, h = it.kvh * p.group + row - qi * p.group;
  const int64_t qt = it.t0 + qi;
  const uint16_t* query = p.q + qt * p.q_t + h * p.q_h;
  u32x4_t q[CHUNKS + 1];
#pragma unroll
  for (int c = 0; c < CHUNKS; ++c)
    if (DK % 64 == 0 || 8 * (part + 8 * c) < DK) q[c] = *reinterpret_cast<const u32x4_t*>(query + 8 * (part + 8 * c));
  m = NEG_INF;
  l = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] = 0;
  for (uint32_t tk = (uint32_t)tk_begin; tk < (uint32_t)tk_end; tk += 64) {
    const uint32_t tok = tk + lane;
    const bool see = tok < (uint32_t)tk_end && (visible(p, it, qt, qi, (int)(tk + (lane & 32))) >> (lane & 31)) & 1;
    bool bad;
    const int64_t crow = find_row(p, it, held, min(tok, (uint32_t)tk_end - 1), bad);
    float s = 0;
#pragma unroll 1
    for (int g = 0; g < 8; ++g) {
      const int64_t r = __shfl(crow, 8 * g + of8);
      float sum = 0;
      u32x4_t a[CHUNKS + 1];
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
        if (DK % 64 == 0 || 8 * (part + 8 * c) < DK) a[c] = cache_eight<MX>(p.pool, 0, r, dk, 8 * (part + 8 * c));
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
        if (DK % 64 == 0 || 8 * (part + 8 * c) < DK) sum = dot8(a[c], q[c], sum);
      if (DK == 0)
#pragma unroll 1
        for (int d = 8 * part; d < dk; d += 64)
          sum = dot8(cache_eight<MX>(p.pool, 0, r, dk, d), *reinterpret_cast<const u32x4_t*>(query + d), sum);
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor(sum, d);
      sum = __shfl(sum, 8 * part);
      if (of8 == g) s = sum;
    }
    s = !see ? NEG_INF : bad ? __builtin_nanf("") : s * p.scale_log2;
    if (__any(__builtin_isnan(s))) {  // and so is everything that follows
      m = l = __builtin_nanf("");
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = m;
      return;
    }
    float top = s;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (top == NEG_INF) continue;
    top += above;
    if (top > m) {
      const float f = exp2_hw(m - top);  // 0 for the first
      m = top;
      l *= f;
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] *= f;
    }
    const float w = see ? exp2_hw(s - m) : 0.0f;
    l += w;
#pragma unroll 1
    for (int j = 0; j < 64; j += PASS * AHEAD) {
      u32x4_t v[AHEAD];
      float wj[AHEAD];
      bool sj[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int from = j + u * PASS + lane / LANES;
        wj[u] = __shfl(w, from);
        sj[u] = __shfl((int)see, from);
        v[u] = cache_eight<MX>(p.pool, vb, __shfl(crow, from), vd, 8 * min(first + step * (lane % LANES), p.d_v / 8 - 1));
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (sj[u])
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            o[2 * k] += wj[u] * bf16_bits_to_f32(v[u][k] & 0xFFFFu);
            o[2 * k + 1] += wj[u] * bf16_bits_to_f32(v[u][k] >> 16);
          }
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
#pragma unroll
  for (int d = LANES; d < 64; d <<= 1)
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] += __shfl_xor(o[k], d);
}

// The workgroup's rows by slow_row, a wave its 32 one by one. Writes what the fast
// path writes.
template <int DK, int DV, bool SHARED, bool MX, int WAVES>
__device__ __forceinline__ void slow_rows(const Item& it, int tk_begin, int tk_end) {
  const AttnParams& p = arguments();
  const int tid = opaque((int)threadIdx.x), lane = tid & 63, wave = tid >> 6, v = lane % (DV / 8);
  const int64_t slot = it.slot * WAVES + wave;
#pragma unroll 1
  for (int r32 = 0; r32 < 32; ++r32) {
    const int row = __builtin_amdgcn_readfirstlane((it.rt * WAVES + wave) * 32 + r32);
    if (row >= it.rows) return;
    float o[8], m, l;
    slow_row<DK, MX, DV / 8>(p, it, row, tk_begin, tk_end, o, m, l);
    const int qi = row / p.group, h = it.kvh * p.group + row - qi * p.group;
    const int64_t qt = it.t0 + qi;
    const float inv = l == 0 ? 0.0f : 1.0f / l;
    if (lane >= DV / 8) continue;
    if (it.whole) {
      *reinterpret_cast<uint4*>(p.out + qt * p.o_t + h * p.o_h + 8 * v) =
          make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                     pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
      if (lane == 0 && p.lse) p.lse[qt * p.H + h] = l == 0 ? NEG_INF : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
    } else {  // column 32 n + 8 g + 4 half + e
      f32x4_t* po = reinterpret_cast<f32x4_t*>(p.part_o) + slot * (DV * 8) + v * 64 + r32;
      po[0] = f32x4_t{o[0], o[1], o[2], o[3]};
      po[32] = f32x4_t{o[4], o[5], o[6], o[7]};
      if (lane == 0) reinterpret_cast<float2*>(p.part_ml)[slot * 32 + r32] = make_float2(m, l);
    }
  }
}

// Rows of an item (bits of `rows`, from row `at` on) whose result over all cache rows
// came out infinite or NaN although their scores are finite. Either a committed
// value is not finite, and the rows, which all see it, have what the formula gives;
// or sums left fp32's range on the way to a mean that lies in it, and the rows are
// done again by slow_row. For a wave, and the columns 8 (first + step v), v < LANES.
template <int DK, bool MX, int LANES>
__device__ __forceinline__ void out_of_range(const Item& it, int at, uint32_t rows, int first, int step) {
  const AttnParams& p = arguments();
  const int lane = opaque((int)threadIdx.x) & 63;
  const bool shared = p.pool.nbuf == (MX ? 2 : 1);
  const int held = min(p.pool.held[it.seq], p.pool.max_pages), c = 8 * min(first + step * (lane % LANES), p.d_v / 8 - 1);
#pragma unroll 1
  for (uint32_t tk = 0; tk < (uint32_t)it.len; tk += 4 * (64 / LANES)) {
    u32x4_t v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      bool bad;
      const int64_t r = find_row(p, it, held, min(tk + u * (64 / LANES) + lane / LANES, (uint32_t)it.len - 1), bad);
      v[u] = cache_eight<MX>(p.pool, shared ? 0 : 1, r, shared ? p.d_k : p.d_v, c);
    }
    bool strange = false;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) strange |= not_finite_pair(v[u][k]);
    if (__any(strange)) return;
  }
  vm_wait<0>();  // what this wave wrote
#pragma unroll 1
  for (; rows; rows &= rows - 1) {
    const int row = __builtin_amdgcn_readfirstlane(at + __builtin_ctz(rows));
    float o[8], m, l;
    slow_row<DK, MX, LANES>(p, it, row, 0, it.total, o, m, l, first, step);
    const int qi = row / p.group, h = it.kvh * p.group + row - qi * p.group;
    const float inv = l == 0 ? 0.0f : 1.0f / l;
    if (lane < LANES)
      *reinterpret_cast<uint4*>(p.out + (int64_t)(it.t0 + qi) * p.o_t + h * p.o_h + c) =
          make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                     pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
  }
}

// Bits set by any of the workgroup's threads, to all of them, with one barrier
// (the place is free again after the next).
template <int WAVES>
__device__ __forceinline__ int any_of(bool bit0, bool bit1, int* place) {
  const int bits = (__any(bit0) ? 1 : 0) | (__any(bit1) ? 2 : 0);
  if ((threadIdx.x & 63) == 0) place[threadIdx.x >> 6] = bits;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) all |= place[w];
  return __builtin_amdgcn_readfirstlane(all);
}

// Page ids of cache rows [tk_begin, tk_end) to s_page, -1 for those outside the
// pool; returns whether there are any. All threads; the list is complete after.
template <int WAVES>
__device__ __forceinline__ bool fill_pages(const AttnParams& p, const Item& it, int* s_page, int page0, int tk_end) {
  const int pages = (tk_end - 1) / p.pool.page_size - page0 + 1;
  const int held = min(__builtin_amdgcn_readfirstlane(p.pool.held[it.seq]), p.pool.max_pages);
  bool bad = false;
  for (int k = opaque((int)threadIdx.x); k < pages; k += 64 * WAVES) {
    int id = page0 + k < held ? p.pool.table[(int64_t)it.seq * p.pool.max_pages + page0 + k] : -1;
    if (id < 0 || id >= p.pool.num_pages) {
      id = -1;
      bad = true;
    }
    s_page[k] = id;
  }
  return any_of<WAVES>(bad, false, s_page + MAX_CHUNK_PAGES);
}

// Cache rows [tk_begin, tk_end) of an item, and its result or partial result.
// `most`: cache rows whose pages fit the list.
template <int DK, int DV, bool SHARED, bool MX, int WAVES>
__device__ __forceinline__ void run_item(const AttnParams& p, const Item& it, uint8_t* lds, int* s_page, int tk_begin,
                                         int tk_end, int most) {
  using S = Shape<DK, DV, SHARED, MX, WAVES>;
  Worker<DK, DV, SHARED, MX, WAVES> w(p, it);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, half = lane >> 5;
  w.tid = tid;
  w.wave = wave;
  w.lds = lds;
  w.s_page = s_page;
  w.m = NEG_INF;
  // K: row l32, chunk half. V: rows 4 half + 0..3, 16 columns per 16 lanes
  w.koff0 = l32 * 128 + ((half ^ swz(l32)) << 4);
  const int q4 = lane & 15, vt = 4 * half + (q4 >> 2);
  w.voff0 = vt * 128 + (((2 * ((lane >> 4) & 1) + ((q4 & 3) >> 1)) ^ swz(vt)) << 4) + (q4 & 1) * 8;

  bool filled = S::WIDE, bad = false;  // the first part's pages are listed
  if constexpr (S::WIDE) {
    __syncthreads();  // LDS is read
    w.ask_queries();
    w.page0 = tk_begin / p.pool.page_size;
    bad = fill_pages<WAVES>(p, it, s_page, w.page0, min(tk_begin + most, tk_end));  // while they come
    w.take_queries();
  } else {
    const auto r = w.row();
#pragma unroll
    for (int kk = 0; kk < S::KK; ++kk)
      w.q[kk] = *reinterpret_cast<const bf16x8_t*>(p.q + r.qt * p.q_t + r.h * p.q_h + 16 * kk + 8 * half);
  }
  bool slow;
  while (true) {
    w.clear();
    slow = false;
    // (only the widest shape's parts can be longer than its list of pages)
    for (int begin = tk_begin; begin < tk_end; begin += most) {
      const int end = S::WIDE ? min(begin + most, tk_end) : tk_end;
      w.tk_begin = begin;
      w.tk_end = end;
      w.page0 = begin / p.pool.page_size;
      __syncthreads();  // LDS is read: the list may change and tiles come in
      if (!filled || begin > tk_begin) bad = fill_pages<WAVES>(p, it, s_page, w.page0, end);
      filled = begin == tk_begin && (!S::WIDE || end == tk_end);  // for a second pass
      slow = bad;
      if (slow) break;
      // tiles before the first draft and wholly inside the part need no mask
      const int full = max(0, (min(end, it.len) - begin) / TILE);
      w.pass((end - begin + TILE - 1) / TILE, full);
      if constexpr (!S::WIDE) break;
    }
    const int seen = any_of<WAVES>(w.odd, w.top > w.m + LAZY, s_page + MAX_CHUNK_PAGES + WAVES);
    slow = slow || (seen & 1);
    if (slow || __builtin_expect(!(seen & 2), 1)) break;
    w.m = w.top;  // the largest score of all: the next pass is the last
  }
  if (__builtin_expect(slow, 0)) {
    slow_rows<DK, DV, SHARED, MX, WAVES>(it, tk_begin, tk_end);
    return;
  }
  const float m = w.m;
  float l = w.l;
  {
    const u32x2_t x = swap_halves(__float_as_uint(l), __float_as_uint(l));
    l = __uint_as_float(x[0]) + __uint_as_float(x[1]);
  }
  const auto r = w.row();
  if (S::WIDE && it.whole) {
    // through LDS, which nobody reads any more, so that a row of the output is
    // written at once (8 bytes a lane to 64 places took 20 us instead of 16 for a
    // sequence of one step): 16-byte piece q of row r lies at place q ^ r
    const float inv = l == 0 ? 0.0f : 1.0f / l;
    uint8_t* rows = lds + wave * (32 * DV * 2);
#pragma unroll
    for (int n = 0; n < S::NT; ++n)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<uint2*>(rows + r.l32 * (DV * 2) + (((4 * n + g) ^ r.l32) << 4) + 8 * r.half) =
            make_uint2(pack_bf16x2(w.o[n][4 * g] * inv, w.o[n][4 * g + 1] * inv),
                       pack_bf16x2(w.o[n][4 * g + 2] * inv, w.o[n][4 * g + 3] * inv));
    const int at = (it.rt * WAVES + wave) * 32;
    int qi = at / p.group, h = at - qi * p.group;
    uint16_t* dst = p.out + (int64_t)(it.t0 + qi) * p.o_t + (int64_t)(it.kvh * p.group + h) * p.o_h + 8 * lane;
    const int live = min(32, it.rows - at);
    uint32_t largest = 0;
    for (int k = 0; k < live; ++k) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(rows + k * (DV * 2) + ((lane ^ k) << 4));
      *reinterpret_cast<u32x4_t*>(dst) = v;
      largest = widest_pairs(widest_pairs(largest, v[0], v[1]), v[2], v[3]);
      dst += p.o_h;
      if (++h == p.group) {
        h = 0;
        dst += p.o_t - (int64_t)p.group * p.o_h;
      }
    }
    if (p.lse && r.live && r.half == 0)
      p.lse[r.qt * p.H + r.h] = l == 0 ? NEG_INF : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
    if (__builtin_expect(__any((largest & 0x7C00u) == 0x7C00u || (largest & 0x7C000000u) == 0x7C000000u), 0)) {
      uint32_t strange = 0;
      for (int k = 0; k < live; ++k) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(rows + k * (DV * 2) + ((lane ^ k) << 4));
        if (__any(not_finite_pair(v[0]) || not_finite_pair(v[1]) || not_finite_pair(v[2]) || not_finite_pair(v[3])))
          strange |= 1u << k;
      }
      strange &= (uint32_t)__ballot(l < __builtin_huge_valf());
      if (strange) out_of_range<DK, MX, DV / 8>(it, at, strange, 0, 1);
    }
    return;
  }
  if (it.whole) {
    const float inv = l == 0 ? 0.0f : 1.0f / l;
    uint16_t* dst = p.out + r.qt * p.o_t + r.h * p.o_h;
    float x = 0;
    if (r.live) {
#pragma unroll
      for (int n = 0; n < S::NT; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          x = widest(widest(x, w.o[n][4 * g], w.o[n][4 * g + 1]), w.o[n][4 * g + 2], w.o[n][4 * g + 3]);
          *reinterpret_cast<uint2*>(dst + 32 * n + 8 * g + 4 * r.half) =
              make_uint2(pack_bf16x2(w.o[n][4 * g] * inv, w.o[n][4 * g + 1] * inv),
                         pack_bf16x2(w.o[n][4 * g + 2] * inv, w.o[n][4 * g + 3] * inv));
        }
      if (p.lse && r.half == 0)
        p.lse[r.qt * p.H + r.h] = l == 0 ? NEG_INF : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
    }
    const uint64_t strange = __ballot(!(x < __builtin_huge_valf()) && l < __builtin_huge_valf());
    if (__builtin_expect(strange != 0, 0))
      out_of_range<DK, MX, DV / 8>(it, (it.rt * WAVES + wave) * 32, (uint32_t)(strange | strange >> 32), 0, 1);
    return;
  }
  if (!r.live) return;
  // partial result, in register order: [slot][wave][32 DV floats as NT * 4 vectors of 64 lanes]
  const int64_t slot = it.slot * WAVES + wave;
  f32x4_t* po = reinterpret_cast<f32x4_t*>(p.part_o) + slot * (DV * 8);
#pragma unroll
  for (int n = 0; n < S::NT; ++n)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      po[(n * 4 + g) * 64 + 32 * r.half + r.l32] = f32x4_t{w.o[n][4 * g], w.o[n][4 * g + 1], w.o[n][4 * g + 2], w.o[n][4 * g + 3]};
  if (r.half == 0) reinterpret_cast<float2*>(p.part_ml)[slot * 32 + r.l32] = make_float2(m, l);
}

// Chunked plan: a workgroup an item. (The fewest waves of a SIMD are those that the
// matrix path alone would have; without them slow_rows takes registers from it.)
template <int DK, int DV, bool SHARED, bool MX, int WAVES>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(DK == 64 ? 4 : DK == 96 ? 3 : 2, 4)))
void tree_attn_kernel(AttnParams p) {
  using S = Shape<DK, DV, SHARED, MX, WAVES>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  __shared__ int s_page[MAX_CHUNK_PAGES + 8];  // and eight words of any_of
  // consecutive items (row tiles that read the same chunk) go to one XCD's L2
  const int64_t per = gridDim.x / 8;
  Item it;
  int chunk;
  if (!find_item(p, (blockIdx.x % 8) * per + blockIdx.x / 8, it, chunk)) return;
  if (it.broken) {
    if (chunk == 0 && it.rt == 0) write_nan(p, it);
    return;
  }
  const int tk_begin = chunk * p.plan.chunk;
  const int tk_end = tk_begin + min(p.plan.chunk, it.total - tk_begin);
  if (it.rt * 32 * WAVES >= it.rows || tk_begin >= tk_end) return;
  run_item<DK, DV, SHARED, MX, WAVES>(p, it, lds, s_page, tk_begin, tk_end, p.plan.chunk);
}

// v of one lane (the same for all that ask), in scalar registers.
__device__ __forceinline__ int64_t of_lane(int64_t v, int lane) {
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
                   (uint32_t)__builtin_amdgcn_readlane((int)v, lane));
}

// Sum of v over the sequences before the thread's own, and over all of them.
// Up to 64 sequences every wave holds all of them; beyond, the workgroup's 256
// threads do.
__device__ __forceinline__ int64_t sum_before(int64_t v, int nseq, int64_t* lds, int64_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t inc = v;
  for (int d = 1; d < min(nseq, 64); d <<= 1) {
    const int64_t o = __shfl_up(inc, d);
    if (lane >= d) inc += o;
  }
  if (nseq <= 64) {
    all = of_lane(inc, nseq - 1);
    return inc - v;
  }
  if (lane == 63) lds[wave] = inc;
  __syncthreads();
  int64_t before = inc - v;
  all = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    before += w < wave ? lds[w] : 0;
    all += lds[w];
  }
  all = of_lane(all, 0);
  return before;
}

// Even plan: a workgroup a run of units. Every workgroup finds its first
// sequence from sums over all of them; the first one leaves the sums for the
// join.
template <bool MX>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
void tree_attn_even_kernel(AttnParams p) {
  using S = Shape<576, 512, true, MX, 4>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  __shared__ int s_page[MAX_CHUNK_PAGES + 8];  // and eight words of any_of
  __shared__ int64_t s_sum[2][4], s_base;
  __shared__ Item s_item;
  const int tid = threadIdx.x;
  Item it;
  // a run of sequences per thread
  const bool many = p.nseq > 64;
  const int per = many ? (p.nseq + 255) / 256 : 1, who = many ? tid : tid & 63;
  const int j0 = min(who * per, p.nseq), j1 = min(j0 + per, p.nseq);
  int64_t work = 0, all;  // steps (fewer than 2^42), and above them items (fewer than 2^21)
  int broken = 0;
  for (int j = j0; j < j1; ++j) {
    load_seq(p, j, it);
    const int64_t n = units_of(p, it, 0);
    work += n + (n ? (int64_t)(p.H_kv * row_tiles_of(it)) << 42 : 0);
    broken |= it.broken && it.n > 0;
  }
  sum_before(work, p.nseq, s_sum[0], all);
  const int64_t W = all & (((int64_t)1 << 42) - 1), all_items = all >> 42;
  if (many ? __syncthreads_or(broken) : __any(broken)) {
    Item bad;
    for (int j = blockIdx.x; j < p.nseq; j += gridDim.x) {
      load_seq_uniform(p, j, bad);
      if (bad.broken)
        for (bad.kvh = 0; bad.kvh < p.H_kv; ++bad.kvh) write_nan(p, bad);
    }
  }
  if (W == 0) return;
  int G = workgroups_for(p, W, all_items);
  const int quantum = quantum_for(W, all_items, G);
  int64_t mine = 0, units;
  for (int j = j0; j < j1; ++j) {
    if (per > 1) load_seq(p, j, it);  // (else `it` is that sequence)
    mine += units_of(p, it, quantum);
  }
  const int64_t before = sum_before(mine, p.nseq, s_sum[1], units);
  if (quantum) G = (int)units;
  const int64_t each_group = divide(units, G);
  const Share share{each_group, units - each_group * G};
  // consecutive runs go to one XCD: row tiles of a sequence share its L2
  const int runs = (G + 7) / 8;
  const int b = (blockIdx.x % 8) * runs + blockIdx.x / 8;
  if (blockIdx.x == 0 && p.plan.total > 0 && tid == who) {
    int64_t at = before;
    for (int j = j0; j < j1; ++j) {
      p.sums[3 + j] = at;
      if (per > 1) load_seq(p, j, it);
      at += units_of(p, it, quantum);
    }
    if (tid == 0) {
      p.sums[0] = share.each;
      p.sums[1] = share.more;
      p.sums[2] = quantum;
    }
  }
  if ((int)(blockIdx.x / 8) >= runs || b >= G) return;
  const int64_t begin = share.first(b), end = share.first(b + 1);
  int64_t base;  // units before the sequence
  const bool mine_first = before <= begin && begin < before + mine;
  if (!many) {
    const int lane = (int)__builtin_ctzll(__ballot(mine_first));
    it.j = lane;
    it.t0 = __builtin_amdgcn_readlane(it.t0, lane);
    it.n = __builtin_amdgcn_readlane(it.n, lane);
    it.seq = __builtin_amdgcn_readlane(it.seq, lane);
    it.len = __builtin_amdgcn_readlane(it.len, lane);
    it.broken = false;
    base = of_lane(before, lane);
  } else {
    if (mine_first) {
      int64_t at = before;
      for (int j = j0; j < j1; ++j) {
        if (per > 1) load_seq(p, j, it);
        const int64_t n = units_of(p, it, quantum);
        if (begin < at + n) {
          s_item = it;
          s_base = at;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
    it = s_item;
    base = of_lane(s_base, 0);
  }
  uniform(p, it);
  for (int64_t unit = begin; unit < end;) {
    const int tiles = tiles_of(it), each = units_of_item(it, quantum);
    const int64_t n = units_of(p, it, quantum);
    if (unit >= base + n) {  // on to the next sequence that has units
      base += n;
      if (it.j + 1 >= p.nseq) break;
      load_seq(p, it.j + 1, it);
      uniform(p, it);
      continue;
    }
    const int item = __builtin_amdgcn_readfirstlane((int)divide(unit - base, each));
    const int at = __builtin_amdgcn_readfirstlane((int)(unit - base - (int64_t)item * each));
    const bool uncut = quantum == 0 && tiles <= SHORT;
    if (uncut && at > 0) {  // the workgroup before has it
      unit += each - at;
      continue;
    }
    const int count = quantum ? 1 : uncut ? each : (int)min((int64_t)(each - at), end - unit);
    const int first = quantum ? (int)divide((int64_t)tiles * at, each) : at;
    const int last = quantum ? (int)divide((int64_t)tiles * (at + 1), each) : at + count;
    it.kvh = item / row_tiles_of(it);
    it.rt = item - it.kvh * row_tiles_of(it);
    it.whole = first == 0 && last == tiles;
    it.slot = 2 * b + (unit == begin ? 0 : 1);
    run_item<576, 512, true, MX, 4>(p, it, lds, s_page, first * TILE, min(last * TILE, it.total), p.plan.chunk);
    unit += count;
  }
}

// Joins the partial results of 32 query rows (a wave of a row tile): out = sum_c
// 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c over the parts c of the cache rows. A
// lane takes 4-element vectors of one query row. A workgroup's way to its first
// partial result is a chain of loads, so many of them should run at once: 1024
// row groups with 100 MB of partial results took 42 us in one block of 64 vectors
// each, 32 in four blocks of 16, 34 in eight. V = 4: four waves share
// `vectors_each` vectors, four in flight each. V = 1, for few rows with many
// parts: a wave takes one vector, and where the workgroup has more than four
// waves they share the parts and add up in LDS. The order of every sum is fixed. (The
// waves of a SIMD are those that out_of_range, which hardly runs, may not lower much.)
template <bool EVEN, int V>
__global__ __launch_bounds__(V == 1 ? 1024 : 256)
__attribute__((amdgpu_waves_per_eu(EVEN ? (V == 1 ? 8 : 6) : (V == 1 ? 7 : 5))))
void join_kernel(AttnParams p, int vectors_each) {
  const int waves = p.plan.waves, vectors = p.d_v / 8;
  const uint32_t blocks = (vectors + vectors_each - 1) / vectors_each;
  const uint32_t b = blockIdx.x / blocks;
  const int vb = (int)(blockIdx.x % blocks) * vectors_each;
  const int wave = (int)(b % waves);
  const uint32_t tile = b / waves;
  const uint32_t head = tile / p.plan.row_tiles;
  Item it;
  int chunk = 0, parts, first = 0;  // parts in order: slots at(0) .. at(parts - 1)
  int64_t slot0 = 0;
  if constexpr (EVEN) {
    it.kvh = (int)(head % p.H_kv);
    it.rt = (int)(tile % p.plan.row_tiles);
    const int j = (int)(head / p.H_kv);
    load_seq_uniform(p, j, it);
    if (it.broken || it.rt >= row_tiles_of(it)) return;
    const Share share{p.sums[0], p.sums[1]};
    const int quantum = (int)p.sums[2], each = units_of_item(it, quantum);
    if (quantum == 0 && each <= SHORT) return;
    const int64_t u0 = p.sums[3 + j] + (int64_t)(it.kvh * row_tiles_of(it) + it.rt) * each;
    // (the bounds keep a workspace that another call writes meanwhile from leading outside it)
    first = min(max(share.of(u0), 0), p.plan.groups - 1);
    parts = min(max(share.of(u0 + each - 1) - first, 0), p.plan.groups - 1 - first) + 1;
    if (parts == 1) return;  // the result is there
    slot0 = 2 * first + (share.first(first) < u0 ? 1 : 0);
  } else {
    if (!find_item(p, (int64_t)head * p.plan.chunks * p.plan.row_tiles + tile % p.plan.row_tiles, it, chunk)) return;
    if (it.broken || it.whole) return;
    parts = (it.total - 1) / p.plan.chunk + 1;
    slot0 = it.slot;
  }
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5, own = threadIdx.x >> 6;
  const int row = (it.rt * waves + wave) * 32 + l32;
  if ((it.rt * waves + wave) * 32 >= it.rows) return;
  // place of part c
  auto at = [&](int c) {
    const int64_t s = c == 0 ? slot0 : EVEN ? 2 * (int64_t)(first + c) : slot0 + (int64_t)c * p.plan.row_tiles;
    return s * waves + wave;
  };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + l32;
  const f32x4_t* po = reinterpret_cast<const f32x4_t*>(p.part_o) + lane;
  const bool live = row < it.rows;  // (partial results of other rows do not exist)
  const int i = live ? row / p.group : 0;
  const int h = it.kvh * p.group + (live ? row - i * p.group : 0);
  const int64_t t = it.t0 + i;
  // this wave's parts: their largest reference
  const int c1 = V == 1 ? own >> 2 : 0, step = V == 1 ? blockDim.x / 256 : 1;
  constexpr int U = V == 1 ? 8 : 4;  // parts at once
  float M = NEG_INF;
  if (live)
    for (int c0 = c1; c0 < parts; c0 += step * 8) {
      float e[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) e[u] = ml[at(min(c0 + step * u, parts - 1)) * 32].x;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (c0 + step * u < parts) M = fmaxf(M, e[u]);
    }
  const float Mu = M == NEG_INF ? 0.0f : M;
  __shared__ float sum[V == 1 ? 16 : 1][6][64];
  const int end = min(vb + vectors_each, vectors);
  const int v0 = __builtin_amdgcn_readfirstlane(vb + (own & 3));  // the wave's vectors: V from here on, four apart
  float l = 0;
  f32x4_t acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = f32x4_t{0, 0, 0, 0};
  if (live)
    for (int c0 = c1; c0 < parts; c0 += step * U) {
      float2 e[U];
      f32x4_t x[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t s = at(min(c0 + step * u, parts - 1));
        e[u] = ml[s * 32];
#pragma unroll
        for (int v = 0; v < V; ++v) x[u][v] = po[(s * vectors + min(v0 + 4 * v, end - 1)) * 64];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (c0 + step * u >= parts) break;
        const float w = exp2_hw(e[u].x - Mu);
        l += w * e[u].y;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[v][k] += w * x[u][v][k];
      }
    }
  float top = M;
  if (V == 1 && step > 1) {
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[own][k][lane] = acc[0][k];
    sum[own][4][lane] = l;
    sum[own][5][lane] = M;
    __syncthreads();
    if (own >= 4) return;
    for (int w = 1; w < step; ++w) top = fmaxf(top, sum[own + 4 * w][5][lane]);
    const float tu = top == NEG_INF ? 0.0f : top;
    const float f0 = exp2_hw(M - tu);
    l *= f0;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[0][k] *= f0;
    for (int w = 1; w < min(step, parts); ++w) {
      const float f = exp2_hw(sum[own + 4 * w][5][lane] - tu);
      l += f * sum[own + 4 * w][4][lane];
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[0][k] += f * sum[own + 4 * w][k][lane];
    }
  }
  const float inv = l == 0 ? 0.0f : 1.0f / l;
  float x = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) x = widest(widest(x, acc[v][0], acc[v][1]), acc[v][2], acc[v][3]);
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (live && v0 + 4 * v < end)
      *reinterpret_cast<uint2*>(p.out + t * p.o_t + h * p.o_h + 8 * (v0 + 4 * v) + 4 * half) =
          make_uint2(pack_bf16x2(acc[v][0] * inv, acc[v][1] * inv), pack_bf16x2(acc[v][2] * inv, acc[v][3] * inv));
  if (p.lse && live && v0 == 0 && half == 0)
    p.lse[t * p.H + h] = l == 0 ? NEG_INF : (top + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
  const uint64_t strange = __ballot(!(x < __builtin_huge_valf()) && l < __builtin_huge_valf());
  if (__builtin_expect(strange != 0, 0)) {
    const int at = (it.rt * waves + wave) * 32;
    const uint32_t rows = (uint32_t)(strange | strange >> 32);
    if (p.mx) out_of_range<0, true, V>(it, at, rows, v0, 4);
    else out_of_range<0, false, V>(it, at, rows, v0, 4);
  }
}

template <int DK, int DV, bool SHARED, bool MX>
void launch_shape(const AttnParams& p, unsigned grid, hipStream_t stream) {
  if (p.plan.waves == 1)
    hipLaunchKernelGGL((tree_attn_kernel<DK, DV, SHARED, MX, 1>), dim3(grid), dim3(64), 0, stream, p);
  else if (p.plan.waves == 2)
    hipLaunchKernelGGL((tree_attn_kernel<DK, DV, SHARED, MX, 2>), dim3(grid), dim3(128), 0, stream, p);
  else
    hipLaunchKernelGGL((tree_attn_kernel<DK, DV, SHARED, MX, 4>), dim3(grid), dim3(256), 0, stream, p);
}

template <int DK, int DV, bool SHARED>
void launch_dtype(const AttnParams& p, unsigned grid, hipStream_t stream) {
  if (p.mx) launch_shape<DK, DV, SHARED, true>(p, grid, stream);
  else launch_shape<DK, DV, SHARED, false>(p, grid, stream);
}

}  // namespace

hipError_t launch_tree_attn(const AttnParams& p, hipStream_t stream) {
  const int64_t tiles = (int64_t)p.nseq * p.H_kv * p.plan.row_tiles;
  const int64_t items = tiles * p.plan.chunks;
  if (items == 0 || p.T == 0) return hipSuccess;
  const unsigned grid = (unsigned)((items + 7) / 8 * 8);
  if (p.plan.groups > 0) {
    const dim3 g((unsigned)((p.plan.groups + 7) / 8 * 8));
    if (p.mx) hipLaunchKernelGGL(tree_attn_even_kernel<true>, g, dim3(256), 0, stream, p);
    else hipLaunchKernelGGL(tree_attn_even_kernel<false>, g, dim3(256), 0, stream, p);
  } else if (p.d_k == 96) launch_dtype<96, 64, true>(p, grid, stream);
  else if (p.d_k == 192) launch_dtype<192, 128, false>(p, grid, stream);
  else if (p.d_k == 128) launch_dtype<128, 128, false>(p, grid, stream);
  else launch_dtype<64, 64, false>(p, grid, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.plan.total == 0) return e;  // no item has parts
  // By the groups of 32 rows: many take 16 of their vectors in a workgroup; few
  // take four, and share parts (at most, or on average) over four times the waves.
  const int64_t groups = tiles * p.plan.waves;
  const int64_t parts = p.plan.groups > 0 ? p.plan.groups / tiles : p.plan.chunks;
  const int vectors = p.d_v / 8, each = groups >= 64 ? std::min(vectors, 16) : 4;
  const dim3 grid2((unsigned)(groups * ((vectors + each - 1) / each)));
  const dim3 threads(each == 4 && parts >= 16 ? 1024 : 256);
  if (p.plan.groups > 0) {
    if (each > 4) hipLaunchKernelGGL((join_kernel<true, 4>), grid2, threads, 0, stream, p, each);
    else hipLaunchKernelGGL((join_kernel<true, 1>), grid2, threads, 0, stream, p, each);
  } else {
    if (each > 4) hipLaunchKernelGGL((join_kernel<false, 4>), grid2, threads, 0, stream, p, each);
    else hipLaunchKernelGGL((join_kernel<false, 1>), grid2, threads, 0, stream, p, each);
  }
  return hipGetLastError();
}

}  // namespace mla
