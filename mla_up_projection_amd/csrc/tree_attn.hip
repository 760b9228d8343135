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
// The cache of a sequence is cut into chunks that different workgroups take;
// their (m, l, O) are joined by a second kernel in chunk order. A sequence of
// one chunk is finished at once.
#include <algorithm>

#include "device_common.h"
#include "internal_decode.h"

namespace mla {
namespace {

constexpr int TILE = 32;         // cache rows per step
constexpr int BLK = TILE * 128;  // LDS bytes of a 64-column block of a tile
constexpr int MAX_CHUNK_PAGES = 1024;
constexpr float LAZY = 8.0f;     // the maximum may lag by this many powers of two
constexpr float NEG_INF = -__builtin_huge_valf();

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// Position of 16-byte chunk c of cache row t within the row's 128 bytes. A row
// spans half the 64 banks, so rows t, t + 2, .. would share theirs; moving
// chunks by the bits of t above the lowest spreads the column reads of K (8
// consecutive rows, one chunk each) and the transposing reads of V (4 rows, 64
// bytes each) over all banks.
__device__ __forceinline__ int swz(int t) { return ((t >> 1) & 1) << 2 | ((t >> 2) & 1) << 1 | ((t >> 3) & 1); }

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// What a workgroup works on.
struct Item {
  int j, kvh, chunk, rt;
  int t0, n, rows;      // first query token, drafts, query rows (n * group)
  int len, total, seq;  // committed rows, with drafts
  int chunks;           // of this sequence
  bool broken;          // it outgrew the plan or its entry is invalid: NaN
};

__device__ __forceinline__ bool find_item(const AttnParams& p, int64_t item, Item& it) {
  it.rt = (int)(item % p.plan.row_tiles);
  item /= p.plan.row_tiles;
  it.chunk = (int)(item % p.plan.chunks);
  item /= p.plan.chunks;
  it.kvh = (int)(item % p.H_kv);
  it.j = (int)(item / p.H_kv);
  if (it.j >= p.nseq) return false;
  const int T = (int)p.T;
  it.t0 = min(max(p.cu[it.j], 0), T);
  it.n = min(max(p.cu[it.j + 1], it.t0), T) - it.t0;
  it.rows = it.n * p.group;
  it.seq = p.seqs[it.j];
  it.broken = it.seq < 0 || it.seq >= p.pool.max_seqs || it.n > p.max_q;
  it.len = it.broken ? 0 : p.pool.lens[it.seq];
  it.broken |= it.len < 0 || it.len > p.max_len - it.n;
  it.total = it.len + it.n;
  it.chunks = it.broken ? 1 : max(1, (it.total + p.plan.chunk - 1) / p.plan.chunk);
  return it.n > 0;
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

// bf16 pair with non-finite elements replaced by zero / by a code (+inf 1,
// -inf 64, NaN 4096, finite 0).
__device__ __forceinline__ uint32_t finite_pair(uint32_t v) {
  if ((v & 0x7F80u) == 0x7F80u) v &= 0xFFFF0000u;
  if ((v & 0x7F800000u) == 0x7F800000u) v &= 0xFFFFu;
  return v;
}
__device__ __forceinline__ uint32_t code16(uint32_t v) {
  if ((v & 0x7F80u) != 0x7F80u) return 0;
  return (v & 0x7Fu) ? 0x4580u : (v & 0x8000u) ? 0x4280u : 0x3F80u;  // bf16 of 4096, 64, 1
}
__device__ __forceinline__ uint32_t code_pair(uint32_t v) { return code16(v & 0xFFFFu) | code16(v >> 16) << 16; }

template <int DK, int DV, bool SHARED, bool MX, int WAVES>
struct Shape {
  static constexpr int NBK = (DK + 63) / 64, NBV = SHARED ? 0 : (DV + 63) / 64;
  static constexpr int KK = DK / 16, NT = DV / 32;
  static constexpr int LDS = (NBK + NBV) * BLK;
};

template <int DK, int DV, bool SHARED, bool MX, int WAVES>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(1, DV > 256 ? 1 : 4)))
void tree_attn_kernel(AttnParams p) {
  using S = Shape<DK, DV, SHARED, MX, WAVES>;
  constexpr int THREADS = 64 * WAVES;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  __shared__ int s_page[MAX_CHUNK_PAGES];
  __shared__ int s_bad;
  // consecutive items (row tiles that read the same chunk) go to one XCD's L2
  const int64_t per = gridDim.x / 8;
  Item it;
  if (!find_item(p, (blockIdx.x % 8) * per + blockIdx.x / 8, it)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l32 = lane & 31, half = lane >> 5;
  if (it.broken) {
    if (it.chunk == 0 && it.rt == 0) write_nan(p, it);
    return;
  }
  const int row0 = it.rt * 32 * WAVES;
  const int tk_begin = it.chunk * p.plan.chunk;
  const int tk_end = min(tk_begin + p.plan.chunk, it.total);
  if (row0 >= it.rows || tk_begin >= tk_end) return;

  // the chunk's pages
  const int ps = p.pool.page_size;
  const int page0 = tk_begin / ps, pages = (tk_end - 1) / ps - page0 + 1;
  const int held = min(p.pool.held[it.seq], p.pool.max_pages);
  if (tid == 0) s_bad = 0;
  __syncthreads();
  for (int k = tid; k < pages; k += THREADS) {
    int id = page0 + k < held ? p.pool.table[(int64_t)it.seq * p.pool.max_pages + page0 + k] : -1;
    if (id < 0 || id >= p.pool.num_pages) {
      id = -1;
      s_bad = 1;
    }
    s_page[k] = id;
  }

  // this lane's query row
  const int row = row0 + wave * 32 + l32;
  const bool live = row < it.rows;
  const int qi = live ? row / p.group : 0;
  const int64_t qt = it.t0 + qi;
  const int h = it.kvh * p.group + (live ? row - qi * p.group : 0);
  bf16x8_t q[S::KK];
#pragma unroll
  for (int kk = 0; kk < S::KK; ++kk)
    q[kk] = *reinterpret_cast<const bf16x8_t*>(p.q + qt * p.q_t + h * p.q_h + 16 * kk + 8 * half);
  f32x16_t o[S::NT];
#pragma unroll
  for (int n = 0; n < S::NT; ++n)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[n][i] = 0;
  float m = NEG_INF, l = 0;
  __syncthreads();
  const bool bad = s_bad;

  // LDS offsets: K fragment (row l32, chunk 2 (kk % 4) + half), V fragment
  // (rows 4 half + 0..3 of an 8-row group, 16 columns per 16 lanes)
  int koff[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) koff[c] = l32 * 128 + (((2 * c + half) ^ swz(l32)) << 4);
  const int q4 = lane & 15;
  int voff[2][2];  // [row 8 group][column half of the block]
#pragma unroll
  for (int e = 0; e < 2; ++e)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int t = 8 * e + 4 * half + (q4 >> 2);
      voff[e][c] = t * 128 + (((4 * c + 2 * ((lane >> 4) & 1) + ((q4 & 3) >> 1)) ^ swz(t)) << 4) + (q4 & 1) * 8;
    }
  const uint8_t* vlds = lds + (SHARED ? 0 : S::NBK * BLK);

  for (int tk = tk_begin; tk < tk_end; tk += TILE) {
    __syncthreads();  // the previous tile is read
    // stage: 16-byte chunk c of row r of block b; rows behind the chunk's end are zeros
    constexpr int CPR = DK / 8, VPR = SHARED ? 0 : DV / 8;  // 16-byte chunks per row
    for (int i = tid; i < TILE * (CPR + VPR); i += THREADS) {
      const bool isk = i < TILE * CPR;
      const int ii = isk ? i : i - TILE * CPR;
      const int cpr = isk ? CPR : VPR;
      const int r = ii / cpr, c = ii - r * cpr;
      const int tok = tk + r;
      u32x4_t v = {0, 0, 0, 0};
      if (tok < tk_end) {
        const int rel = tok - page0 * ps;
        const int pk = rel / ps;
        const int64_t page = max(s_page[pk], 0);
        const int in = rel - pk * ps;
        const int d = isk ? DK : DV;
        const int64_t crow = (page * ps + in) * p.H_kv + it.kvh;  // row of width d
        if (!MX) {
          v = *reinterpret_cast<const u32x4_t*>(p.pool.buf[isk ? 0 : 1] + (crow * d + 8 * c) * 2);
        } else {
          const uint2 code = *reinterpret_cast<const uint2*>(p.pool.buf[isk ? 0 : 2] + crow * d + 8 * c);
          const uint32_t sb = p.pool.buf[isk ? 1 : 3][crow * (d / 32) + c / 4];
          const float sc = __uint_as_float(sb ? sb << 23 : 0x00400000u);
          v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code.x, sc, false));
          v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code.x, sc, true));
          v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code.y, sc, false));
          v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(code.y, sc, true));
          if (sb == 0xFF) v = u32x4_t{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
        }
      }
      *reinterpret_cast<u32x4_t*>(lds + ((isk ? 0 : S::NBK) + c / 8) * BLK + r * 128 + (((c & 7) ^ swz(r)) << 4)) = v;
    }
    __syncthreads();
    // S^T: element i is cache row 8 (i / 4) + 4 half + i % 4, column the lane's query
    f32x16_t s;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 0;
#pragma unroll
    for (int kk = 0; kk < S::KK; ++kk) {
      const bf16x8_t k = *reinterpret_cast<const bf16x8_t*>(lds + (kk >> 2) * BLK + koff[kk & 3]);
      s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[kk], s, 0, 0, 0);
    }
    const bool masked = bad || tk + TILE > it.len;  // else every row sees the whole tile
    uint32_t vis = 0xFFFFFFFFu, nan_rows = 0;
    if (masked) {
      vis = visible(p, it, qt, qi, tk);
      if (tk_end - tk < TILE) vis &= (1u << (tk_end - tk)) - 1;
      if (bad)
        for (int r = 0; r < TILE && tk + r < tk_end; ++r)
          if (s_page[(tk + r - page0 * ps) / ps] < 0) nan_rows |= 1u << r;
    }
    float top = NEG_INF;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int b = 8 * (i / 4) + (i % 4);
      s[i] *= p.scale_log2;
      if (masked) {
        const uint32_t bit = 1u << (b + 4 * half);
        if (nan_rows & bit) s[i] = __builtin_nanf("");
        if (!(vis & bit)) s[i] = NEG_INF;
      }
      top = fmaxf(top, s[i]);
    }
    {
      const u32x2_t x = swap_halves(__float_as_uint(top), __float_as_uint(top));
      top = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
    }
    // The maximum is raised only when a row's grew by more than 2^LAZY: weights
    // stay below 2^LAZY, and O, 32 DV bits a row, is rarely rescaled.
    if (__any(top > m + LAZY || (m == NEG_INF && top > NEG_INF))) {
      const float mn = fmaxf(m, top);
      const float f = mn == NEG_INF ? 1.0f : exp2_hw(m - mn);
      m = mn;
      l *= f;
#pragma unroll
      for (int n = 0; n < S::NT; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[n][i] *= f;
    }
    const float mu = m == NEG_INF ? 0.0f : m;
    float sum = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = exp2_hw(s[i] - mu);
      sum += s[i];
    }
    l += sum;  // of this half's rows; the halves are added at the end
    // P^T for the two 16-row steps: weights rounded to bf16 (half a unit in
    // 2^-8 each, independent of each other, so the sum's error averages out)
    bf16x8_t pt[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const u32x4_t v = {pack_bf16x2(s[8 * c], s[8 * c + 1]), pack_bf16x2(s[8 * c + 2], s[8 * c + 3]),
                         pack_bf16x2(s[8 * c + 4], s[8 * c + 5]), pack_bf16x2(s[8 * c + 6], s[8 * c + 7])};
      pt[c] = __builtin_bit_cast(bf16x8_t, v);
    }
    uint32_t odd = 0;  // non-finite values in a tile that some rows do not see
#pragma unroll
    for (int n = 0; n < S::NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
        const uint8_t* base = vlds + (n >> 1) * BLK + c * 16 * 128;
        const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(base + voff[0][n & 1]));
        const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(base + voff[1][n & 1]));
        const uint2 ua = __builtin_bit_cast(uint2, a), ub = __builtin_bit_cast(uint2, b);
        u32x4_t v = {ua.x, ua.y, ub.x, ub.y};
        if (masked)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t f = finite_pair(v[k]);
            odd |= f ^ v[k];
            v[k] = f;
          }
        o[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, v), pt[c], o[n], 0, 0, 0);
      }
    if (__any(odd)) {
      // the non-finite values by themselves: counts of +inf, -inf and NaN among
      // the rows seen, in one sum (at most 32 of each), then added as such
      u32x4_t one[2];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int b0 = 8 * ((8 * c + 2 * k) / 4) + (2 * k) % 4 + 4 * half;
          one[c][k] = ((vis >> b0) & 1 ? 0x3F80u : 0) | ((vis >> (b0 + 1)) & 1 ? 0x3F800000u : 0);
        }
#pragma unroll
      for (int n = 0; n < S::NT; ++n) {
        f32x16_t cnt;
#pragma unroll
        for (int i = 0; i < 16; ++i) cnt[i] = 0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
          const uint8_t* base = vlds + (n >> 1) * BLK + c * 16 * 128;
          const uint2 ua = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(base + voff[0][n & 1])));
          const uint2 ub = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(base + voff[1][n & 1])));
          const u32x4_t v = {code_pair(ua.x), code_pair(ua.y), code_pair(ub.x), code_pair(ub.y)};
          cnt = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, v), __builtin_bit_cast(bf16x8_t, one[c]), cnt, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t k = (uint32_t)cnt[i];
          if (k >= 4096 || ((k & 63) && (k & 4032))) o[n][i] = __builtin_nanf("");
          else if (k & 63) o[n][i] += __builtin_huge_valf();
          else if (k) o[n][i] -= __builtin_huge_valf();
        }
      }
    }
  }
  {
    const u32x2_t x = swap_halves(__float_as_uint(l), __float_as_uint(l));
    l = __uint_as_float(x[0]) + __uint_as_float(x[1]);
  }
  if (it.chunks == 1) {
    const float inv = l == 0 ? 0.0f : 1.0f / l;
    if (live) {
      uint16_t* dst = p.out + qt * p.o_t + h * p.o_h;
#pragma unroll
      for (int n = 0; n < S::NT; ++n)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<uint2*>(dst + 32 * n + 8 * g + 4 * half) =
              make_uint2(pack_bf16x2(o[n][4 * g] * inv, o[n][4 * g + 1] * inv),
                         pack_bf16x2(o[n][4 * g + 2] * inv, o[n][4 * g + 3] * inv));
      if (p.lse && half == 0)
        p.lse[qt * p.H + h] = l == 0 ? NEG_INF : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
    }
    return;
  }
  // partial result, in register order: [slot][wave][32 DV floats as NT * 4 vectors of 64 lanes]
  const int64_t slot = ((((int64_t)it.j * p.H_kv + it.kvh) * p.plan.row_tiles + it.rt) * p.plan.chunks + it.chunk) * WAVES + wave;
  f32x4_t* po = reinterpret_cast<f32x4_t*>(p.part_o) + slot * (DV * 8);
#pragma unroll
  for (int n = 0; n < S::NT; ++n)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      po[(n * 4 + g) * 64 + lane] = f32x4_t{o[n][4 * g], o[n][4 * g + 1], o[n][4 * g + 2], o[n][4 * g + 3]};
  if (half == 0) reinterpret_cast<float2*>(p.part_ml)[slot * 32 + l32] = make_float2(m, l);
}

// Joins the chunks of a row tile's wave: out = sum_c 2^(m_c - M) O_c / sum_c
// 2^(m_c - M) l_c, chunk by chunk in order. A thread takes one 4-element vector
// of one query row in every chunk.
__global__ __launch_bounds__(256) void join_kernel(AttnParams p, int vec_blocks) {
  const int waves = p.plan.waves;
  int64_t b = blockIdx.x;
  const int vb = (int)(b % vec_blocks);
  b /= vec_blocks;
  const int wave = (int)(b % waves);
  b /= waves;
  Item it;
  // item numbering with the chunk left out
  const int64_t tile = b;
  const int64_t head = tile / p.plan.row_tiles;
  if (!find_item(p, head * p.plan.chunks * p.plan.row_tiles + tile % p.plan.row_tiles, it)) return;
  if (it.broken || it.chunks == 1) return;
  const int lane = threadIdx.x & 63, l32 = lane & 31, half = lane >> 5;
  const int v = vb * 4 + (threadIdx.x >> 6);  // vector of the row: 8-column group n * 4 + g
  const int row = (it.rt * waves + wave) * 32 + l32;
  if (v * 8 >= p.d_v || row >= it.rows) return;
  const int64_t slot0 = (tile * p.plan.chunks) * waves + wave;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + slot0 * 32 + l32;
  const f32x4_t* po = reinterpret_cast<const f32x4_t*>(p.part_o) + slot0 * (p.d_v * 8) + v * 64 + lane;
  float M = NEG_INF;
  for (int c = 0; c < it.chunks; ++c) M = fmaxf(M, ml[(int64_t)c * waves * 32].x);
  const float Mu = M == NEG_INF ? 0.0f : M;
  float l = 0;
  f32x4_t acc = {0, 0, 0, 0};
#pragma unroll 4
  for (int c = 0; c < it.chunks; ++c) {
    const float2 e = ml[(int64_t)c * waves * 32];
    const f32x4_t x = po[(int64_t)c * waves * (p.d_v * 8)];
    const float w = exp2_hw(e.x - Mu);
    l += w * e.y;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] += w * x[k];
  }
  const float inv = l == 0 ? 0.0f : 1.0f / l;
  const int i = row / p.group;
  const int h = it.kvh * p.group + row - i * p.group;
  const int64_t t = it.t0 + i;
  *reinterpret_cast<uint2*>(p.out + t * p.o_t + h * p.o_h + 8 * v + 4 * half) =
      make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  if (p.lse && v == 0 && half == 0)
    p.lse[t * p.H + h] = l == 0 ? NEG_INF : (M + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
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
  if (p.d_k == 576) launch_dtype<576, 512, true>(p, grid, stream);
  else if (p.d_k == 96) launch_dtype<96, 64, true>(p, grid, stream);
  else if (p.d_k == 192) launch_dtype<192, 128, false>(p, grid, stream);
  else if (p.d_k == 128) launch_dtype<128, 128, false>(p, grid, stream);
  else launch_dtype<64, 64, false>(p, grid, stream);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.plan.chunks == 1) return e;
  const int vec_blocks = (p.d_v / 8 + 3) / 4;
  hipLaunchKernelGGL(join_kernel, dim3((unsigned)(tiles * p.plan.waves * vec_blocks)), dim3(256), 0, stream, p, vec_blocks);
  return hipGetLastError();
}

}  // namespace mla
