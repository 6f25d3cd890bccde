// Attention of packed queries over a paged cache in e4m3 (cache.hip), with grouped heads:
//
//   o[t, h] = sum_j p_j v[j] / sum_j p_j,  p_j = exp(scale * (q[t, h] . k[j] - m)),
//
// j over the keys 0 .. L - 1 of t's sequence; causal: the sequence's n queries are its last tokens, and query i
// takes j <= L - n + i. A row without keys is zero.
//
// The rows of a sequence and key head are its queries times the G = H / Hk heads of the group, head
// fastest: row r is head r % G of query r / G, so that all of them share the keys that are read. Scores
// are computed transposed, S^T = K Q^T, so that a lane holds scores of one row and passes its probabilities to
// O^T = V^T P^T without leaving the lane. Codes become bf16 exactly, times their page's power of two, by one
// conversion for two. Probabilities are rounded to bf16 for the second product (as in attention.hip),
// their sum is taken before that.
//
// Two kernels: few rows (up to 16 at a time) stream the keys from memory into operands; many rows
// share tiles of 64 keys in LDS. In both, keys may be split among workgroups, whose results
// join_kernel weighs together.
#include "cache.h"

#include <math.h>

namespace svdq {

namespace {

typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kTile = 64;             // keys of a step
constexpr int kLeastTiles = 2;        // of a split
constexpr float kSlackC = 8.0f;       // powers of two that a score may pass the running maximum by
constexpr float kLowest = -3.4028234663852886e38f;

__device__ __forceinline__ bf16x8 bf16_operand(uint32_t lo, uint32_t hi, float scale) {   // 8 codes
  return __builtin_bit_cast(bf16x8, u32x4{fp8_pair_to_bf16<0>(lo, scale), fp8_pair_to_bf16<1>(lo, scale),
                                          fp8_pair_to_bf16<0>(hi, scale), fp8_pair_to_bf16<1>(hi, scale)});
}

// Rows are numbered in blocks of 2^lg: sequence b's start at floor(cu[b] G / 2^lg) + b, which leaves at most
// one unused number per sequence. Finds the sequence of block t; false where there is none.
struct RowBlock {
  int b, tok0, n;   // sequence, its first packed query and its queries
  int row0;         // first row of the block within the sequence
};
__device__ __forceinline__ bool find_rows(const AttnCacheArgs& a, int G, int lg, int64_t t, RowBlock& o) {
  int b, c0, c1;
  if (a.cu == nullptr) {   // a query each: G rows
    const int per = (G + (1 << lg) - 1) >> lg;
    b = (int)(t / per);
    o = RowBlock{b, b, 1, (int)(t - (int64_t)b * per) << lg};
    return b < a.B;
  }
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = a.B;
  while (true) {
    const int step = (hi - lo + 63) / 64;
    const int idx = lo + lane * step;
    const int64_t c = min(max(a.cu[min(idx, a.B)], 0), (int)a.T);
    const int n = __popcll(__ballot(idx < hi && ((c * G) >> lg) + idx <= t));
    if (n == 0) return false;
    lo += (n - 1) * step;
    if (step == 1) break;
    hi = min(hi, lo + step);
  }
  b = lo;
  c0 = min(max(a.cu[b], 0), (int)a.T);
  c1 = min(max(a.cu[b + 1], 0), (int)a.T);
  const int64_t local = t - (((int64_t)c0 * G) >> lg) - b;
  if (local < 0 || c1 <= c0 || (local << lg) >= (int64_t)(c1 - c0) * G) return false;
  o = RowBlock{b, c0, c1 - c0, (int)(local << lg)};
  return true;
}

// The same for at most 64 sequences, those with the most keys first, so that the longest do not start last: a lane has a
// sequence, whose blocks follow those of longer ones (of equal ones before it).
__device__ __forceinline__ bool find_rows_longest_first(const AttnCacheArgs& a, int G, int lg, int t, RowBlock& o) {
  const int lane = threadIdx.x & 63, b = min(lane, a.B - 1);
  const int c0 = min(max(a.cu[b], 0), (int)a.T), c1 = min(max(a.cu[b + 1], 0), (int)a.T);
  const int keys = a.lengths[b], n = max(c1 - c0, 0);
  const int blocks = lane < a.B ? (int)(((int64_t)n * G + (1 << lg) - 1) >> lg) : 0;
  int at = 0;
  for (int i = 0; i < a.B; ++i) {
    const int other = __builtin_amdgcn_readlane(keys, i);
    if (other > keys || (other == keys && i < lane)) at += __builtin_amdgcn_readlane(blocks, i);
  }
  const uint64_t mine = __ballot(t >= at && t - at < blocks);
  if (mine == 0) return false;
  const int l = __builtin_ctzll(mine);
  o = RowBlock{l, __builtin_amdgcn_readlane(c0, l), __builtin_amdgcn_readlane(n, l),
               (t - __builtin_amdgcn_readlane(at, l)) << lg};
  return true;
}

// keys of a sequence: what its table can hold at most
__device__ __forceinline__ int64_t keys_of(const AttnCacheArgs& a, int b) {
  return min((int64_t)max(a.lengths[b], 0), a.width << a.c.lg_page);
}
// tiles of 64 keys that a split takes, and how many splits have any
__device__ __forceinline__ int tiles_per_split(const AttnCacheArgs& a, int64_t L) {
  const int tiles = (int)((L + kTile - 1) / kTile);
  return max((tiles + a.splits - 1) / a.splits, kLeastTiles);
}

// sum or maximum over the four lanes l16, l16 + 16, .. of a row
template <bool MAX>
__device__ __forceinline__ float across_rows(float v) {
  const Pair p = halves16(v);
  v = MAX ? fmaxf(p.a, p.b) : p.a + p.b;
  const Pair r = halves32(v);
  return MAX ? fmaxf(r.a, r.b) : r.a + r.b;
}

// Few rows. The four waves of a workgroup take 16 rows together, steps of 64 keys in turn; a step's operands
// come straight from memory in 16-byte pieces:
//  S^T: tile t of four holds key 16 (i / 4) + 4 t + i % 4 in matrix row i, so that lane (row, q) receives the
//       scores of keys 16 q .. 16 q + 15 of the step;
//  O^T: the same 16 keys of an element of v are one piece of the transposed page.
// Bound by the cache's bytes: one token on 65537 keys, 32 heads on 8 of 128 (134 MB) 28 us and 4 to join 32 splits (4.8 TB/s
// in the kernel); 32 tokens on 2500 keys each on average (164 MB) 40 and 5, unsplit 42.
constexpr int kWavesF = 4;

template <int D>
__global__ __launch_bounds__(64 * kWavesF, D == 64 ? 4 : 2) void attention_few_kernel(AttnCacheArgs a) {
  constexpr int KP = D / 64;      // 16-byte pieces of a key per lane
  constexpr int JD = D / 16;      // 16-element blocks of the output
  __shared__ float sm[kWavesF][2][16];
  __shared__ __attribute__((aligned(16))) float so[kWavesF][16][D + 4];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int q = lane >> 4, l16 = lane & 15;
  const int G = a.H / a.c.Hk, P = 1 << a.c.lg_page;
  const int split = (int)(blockIdx.x % (unsigned)a.splits);
  const int hk = (int)blockIdx.y;
  RowBlock rb;
  if (!find_rows(a, G, 4, (int64_t)(blockIdx.x / (unsigned)a.splits), rb)) return;
  const int64_t L = keys_of(a, rb.b);
  const int per = tiles_per_split(a, L);
  const bool only = (L + kTile - 1) / kTile <= per;   // one split takes all the keys
  if (split > 0 && (int64_t)split * per * kTile >= L) return;

  // this lane's row; rows past the block's repeat its last
  const int rows = min(16, rb.n * G - rb.row0);
  const int row = rb.row0 + min(l16, rows - 1);
  const int query = row / G, head = hk * G + row % G;
  // keys up to `last` for this row, `end` for any of the block
  const int64_t last = a.causal ? L - rb.n + query : L - 1;
  const int64_t end = a.causal ? L - rb.n + (rb.row0 + rows - 1) / G + 1 : L;
  const int64_t k_begin = (int64_t)split * per * kTile, k_end = min(end, k_begin + (int64_t)per * kTile);

  bf16x8 fq[2 * KP];
  const uint16_t* qp = a.q.p + (int64_t)(rb.tok0 + query) * a.q.st + head * a.q.sh + 16 * q;
#pragma unroll
  for (int s = 0; s < 2 * KP; ++s) fq[s] = *reinterpret_cast<const bf16x8*>(qp + 64 * (s >> 1) + 8 * (s & 1));

  const int32_t* table = a.table + (int64_t)rb.b * a.width;
  const int64_t page_bytes = (int64_t)P * D;
  auto entry_of = [&](int64_t key) {   // the table's entry for a key, looked at when it is used: not waited for here
    const int64_t at = key >> a.c.lg_page;
    return at < a.width ? table[at] : -1;
  };
  auto page_of = [&](int entry) { return (uint32_t)entry < (uint32_t)a.c.pages ? entry : -1; };   // -1: none

  f32x4 acc[JD];
#pragma unroll
  for (int j = 0; j < JD; ++j) acc[j] = f32x4{};
  const float c = a.scale * 1.4426950408889634f;   // exponents in base 2
  // The maximum starts at the least finite score, not the least whose power of two is finite: only differences are
  // taken times c, and a row whose scores all lie below -2^128 / c has its best key too
  float m = kLowest, l = 0.0f;
  const float slack = kSlackC / c;
  bool first = true;

  // A step's codes are requested while the step before is computed (keys as soon as its scores are there, values after
  // its second product), their pages a step earlier still.
  // This lane's pieces: keys kk + 4 t of the step, values of its keys kv .. kv + 15
  const int kk = 16 * (l16 >> 2) + (l16 & 3), kv = 16 * q;
  const int64_t k_first = k_begin + kTile * wave;
  constexpr int kStride = kTile * kWavesF;
  u32x4 wk[4][KP], wv[JD];
  uint32_t ks, vs;                          // scales
  bool k_gone = false, v_gone = false;      // no page
  int ek = entry_of(k_first + kk), ev = entry_of(k_first + kv);
  auto request_k = [&](int64_t k0) {
    const int pk = page_of(ek);
    k_gone = pk < 0;
    const int64_t at = (int64_t)max(pk, 0) * a.c.Hk + hk;
    const uint8_t* p = a.c.k + at * page_bytes + (((int)k0 + kk) & (P - 1)) * D + 16 * q;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int u = 0; u < KP; ++u) wk[t][u] = *reinterpret_cast<const u32x4*>(p + 4 * t * D + 64 * u);
    ks = a.c.ks[at];
  };
  auto request_v = [&](int64_t k0) {
    const int pv = page_of(ev);
    v_gone = pv < 0;
    const int64_t at = (int64_t)max(pv, 0) * a.c.Hk + hk;
    const uint8_t* p = a.c.v + at * page_bytes + l16 * P + (((int)k0 + kv) & (P - 1));
#pragma unroll
    for (int j = 0; j < JD; ++j) wv[j] = *reinterpret_cast<const u32x4*>(p + 16 * j * P);
    vs = a.c.vs[at];
  };
  if (k_first < k_end) {
    const int ek1 = entry_of(k_first + kStride + kk), ev1 = entry_of(k_first + kStride + kv);
    request_k(k_first);
    request_v(k_first);
    ek = ek1;
    ev = ev1;
  }
  for (int64_t k0 = k_first; k0 < k_end; k0 += kStride) {
    f32x4 x[4];
    {
      if (k_gone) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int u = 0; u < KP; ++u) wk[t][u] = zero4();
      }
      const float sc = k_gone ? 1.0f : cache_scale(ks);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        x[t] = f32x4{};
#pragma unroll
        for (int u = 0; u < KP; ++u) {
          x[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_operand(wk[t][u][0], wk[t][u][1], sc), fq[2 * u], x[t], 0, 0, 0);
          x[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_operand(wk[t][u][2], wk[t][u][3], sc), fq[2 * u + 1], x[t], 0, 0, 0);
        }
      }
    }
    const bool more = k0 + kStride < k_end;
    if (more) {
      request_k(k0 + kStride);
      ek = entry_of(k0 + 2 * kStride + kk);
    }
    float mx = -__builtin_inff();
    if (k0 + kTile > last + 1) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (k0 + kv + 4 * t + r > last) x[t][r] = -__builtin_inff();
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) mx = fmaxf(mx, x[t][r]);
    if (__ballot(mx > m + slack) != 0 || first) {
      const float mn = fmaxf(m, across_rows<true>(mx));
      const float alpha = __builtin_amdgcn_exp2f((m - mn) * c);
      m = mn;
      l *= alpha;
#pragma unroll
      for (int j = 0; j < JD; ++j) acc[j] *= alpha;
      first = false;
    }
    uint32_t p[8];
    float sum = 0.0f;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; r += 2) {
        const float p0 = __builtin_amdgcn_exp2f((x[t][r] - m) * c), p1 = __builtin_amdgcn_exp2f((x[t][r + 1] - m) * c);
        sum += p0 + p1;
        p[2 * t + r / 2] = pack_bf16x2(p0, p1);
      }
    l += sum;
    const bf16x8 fp0 = __builtin_bit_cast(bf16x8, u32x4{p[0], p[1], p[2], p[3]});
    const bf16x8 fp1 = __builtin_bit_cast(bf16x8, u32x4{p[4], p[5], p[6], p[7]});
    // values past the sequence, or without a page, are zero: their probabilities are, but what
    // the page holds there may be NaN
    const int64_t left = v_gone ? 0 : L - k0 - kv;
    const float sc = left <= 0 ? 1.0f : cache_scale(vs);
    if (left < 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = (int)max(min(left - 4 * i, (int64_t)4), (int64_t)0);
        const uint32_t keep = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
#pragma unroll
        for (int j = 0; j < JD; ++j) wv[j][i] &= keep;
      }
    }
#pragma unroll
    for (int j = 0; j < JD; ++j) {
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_operand(wv[j][0], wv[j][1], sc), fp0, acc[j], 0, 0, 0);
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_operand(wv[j][2], wv[j][3], sc), fp1, acc[j], 0, 0, 0);
    }
    if (more) {
      request_v(k0 + kStride);
      ev = entry_of(k0 + 2 * kStride + kv);
    }
  }

  // the waves' results together: each relative to its own maximum
  l = across_rows<false>(l);
  if (q == 0) {
    sm[wave][0][l16] = m;
    sm[wave][1][l16] = l;
  }
#pragma unroll
  for (int j = 0; j < JD; ++j) *reinterpret_cast<f32x4*>(&so[wave][l16][16 * j + 4 * q]) = acc[j];
  __syncthreads();
  constexpr int kPer = 16 * D / (64 * kWavesF);   // elements of the output per thread: 8 or 4
  const int r = tid * kPer / D, e0 = tid * kPer % D;
  if (r >= rows) return;
  float M = sm[0][0][r];
#pragma unroll
  for (int w = 1; w < kWavesF; ++w) M = fmaxf(M, sm[w][0][r]);
  float total = 0.0f, o[kPer] = {};
#pragma unroll
  for (int w = 0; w < kWavesF; ++w) {
    const float f = __builtin_amdgcn_exp2f((sm[w][0][r] - M) * c);
    total += sm[w][1][r] * f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] += so[w][r][e0 + e] * f;
  }
  const int orow = rb.row0 + r, otok = rb.tok0 + orow / G, ohead = hk * G + orow % G;
  if (only) {
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    uint32_t w[kPer / 2];
#pragma unroll
    for (int e = 0; e < kPer; e += 2) w[e / 2] = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
    uint16_t* dst = a.o + (int64_t)otok * a.o_st + ohead * a.o_sh + e0;
    if constexpr (kPer == 8) *reinterpret_cast<u32x4*>(dst) = u32x4{w[0], w[1], w[2], w[3]};
    else *reinterpret_cast<u32x2*>(dst) = u32x2{w[0], w[1]};
  } else {
    const int64_t at = ((int64_t)split * a.T + otok) * a.H + ohead;
    float* dst = a.partial + at * D + e0;
#pragma unroll
    for (int e = 0; e < kPer; e += 4) *reinterpret_cast<f32x4*>(dst + e) = f32x4{o[e], o[e + 1], o[e + 2], o[e + 3]};
    if (e0 == 0) {
      float* st = a.partial + (int64_t)a.splits * a.T * a.H * D + 2 * at;
      st[0] = M;
      st[1] = total;
    }
  }
}

// Many rows: 2048 queries on 16896 keys, 30 heads of 128, 550 us in a loop (0.97 PFLOP/s; a bf16 library product reaches
// 1.39), 600 to 635 in the first calls after an idle time (0.84 to 0.89). Matrix and vector units are busy 43% of the time each; without the conversions it is 6% faster, without the
// exponentials 5, without the writes to LDS 13, without the loads 14. Measured and not kept: eight waves with 256 rows
// (slower at every size), conversions between the second product's instructions, three to six reads ahead, other priorities.
// A workgroup of four waves takes 128 rows, 32 a wave, and tiles of 64 keys in LDS: codes travel
// to registers a step ahead, become bf16 and are written to LDS before the next step's barrier. K^T's tile is
// [64][D]; V^T's is [D][64] with each 16 keys in the order of P^T's operand (0-3, 8-11 for the lower half of the
// wave, 4-7, 12-15 for the upper), so that both products read whole 16-byte pieces. Products,
// exponentials and the lazy maximum are arranged as in attention.hip.
// A wave's piece of K is 8 or 16 keys, all in one page; its piece of V is 16 keys of 64 elements (pages of 16 or 32), or with
// WHOLE (pages of 64 or 128: a tile lies in one page) 64 keys of 16 elements, whose rows are read 64 bytes at a time. So
// a page's address and scale are scalar throughout, and a page that the table does not have is a buffer of no bytes,
// which reads zero. Per lane instead: 97 us for 4099 packed queries on 16-token pages, 85 on 64-token ones.
constexpr int kWavesT = 4, kLgRows = 7;
static_assert(kWavesT * 32 == 1 << kLgRows, "32 rows a wave");
constexpr int kAheadC = 2;   // operand reads in flight ahead of a product

__device__ __forceinline__ u32x4 load_codes(__amdgpu_buffer_rsrc_t r, int voff, int soff) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, 0));
}

template <int D, bool CAUSAL, bool WHOLE>
__global__ __launch_bounds__(64 * kWavesT, 2) void attention_tile_kernel(AttnCacheArgs a) {
  constexpr int kRowBytes = 2 * D;
  constexpr int kTileBytes = kTile * kRowBytes;     // of K, and of V
  constexpr int KD = D / 16;                        // 16-element steps of the first product
  constexpr int JD = D / 32;                        // 32-element blocks of the output
  constexpr int kCP = D / 16;                       // 16-byte pieces of a key's codes
  constexpr int kPieces = kTile * kCP / (64 * kWavesT);  // of a tile, per thread; as many of V
  __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * kTileBytes];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int h = lane >> 5, l32 = lane & 31;
  const int G = a.H / a.c.Hk, lg_page = a.c.lg_page, P = 1 << lg_page;

  // row blocks of one head stay on one XCD (its L2 holds their keys)
  const int per_xcd = (int)(gridDim.x / 8);
  const int id = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
  const int blocks = (int)((a.T * G) >> kLgRows) + a.B;
  if (id >= blocks * a.splits * a.c.Hk) return;
  const int hk = id / (blocks * a.splits);
  const int split = id % (blocks * a.splits) / blocks;
  RowBlock rb;
  const int block = id % blocks;
  if (a.cu != nullptr && a.B <= 64 ? !find_rows_longest_first(a, G, kLgRows, block, rb) : !find_rows(a, G, kLgRows, block, rb))
    return;
  const int n_rows = rb.n * G;
  if (CAUSAL) {   // those with the most keys first
    const int last_block = (n_rows - 1) >> kLgRows;
    rb.row0 = (last_block << kLgRows) - rb.row0;
  }
  const int L = __builtin_amdgcn_readfirstlane((int)keys_of(a, rb.b));
  const int per = tiles_per_split(a, L);
  const bool only = (L + kTile - 1) / kTile <= per;
  if (split > 0 && (int64_t)split * per * kTile >= L) return;

  // this wave's rows, this lane's row (past the end: the last) and the keys it sees
  const int row0 = rb.row0 + 32 * wave;
  const int row = min(row0 + l32, n_rows - 1);
  const int query = row / G, head = hk * G + row - query * G;
  const int off = L - rb.n;                                  // causal: query i sees keys up to off + i
  const int last = CAUSAL ? off + query : L - 1;
  // keys up to `low` are seen by every row of the wave, none past `high` by any
  const int low = CAUSAL ? off + min(row0, n_rows - 1) / G : L - 1;
  const int high = CAUSAL ? off + min(row0 + 31, n_rows - 1) / G : L - 1;
  const int wg_high = CAUSAL ? off + min(rb.row0 + 32 * kWavesT - 1, n_rows - 1) / G : L - 1;
  const int kt0 = split * per;
  const int nt = max(min((wg_high >> 6) + 1, kt0 + per) - kt0, 0);              // tiles of the workgroup (>> of -1 is -1)
  const int ntw = row0 < n_rows ? max(min((high >> 6) + 1, kt0 + per) - kt0, 0) : 0;   // and of this wave

  bf16x8 fq[KD];
  {
    const uint16_t* qp = a.q.p + (int64_t)(rb.tok0 + query) * a.q.st + head * a.q.sh + 8 * h;
#pragma unroll
    for (int t = 0; t < KD; ++t) fq[t] = *reinterpret_cast<const bf16x8*>(qp + 16 * t);
  }

  // Pieces of 16 codes: of K, key kr and elements 16 ks .. (piece c: kStepK keys further on); of V, element vd and keys
  // 16 vk .. (kStepV elements further on). The LDS swizzles repeat with those steps.
  auto swz_k = [](int r) { return D == 128 ? (r & 15) : ((r >> 1) & 7); };
  auto swz_v = [](int r) { return (r ^ (r >> 3)) & 7; };
  constexpr int kStepK = 64 * kWavesT / kCP, kStepV = 16 * kWavesT;
  static_assert(kStepK % 16 == 0 && kStepV % 64 == 0, "swizzles");
  constexpr int kRowsK = 64 / kCP;                    // keys of a wave's piece
  const int kr = tid / kCP, ks = tid % kCP;
  const int vd = WHOLE ? tid >> 2 : lane, vk = WHOLE ? tid & 3 : wave;
  const int k_src = (lane / kCP) * D + 16 * ks;       // from the wave's first key
  const int v_src = vd * P + (WHOLE ? 16 * vk : 0);   // from the tile's (WHOLE) or the wave's first key
  const int k_dst = kr * kRowBytes + (((2 * ks) ^ swz_k(kr)) * 16), v_dst = vd * 128 + (((2 * vk) ^ swz_v(vd)) * 16);
  const int32_t* table = a.table + (int64_t)rb.b * a.width;
  const uint32_t page_bytes = (uint32_t)(P * D);
  auto entry_of = [&](int key) {   // the table's entry for a key, looked at when it is used: not waited for here
    const int at = key >> lg_page;
    return at < a.width && key < L ? table[at] : -1;
  };
  auto page_of = [&](int entry) {   // -1: none
    entry = __builtin_amdgcn_readfirstlane(entry);
    return (uint32_t)entry < (uint32_t)a.c.pages ? entry : -1;
  };
  u32x4 wk[kPieces], wv[kPieces];        // codes on their way
  // Table entries of the pieces to be requested next; the scales of those on their way and which have no page (bit c of
  // `gone`). What a load brings is looked at a step later, not where it is requested.
  constexpr int kOwn = WHOLE ? 1 : kPieces;
  int ek[kOwn], ev, gone_k = 0, gone_v = 0;
  uint32_t sk[kOwn], sv;
  auto first_k = [&](int kt, int c) { return (kt0 + kt) * kTile + kRowsK * wave + kStepK * c; };
  auto first_v = [&](int kt) { return (kt0 + kt) * kTile + (WHOLE ? 0 : 16 * wave); };
  auto k_pages = [&](int kt) {
#pragma unroll
    for (int c = 0; c < kOwn; ++c) ek[c] = entry_of(WHOLE ? (kt0 + kt) * kTile : first_k(kt, c));
  };
  auto v_pages = [&](int kt) { ev = entry_of(first_v(kt)); };
  auto request_k = [&](int kt, u32x4 (&wk)[kPieces], uint32_t (&sk)[kOwn], int& gone_k) {
    gone_k = 0;
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      const int page = page_of(ek[o]);
      const int64_t at = (int64_t)max(page, 0) * a.c.Hk + hk;
      const __amdgpu_buffer_rsrc_t r = make_rsrc(a.c.k + at * page_bytes, page < 0 ? 0u : page_bytes);
#pragma unroll
      for (int c = WHOLE ? 0 : o; c < (WHOLE ? kPieces : o + 1); ++c)
        wk[c] = load_codes(r, k_src, (first_k(kt, c) & (P - 1)) * D);
      sk[o] = a.c.ks[at];
      gone_k |= (page < 0 ? 1 : 0) << o;
    }
  };
  auto request_v = [&](int kt) {
    const int page = page_of(ev);
    const int64_t at = (int64_t)max(page, 0) * a.c.Hk + hk;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(a.c.v + at * page_bytes, page < 0 ? 0u : page_bytes);
#pragma unroll
    for (int c = 0; c < kPieces; ++c) wv[c] = load_codes(r, v_src, (first_v(kt) & (P - 1)) + kStepV * P * c);
    sv = a.c.vs[at];
    gone_v = page < 0;
  };
  auto store_k = [&](int kt, const u32x4 (&wk)[kPieces], const uint32_t (&sk)[kOwn], int gone_k) {
    uint8_t* st = smem + (kt & 1) * (2 * kTileBytes);
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      const int o = WHOLE ? 0 : c;
      const float sc = (gone_k >> o) & 1 ? 1.0f : cache_scale((uint32_t)__builtin_amdgcn_readfirstlane((int)sk[o]));
      const u32x4 w = wk[c];
      *reinterpret_cast<bf16x8*>(st + k_dst + kStepK * kRowBytes * c) = bf16_operand(w[0], w[1], sc);
      *reinterpret_cast<bf16x8*>(st + (k_dst ^ 16) + kStepK * kRowBytes * c) = bf16_operand(w[2], w[3], sc);
    }
  };
  auto store_v = [&](int kt) {
    uint8_t* st = smem + (kt & 1) * (2 * kTileBytes) + kTileBytes;
    const int end = L - (kt0 + kt) * kTile;            // keys of the tile: values past the sequence are zero,
    if (end < kTile) {                                 // whatever the page holds
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = max(min(end - 16 * vk - 4 * e, 4), 0);
        const uint32_t keep = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
#pragma unroll
        for (int c = 0; c < kPieces; ++c) wv[c][e] &= keep;
      }
    }
    const float sc = gone_v ? 1.0f : cache_scale((uint32_t)__builtin_amdgcn_readfirstlane((int)sv));
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      const u32x4 w = wv[c];
      *reinterpret_cast<bf16x8*>(st + v_dst + kStepV * 128 * c) = bf16_operand(w[0], w[2], sc);
      *reinterpret_cast<bf16x8*>(st + (v_dst ^ 16) + kStepV * 128 * c) = bf16_operand(w[1], w[3], sc);
    }
  };

  // operand u of the first product (keys 32 (u % 2) of the tile, elements 16 (u / 2) of the head), and of the second
  // (keys 16 (u / JD), elements 32 (u % JD))
  // pieces 2 t + h, permuted by an exclusive or: that of t applies to the address of t = 0. Row 32 j + l32 of V^T is
  // permuted like row l32, with 4 j more
  const int kfrag = l32 * kRowBytes + ((h ^ swz_k(l32)) * 16), vfrag = l32 * 128 + ((h ^ swz_v(l32)) * 16);
  auto read_k = [&](const uint8_t* sk_, int u) {
    return *reinterpret_cast<const bf16x8*>(sk_ + 32 * (u & 1) * kRowBytes + (kfrag ^ (32 * (u >> 1))));
  };
  auto read_v = [&](const uint8_t* sv_, int u) {
    return *reinterpret_cast<const bf16x8*>(sv_ + 32 * (u % JD) * 128 + (vfrag ^ (32 * (u / JD)) ^ (((u % JD) & 1) * 64)));
  };
  constexpr int NK = 2 * KD, NV = 4 * JD;   // products of a tile

  f32x16 acc[JD];
#pragma unroll
  for (int j = 0; j < JD; ++j) acc[j] = f32x16{};
  // exponents in base 2, x c - mc, and scores far from zero, as in attention.hip; the maximum starts as for few rows
  // (its product with c may be infinite, which is `far`)
  const float c = a.scale * 1.4426950408889634f;
  float m = kLowest, mc = 0.0f;
  bool far = true;   // the same in every lane
  const float slack = kSlackC / c;
  // a tile's probabilities first, then l with what its last addition lost, as in attention.hip
  float l = 0.0f, lost = 0.0f, tile_sum = 0.0f;
  auto add_tile = [&] {
    const float y = tile_sum - lost, t = l + y;
    lost = (t - l) - y;
    l = t;
    tile_sum = 0.0f;
  };
  auto pair = [&](const f32x16 (&x)[2], uint32_t (&p)[16], int r) {
    const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r >> 3][2 * (r & 7)], c, -mc));
    const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r >> 3][2 * (r & 7) + 1], c, -mc));
    p[r] = pack_bf16x2(p0, p1);
    tile_sum += p0 + p1;
    asm volatile("" : "+v"(p[r]), "+v"(tile_sum));   // made here: not moved to their use
  };
  auto prob_operand = [&](const uint32_t (&p)[16], int t) {
    return __builtin_bit_cast(bf16x8, u32x4{p[4 * t], p[4 * t + 1], p[4 * t + 2], p[4 * t + 3]});
  };
  auto mask = [&](f32x16 (&x)[2], int kt) {
    const int k0 = (kt0 + kt) * kTile;
    if (k0 + kTile - 1 > low) {
      const int lim = last - k0 - 4 * h;
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        if (32 * (r >> 4) + 8 * ((r & 15) >> 2) + (r & 3) > lim) x[r >> 4][r & 15] = -__builtin_inff();
        if (r % 8 == 7) __builtin_amdgcn_sched_barrier(0);   // few condition registers at a time
      }
    }
  };
  auto raise = [&](float mx) {
    const Pair both = halves32(mx);
    const float mn = fmaxf(m, fmaxf(both.a, both.b));
    float mcn = mn * c;
    const bool far_n = __ballot(fabsf(mcn) > 1048576.0f) != 0;
    if (far_n) mcn = 0.0f;
    const float alpha = __builtin_amdgcn_exp2f(__builtin_fmaf((far ? m : 0.0f) - (far_n ? mn : 0.0f), c, mc - mcn));
    m = mn;
    mc = mcn;
    far = far_n;
    l *= alpha;
    lost *= alpha;
    return alpha;
  };
  auto from_max = [&](f32x16 (&x)[2]) {
    if (far) {
#pragma unroll
      for (int r = 0; r < 32; ++r) x[r >> 4][r & 15] -= m;
    }
  };

  // Start of step kt: one barrier frees K(kt) and V(kt - 1) and publishes K(kt + 1) and V(kt); the codes of the next
  // two tiles are requested, their pages were a step ago
  auto begin_step = [&](int kt) {
    __syncthreads();
    if (kt + 2 < nt) {
      request_k(kt + 2, wk, sk, gone_k);
      k_pages(kt + 3);
    }
    if (kt + 1 < nt) {
      request_v(kt + 1);
      v_pages(kt + 2);
    }
  };
  auto end_step = [&](int kt) {
    if (kt + 2 < nt) store_k(kt + 2, wk, sk, gone_k);
    if (kt + 1 < nt) store_v(kt + 1);
  };
  auto step = [&](f32x16 (&cur)[2], uint32_t (&pc)[16], f32x16 (&nxt)[2], uint32_t (&pn)[16], int kt) {
    begin_step(kt);
    const uint8_t* sk_ = smem + ((kt + 1) & 1) * (2 * kTileBytes);
    const uint8_t* sv_ = smem + (kt & 1) * (2 * kTileBytes) + kTileBytes;
    bf16x8 fk[NK], fv[NV];
#pragma unroll
    for (int u = 0; u < kAheadC; ++u) fk[u] = read_k(sk_, u);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int u = 0; u < NK; ++u) {
      if (u + kAheadC < NK) fk[u + kAheadC] = read_k(sk_, u + kAheadC);
      else fv[u + kAheadC - NK] = read_v(sv_, u + kAheadC - NK);
      nxt[u & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fk[u], fq[u >> 1], u < 2 ? f32x16{} : nxt[u & 1], 0, 0, 0);
#pragma unroll
      for (int r = 8 + 8 * u / NK; r < 8 + 8 * (u + 1) / NK; ++r) pair(cur, pc, r);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
    add_tile();
    mask(nxt, kt + 1);
    constexpr int kMax = NV / 4;   // products that cover the maximum
    auto value = [&](int u) {
      if (u + kAheadC < NV) fv[u + kAheadC] = read_v(sv_, u + kAheadC);
      acc[u % JD] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fv[u], prob_operand(pc, u / JD), acc[u % JD], 0, 0, 0);
    };
    float mx = -__builtin_inff(), alpha = 1.0f;
#pragma unroll
    for (int u = 0; u < kMax; ++u) {
      value(u);
#pragma unroll
      for (int r = 32 * u / kMax; r < 32 * (u + 1) / kMax; ++r) mx = fmaxf(mx, nxt[r >> 4][r & 15]);
      __builtin_amdgcn_sched_barrier(0);
    }
    const bool up = __ballot(mx > m + slack) != 0;
    if (up) alpha = raise(mx);
    from_max(nxt);
#pragma unroll
    for (int u = kMax; u < NV; ++u) {
      value(u);
#pragma unroll
      for (int r = 8 * (u - kMax) / (NV - kMax); r < 8 * (u + 1 - kMax) / (NV - kMax); ++r) pair(nxt, pn, r);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (up) {
#pragma unroll
      for (int j = 0; j < JD; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[j][r] *= alpha;
    }
    end_step(kt);
  };

  if (nt > 0) {   // the first two tiles of K and the first of V, all requested before any is waited for
    u32x4 wk1[kPieces];
    uint32_t sk1[kOwn];
    int next[kOwn], gone1;
    k_pages(1);
#pragma unroll
    for (int c = 0; c < kOwn; ++c) next[c] = ek[c];
    k_pages(0);
    v_pages(0);
    request_k(0, wk, sk, gone_k);
    request_v(0);
#pragma unroll
    for (int c = 0; c < kOwn; ++c) ek[c] = next[c];
    request_k(1, wk1, sk1, gone1);   // (without a second tile: a page that is not there)
    k_pages(2);
    v_pages(1);
    store_k(0, wk, sk, gone_k);
    store_v(0);
    store_k(1, wk1, sk1, gone1);
    __syncthreads();
  }
  int kt = 0;
  if (ntw > 0) {
    f32x16 s0[2], s1[2];
    uint32_t p0[16], p1[16];
#pragma unroll
    for (int u = 0; u < NK; ++u)
      s0[u & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_k(smem, u), fq[u >> 1], u < 2 ? f32x16{} : s0[u & 1], 0, 0, 0);
    mask(s0, 0);
    float mx = s0[0][0];
#pragma unroll
    for (int r = 1; r < 32; ++r) mx = fmaxf(mx, s0[r >> 4][r & 15]);
    raise(mx);
    from_max(s0);
#pragma unroll
    for (int r = 0; r < 8; ++r) pair(s0, p0, r);
    for (; kt + 2 < ntw; kt += 2) {
      step(s0, p0, s1, p1, kt);
      step(s1, p1, s0, p0, kt + 1);
    }
    if (kt + 1 < ntw) {
      step(s0, p0, s1, p1, kt);
      s0[1] = s1[1];
#pragma unroll
      for (int r = 0; r < 8; ++r) p0[r] = p1[r];
      ++kt;
    }
    begin_step(kt);   // the last tile
    const uint8_t* sv_ = smem + (kt & 1) * (2 * kTileBytes) + kTileBytes;
#pragma unroll
    for (int r = 8; r < 16; ++r) pair(s0, p0, r);
    add_tile();
#pragma unroll
    for (int u = 0; u < NV; ++u)
      acc[u % JD] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_v(sv_, u), prob_operand(p0, u / JD), acc[u % JD], 0, 0, 0);
    end_step(kt);
    ++kt;
  }
  for (; kt < nt; ++kt) {   // tiles that only other waves need
    begin_step(kt);
    end_step(kt);
  }

  const Pair sums = halves32(l);
  l = sums.a + sums.b;
  if (!only) {   // this lane holds elements 32 j + 8 (r / 4) + 4 h + r % 4 of its row
    if (row0 + l32 >= n_rows) return;
    // relative to the maximum itself, not to its rounded product
    const float f = far ? 1.0f : __builtin_amdgcn_exp2f(__builtin_fmaf(-m, c, mc));
    const int64_t at = ((int64_t)split * a.T + rb.tok0 + query) * a.H + head;
    float* dst = a.partial + at * D + 4 * h;
#pragma unroll
    for (int j = 0; j < JD; ++j)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<f32x4*>(dst + 32 * j + 2 * r) = f32x4{acc[j][r] * f, acc[j][r + 1] * f, acc[j][r + 2] * f, acc[j][r + 3] * f};
    if (h == 0) {
      float* st = a.partial + (int64_t)a.splits * a.T * a.H * D + 2 * at;
      st[0] = m;
      st[1] = l * f;
    }
    return;
  }
  // O^T through LDS (the tiles' space): each wave turns its block into rows and stores whole
  // 16-byte pieces. Row r's pieces are permuted by piece ^ (r % pieces).
  __syncthreads();
  constexpr int kOP = D / 8, kRowsPerCopy = 64 / kOP;
  uint8_t* out = smem + wave * (32 * kRowBytes);
  static_assert(kWavesT * 32 * kRowBytes <= 4 * kTileBytes, "output staging");
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int j = 0; j < JD; ++j)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *reinterpret_cast<u32x2*>(out + l32 * kRowBytes + (((4 * j + r / 4) ^ (l32 & (kOP - 1))) * 16) + 8 * h) =
          u32x2{pack_bf16x2(acc[j][r] * inv, acc[j][r + 1] * inv), pack_bf16x2(acc[j][r + 2] * inv, acc[j][r + 3] * inv)};
  __syncthreads();
  uint16_t* op = a.o + hk * G * a.o_sh;
#pragma unroll
  for (int u = 0; u < 32 / kRowsPerCopy; ++u) {
    const int r = u * kRowsPerCopy + lane / kOP, piece = lane % kOP;
    const u32x4 w = *reinterpret_cast<const u32x4*>(out + r * kRowBytes + ((piece ^ (r & (kOP - 1))) * 16));
    const int tq = __shfl(query, r), th = __shfl(head, r) - hk * G;
    if (row0 + r < n_rows) *reinterpret_cast<u32x4*>(op + (int64_t)(rb.tok0 + tq) * a.o_st + th * a.o_sh + 8 * piece) = w;
  }
}

// The splits of a row (a query's head) together, four elements a thread. WIDE: a workgroup a row, its groups of D / 4
// threads take the splits in turn; else a group a row, for up to 8 splits, all requested at once. (A wave per row
// that walked through its splits took longer than the attention from 64 splits on.)
constexpr int kWays[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128};   // that keys are split
constexpr int kMaxSplits = kWays[sizeof(kWays) / sizeof(kWays[0]) - 1], kFewSplits = 8;
static_assert(kMaxSplits <= 256, "a thread of join_kernel a split");

template <int D, bool WIDE>
__global__ __launch_bounds__(256) void join_kernel(AttnCacheArgs a) {
  constexpr int kGroups = 256 / (D / 4);
  __shared__ float weight[WIDE ? kMaxSplits : 1];
  __shared__ float part[4];
  __shared__ f32x4 sums[WIDE ? kGroups : 1][D / 4];
  const int tid = threadIdx.x, e = tid % (D / 4), g = tid / (D / 4);
  const int64_t rows = a.T * a.H;
  const int64_t row = WIDE ? (int64_t)blockIdx.x : min((int64_t)blockIdx.x * kGroups + g, rows - 1);
  const int64_t tok = row / a.H;
  int b = (int)tok;
  if (a.cu != nullptr) {   // the sequence of a token: of the wave's rows, those of the same token together
    b = 0;
    if (WIDE) {
      b = wave_count_le(a.cu, a.B + 1, tok) - 1;
    } else {
      int lo = 0, hi = a.B + 1;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (a.cu[mid] <= tok) lo = mid + 1;
        else hi = mid;
      }
      b = lo - 1;
    }
  }
  const bool in = b >= 0 && b < a.B;   // else outside the sequences
  const int64_t L = in ? keys_of(a, b) : 0;
  const int per = tiles_per_split(a, L);
  const int n = (int)(((L + kTile - 1) / kTile + per - 1) / per);   // splits with keys; 0 or 1: written whole
  if (WIDE && n <= 1) return;
  const float c = a.scale * 1.4426950408889634f;
  const float* st = a.partial + (int64_t)a.splits * rows * D;
  const float* src = a.partial + row * D + 4 * e;
  f32x4 o = {};
  float total = 0.0f;
  if constexpr (WIDE) {
    float m = kLowest, l = 0.0f;
    if (tid < n) {
      const float2 v = *reinterpret_cast<const float2*>(st + 2 * (tid * rows + row));
      m = v.x;
      l = v.y;
    }
    const float top = wave_reduce<true>(m);
    if ((tid & 63) == 0) part[tid >> 6] = top;
    __syncthreads();
    const float M = max_or_nan(max_or_nan(part[0], part[1]), max_or_nan(part[2], part[3]));
    const float f = tid < n ? __builtin_amdgcn_exp2f((m - M) * c) : 0.0f;
    if (tid < n) weight[tid] = f;
    const float share = wave_reduce<false>(l * f);
    __syncthreads();   // everyone has the maxima
    if ((tid & 63) == 0) part[tid >> 6] = share;
#pragma unroll 4
    for (int s = g; s < n; s += kGroups) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(src + s * rows * D);
      const float w = weight[s];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __builtin_fmaf(v[i], w, o[i]);
    }
    sums[g][e] = o;
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int i = 1; i < kGroups; ++i) o += sums[i][e];
    total = part[0] + part[1] + part[2] + part[3];
  } else {
    f32x4 v[kFewSplits];
    float2 s[kFewSplits];
    float M = kLowest;
#pragma unroll
    for (int i = 0; i < kFewSplits; ++i) {
      if (i < n) {
        s[i] = *reinterpret_cast<const float2*>(st + 2 * (i * rows + row));
        v[i] = *reinterpret_cast<const f32x4*>(src + i * rows * D);
      }
    }
#pragma unroll
    for (int i = 0; i < kFewSplits; ++i)
      if (i < n) M = fmaxf(M, s[i].x);
#pragma unroll
    for (int i = 0; i < kFewSplits; ++i) {
      if (i < n) {
        const float f = __builtin_amdgcn_exp2f((s[i].x - M) * c);
        total += s[i].y * f;
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = __builtin_fmaf(v[i][r], f, o[r]);
      }
    }
    if (n <= 1 || (int64_t)blockIdx.x * kGroups + g >= rows) return;
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  *reinterpret_cast<u32x2*>(a.o + tok * a.o_st + (row - tok * a.H) * a.o_sh + 4 * e) =
      u32x2{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
}

// Which kernel (0 few rows, 1 tiles) and how many ways the keys are split, by an estimate in microseconds from what the host
// knows: T, B and a bound of the lengths. A workgroup walks through its share in steps (64 keys for each wave of few rows, a
// tile of 64); a step takes at least `least`, and `full` for each workgroup on a CU: those there together up to two, else
// all that come by, and `tail` for the last ones' end. Of several sequences the longest counts `longest` of a step's share
// while all are there, and they average `mean` of it else; one sequence's shares are equal, so the CU with the most counts.
// All steps together take no less than the codes at 7 TB/s. `base` starts and ends the call, a split adds a launch and
// its partial results. As for the linears, a call that is not in a graph takes its caller 10.3 us, and with a workspace and a
// second launch 14, so a split pays only where the device takes longer than that.
// Fitted to both kernels at 345 sizes (1 to 64 sequences of 1 to 4096 queries on 150 to 65000 keys, groups of 1, 4 and
// 8, keys split up to 64 ways, those on the longest 128, from memory: profiles/attention_cache_grid.txt). Where the best takes the device 14 us or more
// the choice is within 4% of it on average and 28% at worst; below, 1.3% and 18% (64 queries on 3064 keys, 8 heads on one:
// 14.1 us split 12 ways, 12.0 split 8). The caller is taken to be eager: a call captured in a graph chooses alike. One token on 65537 keys, 32 heads on 8: 31.6 us split 32 ways, 40 16
// ways, 33 64 ways. 40 tokens on 540 keys: 9.7 us by few rows, 19 by tiles; 512 on 8704: 192 and 105.
struct AttnPlan {
  int kernel, splits;
};
constexpr int64_t kMostPartial = int64_t(1) << 28;   // bytes

AttnPlan plan_attention(int64_t T, int64_t B, int64_t H, int64_t Hk, int64_t D, int64_t max_length, bool packed) {
  static const struct { int rows, keys; double base, least, full, tail, longest, mean; } kernels[] = {
      {16, 4 * kTile, 3.14, 2.01, 1.38, 0.53, 1.15, 0.84}, {128, kTile, 5.35, 1.64, 0.83, 1.06, 1.34, 0.8}};
  const double memory = 2.0 * (double)(Hk * D) * (double)max_length * (B > 1 ? 0.6 * (double)B : 1.0) / 7e6;
  const int64_t G = H / Hk, tiles = (max_length + kTile - 1) / kTile;
  AttnPlan best{0, 1};
  double best_t = 1e300;
  for (int k = 0; k < 2; ++k) {
    const int rows = kernels[k].rows;
    int64_t blocks = packed ? (T * G + rows - 1) / rows : B * ((G + rows - 1) / rows);
    blocks = (blocks < B ? B : blocks) * Hk;
    const double wide = k == 0 ? (double)D / 128.0 : 0.3 + 0.7 * (double)D / 128.0;
    for (int s : kWays) {
      if (s > 1 && (tiles < kLeastTiles * s || (int64_t)s * T * H * (D + 2) * 4 > kMostPartial)) break;
      const double steps = (double)(((tiles + s - 1) / s * kTile + kernels[k].keys - 1) / kernels[k].keys);
      const double on_cu = B > 1 ? (double)(blocks * s) / 256.0 : (double)((blocks * s + 255) / 256);
      const double share = on_cu <= 2.0 ? on_cu * (B > 1 ? kernels[k].longest : 1.0)
                                        : on_cu * (B > 1 ? kernels[k].mean : 1.0) + kernels[k].tail;
      const double device = kernels[k].base + fmax(steps * fmax(kernels[k].least, share * kernels[k].full * wide), memory) +
                            (s > 1 ? 6.46 + 1.92e-6 * (double)(T * H * D) * s : 0.0);
      const double t = fmax(device, s > 1 ? 14.0 : 10.3) + 0.01 * device;
      if (t < best_t) {
        best_t = t;
        best = AttnPlan{k, s};
      }
    }
  }
  return best;
}

template <int D>
void launch_tiles(const AttnCacheArgs& a, hipStream_t stream) {
  const int64_t total = ((a.T * (a.H / a.c.Hk) >> kLgRows) + a.B) * a.splits * a.c.Hk;
  const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(64 * kWavesT);
  const bool whole = a.c.lg_page >= 6;
  if (a.causal && whole) hipLaunchKernelGGL((attention_tile_kernel<D, true, true>), grid, block, 0, stream, a);
  else if (a.causal) hipLaunchKernelGGL((attention_tile_kernel<D, true, false>), grid, block, 0, stream, a);
  else if (whole) hipLaunchKernelGGL((attention_tile_kernel<D, false, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((attention_tile_kernel<D, false, false>), grid, block, 0, stream, a);
}

template <int D>
hipError_t launch_d(const AttnCacheArgs& a, int kernel, hipStream_t stream) {
  const int64_t G = a.H / a.c.Hk;
  if (kernel == 0) {
    const int64_t blocks = a.cu == nullptr ? a.B * ((G + 15) / 16) : (a.T * G >> 4) + a.B;
    hipLaunchKernelGGL(attention_few_kernel<D>, dim3((unsigned)(blocks * a.splits), (unsigned)a.c.Hk), dim3(64 * kWavesF),
                       0, stream, a);
  } else {
    launch_tiles<D>(a, stream);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = a.T * a.H;
  if (a.splits > kFewSplits) hipLaunchKernelGGL((join_kernel<D, true>), dim3((unsigned)rows), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((join_kernel<D, false>), dim3((unsigned)((rows + 1024 / D - 1) / (1024 / D))), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

void attention_cache_plan(int64_t T, int64_t B, int64_t H, int64_t Hk, int64_t D, int64_t max_length, bool packed,
                          int* kernel, int* splits) {
  const AttnPlan p = plan_attention(T, B, H, Hk, D, max_length, packed);
  *kernel = p.kernel;
  *splits = p.splits;
}

size_t attention_cache_partial_bytes(int64_t T, int64_t H, int64_t D, int splits) {
  return splits > 1 ? (size_t)splits * (size_t)T * (size_t)H * (size_t)(D + 2) * 4 : 0;
}

hipError_t launch_attention_cache(const AttnCacheArgs& a, int kernel, hipStream_t stream) {
  return a.c.D == 64 ? launch_d<64>(a, kernel, stream) : launch_d<128>(a, kernel, stream);
}

}  // namespace svdq
