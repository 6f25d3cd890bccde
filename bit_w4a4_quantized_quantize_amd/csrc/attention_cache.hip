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

// keys of a sequence: what its table can hold at most
__device__ __forceinline__ int64_t keys_of(const AttnCacheArgs& a, int b) {
  return min((int64_t)max(a.lengths[b], 0), a.width << a.c.lg_page);
}
// tiles of 64 keys that a split takes, and how many splits have any
__device__ __forceinline__ int tiles_per_split(const AttnCacheArgs& a, int64_t L) {
  const int tiles = (int)((L + kTile - 1) / kTile);
  return max((tiles + a.splits - 1) / a.splits, a.least);
}

// sum or maximum over the four lanes l16, l16 + 16, .. of a row
template <bool MAX>
__device__ __forceinline__ float across_rows(float v) {
  const float u = __shfl_xor(v, 16);
  v = MAX ? fmaxf(v, u) : v + u;
  const float w = __shfl_xor(v, 32);
  return MAX ? fmaxf(v, w) : v + w;
}

// Few rows. The four waves of a workgroup take 16 rows together, steps of 64 keys in turn; a step's operands
// come straight from memory in 16-byte pieces:
//  S^T: tile t of four holds key 16 (i / 4) + 4 t + i % 4 in matrix row i, so that lane (row, q) receives the
//       scores of keys 16 q .. 16 q + 15 of the step;
//  O^T: the same 16 keys of an element of v are one piece of the transposed page.
constexpr int kWavesF = 4;

template <int D>
__global__ __launch_bounds__(64 * kWavesF) void attention_few_kernel(AttnCacheArgs a) {
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
  auto page_of = [&](int64_t key) {   // -1: none
    const int64_t at = key >> a.c.lg_page;
    const int p = at < a.width ? table[at] : -1;
    return (uint32_t)p < (uint32_t)a.c.pages ? p : -1;
  };

  f32x4 acc[JD];
#pragma unroll
  for (int j = 0; j < JD; ++j) acc[j] = f32x4{};
  const float c = a.scale * 1.4426950408889634f;   // exponents in base 2
  float m = kLowest / fmaxf(c, 1.0f), l = 0.0f;
  const float slack = kSlackC / c;
  bool first = true;

  for (int64_t k0 = k_begin + kTile * wave; k0 < k_end; k0 += kTile * kWavesF) {
    // keys: this lane loads pieces of keys kk + 4 t; values: of keys kv .. kv + 15
    const int64_t kk = k0 + 16 * (l16 >> 2) + (l16 & 3), kv = k0 + 16 * q;
    const int pk = page_of(kk), pv = page_of(kv);
    const int64_t pk_at = (int64_t)max(pk, 0) * a.c.Hk + hk, pv_at = (int64_t)max(pv, 0) * a.c.Hk + hk;
    const uint8_t* kp = a.c.k + pk_at * page_bytes + (kk & (P - 1)) * D + 16 * q;
    const uint8_t* vp = a.c.v + pv_at * page_bytes + l16 * P + (kv & (P - 1));
    float ks = cache_scale(a.c.ks[pk_at]), vs = cache_scale(a.c.vs[pv_at]);
    u32x4 wk[4][KP], wv[JD];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int u = 0; u < KP; ++u) wk[t][u] = *reinterpret_cast<const u32x4*>(kp + 4 * t * D + 64 * u);
#pragma unroll
    for (int j = 0; j < JD; ++j) wv[j] = *reinterpret_cast<const u32x4*>(vp + 16 * j * P);
    if (pk < 0) {
      ks = 1.0f;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int u = 0; u < KP; ++u) wk[t][u] = zero4();
    }
    // values past the sequence, or without a page, are zero: their probabilities are, but what
    // the page holds there may be NaN
    const int64_t left = pv < 0 ? 0 : L - kv;
    if (left < 16) {
      if (left <= 0) vs = 1.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = (int)max(min(left - 4 * i, (int64_t)4), (int64_t)0);
        const uint32_t keep = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
#pragma unroll
        for (int j = 0; j < JD; ++j) wv[j][i] &= keep;
      }
    }

    f32x4 x[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      x[t] = f32x4{};
#pragma unroll
      for (int u = 0; u < KP; ++u) {
        x[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_operand(wk[t][u][0], wk[t][u][1], ks), fq[2 * u], x[t], 0, 0, 0);
        x[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_operand(wk[t][u][2], wk[t][u][3], ks), fq[2 * u + 1], x[t], 0, 0, 0);
      }
    }
    float mx = -__builtin_inff();
    if (k0 + kTile > last + 1) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (kv + 4 * t + r > last) x[t][r] = -__builtin_inff();
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
#pragma unroll
    for (int j = 0; j < JD; ++j) {
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_operand(wv[j][0], wv[j][1], vs), fp0, acc[j], 0, 0, 0);
      acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf16_operand(wv[j][2], wv[j][3], vs), fp1, acc[j], 0, 0, 0);
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

// The splits of a row (a query's head) together, a wave each.
template <int D>
__global__ __launch_bounds__(256) void join_kernel(AttnCacheArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t rows = a.T * a.H;
  if (row >= rows) return;
  const int64_t tok = row / a.H;
  int b = (int)tok;
  if (a.cu != nullptr) {
    b = wave_count_le(a.cu, a.B + 1, tok) - 1;
    if (b < 0 || b >= a.B) return;   // outside the sequences
  }
  const int64_t L = keys_of(a, b);
  const int per = tiles_per_split(a, L);
  const int n = (int)(((L + kTile - 1) / kTile + per - 1) / per);   // splits with keys
  if (n <= 1) return;                                              // written whole
  const float c = a.scale * 1.4426950408889634f;
  const float* st = a.partial + (int64_t)a.splits * rows * D;
  float M = kLowest;
  for (int s = 0; s < n; ++s) M = fmaxf(M, st[2 * (s * rows + row)]);
  float total = 0.0f, o[D / 64] = {};
  for (int s = 0; s < n; ++s) {
    const int64_t at = s * rows + row;
    const float f = __builtin_amdgcn_exp2f((st[2 * at] - M) * c);
    total += st[2 * at + 1] * f;
#pragma unroll
    for (int e = 0; e < D / 64; ++e) o[e] += a.partial[at * D + lane * (D / 64) + e] * f;
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  uint16_t* dst = a.o + tok * a.o_st + (row - tok * a.H) * a.o_sh + lane * (D / 64);
  if constexpr (D == 128) *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0] * inv, o[1] * inv);
  else *dst = (uint16_t)f32_to_bf16_rne(o[0] * inv);
}

int plan_splits(int64_t T, int64_t B, int64_t H, int64_t Hk, int64_t max_length, bool packed) {
  const int64_t G = H / Hk;
  const int64_t blocks = packed ? (T * G + 15) / 16 : B * ((G + 15) / 16);
  const int64_t tiles = (max_length + kTile - 1) / kTile;
  int64_t s = (1024 + blocks * Hk - 1) / (blocks * Hk);
  if (s > (tiles + 3) / 4) s = (tiles + 3) / 4;
  return (int)(s < 1 ? 1 : s);
}

template <int D>
hipError_t launch_d(const AttnCacheArgs& a, hipStream_t stream) {
  const int64_t G = a.H / a.c.Hk;
  const int64_t blocks = a.cu == nullptr ? a.B * ((G + 15) / 16) : (a.T * G >> 4) + a.B;
  hipLaunchKernelGGL(attention_few_kernel<D>, dim3((unsigned)(blocks * a.splits), (unsigned)a.c.Hk), dim3(64 * kWavesF),
                     0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL(join_kernel<D>, dim3((unsigned)((a.T * a.H + 3) / 4)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

size_t attention_cache_workspace_bytes(int64_t T, int64_t B, int64_t H, int64_t Hk, int64_t D, int64_t max_length,
                                       bool packed) {
  const int s = plan_splits(T, B, H, Hk, max_length, packed);
  return s > 1 ? (size_t)s * (size_t)T * (size_t)H * (size_t)(D + 2) * 4 : 0;
}

hipError_t launch_attention_cache(AttnCacheArgs a, int64_t max_length, hipStream_t stream) {
  a.splits = plan_splits(a.T, a.B, a.H, a.c.Hk, max_length, a.cu != nullptr);
  a.least = 4;
  return a.c.D == 64 ? launch_d<64>(a, stream) : launch_d<128>(a, stream);
}

}  // namespace svdq
