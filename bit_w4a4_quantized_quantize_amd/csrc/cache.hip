// A cache of keys and values in pages, held in e4m3 with a power-of-two scale per page and head:
//
//   keys   [pages, Hk, P, D]: token-major within a page        value = code * 2^(scale - 127)
//   values [pages, Hk, D, P]: element-major, so that the tokens a product with the probabilities sums over
//                             are contiguous                   scales [pages, Hk], bytes (E8M0, 255 = NaN)
//
// Appending: a page's scale is the least power of two (from 2^-100) that holds its tokens' maximum within 448 when
// its first token is written, and grows when a later one needs more; what was there is rescaled, which is exact but
// for codes that become subnormal. One workgroup per page touched, head and tensor.
#include "cache.h"

namespace svdq {

namespace {

// Threads of a page's workgroup: four tokens of 8 elements each, up to 256 (a page of 128 tokens of 128: two fours each)
template <int D, int P>
constexpr int kThreadsC = P * D / 32 < 64 ? 64 : P * D / 32 > 256 ? 256 : P * D / 32;

// The pages that a sequence of n tokens touches from any start are at most floor((n - 2) / P) + 2, so blocks
// of P packed tokens are numbered with two more per sequence: sequence b starts at floor(cu[b] / P) + 2 b.
// Finds the sequence of block t and its local number; false where there is none.
struct Touched {
  int b, first, count;   // sequence, its first packed token and its tokens
  int64_t local;
};
__device__ __forceinline__ bool touched_block(const CacheTokens& a, int lg, int64_t t, Touched& o) {
  if (a.cu == nullptr) {   // a token per sequence
    o = Touched{(int)t, (int)t, 1, 0};
    return t < a.B;
  }
  // last sequence whose first block is at most t
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = a.B;
  while (true) {
    const int step = (hi - lo + 63) / 64;
    const int idx = lo + lane * step;
    const int c0 = min(max(a.cu[min(idx, a.B)], 0), (int)a.T);
    const int n = __popcll(__ballot(idx < hi && (int64_t)(c0 >> lg) + 2 * (int64_t)idx <= t));
    if (n == 0) return false;
    lo += (n - 1) * step;
    if (step == 1) break;
    hi = min(hi, lo + step);
  }
  const int c0 = min(max(a.cu[lo], 0), (int)a.T), c1 = min(max(a.cu[lo + 1], 0), (int)a.T);
  o = Touched{lo, c0, c1 - c0, t - (c0 >> lg) - 2 * (int64_t)lo};
  return o.local >= 0;
}

// The page of a block and the tokens in it: packed tokens tok0 .. tok0 + (s1 - s0) - 1 go to slots s0 .. s1 - 1.
// `entry` is the table's, to be looked at where it is needed: the tokens are requested meanwhile.
struct Block {
  int entry, tok0, s0, s1;
};
template <int P>
__device__ __forceinline__ bool find_block(const CacheTokens& a, Block& o) {
  constexpr int kLg = __builtin_ctz(P);
  Touched t;
  if (!touched_block(a, kLg, (int64_t)blockIdx.x, t) || t.count <= 0) return false;
  const int64_t start = max(a.starts[t.b], 0), end = start + t.count;
  const int64_t block = (start >> kLg) + t.local;
  const int64_t p0 = block << kLg;
  if (p0 >= end) return false;
  const int64_t from = max(start, p0), to = min(end, p0 + P);
  o = Block{block < a.width ? a.table[(int64_t)t.b * a.width + block] : -1, t.first + (int)(from - start),
            (int)(from - p0), (int)(to - p0)};
  return true;
}

// 16 codes times 2^(from - to), nearest even
__device__ __forceinline__ u32x4 rescale16(u32x4 w, float by) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v0 = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 0) * by, v1 = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 1) * by;
    const float v2 = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 2) * by, v3 = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 3) * by;
    w[i] = fp8_codes4(v0, v1, v2, v3);
  }
  return w;
}

// bytes lo .. hi - 1 of a 16-byte piece (whole if 0, 16)
__device__ __forceinline__ void store_bytes(uint8_t* dst, u32x4 w, int lo, int hi) {
  if (lo <= 0 && hi >= 16) {
    *reinterpret_cast<u32x4*>(dst) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (e >= lo && e < hi) dst[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
  }
}

// An image of a page of values in LDS: row d of P slots, its 16-byte pieces permuted by the rows' eights, so that
// lanes that write (or read) the same slots of every eighth row meet different banks.
template <int D, int P>
struct Image {
  static constexpr int kBytes = D * (P + 16);
  uint8_t* at;
  __device__ __forceinline__ uint8_t* slot(int d, int s) const {
    return at + d * (P + 16) + ((((s >> 4) ^ ((d >> 3) & (P / 16 - 1))) << 4) | (s & 15));
  }
};

// bytes i of four dwords -> dword i (the transpose of 4 x 4 bytes)
__device__ __forceinline__ u32x4 transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t ab0 = __builtin_amdgcn_perm(b, a, 0x05010400u), ab1 = __builtin_amdgcn_perm(b, a, 0x07030602u);
  const uint32_t cd0 = __builtin_amdgcn_perm(d, c, 0x05010400u), cd1 = __builtin_amdgcn_perm(d, c, 0x07030602u);
  return u32x4{__builtin_amdgcn_perm(cd0, ab0, 0x05040100u), __builtin_amdgcn_perm(cd0, ab0, 0x07060302u),
               __builtin_amdgcn_perm(cd1, ab1, 0x05040100u), __builtin_amdgcn_perm(cd1, ab1, 0x07060302u)};
}

// Memory bound: packed prompts of 16411 tokens, 8 heads of 128 on pages of 64 (101 MB, from memory) 24.8 us. 32 single
// tokens take 5.2, the chain of loads that finds the page. Kernels made for their page's size have as many threads as it
// has work (written and read back: pages of 16 tokens 80 -> 46 us, of 32 54 -> 46).
template <int D, int P>
__global__ __launch_bounds__((kThreadsC<D, P>)) void append_kernel(CacheTokens a, CacheShape c, HeadView k, HeadView v) {
  constexpr int kThreads = kThreadsC<D, P>;
  constexpr int kLanes = D / 8;                       // lanes of a token, 8 elements each
  constexpr int kRows = kThreads / kLanes;            // fours of tokens of a pass
  constexpr int kPasses = (P + 4 * kRows - 1) / (4 * kRows);
  __shared__ __attribute__((aligned(16))) uint8_t smem[Image<D, P>::kBytes];
  __shared__ float part[kThreads / 64];
  Block blk;
  if (!find_block<P>(a, blk)) return;
  const int tid = threadIdx.x;
  const int head = (int)blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const HeadView in = is_v ? v : k;
  const int row = 4 * (tid / kLanes), e0 = 8 * (tid % kLanes);
  const int n = blk.s1 - blk.s0;

  u32x4 w[kPasses][4];   // tokens row + 4 kRows u + i
  float amax = 0.0f;
#pragma unroll
  for (int u = 0; u < kPasses; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = row + 4 * kRows * u + i;
      w[u][i] = r < n ? *reinterpret_cast<const u32x4*>(in.p + (int64_t)(blk.tok0 + r) * in.st + head * in.sh + e0) : zero4();
    }
  const int64_t at_page = (int64_t)blk.entry * c.Hk + head;
  if ((uint32_t)blk.entry >= (uint32_t)c.pages) return;   // the table has no page: left out
  uint8_t* scale_at = (is_v ? c.vs : c.ks) + at_page;
  const int old = blk.s0 > 0 ? *scale_at : 0;         // below every scale that is written
#pragma unroll
  for (int u = 0; u < kPasses; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int d = 0; d < 4; ++d)
        amax = max_or_nan(amax, max_or_nan(fabsf(bf16lo_to_f32(w[u][i][d])), fabsf(bf16hi_to_f32(w[u][i][d]))));
  amax = wave_reduce<true>(amax);
  if ((tid & 63) == 0) part[tid >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) amax = max_or_nan(amax, part[i]);
  const bool fine = amax <= 3.4028234663852886e38f;
  const int now = fine ? max(fp8_exponent(amax) + 127, old) : 255;
  if (tid == 0 && now != old) *scale_at = (uint8_t)now;
  // a NaN scale says it all: codes are left as they are, new ones are zero
  // (2^(127 - now); for 254, which only a page filled elsewhere can have, that is 2^-127, a subnormal)
  const float inv = now < 254 ? __uint_as_float((uint32_t)(254 - now) << 23) : now == 254 ? 0x1p-127f : 0.0f;
  const bool grown = blk.s0 > 0 && now > old && now < 255;
  // 2^(old - now); below 2^-126 every code becomes zero
  const float by = now - old < 127 ? __uint_as_float((uint32_t)(127 + old - now) << 23) : 0.0f;
  auto codes = [&](const u32x4& x) {
    float f[8];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      f[2 * d] = bf16lo_to_f32(x[d]);
      f[2 * d + 1] = bf16hi_to_f32(x[d]);
    }
    return fp8_codes8(f, inv);
  };

  uint8_t* page = (is_v ? c.v : c.k) + at_page * (P * D);
  if (!is_v) {
    if (grown) {
      for (int i = tid; i < blk.s0 * (D / 16); i += kThreads) {
        u32x4* at = reinterpret_cast<u32x4*>(page) + i;
        *at = rescale16(*at, by);
      }
    }
#pragma unroll
    for (int u = 0; u < kPasses; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = row + 4 * kRows * u + i;
        if (r < n) *reinterpret_cast<u32x2*>(page + (blk.s0 + r) * D + e0) = codes(w[u][i]);
      }
    return;
  }
  // values: the page's image [D][P] is put together in LDS and leaves by rows
  const Image<D, P> image{smem};
  if (grown) {
    for (int i = tid; i < D * (P / 16); i += kThreads) {
      const int d = i / (P / 16), s = 16 * (i % (P / 16));
      if (s < blk.s0)
        *reinterpret_cast<u32x4*>(image.slot(d, s)) = rescale16(*reinterpret_cast<const u32x4*>(page + d * P + s), by);
    }
    __syncthreads();   // the last piece may hold new tokens' slots too
  }
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
    const int r = row + 4 * kRows * u, s = blk.s0 + r;
    if (r >= n) break;
    u32x2 q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = codes(w[u][i]);
    if (blk.s0 % 4 == 0) {   // four slots at once (those past n are not stored)
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const u32x4 z = transpose4(q[0][g], q[1][g], q[2][g], q[3][g]);
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(image.slot(e0 + 4 * g + e, s)) = z[e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + i < n) {
#pragma unroll
          for (int e = 0; e < 8; ++e) *image.slot(e0 + e, s + i) = (uint8_t)(q[i][e >> 2] >> (8 * (e & 3)));
        }
    }
  }
  __syncthreads();
  const int from = grown ? 0 : blk.s0;
  for (int i = tid; i < D * (P / 16); i += kThreads) {
    const int d = i / (P / 16), s = 16 * (i % (P / 16));
    if (s + 16 > from && s < blk.s1)
      store_bytes(page + d * P + s, *reinterpret_cast<const u32x4*>(image.slot(d, s)), from - s, blk.s1 - s);
  }
}

// 16 codes -> 16 bf16, exact
__device__ __forceinline__ void widen16(u32x4 w, float scale, u32x4 (&o)[2]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i >> 1][2 * (i & 1)] = fp8_pair_to_bf16<0>(w[i], scale);
    o[i >> 1][2 * (i & 1) + 1] = fp8_pair_to_bf16<1>(w[i], scale);
  }
}

// Packed tokens' keys and values back in bf16; zeros where the table has no page.
// Memory bound: the same prompts 19.6 us (5.1 TB/s).
template <int D, int P>
__global__ __launch_bounds__((kThreadsC<D, P>)) void read_kernel(CacheTokens a, CacheShape c, uint16_t* k_out,
                                                                 uint16_t* v_out) {
  constexpr int kThreads = kThreadsC<D, P>;
  __shared__ __attribute__((aligned(16))) uint8_t smem[Image<D, P>::kBytes];
  Block blk;
  if (!find_block<P>(a, blk)) return;
  const int tid = threadIdx.x;
  const int head = (int)blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int n = blk.s1 - blk.s0;
  const bool none = (uint32_t)blk.entry >= (uint32_t)c.pages;
  const int64_t at_page = (none ? 0 : (int64_t)blk.entry) * c.Hk + head;
  const uint8_t* page = (is_v ? c.v : c.k) + at_page * (P * D);
  const uint32_t scale_byte = (is_v ? c.vs : c.ks)[at_page];
  const int64_t out_st = (int64_t)c.Hk * D;
  uint16_t* out = (is_v ? v_out : k_out) + blk.tok0 * out_st + head * D;
  if (is_v) {
    const Image<D, P> image{smem};
    for (int i = tid; i < D * (P / 16); i += kThreads) {
      const int d = i / (P / 16), s = 16 * (i % (P / 16));
      if (s + 16 > blk.s0 && s < blk.s1)
        *reinterpret_cast<u32x4*>(image.slot(d, s)) = *reinterpret_cast<const u32x4*>(page + d * P + s);
    }
    __syncthreads();
    const float scale = cache_scale(scale_byte);
    // 8 elements of four slots an item
    const int first = blk.s0 / 4, fours = (blk.s1 + 3) / 4 - first;
    for (int i = tid; i < fours * (D / 8); i += kThreads) {
      const int s = 4 * (first + i / (D / 8)), e = 8 * (i % (D / 8));
      u32x4 z[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        uint32_t w[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) w[f] = *reinterpret_cast<const uint32_t*>(image.slot(e + 4 * g + f, s));
        z[g] = transpose4(w[0], w[1], w[2], w[3]);
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        if (s + f < blk.s0 || s + f >= blk.s1) continue;
        const u32x4 o = {fp8_pair_to_bf16<0>(z[0][f], scale), fp8_pair_to_bf16<1>(z[0][f], scale),
                         fp8_pair_to_bf16<0>(z[1][f], scale), fp8_pair_to_bf16<1>(z[1][f], scale)};
        *reinterpret_cast<u32x4*>(out + (s + f - blk.s0) * out_st + e) = none ? zero4() : o;
      }
    }
  } else {
    const float scale = cache_scale(scale_byte);
    for (int i = tid; i < n * (D / 16); i += kThreads) {
      const int r = i / (D / 16), e = 16 * (i % (D / 16));
      u32x4 o[2];
      widen16(*reinterpret_cast<const u32x4*>(page + (blk.s0 + r) * D + e), scale, o);
      u32x4* dst = reinterpret_cast<u32x4*>(out + r * out_st + e);
      dst[0] = none ? zero4() : o[0];
      dst[1] = none ? zero4() : o[1];
    }
  }
}

unsigned touched_blocks(const CacheTokens& a, int lg) {
  return (unsigned)(a.cu == nullptr ? a.B : (a.T >> lg) + 2 * (int64_t)a.B);
}

// (kernel of D and the page's tokens, grid of pages touched x heads x keys and values)
#define SVDQ_CACHE_LAUNCH(kernel, d, p, ...)                                                                       \
  hipLaunchKernelGGL((kernel<d, p>), dim3(touched_blocks(a, c.lg_page), (unsigned)c.Hk, 2), dim3(kThreadsC<d, p>), 0, \
                     stream, a, c, __VA_ARGS__)
#define SVDQ_CACHE_PAGES(kernel, d, ...)                                     \
  do {                                                                       \
    if (c.lg_page == 4) SVDQ_CACHE_LAUNCH(kernel, d, 16, __VA_ARGS__);       \
    else if (c.lg_page == 5) SVDQ_CACHE_LAUNCH(kernel, d, 32, __VA_ARGS__);  \
    else if (c.lg_page == 6) SVDQ_CACHE_LAUNCH(kernel, d, 64, __VA_ARGS__);  \
    else SVDQ_CACHE_LAUNCH(kernel, d, 128, __VA_ARGS__);                     \
  } while (0)

}  // namespace

hipError_t launch_cache_append(const CacheTokens& a, const CacheShape& c, const HeadView& k, const HeadView& v,
                               hipStream_t stream) {
  if (c.D == 64) SVDQ_CACHE_PAGES(append_kernel, 64, k, v);
  else SVDQ_CACHE_PAGES(append_kernel, 128, k, v);
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheTokens& a, const CacheShape& c, uint16_t* k_out, uint16_t* v_out,
                             hipStream_t stream) {
  if (c.D == 64) SVDQ_CACHE_PAGES(read_kernel, 64, k_out, v_out);
  else SVDQ_CACHE_PAGES(read_kernel, 128, k_out, v_out);
  return hipGetLastError();
}

}  // namespace svdq
