// Rotary positions with several axes (time, height, width) and the per-head norm
// in front of them, q and k in one launch.
//
//   z = z / sqrt(mean z^2 + eps) * weight (optional), then pair p, the i-th of its
//   axis, turns by positions[t, axis] * theta^(-2 i / axis_dim).
//
// Angles: position * frequency in turns, in fp64, reduced to a fraction of a turn
// in [-1/2, 1/2] before it is rounded to fp32, so that far positions keep their
// phase (an fp32 product loses position * 2^-24 turns). One workgroup per token
// computes its D / 2 angles once for all heads.
#include "common.h"
#include "kernels.h"

#include <type_traits>

namespace svdq {

namespace {

// sum over groups of LANES (8 or 16) neighbouring lanes, the same value in each
template <int LANES>
__device__ __forceinline__ float sum_lanes(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), decltype(ctrl)::value, 0xF,
                                                                 0xF, true));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});    // quad_perm: lane ^ 1
  v += dpp(v, std::integral_constant<int, 0x4E>{});    // quad_perm: lane ^ 2
  v += dpp(v, std::integral_constant<int, 0x141>{});   // mirror of 8 lanes: the other quad
  if (LANES == 16) v += dpp(v, std::integral_constant<int, 0x140>{});   // mirror of 16 lanes: the other 8
  return v;
}

constexpr int kThreadsR = 256;
constexpr int kItems = 2;        // pieces of 8 elements per thread
constexpr int kMaxTokens = 16;   // tokens of a workgroup

// A workgroup takes `per` whole tokens, as many as fill its 512 pieces of 8 elements (one token,
// in several passes, where that has more): its loads go out first, then per * D / 2 angles are
// made in LDS, once for all heads, while they travel. Memory bound, close enough that vector
// instructions show: 16896 tokens of 30 + 30 heads of 128 out of a fused buffer move 519 MB in
// 87-91 us with the norm (5.7-6.0 TB/s, also over four sets of buffers in turn; in place inside the
// fused buffer 100-103); 103 us with the weights applied to the elements instead of the
// angles, an exact square root and quotient, and addresses made per lane. Scalar bases pay for
// one token per workgroup (ONE: 89 -> 87) and cost for several (8190 tokens of 24 + 8 heads of
// 64: 11.0 -> 11.6). Streaming stores are worth 5 us, against four pieces per thread 8, against
// one 2.
template <int D, bool INTER, bool NORM, bool ONE>
__global__ __launch_bounds__(kThreadsR) void rope_kernel(RopeArgs a, int per, int by_heads) {
  constexpr int kLanes = D / 8;            // lanes per head, 8 elements each
  // Per token and pair (u, w), pair 4 l + i of lane l at i * kLanes + l (whole rows of banks per
  // read): cos and sin; with the norm, for q and for k, the factors of u and w in u' and w' with
  // the weights in them: weight_u cos, weight_w sin, weight_w cos, weight_u sin
  extern __shared__ __attribute__((aligned(16))) float turn[];
  constexpr int kTable = NORM ? 8 * (D / 2) : 2 * (D / 2);   // floats of a token
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * per;
  const int here = (int)min((int64_t)per, a.T - t0);
  const int heads = a.H[0] + a.H[1];
  const int sub = tid % kLanes;
  // the 8 elements of this lane: interleaved, 8 consecutive (4 pairs); half-split,
  // 4 from each half (pairs 4 sub .. 4 sub + 3)
  const int e0 = INTER ? 8 * sub : 4 * sub;
  const int e1 = INTER ? 8 * sub + 4 : D / 2 + 4 * sub;
  const int items = here * heads;          // heads of this workgroup

  for (int first = 0; first < items; first += kItems * kThreadsR / kLanes) {
    u32x2 lo[kItems], hi[kItems];
    int tok[kItems];
    uint16_t* dst[kItems];
    bool is_k[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int it = min(first + (u * kThreadsR + tid) / kLanes, items - 1);   // clamped: read, not stored
      tok[u] = ONE ? 0 : (it * by_heads) >> 16;   // it / heads
      const int n = it - tok[u] * heads;
      is_k[u] = n >= a.H[0];
      const int head = is_k[u] ? n - a.H[0] : n;
      const uint16_t* src;
      if constexpr (ONE) {   // the token's bases are scalar
        src = (is_k[u] ? a.in[1].p + t0 * a.in[1].st : a.in[0].p + t0 * a.in[0].st) +
              head * (is_k[u] ? a.in[1].sh : a.in[0].sh);
        dst[u] = (is_k[u] ? a.out[1] + t0 * a.out_st[1] : a.out[0] + t0 * a.out_st[0]) +
                 head * (is_k[u] ? a.out_sh[1] : a.out_sh[0]);
      } else {
        const int64_t t = t0 + tok[u];
        const HeadView in = is_k[u] ? a.in[1] : a.in[0];
        src = in.p + t * in.st + head * in.sh;
        dst[u] = (is_k[u] ? a.out[1] : a.out[0]) + t * (is_k[u] ? a.out_st[1] : a.out_st[0]) +
                 head * (is_k[u] ? a.out_sh[1] : a.out_sh[0]);
      }
      if (INTER) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(src + e0);
        lo[u] = u32x2{w[0], w[1]};
        hi[u] = u32x2{w[2], w[3]};
      } else {
        lo[u] = *reinterpret_cast<const u32x2*>(src + e0);
        hi[u] = *reinterpret_cast<const u32x2*>(src + e1);
      }
    }
    if (first == 0) {
      for (int i = tid; i < here * (D / 2); i += kThreadsR) {
        const int p = i % (D / 2), k = i / (D / 2);
        const double x = (double)a.positions[(t0 + k) * a.axes + a.axis[p]] * a.turns[p];
        float s, c;
        sincospif(2.0f * (float)(x - __builtin_rint(x)), &s, &c);
        float* at = turn + k * kTable;
        const int slot = (p & 3) * kLanes + (p >> 2);
        if constexpr (NORM) {
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const uint16_t* w = side ? a.weight[1] : a.weight[0];
            const float wu = w != nullptr ? bf16lo_to_f32(w[INTER ? 2 * p : p]) : 1.0f;
            const float ww = w != nullptr ? bf16lo_to_f32(w[INTER ? 2 * p + 1 : p + D / 2]) : 1.0f;
            reinterpret_cast<f32x4*>(at)[side * (D / 2) + slot] = f32x4{wu * c, ww * s, ww * c, wu * s};
          }
        } else {
          reinterpret_cast<float2*>(at)[slot] = make_float2(c, s);
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v[2 * i] = bf16lo_to_f32(lo[u][i]);
        v[2 * i + 1] = bf16hi_to_f32(lo[u][i]);
        v[4 + 2 * i] = bf16lo_to_f32(hi[u][i]);
        v[5 + 2 * i] = bf16hi_to_f32(hi[u][i]);
      }
      float o[8];
      const float* at = turn + tok[u] * kTable;
      if constexpr (NORM) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
        ss = sum_lanes<kLanes>(ss) * (1.0f / D) + a.eps;
        // v_rsq_f32 (within one unit of the last place) takes no denormals
        float r = __builtin_amdgcn_rsqf(ss);
        if (__builtin_expect(__ballot(ss < 1e-30f) != 0, 0) && ss < 1e-30f) r = 1.0f / __builtin_sqrtf(ss);
        if ((is_k[u] ? a.weight[1] : a.weight[0]) == nullptr) r = 1.0f;
        const f32x4* f = reinterpret_cast<const f32x4*>(at) + (is_k[u] ? D / 2 : 0) + sub;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = INTER ? 2 * i : i, y = INTER ? 2 * i + 1 : 4 + i;
          const f32x4 w = f[i * kLanes];
          o[x] = (v[x] * w[0] - v[y] * w[1]) * r;
          o[y] = (v[y] * w[2] + v[x] * w[3]) * r;
        }
      } else {
        const float2* f = reinterpret_cast<const float2*>(at) + sub;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = INTER ? 2 * i : i, y = INTER ? 2 * i + 1 : 4 + i;
          const float2 cs = f[i * kLanes];
          o[x] = v[x] * cs.x - v[y] * cs.y;
          o[y] = v[y] * cs.x + v[x] * cs.y;
        }
      }
      if (first + (u * kThreadsR + tid) / kLanes < items) {
        const u32x2 w0 = {pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
        const u32x2 w1 = {pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
        if (INTER) {
          __builtin_nontemporal_store(u32x4{w0[0], w0[1], w1[0], w1[1]}, reinterpret_cast<u32x4*>(dst[u] + e0));
        } else {
          __builtin_nontemporal_store(w0, reinterpret_cast<u32x2*>(dst[u] + e0));
          __builtin_nontemporal_store(w1, reinterpret_cast<u32x2*>(dst[u] + e1));
        }
      }
    }
  }
}

template <int D, bool INTER>
void launch_rope_cfg(const RopeArgs& a, hipStream_t s) {
  const int pieces = (a.H[0] + a.H[1]) * (D / 8);
  const int64_t full = kItems * kThreadsR / pieces;
  // whole tokens per workgroup, fewer while the launch would leave CUs idle
  int64_t per = full < 1 ? 1 : full > kMaxTokens ? kMaxTokens : full;
  while (per > 1 && (a.T + per - 1) / per < 1024) per /= 2;
  const dim3 grid((unsigned)((a.T + per - 1) / per)), block(kThreadsR);
  const bool norm = a.weight[0] != nullptr || a.weight[1] != nullptr;
  // 1 / heads in units of 2^-16, rounded up: exact for the heads of several tokens (at most 64 in all)
  const int by_heads = (65536 + a.H[0] + a.H[1] - 1) / (a.H[0] + a.H[1]);
  const unsigned lds = (unsigned)(per * (D / 2) * (norm ? 32 : 8));   // at most 32 KB
  if (norm && per == 1) hipLaunchKernelGGL((rope_kernel<D, INTER, true, true>), grid, block, lds, s, a, 1, 0);
  else if (norm) hipLaunchKernelGGL((rope_kernel<D, INTER, true, false>), grid, block, lds, s, a, (int)per, by_heads);
  else if (per == 1) hipLaunchKernelGGL((rope_kernel<D, INTER, false, true>), grid, block, lds, s, a, 1, 0);
  else hipLaunchKernelGGL((rope_kernel<D, INTER, false, false>), grid, block, lds, s, a, (int)per, by_heads);
}

// Rotary positions on the first R elements of any head size, one position per token. A workgroup takes `per` whole
// tokens (one token in several passes, where that has more than 512 pieces): loads first, then the tokens' angles
// in LDS, once for all heads. A piece is 8 elements of a head; out of place, those past R are copied. Of the turned part
//   INTER: 8 consecutive ones, four pairs;
//   WIDE: 8 of one half, with 8 of the other read beside them (so not in place; 16 divides R): whole lines are written
//     where a head is turned in part;
//   else: 4 of each half; PART: a head is turned in part.
// Memory bound: 16896 tokens, 30 + 30 heads of 128 (519 MB) 93 us. Stores past the cache pay where a wave writes whole
// lines (R = 64 of 64 elements, 4099 tokens, 24 + 8 heads: 7.8 and 8.5 us without; the long one 93 and 101), and cost where
// it does not (R = 16, 4 of each half: 12.9 and 11.2 without; WIDE, with them, 8.0).
// by_heads, by_pieces: 2^32 / heads and / pieces of a head, rounded up (exact quotients below 2^16).
template <int PAIRS>
struct Turns {
  double at[PAIRS];   // per pair: its frequency in turns
};
template <bool INTER, bool WIDE, bool PART, int PAIRS>
__global__ __launch_bounds__(kThreadsR) void rope_scaled_kernel(RopeScaledArgs a, Turns<PAIRS> turns, int per,
                                                                uint32_t by_heads, uint32_t by_pieces) {
  static_assert(!INTER || !WIDE, "neighbours are in one piece");
  extern __shared__ __attribute__((aligned(16))) float turn[];   // per token and pair: cos and sin
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * per;
  const int here = (int)min((int64_t)per, a.T - t0);
  const int heads = a.H[0] + a.H[1], half = a.R / 2;
  const int turned = a.R / 8, pieces = a.copy ? a.D / 8 : turned;
  const int token_items = heads * pieces, items = here * token_items;

  for (int first = 0; first < items; first += kItems * kThreadsR) {
    u32x4 w[kItems], other[kItems];   // 8 elements (4 + 4: w only), WIDE: those of the other half
    int tok[kItems], piece[kItems];
    uint16_t* dst[kItems];
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const int it = min(first + u * kThreadsR + tid, items - 1);   // clamped: read, not stored
      const int n = pieces == 1 ? it : (int)__umulhi((uint32_t)it, by_pieces);
      piece[u] = it - n * pieces;
      tok[u] = heads == 1 ? n : (int)__umulhi((uint32_t)n, by_heads);
      const int head_all = n - tok[u] * heads;
      const bool is_k = head_all >= a.H[0];
      const int head = is_k ? head_all - a.H[0] : head_all;
      const int64_t t = t0 + tok[u];
      const HeadView in = is_k ? a.in[1] : a.in[0];
      const uint16_t* src = in.p + t * in.st + head * in.sh;
      dst[u] = (is_k ? a.out[1] : a.out[0]) + t * (is_k ? a.out_st[1] : a.out_st[0]) +
               head * (is_k ? a.out_sh[1] : a.out_sh[0]);
      if (INTER || WIDE || piece[u] >= turned) {
        w[u] = *reinterpret_cast<const u32x4*>(src + 8 * piece[u]);
        if (WIDE && piece[u] < turned)
          other[u] = *reinterpret_cast<const u32x4*>(src + 8 * piece[u] + (8 * piece[u] < half ? half : -half));
      } else {
        const u32x2 lo = *reinterpret_cast<const u32x2*>(src + 4 * piece[u]);
        const u32x2 hi = *reinterpret_cast<const u32x2*>(src + half + 4 * piece[u]);
        w[u] = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    }
    if (first == 0) {
      for (int i = tid; i < here * half; i += kThreadsR) {
        const int k = i / half, p = i - k * half;
        const double x = (double)a.positions[t0 + k] * turns.at[p];
        float s, c;
        sincospif(2.0f * (float)(x - __builtin_rint(x)), &s, &c);
        reinterpret_cast<float2*>(turn)[i] = make_float2(a.amplitude * c, a.amplitude * s);
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kItems; ++u) {
      const bool stored = first + u * kThreadsR + tid < items;
      if (piece[u] >= turned) {
        if (stored) __builtin_nontemporal_store(w[u], reinterpret_cast<u32x4*>(dst[u] + 8 * piece[u]));
        continue;
      }
      float v[8], o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16lo_to_f32(w[u][i]);
        v[2 * i + 1] = bf16hi_to_f32(w[u][i]);
      }
      const bool lower = 8 * piece[u] < half;   // WIDE
      const float2* f = reinterpret_cast<const float2*>(turn) + tok[u] * half +
                        (WIDE ? 8 * piece[u] - (lower ? 0 : half) : 4 * piece[u]);
      if (WIDE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float z = i % 2 ? bf16hi_to_f32(other[u][i / 2]) : bf16lo_to_f32(other[u][i / 2]);
          const float2 cs = f[i];
          const float s = lower ? -cs.y : cs.y;
          o[i] = v[i] * cs.x + z * s;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int x = INTER ? 2 * i : i, y = INTER ? 2 * i + 1 : 4 + i;
          const float2 cs = f[i];
          o[x] = v[x] * cs.x - v[y] * cs.y;
          o[y] = v[y] * cs.x + v[x] * cs.y;
        }
      }
      if (!stored) continue;
      const u32x4 r = {pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
      if (INTER || WIDE) {
        __builtin_nontemporal_store(r, reinterpret_cast<u32x4*>(dst[u] + 8 * piece[u]));
      } else {
        u32x2* at = reinterpret_cast<u32x2*>(dst[u] + 4 * piece[u]);
        u32x2* high = reinterpret_cast<u32x2*>(dst[u] + half + 4 * piece[u]);
        if (PART) {
          *at = u32x2{r[0], r[1]};
          *high = u32x2{r[2], r[3]};
        } else {
          __builtin_nontemporal_store(u32x2{r[0], r[1]}, at);
          __builtin_nontemporal_store(u32x2{r[2], r[3]}, high);
        }
      }
    }
  }
}

template <int PAIRS>
void launch_scaled(const RopeScaledArgs& a, const double* frequencies, bool interleaved, bool in_place, hipStream_t stream) {
  const int heads = a.H[0] + a.H[1], pieces = a.copy ? a.D / 8 : a.R / 8;
  const int64_t full = kItems * kThreadsR / ((int64_t)heads * pieces);
  int64_t per = full < 1 ? 1 : full > kMaxTokens ? kMaxTokens : full;
  while (per > 1 && (a.T + per - 1) / per < 1024) per /= 2;
  const dim3 grid((unsigned)((a.T + per - 1) / per)), block(kThreadsR);
  auto by = [](int n) { return (uint32_t)(((uint64_t(1) << 32) + n - 1) / n); };
  const unsigned lds = (unsigned)(per * a.R * 4);   // at most 16 KB
  Turns<PAIRS> turns;
  for (int i = 0; i < PAIRS; ++i) turns.at[i] = i < a.R / 2 ? frequencies[i] : 0.0;
  const bool part = a.R < a.D;
  if (interleaved)
    hipLaunchKernelGGL((rope_scaled_kernel<true, false, false, PAIRS>), grid, block, lds, stream, a, turns, (int)per, by(heads),
                       by(pieces));
  else if (part && !in_place && a.R % 16 == 0)
    hipLaunchKernelGGL((rope_scaled_kernel<false, true, false, PAIRS>), grid, block, lds, stream, a, turns, (int)per, by(heads),
                       by(pieces));
  else if (part)
    hipLaunchKernelGGL((rope_scaled_kernel<false, false, true, PAIRS>), grid, block, lds, stream, a, turns, (int)per, by(heads),
                       by(pieces));
  else
    hipLaunchKernelGGL((rope_scaled_kernel<false, false, false, PAIRS>), grid, block, lds, stream, a, turns, (int)per, by(heads),
                       by(pieces));
}

}  // namespace

hipError_t launch_rope_scaled(const RopeScaledArgs& a, const double* frequencies, bool interleaved, bool in_place,
                              hipStream_t stream) {
  // (a kernel's arguments of 1.2 KB take the caller 0.5 us more than those of 0.4)
  if (a.R <= 64) launch_scaled<32>(a, frequencies, interleaved, in_place, stream);
  else launch_scaled<128>(a, frequencies, interleaved, in_place, stream);
  return hipGetLastError();
}

hipError_t launch_rope(const RopeArgs& a, int D, bool interleaved, hipStream_t stream) {
  if (D == 64) {
    if (interleaved) launch_rope_cfg<64, true>(a, stream);
    else launch_rope_cfg<64, false>(a, stream);
  } else {
    if (interleaved) launch_rope_cfg<128, true>(a, stream);
    else launch_rope_cfg<128, false>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace svdq
