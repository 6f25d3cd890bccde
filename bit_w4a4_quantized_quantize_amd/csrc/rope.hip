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

}  // namespace

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
