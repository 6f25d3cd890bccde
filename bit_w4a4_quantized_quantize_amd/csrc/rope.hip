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
// made in LDS, once for all heads, while they travel. Memory bound: 16896 tokens of 30 + 30
// heads of 128 move 519 MB in 105 us (4.9 TB/s); 110 us without the streaming stores, 114 with
// four pieces per thread in flight and no streaming stores.
template <int D, bool INTER, bool NORM>
__global__ __launch_bounds__(kThreadsR) void rope_kernel(RopeArgs a, int per) {
  constexpr int kLanes = D / 8;            // lanes per head, 8 elements each
  __shared__ float2 turn[kMaxTokens][D / 2];
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
      tok[u] = it / heads;
      const int n = it - tok[u] * heads;
      is_k[u] = n >= a.H[0];
      const int head = is_k[u] ? n - a.H[0] : n;
      const int64_t t = t0 + tok[u];
      const HeadView in = is_k[u] ? a.in[1] : a.in[0];
      const uint16_t* src = in.p + t * in.st + head * in.sh;
      dst[u] = (is_k[u] ? a.out[1] : a.out[0]) + t * (is_k[u] ? a.out_st[1] : a.out_st[0]) +
               head * (is_k[u] ? a.out_sh[1] : a.out_sh[0]);
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
        turn[k][p] = make_float2(c, s);
      }
      __syncthreads();
    }
    float wq[8], wk[8];
    if (NORM) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* w = i ? wk : wq;
        const uint16_t* p = i ? a.weight[1] : a.weight[0];
        u32x2 x0 = {0x3F803F80u, 0x3F803F80u}, x1 = x0;   // ones
        if (p != nullptr) {
          x0 = *reinterpret_cast<const u32x2*>(p + e0);
          x1 = *reinterpret_cast<const u32x2*>(p + e1);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w[2 * e] = bf16lo_to_f32(x0[e]);
          w[2 * e + 1] = bf16hi_to_f32(x0[e]);
          w[4 + 2 * e] = bf16lo_to_f32(x1[e]);
          w[5 + 2 * e] = bf16hi_to_f32(x1[e]);
        }
      }
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
      if (NORM) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
        ss = sum_lanes<kLanes>(ss);
        const bool on = (is_k[u] ? a.weight[1] : a.weight[0]) != nullptr;
        const float r = on ? 1.0f / __builtin_sqrtf(ss * (1.0f / D) + a.eps) : 1.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= r * (is_k[u] ? wk[e] : wq[e]);
      }
      float o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int x = INTER ? 2 * i : i, y = INTER ? 2 * i + 1 : 4 + i;
        const float2 cs = turn[tok[u]][4 * sub + i];
        o[x] = v[x] * cs.x - v[y] * cs.y;
        o[y] = v[y] * cs.x + v[x] * cs.y;
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
  if (a.weight[0] != nullptr || a.weight[1] != nullptr)
    hipLaunchKernelGGL((rope_kernel<D, INTER, true>), grid, block, 0, s, a, (int)per);
  else
    hipLaunchKernelGGL((rope_kernel<D, INTER, false>), grid, block, 0, s, a, (int)per);
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
