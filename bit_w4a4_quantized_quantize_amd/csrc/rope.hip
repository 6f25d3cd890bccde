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

namespace svdq {

namespace {

// One workgroup per token: D/2 cosines and sines into LDS, then D/8 lanes per head.
template <int D, bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a) {
  constexpr int kLanes = D / 8;            // lanes per head, 8 elements each
  constexpr int kHeads = 256 / kLanes;     // heads per pass
  __shared__ float cs[D / 2], sn[D / 2];
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  if (tid < D / 2) {
    const double turn = (double)a.positions[t * a.axes + a.axis[tid]] * a.turns[tid];
    const float f = (float)(turn - __builtin_rint(turn));
    float s, c;
    sincospif(2.0f * f, &s, &c);
    cs[tid] = c;
    sn[tid] = s;
  }
  __syncthreads();
  const int sub = tid % kLanes;
  const int heads = a.H[0] + a.H[1];
  // the 8 elements of this lane: interleaved, 8 consecutive (4 pairs); half-split,
  // 4 from each half (pairs 4 sub .. 4 sub + 3)
  const int e0 = INTER ? 8 * sub : 4 * sub;
  const int e1 = INTER ? 8 * sub + 4 : D / 2 + 4 * sub;
  for (int n0 = 0; n0 < heads; n0 += kHeads) {
    const int n = n0 + tid / kLanes;
    const bool live = n < heads;
    const int which = live && n >= a.H[0];
    const int head = live ? (which ? n - a.H[0] : n) : 0;
    float v[8];
    u32x2 w0 = {0u, 0u}, w1 = {0u, 0u};
    const uint16_t* src = a.in[which].p + t * a.in[which].st + head * a.in[which].sh;
    if (live) {
      w0 = *reinterpret_cast<const u32x2*>(src + e0);
      w1 = *reinterpret_cast<const u32x2*>(src + e1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = bf16lo_to_f32(w0[i]);
      v[2 * i + 1] = bf16hi_to_f32(w0[i]);
      v[4 + 2 * i] = bf16lo_to_f32(w1[i]);
      v[5 + 2 * i] = bf16hi_to_f32(w1[i]);
    }
    const uint16_t* wt = a.weight[which];
    float ss = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[e], v[e], ss);
#pragma unroll
    for (int d = kLanes / 2; d >= 1; d >>= 1) ss += __shfl_xor(ss, d);
    if (wt != nullptr) {
      const float r = 1.0f / __builtin_sqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] *= r * bf16lo_to_f32(wt[e0 + e]);
        v[4 + e] *= r * bf16lo_to_f32(wt[e1 + e]);
      }
    }
    float o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = INTER ? 2 * i : i, w = INTER ? 2 * i + 1 : 4 + i;
      const float c = cs[4 * sub + i], s = sn[4 * sub + i];
      o[u] = v[u] * c - v[w] * s;
      o[w] = v[w] * c + v[u] * s;
    }
    if (live) {
      uint16_t* dst = a.out[which] + t * a.out_st[which] + head * a.out_sh[which];
      *reinterpret_cast<u32x2*>(dst + e0) = u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
      *reinterpret_cast<u32x2*>(dst + e1) = u32x2{pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
    }
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int D, bool interleaved, hipStream_t stream) {
  const dim3 grid((unsigned)a.T), block(256);
  if (D == 64) {
    if (interleaved) hipLaunchKernelGGL((rope_kernel<64, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((rope_kernel<64, false>), grid, block, 0, stream, a);
  } else {
    if (interleaved) hipLaunchKernelGGL((rope_kernel<128, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((rope_kernel<128, false>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace svdq
