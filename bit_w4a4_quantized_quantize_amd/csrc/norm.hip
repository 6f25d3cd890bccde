// Norms before and after a transformer block, fused with its gate, the residual
// scale and the next block's modulation:
//
//   h_out = h + rs * gate[g] * (block / sqrt(mean block^2 + eps)) * post
//   x_out = (h_out / sqrt(mean h_out^2 + eps)) * pre * (1 + scale[g])
//
// One workgroup per row; the row stays in registers between the two sums, so h
// and block are read once and h_out and x_out (or x's int8 codes) written once:
// 16896 x 3840 moves 519 MB in 93 us (5.6 TB/s); to codes, with a block 84 us (5.4), without one
// 42 (4.7): there the vector instructions, about 13 an element, and the two reductions show, so
// the cases with both weights are code of their own (46 -> 42, 96 -> 93 us). Streaming stores are
// worth 3 us, weights requested before each sum 4. Long rows take eight waves: 4096 x 10240 to
// codes 29 us, with sixteen 63. Sums in fp32; x_out comes from h_out before its rounding to bf16.
#include "common.h"
#include "kernels.h"

namespace svdq {

namespace {

__device__ __forceinline__ void unpack8(const u32x4 w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo_to_f32(w[i]);
    v[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  return w;
}

// sum (or maximum) over the workgroup's NW waves, the same value in every lane
template <int NW, bool MAX>
__device__ __forceinline__ float reduce_wg(float v, float* part) {
  v = wave_reduce<MAX>(v);
  if (NW == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) v = MAX ? max_or_nan(v, part[w]) : v + part[w];
  return v;
}

// A row is held by NW waves of NV 8-element pieces per lane, K <= NW * 64 * NV * 8; with NW = 1
// a workgroup's four waves take a row each.
template <int NW, int NV, bool BLOCK>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void norm_gated_kernel(NormArgs a) {
  constexpr int kThreads = 64 * NW;
  constexpr int kRows = NW == 1 ? 4 : 1;
  constexpr bool kBoth = NW < 16;   // sixteen waves have no registers for the extra code
  __shared__ float part[3][NW];
  const int tid = NW == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kRows +
                      (NW == 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) : 0);
  if (row >= a.M) return;
  const int np = (int)(a.K / 8);
  const size_t base = (size_t)row * (size_t)a.K;
  const float rk = 1.0f / (float)a.K;
  auto piece = [](const uint16_t* p, size_t off, int i) {
    return *reinterpret_cast<const u32x4*>(p + off + 8 * (size_t)i);
  };

  // the row's loads go out before its group is looked up, and each norm's weights before its sum
  u32x4 hw[NV], bw[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int i = tid + kThreads * u;
    hw[u] = i < np ? piece(a.h, base, i) : zero4();
    if (BLOCK) bw[u] = i < np ? piece(a.block, base, i) : zero4();
  }
  int g = 0;
  if (a.cu != nullptr) {   // the group of the row: one less than the offsets up to it
    g = wave_count_le(a.cu, a.G + 1, row) - 1;
    if (g < 0 || g >= a.G) return;
  }
  const size_t gbase = (size_t)g * (size_t)a.K;
  auto weights = [&](const uint16_t* p, size_t off, u32x4 (&w)[NV]) {
    if (p == nullptr) return;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = tid + kThreads * u;
      if (i < np) w[u] = piece(p, off, i);
    }
  };
  u32x4 w1[NV], w2[NV];
  float h[NV][8];
  if (BLOCK) {
    weights(a.post, 0, w1);
    weights(a.gate, gbase, w2);
    float b[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      unpack8(bw[u], b[u]);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(b[u][e], b[u][e], ss);
    }
    ss = reduce_wg<NW, false>(ss, part[0]);
    const float r = a.rs / __builtin_sqrtf(ss * rk + a.eps);
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = tid + kThreads * u;
      unpack8(hw[u], h[u]);
      if (i < np) {
        float w[8], gt[8];
        if (a.post != nullptr) unpack8(w1[u], w);
        if (a.gate != nullptr) unpack8(w2[u], gt);
        if (kBoth && a.post != nullptr && a.gate != nullptr) {
#pragma unroll
          for (int e = 0; e < 8; ++e) h[u][e] = __builtin_fmaf(b[u][e], r * w[e] * gt[e], h[u][e]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float f = r;
            if (a.post != nullptr) f *= w[e];
            if (a.gate != nullptr) f *= gt[e];
            h[u][e] = __builtin_fmaf(b[u][e], f, h[u][e]);
          }
        }
        __builtin_nontemporal_store(pack8(h[u]), reinterpret_cast<u32x4*>(a.h_out + base + 8 * (size_t)i));
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < NV; ++u) unpack8(hw[u], h[u]);
  }
  if (a.x_out == nullptr && a.codes == nullptr) return;

  weights(a.pre, 0, w1);
  weights(a.scale, gbase, w2);
  float ss = 0.0f;
#pragma unroll
  for (int u = 0; u < NV; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(h[u][e], h[u][e], ss);
  ss = reduce_wg<NW, false>(ss, part[1]);
  const float r = 1.0f / __builtin_sqrtf(ss * rk + a.eps);
  u32x4 sw[NV];
  weights(a.smooth, 0, sw);
  float amax = 0.0f;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int i = tid + kThreads * u;
    if (i < np) {
      float w[8], sc[8];
      if (a.pre != nullptr) unpack8(w1[u], w);
      if (a.scale != nullptr) unpack8(w2[u], sc);
      if (kBoth && a.pre != nullptr && a.scale != nullptr) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[u][e] *= r * __builtin_fmaf(w[e], sc[e], w[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float f = r;
          if (a.pre != nullptr) f *= w[e];
          if (a.scale != nullptr) f *= 1.0f + sc[e];
          h[u][e] *= f;
        }
      }
      const u32x4 x = pack8(h[u]);
      if (a.codes == nullptr) {
        __builtin_nontemporal_store(x, reinterpret_cast<u32x4*>(a.x_out + base + 8 * (size_t)i));
      } else {   // the codes are those of the bf16 x
        unpack8(x, h[u]);
        if (a.smooth != nullptr) {
          float sm[8];
          unpack8(sw[u], sm);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[u][e] *= sm[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max_or_nan(amax, fabsf(h[u][e]));
      }
    }
  }
  if (a.codes == nullptr) return;
  amax = reduce_wg<NW, true>(amax, part[2]);
  const Int8Scale q = int8_scale(amax);
  if (tid == 0) a.ascales[row] = q.scale;
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int i = tid + kThreads * u;
    if (i < np) *reinterpret_cast<u32x2*>(a.codes + base + 8 * (size_t)i) = int8_codes8(h[u], q.inv);
  }
}

template <int NW, int NV>
void launch_norm_cfg(const NormArgs& a, hipStream_t s) {
  const int64_t wgs = NW == 1 ? (a.M + 3) / 4 : a.M;
  const int64_t gx = wgs < (1 << 20) ? wgs : (1 << 20);   // gridDim.x * threads stays below 2^32
  const dim3 grid((unsigned)gx, (unsigned)((wgs + gx - 1) / gx)), block(NW == 1 ? 256 : 64 * NW);
  if (a.block != nullptr)
    hipLaunchKernelGGL((norm_gated_kernel<NW, NV, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((norm_gated_kernel<NW, NV, false>), grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_norm_gated(const NormArgs& a, hipStream_t stream) {
  if (a.K <= 512) launch_norm_cfg<1, 1>(a, stream);
  else if (a.K <= 1024) launch_norm_cfg<1, 2>(a, stream);
  else if (a.K <= 2048) launch_norm_cfg<4, 1>(a, stream);
  else if (a.K <= 4096) launch_norm_cfg<4, 2>(a, stream);
  else if (a.K <= 8192) launch_norm_cfg<8, 2>(a, stream);
  else if (a.K <= 12288) launch_norm_cfg<8, 3>(a, stream);
  else if (a.K <= 16384) launch_norm_cfg<8, 4>(a, stream);
  else launch_norm_cfg<16, 4>(a, stream);
  return hipGetLastError();
}

}  // namespace svdq
