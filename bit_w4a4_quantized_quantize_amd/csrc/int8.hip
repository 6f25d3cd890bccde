// Linear in 8-bit integers with a scale per token and per output channel:
//
//   v = x * smooth,  a[m] = max_k |v|,  codes = rne(v * (127 / a)),  ascales = a / 127
//   y = bf16( (sum_k codes * weight) * ascales[m] * wscales[n] + bias[n] )
//
// on v_mfma_i32_32x32x32_i8: the sum over k is exact in int32 (127 * 128 * K
// stays below 2^31 up to K = 131072), so its order is free.
#include "common.h"
#include "kernels.h"

namespace svdq {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// 8 bf16 of x times 8 of smooth, in fp32 (exact)
template <bool SMOOTH>
__device__ __forceinline__ void scaled8(const u32x4 x, const u32x4 s, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo_to_f32(x[i]);
    v[2 * i + 1] = bf16hi_to_f32(x[i]);
    if (SMOOTH) {
      v[2 * i] *= bf16lo_to_f32(s[i]);
      v[2 * i + 1] *= bf16hi_to_f32(s[i]);
    }
  }
}

// One workgroup per row: the row's maximum, then its codes (the second read of the
// row comes from the caches).
template <bool SMOOTH>
__global__ __launch_bounds__(256) void quant_int8_kernel(const uint16_t* __restrict__ x,
                                                         const uint16_t* __restrict__ smooth, int K,
                                                         int8_t* __restrict__ codes, float* __restrict__ ascales) {
  __shared__ float part[4];
  const int tid = threadIdx.x;
  const size_t row = blockIdx.x;
  const u32x4* xr = reinterpret_cast<const u32x4*>(x + row * (size_t)K);
  const u32x4* sm = reinterpret_cast<const u32x4*>(smooth);
  const int nv = K / 8;
  float amax = 0.0f;
  for (int i = tid; i < nv; i += 256) {
    float v[8];
    scaled8<SMOOTH>(xr[i], SMOOTH ? sm[i] : zero4(), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
  if ((tid & 63) == 0) part[tid >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const Int8Scale q = int8_scale(amax);
  if (tid == 0) ascales[row] = q.scale;
  u32x2* out = reinterpret_cast<u32x2*>(codes + row * (size_t)K);
  for (int i = tid; i < nv; i += 256) {
    float v[8];
    scaled8<SMOOTH>(xr[i], SMOOTH ? sm[i] : zero4(), v);
    out[i] = int8_codes8(v, q.inv);
  }
}

// Four waves, 2 x 2, each one 32 x 32 tile with its operands straight from memory.
__global__ __launch_bounds__(256) void gemm_int8_kernel(Int8GemmArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int h = lane >> 5, l32 = lane & 31;
  const int64_t m0 = (int64_t)blockIdx.y * 64 + 32 * (wave & 1);
  const int64_t n0 = (int64_t)blockIdx.x * 64 + 32 * (wave >> 1);
  const int64_t K = a.K;
  const int64_t am = m0 + l32 < a.M ? m0 + l32 : a.M - 1;
  const int64_t bn = n0 + l32 < a.N ? n0 + l32 : a.N - 1;
  const int8_t* pa = a.codes + am * K + 16 * h;
  const int8_t* pb = a.weight + bn * K + 16 * h;
  i32x16 acc = {};
  for (int64_t k = 0; k < K; k += 32) {
    i32x4 fa = {}, fb = {};
    if (k + 16 * h < K) {   // K % 16 == 0: a 16-code piece is entirely before or past K
      fa = *reinterpret_cast<const i32x4*>(pa + k);
      fb = *reinterpret_cast<const i32x4*>(pb + k);
    }
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa, fb, acc, 0, 0, 0);
  }
  const int64_t n = n0 + l32;
  if (n >= a.N) return;
  const float ws = a.wscales[n];
  const float b = a.bias != nullptr ? bf16lo_to_f32(a.bias[n]) : 0.0f;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int64_t m = m0 + 8 * (r >> 2) + 4 * h + (r & 3);
    if (m < a.M) a.y[m * a.N + n] = (uint16_t)f32_to_bf16_rne((float)acc[r] * a.ascales[m] * ws + b);
  }
}

}  // namespace

hipError_t launch_quant_int8(const uint16_t* x, const uint16_t* smooth, int64_t M, int64_t K, int8_t* codes,
                             float* ascales, hipStream_t stream) {
  const dim3 grid((unsigned)M);
  if (smooth != nullptr)
    hipLaunchKernelGGL(quant_int8_kernel<true>, grid, dim3(256), 0, stream, x, smooth, (int)K, codes, ascales);
  else
    hipLaunchKernelGGL(quant_int8_kernel<false>, grid, dim3(256), 0, stream, x, smooth, (int)K, codes, ascales);
  return hipGetLastError();
}

size_t gemm_int8_workspace_bytes(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_gemm_int8(const Int8GemmArgs& a, void*, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 63) / 64), (unsigned)((a.M + 63) / 64));
  hipLaunchKernelGGL(gemm_int8_kernel, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace svdq
