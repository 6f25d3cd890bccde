// Linear in 8-bit integers with a scale per token and per output channel:
//
//   v = x * smooth,  a[m] = max_k |v|,  codes = rne(v * (127 / a)),  ascales = a / 127
//   y = bf16( (sum_k codes * weight) * ascales[m] * wscales[n] + bias[n] )
//
// on v_mfma_i32_32x32x32_i8: the sum over k is exact in int32 (127 * 128 * K
// stays below 2^31 up to K = 131072), so its order is free.
//
// Bound by the matrix units' power for many tokens (4096 x 10240, K = 3840: 148-158 us, 2.0-2.2
// POP/s; a large library int8 product reaches 2.24), by the tiles' way from L2 through LDS for
// hundreds (333 x 3840, K = 10240: 30 us), by the weight's bytes for few (one token, 39 MB of weight
// from memory: 12.7 us). The quantiser moves 4096 x 3840 in 8.8 us (5.4 TB/s).
#include "common.h"
#include "kernels.h"
#include <math.h>

#define I8_LDS_PTR(p) ((__attribute__((address_space(3))) void*)(p))

namespace svdq {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

constexpr int kGroupM = 4;

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

// The row's maximum, then its codes. A row is held in registers by NW waves of NV 8-element
// pieces per lane (K <= NW * 64 * NV * 8), with NW = 1 a workgroup's four waves take a row each;
// NV = 0: rows of any length, read twice (the second time from the caches). Memory bound.
template <int NW, int NV, bool SMOOTH>
__global__ __launch_bounds__(NW == 1 ? 256 : 64 * NW) void quant_int8_kernel(const uint16_t* __restrict__ x,
                                                                             const uint16_t* __restrict__ smooth,
                                                                             int64_t M, int K,
                                                                             int8_t* __restrict__ codes,
                                                                             float* __restrict__ ascales) {
  constexpr int kThreads = 64 * NW;
  constexpr int kRows = NW == 1 ? 4 : 1;
  constexpr int kHeld = NV > 0 ? NV : 1;
  __shared__ float part[NW];
  const int tid = NW == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kRows +
                      (NW == 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) : 0);
  if (row >= M) return;
  const u32x4* xr = reinterpret_cast<const u32x4*>(x + (size_t)row * (size_t)K);
  const u32x4* sm = reinterpret_cast<const u32x4*>(smooth);
  const int nv = K / 8;
  float amax = 0.0f;
  float v[kHeld][8];
  if constexpr (NV > 0) {
    u32x4 w[kHeld], f[kHeld];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = tid + kThreads * u;
      w[u] = i < nv ? xr[i] : zero4();
      f[u] = SMOOTH && i < nv ? sm[i] : zero4();
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      scaled8<SMOOTH>(w[u], f[u], v[u]);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = max_or_nan(amax, fabsf(v[u][e]));
    }
  } else {
    for (int i = tid; i < nv; i += kThreads) {
      scaled8<SMOOTH>(xr[i], SMOOTH ? sm[i] : zero4(), v[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = max_or_nan(amax, fabsf(v[0][e]));
    }
  }
  amax = wave_reduce<true>(amax);
  if constexpr (NW > 1) {
    if ((tid & 63) == 0) part[tid >> 6] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) amax = max_or_nan(amax, part[w]);
  }
  const Int8Scale q = int8_scale(amax);
  if (tid == 0) ascales[row] = q.scale;
  u32x2* out = reinterpret_cast<u32x2*>(codes + (size_t)row * (size_t)K);
  if constexpr (NV > 0) {
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int i = tid + kThreads * u;
      if (i < nv) out[i] = int8_codes8(v[u], q.inv);
    }
  } else {
    for (int i = tid; i < nv; i += kThreads) {
      scaled8<SMOOTH>(xr[i], SMOOTH ? sm[i] : zero4(), v[0]);
      out[i] = int8_codes8(v[0], q.inv);
    }
  }
}

template <int NW, int NV>
void launch_quant_cfg(const uint16_t* x, const uint16_t* smooth, int64_t M, int64_t K, int8_t* codes, float* ascales,
                      hipStream_t s) {
  const int64_t wgs = NW == 1 ? (M + 3) / 4 : M;
  const int64_t gx = wgs < (1 << 20) ? wgs : (1 << 20);   // gridDim.x * threads stays below 2^32
  const dim3 grid((unsigned)gx, (unsigned)((wgs + gx - 1) / gx)), block(NW == 1 ? 256 : 64 * NW);
  if (smooth != nullptr)
    hipLaunchKernelGGL((quant_int8_kernel<NW, NV, true>), grid, block, 0, s, x, smooth, M, (int)K, codes, ascales);
  else
    hipLaunchKernelGGL((quant_int8_kernel<NW, NV, false>), grid, block, 0, s, x, smooth, M, (int)K, codes, ascales);
}

// (copies into LDS stay outside template-dependent code, see gemm_mx.hip)
__device__ __forceinline__ void i8_to_lds(__amdgpu_buffer_rsrc_t r, void* lds, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, I8_LDS_PTR(lds), 16, voff, soff, 0, 0);
}
template <int N>
__device__ __forceinline__ void wait_copies() {   // vmcnt(N), the other counters untouched
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}
__device__ __forceinline__ void barrier_no_fence() {   // as in gemm_bf16.hip: the waits are explicit
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Tile of a workgroup: WM x WN waves of TM x TN 32 x 32 outputs. A panel is 128 codes of k:
// chunks of 32 rows x 128 bytes, row r at r * 128 with its eight 16-byte pieces permuted by
// piece ^ swz(r), so that an operand read (32 rows, one piece each) meets every LDS
// bank evenly and a copy reads whole 128-byte row segments.
template <int WM, int WN, int TM, int TN, int S>
struct I8Cfg {
  static constexpr int kWaves = WM * WN;
  static constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN;
  static constexpr int kChunksA = BM / 32, kChunks = (BM + BN) / 32;
  static constexpr int kChunkBytes = 4096;
  static constexpr int kStageBytes = kChunks * kChunkBytes;
  static constexpr int kCopies = kChunks * 4;                    // 1 KB copies of a panel
  static constexpr int kPerWave = kCopies / kWaves;
  static constexpr int kOutBytes = kWaves * 32 * (32 * TN + 8) * 2 + BM * 4;   // output staging and row scales
  static constexpr int kLdsBytes = S * kStageBytes > kOutBytes ? S * kStageBytes : kOutBytes;
  static_assert(kCopies % kWaves == 0, "copies per wave");
};

struct I8Split {
  int panels;        // panels of k per split
  int splits;
  int32_t* partial;  // [splits, M, N] sums when splits > 1
};

template <int WM, int WN, int TM, int TN, int S, bool PIPE>
__global__ __launch_bounds__(64 * WM * WN) void gemm_int8_kernel(Int8GemmArgs a, I8Split sp) {
  using C = I8Cfg<WM, WN, TM, TN, S>;
  static_assert(S == 2 || (PIPE && S == 3), "two or three stages, the plain loop two");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int h = lane >> 5, l32 = lane & 31;
  const int wave_m = wave % WM, wave_n = wave / WM;
  const int M = (int)a.M, N = (int)a.N, K = (int)a.K;

  // XCD-contiguous tile ranges, kGroupM row blocks per column sweep
  const int NBX = (N + C::BN - 1) / C::BN, NBY = (M + C::BM - 1) / C::BM;
  const int per_xcd = (int)(gridDim.x / 8);
  int tile = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
  if (tile >= NBX * NBY * sp.splits) return;
  const int split = tile / (NBX * NBY);
  tile -= split * (NBX * NBY);
  const int per_group = kGroupM * NBX;
  const int first_row = (tile / per_group) * kGroupM;
  const int group_rows = min(NBY - first_row, kGroupM);
  const int m0 = (first_row + (tile % per_group) % group_rows) * C::BM;
  const int n0 = ((tile % per_group) / group_rows) * C::BN;

  const int rows_a = min(C::BM, M - m0), rows_b = min(C::BN, N - n0);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.codes + (size_t)m0 * K, (uint32_t)rows_a * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.weight + (size_t)n0 * K, (uint32_t)rows_b * (uint32_t)K);
  const int p0 = split * sp.panels;
  const int p1 = min(p0 + sp.panels, (K + 127) / 128);

  auto swz = [](int r) { return (r ^ (r >> 3)) & 7; };
  // copy c of a panel: chunk c / 4, rows 8 (c % 4) .. + 7; an offset past the buffer reads
  // zero (rows past the tensor, and pieces past K in the last panel)
  constexpr int kPast = 0x7FFFFFF0;
  int off[C::kPerWave];
#pragma unroll
  for (int u = 0; u < C::kPerWave; ++u) {
    const int c = wave + C::kWaves * u;
    const int r32 = 8 * (c & 3) + (lane >> 3);
    const bool is_a = c / 4 < C::kChunksA;
    const int row = 32 * (is_a ? c / 4 : c / 4 - C::kChunksA) + r32;
    off[u] = row < (is_a ? rows_a : rows_b) ? row * K + 16 * ((lane & 7) ^ swz(r32)) : kPast;
  }
  auto load_panel = [&](int kp) {
    uint8_t* st = smem + ((kp - p0) % S) * C::kStageBytes;
    const int k0 = kp * 128;
    const bool tail = k0 + 128 > K;
#pragma unroll
    for (int u = 0; u < C::kPerWave; ++u) {
      const int c = wave + C::kWaves * u;
      int v = off[u];
      if (tail && k0 + 16 * ((lane & 7) ^ swz(8 * (c & 3) + (lane >> 3))) >= K) v = kPast;
      if (c / 4 < C::kChunksA) i8_to_lds(ra, st + c * 1024, v, k0);
      else i8_to_lds(rb, st + c * 1024, v, k0);
    }
  };

  i32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  int frag[4];   // this lane's operand (row l32, piece 2 t + h of the 32-code step t) within a chunk
#pragma unroll
  for (int t = 0; t < 4; ++t) frag[t] = l32 * 128 + (((2 * t + h) ^ swz(l32)) * 16);
  auto read_set = [&](i32x4 (&dst)[TM + TN], const uint8_t* st, int t) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
      dst[i] = *reinterpret_cast<const i32x4*>(st + (wave_m * TM + i) * C::kChunkBytes + frag[t]);
#pragma unroll
    for (int j = 0; j < TN; ++j)
      dst[TM + j] = *reinterpret_cast<const i32x4*>(st + (C::kChunksA + wave_n * TN + j) * C::kChunkBytes + frag[t]);
  };
  auto multiply = [&](const i32x4 (&f)[TM + TN]) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f[i], f[TM + j], acc[i][j], 0, 0, 0);
  };

  if constexpr (PIPE) {
    // each step's operands are read between the previous step's products, one read after each of
    // the first TM + TN of them; the panel barrier sits before the last step
    i32x4 fr[2][TM + TN];
    auto step = [&](const i32x4 (&cur)[TM + TN], i32x4 (&nxt)[TM + TN], const uint8_t* st, int t, bool rd) {
      __builtin_amdgcn_sched_barrier(0);
      if (rd) read_set(nxt, st, t);
      multiply(cur);
      if (rd) {
        constexpr int kPairs = TM * TN < TM + TN ? TM * TN : TM + TN;
#pragma unroll
        for (int q = 0; q < kPairs; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one matrix instruction
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one LDS read
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // until the copies of a panel have landed: those of `later` panels may be in flight
    auto wait_panel = [&](int later) {
      if (S >= 3 && later >= 1) wait_copies<(S >= 3 ? 1 : 0) * C::kPerWave>();
      else wait_copies<0>();
    };
    if (p0 < p1) {
#pragma unroll
      for (int u = 0; u < S - 1; ++u)
        if (p0 + u < p1) load_panel(p0 + u);
      wait_panel(min(S - 2, p1 - 1 - p0));
      barrier_no_fence();
      if (p0 + S - 1 < p1) load_panel(p0 + S - 1);
      read_set(fr[0], smem, 0);
      for (int kp = p0; kp < p1; ++kp) {
        const uint8_t* cur = smem + ((kp - p0) % S) * C::kStageBytes;
        const uint8_t* nxt = smem + ((kp + 1 - p0) % S) * C::kStageBytes;
        // the waves of two workgroups on a SIMD run out of step by priority (192 x 128 tiles of two
        // stages: 1024 x 10240 59 -> 52 us, 2048 x 11520 112 -> 104; alone on a CU: equal)
        __builtin_amdgcn_s_setprio(1);
        step(fr[0], fr[1], cur, 1, true);
        step(fr[1], fr[0], cur, 2, true);
        step(fr[0], fr[1], cur, 3, true);
        __builtin_amdgcn_s_setprio(0);
        // this stage has been read to the end and panel kp + 1 has landed: publish it, then
        // refill this stage while the last step multiplies
        wait_panel(min(S - 2, p1 - 2 - kp));
        __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0)
        barrier_no_fence();
        if (kp + S < p1) load_panel(kp + S);
        step(fr[1], fr[0], nxt, 0, kp + 1 < p1);
      }
    }
  } else {
    if (p0 < p1) load_panel(p0);
    for (int kp = p0; kp < p1; ++kp) {
      __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0), lgkmcnt(0)
      barrier_no_fence();   // panel kp visible to every wave, the other stage is read to its end
      if (kp + 1 < p1) load_panel(kp + 1);
      const uint8_t* cur = smem + ((kp - p0) & 1) * C::kStageBytes;
      i32x4 f[TM + TN], g[TM + TN];
      read_set(f, cur, 0);
      read_set(g, cur, 1);
      multiply(f);
      read_set(f, cur, 2);
      multiply(g);
      read_set(g, cur, 3);
      multiply(f);
      multiply(g);
    }
  }
  __syncthreads();

  const int m_w = m0 + wave_m * TM * 32, n_w = n0 + wave_n * TN * 32;
  if (sp.splits > 1) {   // the partial sums; int8_reduce_kernel adds them and ends the product
    int32_t* out = sp.partial + (size_t)split * (size_t)M * (size_t)N;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int m = m_w + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3), n = n_w + 32 * j + l32;
          if (m < M && n < N) out[(size_t)m * (size_t)N + n] = acc[i][j][r];
        }
    return;
  }

  // the rows' scales in LDS, then bf16 output through LDS: each wave stages 32-row slices
  // row-major and stores whole 16-byte row pieces
  constexpr int kCols = 32 * TN, kPieces = kCols / 8, kPitch = kCols + 8;
  float* row_scale = reinterpret_cast<float*>(smem + C::kWaves * 32 * kPitch * 2);
  for (int i = tid; i < C::BM; i += 64 * C::kWaves) row_scale[i] = m0 + i < M ? a.ascales[m0 + i] : 0.0f;
  float ws[TN], bias[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int n = n_w + 32 * j + l32;
    ws[j] = n < N ? a.wscales[n] : 0.0f;
    bias[j] = a.bias != nullptr && n < N ? bf16lo_to_f32(a.bias[n]) : 0.0f;
  }
  __syncthreads();
  uint16_t* stage = reinterpret_cast<uint16_t*>(smem + wave * (32 * kPitch * 2));
  // A row of y starts (m N) mod 8 elements past a 16-byte address; it is staged with that shift, so
  // that whole pieces stay aligned on both sides (7345 x 11459, K = 528: 136 us, 204 by elements, 98
  // where 8 divides N)
  int shift[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) shift[r] = ((4 * h + r) * N) & 7;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = 8 * (r >> 2) + 4 * h + (r & 3);
      const float as = row_scale[wave_m * TM * 32 + 32 * i + row];
#pragma unroll
      for (int j = 0; j < TN; ++j)
        stage[row * kPitch + shift[r & 3] + 32 * j + l32] = (uint16_t)f32_to_bf16_rne((float)acc[i][j][r] * as * ws[j] + bias[j]);
    }
    __syncthreads();
    const int cols = min(kCols, N - n_w);
    if (N % 8 == 0) {
#pragma unroll
      for (int u = 0; u < 32 * kPieces / 64; ++u) {
        const int idx = lane + 64 * u;
        const int row = idx / kPieces, c = 8 * (idx % kPieces);
        const int m = m_w + 32 * i + row;
        if (m < M && c < cols)
          *reinterpret_cast<u32x4*>(a.y + (size_t)m * (size_t)N + n_w + c) =
              *reinterpret_cast<const u32x4*>(stage + row * kPitch + c);
      }
    } else {   // a piece more per row, the first and the last one by elements
      for (int idx = lane; idx < 32 * (kPieces + 1); idx += 64) {
        const int row = idx / (kPieces + 1), m = m_w + 32 * i + row;
        const int sh = ((row & 7) * N) & 7, c = 8 * (idx % (kPieces + 1)) - sh;
        if (m >= M || c >= cols) continue;
        uint16_t* dst = a.y + (size_t)m * (size_t)N + n_w;
        const u32x4 v = *reinterpret_cast<const u32x4*>(stage + row * kPitch + sh + c);
        if (c >= 0 && c + 8 <= cols) {
          *reinterpret_cast<u32x4*>(dst + c) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e >= 0 && c + e < cols) dst[c + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
    __syncthreads();
  }
}

// Ends a split product: sum of the partial sums, scales, bias, bf16; W channels per thread, 4 where
// that divides N, else 1 (M * N stays below 2^31: a split has at most 1024 workgroups).
template <int W>
__global__ __launch_bounds__(256) void int8_reduce_kernel(Int8GemmArgs a, const int32_t* __restrict__ partial,
                                                          int splits) {
  const uint32_t per_row = (uint32_t)a.N / W;
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  const uint32_t m = id / per_row, n = W * (id % per_row);
  if (m >= (uint32_t)a.M) return;
  const size_t mn = (size_t)a.M * (size_t)a.N, at = (size_t)m * (size_t)a.N + n;
  const float as = a.ascales[m];
  if constexpr (W == 4) {
    i32x4 s = *reinterpret_cast<const i32x4*>(partial + at);
    for (int i = 1; i < splits; ++i) s += *reinterpret_cast<const i32x4*>(partial + (size_t)i * mn + at);
    const f32x4 ws = *reinterpret_cast<const f32x4*>(a.wscales + n);
    u32x2 b = {0u, 0u};
    if (a.bias != nullptr) b = *reinterpret_cast<const u32x2*>(a.bias + n);
    const float y0 = (float)s[0] * as * ws[0] + bf16lo_to_f32(b[0]), y1 = (float)s[1] * as * ws[1] + bf16hi_to_f32(b[0]);
    const float y2 = (float)s[2] * as * ws[2] + bf16lo_to_f32(b[1]), y3 = (float)s[3] * as * ws[3] + bf16hi_to_f32(b[1]);
    *reinterpret_cast<u32x2*>(a.y + at) = u32x2{pack_bf16x2(y0, y1), pack_bf16x2(y2, y3)};
  } else {
    int32_t s = partial[at];
    for (int i = 1; i < splits; ++i) s += partial[(size_t)i * mn + at];
    const float b = a.bias != nullptr ? bf16lo_to_f32(a.bias[n]) : 0.0f;
    a.y[at] = (uint16_t)f32_to_bf16_rne((float)s * as * a.wscales[n] + b);
  }
}

// Few tokens (M <= 16 MT): bound by the weight's bytes, which stream past the tokens once,
// straight from memory. A workgroup takes 16 output channels, its eight waves share k in
// 64-code steps; v_mfma_i32_16x16x64_i8 with the weight rows as A and the tokens as B, and the
// waves' sums meet in LDS. QUANT: the activations come as x, and each workgroup first makes
// all the tokens' codes for itself in LDS (small M * K: cheaper than a launch of its own), with
// the first weight steps already on their way. LEAD: weight steps in flight per wave.
constexpr int kFewWaves = 8;

__host__ __device__ constexpr int few_pitch(int K) { return (K + 255) / 256 * 256 + 16; }   // LDS bytes of a token

template <int MT, int LEAD, bool QUANT, bool SMOOTH>
__global__ __launch_bounds__(64 * kFewWaves) void gemm_int8_few_kernel(Int8GemmArgs a, const uint16_t* __restrict__ x,
                                                                      const uint16_t* __restrict__ smooth) {
  __shared__ i32x4 part[kFewWaves][MT][64];
  __shared__ float scales[16 * MT];
  __shared__ float row_max[QUANT ? 16 * MT : 1][kFewWaves];
  extern __shared__ __attribute__((aligned(16))) uint8_t tok[];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int q = lane >> 4, l16 = lane & 15;
  const int M = (int)a.M, N = (int)a.N, K = (int)a.K;
  const int n0 = (int)blockIdx.x * 16;
  const int8_t* pw = a.weight + (size_t)min(n0 + l16, N - 1) * K + 16 * q;
  // K % 16 == 0: a 16-code piece is entirely before or past K, and zero past it
  auto weight_at = [&](int k) {
    const i32x4 zero = {};
    return k + 16 * q < K ? *reinterpret_cast<const i32x4*>(pw + k) : zero;
  };
  // a wave takes whole 128-byte lines, two steps each; its step u starts at lead(u)
  constexpr int kLine = 128 * kFewWaves;
  constexpr auto lead = [](int u) { return 64 * (u & 1) + kLine * (u >> 1); };
  const int k_first = 128 * wave;
  i32x4 fw[LEAD];
#pragma unroll
  for (int u = 0; u < LEAD; ++u) fw[u] = weight_at(k_first + lead(u));

  const int8_t* pt[MT];
  if constexpr (QUANT) {
    const int pitch = few_pitch(K), nv = K / 8;
    const u32x4* sm = reinterpret_cast<const u32x4*>(smooth);
    // 8, 4, 2 or 1 waves share a row
    const int wpr = M == 1 ? 8 : M == 2 ? 4 : M <= 4 ? 2 : 1;
    const int sub = (wave % wpr) * 64 + lane, step = 64 * wpr;
    for (int m = wave / wpr; m < M; m += kFewWaves / wpr) {
      const u32x4* xr = reinterpret_cast<const u32x4*>(x + (size_t)m * K);
      float amax = 0.0f;
      for (int i = sub; i < nv; i += step) {
        float v[8];
        scaled8<SMOOTH>(xr[i], SMOOTH ? sm[i] : zero4(), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max_or_nan(amax, fabsf(v[e]));
      }
      amax = wave_reduce<true>(amax);
      if (lane == 0) row_max[m][wave % wpr] = amax;
    }
    __syncthreads();
    for (int m = wave / wpr; m < M; m += kFewWaves / wpr) {
      const u32x4* xr = reinterpret_cast<const u32x4*>(x + (size_t)m * K);
      float amax = row_max[m][0];
      for (int w = 1; w < wpr; ++w) amax = max_or_nan(amax, row_max[m][w]);
      const Int8Scale qs = int8_scale(amax);
      if (sub == 0) scales[m] = qs.scale;
      for (int i = sub; i < nv; i += step) {
        float v[8];
        scaled8<SMOOTH>(xr[i], SMOOTH ? sm[i] : zero4(), v);
        *reinterpret_cast<u32x2*>(tok + m * pitch + 8 * i) = int8_codes8(v, qs.inv);
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) pt[t] = reinterpret_cast<const int8_t*>(tok) + min(16 * t + l16, M - 1) * pitch + 16 * q;
    __syncthreads();
  } else {
#pragma unroll
    for (int t = 0; t < MT; ++t) pt[t] = a.codes + (size_t)min(16 * t + l16, M - 1) * K + 16 * q;
    if (tid < 16 * MT) scales[tid] = tid < M ? a.ascales[tid] : 0.0f;
  }
  i32x4 acc[MT] = {};
  for (int k = k_first; k < K; k += lead(LEAD)) {
    i32x4 ft[LEAD][MT];
#pragma unroll
    for (int u = 0; u < LEAD; ++u)
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const i32x4 zero = {};
        const int at = k + lead(u);
        ft[u][t] = at + 16 * q < K ? *reinterpret_cast<const i32x4*>(pt[t] + at) : zero;
      }
#pragma unroll
    for (int u = 0; u < LEAD; ++u) {
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u], ft[u][t], acc[t], 0, 0, 0);
      fw[u] = weight_at(k + lead(LEAD + u));
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  // wave t ends token group t: lane l holds token l % 16, channels 4 (l / 16) .. + 3
  if (wave < MT) {
    i32x4 s = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += part[w][wave][lane];
    const int m = 16 * wave + l16;
    if (m < M) {
      const float as = scales[m];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = n0 + 4 * q + r;
        if (n < N) {
          const float b = a.bias != nullptr ? bf16lo_to_f32(a.bias[n]) : 0.0f;
          a.y[(size_t)m * (size_t)N + n] = (uint16_t)f32_to_bf16_rne((float)s[r] * as * a.wscales[n] + b);
        }
      }
    }
  }
}

template <int MT, int LEAD>
hipError_t launch_few_cfg(const Int8GemmArgs& a, const uint16_t* x, const uint16_t* smooth, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 15) / 16)), block(64 * kFewWaves);
  if (x == nullptr)
    hipLaunchKernelGGL((gemm_int8_few_kernel<MT, LEAD, false, false>), grid, block, 0, stream, a, x, smooth);
  if constexpr (MT <= 2) {   // few_from_x: at most 32 tokens
    const unsigned lds = (unsigned)a.M * few_pitch((int)a.K);
    if (x != nullptr && smooth == nullptr)
      hipLaunchKernelGGL((gemm_int8_few_kernel<MT, LEAD, true, false>), grid, block, lds, stream, a, x, smooth);
    else if (x != nullptr)
      hipLaunchKernelGGL((gemm_int8_few_kernel<MT, LEAD, true, true>), grid, block, lds, stream, a, x, smooth);
  }
  return hipGetLastError();
}

// Eight steps in flight while a workgroup has its CU to itself, four where more of them fit with
// fewer registers. Weights from memory, one token, four and eight: 3840 x 3840 6.8 and 5.9 us,
// 3840 x 10240 14.7 and 13.9, 10240 x 3840 12.7 and 14.1 (3.1 TB/s of 39 MB, 2.5 us of them a launch).
template <int MT>
hipError_t launch_few_mt(const Int8GemmArgs& a, const uint16_t* x, const uint16_t* smooth, hipStream_t stream) {
  return a.N <= 256 * 16 ? launch_few_cfg<MT, 8>(a, x, smooth, stream) : launch_few_cfg<MT, 4>(a, x, smooth, stream);
}

hipError_t launch_few(const Int8GemmArgs& a, const uint16_t* x, const uint16_t* smooth, hipStream_t stream) {
  return a.M <= 16   ? launch_few_mt<1>(a, x, smooth, stream)
         : a.M <= 32 ? launch_few_mt<2>(a, x, smooth, stream)
         : a.M <= 48 ? launch_few_mt<3>(a, x, smooth, stream)
                     : launch_few_mt<4>(a, x, smooth, stream);
}

// Tile shape, stages and split of k by an estimate in microseconds, fitted to times with weights
// from memory (M from 48 to 6000; ten weights from 1300 x 2064 to 11520 x 3840 and 3840 x 10240; every
// shape with k split 1 to 8 ways: profiles/gemm_int8_tile_grid.txt). A panel takes `share` of its
// CU's time per workgroup, at least `least` where a CU has too few of them; a CU works through
// ceil(workgroups / 256) of them; 5.2 us start and end a product. A split adds a launch (2 us on the
// device) and the partial sums' traffic (1.8 us per way at 333 x 3840). A call that is not in a graph
// takes no less than its caller, about 10 us and 3 more for a split's launch, so a split pays only
// where the device takes longer than that; among those that take the caller's time the shortest on
// the device. The choice is within 1% of the best device time on average and 8% at worst, but for 100
// to 200 tokens of 1300 x 2064 (18% to 9%: 9.8 us unsplit, 8.4 split three ways, where calls in a
// loop take 13). The 3 us added to a split's time instead cost 512 x 3840,
// K = 10240, 17% (41.6 us unsplit, 35.5 split four ways). Three stages, where they leave a CU one
// workgroup, pay while the tiles are few: at 1024 x 3840, K = 3840, 128 x 128 tiles take 24 us with
// three and 31 with two; at 333 x 3840, K = 10240, 192 x 128 tiles and k split four ways 30 and 33; at
// 1024 x 10240, K = 3840, 192 x 128 tiles 61 and 47. 4096 x 3840, K = 10240: 148 us in 256 x 256 tiles
// (240 of them), 165 in 256 x 320; 4096 x 10240, K = 3840: 171 and 158. 48 x 3840, K = 10240: 16 us in
// 64 x 64 tiles with k split four ways, 33 unsplit.
struct I8Plan {
  int shape;     // index into the table
  int splits, panels;
};

I8Plan plan_int8(int64_t M, int64_t N, int64_t K) {
  static const struct { int bm, bn; double share, least; } shapes[] = {
      {256, 320, 1.99, 1.99}, {256, 256, 1.54, 1.67}, {256, 128, 0.92, 1.00}, {192, 128, 0.86, 0.86},
      {192, 128, 0.67, 0.98}, {128, 128, 0.64, 0.64}, {128, 64, 0.36, 0.42},  {64, 64, 0.22, 0.28}};
  const int64_t panels = (K + 127) / 128;
  I8Plan best{0, 1, (int)panels};
  double best_t = 1e300;
  for (int s = 0; s < 8; ++s) {
    const int64_t tiles = ((M + shapes[s].bm - 1) / shapes[s].bm) * ((N + shapes[s].bn - 1) / shapes[s].bn);
    for (int sp = 1; sp <= 8; ++sp) {
      if (sp > 1 && (panels < 2 * sp || tiles * sp > 1024)) break;
      const int64_t per = (panels + sp - 1) / sp;
      const double rounds = (double)((tiles * sp + 255) / 256);
      const double device = 5.2 + (double)per * fmax(shapes[s].least, rounds * shapes[s].share) +
                            (sp > 1 ? 2.0 + 1.4e-6 * (double)(M * N) * sp : 0.0);
      const double t = fmax(device, sp > 1 ? 13.0 : 10.0) + 0.01 * device;
      if (t < best_t) {
        best_t = t;
        best = I8Plan{s, (int)((panels + per - 1) / per), (int)per};
      }
    }
  }
  return best;
}

template <int WM, int WN, int TM, int TN, int S, bool PIPE>
hipError_t launch_int8_cfg(const Int8GemmArgs& a, const I8Split& sp, hipStream_t stream) {
  using C = I8Cfg<WM, WN, TM, TN, S>;
  static std::atomic<uint64_t> lds_set{0};
  const void* fn = reinterpret_cast<const void*>(&gemm_int8_kernel<WM, WN, TM, TN, S, PIPE>);
  hipError_t e = set_lds_limit_once(fn, C::kLdsBytes, lds_set);
  if (e != hipSuccess) return e;
  const int64_t tiles = ((a.N + C::BN - 1) / C::BN) * ((a.M + C::BM - 1) / C::BM) * sp.splits;
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8));
  hipLaunchKernelGGL((gemm_int8_kernel<WM, WN, TM, TN, S, PIPE>), grid, dim3(64 * C::kWaves), C::kLdsBytes, stream, a, sp);
  return hipGetLastError();
}

// Every workgroup reads all the tokens' codes, and one of 16 channels works through all of k: above 8
// tokens only up to 2^17 codes and 2^24 weights (from memory, here and in tiles: 33 x 2064 for 1300
// channels 4.9 and 7.9 us, 48 x 2560 for 3840 8.5 and 9.4, 32 x 3840 for 3840 9.3 and 10.4, 48 x 3840
// 11.1 and 10.6, 16 x 3840 for 10240 16.1 and 13.4, 33 x 8192 for 1024 15.2 and 10.1). With up to 8 the
// tiles gain nothing (8 x 3840 for 10240: 13.9 and 13.4).
bool few_tokens(int64_t M, int64_t N, int64_t K) {
  return M <= 8 || (M <= 64 && M * K <= (int64_t(1) << 17) && N * K <= (int64_t(1) << 24));
}

// The layer from x in one launch: every workgroup makes the tokens' codes again, so only while they
// are few. Against two launches (N = 3840, on the device): 6.9 and 8.2 us for 1 x 3840, 7.7 and 8.5
// for 4 x 3840, 9.3 and 8.9 for 8 x 3840, 17.5 and 15.9 for 4 x 10240 (N = 1300: 7.4 and 6.2 for
// 9 x 2064); one launch saves another 3 us of the caller's time where the calls are not in a graph.
bool few_from_x(int64_t M, int64_t N, int64_t K) {
  // codes and sums together stay inside 64 KB of LDS
  const int64_t rows = M <= 8 ? M : (M + 7) / 8 * 8;   // above 8 a wave makes several rows
  return M <= 32 && few_tokens(M, N, K) && rows * K <= 32768 && M * few_pitch((int)K) <= 46 * 1024;
}

}  // namespace

hipError_t launch_quant_int8(const uint16_t* x, const uint16_t* smooth, int64_t M, int64_t K, int8_t* codes,
                             float* ascales, hipStream_t stream) {
  if (K <= 1024) launch_quant_cfg<1, 2>(x, smooth, M, K, codes, ascales, stream);
  else if (K <= 2048) launch_quant_cfg<4, 1>(x, smooth, M, K, codes, ascales, stream);
  else if (K <= 4096) launch_quant_cfg<4, 2>(x, smooth, M, K, codes, ascales, stream);
  else if (K <= 8192) launch_quant_cfg<8, 2>(x, smooth, M, K, codes, ascales, stream);
  else if (K <= 12288) launch_quant_cfg<8, 3>(x, smooth, M, K, codes, ascales, stream);
  else launch_quant_cfg<8, 0>(x, smooth, M, K, codes, ascales, stream);
  return hipGetLastError();
}

size_t gemm_int8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (few_tokens(M, N, K)) return 0;
  const I8Plan p = plan_int8(M, N, K);
  return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)N * 4 : 0;
}

void gemm_int8_plan(int64_t M, int64_t N, int64_t K, int* tile, int* splits) {
  const bool few = few_tokens(M, N, K);
  const I8Plan p = few ? I8Plan{-1, 1, 0} : plan_int8(M, N, K);
  *tile = p.shape;
  *splits = p.splits;
}

hipError_t launch_gemm_int8(const Int8GemmArgs& a, void* workspace, hipStream_t stream) {
  if (few_tokens(a.M, a.N, a.K)) return launch_few(a, nullptr, nullptr, stream);
  const I8Plan p = plan_int8(a.M, a.N, a.K);
  const I8Split sp{p.panels, p.splits, static_cast<int32_t*>(workspace)};
  hipError_t e = p.shape == 0   ? launch_int8_cfg<4, 2, 2, 5, 2, false>(a, sp, stream)
                 : p.shape == 1 ? launch_int8_cfg<4, 2, 2, 4, 2, true>(a, sp, stream)
                 : p.shape == 2 ? launch_int8_cfg<4, 2, 2, 2, 3, true>(a, sp, stream)
                 : p.shape == 3 ? launch_int8_cfg<2, 2, 3, 2, 3, true>(a, sp, stream)
                 : p.shape == 4 ? launch_int8_cfg<2, 2, 3, 2, 2, true>(a, sp, stream)
                 : p.shape == 5 ? launch_int8_cfg<2, 2, 2, 2, 3, true>(a, sp, stream)
                 : p.shape == 6 ? launch_int8_cfg<2, 2, 2, 1, 3, true>(a, sp, stream)
                                : launch_int8_cfg<2, 2, 1, 1, 3, true>(a, sp, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  const int w = a.N % 4 == 0 ? 4 : 1;
  const dim3 grid((unsigned)((a.M * (a.N / w) + 255) / 256));
  if (w == 4) hipLaunchKernelGGL(int8_reduce_kernel<4>, grid, dim3(256), 0, stream, a, sp.partial, p.splits);
  else hipLaunchKernelGGL(int8_reduce_kernel<1>, grid, dim3(256), 0, stream, a, sp.partial, p.splits);
  return hipGetLastError();
}

size_t linear_int8_codes_bytes(int64_t M, int64_t N, int64_t K) {
  return few_from_x(M, N, K) ? 0 : (size_t)M * (size_t)K;
}

hipError_t launch_linear_int8(const Int8GemmArgs& a, const uint16_t* x, const uint16_t* smooth, int8_t* codes,
                              float* ascales, void* workspace, hipStream_t stream) {
  if (few_from_x(a.M, a.N, a.K)) return launch_few(a, x, smooth, stream);
  hipError_t e = launch_quant_int8(x, smooth, a.M, a.K, codes, ascales, stream);
  if (e != hipSuccess) return e;
  Int8GemmArgs g = a;
  g.codes = codes;
  g.ascales = ascales;
  return launch_gemm_int8(g, workspace, stream);
}

}  // namespace svdq
