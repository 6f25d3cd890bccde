// Linear in 8-bit floating point (OCP e4m3) with a scale per block of 128 input channels:
//
//   v = x * smooth,  e = the least integer >= -100 with max |v| <= 448 * 2^e over 128 channels of a token,
//   codes = e4m3(v * 2^-e),  ascales = 2^e     (weights: over 128 x 128, the same rule)
//   y = bf16( sum_p ascales[p, m] * wscales[n / 128, p] * (sum_{k in p} codes[m, k] * weight[n, k]) + bias[n] )
//
// A power of two costs no precision (e4m3 keeps its three fraction bits down to 2^-15 of a block's maximum) and makes
// v * 2^-e exact, so the codes are bit-exact functions of x. The product takes any fp32 scales.
//
// The instruction adds the products of 8 neighbouring k aligned to the largest exponent among them and drops what lies
// below 2^-13 of it (measured; products within 2^7 of each other lose nothing); groups are added in fp32. The same
// product in bf16 matrix instructions, which keep all bits, would run at half the rate.
//
// A block of 128 is two v_mfma_f32_32x32x64_f8f6f4, the first from zero; their sum is added to the fp32 result times
// the block's two scales. The weight is the A operand, so that a lane holds channels of one token and its
// two scales are one factor per lane.
#include "common.h"
#include "kernels.h"
#include <math.h>

#define F8_LDS_PTR(p) ((__attribute__((address_space(3))) void*)(p))

namespace svdq {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kGroupM = 4;

// 8 bf16 of x times 8 of smooth, in fp32 (exact)
template <bool SMOOTH>
__device__ __forceinline__ void f8_scaled8(const u32x4 x, const u32x4 s, float (&v)[8]) {
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

// maximum over the 16 lanes of a row of the wave, the same value in each
__device__ __forceinline__ float max_row16(float v) {
#define SVDQ_DPP(x, ctrl) \
  __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, 0xF, 0xF, true))
  v = max_or_nan(v, SVDQ_DPP(v, 0xB1));
  v = max_or_nan(v, SVDQ_DPP(v, 0x4E));
  v = max_or_nan(v, SVDQ_DPP(v, 0x141));
  v = max_or_nan(v, SVDQ_DPP(v, 0x140));
#undef SVDQ_DPP
  return v;
}

// A workgroup takes 128 channels of 16 U tokens, 16 lanes of 8 channels each, a thread's loads in flight together; the
// scales, which are stored by blocks, leave 128 bytes at a time. Memory bound: 4096 x 3840 (47 MB from memory) 11.0 us, 333 x
// 10240 4.0. Consecutive blocks of a token in one workgroup instead, scales scattered: 13.5 and 4.7; U = 1 12.0 and 3.7, 4
// 11.7 and 4.4.
template <bool SMOOTH, int U>
__global__ __launch_bounds__(256) void quant_fp8_kernel(const uint16_t* __restrict__ x,
                                                        const uint16_t* __restrict__ smooth, uint32_t M, uint32_t K,
                                                        uint8_t* __restrict__ codes, float* __restrict__ ascales) {
  const uint32_t KB = (K + 127) / 128;
  const uint32_t rows = blockIdx.x / KB, block = blockIdx.x - rows * KB;
  const uint32_t k = 128 * block + 8 * (threadIdx.x & 15);
  u32x4 w[U], f = zero4();
  uint32_t row[U];
  if (SMOOTH && k < K) f = *reinterpret_cast<const u32x4*>(smooth + k);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    row[u] = (rows * U + u) * 16 + threadIdx.x / 16;
    w[u] = row[u] < M && k < K ? *reinterpret_cast<const u32x4*>(x + (size_t)row[u] * K + k) : zero4();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float v[8];
    f8_scaled8<SMOOTH>(w[u], f, v);
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max_or_nan(amax, fabsf(v[e]));
    amax = max_row16(amax);
    const Fp8Scale q = fp8_scale(amax);
    if (row[u] < M && k < K) {
      *reinterpret_cast<u32x2*>(codes + (size_t)row[u] * K + k) = fp8_codes8(v, q.inv);
      if ((threadIdx.x & 15) == 0) ascales[(size_t)block * M + row[u]] = q.scale;
    }
  }
}

// A weight's block of 128 x 128 per workgroup: two threads a row, 64 channels each. Load time.
template <bool SMOOTH>
__global__ __launch_bounds__(256) void quant_weight_fp8_kernel(const uint16_t* __restrict__ w,
                                                               const uint16_t* __restrict__ smooth, int N, int K,
                                                               uint8_t* __restrict__ codes,
                                                               float* __restrict__ wscales) {
  __shared__ float part[4];
  const int n = 128 * (int)blockIdx.y + (int)threadIdx.x / 2;
  const int k0 = 128 * (int)blockIdx.x + 64 * ((int)threadIdx.x & 1);
  const int KB = (K + 127) / 128;
  u32x4 held[8];
  float amax = 0.0f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const bool in = n < N && k0 + 8 * u < K;
    held[u] = in ? *reinterpret_cast<const u32x4*>(w + (size_t)n * K + k0 + 8 * u) : zero4();
    float v[8];
    f8_scaled8<SMOOTH>(held[u], SMOOTH && in ? *reinterpret_cast<const u32x4*>(smooth + k0 + 8 * u) : zero4(), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = max_or_nan(amax, fabsf(v[e]));
  }
  amax = wave_reduce<true>(amax);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) amax = max_or_nan(amax, part[i]);
  const Fp8Scale q = fp8_scale(amax);
  if (threadIdx.x == 0) wscales[(size_t)blockIdx.y * KB + blockIdx.x] = q.scale;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (n < N && k0 + 8 * u < K) {
      float v[8];
      f8_scaled8<SMOOTH>(held[u], SMOOTH ? *reinterpret_cast<const u32x4*>(smooth + k0 + 8 * u) : zero4(), v);
      *reinterpret_cast<u32x2*>(codes + (size_t)n * K + k0 + 8 * u) = fp8_codes8(v, q.inv);
    }
  }
}

// (copies into LDS stay outside template-dependent code, see gemm_mx.hip)
__device__ __forceinline__ void f8_to_lds(__amdgpu_buffer_rsrc_t r, void* lds, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, F8_LDS_PTR(lds), 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void f8_to_lds4(__amdgpu_buffer_rsrc_t r, void* lds, int voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, F8_LDS_PTR(lds), 4, voff, 0, 0, 0);
}
template <int N>
__device__ __forceinline__ void f8_wait_copies() {   // vmcnt(N), lgkmcnt(0)
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
}
__device__ __forceinline__ f32x16 f8_mfma32(i32x8 a, i32x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);   // e4m3 both, unscaled
}
__device__ __forceinline__ f32x4 f8_mfma16(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ i32x8 join8(i32x4 a, i32x4 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }
__device__ __forceinline__ void f8_barrier() {   // as in gemm_bf16.hip: the waits are explicit
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Tile of a workgroup: WM x WN waves of TM x TN blocks of 32 tokens x 32 channels. A panel is the 128 codes of a
// scale block and its scales: chunks of 32 rows x 128 bytes, row r at r * 128 with its eight 16-byte pieces
// permuted by piece ^ swz(r), so that an operand read (32 rows, one piece each) meets every LDS
// bank evenly and a copy reads whole 128-byte row segments.
// 4096 x 10240, K = 3840: 150 us (2.15 PFLOP/s; a library's product with one scale a tensor reaches 3.2). The matrix units
// are busy 55% of the time and the vector units, most of it adding the scaled sums, 48%; without those additions it takes
// 27 us less, without the copies 24. 333 x 3840, K = 10240: 27 us and 5 to add four partial sums; operand traffic
// (190 MB through the L2s, 7 TB/s) and the latency of one workgroup a CU.
template <int WM, int WN, int TM, int TN, int S>
struct F8Cfg {
  static constexpr int kWaves = WM * WN;
  static constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN;
  static constexpr int kChunksA = BM / 32, kChunks = (BM + BN) / 32;
  static constexpr int kChunkBytes = 4096;
  static constexpr int kScalesA = kChunks * kChunkBytes;         // the tokens' scales
  static constexpr int kStageBytes = kScalesA + BM * 4;
  static constexpr int kCopies = kChunks * 4;                    // 1 KB copies of a panel
  static constexpr int kPerWave = kCopies / kWaves;
  static constexpr int kOutBytes = kWaves * 32 * (32 * TN + 8) * 2;   // output staging
  static constexpr int kLdsBytes = S * kStageBytes + 512 > kOutBytes ? S * kStageBytes + 512 : kOutBytes;
  static_assert(kCopies % kWaves == 0, "copies per wave");
};

struct F8Split {
  int panels;        // panels of k per split
  int splits;
  float* partial;    // [splits, M, N] sums when splits > 1
};

template <int WM, int WN, int TM, int TN, int S>
__global__ __launch_bounds__(64 * WM * WN) void gemm_fp8_kernel(Fp8GemmArgs a, F8Split sp) {
  using C = F8Cfg<WM, WN, TM, TN, S>;
  static_assert(S >= 2 && S <= 4, "stages");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int h = lane >> 5, l32 = lane & 31;
  const int wave_m = wave % WM, wave_n = wave / WM;
  const int M = (int)a.M, N = (int)a.N, K = (int)a.K;
  const int KB = (K + 127) / 128;

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
  const int m_w = m0 + wave_m * TM * 32, n_w = n0 + wave_n * TN * 32;

  const int rows_a = min(C::BM, M - m0), rows_b = min(C::BN, N - n0);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(a.codes + (size_t)m0 * K, (uint32_t)rows_a * (uint32_t)K);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(a.weight + (size_t)n0 * K, (uint32_t)rows_b * (uint32_t)K);
  const int p0 = split * sp.panels;
  const int p1 = min(p0 + sp.panels, KB);

  auto swz = [](int r) { return (r ^ (r >> 3)) & 7; };
  // Copy u of a wave: its 8 rows are 8 kWaves further on with each u, at the same pieces. Rows past the tensor are past
  // the buffer and read zero; so do pieces past K in the last panel, at an offset that is.
  constexpr int kPast = 0x7FFFFFF0;
  static_assert(C::kWaves % 4 == 0 && C::kChunksA * 4 % C::kWaves == 0, "a wave's copies are of the tokens, then of the weight");
  constexpr int kCopiesA = C::kChunksA * 4 / C::kWaves;
  const int piece = 16 * ((lane & 7) ^ swz(8 * (wave & 3) + (lane >> 3)));
  int copy_at = (8 * wave + (lane >> 3)) * K + piece;
  const int copy_step = 8 * C::kWaves * K;
  // The scales of a panel: 64 tokens' by each of the first waves; the tile's channels' for 16 panels at a time, by the last
  // wave, panel i of block b in lane 16 b + i (two places in turn).
  const int as_off = 4 * (m0 + 64 * wave + lane);
  const int nb0 = n0 / 128, n_blocks = min((N + 127) / 128 - nb0, 4);
  const int ws_off = 4 * ((lane >> 4) * KB + (lane & 15));
  const __amdgpu_buffer_rsrc_t rws = make_rsrc(a.wscales + (size_t)nb0 * KB, (uint32_t)n_blocks * (uint32_t)KB * 4u);
  static_assert(C::BN <= 384, "at most 4 blocks of 128 channels, aligned to 64");
  // Panel kp's copies, part `part` of kParts (all but the first go out between the next panel's products); panels past
  // the last land as zeros: no branch.
  constexpr int kParts = TN >= 3 ? 3 : TN;
  auto load_panel = [&](int kp, int part) {
    uint8_t* st = smem + ((kp - p0) % S) * C::kStageBytes;
    const int k0 = kp * 128;
    const bool none = kp >= p1;
    const bool past = none || k0 + piece >= K;
    asm volatile("" : "+v"(copy_at));   // the copies' offsets are made here, not kept
#pragma unroll
    for (int u = 0; u < C::kPerWave; ++u) {
      if (u * kParts / C::kPerWave != part) continue;
      const bool is_a = u < kCopiesA;
      const int v = past ? kPast : copy_at + (is_a ? u : u - kCopiesA) * copy_step;
      f8_to_lds(is_a ? ra : rb, st + (wave + C::kWaves * u) * 1024, v, k0);
    }
    if (part == 0) {
      if (wave < C::BM / 64)
        f8_to_lds4(make_rsrc(a.ascales + (size_t)(none ? 0 : kp) * M, (uint32_t)M * 4u), st + C::kScalesA + 256 * wave, as_off);
      if (wave == C::kWaves - 1 && (kp - p0) % 16 == 0)
        f8_to_lds4(rws, smem + S * C::kStageBytes + ((kp - p0) & 16) * 16, ws_off + 4 * (none ? 0 : kp));
    }
  };

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x16{};

  // this lane's operand pieces (row l32, piece 2 t + h) within a chunk: 32 t by exclusive or from t = 0
  int frag = l32 * 128 + ((h ^ swz(l32)) * 16);
  auto operand = [&](const uint8_t* chunk, int s) {
    return join8(*reinterpret_cast<const i32x4*>(chunk + (frag ^ (64 * s))),
                 *reinterpret_cast<const i32x4*>(chunk + (frag ^ (64 * s + 32))));
  };
  const int chunk_m = wave_m * TM * C::kChunkBytes, chunk_n = (C::kChunksA + wave_n * TN) * C::kChunkBytes;

  // Block j of channels: the products of both halves of the panel with each block of tokens, then the sums times their
  // scales. A sum is added while another's matrix instruction runs (the first one's beside the last one's second
  // half, the others' beside the next block's first halves), and each operand is read for the next
  // block (or the next panel) as soon as its last product is issued. One barrier a panel, before its last block: it frees
  // the panel, which is read to its end, and publishes the next one.
  i32x8 ft[TM][2], fw[2];
  f32x16 sum[TM];
  float as[TM], ws;
  const int as_lane = C::kScalesA + 4 * (wave_m * TM * 32 + l32);
  auto read_as = [&](const uint8_t* st, int i) { return *reinterpret_cast<const float*>(st + as_lane + 128 * i); };
  auto read_ws = [&](int kp, int j) {   // a block of 128 holds whole blocks of 32
    const int at = kp - p0;
    return *reinterpret_cast<const float*>(smem + S * C::kStageBytes + (at & 16) * 16 + 64 * ((n_w + 32 * j) / 128 - nb0) +
                                           4 * (at & 15));
  };
  auto add_sum = [&](int i, int j, float s) {
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][j][r] = __builtin_fmaf(sum[i][r], s, acc[i][j][r]);
    asm volatile("" : "+v"(acc[i][j]));   // added here: the sums' registers are free
  };
  constexpr int kFirst = (C::kPerWave + kParts - 1) / kParts;   // copies of a panel's first part
  if (p0 < p1) {
#pragma unroll
    for (int u = 0; u < S; ++u)
#pragma unroll
      for (int part = 0; part < (u < S - 1 ? kParts : 1); ++part) load_panel(p0 + u, part);
    // (waves with copies of scales wait for a little more than panel p0)
    f8_wait_copies<(S - 2) * C::kPerWave + kFirst>();
    f8_barrier();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int i = 0; i < TM; ++i) ft[i][s] = operand(smem + chunk_m + i * C::kChunkBytes, s);
      fw[s] = operand(smem + chunk_n, s);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) as[i] = read_as(smem, i);
    ws = read_ws(p0, 0);
    float scale[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      sum[i] = f32x16{};
      scale[i] = 0.0f;
    }
    for (int kp = p0; kp < p1; ++kp) {
      const uint8_t* cur = smem + ((kp - p0) % S) * C::kStageBytes;
      const uint8_t* nxt = smem + ((kp - p0 + 1) % S) * C::kStageBytes;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const bool last = j == TN - 1;
        if (last) {
          f8_wait_copies<(S - 2) * C::kPerWave>();   // panel kp + 1 has landed, panel kp is read
          f8_barrier();
          load_panel(kp + S, 0);
        } else if (j + 1 < kParts) {
          load_panel(kp + S - 1, j + 1);
        }
        // (after the last panel: whatever its stage holds, not used)
        const uint8_t* next_w = last ? nxt + chunk_n : cur + chunk_n + (j + 1) * C::kChunkBytes;
        asm volatile("" : "+v"(frag));
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          if (i > 0) add_sum(i, (j + TN - 1) % TN, scale[i]);
          scale[i] = as[i] * ws;
          sum[i] = f8_mfma32(fw[0], ft[i][0], f32x16{});
          __builtin_amdgcn_sched_barrier(0);
        }
        fw[0] = operand(next_w, 0);
        if (last) {
#pragma unroll
          for (int i = 0; i < TM; ++i) ft[i][0] = operand(nxt + chunk_m + i * C::kChunkBytes, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          sum[i] = f8_mfma32(fw[1], ft[i][1], sum[i]);
          __builtin_amdgcn_sched_barrier(0);
        }
        fw[1] = operand(next_w, 1);
        if (last) {
#pragma unroll
          for (int i = 0; i < TM; ++i) ft[i][1] = operand(nxt + chunk_m + i * C::kChunkBytes, 1);
        }
        ws = read_ws(last ? kp + 1 : kp, last ? 0 : j + 1);
        if (last) {
#pragma unroll
          for (int i = 0; i < TM; ++i) as[i] = read_as(nxt, i);
        }
        __builtin_amdgcn_sched_barrier(0);
        add_sum(0, j, scale[0]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int i = 1; i < TM; ++i) add_sum(i, TN - 1, scale[i]);
    f8_wait_copies<0>();   // nothing lands in LDS from here on
  }

  // this lane holds channels n_w + 32 j + 8 (r / 4) + 4 h + r % 4 of token m_w + 32 i + l32
  if (sp.splits > 1) {   // the partial sums; fp8_reduce_kernel adds them and ends the product
    float* out = sp.partial + (size_t)split * (size_t)M * (size_t)N;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = m_w + 32 * i + l32;
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const int n = n_w + 32 * j + 2 * r + 4 * h;
          float* dst = out + (size_t)m * (size_t)N + n;
          if (m < M && n < N) {
            if (N % 4 == 0) {
              *reinterpret_cast<f32x4*>(dst) = f32x4{acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (n + e < N) dst[e] = acc[i][j][r + e];
            }
          }
        }
    }
    return;
  }

  // bf16 output through LDS: each wave stages 32 tokens row-major and stores whole 16-byte row pieces. A
  // row of y starts (m N) mod 8 elements past a 16-byte address; it is staged with that shift, so
  // that whole pieces stay aligned on both sides.
  __syncthreads();
  constexpr int kCols = 32 * TN, kPieces = kCols / 8, kPitch = kCols + 8;
  uint16_t* stage = reinterpret_cast<uint16_t*>(smem + wave * (32 * kPitch * 2));
  const int shift = (l32 * N) & 7;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const int c = 32 * j + 2 * r + 4 * h;
        float v[4] = {acc[i][j][r], acc[i][j][r + 1], acc[i][j][r + 2], acc[i][j][r + 3]};
        if (a.bias != nullptr) {
          const int n = n_w + c;
          if (N % 4 == 0) {
            const u32x2 b = n < N ? *reinterpret_cast<const u32x2*>(a.bias + n) : u32x2{0u, 0u};
            v[0] += bf16lo_to_f32(b[0]);
            v[1] += bf16hi_to_f32(b[0]);
            v[2] += bf16lo_to_f32(b[1]);
            v[3] += bf16hi_to_f32(b[1]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] += n + e < N ? bf16lo_to_f32(a.bias[n + e]) : 0.0f;
          }
        }
        uint16_t* dst = stage + l32 * kPitch + shift + c;
        const uint32_t w0 = pack_bf16x2(v[0], v[1]), w1 = pack_bf16x2(v[2], v[3]);
        if (N % 4 == 0) {
          *reinterpret_cast<u32x2*>(dst) = u32x2{w0, w1};
        } else {
          dst[0] = (uint16_t)w0;
          dst[1] = (uint16_t)(w0 >> 16);
          dst[2] = (uint16_t)w1;
          dst[3] = (uint16_t)(w1 >> 16);
        }
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
        const int sh = (row * N) & 7, c = 8 * (idx % (kPieces + 1)) - sh;
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

// Ends a split product: the partial sums in split order, bias, bf16; W channels per thread, 4 where
// that divides N, else 1 (M * N stays below 2^31: a split has at most 1024 workgroups).
template <int W>
__global__ __launch_bounds__(256) void fp8_reduce_kernel(Fp8GemmArgs a, const float* __restrict__ partial, int splits) {
  const uint32_t per_row = (uint32_t)a.N / W;
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  const uint32_t m = id / per_row, n = W * (id % per_row);
  if (m >= (uint32_t)a.M) return;
  const size_t mn = (size_t)a.M * (size_t)a.N, at = (size_t)m * (size_t)a.N + n;
  if constexpr (W == 4) {
    f32x4 s = *reinterpret_cast<const f32x4*>(partial + at);
    for (int i = 1; i < splits; ++i) s += *reinterpret_cast<const f32x4*>(partial + (size_t)i * mn + at);
    u32x2 b = {0u, 0u};
    if (a.bias != nullptr) b = *reinterpret_cast<const u32x2*>(a.bias + n);
    *reinterpret_cast<u32x2*>(a.y + at) =
        u32x2{pack_bf16x2(s[0] + bf16lo_to_f32(b[0]), s[1] + bf16hi_to_f32(b[0])),
              pack_bf16x2(s[2] + bf16lo_to_f32(b[1]), s[3] + bf16hi_to_f32(b[1]))};
  } else {
    float s = partial[at];
    for (int i = 1; i < splits; ++i) s += partial[(size_t)i * mn + at];
    a.y[at] = (uint16_t)f32_to_bf16_rne(a.bias != nullptr ? s + bf16lo_to_f32(a.bias[n]) : s);
  }
}

// Few tokens (M <= 16 MT): bound by the weight's bytes, which stream past the tokens once, straight
// from memory. A workgroup takes 16 output channels, its eight waves share k in blocks of 128;
// v_mfma_f32_16x16x128_f8f6f4 with the weight rows as A and the tokens as B, and the waves' sums
// meet in LDS. QUANT: the activations come as x, and each workgroup first makes all the tokens' codes
// for itself in LDS (small M * K: cheaper than a launch of its own), with the first weight blocks already on their way.
// LEAD: weight blocks in flight per wave.
// One token, 3840 x 3840 (14.8 MB from memory): 6.3 us, a fifth of it the launch; its bytes alone take 2.9.
constexpr int kFewWaves = 8;

__host__ __device__ constexpr int few_pitch(int K) { return (K + 255) / 256 * 256 + 16; }   // LDS bytes of a token
// codes, then scales [ceil(K / 128), M]
__host__ __device__ constexpr int few_lds(int M, int K) { return M * (few_pitch(K) + 4 * ((K + 127) / 128)); }

template <int MT, int LEAD, bool QUANT, bool SMOOTH>
__global__ __launch_bounds__(64 * kFewWaves) void gemm_fp8_few_kernel(Fp8GemmArgs a, const uint16_t* __restrict__ x,
                                                                     const uint16_t* __restrict__ smooth) {
  __shared__ f32x4 part[kFewWaves][MT][64];
  extern __shared__ __attribute__((aligned(16))) uint8_t tok[];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int q = lane >> 4, l16 = lane & 15;
  const int M = (int)a.M, N = (int)a.N, K = (int)a.K;
  const int KB = (K + 127) / 128;
  const int n0 = (int)blockIdx.x * 16;
  // a lane's operand: pieces q and q + 4 of the row's eight 16-byte pieces; K % 16 == 0, so a piece is
  // entirely before or past K, and zero past it
  auto codes_at = [&](const uint8_t* row, int p) {
    const i32x4 zero = {};
    const int k = 128 * p + 16 * q;
    return join8(k < K ? *reinterpret_cast<const i32x4*>(row + 128 * p) : zero,
                 k + 64 < K ? *reinterpret_cast<const i32x4*>(row + 128 * p + 64) : zero);
  };
  const uint8_t* pw = a.weight + (size_t)min(n0 + l16, N - 1) * K + 16 * q;
  const float* ws_at = a.wscales + (size_t)(n0 / 128) * KB;
  constexpr int kStep = kFewWaves * LEAD;
  i32x8 fw[LEAD];
  float ws[LEAD];
  auto request = [&](int u, int p) {
    if (p < KB) {
      fw[u] = codes_at(pw, p);
      ws[u] = ws_at[p];
    }
  };
#pragma unroll
  for (int u = 0; u < LEAD; ++u) request(u, wave + kFewWaves * u);

  const uint8_t* pt[MT];
  const float* as_at = a.ascales;
  if constexpr (QUANT) {
    // 16 lanes a block, 8 channels each; zeros up to the end of a row's last block
    const int pitch = few_pitch(K), items = M * KB;
    float* scales = reinterpret_cast<float*>(tok + M * pitch);
    constexpr int kGroups = 4 * kFewWaves, U = 4;   // U blocks of a thread with their loads in flight together
    for (int g0 = 4 * wave; g0 < items; g0 += U * kGroups) {   // the wave's four
      u32x4 xw[U], sw[U];
      int at[U], to[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (g0 + u * kGroups >= items) break;
        const int g = min(g0 + u * kGroups + q, items - 1);   // (past the end: the last one again)
        const int m = M == 1 ? 0 : g / KB, p = g - m * KB, k = 128 * p + 8 * (tid & 15);
        to[u] = m * pitch + k;
        at[u] = p * M + m;
        xw[u] = k < K ? *reinterpret_cast<const u32x4*>(x + (size_t)m * K + k) : zero4();
        sw[u] = SMOOTH && k < K ? *reinterpret_cast<const u32x4*>(smooth + k) : zero4();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (g0 + u * kGroups >= items) break;
        float v[8], amax = 0.0f;
        f8_scaled8<SMOOTH>(xw[u], sw[u], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = max_or_nan(amax, fabsf(v[e]));
        const Fp8Scale s = fp8_scale(max_row16(amax));
        *reinterpret_cast<u32x2*>(tok + to[u]) = fp8_codes8(v, s.inv);
        if ((tid & 15) == 0) scales[at[u]] = s.scale;
      }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) pt[t] = tok + min(16 * t + l16, M - 1) * pitch + 16 * q;
    as_at = scales;
    __syncthreads();
  } else {
#pragma unroll
    for (int t = 0; t < MT; ++t) pt[t] = a.codes + (size_t)min(16 * t + l16, M - 1) * K + 16 * q;
  }
  f32x4 acc[MT] = {};
  for (int p = wave; p < KB; p += kStep) {
    i32x8 ft[LEAD][MT];
    float as[LEAD][MT];
#pragma unroll
    for (int u = 0; u < LEAD; ++u) {
      const int pu = p + kFewWaves * u;
      if (pu < KB) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          ft[u][t] = QUANT ? join8(*reinterpret_cast<const i32x4*>(pt[t] + 128 * pu),
                                   *reinterpret_cast<const i32x4*>(pt[t] + 128 * pu + 64))
                           : codes_at(pt[t], pu);
          as[u][t] = as_at[(size_t)pu * M + min(16 * t + l16, M - 1)];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < LEAD; ++u) {
      const int pu = p + kFewWaves * u;
      if (pu < KB) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const f32x4 sum = f8_mfma16(fw[u], ft[u][t], f32x4{});
          const float s = as[u][t] * ws[u];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[t][r] = __builtin_fmaf(sum[r], s, acc[t][r]);
        }
        request(u, pu + kStep);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  // wave t ends token group t: lane l holds token l % 16, channels 4 (l / 16) .. + 3
  if (wave < MT) {
    f32x4 s = part[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += part[w][wave][lane];
    const int m = 16 * wave + l16;
    if (m < M) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = n0 + 4 * q + r;
        if (n < N) {
          const float b = a.bias != nullptr ? bf16lo_to_f32(a.bias[n]) : 0.0f;
          a.y[(size_t)m * (size_t)N + n] = (uint16_t)f32_to_bf16_rne(s[r] + b);
        }
      }
    }
  }
}

template <int MT, int LEAD>
hipError_t launch_few_cfg(const Fp8GemmArgs& a, const uint16_t* x, const uint16_t* smooth, hipStream_t stream) {
  const dim3 grid((unsigned)((a.N + 15) / 16)), block(64 * kFewWaves);
  if (x == nullptr)
    hipLaunchKernelGGL((gemm_fp8_few_kernel<MT, LEAD, false, false>), grid, block, 0, stream, a, x, smooth);
  if constexpr (MT == 1) {   // few_from_x: at most 16 tokens
    const unsigned lds = (unsigned)few_lds((int)a.M, (int)a.K);
    if (x != nullptr && smooth == nullptr)
      hipLaunchKernelGGL((gemm_fp8_few_kernel<MT, LEAD, true, false>), grid, block, lds, stream, a, x, smooth);
    else if (x != nullptr)
      hipLaunchKernelGGL((gemm_fp8_few_kernel<MT, LEAD, true, true>), grid, block, lds, stream, a, x, smooth);
  }
  return hipGetLastError();
}

hipError_t launch_few(const Fp8GemmArgs& a, const uint16_t* x, const uint16_t* smooth, hipStream_t stream) {
  return a.M <= 16   ? launch_few_cfg<1, 4>(a, x, smooth, stream)
         : a.M <= 32 ? launch_few_cfg<2, 2>(a, x, smooth, stream)
         : a.M <= 48 ? launch_few_cfg<3, 2>(a, x, smooth, stream)
                     : launch_few_cfg<4, 2>(a, x, smooth, stream);
}

// Every workgroup reads all the tokens' codes, and one of 16 channels works through all of k: above 8 tokens
// only while both are few (with the quantisation, here and in tiles: 32 x 3840 for 3840 channels 12.4 and 13.7 us, 64 x
// 3840 16.5 and 15.1, 64 x 2064 for 1300 8.3 and 11.2, 16 x 10240 for 3840 18.1 and 19.4, 16 x 3840 for 10240 18.7
// and 18.3). With up to 8 the tiles gain nothing (8 x 3840 for 10240: 16.3 and 17.9).
bool few_tokens(int64_t M, int64_t N, int64_t K) {
  return M <= 8 || (M <= 64 && M * K <= 163840 && N * K <= (int64_t(1) << 24));
}

// The layer from x in one launch: every workgroup makes the tokens' codes again, so only while they are few.
// Against two launches (on the device): 6.0 and 8.2 us for 1 x 3840 (3840 channels), 12.5 and 14.1 for 1 x 10240, 8.6 and 9.5
// for 8 x 3840, 16.3 and 16.0 for 4 x 10240; another 3 us of the caller's time where the calls are not in a graph.
bool few_from_x(int64_t M, int64_t N, int64_t K) {
  // codes, scales and sums together stay inside 64 KB of LDS
  return M <= 16 && few_tokens(M, N, K) && M * K <= 32768 && few_lds((int)M, (int)K) <= 56 * 1024;
}

struct F8Plan {
  int shape;     // index into the table
  int splits, panels;
};

// Tile shape and split of k by an estimate in microseconds, fitted to times with weights from memory (M from 20 to
// 6000; eight weights from 1300 x 2064 to 10240 x 3840 and 3840 x 10240; every shape with k split 1 to 8
// ways: profiles/gemm_fp8_tile_grid.txt). A panel takes a workgroup at least `least`, and each of the
// ceil(workgroups / 256) rounds `share` + `full` times the share of the CUs that work (the more do, the slower
// each: power and the L2s); 4.2 us start and end a product; a split adds 0.9 us and the partial sums' traffic.
// As for the 8-bit integers, a call that is not in a graph takes its caller about 10 us and 3 more for a split's
// launch, so a split pays only where the device takes longer than that. The caller is taken to be eager: a call captured
// in a graph chooses alike. Where the best takes the device 13 us or more, the choice is within 0.2% of it on average and 6%
// at worst; with the sizes below it is 1.0% and 27% (100 tokens, 1300 channels, K = 2064: 11.2 us unsplit, 8.8 split), which
// an eager caller does not see and a graph does. The estimate without `full` was 4% off on average. Tiles of 192 x 128 take
// 8 to 14% off where rows fill them and 128's or 256's leave CUs idle (333 x 3840, K = 10240: 36 -> 33; 1500 x 3840, K = 3840:
// 37 -> 32.5).
F8Plan plan_fp8(int64_t M, int64_t N, int64_t K) {
  static const struct { int bm, bn; double least, share, full; } shapes[] = {
      {256, 320, 1.56, 1.33, 0.64}, {256, 256, 1.45, 1.30, 0.49}, {256, 128, 0.86, 0.90, 0.31},
      {128, 128, 0.46, 0.49, 0.27}, {64, 128, 0.33, 0.41, 0.10},  {64, 64, 0.35, 0.29, 0.0},
      {192, 128, 1.03, 0.97, 0.0}};
  const int64_t panels = (K + 127) / 128;
  F8Plan best{0, 1, (int)panels};
  double best_t = 1e300;
  for (int s = 0; s < 7; ++s) {
    const int64_t tiles = ((M + shapes[s].bm - 1) / shapes[s].bm) * ((N + shapes[s].bn - 1) / shapes[s].bn);
    for (int sp = 1; sp <= 8; ++sp) {
      if (sp > 1 && (panels < 2 * sp || tiles * sp > 1024)) break;
      const int64_t per = (panels + sp - 1) / sp, rounds = (tiles * sp + 255) / 256;
      const double fill = (double)(tiles * sp) / (256.0 * (double)rounds);
      const double device = 4.2 + (double)per * fmax(shapes[s].least, (double)rounds * (shapes[s].share + shapes[s].full * fill)) +
                            (sp > 1 ? 0.9 + 2.0e-6 * (double)(M * N) * sp : 0.0);
      const double t = fmax(device, sp > 1 ? 13.0 : 10.0) + 0.01 * device;
      if (t < best_t) {
        best_t = t;
        best = F8Plan{s, (int)((panels + per - 1) / per), (int)per};
      }
    }
  }
  return best;
}

template <int WM, int WN, int TM, int TN, int S>
hipError_t launch_fp8_cfg(const Fp8GemmArgs& a, const F8Split& sp, hipStream_t stream) {
  using C = F8Cfg<WM, WN, TM, TN, S>;
  static std::atomic<uint64_t> lds_set{0};
  const void* fn = reinterpret_cast<const void*>(&gemm_fp8_kernel<WM, WN, TM, TN, S>);
  hipError_t e = set_lds_limit_once(fn, C::kLdsBytes, lds_set);
  if (e != hipSuccess) return e;
  const int64_t tiles = ((a.N + C::BN - 1) / C::BN) * ((a.M + C::BM - 1) / C::BM) * sp.splits;
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8));
  hipLaunchKernelGGL((gemm_fp8_kernel<WM, WN, TM, TN, S>), grid, dim3(64 * C::kWaves), C::kLdsBytes, stream, a, sp);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_fp8(const uint16_t* x, const uint16_t* smooth, int64_t M, int64_t K, uint8_t* codes,
                            float* ascales, hipStream_t stream) {
  constexpr int U = 2;
  const dim3 grid((unsigned)((M + 16 * U - 1) / (16 * U) * ((K + 127) / 128)));
  if (smooth != nullptr)
    hipLaunchKernelGGL((quant_fp8_kernel<true, U>), grid, dim3(256), 0, stream, x, smooth, (uint32_t)M, (uint32_t)K, codes, ascales);
  else
    hipLaunchKernelGGL((quant_fp8_kernel<false, U>), grid, dim3(256), 0, stream, x, smooth, (uint32_t)M, (uint32_t)K, codes, ascales);
  return hipGetLastError();
}

hipError_t launch_quant_weight_fp8(const uint16_t* w, const uint16_t* smooth, int64_t N, int64_t K, uint8_t* codes,
                                   float* wscales, hipStream_t stream) {
  const dim3 grid((unsigned)((K + 127) / 128), (unsigned)((N + 127) / 128));
  if (smooth != nullptr)
    hipLaunchKernelGGL(quant_weight_fp8_kernel<true>, grid, dim3(256), 0, stream, w, smooth, (int)N, (int)K, codes, wscales);
  else
    hipLaunchKernelGGL(quant_weight_fp8_kernel<false>, grid, dim3(256), 0, stream, w, smooth, (int)N, (int)K, codes, wscales);
  return hipGetLastError();
}

size_t gemm_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (few_tokens(M, N, K)) return 0;
  const F8Plan p = plan_fp8(M, N, K);
  return p.splits > 1 ? (size_t)p.splits * (size_t)M * (size_t)N * 4 : 0;
}

void gemm_fp8_plan(int64_t M, int64_t N, int64_t K, int* tile, int* splits) {
  const bool few = few_tokens(M, N, K);
  const F8Plan p = few ? F8Plan{-1, 1, 0} : plan_fp8(M, N, K);
  *tile = p.shape;
  *splits = p.splits;
}

hipError_t launch_gemm_fp8(const Fp8GemmArgs& a, void* workspace, hipStream_t stream) {
  if (few_tokens(a.M, a.N, a.K)) return launch_few(a, nullptr, nullptr, stream);
  const F8Plan p = plan_fp8(a.M, a.N, a.K);
  const F8Split sp{p.panels, p.splits, static_cast<float*>(workspace)};
  hipError_t e = p.shape == 0   ? launch_fp8_cfg<4, 2, 2, 5, 2>(a, sp, stream)
                 : p.shape == 1 ? launch_fp8_cfg<4, 2, 2, 4, 2>(a, sp, stream)
                 : p.shape == 2 ? launch_fp8_cfg<4, 2, 2, 2, 3>(a, sp, stream)
                 : p.shape == 3 ? launch_fp8_cfg<4, 2, 1, 2, 4>(a, sp, stream)
                 : p.shape == 4 ? launch_fp8_cfg<2, 4, 1, 1, 3>(a, sp, stream)
                 : p.shape == 5 ? launch_fp8_cfg<2, 2, 1, 1, 3>(a, sp, stream)
                                : launch_fp8_cfg<2, 4, 3, 1, 3>(a, sp, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  const int w = a.N % 4 == 0 ? 4 : 1;
  const dim3 grid((unsigned)((a.M * (a.N / w) + 255) / 256));
  if (w == 4) hipLaunchKernelGGL(fp8_reduce_kernel<4>, grid, dim3(256), 0, stream, a, sp.partial, p.splits);
  else hipLaunchKernelGGL(fp8_reduce_kernel<1>, grid, dim3(256), 0, stream, a, sp.partial, p.splits);
  return hipGetLastError();
}

size_t linear_fp8_codes_bytes(int64_t M, int64_t N, int64_t K) {
  return few_from_x(M, N, K) ? 0 : (size_t)M * (size_t)K;
}

hipError_t launch_linear_fp8(const Fp8GemmArgs& a, const uint16_t* x, const uint16_t* smooth, uint8_t* codes,
                             float* ascales, void* workspace, hipStream_t stream) {
  if (few_from_x(a.M, a.N, a.K)) return launch_few(a, x, smooth, stream);
  hipError_t e = launch_quant_fp8(x, smooth, a.M, a.K, codes, ascales, stream);
  if (e != hipSuccess) return e;
  Fp8GemmArgs g = a;
  g.codes = codes;
  g.ascales = ascales;
  return launch_gemm_fp8(g, workspace, stream);
}

}  // namespace svdq
