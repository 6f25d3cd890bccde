// Attention over whole packed sequences, full or causal, with grouped heads:
//
//   o[t, h] = sum_j p_j v[j] / sum_j p_j,  p_j = exp(scale * (q[t, h] . k[j] - m)),
//
// j over the tokens of t's sequence (causal: j <= t), in one pass over the keys
// with a running maximum m and sum.
//
// Scores are computed transposed, S^T = K Q^T on v_mfma_f32_32x32x16_bf16, so that
// a lane holds scores of one query (column l % 32) and the maximum, the sum and
// the rescaling are per lane. The accumulator layout of S^T (rows 8 (r / 4) + 4 (l / 32) +
// r % 4) is also the operand layout of P^T in O^T = V^T P^T when the 16 keys of a
// step are taken in the order 4 h + {0..3}, 8 + 4 h + {0..3} for half h, so P goes from one
// product to the next without leaving its lane; V is read in the same order by
// the transposing LDS read (four keys of one column per lane).
#include "common.h"
#include "kernels.h"

#define ATT_LDS(t, p) ((__attribute__((address_space(3))) t*)(p))

namespace svdq {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kWavesA = 8;          // waves of a workgroup, 32 queries each
constexpr int kBM = 32 * kWavesA;   // queries of a workgroup
constexpr int kBN = 64;             // keys of a tile

// copies into LDS stay outside template-dependent code (see gemm_mx.hip)
__device__ __forceinline__ void att_to_lds(__amdgpu_buffer_rsrc_t r, void* lds, int voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, ATT_LDS(void, lds), 16, voff, 0, 0, 0);
}
__device__ __forceinline__ s16x4 att_read_tr(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(ATT_LDS(s16x4, p));
}

// Tiles are numbered so that sequence b starts at floor(cu[b] / kBM) + b, which needs
// no prefix sum and leaves at most one unused number per sequence. Returns the
// sequence of tile `t` (-1: none); the wave's lanes probe 64 offsets at a time.
__device__ __forceinline__ int tile_sequence(const int32_t* cu, int B, int64_t T, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = B;
  while (true) {
    const int step = (hi - lo + 63) / 64;
    const int idx = lo + lane * step;
    bool below = false;
    if (idx < hi) {
      const int64_t c = min(max((int64_t)cu[idx], (int64_t)0), T);
      below = (int)(c / kBM) + idx <= t;
    }
    const int n = __popcll(__ballot(below));
    if (n == 0) return -1;
    lo = lo + (n - 1) * step;
    if (step == 1) return lo;
    hi = min(hi, lo + step);
  }
}

template <int D, bool CAUSAL>
__global__ __launch_bounds__(64 * kWavesA) void attention_kernel(AttnArgs a) {
  constexpr int kRowBytes = 2 * D;
  constexpr int kTileBytes = kBN * kRowBytes;
  constexpr int kPieces = D / 8;                    // 16-byte pieces of a row
  constexpr int kRowsPerCopy = 64 / kPieces;
  constexpr int kCopies = kTileBytes / 1024 / kWavesA;
  constexpr int KD = D / 16;                        // 16-element steps of the first product
  constexpr int JD = D / 32;                        // 32-column blocks of the output
  __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * kTileBytes];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int h = lane >> 5, l32 = lane & 31;

  // heads of one group and the tiles of one head stay on one XCD (its L2 holds their keys)
  const int tiles = (int)(a.T / kBM) + a.B;
  const int per_xcd = (int)(gridDim.x / 8);
  const int id = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
  if (id >= tiles * a.H) return;
  const int head = id / tiles;
  const int tile = id % tiles;
  int b = 0;
  int64_t beg = 0, end = a.T;
  if (a.cu != nullptr) {
    b = tile_sequence(a.cu, a.B, a.T, tile);
    if (b < 0) return;
    beg = min(max((int64_t)a.cu[b], (int64_t)0), a.T);
    end = min(max((int64_t)a.cu[b + 1], (int64_t)0), a.T);
  }
  const int len = (int)(end - beg);
  const int q0 = (tile - (int)(beg / kBM) - b) * kBM;   // first query of the tile in its sequence
  if (q0 >= len) return;
  const int hk = head / (a.H / a.Hk);
  const int q = q0 + 32 * wave + l32;                    // this lane's query
  const bool wave_live = q0 + 32 * wave < len;

  // Q^T operand: this lane's query, elements 16 t + 8 h .. + 7
  bf16x8 fq[KD];
  {
    const uint16_t* qp = a.q.p + (beg + min(q, len - 1)) * a.q.st + head * a.q.sh + 8 * h;
#pragma unroll
    for (int t = 0; t < KD; ++t) fq[t] = *reinterpret_cast<const bf16x8*>(qp + 16 * t);
  }

  const int last_q = min(q0 + kBM, len) - 1;
  const int nt = (CAUSAL ? last_q : len - 1) / kBN + 1;

  // Tile copies: row r of K (V) at r * kRowBytes, its 16-byte pieces permuted by
  // piece ^ swz(r) so that the operand reads hit distinct banks: 16 rows at one
  // piece for K, 4 rows x 4 pieces for V.
  auto swz_k = [](int r) { return D == 128 ? (r & 15) : ((r >> 1) & 7); };
  auto swz_v = [](int r) { return D == 128 ? ((r & 3) << 2) : (((r >> 1) & 1) << 2); };
  const uint16_t* kp = a.k.p + beg * a.k.st + hk * a.k.sh;
  const uint16_t* vp = a.v.p + beg * a.v.st + hk * a.v.sh;
  int koff[kCopies], voff[kCopies];
#pragma unroll
  for (int c = 0; c < kCopies; ++c) {
    const int r = (wave + kWavesA * c) * kRowsPerCopy + lane / kPieces;
    const int slot = lane % kPieces;
    koff[c] = r * (int)a.k.st * 2 + (slot ^ swz_k(r)) * 16;
    voff[c] = r * (int)a.v.st * 2 + (slot ^ swz_v(r)) * 16;
  }
  auto load_tile = [&](int kt) {
    const int row0 = kt * kBN;
    const int rows = min(kBN, len - row0);   // rows past the sequence read as zero
    const __amdgpu_buffer_rsrc_t rk = make_rsrc(kp + row0 * a.k.st, (uint32_t)(((rows - 1) * (int)a.k.st + D) * 2));
    const __amdgpu_buffer_rsrc_t rv = make_rsrc(vp + row0 * a.v.st, (uint32_t)(((rows - 1) * (int)a.v.st + D) * 2));
    uint8_t* st = smem + (kt & 1) * (2 * kTileBytes);
#pragma unroll
    for (int c = 0; c < kCopies; ++c) att_to_lds(rk, st + (wave + kWavesA * c) * 1024, koff[c]);
#pragma unroll
    for (int c = 0; c < kCopies; ++c) att_to_lds(rv, st + kTileBytes + (wave + kWavesA * c) * 1024, voff[c]);
  };

  // operand addresses within a tile
  int kfrag[KD];
#pragma unroll
  for (int t = 0; t < KD; ++t) kfrag[t] = l32 * kRowBytes + (((2 * t + h) ^ swz_k(l32)) * 16);
  const int vrow = 4 * h + ((lane & 15) >> 2);           // + 16 t (+ 8): multiples of 8 leave swz_v alone
  int vfrag[JD];
#pragma unroll
  for (int j = 0; j < JD; ++j) {
    const int piece = 4 * j + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    vfrag[j] = vrow * kRowBytes + ((piece ^ swz_v(vrow)) * 16) + 8 * (lane & 1);
  }

  f32x16 acc[JD];
#pragma unroll
  for (int j = 0; j < JD; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[j][r] = 0.0f;
  float m = -1e30f, l = 0.0f;
  const float c = a.scale * 1.4426950408889634f;   // exponents in base 2

  load_tile(0);
  for (int kt = 0; kt < nt; ++kt) {
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): this wave's copies have landed
    __syncthreads();
    if (kt + 1 < nt) load_tile(kt + 1);
    if (!wave_live || (CAUSAL && kt * kBN > q0 + 32 * wave + 31)) continue;
    const uint8_t* sk = smem + (kt & 1) * (2 * kTileBytes);
    const uint8_t* sv = sk + kTileBytes;

    f32x16 s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[i][r] = 0.0f;
#pragma unroll
      for (int t = 0; t < KD; ++t) {
        const bf16x8 fk = *reinterpret_cast<const bf16x8*>(sk + 32 * i * kRowBytes + kfrag[t]);
        s[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fk, fq[t], s[i], 0, 0, 0);
      }
    }
    // keys past the sequence, or past the query
    const int key0 = kt * kBN + 4 * h;
    if (kt * kBN + kBN > len || (CAUSAL && kt * kBN + kBN - 1 > q0 + 32 * wave)) {
      const int lim = CAUSAL ? min(q, len - 1) : len - 1;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (key0 + 32 * i + 8 * (r >> 2) + (r & 3) > lim) s[i][r] = -__builtin_inff();
    }
    float mx = s[0][0];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[i][r]);
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mn = fmaxf(m, mx);
    const float alpha = __builtin_amdgcn_exp2f((m - mn) * c);
    m = mn;
    l *= alpha;
#pragma unroll
    for (int j = 0; j < JD; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][r] *= alpha;
    const float mc = m * c;
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][2 * r], c, -mc));
        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][2 * r + 1], c, -mc));
        p[8 * i + r] = pack_bf16x2(p0, p1);
        l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, p[8 * i + r]), bf16x2_t{(__bf16)1.0f, (__bf16)1.0f},
                                            l, false);
      }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const u32x4 pw = {p[4 * t], p[4 * t + 1], p[4 * t + 2], p[4 * t + 3]};
      const bf16x8 fp = __builtin_bit_cast(bf16x8, pw);
#pragma unroll
      for (int j = 0; j < JD; ++j) {
        const s16x4 v0 = att_read_tr(sv + 16 * t * kRowBytes + vfrag[j]);
        const s16x4 v1 = att_read_tr(sv + (16 * t + 8) * kRowBytes + vfrag[j]);
        const s16x8 v = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
        acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, v), fp, acc[j], 0, 0, 0);
      }
    }
  }

  l += __shfl_xor(l, 32);
  if (q >= len) return;
  const float inv = 1.0f / l;
  uint16_t* op = a.o + (beg + q) * a.o_st + head * a.o_sh;
#pragma unroll
  for (int j = 0; j < JD; ++j)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *reinterpret_cast<u32x2*>(op + 32 * j + 2 * r + 4 * h) =
          u32x2{pack_bf16x2(acc[j][r] * inv, acc[j][r + 1] * inv), pack_bf16x2(acc[j][r + 2] * inv, acc[j][r + 3] * inv)};
}

template <int D>
void launch_attention_d(const AttnArgs& a, hipStream_t s) {
  const int64_t total = (a.T / kBM + a.B) * a.H;
  const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(64 * kWavesA);
  if (a.causal) hipLaunchKernelGGL((attention_kernel<D, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((attention_kernel<D, false>), grid, block, 0, s, a);
}

}  // namespace

hipError_t launch_attention(const AttnArgs& a, int D, hipStream_t stream) {
  if (D == 64) launch_attention_d<64>(a, stream);
  else launch_attention_d<128>(a, stream);
  return hipGetLastError();
}

}  // namespace svdq
