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
constexpr int kAhead = 3;           // operand reads in flight ahead of a product
constexpr float kSlack = 8.0f;      // powers of two that a score may pass the running maximum by

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

__device__ __forceinline__ void att_barrier() {   // as in gemm_bf16.hip: the waits are explicit
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
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
  int local = tile - (int)(beg / kBM) - b;               // tile within the sequence
  if (local * kBM >= len) return;
  if (CAUSAL) local = (len - 1) / kBM - local;           // those with the most keys first
  const int q0 = local * kBM;
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
  // K in two stages, then V in two
  auto load_k = [&](int kt) {
    const int row0 = kt * kBN;
    const int rows = min(kBN, len - row0);   // rows past the sequence read as zero
    const __amdgpu_buffer_rsrc_t r = make_rsrc(kp + row0 * a.k.st, (uint32_t)(((rows - 1) * (int)a.k.st + D) * 2));
    uint8_t* st = smem + (kt & 1) * kTileBytes;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) att_to_lds(r, st + (wave + kWavesA * c) * 1024, koff[c]);
  };
  auto load_v = [&](int kt) {
    const int row0 = kt * kBN;
    const int rows = min(kBN, len - row0);
    const __amdgpu_buffer_rsrc_t r = make_rsrc(vp + row0 * a.v.st, (uint32_t)(((rows - 1) * (int)a.v.st + D) * 2));
    uint8_t* st = smem + (2 + (kt & 1)) * kTileBytes;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) att_to_lds(r, st + (wave + kWavesA * c) * 1024, voff[c]);
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
  float m = -1e30f, l = 0.0f, mc = 0.0f;
  const float c = a.scale * 1.4426950408889634f;   // exponents in base 2
  const float slack = kSlack / c;

  // Operand u of the first product (rows 32 (u % 2) of the tile, elements 16 (u / 2) of the
  // head), and of the second (keys 16 (u / JD), columns 32 (u % JD))
  auto read_k = [&](const uint8_t* sk, int u) {
    return *reinterpret_cast<const bf16x8*>(sk + 32 * (u & 1) * kRowBytes + kfrag[u >> 1]);
  };
  auto read_v = [&](const uint8_t* sv, int u) {
    const uint8_t* p = sv + 16 * (u / JD) * kRowBytes + vfrag[u % JD];
    const s16x4 v0 = att_read_tr(p), v1 = att_read_tr(p + 8 * kRowBytes);
    return __builtin_bit_cast(bf16x8, (s16x8)__builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  constexpr int NK = 2 * KD, NV = 4 * JD;   // products of a tile
  const bf16x2_t ones = {(__bf16)1.0f, (__bf16)1.0f};
  // probabilities of score pair r (0..15) of a tile
  auto pair = [&](const f32x16 (&s)[2], uint32_t (&p)[16], int r) {
    const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r >> 3][2 * (r & 7)], c, -mc));
    const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r >> 3][2 * (r & 7) + 1], c, -mc));
    p[r] = pack_bf16x2(p0, p1);
    l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, p[r]), ones, l, false);
  };
  auto prob_operand = [&](const uint32_t (&p)[16], int t) {
    return __builtin_bit_cast(bf16x8, u32x4{p[4 * t], p[4 * t + 1], p[4 * t + 2], p[4 * t + 3]});
  };
  auto zero_scores = [&](f32x16 (&s)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[i][r] = 0.0f;
  };
  // keys past the sequence, or past the query
  auto mask = [&](f32x16 (&s)[2], int kt) {
    if (kt * kBN + kBN > len || (CAUSAL && kt * kBN + kBN - 1 > q0 + 32 * wave)) {
      const int lim = (CAUSAL ? min(q, len - 1) : len - 1) - kt * kBN - 4 * h;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * i + 8 * (r >> 2) + (r & 3) > lim) s[i][r] = -__builtin_inff();
    }
  };
  // the running maximum moves only when a score passes it by more than kSlack powers of
  // two: until then the probabilities are at most 2^kSlack, with the same relative rounding
  auto rescale = [&](float mx) {
    if (__ballot(mx > m + slack) == 0) return;
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mn = fmaxf(m, mx);
    const float alpha = __builtin_amdgcn_exp2f((m - mn) * c);
    m = mn;
    mc = m * c;
    l *= alpha;
#pragma unroll
    for (int j = 0; j < JD; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][r] *= alpha;
  };
  // Start of step kt: one barrier frees K(kt) and V(kt - 1) for the copies of K(kt + 2) and
  // V(kt + 1), and publishes K(kt + 1) and V(kt), which were requested a step ago.
  auto next_tiles = [&](int kt) {
    __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0): this wave's copies have landed; lgkmcnt(0)
    att_barrier();
    if (kt + 2 < nt) load_k(kt + 2);
    if (kt + 1 < nt) load_v(kt + 1);
  };
  // A step: the next tile's scores on the matrix unit while this tile's probabilities are
  // made, then the product with V while the maximum of the next scores is found. Each
  // product is issued with its share of the other work and the operand reads of kAhead
  // products later.
  auto step = [&](f32x16 (&cur)[2], f32x16 (&nxt)[2], int kt) {
    next_tiles(kt);
    const uint8_t* sk = smem + ((kt + 1) & 1) * kTileBytes;
    const uint8_t* sv = smem + (2 + (kt & 1)) * kTileBytes;
    uint32_t p[16];
    bf16x8 fk[NK], fv[NV];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fk[u] = read_k(sk, u);
    zero_scores(nxt);
#pragma unroll
    for (int u = 0; u < NK; ++u) {
      if (u + kAhead < NK) fk[u + kAhead] = read_k(sk, u + kAhead);
      else fv[u + kAhead - NK] = read_v(sv, u + kAhead - NK);
      nxt[u & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fk[u], fq[u >> 1], nxt[u & 1], 0, 0, 0);
#pragma unroll
      for (int r = 16 / NK * u; r < 16 / NK * (u + 1); ++r) {
        pair(cur, p, r);
        asm volatile("" : "+v"(p[r]));   // made here: not moved down to its use
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    mask(nxt, kt + 1);
    float mx = -__builtin_inff();
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      if (u + kAhead < NV) fv[u + kAhead] = read_v(sv, u + kAhead);
      acc[u % JD] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fv[u], prob_operand(p, u / JD), acc[u % JD], 0, 0, 0);
#pragma unroll
      for (int r = 32 / NV * u; r < 32 / NV * (u + 1); ++r) mx = fmaxf(mx, nxt[r >> 4][r & 15]);
      __builtin_amdgcn_sched_barrier(0);
    }
    rescale(mx);
  };

  // tiles this wave needs; the others it only helps to load
  const int ntw = !wave_live ? 0 : CAUSAL ? min(nt, (q0 + 32 * wave + 31) / kBN + 1) : nt;
  load_k(0);
  __builtin_amdgcn_s_waitcnt(0x0F70);
  att_barrier();
  load_v(0);
  if (nt > 1) load_k(1);
  int kt = 0;
  if (ntw > 0) {
    f32x16 s0[2], s1[2];
    zero_scores(s0);
#pragma unroll
    for (int u = 0; u < NK; ++u)
      s0[u & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_k(smem, u), fq[u >> 1], s0[u & 1], 0, 0, 0);
    mask(s0, 0);
    float mx = s0[0][0];
#pragma unroll
    for (int r = 1; r < 32; ++r) mx = fmaxf(mx, s0[r >> 4][r & 15]);
    rescale(mx);
    for (; kt + 2 < ntw; kt += 2) {
      step(s0, s1, kt);
      step(s1, s0, kt + 1);
    }
    if (kt + 1 < ntw) {
      step(s0, s1, kt);
      s0[0] = s1[0];
      s0[1] = s1[1];
      ++kt;
    }
    next_tiles(kt);   // the last tile
    const uint8_t* sv = smem + (2 + (kt & 1)) * kTileBytes;
    ++kt;
    uint32_t p[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) pair(s0, p, r);
#pragma unroll
    for (int u = 0; u < NV; ++u)
      acc[u % JD] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_v(sv, u), prob_operand(p, u / JD), acc[u % JD], 0, 0, 0);
  }
  for (; kt < nt; ++kt) next_tiles(kt);

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
