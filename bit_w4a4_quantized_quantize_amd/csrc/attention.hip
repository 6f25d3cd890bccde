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
//
// Bound: the matrix units' power. 30 heads of 128: 16896 tokens 3600-3950 us (1.11-1.22 PFLOP/s at
// 1.65-1.74 GHz; a large library bf16 product reaches 1.33), 4096 tokens 230-255 us (1.0-1.1, 1.9
// rounds of workgroups); 13 causal prompts of 315 tokens on average, 32 heads on 8, 31-37 us (their
// starts and ends); 1024 tokens, 29-30 us (240 workgroups, a wave a SIMD, 16 tiles each one after the
// other). 30 heads of 64, 16896 tokens: 2240 us (0.98: as many exponentials for half the products).
// K and V tiles of 64 keys, double buffered by direct copies to LDS: tiles through
// registers measured equal or 8% slower, 32 keys 18% slower at 4096 tokens. Up to 39 scalars (constants
// of the loop) are spilled into lanes of a vector register; 4 to 13 are read back per two tiles, of about
// 1000 instructions, while the next tiles are requested. No vector register spills.
#include "common.h"
#include "kernels.h"

#define ATT_LDS(t, p) ((__attribute__((address_space(3))) t*)(p))

namespace svdq {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kBN = 64;             // keys of a tile
constexpr int kAhead = 2;           // operand reads in flight ahead of a product
constexpr float kSlack = 8.0f;      // powers of two that a score may pass the running maximum by

// copies into LDS stay outside template-dependent code (see gemm_mx.hip)
__device__ __forceinline__ void att_to_lds(__amdgpu_buffer_rsrc_t r, void* lds, int voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, ATT_LDS(void, lds), 16, voff, 0, 0, 0);
}
__device__ __forceinline__ s16x4 att_read_tr(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(ATT_LDS(s16x4, p));
}
__device__ __forceinline__ void att_barrier() {   // as in gemm_bf16.hip: the waits are explicit
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
template <int N>
__device__ __forceinline__ void att_wait_copies() {   // vmcnt(N)
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0F70);
}

// Tiles of 2^lg queries are numbered so that sequence b starts at floor(cu[b] / 2^lg) + b, which needs
// no prefix sum and leaves at most one unused number per sequence. Finds the sequence of
// tile t and its bounds (clamped to 0..T); false where there is none. The wave's lanes probe
// 64 offsets at a time, so up to 64 sequences cost one load.
__device__ __forceinline__ bool tile_sequence(const int32_t* cu, int B, int64_t T, int lg, int t, int& b, int& beg,
                                              int& end) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = B;
  while (true) {
    const int step = (hi - lo + 63) / 64;
    const int idx = lo + lane * step;
    const int c0 = min(max(cu[min(idx, B)], 0), (int)T), c1 = min(max(cu[min(idx + 1, B)], 0), (int)T);
    const int n = __popcll(__ballot(idx < hi && (c0 >> lg) + idx <= t));
    if (n == 0) return false;
    if (step == 1) {
      b = lo + n - 1;
      beg = __builtin_amdgcn_readlane(c0, n - 1);
      end = __builtin_amdgcn_readlane(c1, n - 1);
      return true;
    }
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
}

// A workgroup of NW waves, each with 32 queries of one head. The waves are dealt to 2^lg_heads
// query heads of one group first (they share K and V, and short or causal sequences waste less
// in few rows of many heads), then to rows: 2^lg_rows queries per head.
template <int D, bool CAUSAL, int NW>
__global__ __launch_bounds__(64 * NW, 2) void attention_kernel(AttnArgs a, int lg_heads) {
  constexpr int kRowBytes = 2 * D;
  constexpr int kTileBytes = kBN * kRowBytes;
  constexpr int kPieces = D / 8;                    // 16-byte pieces of a row
  constexpr int kRowsPerCopy = 64 / kPieces;
  constexpr int kCopies = kTileBytes / 1024 / NW;
  constexpr int KD = D / 16;                        // 16-element steps of the first product
  constexpr int JD = D / 32;                        // 32-column blocks of the output
  constexpr int kLgWaves = NW == 8 ? 3 : 2;
  static_assert(NW == 1 << kLgWaves, "waves");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[4 * kTileBytes];

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lane = tid & 63;
  const int h = lane >> 5, l32 = lane & 31;

  // heads of one group and the tiles of one head stay on one XCD (its L2 holds their keys)
  const int lg_rows = 5 + kLgWaves - lg_heads;
  const int tiles = (int)(a.T >> lg_rows) + a.B;
  const int per_xcd = (int)(gridDim.x / 8);
  const int id = (int)(blockIdx.x % 8) * per_xcd + (int)(blockIdx.x / 8);
  if (id >= tiles * (a.H >> lg_heads)) return;
  const int head0 = (id / tiles) << lg_heads;
  const int tile = id % tiles;
  int b = 0, beg = 0, end = (int)a.T;
  if (a.cu != nullptr && !tile_sequence(a.cu, a.B, a.T, lg_rows, tile, b, beg, end)) return;
  const int len = end - beg;
  int local = tile - (beg >> lg_rows) - b;               // tile within the sequence (negative only where
  if (len <= 0 || local < 0 || local > (len - 1) >> lg_rows) return;   // the offsets decrease)
  if (CAUSAL) local = ((len - 1) >> lg_rows) - local;    // those with the most keys first
  const int q0 = local << lg_rows;
  const int hk = head0 / (a.H / a.Hk);

  // this wave's first row and head, and Q^T's operand (this lane's query, elements
  // 16 t + 8 h .. + 7)
  const int row0 = q0 + 32 * (wave >> lg_heads);
  const int head = head0 + (wave & ((1 << lg_heads) - 1));
  bf16x8 fq[KD];
  {
    const uint16_t* qp = a.q.p + (int64_t)(beg + min(row0 + l32, len - 1)) * a.q.st + head * a.q.sh + 8 * h;
#pragma unroll
    for (int t = 0; t < KD; ++t) fq[t] = *reinterpret_cast<const bf16x8*>(qp + 16 * t);
  }
  const int nt = (CAUSAL ? min(q0 + (1 << lg_rows), len) - 1 : len - 1) / kBN + 1;

  // Tile copies: row r of K (V) at r * kRowBytes, its 16-byte pieces permuted by
  // piece ^ swz(r) so that the operand reads hit distinct banks: 16 rows at one
  // piece for K, 4 rows x 4 pieces for V. Rows past the sequence read as zero.
  auto swz_k = [](int r) { return D == 128 ? (r & 15) : ((r >> 1) & 7); };
  auto swz_v = [](int r) { return D == 128 ? ((r & 3) << 2) : (((r >> 1) & 1) << 2); };
  const uint16_t* kp = a.k.p + (int64_t)beg * a.k.st + hk * a.k.sh;
  const uint16_t* vp = a.v.p + (int64_t)beg * a.v.st + hk * a.v.sh;
  const int kst = (int)a.k.st, vst = (int)a.v.st;
  int koff[kCopies], voff[kCopies];
#pragma unroll
  for (int c = 0; c < kCopies; ++c) {
    const int r = (wave + NW * c) * kRowsPerCopy + lane / kPieces;
    const int slot = lane % kPieces;
    koff[c] = r * kst * 2 + (slot ^ swz_k(r)) * 16;
    voff[c] = r * vst * 2 + (slot ^ swz_v(r)) * 16;
  }
  auto load_k = [&](int kt) {
    const int rows = min(kBN, len - kt * kBN);
    const __amdgpu_buffer_rsrc_t r = make_rsrc(kp + (int64_t)kt * kBN * kst, (uint32_t)(((rows - 1) * kst + D) * 2));
    uint8_t* st = smem + (kt & 1) * (2 * kTileBytes);
#pragma unroll
    for (int c = 0; c < kCopies; ++c) att_to_lds(r, st + (wave + NW * c) * 1024, koff[c]);
  };
  auto load_v = [&](int kt) {
    const int rows = min(kBN, len - kt * kBN);
    const __amdgpu_buffer_rsrc_t r = make_rsrc(vp + (int64_t)kt * kBN * vst, (uint32_t)(((rows - 1) * vst + D) * 2));
    uint8_t* st = smem + (kt & 1) * (2 * kTileBytes) + kTileBytes;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) att_to_lds(r, st + (wave + NW * c) * 1024, voff[c]);
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

  f32x16 acc[JD];
#pragma unroll
  for (int j = 0; j < JD; ++j) acc[j] = f32x16{};
  const float c = a.scale * 1.4426950408889634f;   // exponents in base 2
  // The maximum starts below every finite score whose exponent is finite. Exponents are x c - mc,
  // mc = m c: its rounding is a factor common to the row (raise() carries it over), unless it is so
  // large (`far`) that the factor leaves fp32: then m is taken off the scores first and mc is 0.
  float m = -3.4028234663852886e38f / fmaxf(c, 1.0f), mc = 0.0f;
  bool far = true;   // the same in every lane
  const float slack = kSlack / c;

  // Sum of the probabilities: a tile's own (at most 32 a lane), then l with what its last addition
  // lost, so that the error does not grow with the sequence (one running sum of 2^18 equal ones
  // drifts by up to 1e-3, of 2^24 by 1e-2).
  float l = 0.0f, lost = 0.0f, tile_sum = 0.0f;
  auto add_tile = [&] {
    const float y = tile_sum - lost, t = l + y;
    lost = (t - l) - y;
    l = t;
    tile_sum = 0.0f;
  };
  // Probabilities of score pair r (0..15) of a tile, rounded to bf16 for the product with V, whose
  // matrix instruction takes both operands in one type: o is off from float64 by 0.0024 of its norm,
  // 0.0017 with fp32 probabilities (both with o's own rounding; their rest as a second bf16 operand
  // would double that product). Their sum is taken before (v_dot2 on the rounded pairs holds up the
  // matrix unit).
  auto pair = [&](const f32x16 (&x)[2], uint32_t (&p)[16], int r) {
    const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r >> 3][2 * (r & 7)], c, -mc));
    const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r >> 3][2 * (r & 7) + 1], c, -mc));
    p[r] = pack_bf16x2(p0, p1);
    tile_sum += p0 + p1;
    asm volatile("" : "+v"(p[r]), "+v"(tile_sum));   // made here: not moved to their use
  };
  auto prob_operand = [&](const uint32_t (&p)[16], int t) {
    return __builtin_bit_cast(bf16x8, u32x4{p[4 * t], p[4 * t + 1], p[4 * t + 2], p[4 * t + 3]});
  };
  // keys past the sequence, or past the query
  auto mask = [&](f32x16 (&x)[2], int kt) {
    if (kt * kBN + kBN > len || (CAUSAL && kt * kBN + kBN - 1 > row0)) {
      const int lim = (CAUSAL ? min(row0 + l32, len - 1) : len - 1) - kt * kBN - 4 * h;
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        if (32 * (r >> 4) + 8 * ((r & 15) >> 2) + (r & 3) > lim) x[r >> 4][r & 15] = -__builtin_inff();
        if (r % 8 == 7) __builtin_amdgcn_sched_barrier(0);   // few condition registers at a time
      }
    }
  };
  // The running maximum moves only when a score passes it by more than kSlack powers of
  // two: until then the probabilities are at most 2^kSlack, with the same relative rounding.
  // Returns the factor for what was accumulated so far (l has it already): the difference of what is
  // really taken off the exponents, rounded products included. (m - mn) c in its place would weigh
  // the keys before against those after by up to 2^(1/16), at products of 2^20.
  auto raise = [&](float mx) {
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float mn = fmaxf(m, mx);
    float mcn = mn * c;
    const bool far_n = __ballot(fabsf(mcn) > 1048576.0f) != 0;
    if (far_n) mcn = 0.0f;
    const float alpha = __builtin_amdgcn_exp2f(__builtin_fmaf((far ? m : 0.0f) - (far_n ? mn : 0.0f), c, mc - mcn));
    m = mn;
    mc = mcn;
    far = far_n;
    l *= alpha;
    lost *= alpha;
    return alpha;
  };

  auto from_max = [&](f32x16 (&x)[2]) {
    if (far) {
#pragma unroll
      for (int r = 0; r < 32; ++r) x[r >> 4][r & 15] -= m;
    }
  };

  // Start of step kt: one barrier frees K(kt) and V(kt - 1) for the copies of K(kt + 2) and
  // V(kt + 1), and publishes K(kt + 1) and V(kt), which were requested a step ago.
  auto next_tiles = [&](int kt) {
    __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0): this wave's copies have landed; lgkmcnt(0)
    att_barrier();
    if (kt + 2 < nt) load_k(kt + 2);
    if (kt + 1 < nt) load_v(kt + 1);
  };
  // A step: the next tile's scores on the matrix unit while the second half of this tile's
  // probabilities is made, then the product with V while the next scores' maximum is found
  // and the first half of their probabilities is made. The exponentials cost about as
  // much issue time as the products: spread over both, they hide behind them.
  auto step = [&](f32x16 (&cur)[2], uint32_t (&pc)[16], f32x16 (&nxt)[2], uint32_t (&pn)[16], int kt) {
    next_tiles(kt);
    const uint8_t* sk = smem + ((kt + 1) & 1) * (2 * kTileBytes);
    const uint8_t* sv = smem + (kt & 1) * (2 * kTileBytes) + kTileBytes;
    bf16x8 fk[NK], fv[NV];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fk[u] = read_k(sk, u);
    __builtin_amdgcn_s_setprio(1);   // of the two waves of a SIMD, one runs ahead into the other product
#pragma unroll
    for (int u = 0; u < NK; ++u) {
      if (u + kAhead < NK) fk[u + kAhead] = read_k(sk, u + kAhead);
      else fv[u + kAhead - NK] = read_v(sv, u + kAhead - NK);
      nxt[u & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fk[u], fq[u >> 1], u < 2 ? f32x16{} : nxt[u & 1], 0, 0, 0);
#pragma unroll
      for (int r = 8 + 8 * u / NK; r < 8 + 8 * (u + 1) / NK; ++r) pair(cur, pc, r);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
    add_tile();
    mask(nxt, kt + 1);
    constexpr int kMax = NV / 4;   // products that cover the maximum
    auto value = [&](int u) {
      if (u + kAhead < NV) fv[u + kAhead] = read_v(sv, u + kAhead);
      acc[u % JD] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fv[u], prob_operand(pc, u / JD), acc[u % JD], 0, 0, 0);
    };
    float mx = -__builtin_inff(), alpha = 1.0f;
#pragma unroll
    for (int u = 0; u < kMax; ++u) {
      value(u);
#pragma unroll
      for (int r = 32 * u / kMax; r < 32 * (u + 1) / kMax; ++r) mx = fmaxf(mx, nxt[r >> 4][r & 15]);
      __builtin_amdgcn_sched_barrier(0);
    }
    const bool up = __ballot(mx > m + slack) != 0;
    if (up) alpha = raise(mx);
    from_max(nxt);
#pragma unroll
    for (int u = kMax; u < NV; ++u) {
      value(u);
#pragma unroll
      for (int r = 8 * (u - kMax) / (NV - kMax); r < 8 * (u + 1 - kMax) / (NV - kMax); ++r) pair(nxt, pn, r);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (up) {
#pragma unroll
      for (int j = 0; j < JD; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[j][r] *= alpha;
    }
  };

  // tiles this wave needs; the others it only helps to load
  const int ntw = row0 >= len ? 0 : CAUSAL ? min(nt, (row0 + 31) / kBN + 1) : nt;
  load_k(0);
  load_v(0);
  if (nt > 1) {
    load_k(1);
    att_wait_copies<2 * kCopies>();   // K(0), and Q before it
  } else {
    att_wait_copies<kCopies>();
  }
  att_barrier();
  int kt = 0;
  if (ntw > 0) {
    f32x16 s0[2], s1[2];
    uint32_t p0[16], p1[16];
#pragma unroll
    for (int u = 0; u < NK; ++u)
      s0[u & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_k(smem, u), fq[u >> 1], u < 2 ? f32x16{} : s0[u & 1], 0, 0, 0);
    mask(s0, 0);
    float mx = s0[0][0];
#pragma unroll
    for (int r = 1; r < 32; ++r) mx = fmaxf(mx, s0[r >> 4][r & 15]);
    raise(mx);
    from_max(s0);
#pragma unroll
    for (int r = 0; r < 8; ++r) pair(s0, p0, r);
    for (; kt + 2 < ntw; kt += 2) {
      step(s0, p0, s1, p1, kt);
      step(s1, p1, s0, p0, kt + 1);
    }
    if (kt + 1 < ntw) {
      step(s0, p0, s1, p1, kt);
      s0[1] = s1[1];
#pragma unroll
      for (int r = 0; r < 8; ++r) p0[r] = p1[r];
      ++kt;
    }
    next_tiles(kt);   // the last tile
    const uint8_t* sv = smem + (kt & 1) * (2 * kTileBytes) + kTileBytes;
    ++kt;
#pragma unroll
    for (int r = 8; r < 16; ++r) pair(s0, p0, r);
    add_tile();
#pragma unroll
    for (int u = 0; u < NV; ++u)
      acc[u % JD] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_v(sv, u), prob_operand(p0, u / JD), acc[u % JD], 0, 0, 0);
  }
  for (; kt < nt; ++kt) next_tiles(kt);

  // O^T through LDS (the tiles' space): each wave turns its block into rows and stores whole
  // 16-byte pieces. Row r's pieces are permuted by piece ^ (r % kPieces).
  __syncthreads();
  uint8_t* out = smem + wave * (32 * kRowBytes);
  static_assert(NW * 32 * kRowBytes <= 4 * kTileBytes, "output staging");
  l += __shfl_xor(l, 32);
  const float inv = 1.0f / l;
#pragma unroll
  for (int j = 0; j < JD; ++j)
#pragma unroll
    for (int r = 0; r < 16; r += 4)
      *reinterpret_cast<u32x2*>(out + l32 * kRowBytes + (((4 * j + r / 4) ^ (l32 & (kPieces - 1))) * 16) + 8 * h) =
          u32x2{pack_bf16x2(acc[j][r] * inv, acc[j][r + 1] * inv), pack_bf16x2(acc[j][r + 2] * inv, acc[j][r + 3] * inv)};
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt(0): the wave's own writes
  asm volatile("" ::: "memory");
#pragma unroll
  for (int u = 0; u < 32 / kRowsPerCopy; ++u) {
    const int r = u * kRowsPerCopy + lane / kPieces, piece = lane % kPieces;
    const u32x4 w = *reinterpret_cast<const u32x4*>(out + r * kRowBytes + ((piece ^ (r & (kPieces - 1))) * 16));
    if (row0 + r < len) *reinterpret_cast<u32x4*>(a.o + (int64_t)(beg + row0 + r) * a.o_st + head * a.o_sh + 8 * piece) = w;
  }
}

template <int D, int NW>
void launch_attention_cfg(const AttnArgs& a, hipStream_t s) {
  // as many heads of a group as divide it, up to the workgroup's waves
  int lg_heads = 0;
  while ((2 << lg_heads) <= NW && (a.H / a.Hk) % (2 << lg_heads) == 0) ++lg_heads;
  const int rows = 32 * NW >> lg_heads;
  const int64_t total = (a.T / rows + a.B) * (a.H >> lg_heads);
  const dim3 grid((unsigned)((total + 7) / 8 * 8)), block(64 * NW);
  if (a.causal) hipLaunchKernelGGL((attention_kernel<D, true, NW>), grid, block, 0, s, a, lg_heads);
  else hipLaunchKernelGGL((attention_kernel<D, false, NW>), grid, block, 0, s, a, lg_heads);
}

// Four waves or eight: eight load each tile half as often, four leave two workgroups on a CU (three
// of heads of 64), whose starts and ends overlap, and waste less at the ends of short sequences.
// Measured, 4 and 8 waves, one sequence, 30 heads of 128: 16896 tokens 3920 and 3700 us (causal 2195
// and 2140), 8192 909 and 882 (562 and 585), 4096 235 and 230 (162 and 164), 2048 75 and 106; 13 causal
// prompts of 315 on average, 32 heads on 8: 36.5 and 40.2; 20 sequences of 400, 30 heads on 15: 85 and
// 91. Heads of 64, 30 of them: 16896 2240 and 2335 (1230 and 1320), 8192 553 and 570 (325 and 384), 4096 153
// and 150 (99 and 112); 16 of them, 12000 611 and 619 (318 and 338), 8192 295 and 288 (179 and 158: 3.5 and 4
// rounds of workgroups). So eight from a mean length of 8192 on, for heads of 128 alone: two waves a
// SIMD are all that their registers leave either way, where four-wave workgroups of 64 make three.
template <int D>
void launch_attention_d(const AttnArgs& a, hipStream_t s) {
  if constexpr (D == 128) {
    if (a.T >= 8192 * (int64_t)a.B) return launch_attention_cfg<D, 8>(a, s);
  }
  launch_attention_cfg<D, 4>(a, s);
}

}  // namespace

hipError_t launch_attention(const AttnArgs& a, int D, hipStream_t stream) {
  if (D == 64) launch_attention_d<64>(a, stream);
  else launch_attention_d<128>(a, stream);
  return hipGetLastError();
}

}  // namespace svdq
