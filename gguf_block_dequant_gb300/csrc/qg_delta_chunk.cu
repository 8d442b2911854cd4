// qg_delta_chunk.cu -- the gated delta rule over prompts, 32 tokens at a time on the tensor cores.
//
// With G_i the sum of the log decays of a chunk's tokens up to i and S0 the state before the chunk, the updates u_i of
// the definition solve
//   u_i + sum_{j<i} beta_i e^{G_i - G_j} (k_i . k_j) u_j = beta_i (v_i - e^{G_i} S0^T k_i),
// a unit lower triangular system (1 + A) U = diag(beta) (...).  With T = (1 + A)^-1 diag(beta):
//   R = V - diag(e^G) K S0,   U = T R,
//   O = diag(e^G) Q S0 + [e^{G_i - G_j} q_i . k_j, j <= i] U,   S = e^{G_C} S0 + K^T diag(e^{G_C - G}) U.
// Everything that does not need S0 (norms, T, the decayed Q K^T) comes from one kernel, parallel over chunks and heads;
// a second one walks the chunks of each head with the state in registers.  No exponent is above 0 while log
// decays are not (positive ones are allowed); sums of them are kept in two terms, so that decays between neighbours stay exact
// after strong ones.
//
// Products run on the tensor cores with f32 sums.  Keys, queries, the state and what a chunk adds to it are x = s (hi + lo) in f16,
// s a power of two per row that brings the row's largest magnitude to [2^7, 2^8), hi the multiple of 2^-3 nearest x/s and lo the
// f16 nearest the rest: 23 bits of the row's largest; hi hi + hi lo + lo hi leaves 2^-22 of it and its partner's.  (Two bf16 terms would
// leave 2^-16, tf32 ones cost twice.)  In a row of R and U every element is a token's, in one of T and of the decayed Q K^T every
// element is what becomes of a token's: a token must not lose bits to later, larger ones, nor to earlier ones that are forgotten, so these
// have no scale in common.  They are hi + mid + lo in bf16, whose exponents are f32's: all 24 bits of each, and the six largest of
// their nine products leave 2^-23.
#include <algorithm>
#include <atomic>

#include "qg_delta.cuh"
#include "qg_mma.cuh"
#include "qg_tc.cuh"

__device__ unsigned int g_qg_status_delta_chunk;  // this translation unit's device status word
static std::atomic<bool> g_launched{false};       // whether a kernel that may set it has been launched

namespace {

using qg::DeltaArgs;
constexpr int C = qg::kDeltaChunk;
static_assert(C == 32, "a lane per token");

// ---- the workspace ------------------------------------------------------------------------------
// Sequence b's chunks have the numbers q_start[b] / 32 + b, and on: they rise, and ceil(n / 32) of them fit
// before the next sequence's.  Per (chunk, key head): DK / 64 blocks of hi terms, then those of lo terms, each [32 rows of K, 32
// of Q][64] f16.  Per (chunk, value head): T and A, [32][32 hi, 32 mid] and [32][32 lo] bf16 each, and the factors below.  So every row of
// a block is 128 bytes, and its eight 16-byte pieces are exchanged by the row's low three bits: the 128-byte swizzle of the tensor
// cores' operands, and free of bank conflicts for ldmatrix, turned or not.  Rows of lo terms are 64 bytes, their four pieces exchanged by
// the row's bits 1 and 2: the 64-byte swizzle.
constexpr int kBlock = C * 128;           // bytes of 32 rows of a block; where Q is in one of K and Q
constexpr int kThree = kBlock + C * 64;   // of T or A; its lo terms are kBlock bytes in
template <int DK>
struct Tiles {
  static constexpr int kLo = DK / 64 * 2 * kBlock;  // from the hi terms to the lo terms
  static constexpr int kKQAll = 2 * kLo;
};
struct Factors {
  float fk[C];     // e^{G_j} sk_j: what K S0 is multiplied by
  float fq[C];     // e^{G_i} sq_i
  float wk[C];     // e^{G_C - G_j} sk_j
  float alpha[C], beta[C], sk[C], sq[C];  // token by token, for chunks with infinite or NaN values
  float dec;       // e^{G_C}
  int odd;         // such a value among the queries, keys and gates, a factor that leaves f32, or a state that is forgotten and grows
  float pad[30];
};
constexpr int kTA = 2 * kThree + static_cast<int>(sizeof(Factors));
static_assert(kTA % 16 == 0, "bulk copies");

// byte offset of piece `piece` (16 bytes) of a row of a block
QG_DEVICE uint32_t at_piece(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }
// the same for rows of 64 bytes
QG_DEVICE uint32_t at_piece64(int row, int piece) { return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4); }
// the same in the blocks of K and Q
QG_DEVICE uint32_t kq_at(int row, int piece) { return (piece >> 3) * 2 * kBlock + at_piece(row, piece & 7); }

// the power of two that brings magnitude bits m to [2^7, 2^8), and its inverse; 1 for infinities and NaN
QG_DEVICE void row_scale(uint32_t m, float &s, float &inv) {
  const uint32_t e = max(m >> 23, 8u);
  s = e == 255u ? 1.f : __uint_as_float((e - 7u) << 23);
  inv = e == 255u ? 1.f : __uint_as_float((261u - e) << 23);
}
QG_DEVICE uint32_t mag(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u, kNoBf16 = 0x7F7F8000u;  // magnitudes from the second on round to an infinite bf16
constexpr float kMost = 0x1p127f;  // what is below it can be split
// the larger one, or NaN where one of them is
QG_DEVICE float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// x inv and y inv, below 2^8, as packed f16 terms: hi a multiple of 2^-3 (adding 3 2^19 rounds to one; 11 bits), lo the rest
constexpr float kRound = 1572864.f;
QG_DEVICE void split2(f2 x, f2 inv, uint32_t &hi, uint32_t &lo) {
  const f2 h = add2(fma2(x, inv, mk2(kRound, kRound)), mk2(-kRound, -kRound));
  const f2 l = fma2(x, inv, mk2(-h.x, -h.y));
  hi = pack16<false>(h.x, h.y);
  lo = pack16<false>(l.x, l.y);
}
QG_DEVICE void split2(float x, float y, float inv, uint32_t &hi, uint32_t &lo) { split2(mk2(x, y), mk2(inv, inv), hi, lo); }

// x and y as three packed bf16 terms each: what is left behind two roundings to 8 bits has 8 itself, so nothing is lost
// down to 2^-126; magnitudes of 2^128 - 2^119 and more have no bf16
QG_DEVICE void split3(float x, float y, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
  hi = pack16<true>(x, y);
  x -= lo16<true>(hi);
  y -= hi16<true>(hi);
  mid = pack16<true>(x, y);
  lo = pack16<true>(x - lo16<true>(mid), y - hi16<true>(mid));
}

// N independent tiles c[i] += a b (FIRST: from 0): the tiles take turns, so that no product waits for the sum of the one before
// it (24 cycles; one can start every 8)
template <bool BF16, bool FIRST, int N>
QG_DEVICE void mma_each(float (&c)[N][4], const uint32_t (&a)[4], const uint32_t (&b)[N][2]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (!FIRST)
      mma16816<BF16>(c[i], a, b[i][0], b[i][1]);
    else if constexpr (BF16)
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, "
          "%10, %10};"
          : "=f"(c[i][0]), "=f"(c[i][1]), "=f"(c[i][2]), "=f"(c[i][3])
          : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[i][0]), "r"(b[i][1]), "f"(0.f));
    else
      asm volatile(
          "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, "
          "%10};"
          : "=f"(c[i][0]), "=f"(c[i][1]), "=f"(c[i][2]), "=f"(c[i][3])
          : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[i][0]), "r"(b[i][1]), "f"(0.f));
  }
}
// c[i] += (ah + al) (bh + bl), f16, without al bl
template <bool FIRST, int N>
QG_DEVICE void mma3(float (&c)[N][4], const uint32_t (&ah)[4], const uint32_t (&al)[4], const uint32_t (&bh)[N][2],
                    const uint32_t (&bl)[N][2]) {
  mma_each<false, FIRST>(c, al, bh);
  mma_each<false, false>(c, ah, bl);
  mma_each<false, false>(c, ah, bh);
}
// c[i] += (a[0] + a[1] + a[2]) (b[0] + b[1] + b[2]), bf16, without the three smallest products
template <bool FIRST, int N>
QG_DEVICE void mma6(float (&c)[N][4], const uint32_t (&a)[3][4], const uint32_t (&b)[3][N][2]) {
  mma_each<true, FIRST>(c, a[2], b[0]);
  mma_each<true, false>(c, a[0], b[2]);
  mma_each<true, false>(c, a[1], b[1]);
  mma_each<true, false>(c, a[1], b[0]);
  mma_each<true, false>(c, a[0], b[1]);
  mma_each<true, false>(c, a[0], b[0]);
}
// right operands of two tiles of 8
template <bool TRANS>
QG_DEVICE void load2(uint32_t (&b0)[2], uint32_t (&b1)[2], uint32_t addr) {
  uint32_t r[4];
  if constexpr (TRANS) ldsm4_t(r, addr);
  else ldsm4(r, addr);
  b0[0] = r[0], b0[1] = r[1], b1[0] = r[2], b1[1] = r[3];
}

// 2^y.  What a state keeps from chunk to chunk multiplies up: a state that hardly decays would gather the error of
// ex2 (2^-22) hundreds of times in one direction, so factors near 1, below and above, come from the series, rounded once.
QG_DEVICE float chunk_decay(float y) {
  const float x = y * 0.6931471805599453f;
  if (fabsf(x) > 0.03125f) return ex2(y);
  return fmaf(x, fmaf(x, fmaf(x, fmaf(x, 1.f / 24.f, 1.f / 6.f), 0.5f), 1.f), 1.f);
}

QG_DEVICE int chunk_base(const DeltaArgs &a, int b) { return qg::delta_tok(a, b) / C + b; }

struct ChunkArgs {
  DeltaArgs d;
  unsigned char *kq, *ta;
  int first_len;  // shorter sequences are not this kernel's
  int slots;      // chunk numbers there is room for
};

// ---- what does not need the state -------------------------------------------------------------------
// A CTA of four warps per chunk and key head.  Rows are normalised and split by a warp each; the products of keys with keys and
// queries with keys take a warp per 16 rows; then a warp per value head solves for T, a lane per column (in blocks of 16: in
// one block of 32 it all took 39 us more), and another makes the decayed Q K^T.  30042 tokens, 16 key and 32 value heads:
// 285 us for 1.39 GB moved, 4900 instructions a value head and chunk at 0.43 an issue slot, shared memory's pipe busy 57 % of the
// time, 16 and 18 registers a thread spilled (heads of 128 and of 64).  Latency bounds it, so rows of CTAs to come are sent to L2
// (48 us less), and registers and shared memory are kept to five CTAs an SM (four: 13 us more): decays (powers of two of
// differences of sums in log2) are made again rather than kept, and T is turned in the room of the tiles, from which it and Q K^T
// leave as bulk copies (16 bytes a lane stored to as many lines took 34 us more).  Sums of log decays in two floats rather than
// doubles took no less.
constexpr int kPrepWarps = 4;
// CTAs whose rows a CTA sends to L2 before they start: half of those that run at once (160 to 440 take the same, 80 and 760 20 us more)
constexpr int kPrepAhead = 380;
constexpr int kTurn = C + 4;  // floats of a row there

template <int DK>
__global__ void __launch_bounds__(kPrepWarps * 32, 5) delta_prep_kernel(const ChunkArgs a) {
  extern __shared__ __align__(128) unsigned char tile[];  // K hi, K lo, Q hi, Q lo
  __shared__ __align__(16) float kk[C][kTurn], qk[C][kTurn];
  __shared__ float scale_k[C], scale_q[C];
  __shared__ __align__(16) float2 gsum[kPrepWarps][C];
  __shared__ int bad_rows;
  constexpr int LO = Tiles<DK>::kLo;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = static_cast<int>(blockIdx.x) / a.d.Hk, hk = static_cast<int>(blockIdx.x) % a.d.Hk;
  pdl_wait();
  pdl_launch_dependents();
  // the sequence whose chunk this is: chunk_base(lo) <= slot < chunk_base(hi), as far as is known.  32 places a round, since a
  // round costs a load's latency
  int lo = 0, hi = a.d.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const unsigned below = __ballot_sync(0xFFFFFFFFu, at < hi && chunk_base(a.d, min(at, hi - 1)) <= slot);
    const int k = __ffs(~below) - 1;  // places up to the first above
    const int base = lo;
    lo = base + (below == 0xFFFFFFFFu ? 32 : k) * step;
    hi = min(hi, lo + step);
  }
  const int t00 = qg::delta_tok(a.d, lo), n = qg::delta_tok(a.d, lo + 1) - t00;
  const int first = (slot - chunk_base(a.d, lo)) * C;
  if (n < a.first_len || first < 0 || first >= n) return;
  const int len = min(C, n - first), t0 = t00 + first;

  if (tid == 0) bad_rows = 0;
  __syncthreads();
  // rows: 8 of K and 8 of Q a warp, all of them under way at once
  constexpr int E = DK / 32;
  constexpr int R = C / kPrepWarps;
  float x[2][R][E];
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = warp * R + r;
#pragma unroll
      for (int e = 0; e < E; ++e) x[z][r][e] = 0.f;
      if (i < len) {
        const float *p = (z ? a.d.q + (t0 + i) * a.d.q_stride : a.d.k + (t0 + i) * a.d.k_stride) + hk * DK + lane * E;
        if constexpr (E == 4) {
          const float4 v = __ldg(reinterpret_cast<const float4 *>(p));
          x[z][r][0] = v.x, x[z][r][1] = v.y, x[z][r][2] = v.z, x[z][r][3] = v.w;
        } else {
          const float2 v = __ldg(reinterpret_cast<const float2 *>(p));
          x[z][r][0] = v.x, x[z][r][1] = v.y;
        }
      }
    }
  // rows of a CTA to come go to L2: 32 of K and of Q, DK / 32 lines each
  for (int at = tid; at < C * E; at += kPrepWarps * 32) {
    const int t = t0 + C * (kPrepAhead / a.d.Hk + 1) + at / E;
    if (t < a.d.T) {
      const long long off = hk * DK + at % E * 32;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.d.k + t * a.d.k_stride + off));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(a.d.q + t * a.d.q_stride + off));
    }
  }
  const int group = a.d.Hv / a.d.Hk;
  // the gates of this warp's first item, needed at the end
  auto head_of = [&](int it) {
    const int r = it < group ? it : it - group;
    return a.d.tiled ? hk + r * a.d.Hk : hk * group + r;
  };
  auto gates_of = [&](int it) {
    return lane < len && it < 2 * group ? qg::delta_gates(a.d, t0 + lane, head_of(it)) : make_float2(0.f, 0.f);
  };
  float2 gates = gates_of(warp);
  // norms and scales: lane l works for row l / 2 of the warp's sixteen (8 of K, 8 of Q)
  static_assert(R == 8, "sixteen rows a warp");
  float ss[2 * R];
  uint32_t big = 0;
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float t = 0.f;
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        t = fmaf(x[z][r][e], x[z][r][e], t);
        m = max(m, mag(x[z][r][e]));
      }
      ss[z * R + r] = t;
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      if ((lane >> 1) == z * R + r) big = m;
    }
  reduce_scatter(ss, lane);  // ss[0]: the sum of row lane / 2
  const int mine = lane >> 1;
  float f = mine >= R ? a.d.scale : 1.f;
  if (a.d.l2norm && warp * R + (mine & (R - 1)) < len) f *= 1.f / sqrtf(ss[0] + a.d.eps);
  big = mag(__uint_as_float(big) * f);  // the largest magnitude of the products with f: rounding keeps the order
  float row_s, row_inv;
  row_scale(big, row_s, row_inv);
  float to = f * row_inv;  // a power of two beside f: one rounding
  if (big >= kInfBits) {
    bad_rows = 1;
  } else if (!(fabsf(to) < INFINITY)) {  // rows next to nothing, raised by the norm (zeros, for one)
    row_s = 0x1p-60f;
    to = f * 0x1p60f;
  }
  if ((lane & 1) == 0) (mine >= R ? scale_q : scale_k)[warp * R + (mine & (R - 1))] = row_s;
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = warp * R + r;
      const float w = __shfl_sync(0xFFFFFFFFu, to, 2 * (z * R + r));
      unsigned char *t = tile + z * kBlock;
      const int byte = lane * E * 2;  // of the row
      const uint32_t at = kq_at(i, byte >> 4) + (byte & 15);
      uint32_t h[E / 2], l[E / 2];
#pragma unroll
      for (int e = 0; e < E; e += 2) split2(x[z][r][e], x[z][r][e + 1], w, h[e / 2], l[e / 2]);
      if constexpr (E == 4) {
        *reinterpret_cast<uint2 *>(t + at) = make_uint2(h[0], h[1]);
        *reinterpret_cast<uint2 *>(t + LO + at) = make_uint2(l[0], l[1]);
      } else {
        *reinterpret_cast<uint32_t *>(t + at) = h[0];
        *reinterpret_cast<uint32_t *>(t + LO + at) = l[0];
      }
    }
  fence_proxy_async_smem();
  __syncthreads();
  if (tid == 0)  // the tiles leave as they lie, while the products are made of them
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(
                     a.kq + (static_cast<size_t>(slot) * a.d.Hk + hk) * Tiles<DK>::kKQAll),
                 "r"(smem_u32(tile)), "r"(Tiles<DK>::kKQAll)
                 : "memory");
  // products: warps 0, 1 keys with keys, 2, 3 queries with keys; 16 rows each
  {
    const uint32_t k0 = smem_u32(tile), rows = k0 + (warp >= 2 ? kBlock : 0);
    const int r0 = (warp & 1) * 16;
    float c[4][4];
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
      uint32_t ah[4], al[4];
      const uint32_t at = kq_at(r0 + (lane & 15), 2 * ks + (lane >> 4));
      ldsm4(ah, rows + at);
      ldsm4(al, rows + LO + at);
      uint32_t bh[4][2], bl[4][2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t bt = kq_at(16 * p + (lane & 7) + ((lane >> 4) << 3), 2 * ks + ((lane >> 3) & 1));
        load2<false>(bh[2 * p], bh[2 * p + 1], k0 + bt);
        load2<false>(bl[2 * p], bl[2 * p + 1], k0 + LO + bt);
      }
      if (ks == 0) mma3<true>(c, ah, al, bh, bl);
      else mma3<false>(c, ah, al, bh, bl);
    }
    float(*out)[kTurn] = warp >= 2 ? qk : kk;
    const float *sr = warp >= 2 ? scale_q : scale_k;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int i = r0 + (lane >> 2) + 4 * e, j = 8 * t + 2 * (lane & 3);
        *reinterpret_cast<float2 *>(&out[i][j]) = make_float2(c[t][e] * sr[i] * scale_k[j], c[t][e + 1] * sr[i] * scale_k[j + 1]);
      }
  }
  if (tid == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // T is turned in the tiles' room
  __syncthreads();

  // items: T of every value head, then the decayed Q K^T of every value head
  for (int it = warp; it < 2 * group; it += kPrepWarps) {
    const int h = head_of(it);
    unsigned char *ta = a.ta + (static_cast<size_t>(slot) * a.d.Hv + h) * kTA;
    Factors *f = reinterpret_cast<Factors *>(ta + 2 * kThree);
    const float2 ga = gates;
    gates = gates_of(it + kPrepWarps);
    double sum = ga.x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += y;
    }
    sum *= 1.4426950408889634;  // log2(e)
    const float g_hi = static_cast<float>(sum), g_lo = static_cast<float>(sum - g_hi);
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the room is free
    __syncwarp();
    gsum[warp][lane] = make_float2(g_hi, g_lo);
    __syncwarp();
    // this lane's row: the decay from token j to the lane's, times p[j], for j <= lane - below
    auto decayed = [&](float (&v)[C], const float *p, int below) {
#pragma unroll
      for (int j = 0; j < C; j += 4) {
        const float4 g0 = *reinterpret_cast<const float4 *>(&gsum[warp][j]), g1 = *reinterpret_cast<const float4 *>(&gsum[warp][j + 2]);
        const float4 m = *reinterpret_cast<const float4 *>(p + j);
        auto one = [&](int i, float hi, float lo, float x) { v[i] = i + below <= lane ? ex2((g_hi - hi) + (g_lo - lo)) * x : 0.f; };
        one(j, g0.x, g0.y, m.x);
        one(j + 1, g0.z, g0.w, m.y);
        one(j + 2, g1.x, g1.y, m.z);
        one(j + 3, g1.z, g1.w, m.w);
      }
    };
    unsigned char *const room = tile + warp * kThree;
    // a lane per row: its pieces leave by way of the room, 6 KB at once
    auto write_row = [&](const float (&v)[C], unsigned char *dst) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        uint32_t h4[4], m4[4], l4[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split3(v[8 * p + 2 * e], v[8 * p + 2 * e + 1], h4[e], m4[e], l4[e]);
        *reinterpret_cast<uint4 *>(room + at_piece(lane, p)) = make_uint4(h4[0], h4[1], h4[2], h4[3]);
        *reinterpret_cast<uint4 *>(room + at_piece(lane, 4 + p)) = make_uint4(m4[0], m4[1], m4[2], m4[3]);
        *reinterpret_cast<uint4 *>(room + kBlock + at_piece64(lane, p)) = make_uint4(l4[0], l4[1], l4[2], l4[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0)
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(dst),
                     "r"(smem_u32(room)), "r"(kThree)
                     : "memory");
    };
    float w[C];
    if (it >= group) {
      decayed(w, qk[lane], 0);
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < C; ++j) top = max_nan(top, fabsf(w[j]));
      write_row(w, ta + kThree);
      const float2 gl = gsum[warp][C - 1];
      const float eg = ex2(g_hi + g_lo);
      f->fk[lane] = eg * scale_k[lane];
      f->fq[lane] = eg * scale_q[lane];
      const float wk = ex2((gl.x - g_hi) + (gl.y - g_lo)) * scale_k[lane];
      f->wk[lane] = wk;
      f->alpha[lane] = expf(ga.x);
      f->beta[lane] = ga.y;
      f->sk[lane] = scale_k[lane];
      f->sq[lane] = scale_q[lane];
      const bool bad = !(fabsf(ga.x) < INFINITY && fabsf(ga.y) < INFINITY && top < kMost && eg < kMost && wk < kMost);
      // a decay that leaves nothing must not be made up for by ones that grow: sums of log decays cannot tell
      const bool again = __any_sync(0xFFFFFFFFu, ga.x <= qg::kDeltaForgets) && __any_sync(0xFFFFFFFFu, ga.x > 0.f);
      const int odd = __any_sync(0xFFFFFFFFu, bad) || again || bad_rows;
      if (lane == 0) {
        f->dec = chunk_decay(gl.x + gl.y);
        f->odd = odd;
      }
      continue;
    }
    float(*const M)[kTurn] = reinterpret_cast<float(*)[kTurn]>(room);
    // a lane per row of A
    decayed(w, kk[lane], 1);
#pragma unroll
    for (int j = 0; j < C; j += 4)
      *reinterpret_cast<float4 *>(&M[lane][j]) = make_float4(ga.y * w[j], ga.y * w[j + 1], ga.y * w[j + 2], ga.y * w[j + 3]);
    __syncwarp();
    // (1 + A) T = 1 in blocks of 16.  Both diagonal blocks at once, a lane per column, from the top, four sums a row
    constexpr int H = C / 2;
    const int blk = lane / H, col = lane % H;
    float x[H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
      float acc[4] = {i == col ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j4 = 0; j4 < i; j4 += 4) {
        const float4 m = *reinterpret_cast<const float4 *>(&M[blk * H + i][blk * H + j4]);
        acc[0] = fmaf(-m.x, x[j4], acc[0]);
        if (j4 + 1 < i) acc[1] = fmaf(-m.y, x[j4 + 1], acc[1]);
        if (j4 + 2 < i) acc[2] = fmaf(-m.z, x[j4 + 2], acc[2]);
        if (j4 + 3 < i) acc[3] = fmaf(-m.w, x[j4 + 3], acc[3]);
      }
      x[i] = i < col ? 0.f : (acc[0] + acc[1]) + (acc[2] + acc[3]);
    }
    // then T21 = -T22 (A21 T11): lanes col and col + 16 make column col, rows of one parity each
    float y[H];
    {
      float t[H];
#pragma unroll
      for (int j = 0; j < H; ++j) t[j] = __shfl_sync(0xFFFFFFFFu, x[j], col);
#pragma unroll
      for (int r = 0; r < H; r += 2) {
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < H; j += 4) {
          const float4 m = *reinterpret_cast<const float4 *>(&M[H + r + blk][j]);
          acc[0] = fmaf(-m.x, t[j], acc[0]);
          acc[1] = fmaf(-m.y, t[j + 1], acc[1]);
          acc[2] = fmaf(-m.z, t[j + 2], acc[2]);
          acc[3] = fmaf(-m.w, t[j + 3], acc[3]);
        }
        const float own = (acc[0] + acc[1]) + (acc[2] + acc[3]), other = __shfl_xor_sync(0xFFFFFFFFu, own, H);
        y[r] = blk ? other : own;
        y[r + 1] = blk ? own : other;
      }
    }
    __syncwarp();
    const float beta_col = __shfl_sync(0xFFFFFFFFu, ga.y, col);
#pragma unroll
    for (int i = 0; i < H; ++i) M[blk * H + i][lane] = blk ? x[i] : x[i] * ga.y;  // T22 goes into a product first
    __syncwarp();
#pragma unroll
    for (int r = 0; r < H; r += 2) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < r + 2; j += 4) {
        const float4 m = *reinterpret_cast<const float4 *>(&M[H + r + blk][H + j]);
        acc[0] = fmaf(m.x, y[j], acc[0]);
        acc[1] = fmaf(m.y, y[j + 1], acc[1]);
        if (j + 2 < r + 2) {
          acc[2] = fmaf(m.z, y[j + 2], acc[2]);
          acc[3] = fmaf(m.w, y[j + 3], acc[3]);
        }
      }
      M[H + r + blk][col] = beta_col * ((acc[0] + acc[1]) + (acc[2] + acc[3]));
    }
    __syncwarp();
    if (blk) {
#pragma unroll
      for (int i = 0; i < H; ++i) M[H + i][lane] = x[i] * ga.y;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < C; j += 4) {
      const float4 m = *reinterpret_cast<const float4 *>(&M[lane][j]);
      w[j] = m.x, w[j + 1] = m.y, w[j + 2] = m.z, w[j + 3] = m.w;
    }
    __syncwarp();  // rows of T are read before their pieces take the room
    write_row(w, ta);
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ---- the walk ------------------------------------------------------------------------------------------
// A warp owns 16 columns of a head's state, as S^T in the accumulator layout (rows: columns of S): it is the left operand of
// both products with the old state, U^T in turn the left operand of the next two, so nothing but the tiles from the
// kernel above passes through shared memory, and warps never wait for one another.  The tiles come through a ring of
// bulk copies; the warp that leaves a stage last asks for its next contents.  For heads whose columns are no multiple of 128 (64
// columns with four warps take 3.6 us a chunk, 360 products of 8 cycles each a warp, where 128 take 3.1 below).
template <int DK, int W, int NST>
struct WalkSmem {
  static constexpr int kStage = (Tiles<DK>::kKQAll + kTA + 1023) / 1024 * 1024;  // pieces are found by exclusive or
  static constexpr int kBytes = NST * kStage;
};

template <int DK, int W, int NST>
__global__ void __launch_bounds__(W * 32) delta_walk_kernel(const ChunkArgs a) {
  extern __shared__ __align__(1024) unsigned char ring[];
  __shared__ uint64_t full[NST];
  __shared__ int left[NST];  // warps that are done with a stage's contents
  constexpr int LO = Tiles<DK>::kLo, kStage = WalkSmem<DK, W, NST>::kStage;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int parts = a.d.Dv / (16 * W);
  const int part = static_cast<int>(blockIdx.x) % parts, bh = static_cast<int>(blockIdx.x) / parts;
  const int h = bh % a.d.Hv, b = bh / a.d.Hv;
  pdl_wait();
  pdl_launch_dependents();
  const int t00 = qg::delta_tok(a.d, b), n = qg::delta_tok(a.d, b + 1) - t00;
  if (n < a.first_len || n <= 0) return;
  const int chunks = (n + C - 1) / C;
  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&full[i], 1);
      left[i] = 0;
    }
    fence_mbar_init();
  }
  __syncthreads();
  const int slot0 = chunk_base(a.d, b), hk = qg::delta_key_head(a.d, h);
  if (slot0 + chunks > a.slots) return;

  auto ask = [&](int c) {
    unsigned char *dst = ring + (c % NST) * kStage;
    uint64_t *bar = &full[c % NST];
    mbar_arrive_expect_tx(bar, Tiles<DK>::kKQAll + kTA);
    bulk_g2s(dst, a.kq + (static_cast<size_t>(slot0 + c) * a.d.Hk + hk) * Tiles<DK>::kKQAll, Tiles<DK>::kKQAll, bar);
    bulk_g2s(dst + Tiles<DK>::kKQAll, a.ta + (static_cast<size_t>(slot0 + c) * a.d.Hv + h) * kTA, kTA, bar);
  };
  if (tid == 0) {
    asm volatile("fence.proxy.async;" ::: "memory");  // the tiles were written by plain stores
    for (int c = 0; c < min(NST, chunks); ++c) ask(c);
  }

  const int q4 = lane & 3, r8 = lane >> 2;
  const int d0 = h * a.d.Dv + (part * W + warp) * 16 + r8;  // this lane's columns of S: d0 and d0 + 8
  const bool teller = tid == 0 && part == 0 && h == 0;
  // the state: s[ct] holds rows 8 ct + 2 q4, + 1 of S for column d0, then for d0 + 8
  float s[DK / 8][4];
  {
    const int in = a.d.state_in ? __ldg(a.d.state_in + b) : -1;
    if (teller && (in < -1 || in >= a.d.n_slots)) atomicOr(&g_qg_status_delta_chunk, QG_STATUS_BIT_ID);
    const bool have = in >= 0 && in < a.d.n_slots;
    const float *p = a.d.states + (have ? in : 0) * a.d.slot_stride + static_cast<long long>(h) * DK * a.d.Dv + (d0 - h * a.d.Dv);
#pragma unroll
    for (int ct = 0; ct < DK / 8; ++ct)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[ct][e] = have ? p[static_cast<long long>(8 * ct + 2 * q4 + (e & 1)) * a.d.Dv + 8 * (e >> 1)] : 0.f;
  }
  const float *vp = a.d.v + d0;
  float *op = a.d.out + d0;
  // this lane's tokens of a chunk are 8 t + 2 q4 and the one after
  const float *vnext = vp + static_cast<long long>(t00 + 2 * q4) * a.d.v_stride;
  float *onext = op + static_cast<long long>(t00 + 2 * q4) * a.d.out_stride;
  auto load_v = [&](int c, float (&v)[4][4]) {  // called once for every chunk in turn
    const float *p = vnext;
    if ((c + 1) * C <= n) {
#pragma unroll
      for (int t = 0; t < 4; ++t, p += 8 * a.d.v_stride) {
        v[t][0] = __ldg(p);
        v[t][1] = __ldg(p + a.d.v_stride);
        v[t][2] = __ldg(p + 8);
        v[t][3] = __ldg(p + a.d.v_stride + 8);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t, p += 8 * a.d.v_stride) {
        const int j = c * C + 8 * t + 2 * q4;
        v[t][0] = j < n ? __ldg(p) : 0.f;
        v[t][1] = j + 1 < n ? __ldg(p + a.d.v_stride) : 0.f;
        v[t][2] = j < n ? __ldg(p + 8) : 0.f;
        v[t][3] = j + 1 < n ? __ldg(p + a.d.v_stride + 8) : 0.f;
      }
    }
    vnext += C * a.d.v_stride;
  };
  float v[4][4];
  load_v(0, v);
  // where this lane's rows of the tiles start for ldmatrix: pieces are then found by exclusive or.  Keys and queries as right
  // operands of S0 (a row per token), keys as right operands of U (turned)
  const int brow = (lane & 7) + ((lane >> 4) << 3), bpiece = (lane >> 3) & 1;
  const uint32_t off_b = at_piece(brow, bpiece), off_lo = at_piece64(brow, bpiece), off_t = at_piece(lane & 15, lane >> 4);

  for (int c = 0; c < chunks; ++c) {
    const int st = c % NST;
    if (!mbar_wait(&full[st], (c / NST) & 1)) {
      if (lane == 0) atomicOr(&g_qg_status_delta_chunk, QG_STATUS_BIT_TIMEOUT);
      return;
    }
    const uint32_t kt = smem_u32(ring + st * kStage), tt = kt + Tiles<DK>::kKQAll, at = tt + kThree;
    const Factors *f = reinterpret_cast<const Factors *>(ring + st * kStage + Tiles<DK>::kKQAll + 2 * kThree);
    float o[4][4];
    bool odd = false;
    {
      // rows of S^T in two terms (a NaN does not count for the scale; it makes its row's products NaN)
      float m0 = 0.f, m1 = 0.f;
#pragma unroll
      for (int ct = 0; ct < DK / 8; ++ct) {
        m0 = fmaxf(m0, fmaxf(fabsf(s[ct][0]), fabsf(s[ct][1])));
        m1 = fmaxf(m1, fmaxf(fabsf(s[ct][2]), fabsf(s[ct][3])));
      }
      m0 = fmaxf(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, 1));
      m1 = fmaxf(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, 1));
      m0 = fmaxf(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, 2));
      m1 = fmaxf(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, 2));
      float s0, i0, s1, i1;
      row_scale(mag(m0), s0, i0);
      row_scale(mag(m1), s1, i1);
      float x[8][4];  // (K S0)^T, then (Q S0)^T
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        uint32_t ah[4], al[4];
        split2(s[2 * ks][0], s[2 * ks][1], i0, ah[0], al[0]);
        split2(s[2 * ks][2], s[2 * ks][3], i1, ah[1], al[1]);
        split2(s[2 * ks + 1][0], s[2 * ks + 1][1], i0, ah[2], al[2]);
        split2(s[2 * ks + 1][2], s[2 * ks + 1][3], i1, ah[3], al[3]);
        uint32_t bh[8][2], bl[8][2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint32_t at = ((kt + off_b) ^ ((ks & 3) << 5)) + (ks >> 2) * 2 * kBlock + p * 16 * 128;
          load2<false>(bh[2 * p], bh[2 * p + 1], at);
          load2<false>(bl[2 * p], bl[2 * p + 1], at + LO);
          load2<false>(bh[4 + 2 * p], bh[5 + 2 * p], at + kBlock);
          load2<false>(bl[4 + 2 * p], bl[5 + 2 * p], at + kBlock + LO);
        }
        if (ks == 0) mma3<true>(x, ah, al, bh, bl);
        else mma3<false>(x, ah, al, bh, bl);
      }
      // R^T = V^T - e^G (K S0)^T, in v; O^T = e^G (Q S0)^T
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float2 fk = *reinterpret_cast<const float2 *>(f->fk + 8 * t + 2 * q4);
        const float2 fq = *reinterpret_cast<const float2 *>(f->fq + 8 * t + 2 * q4);
        v[t][0] = fmaf(-fk.x * s0, x[t][0], v[t][0]);
        v[t][1] = fmaf(-fk.y * s0, x[t][1], v[t][1]);
        v[t][2] = fmaf(-fk.x * s1, x[t][2], v[t][2]);
        v[t][3] = fmaf(-fk.y * s1, x[t][3], v[t][3]);
        o[t][0] = x[4 + t][0] * (fq.x * s0);
        o[t][1] = x[4 + t][1] * (fq.y * s0);
        o[t][2] = x[4 + t][2] * (fq.x * s1);
        o[t][3] = x[4 + t][3] * (fq.y * s1);
      }
    }
    // the largest magnitudes of the two rows of a [16][32] accumulator
    auto largest = [&](const float (&w)[4][4], uint32_t &m0, uint32_t &m1) {
      m0 = m1 = 0;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        m0 = max(m0, max(mag(w[t][0]), mag(w[t][1])));
        m1 = max(m1, max(mag(w[t][2]), mag(w[t][3])));
      }
    };
    // whether all of it can be split
    auto fits = [&](const float (&w)[4][4]) {
      uint32_t m0, m1;
      largest(w, m0, m1);
      return !__any_sync(0xFFFFFFFFu, max(m0, m1) >= kNoBf16);
    };
    auto split = [&](const float (&w)[4][4], uint32_t (&a)[2][3][4]) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float *x = &w[2 * ks + (i >> 1)][2 * (i & 1)];
          split3(x[0], x[1], a[ks][0][i], a[ks][1][i], a[ks][2][i]);
        }
    };
    // w (16 x 32) times a lower triangular square tile's transpose
    auto times_tile = [&](const uint32_t (&a)[2][3][4], uint32_t tile, float (&w)[4][4]) {
      uint32_t b[3][4][2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t at = tile + off_b + p * 16 * 128;
        load2<false>(b[0][2 * p], b[0][2 * p + 1], at);
        load2<false>(b[1][2 * p], b[1][2 * p + 1], at ^ 64);
        load2<false>(b[2][2 * p], b[2][2 * p + 1], tile + kBlock + off_lo + p * 16 * 64);
      }
      mma6<true>(w, a[0], b);
      // the first 16 rows end with their diagonal
      float (&lower)[2][4] = *reinterpret_cast<float(*)[2][4]>(&w[2]);
      uint32_t b2[3][2][2];
      const uint32_t at = ((tile + off_b) ^ 32) + 16 * 128;
      load2<false>(b2[0][0], b2[0][1], at);
      load2<false>(b2[1][0], b2[1][1], at ^ 64);
      load2<false>(b2[2][0], b2[2][1], ((tile + kBlock + off_lo) ^ 32) + 16 * 64);
      mma6<false>(lower, a[1], b2);
    };
    float u[4][4];
    {
      odd = f->odd || !fits(v);
      if (!odd) {
        uint32_t a3[2][3][4];
        split(v, a3);
        times_tile(a3, tt, u);
        float w[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float2 x = *reinterpret_cast<const float2 *>(f->wk + 8 * t + 2 * q4);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[t][e] = max_nan(fabsf(u[t][e]), fabsf(u[t][e] * (e & 1 ? x.y : x.x)));
        }
        odd = !fits(w);
      }
      if (!odd) {
        uint32_t a3[2][3][4];
        split(u, a3);
        float w[4][4];
        times_tile(a3, at, w);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[t][e] += w[t][e];
        float *p = onext;
        const int left_over = n - c * C - 2 * q4;
#pragma unroll
        for (int t = 0; t < 4; ++t, p += 8 * a.d.out_stride) {
          if (8 * t < left_over) p[0] = o[t][0], p[8] = o[t][2];
          if (8 * t + 1 < left_over) p[a.d.out_stride] = o[t][1], p[a.d.out_stride + 8] = o[t][3];
        }
      }
    }
    if (!odd) {
      if (c + 1 < chunks) load_v(c + 1, v);
      // S^T <- e^{G_C} S^T + (U^T diag(e^{G_C - G})) K
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float2 x = *reinterpret_cast<const float2 *>(f->wk + 8 * t + 2 * q4);
        u[t][0] *= x.x;
        u[t][1] *= x.y;
        u[t][2] *= x.x;
        u[t][3] *= x.y;
      }
      uint32_t m0, m1;
      largest(u, m0, m1);
      m0 = max(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, 1));
      m1 = max(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, 1));
      m0 = max(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, 2));
      m1 = max(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, 2));
      float s0, i0, s1, i1;
      row_scale(m0, s0, i0);
      row_scale(m1, s1, i1);
      uint32_t ah[2][4], al[2][4];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float *x = &u[2 * ks + (i >> 1)][2 * (i & 1)];
          split2(x[0], x[1], i & 1 ? i1 : i0, ah[ks][i], al[ks][i]);
        }
      const float dec = f->dec;
#pragma unroll
      for (int c4 = 0; c4 < DK / 8; c4 += 4) {
        float w[4][4];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          uint32_t bh[4][2], bl[4][2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t at = ((kt + off_t) ^ (((c4 + 2 * p) & 7) << 4)) + (c4 >> 3) * 2 * kBlock + ks * 16 * 128;
            load2<true>(bh[2 * p], bh[2 * p + 1], at);
            load2<true>(bl[2 * p], bl[2 * p + 1], at + LO);
          }
          if (ks == 0) mma3<true>(w, ah[ks], al[ks], bh, bl);
          else mma3<false>(w, ah[ks], al[ks], bh, bl);
        }
        // not on the packed unit: it counts denormal states as zero
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          s[c4 + t][0] = fmaf(s0, w[t][0], dec * s[c4 + t][0]);
          s[c4 + t][1] = fmaf(s0, w[t][1], dec * s[c4 + t][1]);
          s[c4 + t][2] = fmaf(s1, w[t][2], dec * s[c4 + t][2]);
          s[c4 + t][3] = fmaf(s1, w[t][3], dec * s[c4 + t][3]);
        }
      }
    } else {
      // an infinite or NaN value among these tokens or their updates: one after another, so that none reaches an earlier one
      const int len = min(C, n - c * C);
      const unsigned char *tile = ring + st * kStage;
      for (int j = 0; j < len; ++j) {
        const float al = f->alpha[j], be = f->beta[j], sk = f->sk[j], sq = f->sq[j];
        auto both = [&](int ct, float2 &k, float2 &q) {
          const uint32_t off = kq_at(j, ct) + 4 * q4;
          const uint32_t kh = *reinterpret_cast<const uint32_t *>(tile + off);
          const uint32_t kl = *reinterpret_cast<const uint32_t *>(tile + LO + off);
          const uint32_t qh = *reinterpret_cast<const uint32_t *>(tile + kBlock + off);
          const uint32_t ql = *reinterpret_cast<const uint32_t *>(tile + kBlock + LO + off);
          k = make_float2(sk * (lo16<false>(kh) + lo16<false>(kl)), sk * (hi16<false>(kh) + hi16<false>(kl)));
          q = make_float2(sq * (lo16<false>(qh) + lo16<false>(ql)), sq * (hi16<false>(qh) + hi16<false>(ql)));
        };
        float x0 = 0.f, x1 = 0.f, y0 = 0.f, y1 = 0.f, z = 0.f;
#pragma unroll
        for (int ct = 0; ct < DK / 8; ++ct) {
          float2 k, q;
          both(ct, k, q);
          x0 = fmaf(s[ct][0], k.x, fmaf(s[ct][1], k.y, x0));
          x1 = fmaf(s[ct][2], k.x, fmaf(s[ct][3], k.y, x1));
          y0 = fmaf(s[ct][0], q.x, fmaf(s[ct][1], q.y, y0));
          y1 = fmaf(s[ct][2], q.x, fmaf(s[ct][3], q.y, y1));
          z = fmaf(k.x, q.x, fmaf(k.y, q.y, z));
        }
#pragma unroll
        for (int m = 1; m <= 2; m <<= 1) {
          x0 += __shfl_xor_sync(0xFFFFFFFFu, x0, m);
          x1 += __shfl_xor_sync(0xFFFFFFFFu, x1, m);
          y0 += __shfl_xor_sync(0xFFFFFFFFu, y0, m);
          y1 += __shfl_xor_sync(0xFFFFFFFFu, y1, m);
          z += __shfl_xor_sync(0xFFFFFFFFu, z, m);
        }
        const long long row = t00 + c * C + j;
        const float u0 = be * (__ldg(vp + row * a.d.v_stride) - al * x0);
        const float u1 = be * (__ldg(vp + row * a.d.v_stride + 8) - al * x1);
        if (q4 == 0) {
          op[row * a.d.out_stride] = fmaf(z, u0, al * y0);
          op[row * a.d.out_stride + 8] = fmaf(z, u1, al * y1);
        }
#pragma unroll
        for (int ct = 0; ct < DK / 8; ++ct) {
          float2 k, q;
          both(ct, k, q);
          s[ct][0] = fmaf(k.x, u0, al * s[ct][0]);
          s[ct][1] = fmaf(k.y, u0, al * s[ct][1]);
          s[ct][2] = fmaf(k.x, u1, al * s[ct][2]);
          s[ct][3] = fmaf(k.y, u1, al * s[ct][3]);
        }
      }
      if (c + 1 < chunks) load_v(c + 1, v);
    }
    onext += C * a.d.out_stride;
    __syncwarp();
    if (lane == 0) {
      __threadfence_block();
      if (atomicAdd(&left[st], 1) == W - 1) {
        left[st] = 0;
        __threadfence_block();
        if (c + NST < chunks) ask(c + NST);
      }
    }
  }

  if (a.d.state_out) {
    const int to = __ldg(a.d.state_out + b);
    if (to >= 0 && to < a.d.n_slots) {
      float *p = a.d.states + to * a.d.slot_stride + static_cast<long long>(h) * DK * a.d.Dv + (d0 - h * a.d.Dv);
#pragma unroll
      for (int ct = 0; ct < DK / 8; ++ct)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[static_cast<long long>(8 * ct + 2 * q4 + (e & 1)) * a.d.Dv + 8 * (e >> 1)] = s[ct][e];
    } else if (to != -1 && teller) {
      atomicOr(&g_qg_status_delta_chunk, QG_STATUS_BIT_ID);
    }
  }
}

// ---- the walk with a head to an SM ---------------------------------------------------------------------
// For heads of whole 128 columns: a CTA walks 128 columns of a head's state on tcgen05.  Row d of every product is column d of
// the state, so a lane of tensor memory is one column and its thread works alone: the state stays in registers (two threads
// a column, half of its rows each), left operands go to tensor memory as f16 pairs (hi in one range of columns, lo in
// another), right operands are the tiles in shared memory, with K read as it lies for S0^T K^T and turned for U^T K.
//   both groups  S^T in two terms (each half of its rows); R = V - ... and U, in three terms, and W, U with the decays to the
//                chunk's end, in two (each half of the tokens); the outputs of the chunk before; S^T <- e^{G_C} S^T + D
//   a producer   bulk copies into the ring (a row of values each lane: that would hold control up by 1700 cycles)
//   control      the products X = S^T K^T, O = S^T Q^T, U = R T^T, D = W K, O2 = U A^T
// Every wait ends with its phase or after kTcWaitCycles, which makes the CTA give up.
// The chain of a chunk bounds it, 5800 cycles or 3.1 us where its products alone are 3400: state in two terms 740, X and meanwhile the
// outputs of the chunk before 2050, R 450, U 550, W 510 and U's terms 290, D 750, the state's update 480 (stamps in a copy of the build; five
// prompts of 30042 tokens in all, the longest of 7842: 761 us; the tensor cores' pipe is busy 26 % of a head's time).
constexpr int kTcThreads = 384;                    // two groups of four warps, control, the producer and two idle warps
constexpr int kTcRegs = 168, kTcRegsWork = 208, kTcRegsRest = 88;
static_assert(2 * kTcRegsWork + kTcRegsRest <= 3 * kTcRegs, "the warpgroups' shares come from the launch's total");
constexpr int kTcStages = 3;
constexpr long long kTcWaitCycles = 1LL << 29;  // a quarter of a second: a wait is for microseconds
constexpr int kOrder = 128;  // sequences that are put in order, longest first
// columns of tensor memory
// X and O are in two places by the chunk's parity, since O is read while the next is made.  They are two products: 32 columns
// take 41 cycles a step and 64 take 70, and only X is waited for.  R's terms make way for U's, which are written once R's product is
// done, and U's sums for W's terms: each half of the tokens has its hi and lo terms where it has read its sums.
enum { TXO = 0, TU = 128, TO2 = 160, TD = 192, TS = 320, TR = 448, TUA = 448, TW = TU };

template <int DK>
struct TcSmem {
  static constexpr int kV = Tiles<DK>::kKQAll + kTA;  // where a stage's values are: [32][128] f32
  static constexpr int kStage = (kV + C * 512 + 1023) / 1024 * 1024;
  static constexpr int kBytes = kTcStages * kStage + 1024;
};
struct TcShared {
  uint64_t full[kTcStages], empty[kTcStages];           // by the copies, and by control
  uint64_t s_ready, r_ready, u_ready, w_ready, o_free;  // by the working warps
  uint64_t x_done, u_done, d_done, o_done;              // by the tensor cores
  uint32_t tmem;
  int abort, seq;
  int odd_chunk, u_odd;     // the last chunk that goes token by token; the last one whose updates say that it must
  float smax[2][128];       // largest of a column's halves
  float wmax[2][128];       // the same of W: halves of the tokens
  __align__(16) float4 ex[2][2][128];  // token by token: partial products of the halves, by the token's parity
};

// D = (A hi + A lo) (B hi + B lo) without lo lo, the small products first.  A: 8 columns of tensor memory a step, STEP from one to
// the next; B: the descriptor of its hi tile, lo LO bytes behind it; KROWS: the tile's rows are columns of the product, 16 elements of
// each a step; TURNED: 16 rows a step.  Unrolled, with nothing but sums of constants between the instructions: a loop that
// makes each descriptor took 70 cycles a product.
enum { KROWS, TURNED };
template <int KIND, int STEPS, int LO, int STEP = 8>
QG_DEVICE void product(uint32_t el, uint32_t d, uint32_t a_hi, uint32_t a_lo, uint64_t b, uint32_t id) {
#pragma unroll
  for (int term = 0; term < 3; ++term)
#pragma unroll
    for (int ks = 0; ks < STEPS; ++ks) {
      const int off = (KIND == TURNED ? ks * 16 * 128 : (ks >> 2) * 2 * kBlock + (ks & 3) * 32) + (term == 1 ? LO : 0);
      tc_mma_ta_el(el, d, (term == 0 ? a_lo : a_hi) + STEP * ks, b + (off >> 4), id, term || ks);
    }
}
// D = A B of three terms each, without the three smallest products: 32 tokens.  A: 16 columns a term; B: its hi and mid terms, its lo
QG_DEVICE void product3(uint32_t el, uint32_t d, uint32_t a, uint64_t b, uint64_t b_lo, uint32_t id) {
  constexpr int kA[6] = {2, 0, 1, 1, 0, 0}, kB[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
  for (int i = 0; i < 6; ++i)
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
      tc_mma_ta_el(el, d, a + 16 * kA[i] + 8 * ks, (kB[i] == 2 ? b_lo : b + (64 * kB[i] >> 4)) + (32 * ks >> 4), id, i || ks);
}

template <int DK>
__global__ void __launch_bounds__(kTcThreads, 1) delta_walk_tc_kernel(const ChunkArgs a) {
  extern __shared__ unsigned char ring_raw[];
  __shared__ TcShared sh;
  constexpr int LO = Tiles<DK>::kLo, kStage = TcSmem<DK>::kStage;
  constexpr int HK = DK / 2;  // rows of the state a thread holds
  unsigned char *ring = ring_raw + ((1024u - (smem_u32(ring_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int parts = a.d.Dv / 128, per_seq = a.d.Hv * parts;
  const int part = static_cast<int>(blockIdx.x) % parts, h = static_cast<int>(blockIdx.x) / parts % a.d.Hv;
  const int place = static_cast<int>(blockIdx.x) / per_seq;
  pdl_wait();
  pdl_launch_dependents();
  auto length = [&](int i) { return qg::delta_tok(a.d, i + 1) - qg::delta_tok(a.d, i); };
  // the longest sequences first: theirs is the longest chain of chunks
  if (tid == 0) sh.seq = place;
  __syncthreads();
  if (a.d.B > 1 && a.d.B <= kOrder && tid < a.d.B) {
    const int mine = length(tid);
    int rank = 0;
    for (int i = 0; i < a.d.B; ++i) {
      const int l = length(i);
      rank += l > mine || (l == mine && i < tid);
    }
    if (rank == place) sh.seq = tid;
  }
  __syncthreads();
  const int b = sh.seq;
  const int t00 = qg::delta_tok(a.d, b), n = length(b);
  if (n < a.first_len || n <= 0) return;
  const int chunks = (n + C - 1) / C, slot0 = chunk_base(a.d, b), hk = qg::delta_key_head(a.d, h);
  if (slot0 + chunks > a.slots) return;

  if (tid == 0) {
    for (int i = 0; i < kTcStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.s_ready, 8);
    mbar_init(&sh.r_ready, 8);
    mbar_init(&sh.u_ready, 8);
    mbar_init(&sh.w_ready, 8);
    mbar_init(&sh.o_free, 8);
    mbar_init(&sh.x_done, 1);
    mbar_init(&sh.u_done, 1);
    mbar_init(&sh.d_done, 1);
    mbar_init(&sh.o_done, 1);
    fence_mbar_init();
    sh.abort = 0;
    sh.odd_chunk = sh.u_odd = -1;
  }
  if (warp == 8) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sh.tmem;
  volatile int *const abort_flag = &sh.abort;
  auto wait = [&](uint64_t *bar, uint32_t parity) {  // the whole warp, and gives up as a whole
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
      const long long start = clock64();  // the SM's own clock: the global timer takes a microsecond to read
      while (!(ok = mbar_try_wait(bar, parity))) {
        if (*abort_flag) break;
        if (clock64() - start > kTcWaitCycles) {
          *abort_flag = 1;
          atomicOr(&g_qg_status_delta_chunk, QG_STATUS_BIT_TIMEOUT);
          break;
        }
      }
    }
    return __all_sync(0xFFFFFFFFu, ok);
  };
  auto factors = [&](int c) { return reinterpret_cast<const Factors *>(ring + (c % kTcStages) * kStage + Tiles<DK>::kKQAll + 2 * kThree); };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcRegsRest));
    if (warp == 9) {
      auto ask = [&](int c) {  // a lane asks for a token's values
        unsigned char *dst = ring + (c % kTcStages) * kStage;
        uint64_t *bar = &sh.full[c % kTcStages];
        const int rows = min(C, n - c * C);
        if (lane == 0) mbar_arrive_expect_tx(bar, Tiles<DK>::kKQAll + kTA + 512 * rows);
        __syncwarp();
        if (lane < rows)
          bulk_g2s(dst + TcSmem<DK>::kV + 512 * lane,
                   a.d.v + (t00 + static_cast<long long>(c) * C + lane) * a.d.v_stride + h * a.d.Dv + part * 128, 512, bar);
        if (lane == 0) {
          bulk_g2s(dst, a.kq + (static_cast<size_t>(slot0 + c) * a.d.Hk + hk) * Tiles<DK>::kKQAll, Tiles<DK>::kKQAll, bar);
          bulk_g2s(dst + Tiles<DK>::kKQAll, a.ta + (static_cast<size_t>(slot0 + c) * a.d.Hv + h) * kTA, kTA, bar);
        }
        __syncwarp();
      };
      asm volatile("fence.proxy.async;" ::: "memory");  // the tiles were written by plain stores
      int c = 0;
      for (; c < chunks; ++c) {
        if (c >= kTcStages && !wait(&sh.empty[c % kTcStages], (c / kTcStages - 1) & 1)) break;
        ask(c);
      }
      if (c < chunks)  // copies still under way land before the CTA ends
        for (int i = max(0, c - kTcStages); i < c; ++i) cleanup_wait(&sh.full[i % kTcStages], (i / kTcStages) & 1);
    } else if (warp == 8) {
      const uint32_t el = elect_lane();
      constexpr uint32_t id32 = make_idesc16(128, 32, false, false), idk = make_idesc16(128, DK, false, true);
      constexpr uint32_t id3 = make_idesc16(128, 32, true, false);
      // what the right operands' descriptors say beside the address
      const uint64_t rows0 = sw128_desc(0), turned0 = sw128_desc_mn(0, 2 * kBlock), lo0 = sw64_desc(0);
      uint32_t n_r = 0, n_o = 0;  // phases of r_ready (u_ready, w_ready) and of o_free
      bool before_odd = true;     // no output to be read of a chunk before
      bool ok = true;
      for (int c = 0; c < chunks && ok; ++c) {
        const int st = c % kTcStages;
        ok = wait(&sh.s_ready, c & 1) && wait(&sh.full[st], (c / kTcStages) & 1);
        if (!ok) break;
        const uint32_t kt = smem_u32(ring + st * kStage), tt = kt + Tiles<DK>::kKQAll;
        const uint64_t kd = rows0 + (kt >> 4), kturned = turned0 + (kt >> 4);
        const bool odd = factors(c)->odd;
        tc_fence_after();
        if (!odd) {
          product<KROWS, DK / 16, LO>(el, tm + TXO + 64 * (c & 1), tm + TS, tm + TS + DK / 2, kd, id32);
          tc_commit_el(el, &sh.x_done);
          product<KROWS, DK / 16, LO>(el, tm + TXO + 64 * (c & 1) + 32, tm + TS, tm + TS + DK / 2, kd + (kBlock >> 4), id32);
        } else if (el) {
          sh.odd_chunk = c;
          __threadfence_block();
          mbar_arrive(&sh.x_done);
          mbar_arrive(&sh.d_done);
        }
        __syncwarp();
        if (odd) {
          if (!before_odd && !(ok = wait(&sh.o_free, n_o++ & 1))) break;
          if (c > 0 && el) mbar_arrive(&sh.empty[(c - 1) % kTcStages]);
          before_odd = true;
          continue;
        }
        if (!(ok = wait(&sh.r_ready, n_r & 1))) break;
        tc_fence_after();
        product3(el, tm + TU, tm + TR, rows0 + (tt >> 4), lo0 + ((tt + kBlock) >> 4), id3);
        tc_commit_el(el, &sh.u_done);
        if (!(ok = wait(&sh.w_ready, n_r & 1))) break;
        tc_fence_after();
        const bool late = *reinterpret_cast<volatile int *>(&sh.u_odd) == c;
        if (!late) {
          product<TURNED, 2, LO, 16>(el, tm + TD, tm + TW, tm + TW + 8, kturned, idk);
          tc_commit_el(el, &sh.d_done);
        }
        // everyone has left the chunk before, and its outputs have been read
        if (!before_odd && !(ok = wait(&sh.o_free, n_o++ & 1))) break;
        if (c > 0 && el) mbar_arrive(&sh.empty[(c - 1) % kTcStages]);
        before_odd = late;
        if (!(ok = wait(&sh.u_ready, n_r & 1))) break;
        ++n_r;
        tc_fence_after();
        if (!late) {
          product3(el, tm + TO2, tm + TUA, rows0 + ((tt + kThree) >> 4), lo0 + ((tt + kThree + kBlock) >> 4), id3);
          tc_commit_el(el, &sh.o_done);
        } else if (el) {  // U's product is done, and with it those before it: nobody reads or writes tensor memory now
          sh.odd_chunk = c;
          __threadfence_block();
          mbar_arrive(&sh.d_done);
          mbar_arrive(&sh.o_done);
        }
        __syncwarp();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcRegsWork));
    const int group = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tm + (static_cast<uint32_t>(warp & 3) << 21);  // this warp's lanes of tensor memory
    const int d0 = h * a.d.Dv + part * 128 + row;
    const bool teller = tid == 0 && part == 0 && h == 0;
    float s[HK];  // rows group * HK and on of column d0
    const long long state_at = (static_cast<long long>(h) * DK + group * HK) * a.d.Dv + part * 128 + row;
    {
      const int in = a.d.state_in ? __ldg(a.d.state_in + b) : -1;
      if (teller && (in < -1 || in >= a.d.n_slots)) atomicOr(&g_qg_status_delta_chunk, QG_STATUS_BIT_ID);
      const bool have = in >= 0 && in < a.d.n_slots;
      const float *p = a.d.states + (have ? in : 0) * a.d.slot_stride + state_at;
#pragma unroll
      for (int i = 0; i < HK; ++i) s[i] = have ? p[static_cast<long long>(i) * a.d.Dv] : 0.f;
    }
    const float *vp = a.d.v + static_cast<long long>(t00) * a.d.v_stride + d0;
    float *op = a.d.out + static_cast<long long>(t00) * a.d.out_stride + d0;
    // a chunk's values of this column, 0 behind the last token.  They come with the tiles: loads of the working warps would
    // be waited for together with the next barrier or tensor-memory load (4.3 microseconds a chunk)
    auto value = [&](int c, int j) {
      const float *p = reinterpret_cast<const float *>(ring + (c % kTcStages) * kStage + TcSmem<DK>::kV);
      return c * C + j < n ? p[j * 128 + row] : 0.f;
    };
    // this half's 16 tokens in three terms to its 8 columns of each
    constexpr int H = C / 2;
    const int j0 = group * H;
    auto put = [&](const float (&w)[H], uint32_t col) {
      uint32_t hi[H / 2], mid[H / 2], lo[H / 2];
#pragma unroll
      for (int j = 0; j < H; j += 2) split3(w[j], w[j + 1], hi[j / 2], mid[j / 2], lo[j / 2]);
      tmem_st8(lanes + col + 8 * group, hi);
      tmem_st8(lanes + col + 16 + 8 * group, mid);
      tmem_st8(lanes + col + 32 + 8 * group, lo);
    };
    auto tell = [&](uint64_t *bar) {  // what this warp has put into, or taken from, tensor memory
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto largest = [&] {
      float m4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < HK; ++i) m4[i & 3] = max_nan(m4[i & 3], fabsf(s[i]));
      return max_nan(max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3]));
    };
    float m = largest();
    float scale_s = 1.f, scale_before = 1.f, largest_s = 0.f;
    uint32_t n_u = 0;      // phases of u_done and o_done
    bool pending = false;  // outputs of the chunk before wait to be written
    auto outputs = [&](int c, float ss) {  // ss: the state's scale then
      if (!wait(&sh.o_done, (n_u - 1) & 1)) return false;
      tc_fence_after();
      const Factors *f = factors(c);
      float *p = op + (static_cast<long long>(c) * C + j0) * a.d.out_stride;
      const int left = n - c * C - j0;
      float x[H], y[H];
      tmem_ld16(lanes + TXO + 64 * (c & 1) + 32 + j0, x);
      tmem_ld16(lanes + TO2 + j0, y);
#pragma unroll
      for (int j = 0; j < H; j += 4) {
        const float4 fq = *reinterpret_cast<const float4 *>(f->fq + j0 + j);
        x[j] = fmaf(fq.x * ss, x[j], y[j]);
        x[j + 1] = fmaf(fq.y * ss, x[j + 1], y[j + 1]);
        x[j + 2] = fmaf(fq.z * ss, x[j + 2], y[j + 2]);
        x[j + 3] = fmaf(fq.w * ss, x[j + 3], y[j + 3]);
      }
#pragma unroll
      for (int j = 0; j < H; ++j) asm volatile("" : "+f"(x[j]));  // the factors are read before the stage is given up
      tell(&sh.o_free);
#pragma unroll
      for (int j = 0; j < H; ++j, p += a.d.out_stride)
        if (j < left) *p = x[j];
      return true;
    };

    int c = 0;
    for (; c < chunks; ++c) {
      // ---- the state in two terms
      {
        sh.smax[group][row] = m;
        named_bar_sync(1, 256);
        scale_before = scale_s;
        float inv;
        largest_s = max_nan(m, sh.smax[group ^ 1][row]);
        row_scale(mag(largest_s), scale_s, inv);
#pragma unroll
        for (int i = 0; i < HK; i += 32) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) split2(s[i + j], s[i + j + 1], inv, hi[j / 2], lo[j / 2]);
          tmem_st16(lanes + TS + (group * HK + i) / 2, hi);
          tmem_st16(lanes + TS + DK / 2 + (group * HK + i) / 2, lo);
        }
        tmem_st_wait();
        tell(&sh.s_ready);
      }
      const Factors *f = factors(c);
      if (!wait(&sh.full[c % kTcStages], (c / kTcStages) & 1)) break;
      // while the product runs: this half's values, and the outputs of the chunk before
      float x[H], w[H];
#pragma unroll
      for (int j = 0; j < H; ++j) w[j] = value(c, j0 + j);
#pragma unroll
      for (int j = 0; j < H; ++j) asm volatile("" : "+f"(w[j]));
      if (pending && !outputs(c - 1, scale_before)) break;
      pending = false;
      if (!wait(&sh.x_done, c & 1)) break;
      const float dec = f->dec;
      float scale_w = 1.f;
      auto by_token = [&] { return *reinterpret_cast<volatile int *>(&sh.odd_chunk) == c; };
      if (!by_token()) {
        tc_fence_after();
        tmem_ld16(lanes + TXO + 64 * (c & 1) + j0, x);
#pragma unroll
        for (int j = 0; j < H; j += 4) {
          const float4 fk = *reinterpret_cast<const float4 *>(f->fk + j0 + j);
          x[j] = fmaf(-fk.x * scale_s, x[j], w[j]);
          x[j + 1] = fmaf(-fk.y * scale_s, x[j + 1], w[j + 1]);
          x[j + 2] = fmaf(-fk.z * scale_s, x[j + 2], w[j + 2]);
          x[j + 3] = fmaf(-fk.w * scale_s, x[j + 3], w[j + 3]);
        }
        put(x, TR);
        tmem_st_wait();
        tell(&sh.r_ready);
        if (!wait(&sh.u_done, n_u & 1)) break;
        tc_fence_after();
        tmem_ld16(lanes + TU + j0, x);
        float big = 0.f, big_u = 0.f;
#pragma unroll
        for (int j = 0; j < H; ++j) big_u = max_nan(big_u, fabsf(x[j]));
#pragma unroll
        for (int j = 0; j < H; j += 4) {
          const float4 wk = *reinterpret_cast<const float4 *>(f->wk + j0 + j);
          w[j] = x[j] * wk.x;
          w[j + 1] = x[j + 1] * wk.y;
          w[j + 2] = x[j + 2] * wk.z;
          w[j + 3] = x[j + 3] * wk.w;
          big = fmaxf(fmaxf(big, fmaxf(fabsf(w[j]), fabsf(w[j + 1]))), fmaxf(fabsf(w[j + 2]), fabsf(w[j + 3])));
        }
        // infinite or NaN (a zero of T times an infinite R is): the chunk goes token by token.  Not where the column's state is
        // that already: then every token's output is
        if (largest_s < INFINITY && !(big_u < kMost && big < kMost)) sh.u_odd = c;
        sh.wmax[group][row] = big;
        named_bar_sync(2 + (warp & 3), 64);  // with the warp that has these columns' other tokens
        float inv_w;
        row_scale(mag(fmaxf(big, sh.wmax[group ^ 1][row])), scale_w, inv_w);
        {
          uint32_t hi[H / 2], lo[H / 2];
#pragma unroll
          for (int j = 0; j < H; j += 2) split2(w[j], w[j + 1], inv_w, hi[j / 2], lo[j / 2]);
          tmem_st8(lanes + TW + 16 * group, hi);
          tmem_st8(lanes + TW + 16 * group + 8, lo);
        }
        tmem_st_wait();
        tell(&sh.w_ready);
        put(x, TUA);
        tmem_st_wait();
        tell(&sh.u_ready);
        ++n_u;
        if (!wait(&sh.d_done, c & 1)) break;
      } else if (!wait(&sh.d_done, c & 1)) {
        break;
      }
      if (!by_token()) {
        tc_fence_after();
        float m4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < HK; i += 32) {
          float d[32];
          tmem_ld32_nowait(lanes + TD + group * HK + i, d);
          tmem_ld_wait(d);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const f2 y = fma2(mk2(scale_w, scale_w), mk2(d[j], d[j + 1]), mul2(mk2(dec, dec), mk2(s[i + j], s[i + j + 1])));
            s[i + j] = y.x;
            s[i + j + 1] = y.y;
            m4[(j >> 1) & 3] = max_nan(m4[(j >> 1) & 3], max_nan(fabsf(y.x), fabsf(y.y)));
          }
        }
        m = max_nan(max_nan(m4[0], m4[1]), max_nan(m4[2], m4[3]));
        tc_fence_before();
        pending = true;
        continue;
      }
      // ---- token by token: an infinite or NaN value must not reach an earlier one.  The state is still the one before the chunk
      const int len = min(C, n - c * C);
      const unsigned char *tile = ring + (c % kTcStages) * kStage;
      bool gone = false;
      for (int j = 0; j < len; ++j) {
        const float al = f->alpha[j], be = f->beta[j], sk = f->sk[j], sq = f->sq[j];
        auto pair = [&](int i, float2 &k, float2 &q) {  // rows i and i + 1 of this thread's half
          const uint32_t off = kq_at(j, (group * HK + i) >> 3) + (i & 7) * 2;
          const uint32_t kh = *reinterpret_cast<const uint32_t *>(tile + off);
          const uint32_t kl = *reinterpret_cast<const uint32_t *>(tile + LO + off);
          const uint32_t qh = *reinterpret_cast<const uint32_t *>(tile + kBlock + off);
          const uint32_t ql = *reinterpret_cast<const uint32_t *>(tile + kBlock + LO + off);
          k = make_float2(sk * (lo16<false>(kh) + lo16<false>(kl)), sk * (hi16<false>(kh) + hi16<false>(kl)));
          q = make_float2(sq * (lo16<false>(qh) + lo16<false>(ql)), sq * (hi16<false>(qh) + hi16<false>(ql)));
        };
        float x = 0.f, y = 0.f, z = 0.f;
#pragma unroll
        for (int i = 0; i < HK; i += 2) {
          float2 k, q;
          pair(i, k, q);
          x = fmaf(s[i], k.x, fmaf(s[i + 1], k.y, x));
          y = fmaf(s[i], q.x, fmaf(s[i + 1], q.y, y));
          z = fmaf(k.x, q.x, fmaf(k.y, q.y, z));
        }
        sh.ex[j & 1][group][row] = make_float4(x, y, z, 0.f);
        named_bar_sync(1, 256);
        gone = __any_sync(0xFFFFFFFFu, *abort_flag != 0);
        if (gone) break;
        const float4 other = sh.ex[j & 1][group ^ 1][row];
        const long long t = static_cast<long long>(c) * C + j;
        const float u = be * (__ldg(vp + t * a.d.v_stride) - al * (x + other.x));
        if (group == 0) op[t * a.d.out_stride] = fmaf(z + other.z, u, al * (y + other.y));
#pragma unroll
        for (int i = 0; i < HK; i += 2) {
          float2 k, q;
          pair(i, k, q);
          s[i] = fmaf(k.x, u, al * s[i]);
          s[i + 1] = fmaf(k.y, u, al * s[i + 1]);
        }
      }
      if (gone) break;
      m = largest();
    }
    // a warp that gave up does not keep the others at the barriers that they may be at; behind them they see that it did (nothing
    // that they wait for next comes without this warp)
    if (c < chunks) {
      asm volatile("bar.arrive 1, 256;" ::: "memory");
      asm volatile("bar.arrive %0, 64;" ::"r"(2 + (warp & 3)) : "memory");
    }
    if (c == chunks && pending) outputs(chunks - 1, scale_s);
    if (c == chunks && a.d.state_out) {
      const int to = __ldg(a.d.state_out + b);
      if (to >= 0 && to < a.d.n_slots) {
        float *p = a.d.states + to * a.d.slot_stride + state_at;
#pragma unroll
        for (int i = 0; i < HK; ++i) p[static_cast<long long>(i) * a.d.Dv] = s[i];
      } else if (to != -1 && teller) {
        atomicOr(&g_qg_status_delta_chunk, QG_STATUS_BIT_ID);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(sh.tmem, 512);
}

template <int DK, int W, int NST>
cudaError_t walk(const ChunkArgs &a, cudaStream_t s) {
  constexpr int smem = WalkSmem<DK, W, NST>::kBytes;
  if (!qg::set_smem_attr(reinterpret_cast<const void *>(delta_walk_kernel<DK, W, NST>), smem)) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(a.d.B) * a.d.Hv * (a.d.Dv / (16 * W)));
  return qg::launch_pdl(delta_walk_kernel<DK, W, NST>, grid, dim3(W * 32), smem, s, a);
}

template <int DK>
cudaError_t both(const ChunkArgs &a, cudaStream_t s) {
  constexpr int smem = std::max(Tiles<DK>::kKQAll, kPrepWarps * kThree);
  static_assert(C * kTurn * 4 <= kThree, "T is turned in a warp's room");
  if (!qg::set_smem_attr(reinterpret_cast<const void *>(delta_prep_kernel<DK>), smem)) return cudaErrorInvalidValue;
  cudaError_t e = qg::launch_pdl(delta_prep_kernel<DK>, dim3(static_cast<unsigned>(a.slots) * a.d.Hk), dim3(kPrepWarps * 32), smem, s, a);
  if (e != cudaSuccess) return e;
  // a build of other registers than the split's goes the other way, which takes every width
  static const bool fits = qg::split_fits(reinterpret_cast<const void *>(delta_walk_tc_kernel<DK>), kTcRegs);
  if (a.d.Dv % 128 == 0 && fits) {
    constexpr int tc = TcSmem<DK>::kBytes;
    if (!qg::set_smem_attr(reinterpret_cast<const void *>(delta_walk_tc_kernel<DK>), tc)) return cudaErrorInvalidValue;
    return qg::launch_pdl(delta_walk_tc_kernel<DK>, dim3(static_cast<unsigned>(a.d.B) * a.d.Hv * (a.d.Dv / 128)), dim3(kTcThreads), tc, s, a);
  }
  return a.d.Dv % 64 == 0 ? walk<DK, 4, 2>(a, s) : walk<DK, 2, 2>(a, s);
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
int chunk_slots(const DeltaArgs &a) { return a.T / C + a.B; }
size_t kq_bytes(const DeltaArgs &a) { return static_cast<size_t>(chunk_slots(a)) * a.Hk * 4 * C * a.Dk * 2; }

}  // namespace

namespace qg {

size_t delta_chunk_workspace(const DeltaArgs &a) {
  return round256(kq_bytes(a)) + static_cast<size_t>(chunk_slots(a)) * a.Hv * kTA;
}

cudaError_t delta_chunks(const DeltaArgs &d, int first_len, void *ws, cudaStream_t s) {
  unsigned char *p = static_cast<unsigned char *>(ws);
  const ChunkArgs a{d, p, p + round256(kq_bytes(d)), first_len, chunk_slots(d)};
  g_launched = true;
  return d.Dk == 64 ? both<64>(a, s) : both<128>(a, s);
}

unsigned int read_status_delta_chunk(bool clear) {
  unsigned int v = 0;
  if (!g_launched) return v;
  if (cudaMemcpyFromSymbol(&v, g_qg_status_delta_chunk, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_qg_status_delta_chunk, &z, sizeof(z));
  }
  return v;
}

}  // namespace qg
