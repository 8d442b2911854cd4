// qg_attn.cu -- causal attention over the paged cache: the kernel for few rows per segment (a
// decode step's tokens), the kernel that joins the pieces of a row, and the entry points.
//
// o = sum_j p_j V_j / sum_j p_j with p_j = 2^(c q.K_j - m), m from the running maximum, in one pass
// over the keys.  A decode step reads every cached row once and does 4 operations per cached value
// and query head, far below the tensor cores' rate, so HBM bounds it: the design keeps
// asynchronous copies in flight on every SM and spends few instructions per byte.
//
// Measured (one GB300, calls replayed from a graph; floor: bytes at the measured copy bandwidth):
//   64 ragged sequences of up to 8191 tokens, 8 cached heads of 128, bf16   199 us, floor 177 (the kernel
//     alone 191: 6.3 TB/s, 93 % of the copy)
//   one sequence of 4097 tokens, f16 cache, f32 output                      16.9 us, floor 2.5: two
//     launches whose fixed parts (the scan, the look-ups, cold code) take most of it
#include <math.h>

#include <algorithm>
#include <atomic>

#include "qg_attn.cuh"
#include "qg_mma.cuh"

__device__ unsigned int g_qg_status_attn;  // this translation unit's device status word
static std::atomic<bool> g_launched{false};   // whether a kernel that may set it has been launched

namespace {

using namespace qg;

template <int D>
struct NarrowCfg {
  static constexpr int NW = D == 256 ? 4 : 8;                 // warps per CTA
  static constexpr uint32_t TILE = kNarrowKeys * D * 2;       // bytes of a key (or value) tile
  static constexpr int NST = D == 64 ? 6 : 3;                 // tiles a warp has room for
  static constexpr uint32_t SMEM = NW * NST * 2 * TILE;       // 192 KB
};

// The products multiply every value of a tile by every row's weight, and zero times infinity is NaN.  So
// where some row must not see a key that is there, infinite and NaN values of the tile leave it
// before the product and are added to the rows that do see them (by the warp; its lanes' columns
// are 8 d + 2 qc and the one after; 16 keys from key0 on; lim: keys that the lane's two rows see).
template <int D, bool BF16>
QG_DEVICE void add_nonfinite(const uint8_t *v, int key0, int qc, const int (&lim)[2], float (&o)[D / 8][4]) {
#pragma unroll 1
  for (int k = 0; k < kNarrowKeys; ++k) {
#pragma unroll
    for (int d = 0; d < D / 8; ++d) {
      const uint32_t w = *reinterpret_cast<const uint32_t *>(v + k * (D * 2) + (d ^ (k & 7)) * 16 + 4 * qc);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (!nonfinite16<BF16>(c ? w >> 16 : w)) continue;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (key0 + k < lim[e]) o[d][2 * e + c] += c ? hi16<BF16>(w) : lo16<BF16>(w);
      }
    }
  }
}

// Each warp is a worker of its own: it walks its pieces with a private ring of key and value
// tiles (16 keys, cp.async, no barrier wider than the warp), the piece's 16 query rows in
// mma fragments, and writes the piece's unnormalised output, maximum and sum.  mma.sync
// m16n8k16 fits here where tcgen05's 128-row tiles would be nearly empty: it runs at a fifth of
// its rate beside the copies (tensor pipe 18 %, issue 26 % busy at 6.3 TB/s).  Eight warps of three
// 8 KB stages keep 128 KB in flight on an SM, three times what its share of the bandwidth needs.
template <int D, bool BF16, bool OUT32>
__global__ void __launch_bounds__(NarrowCfg<D>::NW * 32, 1) attn_narrow_kernel(const __grid_constant__ AttnArgs a) {
  using C = NarrowCfg<D>;
  constexpr int NT = C::NW * 32;
  constexpr int KS = D / 16;       // 16-element steps of q.K
  constexpr int DT = D / 8;        // 8-column tiles of the output
  constexpr int CH = D / 8;        // 16-byte chunks per row
  constexpr int RPI = 32 / CH;     // rows per copy instruction of the warp
  static_assert(CH <= 32, "a row is at most one chunk per lane");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ LineScan<NT> scan;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const Line &ln = a.narrow;
  const long long total = line_scan<NT>(a, ln, &scan, blockIdx.x == 0);
  if (blockIdx.x == 0) {  // lengths outside the page lists are cut there and reported
    for (int i = threadIdx.x; i < a.b.G + a.b.B; i += NT) {
      const int raw = i < a.b.G ? __ldg(a.b.prefix_len + i) : __ldg(a.b.kv_len + i - a.b.G);
      const int cap = kv_cap(i < a.b.G ? a.b.max_prefix_pages : a.b.max_pages, a.pool.page_shift);
      if (raw < 0 || raw > cap) atomicOr(&g_qg_status_attn, QG_STATUS_BIT_ID);
    }
  }
  if (total == 0) return;
  const int nw = line_workers(ln, total);
  const int w = warp * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
  if (w >= nw) return;
  const Cut cut = line_cut(total, nw);
  const long long at = line_start(cut, w), end = line_start(cut, w + 1);
  if (at >= end) return;
  Cursor cur;
  if (!cursor_find(a, ln, scan, at, &cur)) return;

  const uint32_t ring = smem_u32(smem) + static_cast<uint32_t>(warp) * (C::NST * 2 * C::TILE);
  const int shift = a.pool.page_shift;
  const int qr = lane >> 2, qc = lane & 3;      // fragment row and column pair
  const int crow = lane / CH, cchunk = lane % CH;  // copy: row within an instruction, chunk

  for (bool more = true; more; more = cursor_next(a, ln, scan, &cur, end)) {
    int j0, j1, n_tiles;
    cursor_tiles(ln, cur, at, end, &j0, &j1, &n_tiles);
    if (j0 >= j1) continue;
    const Seg g = cur.g;

    // ---- this lane's two rows: query fragments and key limits
    const int tile_t0 = cur.r * ln.tpt;
    const int tokens = min(ln.tpt, g.nt - tile_t0);
    const int nrows = tokens * a.Gq;
    int lim[2];
    uint32_t qf[KS][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = qr + 8 * e;
      lim[e] = 0;
      const uint16_t *qp = nullptr;
      if (row < nrows) {
        const int t = g.t0 + tile_t0 + row / a.Gq;
        lim[e] = row_limit(a, g, t);
        qp = a.q + t * a.q_stride + static_cast<long long>(cur.h * a.Gq + row % a.Gq) * D + 2 * qc;
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qf[ks][e] = qp ? __ldg(reinterpret_cast<const uint32_t *>(qp + 16 * ks)) : 0u;
        qf[ks][2 + e] = qp ? __ldg(reinterpret_cast<const uint32_t *>(qp + 16 * ks + 8)) : 0u;
      }
    }
    // keys below every valid row's limit need no mask
    int all = min(qr < nrows ? lim[0] : 0x7FFFFFFF, qr + 8 < nrows ? lim[1] : 0x7FFFFFFF);
    all = __reduce_min_sync(0xFFFFFFFFu, all);

    // lane r < 16: element offset of key row 16 j + r, -1 past the end
    const long long hoff = cur.h * a.pool.head_stride;
    auto row_off = [&](int j) -> long long {
      const int key = 16 * j + (lane & 15);
      if (key >= g.len || j >= j1) return -1;
      const int page = __ldg(g.table + (key >> shift));
      if (page < 0 || page >= a.pool.n_pages) {
        atomicOr(&g_qg_status_attn, QG_STATUS_BIT_ID);
        return -1;
      }
      return page * a.pool.page_stride + (key & ((1 << shift) - 1)) * a.pool.token_stride + hoff;
    };
    auto issue = [&](int j, long long off) {
      if (j < j1) {
        const uint32_t kb = ring + static_cast<uint32_t>(j % C::NST) * (2 * C::TILE);
#pragma unroll
        for (int i = 0; i < kNarrowKeys / RPI; ++i) {
          const int row = i * RPI + crow;
          const long long o = __shfl_sync(0xFFFFFFFFu, off, row & 15);
          const uint32_t dst = kb + static_cast<uint32_t>(row) * (D * 2) + static_cast<uint32_t>((cchunk ^ (row & 7)) * 16);
          const long long src = (o < 0 ? 0 : o) + 8 * cchunk;
          const uint32_t n = o < 0 ? 0u : 16u;
          cp_async16_zfill(dst, a.pool.k + src, n);
          cp_async16_zfill(dst + C::TILE, a.pool.v + src, n);
        }
      }
      cp_async_commit();
    };

    float o[DT][4];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
    // m: the reference of the row's weights, its running maximum less what f16 weights are
    // raised by (2^14: the second term of a small one would otherwise lie among the subnormals)
    constexpr float RAISE = BF16 ? 0.f : 14.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    long long off = row_off(j0);
#pragma unroll
    for (int i = 0; i < C::NST - 1; ++i) {
      const long long nx = row_off(j0 + i + 1);
      issue(j0 + i, off);
      off = nx;
    }
    for (int j = j0; j < j1; ++j) {
      const long long nx = row_off(j + C::NST);
      cp_async_wait<C::NST - 2>();
      __syncwarp();  // tile j has landed, and every lane has read tile j - 1, which the next copy replaces
      issue(j + C::NST - 1, off);
      off = nx;
      const uint32_t kb = ring + static_cast<uint32_t>(j % C::NST) * (2 * C::TILE), vb = kb + C::TILE;
      // ---- scores of 16 rows x 16 keys
      float s[2][4], s2[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[0][e] = s[1][e] = s2[0][e] = s2[1][e] = 0.f;
      const int mat = lane >> 3, krow = (lane & 7) + ((mat >> 1) << 3);
      const uint32_t ka = kb + static_cast<uint32_t>(krow) * (D * 2);
#pragma unroll
      for (int ks = 0; ks < KS; ks += 2) {
        uint32_t b[4];
        ldsm4(b, ka + static_cast<uint32_t>(((2 * ks + (mat & 1)) ^ (krow & 7)) * 16));
        mma16816<BF16>(s[0], qf[ks], b[0], b[1]);
        mma16816<BF16>(s[1], qf[ks], b[2], b[3]);
        ldsm4(b, ka + static_cast<uint32_t>(((2 * ks + 2 + (mat & 1)) ^ (krow & 7)) * 16));
        mma16816<BF16>(s2[0], qf[ks + 1], b[0], b[1]);
        mma16816<BF16>(s2[1], qf[ks + 1], b[2], b[3]);
      }
      float x[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = (s[nt][e] + s2[nt][e]) * a.scale_log2;
      if (16 * j + 16 > all) {  // masked keys by selection: whatever the products hold
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * j + 8 * nt + 2 * qc + (e & 1) >= lim[e >> 1]) x[nt][e] = -INFINITY;
      }
      // ---- running maximum and sum of each row (four lanes share a row)
      uint32_t ph[4], plo[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(fmaxf(x[0][2 * e], x[0][2 * e + 1]), fmaxf(x[1][2 * e], x[1][2 * e + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        const float mn = fmaxf(m[e], mx - RAISE);
        const float ms = mn == -INFINITY ? 0.f : mn;
        if (__any_sync(0xFFFFFFFFu, mn > m[e])) {
          const float al = ex2(m[e] - ms);
          l[e] *= al;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            o[d][2 * e] *= al;
            o[d][2 * e + 1] *= al;
          }
        }
        m[e] = mn;
        const float p0 = ex2(x[0][2 * e] - ms), p1 = ex2(x[0][2 * e + 1] - ms);
        const float p2 = ex2(x[1][2 * e] - ms), p3 = ex2(x[1][2 * e + 1] - ms);
        l[e] += (p0 + p1) + (p2 + p3);
        ph[e] = pack16<BF16>(p0, p1);
        ph[2 + e] = pack16<BF16>(p2, p3);
        if constexpr (OUT32) {  // what the rounding left, as a second operand
          plo[e] = pack16<BF16>(p0 - lo16<BF16>(ph[e]), p1 - hi16<BF16>(ph[e]));
          plo[2 + e] = pack16<BF16>(p2 - lo16<BF16>(ph[2 + e]), p3 - hi16<BF16>(ph[2 + e]));
        }
      }
      // ---- o += p V
      if (all < min(g.len, 16 * j + 16)) {
        uint4 *vt = reinterpret_cast<uint4 *>(smem + (vb - smem_u32(smem)));
        uint32_t some = 0;
        for (int i = lane; i < kNarrowKeys * CH; i += 32) some |= any_nonfinite<BF16>(vt[i]);
        if (__any_sync(0xFFFFFFFFu, some)) {
          add_nonfinite<D, BF16>(reinterpret_cast<const uint8_t *>(vt), 16 * j, qc, lim, o);
          __syncwarp();
          for (int i = lane; i < kNarrowKeys * CH; i += 32) vt[i] = make_finite<BF16>(vt[i]);
          __syncwarp();
        }
      }
      const int vrow = (lane & 7) + ((mat & 1) << 3);
      const uint32_t va = vb + static_cast<uint32_t>(vrow) * (D * 2);
#pragma unroll
      for (int d = 0; d < DT; d += 2) {
        uint32_t b[4];
        ldsm4_t(b, va + static_cast<uint32_t>(((d + (mat >> 1)) ^ (vrow & 7)) * 16));
        mma16816<BF16>(o[d], ph, b[0], b[1]);
        mma16816<BF16>(o[d + 1], ph, b[2], b[3]);
        if constexpr (OUT32) {
          mma16816<BF16>(o[d], plo, b[0], b[1]);
          mma16816<BF16>(o[d + 1], plo, b[2], b[3]);
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();  // every lane has read the last tiles: the next piece's copies may replace them

    // ---- write the piece
    const bool alone = j0 == 0 && j1 == n_tiles && seg_whole(a, g, cur.s >> 1);
    const long long slot = piece_slot(ln, cur.unit, w);
    if (slot < 0 && !alone) {
      if (lane == 0) atomicOr(&g_qg_status_attn, QG_STATUS_BIT_ID);
      continue;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float ls = l[e];
      ls += __shfl_xor_sync(0xFFFFFFFFu, ls, 1);
      ls += __shfl_xor_sync(0xFFFFFFFFu, ls, 2);
      const int row = qr + 8 * e;
      if (row >= nrows) continue;
      if (alone) {
        const float inv = ls == 0.f ? 0.f : 1.0f / ls;
        const int t = g.t0 + tile_t0 + row / a.Gq;
        const size_t base = (static_cast<size_t>(t) * a.Hq + cur.h * a.Gq + row % a.Gq) * D + 2 * qc;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          if constexpr (OUT32)
            *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + base + 8 * d) =
                make_float2(o[d][2 * e] * inv, o[d][2 * e + 1] * inv);
          else
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + base + 8 * d) =
                pack16<BF16>(o[d][2 * e] * inv, o[d][2 * e + 1] * inv);
        }
      } else {
        float *po = ln.part_o + (slot * kNarrowRows + row) * D + 2 * qc;
#pragma unroll
        for (int d = 0; d < DT; ++d)
          *reinterpret_cast<float2 *>(po + 8 * d) = make_float2(o[d][2 * e], o[d][2 * e + 1]);
        if (qc == 0) ln.part_ml[slot * kNarrowRows + row] = make_float2(m[e], ls);
      }
    }
  }
}

// ---- joining ------------------------------------------------------------------------------------
// One token's rows in one segment: what its pieces' slots follow from, for every head.
struct RowSeg {
  const Line *l;            // null: no keys there
  int s;                    // the segment
  long long p0, cost;       // place of head 0's unit, places per head
  Cut cut;                  // the line's parts
  int unit, rt, x;          // head 0's unit, units per head, keys of a unit
  int row, halves;          // first row in the tile; 2: each slot holds two partial results of a row
};

// from the lengths alone; row_seg_place adds what the attention kernels published
QG_DEVICE RowSeg row_seg(const AttnArgs &a, int s, int t) {
  RowSeg q;
  q.l = nullptr;
  q.s = s;
  const Seg g = seg_load(a, s);
  const bool nar = seg_in(a.narrow, g);
  if (!nar && !(a.wide.workers && seg_in(a.wide, g))) return q;
  const Line &l = nar ? a.narrow : a.wide;
  if (t < g.t0 || t >= g.t0 + g.nt) return q;  // starts that do not rise
  const int r = (t - g.t0) / l.tpt, i = t - g.t0 - r * l.tpt;
  q.x = unit_keys(l, g, r);
  if (q.x == 0) return q;
  q.l = &l;
  q.rt = seg_tiles(l, g);
  q.p0 = seg_cost_to(l, g, r);
  q.cost = seg_cost_to(l, g, q.rt);
  q.unit = r;
  q.halves = 1;
  if (nar) {
    q.row = i * a.Gq;
  } else {
    const int half = l.tpt / 2;
    q.row = (i / half) * kWideHalf + (i % half) * a.Gq;
    // one half's rows alone: the kernel's two streams took the key tiles in turn
    if (g.nt - r * l.tpt <= half) q.halves = 2;
  }
  return q;
}

QG_DEVICE void row_seg_place(const AttnArgs &a, RowSeg *q) {
  if (!q->l) return;
  const long long total = __ldcg(q->l->seg_pos + 2 * a.b.B);
  q->cut = line_cut(total, line_workers(*q->l, total));
  q->p0 += __ldcg(q->l->seg_pos + q->s);
  q->unit += __ldcg(q->l->seg_unit + q->s);
}

// The pieces of one row: slots first, first + 1, ... (count of them), row `row` of a `rows`-row
// tile (and the one kWideHalf rows on, with two halves).
struct Pieces {
  const float *o;
  const float2 *ml;
  size_t first;
  int count, rows, row, halves;
};
QG_DEVICE Pieces pieces_of(const RowSeg &q, int h, int gq) {
  Pieces p;
  p.count = 0;
  p.halves = 1;
  if (!q.l) return p;
  const Line &l = *q.l;
  const long long p0 = q.p0 + h * q.cost;
  const int w0 = line_owner(q.cut, p0);
  int w1 = line_owner(q.cut, p0 + q.x - 1);
  // the last one's part may lie within the last key tile, which is then its neighbour's
  if (w1 > w0 && tiles_of(l, static_cast<int>(line_start(q.cut, w1) - p0)) >= tiles_of(l, q.x)) --w1;
  p.o = l.part_o;
  p.ml = l.part_ml;
  p.first = static_cast<size_t>(q.unit + h * q.rt) + static_cast<size_t>(w0);
  p.count = w1 - w0 + 1;
  p.rows = l.rows;
  p.row = q.row + gq;
  p.halves = q.halves;
  if (piece_slot(l, q.unit + h * q.rt, w1) < 0) p.count = 0;  // not written
  return p;
}
// whether a worker wrote the row itself: all its keys are in one piece
QG_DEVICE bool written(const Pieces &own, const Pieces &pre) {
  return own.count == 1 && own.halves == 1 && pre.count == 0;
}

// Online softmax over pieces i0, i0 + step, ...: lane holds D/32 consecutive outputs.
template <int NV>
struct Acc {
  float m, l, o[NV];
};
template <int NV>
QG_DEVICE void acc_add(Acc<NV> &x, float m, float l, const float (&o)[NV]) {
  if (l == 0.f) return;  // nothing seen (and o not written); the sum of NaN scores is NaN, under a maximum of -inf
  const float mn = fmaxf(x.m, m);
  const float fa = ex2(x.m - mn), fb = ex2(m - mn);
  x.m = mn;
  x.l = x.l * fa + l * fb;
#pragma unroll
  for (int i = 0; i < NV; ++i) x.o[i] = x.o[i] * fa + o[i] * fb;
}
QG_DEVICE size_t piece_row(const Pieces &p, int i) {
  const int slot = p.halves == 2 ? i >> 1 : i, half = p.halves == 2 ? i & 1 : 0;
  return (p.first + slot) * p.rows + p.row + half * kWideHalf;
}
template <int D>
QG_DEVICE void load_o(const Pieces &p, int i, int r, int lane, float (&v)[D / 32]) {
  const float *src = p.o + (piece_row(p, i) + r) * D + lane * (D / 32);
  if constexpr (D == 64) {
    const float2 u = __ldcg(reinterpret_cast<const float2 *>(src));
    v[0] = u.x;
    v[1] = u.y;
  } else {
#pragma unroll
    for (int q = 0; q < D / 128; ++q) {
      const float4 u = __ldcg(reinterpret_cast<const float4 *>(src) + q);
      v[4 * q] = u.x;
      v[4 * q + 1] = u.y;
      v[4 * q + 2] = u.z;
      v[4 * q + 3] = u.w;
    }
  }
}
// R neighbouring rows of the tile (the first nr of them), U pieces of each in flight.
template <int D, int R, int U>
QG_DEVICE void acc_pieces(Acc<D / 32> (&x)[R], int nr, const Pieces &p, int i0, int step, int lane) {
  const int count = p.count * p.halves;
  for (int i = i0; i < count; i += U * step) {
    float v[R][U][D / 32];
    float2 ml[R][U];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < U; ++k) {
        ml[r][k] = make_float2(-INFINITY, 0.f);
        if (r < nr && i + k * step < count) {
          ml[r][k] = __ldcg(p.ml + piece_row(p, i + k * step) + r);
          load_o<D>(p, i + k * step, r, lane, v[r][k]);
        }
      }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (r < nr && i + k * step < count) acc_add(x[r], ml[r][k].x, ml[r][k].y, v[r][k]);
  }
}
template <int NV, int R>
QG_DEVICE void acc_clear(Acc<NV> (&x)[R]) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    x[r].m = -INFINITY;
    x[r].l = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) x[r].o[i] = 0.f;
  }
}

template <int D, bool BF16, bool OUT32>
QG_DEVICE void write_row(const AttnArgs &a, int t, int hq, int lane, const Acc<D / 32> &x) {
  constexpr int NV = D / 32;
  const float inv = x.l == 0.f ? 0.f : 1.0f / x.l;
  const size_t base = (static_cast<size_t>(t) * a.Hq + hq) * D + lane * NV;
  if constexpr (OUT32) {
#pragma unroll
    for (int i = 0; i < NV; i += 2)
      *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + base + i) = make_float2(x.o[i] * inv, x.o[i + 1] * inv);
  } else {
#pragma unroll
    for (int i = 0; i < NV; i += 2)
      *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + base + i) =
          pack16<BF16>(x.o[i] * inv, x.o[i + 1] * inv);
  }
}

// The two segments of token t that hold keys for it: its sequence's own, and its run's.
QG_DEVICE void token_segs(const AttnArgs &a, int t, RowSeg *own, RowSeg *pre) {
  own->l = pre->l = nullptr;
  const int b = kv_seq_of(a.b, t);
  if (b < 0) {
    atomicOr(&g_qg_status_attn, QG_STATUS_BIT_ID);
    return;
  }
  *own = row_seg(a, 2 * b + 1, t);
  const int gr = kv_group_of(a.b, b);
  if (gr >= 0 && !seq_long(a, b)) *pre = row_seg(a, 2 * run_first(a, gr, b), t);
}

// How the rows are shared out:
//   kRowBlock  a block of 8 warps per row, the row's pieces spread over the warps: few rows with
//              many pieces each;
//   kRowWarp   a warp per row: a batch's decode step;
//   kTokens    a block per 32 tokens and cached head: its first warp's lanes ask which tokens need
//              joining at all, its warps join those: prompts, most of whose rows their workers
//              wrote.  (A block for all heads was slower: a cut falls on all of a tile's tokens.)
enum { kRowBlock, kRowWarp, kTokens };
struct JoinItem {
  Pieces own, pre;
  int t;
};
constexpr int kTokensThreads = 128;
template <int D, bool BF16, bool OUT32, int MODE>
__global__ void __launch_bounds__(MODE == kTokens ? kTokensThreads : 256) attn_join_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int NV = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // What follows from the lengths is worked out while the attention kernels drain: their own wait
  // came after everything before the call.
  RowSeg so, sp;
  so.l = sp.l = nullptr;
  auto place = [&] {
    pdl_wait();
    pdl_launch_dependents();
    row_seg_place(a, &so);
    row_seg_place(a, &sp);
  };
  if constexpr (MODE == kTokens) {
    __shared__ JoinItem items[32];
    __shared__ int n_items;
    const int h = static_cast<int>(blockIdx.y);
    if (warp == 0) {
      const int t = static_cast<int>(blockIdx.x) * 32 + lane;
      JoinItem it;
      bool need = false;
      if (t < a.b.T) token_segs(a, t, &so, &sp);
      place();
      if (t < a.b.T) {
        it = JoinItem{pieces_of(so, h, 0), pieces_of(sp, h, 0), t};
        need = !written(it.own, it.pre);
      }
      const uint32_t all = __ballot_sync(0xFFFFFFFFu, need);
      if (need) items[__popc(all & ((1u << lane) - 1u))] = it;
      if (lane == 0) n_items = __popc(all);
    } else {
      pdl_wait();
    }
    __syncthreads();
    constexpr int R = 2;  // a head's query rows, two at a time
    const int groups = (a.Gq + R - 1) / R, tasks = n_items * groups;
    for (int k = warp; k < tasks; k += kTokensThreads / 32) {
      const JoinItem &it = items[k / groups];
      const int q0 = (k % groups) * R, nr = min(R, a.Gq - q0);
      Pieces own = it.own, pre = it.pre;
      own.row += q0;
      pre.row += q0;
      Acc<NV> x[R];
      acc_clear(x);
      acc_pieces<D, R, 2>(x, nr, own, 0, 1, lane);
      acc_pieces<D, R, 2>(x, nr, pre, 0, 1, lane);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (r < nr) write_row<D, BF16, OUT32>(a, it.t, h * a.Gq + q0 + r, lane, x[r]);
    }
  } else {
    const int item = MODE == kRowBlock ? static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x) * 8 + warp;
    const int t = item / a.Hq, hq = item - t * a.Hq;
    if (t < a.b.T) token_segs(a, t, &so, &sp);
    place();
    if (t >= a.b.T) return;
    const Pieces own = pieces_of(so, hq / a.Gq, hq % a.Gq), pre = pieces_of(sp, hq / a.Gq, hq % a.Gq);
    if (written(own, pre)) return;
    Acc<NV> x[1];
    acc_clear(x);
    constexpr int W = MODE == kRowBlock ? 8 : 1;  // warps per row
    acc_pieces<D, 1, 4>(x, 1, own, MODE == kRowBlock ? warp : 0, W, lane);
    acc_pieces<D, 1, 4>(x, 1, pre, MODE == kRowBlock ? warp : 0, W, lane);
    if constexpr (MODE == kRowBlock) {
      __shared__ float sh[8][D];
      __shared__ float2 sml[8];
#pragma unroll
      for (int i = 0; i < NV; ++i) sh[warp][lane * NV + i] = x[0].o[i];
      if (lane == 0) sml[warp] = make_float2(x[0].m, x[0].l);
      __syncthreads();
      if (warp) return;
#pragma unroll
      for (int q = 1; q < 8; ++q) {
        float v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = sh[q][lane * NV + i];
        acc_add(x[0], sml[q].x, sml[q].y, v);
      }
    }
    write_row<D, BF16, OUT32>(a, t, hq, lane, x[0]);
  }
}

// ---- workspace ----------------------------------------------------------------------------------
constexpr size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
  size_t bytes;
  long long n_slots, w_slots;       // pieces the two lines can have
  size_t n_pos, n_unit, n_o, n_ml;  // offsets of the narrow line's arrays
  size_t w_pos, w_unit, w_o, w_ml;  // of the wide line's
  size_t flags;                     // of value_flags
  int wide_workers, narrow_workers;
};

// rows bound: a unit per (cached head, row tile); tiles of a segment: tokens / tpt + 1
Plan make_plan(const KvPool &pool, const KvBatch &b, int Gq, int sms) {
  Plan p = {};
  const int tn = kNarrowRows / Gq, tw = 2 * (kWideHalf / Gq);
  const long long nseg = 2LL * b.B;
  const bool wide = attn_wide_supported(pool.D) && b.T > tn;
  p.narrow_workers = sms * (pool.D == 256 ? 4 : 8);
  p.wide_workers = wide ? sms : 0;
  // long sequences have more than kWideHalf / Gq tokens; runs: one per group and one after each
  // long sequence.  A token is in its own segment and in at most one run.
  const long long longs = b.q_start ? std::min<long long>(b.B, b.T / (kWideHalf / Gq + 1)) : 0;
  const long long runs = b.G ? std::min<long long>(b.B, b.G + (wide ? longs : 0)) : 0;
  long long un = b.B + runs;                                      // wide line there: one row tile each
  if (!wide) un += (b.G ? 2 : 1) * (static_cast<long long>(b.T) / tn);
  const long long sn = un * pool.Hkv + p.narrow_workers;
  p.n_slots = sn;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at += up256(n);
    return r;
  };
  p.n_pos = take((nseg + 1) * 8);
  p.n_unit = take((nseg + 1) * 4);
  p.n_ml = take(static_cast<size_t>(sn) * kNarrowRows * 8);
  p.n_o = take(static_cast<size_t>(sn) * kNarrowRows * pool.D * 4);
  if (wide) {
    // of each kind, at most T / (tn + 1) segments have the more than tn tokens of the wide line; n tokens make
    // at most 1 + n / tw tiles, own segments of sequences that are not long one, and long sequences' tokens are in
    // no run: so all the tiles beyond a segment's first come from T tokens, each counted once
    const long long most = b.T / (tn + 1);
    const long long uw = (b.q_start ? std::min<long long>(b.B, most) : 0) + (b.G ? std::min<long long>(runs, most) : 0) +
                         (b.q_start || b.G ? static_cast<long long>(b.T) / tw : 0);
    const long long sw = uw * pool.Hkv + p.wide_workers;
    p.w_slots = sw;
    p.w_pos = take((nseg + 1) * 8);
    p.w_unit = take((nseg + 1) * 4);
    p.w_ml = take(static_cast<size_t>(sw) * kWideRows * 8);
    p.w_o = take(static_cast<size_t>(sw) * kWideRows * pool.D * 4);
    p.flags = take(b.q_start ? static_cast<size_t>(2 * pool.Hkv) * ((b.T + 31) / 32) * 4 : 0);
  }
  p.bytes = at;
  return p;
}

qg_status attn_check(const qg_kv_cache *cache, const qg_kv_batch *batch, int Hq, AttnArgs *a) {
  qg_status st = kv_check_cache(cache, &a->pool);
  if (st != QG_OK) return st;
  st = kv_check_batch(batch, true, true, &a->b);
  if (st != QG_OK) return st;
  if (Hq < 1 || Hq % a->pool.Hkv) return QG_EINVAL_SHAPE;
  if (Hq / a->pool.Hkv > kNarrowRows) return QG_EUNSUPPORTED;
  a->Hq = Hq;
  a->Gq = Hq / a->pool.Hkv;
  a->D = a->pool.D;
  return QG_OK;
}

template <int D, bool BF16, bool OUT32>
qg_status attn_run(const AttnArgs &a, int sms, cudaStream_t s) {
  using C = NarrowCfg<D>;
  auto narrow = attn_narrow_kernel<D, BF16, OUT32>;
  if (!set_smem_attr(reinterpret_cast<const void *>(narrow), C::SMEM)) return QG_ECUDA;
  g_launched = true;
  if (a.value_flags) {
    const qg_status st = attn_flags_launch(a, BF16, s);
    if (st != QG_OK) return st;
  }
  if (launch_pdl(narrow, dim3(static_cast<unsigned>(sms)), dim3(C::NW * 32), C::SMEM, s, a) != cudaSuccess)
    return QG_ECUDA;
  if (a.wide.workers) {
    const qg_status st = attn_wide_launch(a, BF16, s);
    if (st != QG_OK) return st;
  }
  const long long rows = static_cast<long long>(a.b.T) * a.Hq;
  cudaError_t e;
  // 2048 rows of about 20 pieces: 30 us with a block per row, 12 with a warp; 7832 tokens of 32
  // rows, few to be joined: 57 us with a warp per token, 14 with blocks of 32 tokens
  if (rows <= 3LL * sms)
    e = launch_pdl(attn_join_kernel<D, BF16, OUT32, kRowBlock>, dim3(static_cast<unsigned>(rows)), dim3(256), 0, s, a);
  else if (rows <= 8192)
    e = launch_pdl(attn_join_kernel<D, BF16, OUT32, kRowWarp>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, s, a);
  else
    e = launch_pdl(attn_join_kernel<D, BF16, OUT32, kTokens>, dim3(static_cast<unsigned>((a.b.T + 31) / 32), a.pool.Hkv),
                   dim3(kTokensThreads), 0, s, a);
  if (e != cudaSuccess) return QG_ECUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ECUDA;
}

template <int D>
qg_status attn_dispatch(const AttnArgs &a, bool bf16, int sms, cudaStream_t s) {
  if (bf16) return a.out32 ? attn_run<D, true, true>(a, sms, s) : attn_run<D, true, false>(a, sms, s);
  return a.out32 ? attn_run<D, false, true>(a, sms, s) : attn_run<D, false, false>(a, sms, s);
}

}  // namespace

namespace qg {
unsigned int read_status_attn(bool clear) {
  unsigned int v = 0;
  if (!g_launched) return v;
  if (cudaMemcpyFromSymbol(&v, g_qg_status_attn, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_qg_status_attn, &z, sizeof(z));
  }
  return v;
}
}  // namespace qg

extern "C" {

size_t qg_attn_workspace_size(const qg_kv_cache *cache, const qg_kv_batch *batch, int Hq) {
  AttnArgs a = {};
  if (attn_check(cache, batch, Hq, &a) != QG_OK) return 0;
  const DeviceInfo &dev = device_info();
  return make_plan(a.pool, a.b, a.Gq, dev.ok ? dev.sms : 152).bytes;
}

qg_status qg_attn_paged(const qg_kv_cache *cache, const qg_kv_batch *batch, int Hq, const void *q, int64_t q_stride,
                        float scale, void *out, int out_dtype, void *workspace, size_t workspace_bytes,
                        qg_stream_t stream) {
  AttnArgs a = {};
  const qg_status st = attn_check(cache, batch, Hq, &a);
  if (st != QG_OK) return st;
  if (a.b.T == 0) return QG_OK;
  if (!q || !out) return QG_EINVAL_PTR;
  if (out_dtype != QG_DT_F32 && out_dtype != cache->dtype) return QG_EUNSUPPORTED;
  if (!isfinite(scale) || q_stride < static_cast<int64_t>(Hq) * a.D || q_stride > (int64_t(1) << 38))
    return QG_EINVAL_SHAPE;
  if (!aligned16(q) || !aligned16(out) || q_stride % 8) return QG_EALIGN;
  const DeviceInfo &dev = device_info();
  const Plan p = make_plan(a.pool, a.b, a.Gq, dev.ok ? dev.sms : 152);
  if (!workspace || workspace_bytes < p.bytes) return QG_EWORKSPACE;
  if (!aligned16(workspace)) return QG_EALIGN;
  if (!dev.ok) return QG_ECUDA;
  a.q = static_cast<const uint16_t *>(q);
  a.q_stride = q_stride;
  a.out = out;
  a.out32 = out_dtype == QG_DT_F32;
  a.scale_log2 = scale * 1.4426950408889634f;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  auto line = [&](int rows, int kshift, int workers, long long slots, size_t pos, size_t unit, size_t o, size_t ml) {
    Line l = {};
    l.rows = rows;
    l.kshift = kshift;
    l.tpt = rows == kNarrowRows ? rows / a.Gq : 2 * (kWideHalf / a.Gq);
    l.workers = workers;
    l.slots = slots;
    l.seg_pos = reinterpret_cast<long long *>(ws + pos);
    l.seg_unit = reinterpret_cast<int *>(ws + unit);
    l.part_o = reinterpret_cast<float *>(ws + o);
    l.part_ml = reinterpret_cast<float2 *>(ws + ml);
    return l;
  };
  a.narrow = line(kNarrowRows, kNarrowShift, p.narrow_workers, p.n_slots, p.n_pos, p.n_unit, p.n_o, p.n_ml);
  a.long_tokens = p.wide_workers ? kWideHalf / a.Gq : INT32_MAX;
  a.narrow.hi = p.wide_workers ? a.narrow.tpt : INT32_MAX;
  if (p.wide_workers) {
    a.wide = line(kWideRows, kWideShift, p.wide_workers, p.w_slots, p.w_pos, p.w_unit, p.w_o, p.w_ml);
    a.wide.lo = a.narrow.tpt;
    a.wide.hi = INT32_MAX;
    // The warp that walks the line waits for whole pieces, and the others for it while it passes over empty
    // segments: a quarter of a second, 2^13 cycles for each key that a piece can have by the page lists (about
    // 27 are needed, thousands where an infinite value is read again) and 2^14 for each segment, a minute at most.
    const long long most = static_cast<long long>(a.b.max_pages + static_cast<long long>(a.b.max_prefix_pages)) << a.pool.page_shift;
    a.wait_cycles = std::min((1LL << 29) + (most << 13) + (static_cast<long long>(a.b.B) << 15), 1LL << 37);
    // without q_start no token comes after another of its sequence
    if (a.b.q_start) a.value_flags = reinterpret_cast<uint32_t *>(ws + p.flags);
  }
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = cache->dtype == QG_DT_BF16;
  switch (a.D) {
    case 64: return attn_dispatch<64>(a, bf16, dev.sms, s);
    case 128: return attn_dispatch<128>(a, bf16, dev.sms, s);
    default: return attn_dispatch<256>(a, bf16, dev.sms, s);
  }
}

}  // extern "C"
