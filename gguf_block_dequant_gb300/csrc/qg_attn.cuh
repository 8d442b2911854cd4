// qg_attn.cuh -- the work of one attention call, as its kernels share it.
//
// A SEGMENT is a list of cached keys with the query tokens that read it: a group's prefix with
// the tokens of a run of the group's sequences, or a sequence's own keys with its own tokens.  A
// LONG sequence, with more query rows than the 128 of a tensor-core tile, gains nothing from
// sharing the read of a prefix: its own segment has the prefix's keys first, and its rows need
// no joining; runs are what long sequences leave of a group.  The rows
// of a segment and a cached head are its (token, query head of that cached head) pairs; they
// are cut into ROW TILES of `tpt` whole tokens.  A UNIT is (segment, cached head, row tile),
// and its cost is the number of keys its last row sees.  All units in (segment, head, row
// tile) order, key by key, form one LINE; worker w of n takes the w-th of n
// equal parts of it, the part's ends raised to whole key tiles of their units.  So ragged
// lengths balance without the host knowing them, and every kernel can work out from the lengths
// alone who did what: costs in keys rather than tiles make a segment's cost an arithmetic series
// (the sum of rounded-up tile counts took tens of thousands of cycles to invert).  A worker's
// part of one unit is a PIECE; unit u and worker w rise along the line and one of them rises
// from piece to piece, so u + w numbers the pieces' slots in the workspace without gaps mattering.
//
// Two kernels with a line each share a call: segments with few rows (at most one row tile of 16)
// and segments with more (row tiles of two times 128).  The joining kernel reads both lines.  The
// border, measured on 8 groups under 2999 tokens each: groups of 24 rows a head take 60 us on the
// wide kernel and 64 as two narrow row tiles, groups of 32 rows 61 and 99.
#pragma once

#include "qg_kv.cuh"

namespace qg {

constexpr int kNarrowRows = 16, kNarrowShift = 4, kNarrowKeys = 1 << kNarrowShift;
constexpr int kWideHalf = 128, kWideRows = 2 * kWideHalf, kWideShift = 7, kWideKeys = 1 << kWideShift;

// A line: row and key tile sizes, and which segments belong to it.
struct Line {
  int rows, kshift;      // rows per tile, keys per tile (its logarithm)
  int tpt;               // tokens per row tile: rows / Gq (wide: two halves of 128 / Gq)
  int lo, hi;            // segments with lo < tokens <= hi belong to it
  int workers;
  long long slots;       // capacity of the pieces' arrays
  float *part_o;         // [slot][rows][D]
  float2 *part_ml;       // [slot][rows]: running maximum (log2 units) and sum
  long long *seg_pos;    // [2 B + 1] place of each segment's first key on the line
  int *seg_unit;         // [2 B + 1] first unit of each segment
};

struct AttnArgs {
  KvPool pool;
  KvBatch b;
  const uint16_t *q;
  void *out;
  long long q_stride;
  float scale_log2;      // scale * log2(e): exponentials are powers of two
  int Hq, Gq, D;
  int out32;
  int long_tokens;       // sequences of more new tokens are long
  long long wait_cycles; // limit of a wait inside the wide kernel
  uint32_t *value_flags; // [2][heads][tokens / 32] (qg_attn_tc.cu); null without q_start or a wide line
  Line narrow, wide;     // wide.workers == 0: the narrow line has every segment, nothing is long
};

struct Seg {
  int t0, nt;            // token rows
  int prefix;            // 1: a run of a group's sequences and the group's prefix
  int len;               // keys (own ones of a sequence)
  int plen;              // a long sequence's keys before its own
  const int32_t *table, *ptable;
};

QG_DEVICE int kv_prefix_len(const AttnArgs &a, int g) {
  return kv_clamp(__ldg(a.b.prefix_len + g), 0, kv_cap(a.b.max_prefix_pages, a.pool.page_shift));
}
QG_DEVICE const int32_t *kv_prefix_table(const AttnArgs &a, int g) {
  return a.b.prefix_pages + static_cast<size_t>(g) * a.b.max_prefix_pages;
}
QG_DEVICE bool seq_long(const AttnArgs &a, int b) {
  return a.b.q_start && kv_tok(a.b, b + 1) - kv_tok(a.b, b) > a.long_tokens;
}
// first sequence of the run that b, not long, of group g is in
QG_DEVICE int run_first(const AttnArgs &a, int g, int b) {
  const int lo = kv_clamp(__ldg(a.b.group_start + g), 0, b);
  if (!a.b.q_start || !a.wide.workers) return lo;
  while (b > lo && !seq_long(a, b - 1)) --b;
  return b;
}

// segment 2 b: the run of sequences that starts at b (empty when none does); 2 b + 1: b's own
QG_DEVICE Seg seg_load(const AttnArgs &a, int s) {
  const int b = s >> 1;
  Seg g;
  g.prefix = !(s & 1);
  g.nt = g.len = g.plen = 0;
  g.table = g.ptable = nullptr;
  g.t0 = kv_tok(a.b, b);
  const int gr = kv_group_of(a.b, b);
  const bool lg = seq_long(a, b);
  if (s & 1) {
    g.nt = max(0, kv_tok(a.b, b + 1) - g.t0);
    g.len = kv_own_len(a.b, a.pool.page_shift, b);
    g.table = a.b.pages + static_cast<size_t>(b) * a.b.max_pages;
    if (lg && gr >= 0) {
      g.plen = kv_prefix_len(a, gr);
      g.ptable = kv_prefix_table(a, gr);
    }
  } else if (gr >= 0 && !lg) {
    const int lo = __ldg(a.b.group_start + gr), hi = kv_clamp(__ldg(a.b.group_start + gr + 1), b + 1, a.b.B);
    if (b != max(lo, 0) && !seq_long(a, b - 1)) return g;  // the run began earlier
    int e = hi;
    if (a.b.q_start && a.wide.workers)
      for (e = b + 1; e < hi && !seq_long(a, e);) ++e;
    g.nt = max(0, kv_tok(a.b, e) - g.t0);
    g.len = kv_prefix_len(a, gr);
    g.table = kv_prefix_table(a, gr);
  }
  return g;
}

// A piece's slot, -1 past the arrays: only where token or group starts do not rise, so that
// segments hold more tokens than there are.
QG_DEVICE long long piece_slot(const Line &l, long long unit, int w) {
  const long long s = unit + w;
  return s < l.slots ? s : -1;
}

QG_DEVICE bool seg_in(const Line &l, const Seg &g) { return g.nt > l.lo && g.nt <= l.hi && (g.len | g.plen) > 0; }
QG_DEVICE int seg_tiles(const Line &l, const Seg &g) { return (g.nt + l.tpt - 1) / l.tpt; }  // row tiles

QG_DEVICE int tiles_of(const Line &l, int keys) { return (keys + (1 << l.kshift) - 1) >> l.kshift; }
// keys of row tile r: up to the last key its last token sees (a long sequence's prefix counts
// in whole tiles, so that its own keys start one)
QG_DEVICE int unit_keys(const Line &l, const Seg &g, int r) {
  if (g.prefix) return g.len;
  return (tiles_of(l, g.plen) << l.kshift) + kv_clamp(g.len - g.nt + min(g.nt, (r + 1) * l.tpt), 0, g.len);
}
// keys of row tiles 0 .. r-1
QG_DEVICE long long seg_cost_to(const Line &l, const Seg &g, int r) {
  if (g.prefix) return static_cast<long long>(r) * g.len;
  // own keys: tile i < rt - 1 sees base + (i + 1) tpt of them (none while that is not positive)
  const int rt = seg_tiles(l, g), base = g.len - g.nt, m = min(r, rt - 1);
  const int i0 = base < 0 ? min(m, -base / l.tpt) : 0;  // tiles that see nothing
  const long long n = m - i0;
  long long c = n * (base + (i0 + 1) * l.tpt) + n * (n - 1) / 2 * l.tpt;
  if (r == rt) c += g.len;
  return c + static_cast<long long>(r) * (tiles_of(l, g.plen) << l.kshift);
}

// workers that take part: about `kMinTiles` tiles each and never less than one, so that a worker
// whose part lies within a unit has a tile of it (the joining kernel counts on that)
constexpr int kMinTiles = 2;
QG_DEVICE int line_workers(const Line &l, long long total) {
  const long long n = (total + (kMinTiles << l.kshift) - 1) / (kMinTiles << l.kshift);
  return n < l.workers ? static_cast<int>(n) : l.workers;
}
// quotient of non-negative numbers, in 32 bits where they fit (a 64-bit division is a call)
QG_DEVICE long long div_pos(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}
// The line cut into n parts: part w starts at floor(w * total / n), evenly spread, so that equal
// units end where parts do whenever their numbers allow it.
struct Cut {
  long long size, total;
  int rest, n;
};
QG_DEVICE Cut line_cut(long long total, int n) {
  Cut c;
  c.n = n;
  c.total = total;
  c.size = div_pos(total, n);
  c.rest = static_cast<int>(total - c.size * n);
  return c;
}
QG_DEVICE long long line_start(const Cut &c, int w) {
  return w * c.size + static_cast<uint32_t>(w * c.rest) / static_cast<uint32_t>(c.n);
}
QG_DEVICE int line_owner(const Cut &c, long long p) {
  // the estimate's relative error is a few 2^-24 and there are a few thousand workers at most
  int w = static_cast<int>(static_cast<float>(p) * (static_cast<float>(c.n) / static_cast<float>(c.total)));
  w = min(w, c.n - 1);
  while (w > 0 && line_start(c, w) > p) --w;
  while (w + 1 < c.n && line_start(c, w + 1) <= p) ++w;
  return w;
}

// keys of the segment's (own) list that token t sees (t in the segment's token rows)
QG_DEVICE int row_limit(const AttnArgs &a, const Seg &g, int t) {
  if (!g.prefix) return kv_clamp(g.len - g.nt + (t - g.t0) + 1, 0, g.len);
  const int b = kv_seq_of(a.b, t);
  if (b < 0) return 0;
  const int t0 = kv_tok(a.b, b), n = kv_tok(a.b, b + 1) - t0;
  const long long seen = static_cast<long long>(g.len) + kv_own_len(a.b, a.pool.page_shift, b) - n + (t - t0) + 1;
  return seen < 0 ? 0 : seen > g.len ? g.len : static_cast<int>(seen);
}
// keys of a long sequence's prefix that token t sees
QG_DEVICE int row_prefix_limit(const Seg &g, int t) {
  const long long seen = static_cast<long long>(g.plen) + g.len - g.nt + (t - g.t0) + 1;
  return seen < 0 ? 0 : seen > g.plen ? g.plen : static_cast<int>(seen);
}

// ---- the block's view of a line ---------------------------------------------------------------
// Thread i of the block owns segments [i*chunk, (i+1)*chunk); pos[i], unit[i] are the line's
// keys and units before them.  Filled by all threads of the block.
constexpr int kKeptSegs = 128;
template <int NT>
struct LineScan {
  long long pos[NT + 1];
  int unit[NT + 1];
  Seg seg[kKeptSegs];  // the segments themselves, where there are no more (a thread owns one each)
};

template <int NT>
QG_DEVICE long long line_scan(const AttnArgs &a, const Line &l, LineScan<NT> *sc, bool publish) {
  const int nseg = 2 * a.b.B;
  const int chunk = (nseg + NT - 1) / NT;
  const int s0 = min(nseg, static_cast<int>(threadIdx.x) * chunk), s1 = min(nseg, s0 + chunk);
  long long c = 0;
  int u = 0;
  for (int s = s0; s < s1; ++s) {
    const Seg g = seg_load(a, s);
    if (nseg <= kKeptSegs) sc->seg[s] = g;
    if (!seg_in(l, g)) continue;
    const int rt = seg_tiles(l, g);
    c += a.pool.Hkv * seg_cost_to(l, g, rt);
    u += a.pool.Hkv * rt;
  }
  // inclusive scan over the block: within warps, then over the warps' totals
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ci = c;
  int ui = u;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long pc = __shfl_up_sync(0xFFFFFFFFu, ci, o);
    const int pu = __shfl_up_sync(0xFFFFFFFFu, ui, o);
    if (lane >= o) {
      ci += pc;
      ui += pu;
    }
  }
  __shared__ long long wc[NT / 32];
  __shared__ int wu[NT / 32];
  if (lane == 31) {
    wc[warp] = ci;
    wu[warp] = ui;
  }
  __syncthreads();
  long long bc = 0;
  int bu = 0;
  for (int w = 0; w < warp; ++w) {
    bc += wc[w];
    bu += wu[w];
  }
  sc->pos[threadIdx.x] = bc + ci - c;
  sc->unit[threadIdx.x] = bu + ui - u;
  if (threadIdx.x == NT - 1) {
    sc->pos[NT] = bc + ci;
    sc->unit[NT] = bu + ui;
  }
  if (publish) {
    long long p = bc + ci - c;
    int uu = bu + ui - u;
    for (int s = s0; s < s1; ++s) {
      l.seg_pos[s] = p;
      l.seg_unit[s] = uu;
      if (chunk == 1) continue;  // nothing of this thread's follows
      const Seg g = seg_load(a, s);
      if (!seg_in(l, g)) continue;
      const int rt = seg_tiles(l, g);
      p += a.pool.Hkv * seg_cost_to(l, g, rt);
      uu += a.pool.Hkv * rt;
    }
    if (threadIdx.x == NT - 1) {
      l.seg_pos[nseg] = bc + ci;
      l.seg_unit[nseg] = bu + ui;
    }
  }
  __syncthreads();
  return sc->pos[NT];
}

// A unit on the line and the segment it is of.
struct Cursor {
  int s;
  Seg g;
  long long pos;   // place of the unit's first key
  int unit;        // the unit's number
  int rt;          // row tiles of the segment
  int h, r, x;     // head, row tile, keys
};

// to the first unit of a segment at or after s (pos and unit are those of s)
template <int NT>
QG_DEVICE bool cursor_seg(const AttnArgs &a, const Line &l, const LineScan<NT> &sc, Cursor *c, int s) {
  const int nseg = 2 * a.b.B;
  for (; s < nseg; ++s) {
    c->g = nseg <= kKeptSegs ? sc.seg[s] : seg_load(a, s);
    if (!seg_in(l, c->g)) continue;
    c->s = s;
    c->rt = seg_tiles(l, c->g);
    c->h = c->r = 0;
    c->x = unit_keys(l, c->g, 0);
    return true;
  }
  return false;
}
// to the next unit; false when the part of the line that ends at `end` has no more (asked first:
// a walk over the empty segments at the end of the line is a chain of loads)
template <int NT>
QG_DEVICE bool cursor_next(const AttnArgs &a, const Line &l, const LineScan<NT> &sc, Cursor *c, long long end) {
  if (c->pos + c->x >= end) return false;
  c->pos += c->x;
  ++c->unit;
  if (++c->r == c->rt) {
    c->r = 0;
    if (++c->h == a.pool.Hkv) return cursor_seg(a, l, sc, c, c->s + 1);
  }
  c->x = unit_keys(l, c->g, c->r);
  return true;
}
// to the unit that holds place `at`
template <int NT>
QG_DEVICE bool cursor_find(const AttnArgs &a, const Line &l, const LineScan<NT> &sc, long long at, Cursor *c) {
  int lo = 0, hi = NT;  // the last thread whose segments start at or before `at`
  while (hi - lo > 1) {
    const int m = (lo + hi) / 2;
    if (sc.pos[m] <= at) lo = m;
    else hi = m;
  }
  const int chunk = (2 * a.b.B + NT - 1) / NT;
  c->pos = sc.pos[lo];
  c->unit = sc.unit[lo];
  if (!cursor_seg(a, l, sc, c, lo * chunk)) return false;
  long long cost;
  while (true) {  // the segment
    cost = seg_cost_to(l, c->g, c->rt);
    if (c->pos + a.pool.Hkv * cost > at) break;
    c->pos += a.pool.Hkv * cost;
    c->unit += a.pool.Hkv * c->rt;
    if (!cursor_seg(a, l, sc, c, c->s + 1)) return false;
  }
  c->h = static_cast<int>(div_pos(at - c->pos, cost));
  c->pos += c->h * cost;
  lo = 0, hi = c->rt;  // the last row tile that starts at or before `at`
  while (hi - lo > 1) {
    const int m = (lo + hi) / 2;
    if (c->pos + seg_cost_to(l, c->g, m) <= at) lo = m;
    else hi = m;
  }
  c->r = lo;
  c->pos += seg_cost_to(l, c->g, lo);
  c->unit += c->h * c->rt + lo;
  c->x = unit_keys(l, c->g, lo);
  return true;
}
// the key tiles [j0, j1) of the cursor's unit in the part [at, end) of the line (none: j0 == j1);
// n: tiles of the unit
QG_DEVICE void cursor_tiles(const Line &l, const Cursor &c, long long at, long long end, int *j0, int *j1, int *n) {
  const int up = (1 << l.kshift) - 1;
  const int o0 = at > c.pos ? static_cast<int>(at - c.pos) : 0;
  const int o1 = end - c.pos < c.x ? static_cast<int>(end - c.pos) : c.x;
  *j0 = (o0 + up) >> l.kshift;
  *j1 = (o1 + up) >> l.kshift;
  *n = (c.x + up) >> l.kshift;
}

// whether the own segment g of sequence b has all the keys its rows see
QG_DEVICE bool seg_whole(const AttnArgs &a, const Seg &g, int b) {
  if (g.prefix) return false;
  if (seq_long(a, b)) return true;
  const int gr = kv_group_of(a.b, b);
  return gr < 0 || kv_prefix_len(a, gr) == 0;
}

// attention over many rows per segment on the tcgen05 tensor cores (qg_attn_tc.cu)
qg_status attn_flags_launch(const AttnArgs &a, bool bf16, cudaStream_t s);
qg_status attn_wide_launch(const AttnArgs &a, bool bf16, cudaStream_t s);
bool attn_wide_supported(int D);

}  // namespace qg
