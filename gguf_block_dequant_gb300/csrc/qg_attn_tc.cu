// qg_attn_tc.cu -- attention for segments with many query rows (a shared prefix under a batch, a
// prompt's own tokens) on the tcgen05 tensor cores.
//
// S = Q K^T and O += P V with the scores and the output in tensor memory; the weights P go back
// to tensor memory as the second product's left operand, so nothing but Q, K and V passes
// through shared memory.  One persistent CTA per SM, warp-specialised:
//   warps 0-3, 4-7  two softmax streams, a thread per row: scores from tensor memory, running
//                   maximum and sum, weights back in 16 bits, at the end the piece's output;
//   warp 8          TMEM allocation and the single MMA-issuing thread;
//   warp 9          the TMA producer: query tiles, and key and value tiles gathered page by page
//                   (a box is 64 elements of the rows a page has in the tile) into
//                   128-byte-swizzled shared memory;
//   warp 10         walks the CTA's part of the line and leaves each piece's description in a small
//                   ring, so that the others keep none of that in registers;
//   warp 11         idle: it completes the warpgroup whose registers the softmax warps take over
//                   (a thread holds its row's 128 scores).
// Two streams keep the tensor cores busy during the exponentials.  With more than 128 rows the
// streams take 128 rows each and share every key tile; with fewer they take the key tiles in
// turn, each with its own maximum, sum and output, joined later like any two pieces.
//
// The running maximum a row's weights refer to is raised (and its output rescaled) only when the
// row's maximum has grown by more than 2^8: weights stay below 2^8, exact in their ratios, and
// the output in tensor memory is hardly ever touched between the products.  Those sums are the tensor
// cores' f32, whose additions round towards zero: n keys are n / 16 of them (twice that with two
// weight terms), each low by up to 2^-23, which at 1 M keys of equal values a piece is 0.3 to 0.5 %.
//
// Measured (one GB300, whole calls replayed from a graph): prompts of 7832 tokens under a prefix of
// 4001, 32 heads over 8 of 128, bf16: 595 us, 1.17 PFLOP/s (0.61 of the measured cuBLAS rate); 64
// one-token sequences under a prefix of 32768 (512 rows a cached head): 77 us, of which this
// kernel about 40.  What bounds it: a pair of 128-row tiles and 128 keys takes about 3500 cycles, with the softmax
// left out 3080 (2048 at the tensor cores' full rate: Q K^T reads both operands from shared
// memory, 8 KB for 64 cycles' work), with a quarter of the products 3200.  So two chains of about one
// length, the products' and scores -> weights -> P V -> next scores (the weights overwrite the
// scores' columns), overlap only to 3500: shortening one alone gains a tenth at most.
// The kernel's time also depends on how much code lies around its hot loops: parts that never run
// cost up to 28 us of the prompts' 595.
// The issuing warp's own instructions count: asking for the tiles' barriers while products are
// queued, and letting go of V before the next scores, took 580 us to 563.  Tried and slower: an MMA
// warp per stream (594 to 757), weights handed over in halves (636 to 645), more chains for the
// maximum and sum (611 to 620), test_wait for try_wait (579 to 612).
#include <cuda.h>

#include <atomic>
#include <mutex>

#include "qg_attn.cuh"
#include "qg_mma.cuh"
#include "qg_pipe.cuh"
#include "qg_tc.cuh"

__device__ unsigned int g_qg_status_attn_tc;  // this translation unit's device status word
static std::atomic<bool> g_launched{false};   // whether a kernel that may set it has been launched

namespace {

using namespace qg;

constexpr int kSoftWarps = 8, kMmaWarp = 8, kProdWarp = 9, kWalkWarp = 10;
constexpr int kPieces = 2;  // descriptions in the ring
constexpr int kThreads = 12 * 32;
// registers: launched with 168 a thread; two warpgroups go up to 208, the third down to 88
constexpr int kRegs = 168, kRegsSoft = 208, kRegsRest = 88;
static_assert(2 * kRegsSoft + kRegsRest <= 3 * kRegs, "the warpgroups' shares come from the launch's total");

// epilogue staging: 32 rows of 64 bytes per softmax warp, 80 bytes apart
constexpr uint32_t kStagePitch = 80, kStageBytes = 32 * kStagePitch;
QG_DEVICE void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
constexpr uint32_t BAR_BYTES = 640;
constexpr uint32_t SCAN_BYTES = (sizeof(LineScan<kThreads>) + 15) / 16 * 16;

template <int D>
struct WideCfg {
  static constexpr uint32_t HALF = 128 * 128;             // bytes of 128 rows x 64 elements
  static constexpr uint32_t TILE = HALF * (D / 64);       // a key, value or query tile
  static constexpr int NST = D == 64 ? 8 : 4;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_KV = 2 * TILE;
  static constexpr uint32_t OFF_BAR = OFF_KV + NST * TILE;
  static constexpr uint32_t OFF_SCAN = OFF_BAR + BAR_BYTES;
  static constexpr uint32_t OFF_STAGE = OFF_SCAN + SCAN_BYTES;
  static constexpr uint32_t SMEM = OFF_STAGE + kSoftWarps * kStageBytes + 1024;  // + alignment slack
  static_assert(SMEM <= 226 * 1024, "one CTA's shared memory");
  static constexpr uint32_t COLS = 512;                   // S0 S1 (128 each), O0 O1 (D each)
};

// A place in the tile ring and the parity of its present use.
template <int N>
struct Ring {
  int st = 0;
  uint32_t par = 0;
  QG_DEVICE void next() {
    if (++st == N) {
      st = 0;
      par ^= 1u;
    }
  }
};

// A worker's part of one unit (j0 == j1: there is no more).
struct Piece {
  Seg g;
  int h, t0;       // cached head, first token row of the unit
  int tokens;      // of the unit
  int j0, j1, jp;  // key tiles; the first jp of the unit are those of a long sequence's prefix
  bool paired;     // two halves of rows; otherwise the streams take the key tiles in turn
  bool alone;      // the piece is all there is of its rows
  bool dirty;      // z0, z1 hold something
  long long slot;  // -1: the workspace has none (token starts that do not rise)
  int z0[2], z1[2];  // of a long sequence's prefix and of the list: first key and end of what loses its infinite
                     // and NaN values (nothing: equal)
};
struct WideBars {
  Piece piece[kPieces];
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t full[8], empty[8];
  uint64_t q_full, q_empty, tail;
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint32_t tmem;
  int abort;
};

using Scan = LineScan<kThreads>;
struct Walk {
  const Scan *scan;
  Cursor cur;
  long long at, end;
  int w;
};
QG_DEVICE bool walk_next(const AttnArgs &a, Walk *k, Piece *p) {
  const Line &l = a.wide;
  Cursor &c = k->cur;
  while (c.pos < k->end) {
    int n;
    cursor_tiles(l, c, k->at, k->end, &p->j0, &p->j1, &n);
    const bool some = p->j0 < p->j1;
    if (some) {
      p->g = c.g;
      p->h = c.h;
      p->t0 = c.g.t0 + c.r * l.tpt;
      p->tokens = min(l.tpt, c.g.nt - c.r * l.tpt);
      p->paired = p->tokens > l.tpt / 2;
      p->jp = tiles_of(l, c.g.plen);
      p->alone = p->paired && p->j0 == 0 && p->j1 == n && seg_whole(a, c.g, c.s >> 1);
      p->slot = piece_slot(l, c.unit, k->w);
    }
    if (!cursor_next(a, l, *k->scan, &c, k->end)) c.pos = k->end;
    if (some) return true;
  }
  return false;
}

// Bounded wait by the SM's own clock: gives up when another role has, or after a.wait_cycles.
QG_DEVICE bool clock_wait(const AttnArgs &a, uint64_t *b, uint32_t parity, WideBars *bar) {
  if (mbar_try_wait(b, parity)) return true;
  const long long t0 = clock64();
  volatile int *abort = &bar->abort;
  while (true) {
    if (mbar_try_wait(b, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > a.wait_cycles) break;
  }
  *abort = 1;
  atomicOr(&g_qg_status_attn_tc, QG_STATUS_BIT_TIMEOUT);
  return false;
}
// the whole warp waits, and gives up as a whole
QG_DEVICE bool warp_wait(const AttnArgs &a, uint64_t *b, uint32_t parity, WideBars *bar) {
  return __all_sync(0xFFFFFFFFu, clock_wait(a, b, parity, bar));
}

// ---- the walk -----------------------------------------------------------------------------------
// Zero times an infinite or NaN value is not zero.  So where some row of a unit must not see a key,
// such values of its leave the tile before the product, and the softmax warps add them to the rows
// that do see it.  The keys in question are those at the new tokens' own positions, since a token
// sees all before its own: value_flags_kernel has a bit for each.
//
QG_DEVICE bool any_flag(const AttnArgs &a, int row, int ta, int tb, int lane) {  // of tokens [ta, tb), and of a few around them
  const uint32_t *flags = a.value_flags + static_cast<size_t>(row) * ((a.b.T + 31) / 32);
  uint32_t f = 0;
#pragma unroll 1
  for (int w = (ta >> 5) + lane; 32 * w < tb; w += 32) f |= __ldcg(flags + w);
  return __any_sync(0xFFFFFFFFu, f != 0);
}
QG_DEVICE void piece_values(const AttnArgs &a, Piece *p, int lane) {
  p->dirty = false;
  p->z0[0] = p->z1[0] = p->z0[1] = p->z1[1] = 0;
  if (!a.value_flags) return;
  const Seg &g = p->g;
  const int h = p->h, te = g.t0 + g.nt;
  // own positions: token t has key t + d
  const int d = g.len - g.nt - g.t0;
  const int ta = max(p->t0 + 1, (max(p->j0 - p->jp, 0) << kWideShift) - d), tb = min(te, ((p->j1 - p->jp) << kWideShift) - d);
  if (!g.prefix && any_flag(a, a.pool.Hkv + h, ta, tb, lane)) {
    p->dirty = true;
    p->z0[1] = max(ta + d, 0);
    p->z1[1] = tb + d;
  }
  // positions in a prefix, of tokens before their sequence's first slot: under a shared one the unit's
  // tokens and those that follow of its last sequence, else the long sequence's.  Rare: all of the prefix is taken.
  if ((g.prefix || (g.plen && g.len < g.nt)) &&
      any_flag(a, h, p->t0, g.prefix ? min(te, p->t0 + p->tokens + a.wide.tpt / 2) : te, lane)) {
    p->dirty = true;
    (g.prefix ? p->z1[1] : p->z1[0]) = g.prefix ? g.len : g.plen;
  }
}
QG_DEVICE void walk_line(const AttnArgs &a, Walk walk, WideBars *bar, int lane) {
  for (uint32_t n = 0;; ++n) {
    Piece p;
    const bool more = walk_next(a, &walk, &p);
    if (!more) p.j0 = p.j1 = 0;
    else if (p.slot < 0 && !p.alone && lane == 0) atomicOr(&g_qg_status_attn_tc, QG_STATUS_BIT_ID);
    if (more) piece_values(a, &p, lane);
    const uint32_t i = n % kPieces;
    if (!warp_wait(a, &bar->piece_empty[i], ((n / kPieces) & 1) ^ 1, bar)) return;
    if (lane == 0) {
      bar->piece[i] = p;
      mbar_arrive(&bar->piece_full[i]);
    }
    __syncwarp();
    if (!more) return;
  }
}
// the n-th piece, nullptr at the end (or after an abort)
QG_DEVICE const Piece *piece_get(const AttnArgs &a, WideBars *bar, uint32_t n) {
  const uint32_t i = n % kPieces;
  if (!warp_wait(a, &bar->piece_full[i], (n / kPieces) & 1, bar)) return nullptr;
  const Piece *p = &bar->piece[i];
  return p->j0 < p->j1 ? p : nullptr;
}
QG_DEVICE void piece_done(WideBars *bar, uint32_t n, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar->piece_empty[n % kPieces]);
}

// ---- producer ---------------------------------------------------------------------------------
QG_DEVICE void tma_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}
QG_DEVICE void tma_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// Tensor maps of a call: queries (D, Hq, tokens), keys and values (D, page rows, heads, pages).  A page
// number outside the pool is a coordinate outside the map and reads zeros.
struct WideMaps {
  CUtensorMap q, k, v;
};

template <int D, bool BF16>
QG_DEVICE void produce(const AttnArgs &a, const WideMaps &maps, uint8_t *smem, WideBars *bar, int lane) {
  using C = WideCfg<D>;
  constexpr int H = D / 64;              // 64-element halves of a row
  const uint32_t sb = smem_u32(smem);
  const int shift = a.pool.page_shift;
  const int bshift = min(shift, 7), rows = 1 << bshift;  // rows of a box
  const int half = a.wide.tpt / 2;
  Ring<C::NST> ring;
  uint32_t np = 0, ntail = 0;
  for (const Piece *pp; (pp = piece_get(a, bar, np)) != nullptr; piece_done(bar, np++, lane)) {
    const Piece p = *pp;
    if (!warp_wait(a, &bar->q_empty, (np & 1) ^ 1, bar)) return;
    const int ns = p.paired ? 2 : 1;
    if (lane == 0) mbar_arrive_expect_tx(&bar->q_full, static_cast<uint32_t>(ns * H * half * a.Gq) * 128u);
    __syncwarp();
    // a box is half a row tile: its rows are tokens by heads, the order of the tile's rows
    // (tokens past the unit's belong to rows that nobody reads)
    if (lane < ns * H)
      tma_3d(sb + C::OFF_Q + lane * C::HALF, &maps.q, 64 * (lane % H), p.h * a.Gq, p.t0 + (lane / H) * half, &bar->q_full);
    for (int j = p.j0; j < p.j1; ++j) {
      const bool pre = j < p.jp;
      const int key0 = (pre ? j : j - p.jp) * kWideKeys;
      const int32_t *table = pre ? p.g.ptable : p.g.table;
      const int left = min(kWideKeys, (pre ? p.g.plen : p.g.len) - key0);
      const int boxes = (left + rows - 1) >> bshift;
      int page[4];  // this lane's boxes: lane, lane + 32, ...
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        page[i] = 0;
        if (lane + 32 * i < boxes) {
          page[i] = __ldg(table + ((key0 + ((lane + 32 * i) << bshift)) >> shift));
          bad |= page[i] < 0 || page[i] >= a.pool.n_pages;
        }
      }
      if (bad) atomicOr(&g_qg_status_attn_tc, QG_STATUS_BIT_ID);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ring.next()) {
        const int st = ring.st;
        if (!warp_wait(a, &bar->empty[st], ring.par ^ 1u, bar)) return;
        // a value tile is held back when values past the last key are to become zeros (whatever their
        // rows or the stage held), or infinite and NaN ones.  Keys may be anything: their scores are
        // replaced.
        int z0 = 0, z1 = 0;  // rows of the latter
        if (kv && p.dirty) {
          z0 = max((pre ? p.z0[0] : p.z0[1]) - key0, 0);
          z1 = min((pre ? p.z1[0] : p.z1[1]) - key0, left);
        }
        const bool held = kv && (left < kWideKeys || z0 < z1);
        uint64_t *land = held ? &bar->tail : &bar->full[st];
        if (lane == 0) mbar_arrive_expect_tx(land, static_cast<uint32_t>(boxes * H * rows) * 128u);
        __syncwarp();
        const uint32_t off = C::OFF_KV + static_cast<uint32_t>(st) * C::TILE;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int b = lane + 32 * i;
          if (b < boxes) {
            const int row = (key0 + (b << bshift)) & ((1 << shift) - 1);
#pragma unroll
            for (int h = 0; h < H; ++h)
              tma_4d(sb + off + h * C::HALF + static_cast<uint32_t>(b << bshift) * 128u, kv ? &maps.v : &maps.k, 64 * h, row,
                     p.h, page[i], land);
          }
        }
        if (held) {
          if (!warp_wait(a, &bar->tail, ntail++ & 1, bar)) return;
#pragma unroll 1
          for (int h = 0; h < H; ++h) {
            uint4 *v = reinterpret_cast<uint4 *>(smem + off + h * C::HALF);
#pragma unroll 4
            for (int x = left * 8 + lane; x < kWideKeys * 8; x += 32) v[x] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
            for (int x = z0 * 8 + lane; x < z1 * 8; x += 32) v[x] = make_finite<BF16>(v[x]);
          }
          fence_proxy_async_smem();  // stored through the generic proxy, read by the tensor cores
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar->full[st]);
        }
      }
    }
  }
}

// ---- MMA issue --------------------------------------------------------------------------------
template <int D, bool BF16, bool OUT32>
QG_DEVICE void issue_mma(const AttnArgs &a, uint32_t smem, WideBars *bar, int lane) {
  using C = WideCfg<D>;
  constexpr uint32_t id_s = make_idesc16(128, kWideKeys, BF16, false), id_o = make_idesc16(128, D, BF16, true);
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, bar->tmem, 0), el = elect_lane();
  auto wait = [&](uint64_t *b, uint32_t parity) {
    const bool r = warp_wait(a, b, parity, bar);
    tc_fence_after();
    return r;
  };
  uint32_t np = 0;
  uint32_t n_p[2] = {0, 0};   // weights taken from each stream
  uint32_t n_o[2] = {0, 0};   // outputs begun for each stream
  // descriptors differ in their start address alone (low word, 16-byte units)
  const uint64_t dq = sw128_desc(smem + C::OFF_Q), dk = sw128_desc(smem + C::OFF_KV),
                 dv = sw128_desc_mn(smem + C::OFF_KV, C::HALF);
  auto scores = [&](int s, int qt, int st) {  // S_s = Q_qt K^T
    const uint64_t q = dq + static_cast<uint32_t>(qt) * (C::TILE / 16), k = dk + static_cast<uint32_t>(st) * (C::TILE / 16);
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      const uint32_t o = ((x >> 2) * C::HALF + (x & 3) * 32) / 16;
      tc_mma_el(el, tmem + 128u * s, q + o, k + o, id_s, x != 0);
    }
    tc_commit_el(el, &bar->s_full[s]);
  };
  auto output = [&](int s, int st, bool first) {  // O_s += P_s V
    const uint64_t v = dv + static_cast<uint32_t>(st) * (C::TILE / 16);
    const uint32_t ps = tmem + 128u * s, o = tmem + 256u + D * s;
#pragma unroll
    for (int x = 0; x < kWideKeys / 16; ++x) {
      const uint32_t p = ps + 32u * (x >> 1) + 8u * (x & 1);
      tc_mma_ta_el(el, o, p, v + x * (2048 / 16), id_o, x == 0 ? !first : 1u);
      if constexpr (OUT32) tc_mma_ta_el(el, o, p + 16u, v + x * (2048 / 16), id_o, 1);
    }
  };
  auto landed = [&](const Ring<C::NST> &r) { return wait(&bar->full[r.st], r.par); };
  auto release = [&](const Ring<C::NST> &r) { tc_commit_el(el, &bar->empty[r.st]); };
  // weights of stream s are in tensor memory; before its first output of the piece, the last
  // piece's has been read
  auto weights = [&](int s, bool first) {
    if (!wait(&bar->p_full[s], n_p[s]++ & 1)) return false;
    if (first && !wait(&bar->o_empty[s], (n_o[s]++ & 1) ^ 1)) return false;
    return true;
  };
  // tiles come as K0 V0 K1 V1 ...; kt and vt are the next key and value tiles to be used
  Ring<C::NST> kt, vt;
  vt.next();
  for (const Piece *pp; (pp = piece_get(a, bar, np)) != nullptr; ++np) {
    const int n = pp->j1 - pp->j0;
    const bool paired = pp->paired;
    piece_done(bar, np, lane);
    if (!wait(&bar->q_full, np & 1)) return;
    if (paired) {
      for (int j = 0; j <= n; ++j) {
        // The tiles' barriers are asked while products are queued, not between a stream's weights and
        // its products: K_j before its first scores, V_j (the next to be used) before its second.
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (j > 0) {
            if (!weights(s, j == 1)) return;
            output(s, vt.st, j == 1);
            if (j == n) tc_commit_el(el, &bar->o_full[s]);
            if (s == 1) {
              release(vt);
              vt.next();
              vt.next();
            }
          }
          if (j < n) {
            if (s == 0 && !landed(kt)) return;
            if (s == 1 && !landed(vt)) return;
            scores(s, s, kt.st);
          }
        }
        if (j < n) {
          release(kt);
          kt.next();
          kt.next();
          if (j == n - 1) tc_commit_el(el, &bar->q_empty);
        }
      }
    } else {
      for (int j = 0; j < n + 2; ++j) {
        const int s = j & 1;
        if (j >= 2 && j - 2 < n) {
          if (!landed(vt) || !weights(s, j < 4)) return;
          output(s, vt.st, j < 4);
          release(vt);
          vt.next();
          vt.next();
          if (j >= n) tc_commit_el(el, &bar->o_full[s]);
        }
        if (j < n) {
          if (!landed(kt)) return;
          scores(s, 0, kt.st);
          release(kt);
          kt.next();
          kt.next();
          if (j == n - 1) tc_commit_el(el, &bar->q_empty);
        }
      }
    }
  }
}

// ---- softmax ----------------------------------------------------------------------------------
// Adds the values that left the piece's tiles to the rows that see them (infinite
// or NaN: whatever their positive weight is).  Rare, and read from the cache once more.  lim_*: keys
// that this thread's row sees of a long sequence's prefix and of the list.
template <int D, bool BF16>
__device__ __noinline__ void add_zeroed(const AttnArgs &a, const Piece &p, uint32_t to, int s, int lim_prefix, int lim_list) {
  const int shift = a.pool.page_shift;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int lim = part ? lim_list : lim_prefix;
    const int z0 = p.z0[part], z1 = min(p.z1[part], __reduce_max_sync(0xFFFFFFFFu, lim));
    const int32_t *table = part ? p.g.table : p.g.ptable;
#pragma unroll 1
    for (int c = 0; c < D && z0 < z1; c += 16) {
      float o[16];
      tmem_ld16(to + c, o);
#pragma unroll 1
      for (int key = z0; key < z1; ++key) {
        const int j = (key >> kWideShift) + (part ? p.jp : 0);
        if (!p.paired && ((j - p.j0) & 1) != s) continue;  // the other stream's tile
        const int page = __ldg(table + (key >> shift));
        if (page < 0 || page >= a.pool.n_pages) continue;
        const uint4 *v = reinterpret_cast<const uint4 *>(a.pool.v + page * a.pool.page_stride +
                                                         (key & ((1 << shift) - 1)) * a.pool.token_stride +
                                                         p.h * a.pool.head_stride + c);
        const bool sees = key < lim;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 q = __ldg(v + i);
          const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (sees && nonfinite16<BF16>(w[e])) o[8 * i + 2 * e] += lo16<BF16>(w[e]);
            if (sees && nonfinite16<BF16>(w[e] >> 16)) o[8 * i + 2 * e + 1] += hi16<BF16>(w[e]);
          }
        }
      }
      uint32_t r[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(o[i]);
      tmem_st16(to + c, r);
      tmem_st_wait();
    }
  }
}

template <int D, bool BF16, bool OUT32>
QG_DEVICE void softmax(const AttnArgs &a, WideBars *bar, int s, int warp4, int lane, uint32_t stage) {
  const uint32_t lanes = static_cast<uint32_t>(32 * warp4) << 16;
  const uint32_t ts = bar->tmem + lanes + 128u * s, to = bar->tmem + lanes + 256u + D * s;
  const int row = 32 * warp4 + lane, half = a.wide.tpt / 2;
  const float sl = fabsf(a.scale_log2);
  const bool neg = a.scale_log2 < 0.f;
  uint32_t n_s = 0, n_o = 0, np = 0;
  for (const Piece *pp; (pp = piece_get(a, bar, np)) != nullptr; piece_done(bar, np++, lane)) {
    const Piece &p = *pp;
    // this thread's row
    const int sub = p.paired ? s : 0;
    const int tok = min(half, p.tokens - sub * half);
    const bool valid = row < tok * a.Gq && (p.alone || p.slot >= 0);
    const int t = p.t0 + sub * half + (valid ? row / a.Gq : 0);
    const int lim = valid ? row_limit(a, p.g, t) : 0, limp = valid ? row_prefix_limit(p.g, t) : 0;
    const int all = __reduce_min_sync(0xFFFFFFFFu, valid ? lim : 0x7FFFFFFF);
    const int allp = __reduce_min_sync(0xFFFFFFFFu, valid ? limp : 0x7FFFFFFF);
    // the row's maximum that its weights refer to, and the reference itself: the maximum in log2
    // units less what f16 weights are raised by (2^7, up to 2^15 with the lag: the second term of a
    // small one would otherwise lie among the subnormals).  Rescaling uses the references as they
    // were rounded.
    constexpr float RAISE = BF16 ? 0.f : 7.f;
    float m = -INFINITY, ref = -INFINITY, l = 0.f;
    const bool idle = !__any_sync(0xFFFFFFFFu, valid);  // no row of this warp is anyone's: whatever its weights are
    const int step = p.paired ? 1 : 2, first = p.paired ? p.j0 : p.j0 + s, j1 = p.j1, jp = p.jp;
    for (int j = first; j < j1; j += step) {
      if (!warp_wait(a, &bar->s_full[s], n_s++ & 1, bar)) return;
      tc_fence_after();
      if (idle) {
        if (lane == 0) mbar_arrive(&bar->p_full[s]);
        continue;
      }
      const bool pre = j < jp;
      const int key0 = (pre ? j : j - jp) * kWideKeys;
      const int left = (pre ? limp : lim) - key0;  // keys of the tile that the row sees
      const bool masked = key0 + kWideKeys > (pre ? allp : all);
      float x[kWideKeys];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32_nowait(ts + 32 * c, &x[32 * c]);
      tmem_ld_wait(x);
      if (neg) {
#pragma unroll
        for (int i = 0; i < kWideKeys; ++i) x[i] = -x[i];
      }
      if (masked) {
#pragma unroll
        for (int i = 0; i < kWideKeys; ++i)
          if (i >= left) x[i] = -INFINITY;
      }
      float mx4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int i = 4; i < kWideKeys; i += 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) mx4[e] = fmaxf(mx4[e], x[i + e]);
      }
      const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
      // the reference maximum moves when the row's outgrew it by 2^8 (or it is the first)
      const bool move = mx > m && (m == -INFINITY || (mx - m) * sl > 8.0f);
      float al = 1.0f;
      if (move) {
        const float r = fmaf(mx, sl, -RAISE);
        al = ex2(ref - r);  // 0 from -inf
        m = mx;
        ref = r;
        l *= al;
      }
      if (j != first && __any_sync(0xFFFFFFFFu, move)) {
        // every product into O has finished: S's barrier came after them
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          float o[16];
          tmem_ld16(to + 16 * c, o);
          uint32_t r[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(o[i] * al);
          tmem_st16(to + 16 * c, r);
        }
      }
      const float nm = ref == -INFINITY ? 0.f : -ref;
      f2 sum = mk2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float *y = &x[32 * c];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const f2 e = fma2(mk2(y[i], y[i + 1]), mk2(sl, sl), mk2(nm, nm));
          y[i] = ex2(e.x);
          y[i + 1] = ex2(e.y);
        }
        if (masked) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i >= left) y[i] = 0.f;
        }
        uint32_t hi[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          sum = add2(sum, mk2(y[i], y[i + 1]));
          hi[i / 2] = pack16<BF16>(y[i], y[i + 1]);
        }
        tmem_st16(ts + 32 * c, hi);
        if constexpr (OUT32) {  // what the rounding left
          uint32_t lo[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            lo[i / 2] = pack16<BF16>(y[i] - lo16<BF16>(hi[i / 2]), y[i + 1] - hi16<BF16>(hi[i / 2]));
          tmem_st16(ts + 32 * c + 16, lo);
        }
      }
      l += sum.x + sum.y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->p_full[s]);
    }
    // ---- the piece's output
    const bool any = first < j1;
    if (any) {
      if (!warp_wait(a, &bar->o_full[s], n_o++ & 1, bar)) return;
      tc_fence_after();
      if (p.dirty) add_zeroed<D, BF16>(a, p, to, s, limp, lim);
    }
    const float inv = !p.alone ? 1.0f : l == 0.f ? 0.f : 1.0f / l;
    const size_t prow = p.slot * kWideRows + s * kWideHalf + row;
    if (valid && !p.alone) a.wide.part_ml[prow] = make_float2(ref, l);
    if (any) {
      const bool wide_out = !p.alone || OUT32;  // f32 values; otherwise 16-bit ones
      const size_t orow = (static_cast<size_t>(t) * a.Hq + p.h * a.Gq + (valid ? row % a.Gq : 0)) * D;
      uint8_t *mine = nullptr;
      if (valid)
        mine = !p.alone ? reinterpret_cast<uint8_t *>(a.wide.part_o + prow * D)
               : OUT32  ? reinterpret_cast<uint8_t *>(static_cast<float *>(a.out) + orow)
                        : reinterpret_cast<uint8_t *>(static_cast<uint16_t *>(a.out) + orow);
      // 64 bytes of every row at a time through the warp's staging rows, so that four lanes write
      // a row's 64 bytes together: a thread writing its own row costs a cache line per lane and
      // store, and held up every other warp's loads for thousands of cycles
      uint8_t *dst[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dst[i] = reinterpret_cast<uint8_t *>(__shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(mine), 8 * i + (lane >> 2)));
      const uint32_t put = stage + lane * kStagePitch, get = stage + (lane >> 2) * kStagePitch + (lane & 3) * 16;
      const int cols = wide_out ? 16 : 32;
#pragma unroll 1
      for (int c = 0; c < D; c += cols) {
        float o[32];
        uint32_t q[16];
        tmem_ld16(to + c, reinterpret_cast<float(&)[16]>(o[0]));
        if (wide_out) {
#pragma unroll
          for (int i = 0; i < 16; ++i) q[i] = __float_as_uint(o[i] * inv);
        } else {
          tmem_ld16(to + c + 16, reinterpret_cast<float(&)[16]>(o[16]));
#pragma unroll
          for (int i = 0; i < 16; ++i) q[i] = pack16<BF16>(o[2 * i] * inv, o[2 * i + 1] * inv);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) sts_v4(put + 16 * i, q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = lds_v4(get + 8 * i * kStagePitch);
          if (dst[i]) {
            *reinterpret_cast<uint4 *>(dst[i] + (lane & 3) * 16) = v;
            dst[i] += 64;
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->o_empty[s]);
    }
  }
}

// A bit for each new token and cached head: the value at the token's position has infinite or NaN elements.
// Positions in the prefix (of tokens before their sequence's first slot) and own ones have words of
// their own, [2][heads][tokens / 32].  A warp per 32 tokens and head; reads the new tokens' values once
// (prompts of 7832 tokens, 16 MB: 8.5 us, a launch and a chain of look-ups more than the bytes).  Looked up
// inside the wide kernel, a piece ahead or in the landed tiles, it cost the call 40 to 120 us.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) value_flags_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int CH = D / 8, RPL = 32 / CH;  // 16-byte chunks of a row, rows a load of the warp takes
  const int lane = threadIdx.x & 31, words = (a.b.T + 31) / 32;
  pdl_wait();
  pdl_launch_dependents();
  const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(words) * a.pool.Hkv) return;
  const int h = static_cast<int>(item / words), w = static_cast<int>(item - static_cast<long long>(h) * words);
  // lane's token: where its value lies (-1: nowhere)
  long long off = -1;
  bool in_prefix = false;
  const int t = 32 * w + lane, shift = a.pool.page_shift;
  const int b = t < a.b.T ? kv_seq_of(a.b, t) : -1;
  if (b >= 0) {
    int slot = kv_own_len(a.b, shift, b) - (kv_tok(a.b, b + 1) - t);
    const int32_t *table = a.b.pages + static_cast<size_t>(b) * a.b.max_pages;
    if (slot < 0) {
      const int g = kv_group_of(a.b, b);
      if (g >= 0) {
        in_prefix = true;
        slot += kv_prefix_len(a, g);
        table = kv_prefix_table(a, g);
      }
    }
    if (slot >= 0) {
      const int page = __ldg(table + (slot >> shift));
      if (page >= 0 && page < a.pool.n_pages)
        off = page * a.pool.page_stride + (slot & ((1 << shift) - 1)) * a.pool.token_stride + h * a.pool.head_stride;
    }
  }
  uint32_t f = 0;
#pragma unroll 8
  for (int i = 0; i < 32 / RPL; ++i) {
    const long long o = __shfl_sync(0xFFFFFFFFu, off, i * RPL + lane / CH);
    const uint4 v = o < 0 ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4 *>(a.pool.v + o) + lane % CH);
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, any_nonfinite<BF16>(v) != 0);
#pragma unroll
    for (int r = 0; r < RPL; ++r)
      if (some >> (CH * r) & ((1u << CH) - 1u)) f |= 1u << (i * RPL + r);
  }
  const uint32_t pre = __ballot_sync(0xFFFFFFFFu, in_prefix);
  if (lane == 0) {
    a.value_flags[static_cast<size_t>(h) * words + w] = f & pre;
    a.value_flags[static_cast<size_t>(a.pool.Hkv + h) * words + w] = f & ~pre;
  }
}

template <int D, bool BF16, bool OUT32>
__global__ void __launch_bounds__(kThreads, 1) attn_wide_kernel(const __grid_constant__ AttnArgs a,
                                                                   const __grid_constant__ WideMaps maps) {
  using C = WideCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  WideBars *bar = reinterpret_cast<WideBars *>(smem + C::OFF_BAR);
  Scan *scan = reinterpret_cast<Scan *>(smem + C::OFF_SCAN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&bar->full[i], 1);
      mbar_init(&bar->empty[i], 1);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&bar->piece_full[i], 1);
      mbar_init(&bar->piece_empty[i], kSoftWarps + 2);
    }
    mbar_init(&bar->q_full, 1);
    mbar_init(&bar->tail, 1);
    mbar_init(&bar->q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->s_full[s], 1);
      mbar_init(&bar->p_full[s], 4);
      mbar_init(&bar->o_full[s], 1);
      mbar_init(&bar->o_empty[s], 4);
    }
    bar->abort = 0;
    fence_mbar_init();
  }
  // No wait for the narrow kernel here: it has waited for all that came before the call, and this
  // one reads and writes nothing of its.  A CTA starts as soon as its SM is free; the wait at the
  // end keeps the order for what follows.
  const Line &ln = a.wide;
  const long long total = line_scan<kThreads>(a, ln, scan, blockIdx.x == 0);
  const int nw = line_workers(ln, total);
  Walk walk;
  walk.scan = scan;
  walk.w = static_cast<int>(blockIdx.x);
  if (total == 0 || walk.w >= nw) {
    pdl_wait();
    return;
  }
  const Cut cut = line_cut(total, nw);
  walk.at = line_start(cut, walk.w);
  walk.end = line_start(cut, walk.w + 1);
  if (walk.at >= walk.end || !cursor_find(a, ln, *scan, walk.at, &walk.cur)) {  // the same for the whole block
    pdl_wait();
    return;
  }
  if (warp == kMmaWarp) tmem_alloc(&bar->tmem, C::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t sb = smem_u32(smem);
  if (warp < kSoftWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    softmax<D, BF16, OUT32>(a, bar, warp >> 2, warp & 3, lane, sb + C::OFF_STAGE + warp * kStageBytes);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == kMmaWarp) {
      issue_mma<D, BF16, OUT32>(a, sb, bar, lane);
      if (lane == 0) {
        // after an abort the products in flight finish before the tensor memory is released (a
        // normal run waited for each); q_empty counts pieces, so any further phase will do
        if (*static_cast<volatile int *>(&bar->abort)) {
          const uint64_t st = *reinterpret_cast<volatile uint64_t *>(&bar->q_empty);
          tc_commit(&bar->q_empty);
          for (uint32_t i = 0; i < (1u << 16) && *reinterpret_cast<volatile uint64_t *>(&bar->q_empty) == st; ++i)
            __nanosleep(32);
        }
      }
    } else if (warp == kProdWarp) {
      produce<D, BF16>(a, maps, smem, bar, lane);
      // after an abort the copies in flight land before the CTA's shared memory is released
      if (*static_cast<volatile int *>(&bar->abort)) __nanosleep(1000000);
    } else if (warp == kWalkWarp) {
      walk_line(a, walk, bar, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(bar->tmem, C::COLS);
  }
  pdl_wait();
  pdl_launch_dependents();  // not before: blocks that wait beside this kernel cost it 5 %
}

bool make_maps(const AttnArgs &a, bool bf16, WideMaps *m) {
  const auto enc = encode_fn();
  if (!enc) return false;
  const CUtensorMapDataType type = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  const cuuint64_t D = static_cast<cuuint64_t>(a.D), ps = 1ull << a.pool.page_shift;
  {
    const cuuint64_t dim[3] = {D, static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.b.T)};
    const cuuint64_t stride[2] = {D * 2, static_cast<cuuint64_t>(a.q_stride) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.Gq), static_cast<cuuint32_t>(a.wide.tpt / 2)};
    if (enc(&m->q, type, 3, const_cast<uint16_t *>(a.q), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  const cuuint64_t dim[4] = {D, ps, static_cast<cuuint64_t>(a.pool.Hkv), static_cast<cuuint64_t>(a.pool.n_pages)};
  // a dimension of one has no stride of its own: any valid one
  const cuuint64_t stride[3] = {ps > 1 ? static_cast<cuuint64_t>(a.pool.token_stride) * 2 : D * 2,
                                a.pool.Hkv > 1 ? static_cast<cuuint64_t>(a.pool.head_stride) * 2 : D * 2,
                                a.pool.n_pages > 1 ? static_cast<cuuint64_t>(a.pool.page_stride) * 2 : D * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(ps < kWideKeys ? ps : kWideKeys), 1, 1};
  for (int i = 0; i < 2; ++i)
    if (enc(i ? &m->v : &m->k, type, 4, i ? a.pool.v : a.pool.k, dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

static_assert(sizeof(WideBars) <= BAR_BYTES, "barriers and descriptions");

template <int D, bool BF16, bool OUT32>
qg_status wide_run(const AttnArgs &a, cudaStream_t s) {
  const auto k = attn_wide_kernel<D, BF16, OUT32>;
  static const bool fits = qg::split_fits(reinterpret_cast<const void *>(k), kRegs);  // the split above
  WideMaps maps;
  if (!fits || !make_maps(a, BF16, &maps) || !set_smem_attr(reinterpret_cast<const void *>(k), WideCfg<D>::SMEM))
    return QG_ECUDA;
  g_launched = true;
  return launch_pdl(k, dim3(static_cast<unsigned>(a.wide.workers)), dim3(kThreads), WideCfg<D>::SMEM, s, a, maps) ==
                 cudaSuccess
             ? QG_OK
             : QG_ECUDA;
}

}  // namespace

namespace qg {

bool attn_wide_supported(int D) { return D == 64 || D == 128; }

// before the narrow kernel, whose wait orders it before the wide one
qg_status attn_flags_launch(const AttnArgs &a, bool bf16, cudaStream_t s) {
  const long long items = static_cast<long long>((a.b.T + 31) / 32) * a.pool.Hkv;
  const dim3 grid(static_cast<unsigned>((items + 7) / 8)), block(256);
  cudaError_t e;
  if (a.D == 64) e = bf16 ? launch_pdl(value_flags_kernel<64, true>, grid, block, 0, s, a) : launch_pdl(value_flags_kernel<64, false>, grid, block, 0, s, a);
  else e = bf16 ? launch_pdl(value_flags_kernel<128, true>, grid, block, 0, s, a) : launch_pdl(value_flags_kernel<128, false>, grid, block, 0, s, a);
  return e == cudaSuccess ? QG_OK : QG_ECUDA;
}

qg_status attn_wide_launch(const AttnArgs &a, bool bf16, cudaStream_t s) {
  if (a.D == 64) {
    if (bf16) return a.out32 ? wide_run<64, true, true>(a, s) : wide_run<64, true, false>(a, s);
    return a.out32 ? wide_run<64, false, true>(a, s) : wide_run<64, false, false>(a, s);
  }
  if (bf16) return a.out32 ? wide_run<128, true, true>(a, s) : wide_run<128, true, false>(a, s);
  return a.out32 ? wide_run<128, false, true>(a, s) : wide_run<128, false, false>(a, s);
}

unsigned int read_status_attn_tc(bool clear) {
  unsigned int v = 0;
  if (!g_launched) return v;
  if (cudaMemcpyFromSymbol(&v, g_qg_status_attn_tc, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_qg_status_attn_tc, &z, sizeof(z));
  }
  return v;
}

}  // namespace qg
