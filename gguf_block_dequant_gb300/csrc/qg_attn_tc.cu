// qg_attn_tc.cu -- attention for segments with many query rows (a shared prefix under a batch, a
// prompt's own tokens) on the tcgen05 tensor cores.
//
// S = Q K^T and O += P V with the scores and the output in tensor memory; the weights P go back
// to tensor memory as the second product's left operand, so nothing but Q, K and V passes
// through shared memory.  One persistent CTA per SM, warp-specialised:
//   warps 0-3, 4-7  two softmax streams, a thread per row: scores from tensor memory, running
//                   maximum and sum, weights back in 16 bits, at the end the piece's output;
//   warp 8          TMEM allocation and the single MMA-issuing thread;
//   warps 9-11      producers: gather K and V rows through the page list (16-byte cp.async, the
//                   pages may be of any size and stride) into 128-byte-swizzled tiles.
// Two streams keep the tensor cores busy during the exponentials.  With more than 128 rows the
// streams take 128 rows each and share every key tile; with fewer they take the key tiles in
// turn, each with its own maximum, sum and output, joined later like any two pieces.
//
// The running maximum a row's weights refer to is raised (and its output rescaled) only when the
// row's maximum has grown by more than 2^8: weights stay below 2^8, exact in their ratios, and
// the output in tensor memory is hardly ever touched between the products.
#include "qg_attn.cuh"
#include "qg_mma.cuh"
#include "qg_tc.cuh"

__device__ unsigned int g_qg_status_attn_tc;  // this translation unit's device status word

namespace {

using namespace qg;

constexpr int kSoftWarps = 8, kMmaWarp = 8, kProdWarps = 3;  // 12 warps: 168 registers a thread
constexpr int kThreads = (kSoftWarps + 1 + kProdWarps) * 32;
constexpr int kLag = 2;  // copies a producer keeps in flight behind the newest

template <int D>
struct WideCfg {
  static constexpr uint32_t HALF = 128 * 128;             // bytes of 128 rows x 64 elements
  static constexpr uint32_t TILE = HALF * (D / 64);       // a key, value or query tile
  static constexpr int NST = D == 64 ? 8 : 4;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_KV = 2 * TILE;
  static constexpr uint32_t OFF_BAR = OFF_KV + NST * TILE;
  static constexpr uint32_t SMEM = OFF_BAR + 256 + 1024;  // + alignment slack
  static constexpr uint32_t COLS = 512;                   // S0 S1 (128 each), O0 O1 (D each)
};

struct WideBars {
  uint64_t full[8], empty[8];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint32_t tmem;
  int abort;
};

// A worker's part of one unit, as every role of the CTA works it out for itself.
struct Piece {
  Seg g;
  int h, t0;       // cached head, first token row of the unit
  int tokens;      // of the unit
  int j0, j1;      // key tiles
  bool paired;     // two halves of rows; otherwise the streams take the key tiles in turn
  bool alone;      // the piece is all there is of its rows
  size_t slot;
};
struct Walk {
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
      p->alone = p->paired && !c.g.prefix && p->j0 == 0 && p->j1 == n && !has_prefix(a, c.s - a.b.G);
      p->slot = static_cast<size_t>(c.unit) + static_cast<size_t>(k->w);
    }
    if (!cursor_next(a, l, &c)) c.pos = k->end;
    if (some) return true;
  }
  return false;
}

// Bounded wait by the SM's own clock: gives up when another role has, or after about a quarter
// of a second.
constexpr long long kWaitCycles = 1LL << 29;
QG_DEVICE bool clock_wait(uint64_t *b, uint32_t parity, volatile int *abort) {
  if (mbar_try_wait(b, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(b, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitCycles) break;
  }
  *abort = 1;
  atomicOr(&g_qg_status_attn_tc, QG_STATUS_BIT_TIMEOUT);
  return false;
}
// the whole warp waits, and gives up as a whole
QG_DEVICE bool warp_wait(uint64_t *b, uint32_t parity, volatile int *abort) {
  return __all_sync(0xFFFFFFFFu, clock_wait(b, parity, abort));
}

// ---- producer ---------------------------------------------------------------------------------
// 16-byte chunk c of row r of a tile: half c / 8, 128-byte rows, chunks swizzled by r & 7
QG_DEVICE uint32_t tile_off(int r, int c) {
  return static_cast<uint32_t>(c >> 3) * (128u * 128u) + static_cast<uint32_t>(r) * 128u +
         static_cast<uint32_t>(((c & 7) ^ (r & 7)) * 16);
}

template <int D>
QG_DEVICE void produce(const AttnArgs &a, Walk walk, uint32_t smem, WideBars *bar, int tid) {
  using C = WideCfg<D>;
  constexpr int CH = D / 8;            // chunks per row
  constexpr int RPT = kProdWarps * 32 / CH;     // rows the producers cover at once
  constexpr int NR = (128 + RPT - 1) / RPT;     // and the times they do
  const int c = tid % CH, r0 = tid / CH;
  volatile int *abort = &bar->abort;
  // copies are reported to their barriers kLag commits later: until then they may be in flight
  uint64_t *pend[kLag] = {};
  auto report = [&](uint64_t *b) {
    fence_proxy_async_smem();  // copied through the generic proxy, read by the tensor cores
    __syncwarp();
    if (b && (threadIdx.x & 31) == 0) mbar_arrive(b);
  };
  auto push = [&](uint64_t *b) {
    cp_async_commit();
    cp_async_wait<kLag>();
    report(pend[0]);
#pragma unroll
    for (int i = 0; i + 1 < kLag; ++i) pend[i] = pend[i + 1];
    pend[kLag - 1] = b;
  };
  auto flush = [&] {
    cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < kLag; ++i) {
      report(pend[i]);
      pend[i] = nullptr;
    }
  };
  // a wait that may last: what others need to end it may be among the copies not yet reported
  auto acquire = [&](uint64_t *b, uint32_t parity) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(b, parity))) return true;
    flush();
    return warp_wait(b, parity, abort);
  };
  const int shift = a.pool.page_shift, mask = (1 << shift) - 1;
  long long it = 0;
  int np = 0;
  bool ok = true;
  Piece p;
  for (; ok && walk_next(a, &walk, &p); ++np) {
    if (!acquire(&bar->q_empty, static_cast<uint32_t>((np & 1) ^ 1))) break;
    const int half = a.wide.tpt / 2;
    for (int s = 0; s < (p.paired ? 2 : 1); ++s) {
      const int tok = min(half, p.tokens - s * half), rows = tok * a.Gq;
#pragma unroll 4
      for (int r = r0; r < 128; r += RPT) {
        const bool in = r < rows;
        const int t = p.t0 + s * half + (in ? r / a.Gq : 0);
        const uint16_t *src = a.q + t * a.q_stride + static_cast<long long>(p.h * a.Gq + (in ? r % a.Gq : 0)) * D + 8 * c;
        cp_async16_zfill(smem + C::OFF_Q + s * C::TILE + tile_off(r, c), src, in ? 16u : 0u);
      }
    }
    push(&bar->q_full);
    const long long hoff = p.h * a.pool.head_stride + 8 * c;
    for (int j = p.j0; j < p.j1 && ok; ++j) {
      // this thread's rows of the key tile: r0, r0 + RPT, ...
      long long off[NR];
      bool bad = false;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int r = r0 + i * RPT, key = j * kWideKeys + r;
        off[i] = -1;
        if (r < 128 && key < p.g.len) {
          const int page = __ldg(p.g.table + (key >> shift));
          if (page >= 0 && page < a.pool.n_pages)
            off[i] = page * a.pool.page_stride + (key & mask) * a.pool.token_stride + hoff;
          else
            bad = true;
        }
      }
      if (bad) atomicOr(&g_qg_status_attn_tc, QG_STATUS_BIT_ID);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++it) {
        const int st = static_cast<int>(it % C::NST);
        if (!acquire(&bar->empty[st], static_cast<uint32_t>(((it / C::NST) & 1) ^ 1))) {
          ok = false;
          break;
        }
        const uint16_t *base = kv ? a.pool.v : a.pool.k;
        const uint32_t dst = smem + C::OFF_KV + static_cast<uint32_t>(st) * C::TILE;
#pragma unroll
        for (int i = 0; i < NR; ++i)
          if (r0 + i * RPT < 128)
            cp_async16_zfill(dst + tile_off(r0 + i * RPT, c), base + (off[i] < 0 ? 0 : off[i]), off[i] < 0 ? 0u : 16u);
        push(&bar->full[st]);
      }
    }
  }
  flush();
}

// ---- MMA issue --------------------------------------------------------------------------------
template <int D, bool BF16, bool OUT32>
QG_DEVICE void issue_mma(const AttnArgs &a, Walk walk, uint32_t smem, WideBars *bar) {
  using C = WideCfg<D>;
  constexpr uint32_t id_s = make_idesc16(128, kWideKeys, BF16, false), id_o = make_idesc16(128, D, BF16, true);
  volatile int *abort = &bar->abort;
  const uint32_t tmem = bar->tmem;
  auto wait = [&](uint64_t *b, uint32_t parity) {
    const bool r = clock_wait(b, parity, abort);
    tc_fence_after();
    return r;
  };
  long long it = 0;           // ring position of the piece's first key tile
  int np = 0;
  uint32_t n_p[2] = {0, 0};   // weights taken from each stream
  uint32_t n_o[2] = {0, 0};   // outputs begun for each stream
  auto scores = [&](int s, int qt, int j) {  // S_s = Q_qt K_j^T
    const uint32_t q = smem + C::OFF_Q + qt * C::TILE;
    const uint32_t k = smem + C::OFF_KV + static_cast<uint32_t>((it + 2 * j) % C::NST) * C::TILE;
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      const uint32_t o = (x >> 2) * C::HALF + (x & 3) * 32;
      tc_mma_bf16(tmem + 128u * s, sw128_desc(q + o), sw128_desc(k + o), id_s, x != 0);
    }
    tc_commit(&bar->s_full[s]);
  };
  auto output = [&](int s, int j, bool first) {  // O_s += P_s V_j
    const uint32_t v = smem + C::OFF_KV + static_cast<uint32_t>((it + 2 * j + 1) % C::NST) * C::TILE;
#pragma unroll
    for (int x = 0; x < kWideKeys / 16; ++x) {
      const uint32_t p = tmem + 128u * s + 32u * (x >> 1) + 8u * (x & 1);
      const uint64_t d = sw128_desc_mn(v + x * 2048, C::HALF);
      tc_mma_ta(tmem + 256u + D * s, p, d, id_o, !(first && x == 0));
      if constexpr (OUT32) tc_mma_ta(tmem + 256u + D * s, p + 16u, d, id_o, 1);
    }
  };
  auto full = [&](int i) {  // ring position it + i has landed
    return wait(&bar->full[(it + i) % C::NST], static_cast<uint32_t>(((it + i) / C::NST) & 1));
  };
  auto free_tile = [&](int i) { tc_commit(&bar->empty[(it + i) % C::NST]); };
  // weights of stream s are in tensor memory; before its first output of the piece, the last
  // piece's has been read
  auto weights = [&](int s, bool first) {
    if (!wait(&bar->p_full[s], n_p[s]++ & 1)) return false;
    if (first && !wait(&bar->o_empty[s], (n_o[s]++ & 1) ^ 1)) return false;
    return true;
  };
  bool ok = true;
  Piece p;
  for (; ok && walk_next(a, &walk, &p); ++np) {
    const int n = p.j1 - p.j0;
    ok = wait(&bar->q_full, np & 1);
    if (p.paired) {
      for (int j = 0; j <= n && ok; ++j) {
        if (j < n) ok = full(2 * j);
        if (j > 0) ok = ok && full(2 * j - 1);
        for (int s = 0; s < 2 && ok; ++s) {
          if (j > 0) {
            ok = weights(s, j == 1);
            if (!ok) break;
            output(s, j - 1, j == 1);
            if (j == n) tc_commit(&bar->o_full[s]);
          }
          if (j < n) scores(s, s, j);
        }
        if (!ok) break;
        if (j < n) free_tile(2 * j);
        if (j > 0) free_tile(2 * j - 1);
        if (j == n - 1) tc_commit(&bar->q_empty);
      }
    } else {
      for (int j = 0; j < n + 2 && ok; ++j) {
        const int s = j & 1;
        if (j >= 2 && j - 2 < n) {
          ok = full(2 * (j - 2) + 1) && weights(s, j - 2 < 2);
          if (!ok) break;
          output(s, j - 2, j - 2 < 2);
          free_tile(2 * (j - 2) + 1);
          if (j >= n) tc_commit(&bar->o_full[s]);
        }
        if (j < n) {
          ok = full(2 * j);
          if (!ok) break;
          scores(s, 0, j);
          free_tile(2 * j);
          if (j == n - 1) tc_commit(&bar->q_empty);
        }
      }
    }
    it += 2 * n;
  }
}

// ---- softmax ----------------------------------------------------------------------------------
template <int D, bool BF16, bool OUT32>
QG_DEVICE void softmax(const AttnArgs &a, Walk walk, WideBars *bar, int s, int warp4, int lane) {
  volatile int *abort = &bar->abort;
  const uint32_t lanes = static_cast<uint32_t>(32 * warp4) << 16;
  const uint32_t ts = bar->tmem + lanes + 128u * s, to = bar->tmem + lanes + 256u + D * s;
  const int row = 32 * warp4 + lane, half = a.wide.tpt / 2;
  const float sl = fabsf(a.scale_log2);
  const bool neg = a.scale_log2 < 0.f;
  uint32_t n_s = 0, n_o = 0;
  Piece p;
  while (walk_next(a, &walk, &p)) {
    // this thread's row
    const int sub = p.paired ? s : 0;
    const int tok = min(half, p.tokens - sub * half);
    const bool valid = row < tok * a.Gq;
    const int t = p.t0 + sub * half + (valid ? row / a.Gq : 0);
    const int lim = valid ? row_limit(a, p.g, t) : 0;
    const int all = __reduce_min_sync(0xFFFFFFFFu, valid ? lim : 0x7FFFFFFF);
    float m = -INFINITY, l = 0.f;
    const int step = p.paired ? 1 : 2, first = p.paired ? p.j0 : p.j0 + s;
    for (int j = first; j < p.j1; j += step) {
      if (!warp_wait(&bar->s_full[s], n_s++ & 1, abort)) return;
      tc_fence_after();
      const int left = lim - j * kWideKeys;  // keys of the tile that the row sees
      const bool masked = j * kWideKeys + kWideKeys > all;
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float x[32];
        tmem_ld32(ts + 32 * c, x);
        if (neg) {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = -x[i];
        }
        if (masked) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i >= left) x[i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2) mx = fmaxf(mx, fmaxf(x[i], x[i + 1]));
      }
      // the reference maximum moves when the row's outgrew it by 2^8 (or it is the first)
      const bool move = mx > m && (m == -INFINITY || (mx - m) * sl > 8.0f);
      float al = 1.0f;
      if (move) {
        al = m == -INFINITY ? 0.f : ex2((m - mx) * sl);
        m = mx;
        l *= al;
      }
      if (j != first && __any_sync(0xFFFFFFFFu, move)) {
        // every product into O has finished: S's barrier came after them
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(to + 32 * c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= al;
          tmem_st32(to + 32 * c, o);
        }
      }
      const float nm = m == -INFINITY ? 0.f : -m * sl;
      f2 sum = mk2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float x[32];
        tmem_ld32(ts + 32 * c, x);
        if (neg) {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = -x[i];
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const f2 y = fma2(mk2(x[i], x[i + 1]), mk2(sl, sl), mk2(nm, nm));
          x[i] = ex2(y.x);
          x[i + 1] = ex2(y.y);
        }
        if (masked) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i >= left) x[i] = 0.f;
        }
        uint32_t hi[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          sum = add2(sum, mk2(x[i], x[i + 1]));
          hi[i / 2] = pack16<BF16>(x[i], x[i + 1]);
        }
        tmem_st16(ts + 32 * c, hi);
        if constexpr (OUT32) {  // what the rounding left
          uint32_t lo[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            lo[i / 2] = pack16<BF16>(x[i] - lo16<BF16>(hi[i / 2]), x[i + 1] - hi16<BF16>(hi[i / 2]));
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
    const bool any = first < p.j1;
    if (any) {
      if (!warp_wait(&bar->o_full[s], n_o++ & 1, abort)) return;
      tc_fence_after();
    }
    const float inv = p.alone ? (l > 0.f ? 1.0f / l : 0.f) : 1.0f;
    const size_t prow = p.slot * kWideRows + s * kWideHalf + row;
    const size_t orow = (static_cast<size_t>(t) * a.Hq + p.h * a.Gq + (valid ? row % a.Gq : 0)) * D;
    if (valid && !p.alone) a.wide.part_ml[prow] = make_float2(m == -INFINITY ? m : m * sl, l);
    if (any) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float o[32];
        tmem_ld32(to + 32 * c, o);
        if (valid) {
          if (!p.alone || OUT32) {
            float4 *dst = reinterpret_cast<float4 *>((p.alone ? static_cast<float *>(a.out) + orow
                                                              : a.wide.part_o + prow * D) + 32 * c);
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              dst[i / 4] = make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
          } else {
            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + orow + 32 * c);
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              dst[i / 8] = make_uint4(pack16<BF16>(o[i] * inv, o[i + 1] * inv), pack16<BF16>(o[i + 2] * inv, o[i + 3] * inv),
                                      pack16<BF16>(o[i + 4] * inv, o[i + 5] * inv), pack16<BF16>(o[i + 6] * inv, o[i + 7] * inv));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->o_empty[s]);
    }
  }
}

template <int D, bool BF16, bool OUT32>
__global__ void __launch_bounds__(kThreads, 1) attn_wide_kernel(const __grid_constant__ AttnArgs a) {
  using C = WideCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  WideBars *bar = reinterpret_cast<WideBars *>(smem + C::OFF_BAR);
  LineScan<kThreads> *scan = reinterpret_cast<LineScan<kThreads> *>(smem);  // before any tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&bar->full[i], kProdWarps);
      mbar_init(&bar->empty[i], 1);
    }
    mbar_init(&bar->q_full, kProdWarps);
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
  pdl_wait();
  pdl_launch_dependents();
  const Line &ln = a.wide;
  const long long total = line_scan<kThreads>(a, ln, scan, blockIdx.x == 0);
  const int nw = line_workers(ln, total);
  Walk walk;
  walk.w = static_cast<int>(blockIdx.x);
  if (total == 0 || walk.w >= nw) return;
  walk.at = line_start(walk.w, total, nw);
  walk.end = line_start(walk.w + 1, total, nw);
  if (walk.at >= walk.end || !cursor_find(a, ln, *scan, walk.at, &walk.cur)) return;  // the same for the whole block
  if (warp == kMmaWarp) tmem_alloc(&bar->tmem, C::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t sb = smem_u32(smem);
  if (warp < kSoftWarps) {
    softmax<D, BF16, OUT32>(a, walk, bar, warp >> 2, warp & 3, lane);
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      issue_mma<D, BF16, OUT32>(a, walk, sb, bar);
      // after an abort the products in flight finish before the tensor memory is released (a
      // normal run waited for each); q_empty counts pieces, so any further phase will do
      if (bar->abort) {
        const uint64_t st = *reinterpret_cast<volatile uint64_t *>(&bar->q_empty);
        tc_commit(&bar->q_empty);
        for (uint32_t i = 0; i < (1u << 16) && *reinterpret_cast<volatile uint64_t *>(&bar->q_empty) == st; ++i) __nanosleep(32);
      }
    }
  } else {
    produce<D>(a, walk, sb, bar, static_cast<int>(threadIdx.x) - 32 * (kMmaWarp + 1));
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(bar->tmem, C::COLS);
  }
}

template <int D, bool BF16, bool OUT32>
qg_status wide_run(const AttnArgs &a, cudaStream_t s) {
  auto k = attn_wide_kernel<D, BF16, OUT32>;
  if (!set_smem_attr(reinterpret_cast<const void *>(k), WideCfg<D>::SMEM)) return QG_ECUDA;
  return launch_pdl(k, dim3(static_cast<unsigned>(a.wide.workers)), dim3(kThreads), WideCfg<D>::SMEM, s, a) == cudaSuccess
             ? QG_OK
             : QG_ECUDA;
}

}  // namespace

namespace qg {

bool attn_wide_supported(int D) { return D == 64 || D == 128; }

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
  if (cudaMemcpyFromSymbol(&v, g_qg_status_attn_tc, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_qg_status_attn_tc, &z, sizeof(z));
  }
  return v;
}

}  // namespace qg
