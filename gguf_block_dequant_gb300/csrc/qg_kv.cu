// qg_kv.cu -- the paged cache's two writers: qg_kv_append (per-head norm, position rotation and
// the write of a step's new tokens) and qg_beam_reorder (a beam search's states after a
// selection), with the rotation table and the host checks of the cache structs.
#include <math.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "qg_kv.cuh"
#include "qg_mma.cuh"

__device__ unsigned int g_qg_status_kv;  // this translation unit's device status word
static std::atomic<bool> g_launched{false};   // whether a kernel that may set it has been launched

namespace {

using qg::KvBatch;
using qg::KvPool;

// ---- append ---------------------------------------------------------------------------------
// A row (one head of one token: D floats in, D 16-bit values out) is one warp's work; lane l
// holds D/64 pairs, so a rotation never leaves its lane.  HBM bounds it with many tokens (11604
// tokens of 48 rows: 78 us, 5.5 TB/s, 0.81 of the copy bandwidth), one latency with few (one
// token 2.6 us).  Angles: position * freq as a 64-bit
// fraction of a turn (the product's overflow is whole turns), its top bits rounded once to
// f32, then the sine and cosine of pi times twice that.  They depend on the token alone, as does
// the search for its sequence, page and row: a warp does all that once for its rows, so with many
// tokens (where bytes and then instructions are the bound) two warps share a token's rows, and
// with few (where latency is) eight do and a token's rows spread over several blocks.
struct AppendArgs {
  KvPool pool;
  KvBatch b;
  const float *q, *k, *v, *q_norm, *k_norm;
  long long q_stride, k_stride, v_stride;
  const unsigned long long *freqs;
  uint16_t *q_out;
  float eps;
  int Hq, rot, rows_per_block;
  int wpt;  // warps per token: 2 or 8
};

constexpr int kAppendWarps = 8;
constexpr int kAppendRows = 2;  // rows a warp works on while as many are under way (2: 78 us, 3: 82, 4: 80)

template <int NP>
struct Pairs {
  float a[NP], b[NP];
};

// lane's pairs start at element (first) `ea` and (second) `eb`; PAIRS: they alternate from ea
template <int NP, bool PAIRS>
QG_DEVICE Pairs<NP> load_pairs(const float *p, int ea, int eb) {
  Pairs<NP> r;
  if constexpr (PAIRS) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 v = __ldg(reinterpret_cast<const float2 *>(p + ea + 2 * i));
      r.a[i] = v.x;
      r.b[i] = v.y;
    }
  } else if constexpr (NP == 1) {
    r.a[0] = __ldg(p + ea);
    r.b[0] = __ldg(p + eb);
  } else {
#pragma unroll
    for (int i = 0; i < NP; i += 2) {
      const float2 u = __ldg(reinterpret_cast<const float2 *>(p + ea + i));
      const float2 w = __ldg(reinterpret_cast<const float2 *>(p + eb + i));
      r.a[i] = u.x;
      r.a[i + 1] = u.y;
      r.b[i] = w.x;
      r.b[i + 1] = w.y;
    }
  }
  return r;
}

template <int NP, bool PAIRS, bool BF16>
QG_DEVICE void store_pairs(uint16_t *p, int ea, int eb, const Pairs<NP> &r) {
  if constexpr (PAIRS) {
#pragma unroll
    for (int i = 0; i < NP; ++i) *reinterpret_cast<uint32_t *>(p + ea + 2 * i) = pack16<BF16>(r.a[i], r.b[i]);
  } else if constexpr (NP == 1) {
    const uint32_t w = pack16<BF16>(r.a[0], r.b[0]);
    p[ea] = static_cast<uint16_t>(w);
    p[eb] = static_cast<uint16_t>(w >> 16);
  } else {
#pragma unroll
    for (int i = 0; i < NP; i += 2) {
      *reinterpret_cast<uint32_t *>(p + ea + i) = pack16<BF16>(r.a[i], r.a[i + 1]);
      *reinterpret_cast<uint32_t *>(p + eb + i) = pack16<BF16>(r.b[i], r.b[i + 1]);
    }
  }
}

template <int D, bool PAIRS, bool BF16>
__global__ void __launch_bounds__(kAppendWarps * 32) kv_append_kernel(const AppendArgs a) {
  constexpr int NP = D / 64;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int tpb = kAppendWarps / a.wpt, sub = warp % a.wpt;
  const int t = static_cast<int>(blockIdx.x) * tpb + warp / a.wpt;
  if (t >= a.b.T) return;
  const bool teller = sub == 0 && lane == 0;
  // this lane's pairs: those below rot/2 turn, the others (elements rot .. D-1) stay
  const int p0 = NP * lane, hr = a.rot / 2;
  int ea, eb;
  if (PAIRS) {
    ea = 2 * p0;
    eb = 0;
  } else if (p0 < hr) {
    ea = p0;
    eb = p0 + hr;
  } else {
    ea = a.rot + (p0 - hr);
    eb = ea + (D - a.rot) / 2;
  }
  const int rows = a.Hq + 2 * a.pool.Hkv;
  const int r_end = min(rows, (static_cast<int>(blockIdx.y) + 1) * a.rows_per_block);
  auto load_rows = [&](int r0, Pairs<NP> (&x)[kAppendRows]) {
#pragma unroll
    for (int j = 0; j < kAppendRows; ++j) {
      const int r = r0 + j * a.wpt;
      if (r < r_end) {
        const float *p = r < a.Hq ? a.q + t * a.q_stride + static_cast<long long>(r) * D
                         : r < a.Hq + a.pool.Hkv
                             ? a.k + t * a.k_stride + static_cast<long long>(r - a.Hq) * D
                             : a.v + t * a.v_stride + static_cast<long long>(r - a.Hq - a.pool.Hkv) * D;
        x[j] = load_pairs<NP, PAIRS>(p, ea, eb);
      }
    }
  };
  // the first rows are under way while the token's place is looked up (a chain of loads)
  Pairs<NP> x[kAppendRows];
  int r0 = static_cast<int>(blockIdx.y) * a.rows_per_block + sub;
  load_rows(r0, x);
  Pairs<NP> wq, wk;
  if (a.q_norm) wq = load_pairs<NP, PAIRS>(a.q_norm, ea, eb);
  if (a.k_norm) wk = load_pairs<NP, PAIRS>(a.k_norm, ea, eb);
  const int b = qg::kv_seq_of(a.b, t);
  if (b < 0) {
    if (teller) atomicOr(&g_qg_status_kv, QG_STATUS_BIT_ID);
    return;
  }
  const int t0 = a.b.q_start ? __ldg(a.b.q_start + b) : b;
  const int t1 = a.b.q_start ? __ldg(a.b.q_start + b + 1) : b + 1;
  const long long slot = static_cast<long long>(__ldg(a.b.kv_len + b)) - (t1 - t0) + (t - t0);
  const int g = qg::kv_group_of(a.b, b);
  const long long pos = slot + (g >= 0 ? max(0, __ldg(a.b.prefix_len + g)) : 0);
  // the token's cache row; a token without one is not written
  long long row = -1;
  const int shift = a.pool.page_shift;
  if (slot >= 0 && slot < qg::kv_cap(a.b.max_pages, shift)) {
    const int page = __ldg(a.b.pages + static_cast<size_t>(b) * a.b.max_pages + (slot >> shift));
    if (page >= 0 && page < a.pool.n_pages)
      row = page * a.pool.page_stride + (slot & ((1LL << shift) - 1)) * a.pool.token_stride;
  }
  if (row < 0 && teller) atomicOr(&g_qg_status_kv, QG_STATUS_BIT_ID);

  float cs[NP], sn[NP];
  if (p0 < hr) {  // hr is a multiple of 4: a lane's pairs all turn or all stay
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const long long turn = static_cast<long long>(static_cast<unsigned long long>(pos) * __ldg(a.freqs + p0 + i));
      // a fraction in [-1/2, 1/2) of a turn, 2^-64 units; 2^-63 of it in half turns
      sincospif(static_cast<float>(turn) * 1.0842021724855044e-19f, &sn[i], &cs[i]);
    }
  }

  for (; r0 < r_end; r0 += a.wpt * kAppendRows) {
    Pairs<NP> next[kAppendRows];
    load_rows(r0 + a.wpt * kAppendRows, next);
#pragma unroll
    for (int j = 0; j < kAppendRows; ++j) {
      const int r = r0 + j * a.wpt;
      if (r >= r_end) continue;
      const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.pool.Hkv;
      if (!is_v) {
        if (is_q ? a.q_norm : a.k_norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < NP; ++i) ss = fmaf(x[j].a[i], x[j].a[i], fmaf(x[j].b[i], x[j].b[i], ss));
          const float s = rsqrtf(warp_sum(ss) * (1.0f / D) + a.eps);
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            x[j].a[i] = x[j].a[i] * s * (is_q ? wq.a[i] : wk.a[i]);
            x[j].b[i] = x[j].b[i] * s * (is_q ? wq.b[i] : wk.b[i]);
          }
        }
        if (p0 < hr) {
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const float u = x[j].a[i], v = x[j].b[i];
            x[j].a[i] = u * cs[i] - v * sn[i];
            x[j].b[i] = u * sn[i] + v * cs[i];
          }
        }
      }
      if (is_q) {
        store_pairs<NP, PAIRS, BF16>(a.q_out + (static_cast<long long>(t) * a.Hq + r) * D, ea, eb, x[j]);
      } else if (row >= 0) {
        const int h = is_v ? r - a.Hq - a.pool.Hkv : r - a.Hq;
        store_pairs<NP, PAIRS, BF16>((is_v ? a.pool.v : a.pool.k) + row + h * a.pool.head_stride, ea, eb, x[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kAppendRows; ++j) x[j] = next[j];
  }
}

// ---- reorder --------------------------------------------------------------------------------
// A request's W part-filled pages are permuted in place, 16 bytes at a time: a thread owns one
// 16-byte place of the page and holds what every moved beam is to receive before it stores any
// of it, so cycles of parents need no second buffer and no order between threads.  HBM-bound
// when there is much to move (48 beams, 36 layers, 38 MB: 9.9 us), else a launch (3.6 us).  The page
// lists are permuted the same way, a thread per column.  Full pages move by their numbers only.
constexpr int kMaxLayers = 128;
struct ReorderArgs {
  uint16_t *pool[2 * kMaxLayers];
  long long page_stride, token_stride, head_stride;
  int n_pages, page_shift, Hkv, c16;  // c16: 16-byte chunks per head row
  int n_pools, N, W, max_pages;
  const int32_t *kv_len, *parents;
  int32_t *pages;
};

template <int WM>
__global__ void __launch_bounds__(256) beam_reorder_kernel(const __grid_constant__ ReorderArgs a) {
  __shared__ int par[WM], page[WM];
  __shared__ int moved;
  pdl_wait();
  pdl_launch_dependents();
  const int n = blockIdx.x % a.N, pool = blockIdx.x / a.N;  // pool == n_pools: the page lists
  const int W = a.W;
  if (threadIdx.x == 0) moved = 0;
  __syncthreads();
  const int len = __ldg(a.kv_len + static_cast<size_t>(n) * W);
  const int full = len >> a.page_shift, rem = len & ((1 << a.page_shift) - 1);
  bool bad = len < 0 || full > a.max_pages || (rem && full >= a.max_pages);
  for (int i = threadIdx.x; i < W; i += blockDim.x) {
    const size_t s = static_cast<size_t>(n) * W + i;
    if (__ldg(a.kv_len + s) != len) bad = true;
    int p = __ldg(a.parents + s);
    if (p < 0 || p >= W) {
      p = i;
      atomicOr(&g_qg_status_kv, QG_STATUS_BIT_ID);
    }
    par[i] = p;
    if (p != i) moved = 1;
    page[i] = 0;
    if (!bad && rem) {  // the lists' blocks ask as well: a request moves as a whole or not at all
      const int pg = a.pages[s * a.max_pages + full];
      page[i] = pg;
      if (pg < 0 || pg >= a.n_pages) bad = true;
    }
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicOr(&g_qg_status_kv, QG_STATUS_BIT_ID);
    return;
  }
  if (!moved) return;
  const int stride = static_cast<int>(gridDim.y * blockDim.x);
  const int first = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x);
  if (pool == a.n_pools) {
    int32_t *tab = a.pages + static_cast<size_t>(n) * W * a.max_pages;
    for (int c = first; c < full; c += stride) {
      int32_t v[WM];
#pragma unroll
      for (int i = 0; i < WM; ++i)
        if (i < W) v[i] = tab[static_cast<size_t>(par[i]) * a.max_pages + c];
#pragma unroll
      for (int i = 0; i < WM; ++i)
        if (i < W && par[i] != i) tab[static_cast<size_t>(i) * a.max_pages + c] = v[i];
    }
    return;
  }
  uint16_t *base = a.pool[pool];
  const int per_row = a.Hkv * a.c16;
  for (long long x = first; x < static_cast<long long>(rem) * per_row; x += stride) {
    const int r = static_cast<int>(x / per_row), y = static_cast<int>(x - static_cast<long long>(r) * per_row);
    const int h = y / a.c16, c = y - h * a.c16;
    uint16_t *p = base + r * a.token_stride + h * a.head_stride + 8 * c;
    uint4 v[WM];
#pragma unroll
    for (int i = 0; i < WM; ++i)
      if (i < W && par[i] != i) v[i] = *reinterpret_cast<const uint4 *>(p + page[par[i]] * a.page_stride);
#pragma unroll
    for (int i = 0; i < WM; ++i)
      if (i < W && par[i] != i) *reinterpret_cast<uint4 *>(p + page[i] * a.page_stride) = v[i];
  }
}

template <int D, bool PAIRS>
cudaError_t append_launch(bool bf16, dim3 grid, cudaStream_t s, const AppendArgs &a) {
  const dim3 block(kAppendWarps * 32);
  return bf16 ? qg::launch_pdl(kv_append_kernel<D, PAIRS, true>, grid, block, 0, s, a)
              : qg::launch_pdl(kv_append_kernel<D, PAIRS, false>, grid, block, 0, s, a);
}

}  // namespace

namespace qg {

qg_status kv_check_cache(const qg_kv_cache *c, KvPool *pool) {
  if (!c || !c->k || !c->v) return QG_EINVAL_PTR;
  if (c->dtype != QG_DT_F16 && c->dtype != QG_DT_BF16) return QG_EUNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QG_EUNSUPPORTED;
  if (c->n_pages < 1 || c->n_heads < 1 || c->n_heads > 1024 || c->page_size < 1 || c->page_size > 65536 ||
      (c->page_size & (c->page_size - 1)))
    return QG_EINVAL_SHAPE;
  const int64_t lim = int64_t(1) << 38;  // products with an index stay inside 64 bits, bytes inside a tensor map's 2^40
  if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0 || c->page_stride > lim ||
      c->token_stride > lim || c->head_stride > lim)
    return QG_EINVAL_SHAPE;
  if (!aligned16(c->k) || !aligned16(c->v) || c->page_stride % 8 || c->token_stride % 8 || c->head_stride % 8)
    return QG_EALIGN;
  pool->k = static_cast<uint16_t *>(c->k);
  pool->v = static_cast<uint16_t *>(c->v);
  pool->page_stride = c->page_stride;
  pool->token_stride = c->token_stride;
  pool->head_stride = c->head_stride;
  pool->n_pages = c->n_pages;
  pool->page_shift = 0;
  while ((1 << pool->page_shift) < c->page_size) ++pool->page_shift;
  pool->Hkv = c->n_heads;
  pool->D = c->head_dim;
  return QG_OK;
}

qg_status kv_check_batch(const qg_kv_batch *b, bool tokens, bool prefix, KvBatch *kb) {
  if (!b) return QG_EINVAL_PTR;
  if (b->n_seqs < 0 || b->n_seqs > 65535 || b->max_pages < 1) return QG_EINVAL_SHAPE;
  if (b->n_seqs > 0 && (!b->kv_len || !b->pages)) return QG_EINVAL_PTR;
  auto odd = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
  if (odd(b->kv_len) || odd(b->pages)) return QG_EALIGN;
  *kb = KvBatch{};
  kb->B = b->n_seqs;
  kb->max_pages = b->max_pages;
  kb->kv_len = b->kv_len;
  kb->pages = b->pages;
  if (!tokens) return QG_OK;
  if (b->n_tokens < 0 || b->n_tokens > (1 << 24) || b->n_groups < 0 || b->n_groups > b->n_seqs) return QG_EINVAL_SHAPE;
  if (!b->q_start && b->n_tokens != b->n_seqs) return QG_EINVAL_SHAPE;
  if (b->q_start && odd(b->q_start)) return QG_EALIGN;
  if (b->n_groups > 0) {
    if (!b->group_start || !b->prefix_len || (prefix && !b->prefix_pages)) return QG_EINVAL_PTR;
    if (odd(b->group_start) || odd(b->prefix_len) || (prefix && odd(b->prefix_pages))) return QG_EALIGN;
    if (prefix && b->max_prefix_pages < 1) return QG_EINVAL_SHAPE;
    kb->G = b->n_groups;
    kb->group_start = b->group_start;
    kb->prefix_len = b->prefix_len;
    kb->prefix_pages = b->prefix_pages;
    kb->max_prefix_pages = b->max_prefix_pages;
  }
  kb->T = b->n_tokens;
  kb->q_start = b->q_start;
  return QG_OK;
}

unsigned int read_status_kv(bool clear) {
  unsigned int v = 0;
  if (!g_launched) return v;
  if (cudaMemcpyFromSymbol(&v, g_qg_status_kv, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_qg_status_kv, &z, sizeof(z));
  }
  return v;
}

}  // namespace qg

extern "C" {

qg_status qg_rope_freqs(int rot, double theta, const float *factors, uint64_t *out) {
  if (!out) return QG_EINVAL_PTR;
  if (rot <= 0 || rot % 2 || rot > 65536 || !(theta > 1.0) || !std::isfinite(theta)) return QG_EINVAL_SHAPE;
  for (int i = 0; i < rot / 2; ++i) {
    const double f = std::pow(theta, -2.0 * i / rot) / (factors ? static_cast<double>(factors[i]) : 1.0);
    const double turns = f / 6.283185307179586476925286766559;
    if (!(turns >= 0.0 && turns < 1.0)) return QG_EINVAL_SHAPE;
    const double x = std::floor(std::ldexp(turns, 64) + 0.5);  // < 2^64: turns <= 1 - 2^-53
    out[i] = static_cast<uint64_t>(x);
  }
  return QG_OK;
}

qg_status qg_kv_append(const qg_kv_cache *cache, const qg_kv_batch *batch, int Hq, const float *q, int64_t q_stride,
                       const float *k, int64_t k_stride, const float *v, int64_t v_stride, const float *q_norm,
                       const float *k_norm, float eps, const uint64_t *freqs, int rot, int rope_pairs, void *q_out,
                       qg_stream_t stream) {
  AppendArgs a = {};
  qg_status st = qg::kv_check_cache(cache, &a.pool);
  if (st != QG_OK) return st;
  st = qg::kv_check_batch(batch, true, false, &a.b);
  if (st != QG_OK) return st;
  const int D = a.pool.D, Hkv = a.pool.Hkv;
  if (Hq < 0 || Hq % Hkv || Hq > 16384 || rot < 0 || rot > D || rot % 8 || !(eps >= 0.f) || (rope_pairs & ~1))
    return QG_EINVAL_SHAPE;
  if (a.b.T == 0) return QG_OK;
  if (!k || !v || (Hq > 0 && (!q || !q_out)) || (rot > 0 && !freqs)) return QG_EINVAL_PTR;
  const int64_t lim = int64_t(1) << 38;
  if ((Hq > 0 && q_stride < static_cast<int64_t>(Hq) * D) || k_stride < static_cast<int64_t>(Hkv) * D ||
      v_stride < static_cast<int64_t>(Hkv) * D || q_stride > lim || k_stride > lim || v_stride > lim)
    return QG_EINVAL_SHAPE;
  if (!qg::aligned16(k) || !qg::aligned16(v) || k_stride % 4 || v_stride % 4 ||
      (Hq > 0 && (!qg::aligned16(q) || !qg::aligned16(q_out) || q_stride % 4)) || (q_norm && !qg::aligned16(q_norm)) ||
      (k_norm && !qg::aligned16(k_norm)) || (reinterpret_cast<uintptr_t>(freqs) & 7u))
    return QG_EALIGN;
  const qg::DeviceInfo &dev = qg::device_info();
  if (!dev.ok) return QG_ECUDA;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.freqs = reinterpret_cast<const unsigned long long *>(freqs);
  a.q_out = static_cast<uint16_t *>(q_out);
  a.eps = eps;
  a.Hq = Hq;
  a.rot = rot;
  // two warps per token from eight tokens for every SM on (11604 tokens of 48 rows: 95 us with
  // eight, 78 with two); with few tokens their rows go to several blocks, one row per warp
  const int rows = Hq + 2 * Hkv;
  a.wpt = a.b.T >= 8 * dev.sms ? 2 : kAppendWarps;
  const int most = (rows + kAppendWarps - 1) / kAppendWarps;
  const int gy = a.wpt == 2 ? 1 : std::max(1, std::min(most, 2 * dev.sms / a.b.T));
  a.rows_per_block = (rows + gy - 1) / gy;
  const int tpb = kAppendWarps / a.wpt;
  const dim3 grid(static_cast<unsigned>((a.b.T + tpb - 1) / tpb),
                  static_cast<unsigned>((rows + a.rows_per_block - 1) / a.rows_per_block));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = cache->dtype == QG_DT_BF16;
  g_launched = true;
  cudaError_t e;
  if (D == 64) e = rope_pairs ? append_launch<64, true>(bf16, grid, s, a) : append_launch<64, false>(bf16, grid, s, a);
  else if (D == 128) e = rope_pairs ? append_launch<128, true>(bf16, grid, s, a) : append_launch<128, false>(bf16, grid, s, a);
  else e = rope_pairs ? append_launch<256, true>(bf16, grid, s, a) : append_launch<256, false>(bf16, grid, s, a);
  if (e != cudaSuccess) return QG_ECUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ECUDA;
}

qg_status qg_beam_reorder(const qg_kv_cache *caches, int n_layers, const qg_kv_batch *batch, int W,
                          const int32_t *parents, qg_stream_t stream) {
  if (!caches || (!parents && batch && batch->n_seqs > 0)) return QG_EINVAL_PTR;
  if (n_layers < 1 || n_layers > kMaxLayers || W < 1 || W > 32) return QG_EINVAL_SHAPE;
  ReorderArgs a;
  KvPool first = {};
  for (int l = 0; l < n_layers; ++l) {
    KvPool p = {};
    const qg_status st = qg::kv_check_cache(caches + l, &p);
    if (st != QG_OK) return st;
    if (l == 0) first = p;
    if (p.page_stride != first.page_stride || p.token_stride != first.token_stride ||
        p.head_stride != first.head_stride || p.n_pages != first.n_pages || p.page_shift != first.page_shift ||
        p.Hkv != first.Hkv || p.D != first.D || caches[l].dtype != caches[0].dtype)
      return QG_EINVAL_SHAPE;
    a.pool[2 * l] = p.k;
    a.pool[2 * l + 1] = p.v;
  }
  KvBatch kb = {};
  const qg_status st = qg::kv_check_batch(batch, false, false, &kb);
  if (st != QG_OK) return st;
  if (kb.B % W) return QG_EINVAL_SHAPE;
  if (reinterpret_cast<uintptr_t>(parents) & 3u) return QG_EALIGN;
  if (kb.B == 0 || W == 1) return QG_OK;
  a.page_stride = first.page_stride;
  a.token_stride = first.token_stride;
  a.head_stride = first.head_stride;
  a.n_pages = first.n_pages;
  a.page_shift = first.page_shift;
  a.Hkv = first.Hkv;
  a.c16 = first.D / 8;
  a.n_pools = 2 * n_layers;
  a.N = kb.B / W;
  a.W = W;
  a.max_pages = kb.max_pages;
  a.kv_len = kb.kv_len;
  a.parents = parents;
  a.pages = kb.pages;
  // a block takes 256 of a page's 16-byte places at a time
  const long long places = static_cast<long long>(caches[0].page_size) * first.Hkv * a.c16;
  const dim3 grid(static_cast<unsigned>((a.n_pools + 1) * a.N),
                  static_cast<unsigned>(std::min<long long>(64, (places + 255) / 256)));
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  g_launched = true;
  cudaError_t e;
  if (W <= 4) e = qg::launch_pdl(beam_reorder_kernel<4>, grid, dim3(256), 0, s, a);
  else if (W <= 8) e = qg::launch_pdl(beam_reorder_kernel<8>, grid, dim3(256), 0, s, a);
  else if (W <= 16) e = qg::launch_pdl(beam_reorder_kernel<16>, grid, dim3(256), 0, s, a);
  else e = qg::launch_pdl(beam_reorder_kernel<32>, grid, dim3(256), 0, s, a);
  if (e != cudaSuccess) return QG_ECUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ECUDA;
}

}  // extern "C"
