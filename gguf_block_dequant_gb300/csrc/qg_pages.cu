// qg_pages.cu -- pages with holders: qg_kv_fork (share, truncate, free), qg_kv_reserve (new pages, begun
// shared ones copied) and qg_kv_compact (chosen tokens into pages of their own).
#include <algorithm>
#include <atomic>

#include "qg_kv.cuh"

__device__ unsigned int g_qg_status_pages;   // this translation unit's device status word
static std::atomic<bool> g_launched{false};  // whether a kernel that may set it has been launched

namespace {

using qg::KvBatch;

QG_DEVICE void bad() { atomicOr(&g_qg_status_pages, QG_STATUS_BIT_ID); }

// what a length is worth: its pages, -1 when it does not fit the page list
QG_DEVICE int pages_of(int len, int shift, int max_pages) {
  if (len < 0) return -1;
  const int n = static_cast<int>((static_cast<long long>(len) + (1 << shift) - 1) >> shift);
  return n <= max_pages ? n : -1;
}

// ---- fork ---------------------------------------------------------------------------------------
// A block per sequence; all it costs is a launch and the page numbers (a few words a page).  A source must
// stay as it is, so no block reads what another writes, and counts only meet in atomics.
struct ForkArgs {
  int32_t *kv_len, *pages, *refs;
  const int32_t *src, *keep;
  int B, max_pages, n_pages, shift;
};

__global__ void __launch_bounds__(128) kv_fork_kernel(const ForkArgs a) {
  const int b = blockIdx.x, tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int s = a.src ? __ldg(a.src + b) : b;
  const int old_len = a.kv_len[b], old_pages = pages_of(old_len, a.shift, a.max_pages);
  const int want = a.keep ? __ldg(a.keep + b) : -1;  // -1: all
  bool ok = s >= -1 && s < a.B && old_pages >= 0 && want >= -1;
  int len = 0, n = 0;
  if (ok && s >= 0) {
    const int there = s == b ? old_len : a.kv_len[s];
    if (s != b)  // the source stays as it is
      ok = __ldg(a.src + s) == s && (!a.keep || __ldg(a.keep + s) == -1) && pages_of(there, a.shift, a.max_pages) >= 0;
    len = want < 0 ? there : min(there, want);
    n = pages_of(len, a.shift, a.max_pages);
  }
  if (!ok) {
    if (tid == 0) bad();
    return;
  }
  int32_t *row = a.pages + static_cast<size_t>(b) * a.max_pages;
  auto count = [&](int p, int by) {
    if (p < 0 || p >= a.n_pages) return bad();
    if (atomicAdd(a.refs + p, by) <= 0 && by < 0) {
      atomicAdd(a.refs + p, 1);
      bad();
    }
  };
  for (int i = tid + (s == b ? n : 0); i < old_pages; i += blockDim.x) count(row[i], -1);
  if (s >= 0 && s != b) {
    __syncthreads();  // the old numbers are read
    const int32_t *from = a.pages + static_cast<size_t>(s) * a.max_pages;
    for (int i = tid; i < n; i += blockDim.x) {
      const int p = from[i];
      row[i] = p;
      count(p, 1);
    }
  }
  __syncthreads();
  if (tid == 0 && len != old_len) a.kv_len[b] = len;
}

// ---- reserve --------------------------------------------------------------------------------------
// One block does the books: what each sequence needs (a scan gives its place among the free pages), the
// free pages in rising order (a scan over the counts until there are enough), then the page lists and the
// counts.  A second kernel copies the begun pages that were shared, its blocks over layers and sequences.  Latency bounds the books
// (about 4 us for 60 sequences and 160 pages: three loads in a chain, three block scans); a large pool costs a round of
// kBookThreads x kBookEach counts each, with the next round's on their way.
// Workspace: the number of copies; (old page, new page, rows) of each; the needs' running sums; the free pages.
constexpr int kBookThreads = 512;
constexpr int kBookFree = 4096;  // free pages kept in shared memory
constexpr int kBookEach = 8;     // counts of a thread and round
struct ReserveArgs {
  int32_t *kv_len, *pages, *refs, *missing;
  const int32_t *add;
  int32_t *n_copies, *copies, *upto, *free_ids;
  int B, max_pages, n_pages, shift;
};

struct Need {
  int first, n;     // first column that gets a page, and how many do
  bool ok, copies;  // the first of them replaces a begun page
};

QG_DEVICE Need need_of(const ReserveArgs &a, int b) {
  Need r{0, 0, true, false};
  const int add = __ldg(a.add + b), len = a.kv_len[b];
  if (add == 0) return r;
  const int have = pages_of(len, a.shift, a.max_pages);
  const long long to = static_cast<long long>(len) + add;
  const int want = to > 0x7FFFFFFF ? -1 : pages_of(static_cast<int>(to), a.shift, a.max_pages);
  if (add < 0 || have < 0 || want < 0) {
    r.ok = false;
    return r;
  }
  r.first = have;
  r.n = want - have;
  if (len & ((1 << a.shift) - 1)) {
    const int p = a.pages[static_cast<size_t>(b) * a.max_pages + have - 1];
    if (p < 0 || p >= a.n_pages) {
      r.ok = false;
      r.n = 0;
    } else if (a.refs[p] > 1) {
      r.copies = true;
      --r.first;
      ++r.n;
    }
  }
  return r;
}

// exclusive running sum over the block; *total gets the sum
template <typename T>
QG_DEVICE T block_scan(T v, T *total) {
  __shared__ T part[kBookThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  constexpr int W = kBookThreads / 32;
  __syncthreads();
  if (lane == 31) part[warp] = x;
  __syncthreads();
  T y = part[lane & (W - 1)];
#pragma unroll
  for (int o = 1; o < W; o <<= 1) {
    const T z = __shfl_up_sync(0xFFFFFFFFu, y, o);
    if (lane >= o) y += z;
  }
  *total = __shfl_sync(0xFFFFFFFFu, y, W - 1);
  const T before = __shfl_sync(0xFFFFFFFFu, y, warp ? warp - 1 : 0);
  return (warp ? before : 0) + x - v;
}

__global__ void __launch_bounds__(kBookThreads) kv_reserve_kernel(const ReserveArgs a) {
  __shared__ int s_free[kBookFree];  // the first free pages that are taken
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  // the counts of the first pages are under way while the needs are worked out (a chain of loads)
  constexpr int kRound = kBookThreads * kBookEach;
  int ref[kBookEach];
  auto load = [&](int p0) {
#pragma unroll
    for (int i = 0; i < kBookEach; ++i) {
      const int p = p0 + tid * kBookEach + i;
      ref[i] = p < a.n_pages ? a.refs[p] : 1;
    }
  };
  load(0);
  // needs and copies in one sum, the copies above bit 47: 65535 sequences need less than that many pages, and copy fewer than 2^16.
  // upto[b]: free pages taken before b
  constexpr int kHigh = 47;
  long long sums = 0, sum;
  Need r{0, 0, true, false};
  int at = 0;
  const bool one_round = a.B <= kBookThreads;
  for (int b0 = 0; b0 < a.B; b0 += kBookThreads) {
    const int b = b0 + tid;
    r = Need{0, 0, true, false};
    int len = 0, old_page = 0;
    if (b < a.B) {
      r = need_of(a, b);
      if (r.copies) {
        len = a.kv_len[b];
        old_page = a.pages[static_cast<size_t>(b) * a.max_pages + r.first];
      }
    }
    if (!r.ok) bad();
    const long long mine = r.n + (static_cast<long long>(r.copies) << kHigh);
    const long long before = sums + block_scan<long long>(mine, &sum);
    sums += sum;
    const long long need = before & ((1LL << kHigh) - 1);
    at = static_cast<int>(min(need, static_cast<long long>(a.n_pages)));
    if (b < a.B) {
      if (!one_round) a.upto[b] = at;
      if (r.copies) {
        const int c = static_cast<int>(before >> kHigh);
        a.copies[3 * c] = old_page;
        a.copies[3 * c + 1] = at;  // becomes the page
        a.copies[3 * c + 2] = len & ((1 << a.shift) - 1);
      }
    }
  }
  const long long need = sums & ((1LL << kHigh) - 1);
  const int copies = static_cast<int>(sums >> kHigh);
  // the lowest free pages
  int found = 0, total;
  for (int p0 = 0; p0 < a.n_pages && found < need; p0 += kRound) {
    int mine = 0, now[kBookEach];
#pragma unroll
    for (int i = 0; i < kBookEach; ++i) {
      now[i] = ref[i];
      mine += now[i] == 0;
    }
    if (a.n_pages - p0 > kRound) load(p0 + kRound);
    int i = found + block_scan<int>(mine, &total);
    found += total;
#pragma unroll
    for (int e = 0; e < kBookEach; ++e)
      if (now[e] == 0) {
        const int p = p0 + tid * kBookEach + e;
        if (i < need) {
          if (i < kBookFree) s_free[i] = p;
          else a.free_ids[i] = p;
        }
        ++i;
      }
  }
  if (tid == 0) {
    *a.missing = static_cast<int>(max(0LL, min(need - found, 0x7FFFFFFFLL)));
    *a.n_copies = found < need ? 0 : copies;
  }
  if (found < need) return;
  __syncthreads();
  auto free_page = [&](int i) { return i < kBookFree ? s_free[i] : a.free_ids[i]; };
  // every sequence's need is worked out before any count changes below
  for (int c = tid; c < copies; c += kBookThreads) a.copies[3 * c + 1] = free_page(a.copies[3 * c + 1]);
  for (int b = tid; b < a.B; b += kBookThreads) {
    if (!one_round) {
      r = need_of(a, b);
      at = a.upto[b];
    }
    if (!r.ok) continue;
    for (int i = 0; i < r.n; ++i) a.pages[static_cast<size_t>(b) * a.max_pages + r.first + i] = free_page(at + i);
    const int more = __ldg(a.add + b);
    if (more) a.kv_len[b] += more;
  }
  __syncthreads();
  for (int i = tid; i < need; i += kBookThreads) a.refs[free_page(i)] = 1;
  for (int c = tid; c < copies; c += kBookThreads) atomicSub(a.refs + a.copies[3 * c], 1);
}

// x / d for x < 2^31 and the d that `mul` and `shift` were made for: mul = ceil(2^shift / d), shift = 31 + ceil(log2 d)
struct Divisor {
  unsigned long long mul;
  int shift;
  QG_DEVICE int of(int x) const { return static_cast<int>((static_cast<unsigned>(x) * mul) >> shift); }
};
Divisor divisor(int d) {
  int l = 0;
  while ((1LL << l) < d) ++l;
  return {((1ULL << (31 + l)) + d - 1) / d, 31 + l};
}

// one geometry for all layers
constexpr int kMaxLayers = 128;
struct Pools {
  uint16_t *pool[2 * kMaxLayers];
  long long page_stride, token_stride, head_stride;
  int n_pools, n_pages, shift, Hkv, per_row, c_shift;  // 16-byte pieces of a token, and log2 of those of a head's row
  Divisor by_row;                                      // by per_row
};
// offset of piece x of a page or token run, and its token
QG_DEVICE long long piece_at(const Pools &a, int x, int &token) {
  token = a.by_row.of(x);
  const int y = x - token * a.per_row, h = y >> a.c_shift;
  return h * a.head_stride + 8 * (y - (h << a.c_shift));
}

// A thread moves 16 bytes at a time, eight under way; HBM-bound once there is much to move (48 begun pages in
// 36 layers, 79 MB: fork, books and copy together 20.5 us, the copy about 13).
__global__ void __launch_bounds__(256) page_copy_kernel(const __grid_constant__ Pools a, const int32_t *n_copies,
                                                        const int32_t *copies) {
  pdl_wait();
  pdl_launch_dependents();
  uint16_t *pool = a.pool[blockIdx.x];
  const int n = *n_copies;
  for (int c = blockIdx.y; c < n; c += gridDim.y) {
    const uint16_t *from = pool + copies[3 * c] * a.page_stride;
    uint16_t *to = pool + copies[3 * c + 1] * a.page_stride;
    const int pieces = copies[3 * c + 2] * a.per_row;
    for (int x = threadIdx.x; x < pieces; x += 8 * 256) {
      uint4 v[8];
      long long o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (x + 256 * i < pieces) {
          int r;
          o[i] = piece_at(a, x + 256 * i, r);
          o[i] += r * a.token_stride;
          v[i] = *reinterpret_cast<const uint4 *>(from + o[i]);
        }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (x + 256 * i < pieces) *reinterpret_cast<uint4 *>(to + o[i]) = v[i];
    }
  }
}

// ---- compact --------------------------------------------------------------------------------------
// A block owns a few tokens: it looks their places up once (a chain of loads) and moves them in several
// pools, 16 bytes a thread and several under way: HBM bounds it (1550 tokens in 36 layers, 460 MB: 73.5 us, 6.3 TB/s, 0.94 of
// the copy).
constexpr int kCompactTokens = 8;
struct CompactArgs {
  Pools p;
  const int32_t *kv_len, *pages, *src, *keep_start, *keep;
  int B, max_pages, n_keep, pools_per_block;
};

__global__ void __launch_bounds__(256) kv_compact_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ long long from[kCompactTokens], to[kCompactTokens];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  if (tid < kCompactTokens) {
    const long long i = static_cast<long long>(blockIdx.x) * kCompactTokens + tid;
    long long f = -1, t = -1;
    const int b = i < a.n_keep ? qg::kv_search(a.keep_start, a.B, static_cast<int>(i)) : -1;
    const int s = b >= 0 ? __ldg(a.src + b) : -1;
    if (s != -1) {
      const int dst = static_cast<int>(i) - __ldg(a.keep_start + b), slot = __ldg(a.keep + i);
      const int cap = qg::kv_cap(a.max_pages, a.p.shift);
      bool ok = s >= 0 && s < a.B && s != b && dst >= 0 && dst < min(cap, __ldg(a.kv_len + b));
      ok = ok && slot >= 0 && slot < min(cap, __ldg(a.kv_len + s));
      if (ok) {
        const int pf = __ldg(a.pages + static_cast<size_t>(s) * a.max_pages + (slot >> a.p.shift));
        const int pt = __ldg(a.pages + static_cast<size_t>(b) * a.max_pages + (dst >> a.p.shift));
        ok = pf >= 0 && pf < a.p.n_pages && pt >= 0 && pt < a.p.n_pages;
        const int m = (1 << a.p.shift) - 1;
        if (ok) {
          f = pf * a.p.page_stride + (slot & m) * a.p.token_stride;
          t = pt * a.p.page_stride + (dst & m) * a.p.token_stride;
        }
      }
      if (!ok && blockIdx.y == 0) bad();
    }
    from[tid] = f;
    to[tid] = t;
  }
  __syncthreads();
  const int q0 = blockIdx.y * a.pools_per_block, q1 = min(a.p.n_pools, q0 + a.pools_per_block);
  const int all = (q1 - q0) * kCompactTokens * a.p.per_row;
  for (int x = tid; x < all; x += 8 * 256) {
    uint4 v[8];
    uint16_t *dst[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int y = x + 256 * i;
      dst[i] = nullptr;
      if (y < all) {
        int t;  // the tile's tokens in the first pool, then in the next
        const long long o = piece_at(a.p, y, t);
        const int r = t % kCompactTokens;
        if (to[r] >= 0) {
          uint16_t *pool = a.p.pool[q0 + t / kCompactTokens];
          v[i] = *reinterpret_cast<const uint4 *>(pool + from[r] + o);
          dst[i] = pool + to[r] + o;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (dst[i]) *reinterpret_cast<uint4 *>(dst[i]) = v[i];
  }
}

qg_status check_pools(const qg_kv_cache *caches, int n_layers, Pools *out) {
  if (!caches) return QG_EINVAL_PTR;
  if (n_layers < 1 || n_layers > kMaxLayers) return QG_EINVAL_SHAPE;
  qg::KvPool first = {};
  for (int l = 0; l < n_layers; ++l) {
    qg::KvPool p = {};
    const qg_status st = qg::kv_check_cache(caches + l, &p);
    if (st != QG_OK) return st;
    if (l == 0) first = p;
    if (p.page_stride != first.page_stride || p.token_stride != first.token_stride ||
        p.head_stride != first.head_stride || p.n_pages != first.n_pages || p.page_shift != first.page_shift ||
        p.Hkv != first.Hkv || p.D != first.D || caches[l].dtype != caches[0].dtype)
      return QG_EINVAL_SHAPE;
    out->pool[2 * l] = p.k;
    out->pool[2 * l + 1] = p.v;
  }
  out->page_stride = first.page_stride;
  out->token_stride = first.token_stride;
  out->head_stride = first.head_stride;
  out->n_pools = 2 * n_layers;
  out->n_pages = first.n_pages;
  out->shift = first.page_shift;
  out->Hkv = first.Hkv;
  out->per_row = first.Hkv * (first.D / 8);
  out->c_shift = first.D == 64 ? 3 : first.D == 128 ? 4 : 5;
  out->by_row = divisor(out->per_row);
  return QG_OK;
}

bool odd4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }
size_t round16(size_t n) { return (n + 15) & ~size_t(15); }

}  // namespace

namespace qg {

unsigned int read_status_pages(bool clear) {
  unsigned int v = 0;
  if (!g_launched) return v;
  if (cudaMemcpyFromSymbol(&v, g_qg_status_pages, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_qg_status_pages, &z, sizeof(z));
  }
  return v;
}

}  // namespace qg

extern "C" {

qg_status qg_kv_fork(const qg_kv_cache *cache, const qg_kv_batch *batch, int32_t *refs, const int32_t *src,
                     const int32_t *keep, qg_stream_t stream) {
  Pools p;
  qg_status st = check_pools(cache, 1, &p);
  if (st != QG_OK) return st;
  KvBatch kb = {};
  st = qg::kv_check_batch(batch, false, false, &kb);
  if (st != QG_OK) return st;
  if (kb.B == 0) return QG_OK;
  if (!refs) return QG_EINVAL_PTR;
  if (odd4(refs) || odd4(src) || odd4(keep)) return QG_EALIGN;
  ForkArgs a{const_cast<int32_t *>(kb.kv_len), kb.pages, refs, src, keep, kb.B, kb.max_pages, p.n_pages, p.shift};
  g_launched = true;
  const cudaError_t e = qg::launch_pdl(kv_fork_kernel, dim3(kb.B), dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return QG_ECUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ECUDA;
}

size_t qg_kv_reserve_workspace_size(const qg_kv_cache *caches, const qg_kv_batch *batch) {
  Pools p;
  KvBatch kb = {};
  if (check_pools(caches, 1, &p) != QG_OK || qg::kv_check_batch(batch, false, false, &kb) != QG_OK) return 0;
  return 16 + round16(sizeof(int32_t) * 3 * kb.B) + round16(sizeof(int32_t) * kb.B) + round16(sizeof(int32_t) * p.n_pages);
}

qg_status qg_kv_reserve(const qg_kv_cache *caches, int n_layers, const qg_kv_batch *batch, int32_t *refs,
                        const int32_t *add, int32_t *missing, void *workspace, size_t workspace_bytes,
                        qg_stream_t stream) {
  Pools p;
  qg_status st = check_pools(caches, n_layers, &p);
  if (st != QG_OK) return st;
  KvBatch kb = {};
  st = qg::kv_check_batch(batch, false, false, &kb);
  if (st != QG_OK) return st;
  if (kb.B == 0) return QG_OK;
  if (!refs || !add || !missing) return QG_EINVAL_PTR;
  if (odd4(refs) || odd4(add) || odd4(missing)) return QG_EALIGN;
  if (!workspace || workspace_bytes < qg_kv_reserve_workspace_size(caches, batch)) return QG_EWORKSPACE;
  if (!qg::aligned16(workspace)) return QG_EALIGN;
  const qg::DeviceInfo &dev = qg::device_info();
  if (!dev.ok) return QG_ECUDA;
  char *ws = static_cast<char *>(workspace);
  ReserveArgs a{const_cast<int32_t *>(kb.kv_len), kb.pages, refs, missing, add};
  a.n_copies = reinterpret_cast<int32_t *>(ws);
  a.copies = reinterpret_cast<int32_t *>(ws += 16);
  a.upto = reinterpret_cast<int32_t *>(ws += round16(sizeof(int32_t) * 3 * kb.B));
  a.free_ids = reinterpret_cast<int32_t *>(ws += round16(sizeof(int32_t) * kb.B));
  a.B = kb.B;
  a.max_pages = kb.max_pages;
  a.n_pages = p.n_pages;
  a.shift = p.shift;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  g_launched = true;
  cudaError_t e = qg::launch_pdl(kv_reserve_kernel, dim3(1), dim3(kBookThreads), 0, s, a);
  if (e == cudaSuccess && p.shift > 0) {  // pages of one token are never begun
    const dim3 grid(p.n_pools, std::max(1, std::min(kb.B, 16 * dev.sms / p.n_pools)));
    e = qg::launch_pdl(page_copy_kernel, grid, dim3(256), 0, s, p, static_cast<const int32_t *>(a.n_copies),
                       static_cast<const int32_t *>(a.copies));
  }
  if (e != cudaSuccess) return QG_ECUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ECUDA;
}

qg_status qg_kv_compact(const qg_kv_cache *caches, int n_layers, const qg_kv_batch *batch, const int32_t *src,
                        const int32_t *keep_start, const int32_t *keep, int n_keep, qg_stream_t stream) {
  CompactArgs a;
  qg_status st = check_pools(caches, n_layers, &a.p);
  if (st != QG_OK) return st;
  KvBatch kb = {};
  st = qg::kv_check_batch(batch, false, false, &kb);
  if (st != QG_OK) return st;
  if (n_keep < 0 || n_keep > (1 << 24)) return QG_EINVAL_SHAPE;
  if (kb.B == 0 || n_keep == 0) return QG_OK;
  if (!src || !keep_start || !keep) return QG_EINVAL_PTR;
  if (odd4(src) || odd4(keep_start) || odd4(keep)) return QG_EALIGN;
  const qg::DeviceInfo &dev = qg::device_info();
  if (!dev.ok) return QG_ECUDA;
  a.kv_len = kb.kv_len;
  a.pages = kb.pages;
  a.src = src;
  a.keep_start = keep_start;
  a.keep = keep;
  a.B = kb.B;
  a.max_pages = kb.max_pages;
  a.n_keep = n_keep;
  const int tiles = (n_keep + kCompactTokens - 1) / kCompactTokens;
  // about eight blocks an SM, at most all pools to one block
  const int parts = std::max(1, std::min(a.p.n_pools, 8 * dev.sms / tiles));
  a.pools_per_block = (a.p.n_pools + parts - 1) / parts;
  const dim3 grid(tiles, (a.p.n_pools + a.pools_per_block - 1) / a.pools_per_block);
  g_launched = true;
  const cudaError_t e = qg::launch_pdl(kv_compact_kernel, grid, dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return QG_ECUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ECUDA;
}

}  // extern "C"
