// qg_beam.cu -- one beam-search selection: the K best continuations of each request's W beams
// over the vocabulary.
//
// cand(w, v) = score_w + (logit[w][v] - m_w) - log sum_v exp(logit[w][v] - m_w).  Within a row the
// order is the logits' order, so the first kernel needs one pass over the logits (the bytes that
// bound it): a CTA streams a slice of one row through registers, keeps the slice's maximum and
// sum of exponentials, and a short list of the values above the K-th best so far, which after
// the first chunk hardly any value joins.  The second joins a request's slices: the row sums in
// f32 (their logarithms in 64 bits), each row's K best, then the K best of W*K candidates ranked in
// 64 bits.  So candidates of one row are in exact order, and those of two rows to about 1e-7, the sums' error.
//
// Measured: 16 requests of 8 beams over 151936 tokens (72 MB) 27 us, floor 10.7 (what it spends above
// the bytes: 12 instructions a value, a chunk's barriers, 256 CTAs on 152 SMs, the merge's 5 us);
// one request of 4 beams 10.5 us, two launches.
#include <math.h>

#include <algorithm>

#include "qg_common.cuh"
#include "qg_host.h"
#include "qg_mma.cuh"

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kPT = 16;                  // values per thread and chunk
constexpr int kChunk = kThreads * kPT;
constexpr int kMaxK = 64;
constexpr int kList = 2048;              // candidates a slice holds

// f32 (no NaN) -> unsigned that rises with the value; both zeros are one
QG_DEVICE uint32_t ord_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
QG_DEVICE float ord_val(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o); }
// one 64-bit key per (value, index): larger is better, equal values by the lowest index.  0 is
// below every key of a real value.
QG_DEVICE unsigned long long key_of(float x, uint32_t idx) {
  return (static_cast<unsigned long long>(ord_of(x)) << 32) | (0xFFFFFFFFu - idx);
}
QG_DEVICE uint32_t key_idx(unsigned long long k) { return 0xFFFFFFFFu - static_cast<uint32_t>(k); }
QG_DEVICE float key_val(unsigned long long k) { return ord_val(static_cast<uint32_t>(k >> 32)); }

struct SelectArgs {
  const float *logits, *scores;
  const uint8_t *done;
  float *out_scores;
  int32_t *parents, *tokens;
  uint8_t *done_out;
  unsigned long long *keys;  // [N*W][S][K], 0: none
  float2 *ms;                // [N*W][S] slice maximum and sum of exp(x - maximum)
  long long V;
  int N, W, K, S, eos, slice, vec4;
};

// largest key of the warp: the largest upper word, then the largest lower one beside it
QG_DEVICE unsigned long long warp_max64(unsigned long long v) {
  const uint32_t h = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(v >> 32));
  const uint32_t l = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(v >> 32) == h ? static_cast<uint32_t>(v) : 0u);
  return static_cast<unsigned long long>(h) << 32 | l;
}

// The slice's candidates and what it takes to thin them out to the K best, in falling order.
struct SliceShared {
  unsigned long long list[kList], best[kMaxK], top[kWarps];
  float red[kWarps];
  int count;
};
QG_DEVICE void thin(SliceShared &sh, int K) {  // by the whole CTA; keys differ, so a key's rank is the number of larger ones
  __syncthreads();
  const int c = sh.count;
  for (int i = threadIdx.x; i < c; i += kThreads) {
    const unsigned long long k = sh.list[i];
    int r = 0;
    for (int j = 0; j < c; ++j) r += sh.list[j] > k;
    if (r < K) sh.best[r] = k;
  }
  __syncthreads();
  const int n = min(c, K);
  if (threadIdx.x < n) sh.list[threadIdx.x] = sh.best[threadIdx.x];
  if (threadIdx.x == 0) sh.count = n;
  __syncthreads();
}

// Value i of thread t of a chunk is its element 4 (kThreads (i / 4) + t) + i % 4.
QG_DEVICE int chunk_elem(int i) { return 4 * (kThreads * (i >> 2) + static_cast<int>(threadIdx.x)) + (i & 3); }
QG_DEVICE void load_chunk(const SelectArgs &a, const float *x, int n, float (&v)[kPT]) {
  const bool whole = a.vec4 && n >= kChunk;
#pragma unroll
  for (int i = 0; i < kPT; i += 4) {
    const int e = chunk_elem(i);
    if (whole || (a.vec4 && e + 4 <= n)) {
      const float4 q = __ldg(reinterpret_cast<const float4 *>(x + e));
      v[i] = q.x;
      v[i + 1] = q.y;
      v[i + 2] = q.z;
      v[i + 3] = q.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i + j] = e + j < n ? __ldg(x + e + j) : -INFINITY;
    }
  }
}

__global__ void __launch_bounds__(kThreads, 2) select_slice_kernel(const SelectArgs a) {
  __shared__ SliceShared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int row = blockIdx.y, sl = blockIdx.x;
  const size_t out = static_cast<size_t>(row) * a.S + sl;
  unsigned long long *keys = a.keys + out * a.K;
  if (a.done && __ldg(a.done + row)) {
    // an ended beam: eos at probability 1, every other token at none; slice 0 tells it all
    if (sl == 0) {
      const bool has = a.eos >= 0 && a.eos < a.V;
      for (int i = threadIdx.x; i < a.K; i += kThreads) {
        unsigned long long k = 0;
        if (has && i == 0) k = key_of(0.f, static_cast<uint32_t>(a.eos));
        else {
          long long v = has ? i - 1 : i;  // the lowest indices other than eos
          if (has && v >= a.eos) ++v;
          if (v < a.V) k = key_of(-INFINITY, static_cast<uint32_t>(v));
        }
        keys[i] = k;
      }
      if (threadIdx.x == 0) a.ms[out] = make_float2(0.f, 1.f);
    } else {
      for (int i = threadIdx.x; i < a.K; i += kThreads) keys[i] = 0;
      if (threadIdx.x == 0) a.ms[out] = make_float2(-INFINITY, 0.f);
    }
    return;
  }
  const long long base = static_cast<long long>(sl) * a.slice;
  const int len = static_cast<int>(min(static_cast<long long>(a.slice), a.V - base));
  const float *x = a.logits + static_cast<size_t>(row) * a.V + base;
  if (threadIdx.x == 0) sh.count = 0;
  float m = -INFINITY, sum = 0.f;      // this thread's maximum and sum of exp(x - m)
  bool full = false;                   // the list holds K: only values above tau can matter
  uint32_t tau = 0;                    // order word of the K-th best
  float v[kPT], w[kPT];
  load_chunk(a, x, len, w);
  __syncthreads();  // the list is empty before any thread asks how long it is
  for (int c0 = 0; c0 < len; c0 += kChunk) {
    const int n = len - c0;
#pragma unroll
    for (int i = 0; i < kPT; ++i) v[i] = fmaxf(w[i], -INFINITY);  // NaN counts as -inf
    if (c0 + kChunk < len) load_chunk(a, x + c0 + kChunk, n - kChunk, w);
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPT; ++i) mx = fmaxf(mx, v[i]);
    const uint32_t mo = ord_of(mx);
    if (mx > m) {
      sum *= expf(m - mx);  // 0 from -inf (and of +inf - +inf never: mx > m)
      m = mx;
    }
    if (m > -INFINITY && m < INFINITY) {
      // 2^((x - m) log2 e), two values an instruction.  The exponent's rounding is relative to x - m, and
      // a term's share of the sum falls faster than that grows: a few 2^-24 of the sum.
      const f2 nm = mk2(-m, -m), l2e = mk2(1.4426950408889634f, 1.4426950408889634f);
      f2 p0 = mk2(0.f, 0.f), p1 = p0;
#pragma unroll
      for (int i = 0; i < kPT; i += 4) {
        const f2 y0 = mul2(add2(mk2(v[i], v[i + 1]), nm), l2e), y1 = mul2(add2(mk2(v[i + 2], v[i + 3]), nm), l2e);
        p0 = add2(p0, mk2(ex2(y0.x), ex2(y0.y)));
        p1 = add2(p1, mk2(ex2(y1.x), ex2(y1.y)));
      }
      p0 = add2(p0, p1);
      sum += p0.x + p0.y;
    }
    // ---- candidates.  A later value equal to the K-th best loses to it by its index.
    uint32_t t = full ? tau + 1u : 0u;
    const bool any = full ? mo >= t : chunk_elem(0) < n;
    const int have = sh.count;  // nobody adds to the list before the barrier
    int hits = __syncthreads_count(any);
    if (hits == 0) continue;
    const int K = min(a.K, n);
    bool exact = false;
    if (hits * kPT > kList - kMaxK) {
      // raise t while at least K threads' maxima reach it (so K values do): few values pass
      uint32_t lo = t, hi = 0xFFFFFFFFu;
      while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int c = __syncthreads_count(mo >= mid && any);
        if (c >= K) {
          lo = mid;
          hits = c;
          if (c <= K + 16) break;
        } else {
          hi = mid;
        }
      }
      t = lo;
      exact = hits * kPT > kList - kMaxK;  // many equal maxima
    }
    if (have + (exact ? K : hits * kPT) > kList) thin(sh, a.K);
    if (!exact) {
      // few threads have any, and those mostly one: a mask of them, then each read again (16 copies of
      // the append took two fifths of the kernel's time)
      if (any && mo >= t) {
        const float tf = t ? ord_val(t) : -INFINITY;
        uint32_t mask = 0;
#pragma unroll
        for (int i = 0; i < kPT; ++i) mask |= (chunk_elem(i) < n && v[i] >= tf ? 1u : 0u) << i;
        for (; mask; mask &= mask - 1) {
          const int e = chunk_elem(__ffs(static_cast<int>(mask)) - 1);
          const float f = fmaxf(__ldg(x + c0 + e), -INFINITY);
          sh.list[atomicAdd(&sh.count, 1)] = key_of(f, static_cast<uint32_t>(base + c0 + e));
        }
      }
    } else {
      // the chunk's K best, one maximum at a time
      unsigned long long last = ~0ull;
      for (int r = 0; r < K; ++r) {
        unsigned long long k = 0;
#pragma unroll
        for (int i = 0; i < kPT; ++i) {
          const int e = chunk_elem(i);
          if (e < n) {
            const unsigned long long u = key_of(v[i], static_cast<uint32_t>(base + c0 + e));
            if (u < last && u > k) k = u;
          }
        }
        k = warp_max64(k);
        if (lane == 0) sh.top[warp] = k;
        __syncthreads();
        k = sh.top[0];
#pragma unroll
        for (int q = 1; q < kWarps; ++q) k = sh.top[q] > k ? sh.top[q] : k;
        last = k;
        if (threadIdx.x == 0) sh.list[sh.count++] = k;
        __syncthreads();
      }
    }
    __syncthreads();
    // a short list makes a high tau: thin it early, and whenever it has grown
    if (sh.count >= a.K && (!full || sh.count > a.K + 32)) {
      thin(sh, a.K);
      full = true;
      tau = static_cast<uint32_t>(sh.list[a.K - 1] >> 32);
    }
  }
  thin(sh, a.K);
  for (int i = threadIdx.x; i < a.K; i += kThreads) keys[i] = i < sh.count ? sh.list[i] : 0;
  // ---- the slice's maximum and sum
  float bm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xFFFFFFFFu, bm, o));
  if (lane == 0) sh.red[warp] = bm;
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kWarps; ++q) bm = fmaxf(bm, sh.red[q]);
  __syncthreads();
  sum = warp_sum(sum > 0.f ? sum * expf(m - bm) : 0.f);
  if (lane == 0) sh.red[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) s += sh.red[q];
    a.ms[out] = make_float2(bm, s);
  }
}

// One CTA per request, all its slices' lists in shared memory.  A warp takes a row at a time: its
// slices' sums, then its K best keys (the lists fall, so a list's next key is the only one that
// can come next; lane q holds the heads of lists q, q + 32, ...), then all W*K candidates are
// ranked against each other.
constexpr int kMergeThreads = 512;
constexpr int kMaxSlices = 128, kMaxW = 64;
__global__ void __launch_bounds__(kMergeThreads) select_merge_kernel(const SelectArgs a) {
  extern __shared__ uint8_t smem[];
  const int per_row = a.S * a.K, total = a.W * a.K;
  unsigned long long *lists = reinterpret_cast<unsigned long long *>(smem);           // [W][S][K]
  unsigned long long *rank = lists + static_cast<size_t>(a.W) * per_row;              // [W*K] order word of a candidate
  float *val = reinterpret_cast<float *>(rank + total);                               // [W*K] its logit
  uint32_t *tok = reinterpret_cast<uint32_t *>(val + total);                          // [W*K] its token
  __shared__ float row_max[kMaxW], row_sum[kMaxW];
  __shared__ double row_off[kMaxW];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = kMergeThreads / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int req = blockIdx.x;
  for (int i = threadIdx.x; i < a.W * per_row; i += kMergeThreads)
    lists[i] = __ldcg(a.keys + static_cast<size_t>(req) * a.W * per_row + i);
  for (int w = warp; w < a.W; w += nwarps) {
    const float2 *ms = a.ms + static_cast<size_t>(req * a.W + w) * a.S;
    float m = -INFINITY, sum = 0.f;
    for (int s = lane; s < a.S; s += 32) m = fmaxf(m, __ldcg(&ms[s]).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    if (isfinite(m))
      for (int s = lane; s < a.S; s += 32) {
        const float2 p = __ldcg(&ms[s]);
        if (p.y > 0.f) sum += p.y * expf(p.x - m);
      }
    sum = warp_sum(sum);
    if (lane == 0) {
      row_max[w] = m;
      row_sum[w] = sum;
    }
  }
  __syncthreads();
  // 64-bit arithmetic is scarce on this part: one warp's worth of logarithms, two sums a
  // candidate, and integer comparisons of the results' order words
  if (threadIdx.x < a.W)
    row_off[threadIdx.x] = static_cast<double>(__ldg(a.scores + req * a.W + threadIdx.x)) -
                           log(static_cast<double>(row_sum[threadIdx.x]));
  for (int w = warp; w < a.W; w += nwarps) {
    const float sc = __ldg(a.scores + req * a.W + w);
    if (!isfinite(row_max[w]) || !isfinite(sc)) {  // no distribution, or a beam not continued
      for (int i = lane; i < a.K; i += 32) {
        val[w * a.K + i] = -INFINITY;
        tok[w * a.K + i] = i < a.V ? static_cast<uint32_t>(i) : 0xFFFFFFFFu;
      }
      continue;
    }
    const unsigned long long *kr = lists + w * per_row;
    if (per_row <= 64) {  // few keys: each one's rank is the number of larger ones
      for (int i = lane; i < a.K; i += 32) {
        val[w * a.K + i] = -INFINITY;
        tok[w * a.K + i] = 0xFFFFFFFFu;
      }
      __syncwarp();
      const unsigned long long k0 = lane < per_row ? kr[lane] : 0ull, k1 = lane + 32 < per_row ? kr[lane + 32] : 0ull;
      int r0 = 0, r1 = 0;
      for (int j = 0; j < per_row; ++j) {
        const unsigned long long k = kr[j];
        r0 += k > k0;
        r1 += k > k1;
      }
      if (k0 && r0 < a.K) {
        val[w * a.K + r0] = key_val(k0);
        tok[w * a.K + r0] = key_idx(k0);
      }
      if (k1 && r1 < a.K) {
        val[w * a.K + r1] = key_val(k1);
        tok[w * a.K + r1] = key_idx(k1);
      }
      continue;
    }
    // lane's lists: positions and heads
    constexpr int kHeads = kMaxSlices / 32;
    int at[kHeads];
    unsigned long long head[kHeads];
#pragma unroll
    for (int q = 0; q < kHeads; ++q) {
      const int s = lane + 32 * q;
      at[q] = 0;
      head[q] = s < a.S ? kr[s * a.K] : 0ull;
    }
    for (int r = 0; r < a.K; ++r) {
      unsigned long long k = 0;
#pragma unroll
      for (int q = 0; q < kHeads; ++q) k = head[q] > k ? head[q] : k;
      k = warp_max64(k);
      if (lane == 0) {
        val[w * a.K + r] = k ? key_val(k) : -INFINITY;
        tok[w * a.K + r] = k ? key_idx(k) : 0xFFFFFFFFu;
      }
      if (k) {
#pragma unroll
        for (int q = 0; q < kHeads; ++q)
          if (head[q] == k) {
            ++at[q];
            head[q] = at[q] < a.K ? kr[(lane + 32 * q) * a.K + at[q]] : 0ull;
          }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += kMergeThreads) {
    const int w = i / a.K;
    // off + (logit - m): a row of huge equal logits would absorb the rest otherwise
    const double x = val[i] == -INFINITY ? -INFINITY
                                         : row_off[w] + (static_cast<double>(val[i]) - static_cast<double>(row_max[w]));
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x + 0.0));
    // 0, below every real candidate, for a place without one
    rank[i] = tok[i] == 0xFFFFFFFFu ? 0ull : u >> 63 ? ~u : u | 0x8000000000000000ull;
  }
  __syncthreads();
  // eight threads count a candidate's betters
  const int part = static_cast<int>(threadIdx.x) & 7;
  for (int i0 = 0; i0 < total; i0 += kMergeThreads / 8) {
    const int i = i0 + (static_cast<int>(threadIdx.x) >> 3);
    const unsigned long long x = i < total ? rank[i] : 0ull;
    const int w = i / a.K;
    const uint32_t v = i < total ? tok[i] : 0u;
    int r = 0;
    if (x) {
      for (int j = part; j < total; j += 8) {
        const unsigned long long y = rank[j];
        r += y > x;
        if (y == x && j != i) {  // equal: the lowest beam, then the lowest token
          const int wj = j / a.K;
          r += wj < w || (wj == w && tok[j] < v);
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
    if (x == 0 || part) continue;
    if (r < a.K) {
      const size_t o = static_cast<size_t>(req) * a.K + r;
      const unsigned long long u = x >> 63 ? x & 0x7FFFFFFFFFFFFFFFull : ~x;
      a.out_scores[o] = static_cast<float>(__longlong_as_double(static_cast<long long>(u)));
      a.parents[o] = w;
      a.tokens[o] = static_cast<int32_t>(v);
      if (a.done_out)
        a.done_out[o] = (a.done && __ldg(a.done + req * a.W + w)) || static_cast<int>(v) == a.eos ? 1 : 0;
    }
  }
}

// Slices of a row: two CTAs for every SM in all, but no slice under 4096 values (4 rows of 151936: 12.2 us at 2048, 10.7 at 4096,
// 10.9 at 8192; 128 rows: one CTA an SM 43 us, two 35, three 41; before the appends were made
// cheaper), and lists that
// fit the merge's shared memory.
struct Slices {
  int S, slice;
};
Slices make_slices(long long rows, long long W, long long K, long long V, int sms) {
  long long S = std::min<long long>({2LL * sms / rows, (V + 4095) / 4096, kMaxSlices, 16384 / (W * K)});
  S = std::max<long long>(S, 1);
  const long long slice = ((V + S - 1) / S + 3) / 4 * 4;
  return {static_cast<int>((V + slice - 1) / slice), static_cast<int>(slice)};
}
size_t merge_smem(int W, int K, int S) { return static_cast<size_t>(W) * K * (8 * static_cast<size_t>(S) + 16); }

bool select_shape(int N, int W, int K, int64_t V) {
  return N >= 0 && W >= 1 && W <= 64 && K >= 1 && K <= kMaxK && V >= 1 && V <= (1 << 20) &&
         static_cast<long long>(W) * V >= K && static_cast<long long>(N) * W <= 65535;
}

}  // namespace

extern "C" {

size_t qg_beam_workspace_size(int N, int W, int K, int64_t V) {
  if (!select_shape(N, W, K, V)) return 0;
  const qg::DeviceInfo &dev = qg::device_info();
  const long long rows = static_cast<long long>(N) * W;
  const size_t S = static_cast<size_t>(make_slices(std::max(rows, 1LL), W, K, V, dev.ok ? dev.sms : 152).S);
  return (rows * S * 8 + 255) / 256 * 256 + rows * S * K * 8;
}

qg_status qg_beam_select(const float *logits, const float *scores, const uint8_t *done, int eos, int N, int W, int K,
                         int64_t V, float *out_scores, int32_t *parents, int32_t *tokens, uint8_t *done_out,
                         void *workspace, size_t workspace_bytes, qg_stream_t stream) {
  if (!select_shape(N, W, K, V) || eos >= V) return QG_EINVAL_SHAPE;
  if (N == 0) return QG_OK;
  if (!logits || !scores || !out_scores || !parents || !tokens) return QG_EINVAL_PTR;
  auto odd = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
  if (odd(logits) || odd(scores) || odd(out_scores) || odd(parents) || odd(tokens)) return QG_EALIGN;
  if (!workspace || workspace_bytes < qg_beam_workspace_size(N, W, K, V)) return QG_EWORKSPACE;
  if (!qg::aligned16(workspace)) return QG_EALIGN;
  const qg::DeviceInfo &dev = qg::device_info();
  if (!dev.ok) return QG_ECUDA;
  SelectArgs a = {};
  const long long rows = static_cast<long long>(N) * W;
  const Slices sl = make_slices(rows, W, K, V, dev.sms);
  a.slice = sl.slice;
  a.S = sl.S;
  a.logits = logits;
  a.scores = scores;
  a.done = done;
  a.out_scores = out_scores;
  a.parents = parents;
  a.tokens = tokens;
  a.done_out = done_out;
  a.ms = static_cast<float2 *>(workspace);
  a.keys = reinterpret_cast<unsigned long long *>(static_cast<uint8_t *>(workspace) +
                                                  (static_cast<size_t>(rows) * a.S * 8 + 255) / 256 * 256);
  a.V = V;
  a.N = N;
  a.W = W;
  a.K = K;
  a.eos = eos;
  a.vec4 = V % 4 == 0 && qg::aligned16(logits);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(a.S), static_cast<unsigned>(rows)), block(kThreads);
  const size_t smem = merge_smem(W, K, a.S);
  if (smem > 48 * 1024 && !qg::set_smem_attr(reinterpret_cast<const void *>(select_merge_kernel), static_cast<uint32_t>(smem)))
    return QG_ECUDA;
  if (qg::launch_pdl(select_slice_kernel, grid, block, 0, s, a) != cudaSuccess) return QG_ECUDA;
  if (qg::launch_pdl(select_merge_kernel, dim3(static_cast<unsigned>(N)), dim3(kMergeThreads), smem, s, a) != cudaSuccess)
    return QG_ECUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ECUDA;
}

}  // extern "C"
