// qg_draft.cu -- the token steps of drafted decode: qg_token_probs (probabilities from logits) and
// qg_draft_verify (how many drafts the target accepts, and the token drawn behind them).
#include <algorithm>
#include <atomic>

#include "qg_common.cuh"
#include "qg_host.h"

__device__ unsigned int g_qg_status_draft;   // this translation unit's device status word
static std::atomic<bool> g_launched{false};  // whether a kernel that may set it has been launched

namespace {

// ---- clusters ---------------------------------------------------------------------------------
QG_DEVICE void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
QG_DEVICE uint32_t remote_addr(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
QG_DEVICE float remote_f32(const float *p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote_addr(p, rank)) : "memory");
  return v;
}
QG_DEVICE double remote_f64(const double *p, uint32_t rank) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(remote_addr(p, rank)) : "memory");
  return v;
}
QG_DEVICE int remote_s32(const int *p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote_addr(p, rank)) : "memory");
  return v;
}

template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kern)(KArgs...), unsigned blocks, unsigned threads, size_t smem, int cluster,
                           cudaStream_t s, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// ---- probabilities ------------------------------------------------------------------------------
// A row is split over a cluster of CTAs; each keeps its slice in shared memory, so a logit is read once
// and a probability written once (8 bytes an element: HBM bounds it).  Slices are laid out as in global
// memory modulo 16 bytes, so that rows of odd lengths still move 16 bytes at a time.  Each CTA sums
// exp((x - its own maximum) / t); one exchange of (maximum, sum) gives every CTA its factor.  What does
// not fit (vocabularies over 8 x kKeep) is read again.
constexpr int kProbThreads = 512;
constexpr int kKeep = 48 * 1024;  // floats of a slice that stay in shared memory

struct ProbArgs {
  const float *logits, *temperature;
  float *probs;
  int T, V, cs, slice;  // CTAs per row, elements per CTA (a multiple of 4)
};

QG_DEVICE void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__global__ void __launch_bounds__(kProbThreads) token_probs_kernel(const ProbArgs a) {
  extern __shared__ float4 keep4[];
  float *const keep = reinterpret_cast<float *>(keep4);
  __shared__ float red[kProbThreads / 32];
  __shared__ int redi[kProbThreads / 32];
  __shared__ float cta_m, cta_s;
  __shared__ int cta_i;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = static_cast<int>(blockIdx.x) / a.cs, rank = static_cast<int>(blockIdx.x) % a.cs;
  pdl_wait();
  pdl_launch_dependents();
  const float tau = a.temperature ? __ldg(a.temperature + row) : 1.f;
  const bool greedy = !(tau > 0.f);
  const float inv2 = greedy ? 2.f : 2.f / tau;  // t of inf: 0, a denormal t: inf (0 * inf is caught below)
  const long long base = static_cast<long long>(row) * a.V;
  const int lo = min(a.V, rank * a.slice), hi = min(a.V, lo + a.slice), n = hi - lo;
  const float *src = a.logits + base + lo;
  float *dst = a.probs + base + lo;
  const int pad = static_cast<int>((base + lo) & 3);  // slice element i sits at keep[pad + i]
  const int held = min(n, kKeep - 4);
  const int head = min(held, (4 - pad) & 3), body = (held - head) >> 2, tail = held - head - 4 * body;
  for (int i = tid; i < body; i += kProbThreads)
    cp_async16(smem_u32(keep + pad + head + 4 * i), src + head + 4 * i);
  if (tid < head) cp_async4(smem_u32(keep + pad + tid), src + tid);
  if (tid < tail) cp_async4(smem_u32(keep + pad + head + 4 * body + tid), src + head + 4 * body + tid);
  cp_async_wait_all();
  __syncthreads();

  auto clean = [](float x) { return x == x ? x : -INFINITY; };
  auto get = [&](int i) { return clean(i < held ? keep[pad + i] : src[i]); };
  // maximum, with its lowest index (greedy rows need it)
  float m = -INFINITY;
  int at = 0x7FFFFFFF;
  for (int i = tid; i < n; i += kProbThreads) {
    const float x = get(i);
    if (x > m || at == 0x7FFFFFFF) {
      m = x;
      at = lo + i;
    }
  }
  auto better = [](float x, int i, float y, int j) { return x > y || (x == y && i < j); };
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float y = __shfl_xor_sync(0xFFFFFFFFu, m, o);
    const int j = __shfl_xor_sync(0xFFFFFFFFu, at, o);
    if (better(y, j, m, at)) {
      m = y;
      at = j;
    }
  }
  if (lane == 0) {
    red[warp] = m;
    redi[warp] = at;
  }
  __syncthreads();
  m = red[0];
  at = redi[0];
#pragma unroll
  for (int w = 1; w < kProbThreads / 32; ++w)
    if (better(red[w], redi[w], m, at)) {
      m = red[w];
      at = redi[w];
    }
  __syncthreads();

  // exponentials against the slice's own maximum; a slice of -inf has none
  const bool finite = m > -INFINITY && m < INFINITY;
  auto power = [&](float x, float y) {  // e^((x - y) / t) for x <= y, y finite; half the difference stays finite
    const float d = fmaf(0.5f, x, -0.5f * y);
    return d == 0.f ? 1.f : x == -INFINITY ? 0.f : expf(d * inv2);
  };
  auto weight = [&](float x) { return power(x, m); };
  float s = 0.f;
  if (!greedy && finite)
    for (int i = tid; i < n; i += kProbThreads) {
      const float e = weight(get(i));
      if (i < held) keep[pad + i] = e;
      s += e;
    }
  s = warp_sum(s);
  if (lane == 0) red[warp] = s;
  __syncthreads();
  if (tid == 0) {
    float t = 0.f;
    for (int w = 0; w < kProbThreads / 32; ++w) t += red[w];
    cta_m = m;
    cta_s = t;
    cta_i = at;
  }
  float M = m, S = 0.f;
  int best = at;
  if (a.cs == 1) {
    __syncthreads();
    S = cta_s;
  } else {
    cluster_sync();
    for (int r = 0; r < a.cs; ++r) {
      const float y = remote_f32(&cta_m, r);
      const int j = remote_s32(&cta_i, r);
      if (better(y, j, M, best)) {
        M = y;
        best = j;
      }
    }
    for (int r = 0; r < a.cs; ++r) {
      const float y = remote_f32(&cta_m, r), z = remote_f32(&cta_s, r);
      if (y > -INFINITY && M < INFINITY) S += z * power(y, M);
    }
    cluster_sync();  // nobody leaves while its shared memory is being read
  }
  const bool none = !(M > -INFINITY && M < INFINITY);
  const float f = none || greedy || !finite ? 0.f : power(m, M) / S;
  auto prob = [&](int i) {
    if (none) return 0.f;
    if (greedy) return lo + i == best ? 1.f : 0.f;
    if (!finite) return 0.f;
    return (i < held ? keep[pad + i] : weight(get(i))) * f;
  };
  const int h2 = min(n, (4 - pad) & 3), b2 = (n - h2) >> 2, t2 = n - h2 - 4 * b2;
  for (int i = tid; i < b2; i += kProbThreads) {
    const int e = h2 + 4 * i;
    *reinterpret_cast<float4 *>(dst + e) = make_float4(prob(e), prob(e + 1), prob(e + 2), prob(e + 3));
  }
  if (tid < h2) dst[tid] = prob(tid);
  if (tid < t2) dst[h2 + 4 * b2 + tid] = prob(h2 + 4 * b2 + tid);
}

// ---- verification -------------------------------------------------------------------------------
// A cluster per sequence.  Every CTA finds the first draft that is not accepted (a gather per draft), then the
// row of residuals is summed in slices: one read of that row of probs and of draft_probs, which bounds it.
// The draw must not depend on how the sum is split: each thread sums in two f32 terms (the error of
// every addition is kept, about 2^-46 of the sum), and threads, warps and CTAs are joined in f64.  The CTA
// and then the warp whose range holds the threshold are found from their sums; that warp walks its range.
constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;

struct VerifyArgs {
  const float *probs, *draft, *u, *u_next;
  const int32_t *tokens, *q_start, *kv_len;
  int32_t *accepted, *next_token, *kept_len;
  int B, T, V, cs, slice, sub;  // CTAs per sequence, elements per CTA and per warp (multiples of 4)
};

// probabilities as they count: NaN and negative ones 0, none above 2^100 (a sum of 2^20 stays finite)
QG_DEVICE float as_prob(float p) { return fminf(fmaxf(p, 0.f), 1.2676506002282294e30f); }

struct Residual {
  const float *p, *q;  // q NULL: p alone
  int x;               // with a certain draft, the token whose probability loses 1 (-1: none)
  QG_DEVICE float at(int v) const {
    float r = as_prob(__ldg(p + v));
    if (q) r = fmaxf(r - as_prob(__ldg(q + v)), 0.f);
    else if (v == x) r = fmaxf(r - 1.f, 0.f);
    return r;
  }
  // four elements from a place where p's (and q's) addresses are 16-byte aligned
  QG_DEVICE float4 at4(int v) const {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p + v));
    float4 r = make_float4(as_prob(a.x), as_prob(a.y), as_prob(a.z), as_prob(a.w));
    if (q) {
      const float4 b = __ldg(reinterpret_cast<const float4 *>(q + v));
      r = make_float4(fmaxf(r.x - as_prob(b.x), 0.f), fmaxf(r.y - as_prob(b.y), 0.f), fmaxf(r.z - as_prob(b.z), 0.f),
                      fmaxf(r.w - as_prob(b.w), 0.f));
    } else if (x >= v && x < v + 4) {
      float *e = x == v ? &r.x : x == v + 1 ? &r.y : x == v + 2 ? &r.z : &r.w;
      *e = fmaxf(*e - 1.f, 0.f);
    }
    return r;
  }
};

// (s, e) += x with the rounding error of the addition kept in e
QG_DEVICE void add_kept(float &s, float &e, float x) {
  const float t = __fadd_rn(s, x);
  const float b = __fadd_rn(t, -s);
  e = __fadd_rn(e, __fadd_rn(__fadd_rn(s, -__fadd_rn(t, -b)), __fadd_rn(x, -b)));
  s = t;
}

__global__ void __launch_bounds__(kVerThreads) draft_verify_kernel(const VerifyArgs a) {
  __shared__ double wsum[kVerWarps], cta_sum;
  __shared__ int wlast[kVerWarps], cta_last, stop, found, tail;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = static_cast<int>(blockIdx.x) / a.cs, rank = static_cast<int>(blockIdx.x) % a.cs;
  pdl_wait();
  pdl_launch_dependents();
  auto start = [&](int i) { return a.q_start ? max(0, min(a.T, __ldg(a.q_start + i))) : min(i, a.T); };
  const int t0 = start(b), t1 = start(b + 1);
  if (t1 <= t0) {  // the whole cluster leaves
    if (rank == 0 && tid == 0) {
      a.accepted[b] = 0;
      a.next_token[b] = -1;
      if (a.kept_len) a.kept_len[b] = a.kv_len[b];
    }
    return;
  }
  if (tid == 0) stop = t1 - 1;
  __syncthreads();
  for (int t = t0 + tid; t < t1 - 1; t += kVerThreads) {
    const int x = __ldg(a.tokens + t + 1);
    bool ok = false;
    if (x < 0 || x >= a.V) {
      if (rank == 0) atomicOr(&g_qg_status_draft, QG_STATUS_BIT_ID);
    } else {
      const size_t at = static_cast<size_t>(t) * a.V + x;
      const float un = fmaxf(__ldg(a.u + t), 0.f);
      const float q = a.draft ? as_prob(__ldg(a.draft + at)) : 1.f;
      ok = static_cast<double>(un) * q < static_cast<double>(as_prob(__ldg(a.probs + at)));  // exact products
    }
    if (!ok) atomicMin(&stop, t);
  }
  __syncthreads();
  const int t = stop;
  const bool refused = t < t1 - 1;
  const size_t row = static_cast<size_t>(t) * a.V;
  Residual r{a.probs + row, nullptr, -1};
  if (refused) {
    if (a.draft) r.q = a.draft + row;
    else r.x = __ldg(a.tokens + t + 1);
  }
  const double u = fmaxf(__ldg(a.u_next + b), 0.f);

  // element v sits at a 16-byte boundary when (row + v) % 4 == 0; slices and warps' ranges start at such places
  const int skew = static_cast<int>((4 - (row & 3)) & 3);
  auto edge = [&](int v) { return v <= 0 ? 0 : min(a.V, v + skew); };
  const int wlo = edge(rank * a.slice + min(a.slice, warp * a.sub));
  const int whi = edge(rank * a.slice + min(a.slice, (warp + 1) * a.sub));
  for (int pass = 0; pass < 2; ++pass) {
    // this warp's sum and its last element with mass
    float s = 0.f, e = 0.f;
    int last = -1;
    auto take = [&](float x, int v) {
      add_kept(s, e, x);
      if (x > 0.f) last = v;
    };
    const int head = min(whi - wlo, wlo == 0 ? skew : 0);
    const int body = (whi - wlo - head) >> 2, from = wlo + head;
    if (lane < head) take(r.at(wlo + lane), wlo + lane);
#pragma unroll 4
    for (int i = lane; i < body; i += 32) {
      const float4 x = r.at4(from + 4 * i);
      take(x.x, from + 4 * i);
      take(x.y, from + 4 * i + 1);
      take(x.z, from + 4 * i + 2);
      take(x.w, from + 4 * i + 3);
    }
    for (int v = from + 4 * body + lane; v < whi; v += 32) take(r.at(v), v);
    double d = static_cast<double>(s) + e;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      d += __shfl_xor_sync(0xFFFFFFFFu, d, o);
      last = max(last, __shfl_xor_sync(0xFFFFFFFFu, last, o));
    }
    if (lane == 0) {
      wsum[warp] = d;
      wlast[warp] = last;
    }
    __syncthreads();
    double own = 0.0;  // the same additions in every thread
    int own_last = -1;
    for (int w = 0; w < kVerWarps; ++w) {
      own += wsum[w];
      own_last = max(own_last, wlast[w]);
    }
    double total = own;
    int all_last = own_last;
    if (a.cs > 1) {
      if (tid == 0) {
        cta_sum = own;
        cta_last = own_last;
      }
      cluster_sync();
      total = 0.0;
      for (int k = 0; k < a.cs; ++k) {
        total += remote_f64(&cta_sum, k);
        all_last = max(all_last, remote_s32(&cta_last, k));
      }
    }
    if (!(total > 0.0) && pass == 0 && refused) {  // nothing is left of the difference: the row itself
      r.q = nullptr;
      r.x = -1;
      if (a.cs > 1) cluster_sync();  // the sums are written again
      __syncthreads();
      continue;
    }
    const double want = u * total;
    if (!(want < total)) {  // no mass at all; a random number of 1 or more, or rounding: the last one with mass
      if (rank == 0 && tid == 0) a.next_token[b] = total > 0.0 ? all_last : -1;
    } else {
      // the CTA whose range holds the threshold: every CTA makes the same additions and finds the same one
      double run = 0.0;
      int pick = 0;
      if (a.cs > 1)
        for (; pick < a.cs - 1; ++pick) {
          const double x = remote_f64(&cta_sum, pick);
          if (want < run + x) break;
          run += x;
        }
      if (pick == rank) {
        const double here = want - run;
        // its warp's range, in which then every thread takes a few elements
        int w = -1, some = 0;
        double rest = INFINITY, at = 0.0;
        for (int i = 0; i < kVerWarps; ++i) {
          if (w < 0 && here < at + wsum[i]) {
            w = i;
            rest = here - at;
          }
          if (wsum[i] > 0.0) some = i;
          at += wsum[i];
        }
        if (w < 0) w = some;  // rounding: the last range with mass, and in it the last element
        const int lo = edge(rank * a.slice + min(a.slice, w * a.sub));
        const int hi = edge(rank * a.slice + min(a.slice, (w + 1) * a.sub));
        const int each = (hi - lo + kVerThreads - 1) / kVerThreads;
        const int v0 = min(hi, lo + tid * each), v1 = min(hi, v0 + each);
        double c = 0.0;
        for (int v = v0; v < v1; ++v) c += r.at(v);
        double incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const double y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
          if (lane >= o) incl += y;
        }
        __syncthreads();  // everyone has read wsum
        if (lane == 31) wsum[warp] = incl;
        if (tid == 0) {
          found = 0x7FFFFFFF;
          tail = -1;
        }
        __syncthreads();
        double sum = __shfl_up_sync(0xFFFFFFFFu, incl, 1);
        if (lane == 0) sum = 0.0;
        for (int i = 0; i < warp; ++i) sum += wsum[i];
        for (int v = v0; v < v1; ++v) {
          const float x = r.at(v);
          if (!(x > 0.f)) continue;
          sum += x;
          atomicMax(&tail, v);
          if (sum > rest) {
            atomicMin(&found, v);
            break;
          }
        }
        __syncthreads();
        if (tid == 0) a.next_token[b] = found != 0x7FFFFFFF ? found : tail;
      }
    }
    break;
  }
  if (a.cs > 1) cluster_sync();  // nobody leaves while its shared memory is being read
  if (rank == 0 && tid == 0) {
    a.accepted[b] = t - t0;
    if (a.kept_len) a.kept_len[b] = a.kv_len[b] - (t1 - 1 - t);
  }
}

}  // namespace

namespace qg {

unsigned int read_status_draft(bool clear) {
  unsigned int v = 0;
  if (!g_launched) return v;
  if (cudaMemcpyFromSymbol(&v, g_qg_status_draft, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_qg_status_draft, &z, sizeof(z));
  }
  return v;
}

}  // namespace qg

extern "C" {

qg_status qg_token_probs(const float *logits, const float *temperature, int T, int64_t V, float *probs,
                         qg_stream_t stream) {
  if (T < 0 || T > 65535 || V < 1 || V > (1 << 20)) return QG_EINVAL_SHAPE;
  if (T == 0) return QG_OK;
  if (!logits || !probs) return QG_EINVAL_PTR;
  if (!qg::aligned16(logits) || !qg::aligned16(probs) || (reinterpret_cast<uintptr_t>(temperature) & 3u)) return QG_EALIGN;
  const qg::DeviceInfo &dev = qg::device_info();
  if (!dev.ok) return QG_ECUDA;
  // CTAs per row: enough to hold the row at two CTAs per SM, and to occupy the SMs when there are few rows
  int cs = 1;
  while (cs < 8 && (V > int64_t(cs) * 24 * 1024 || (int64_t(T) * cs < 2 * dev.sms && V > int64_t(cs) * 4096))) cs *= 2;
  ProbArgs a{logits, temperature, probs, T, static_cast<int>(V), cs, 0};
  a.slice = static_cast<int>((V + cs - 1) / cs + 3) & ~3;
  const size_t smem = (static_cast<size_t>(std::min(a.slice, kKeep - 4)) + 4) * sizeof(float);
  if (!qg::set_smem_attr(reinterpret_cast<const void *>(token_probs_kernel), static_cast<uint32_t>(smem))) return QG_ECUDA;
  const cudaError_t e = launch_cluster(token_probs_kernel, static_cast<unsigned>(T) * cs, kProbThreads, smem, cs,
                                       reinterpret_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return QG_ECUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ECUDA;
}

qg_status qg_draft_verify(const float *probs, const float *draft_probs, const int32_t *tokens, const float *u,
                          const float *u_next, const int32_t *q_start, int n_seqs, int n_rows, int64_t V,
                          int32_t *accepted, int32_t *next_token, const int32_t *kv_len, int32_t *kept_len,
                          qg_stream_t stream) {
  if (n_seqs < 0 || n_seqs > 65535 || n_rows < 0 || n_rows > (1 << 24) || V < 1 || V > (1 << 20)) return QG_EINVAL_SHAPE;
  if (!q_start && n_rows != n_seqs) return QG_EINVAL_SHAPE;
  if (n_seqs == 0) return QG_OK;
  if (!accepted || !next_token || !u_next || (n_rows > 0 && !probs) || (q_start && n_rows > 0 && (!tokens || !u)) ||
      !kv_len != !kept_len)
    return QG_EINVAL_PTR;
  auto odd = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
  if (!qg::aligned16(probs) || !qg::aligned16(draft_probs) || odd(tokens) || odd(u) || odd(u_next) || odd(q_start) ||
      odd(accepted) || odd(next_token) || odd(kv_len) || odd(kept_len))
    return QG_EALIGN;
  const qg::DeviceInfo &dev = qg::device_info();
  if (!dev.ok) return QG_ECUDA;
  int cs = 1;
  while (cs < 8 && int64_t(n_seqs) * cs < 4 * dev.sms && V > int64_t(cs) * 4096) cs *= 2;
  VerifyArgs a{probs, draft_probs, u, u_next, tokens, q_start, kv_len, accepted, next_token, kept_len,
               n_seqs, n_rows, static_cast<int>(V), cs, 0, 0};
  a.slice = static_cast<int>((V + cs - 1) / cs + 3) & ~3;
  a.sub = ((a.slice + kVerWarps - 1) / kVerWarps + 3) & ~3;
  g_launched = true;
  const cudaError_t e = launch_cluster(draft_verify_kernel, static_cast<unsigned>(n_seqs) * cs, kVerThreads, 0, cs,
                                       reinterpret_cast<cudaStream_t>(stream), a);
  if (e != cudaSuccess) return QG_ECUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ECUDA;
}

}  // extern "C"
