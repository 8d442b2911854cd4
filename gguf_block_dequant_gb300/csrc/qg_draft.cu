// qg_draft.cu -- the token steps of drafted decode: qg_token_probs (probabilities from logits) and
// qg_draft_verify (how many drafts the target accepts, and the token drawn behind them).
#include <algorithm>
#include <atomic>

#include "qg_common.cuh"
#include "qg_host.h"
#include "qg_mma.cuh"

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
QG_DEVICE int remote_s32(const int *p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote_addr(p, rank)) : "memory");
  return v;
}

// 16 bytes into the same place of CTA `rank`'s shared memory, counted on its barrier
QG_DEVICE void tell_remote(const float4 *place, float4 v, const uint64_t *bar, uint32_t rank) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
          remote_addr(place, rank)),
      "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(remote_addr(bar, rank))
      : "memory");
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

// how many clusters of a kernel the current device holds at once (asked once a device; the one kernel that asks)
int clusters_at_once(const void *kern, unsigned threads, size_t smem, int cluster) {
  static std::atomic<int> known[64];
  int d = 0;
  if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= 64) return 0;
  int n = known[d];
  if (n == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      return 0;
    }
    known[d] = n;
  }
  return n;
}

// ---- probabilities ------------------------------------------------------------------------------
// A row is split over a cluster of CTAs; each keeps its slice in registers, so a logit is read once and a
// probability written once (8 bytes an element: HBM bounds it).  Slices start at 16-byte boundaries of the
// whole tensor, so that rows of odd lengths still move 16 bytes at a time; only a row's two ends are moved by
// elements (5 rows of 151936: 4.8 us, the launch, the reads, the exchange and the writes one after another).  Each CTA sums the exponentials against its own maximum; one exchange of (maximum, sum) gives every
// CTA its factor.  Exponentials are powers of two of (x/2 - m/2) (2 log2(e) / t): the half difference stays finite, six
// instructions an element.
constexpr int kProbThreads = 512;
constexpr int kProbWarps = kProbThreads / 32;
constexpr int kKeep = 48 * 1024;  // floats of a slice that stay in shared memory

struct ProbArgs {
  const float *logits, *temperature;
  float *probs;
  int T, V, cs, slice;  // CTAs per row, elements per CTA (a multiple of 4)
};

QG_DEVICE void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// the best of the CTA's (value, index) pairs, the lowest index among equals
QG_DEVICE void best_of(float &m, int &at, float *red, int *redi) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float y = __shfl_xor_sync(0xFFFFFFFFu, m, o);
    const int j = __shfl_xor_sync(0xFFFFFFFFu, at, o);
    if (y > m || (y == m && j < at)) m = y, at = j;
  }
  if (lane == 0) red[warp] = m, redi[warp] = at;
  __syncthreads();
  m = red[lane & (kProbWarps - 1)];
  at = redi[lane & (kProbWarps - 1)];
#pragma unroll
  for (int o = kProbWarps / 2; o; o >>= 1) {
    const float y = __shfl_xor_sync(0xFFFFFFFFu, m, o);
    const int j = __shfl_xor_sync(0xFFFFFFFFu, at, o);
    if (y > m || (y == m && j < at)) m = y, at = j;
  }
}

template <int NV>
__global__ void __launch_bounds__(kProbThreads) probs_kernel(const ProbArgs a) {
  __shared__ float red[kProbWarps], reds[kProbWarps];
  __shared__ int redi[kProbWarps];
  __shared__ __align__(16) float4 told[8];  // (maximum, sum, index) of each CTA
  __shared__ uint64_t told_bar;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = static_cast<int>(blockIdx.x) / a.cs, rank = static_cast<int>(blockIdx.x) % a.cs;
  if (a.cs > 1) {
    if (tid == 0) {
      mbar_init(&told_bar, 1);
      fence_mbar_init();
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // its other half is where it is needed
  }
  pdl_wait();
  pdl_launch_dependents();
  const long long r0 = static_cast<long long>(row) * a.V, r1 = r0 + a.V;  // elements of the tensor
  const long long g0 = (r0 & ~3LL) + static_cast<long long>(rank) * a.slice;
  const int count = static_cast<int>(min(static_cast<long long>(a.slice), r1 - g0));  // may be negative: an empty slice
  float4 x[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = 4 * (tid + k * kProbThreads);
    const long long g = g0 + i;
    x[k] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (i < count) {
      if (g >= r0 && g + 4 <= r1) {
        x[k] = *reinterpret_cast<const float4 *>(a.logits + g);
      } else {
        if (g >= r0) x[k].x = a.logits[g];
        if (g + 1 >= r0 && g + 1 < r1) x[k].y = a.logits[g + 1];
        if (g + 2 >= r0 && g + 2 < r1) x[k].z = a.logits[g + 2];
        if (g + 3 >= r0 && g + 3 < r1) x[k].w = a.logits[g + 3];
      }
    }
  }
  const float tau = a.temperature ? __ldg(a.temperature + row) : 1.f;
  const bool greedy = !(tau > 0.f);
  // fmaxf leaves NaN out
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < NV; ++k) m = fmaxf(m, fmaxf(fmaxf(x[k].x, x[k].y), fmaxf(x[k].z, x[k].w)));
  int at = 0x7FFFFFFF;
  if (greedy) {  // the lowest index of this thread's largest
#pragma unroll
    for (int k = NV - 1; k >= 0; --k) {
      const int i = 4 * (tid + k * kProbThreads) + static_cast<int>(g0 - r0);
      if (x[k].w == m) at = i + 3;
      if (x[k].z == m) at = i + 2;
      if (x[k].y == m) at = i + 1;
      if (x[k].x == m) at = i;
    }
  }
  best_of(m, at, red, redi);
  const bool finite = m > -INFINITY && m < INFINITY;
  // 2 log2(e) / t within f32: a difference of 0 stays 0 and an infinite one infinite
  const float c = fminf(fmaxf(2.8853900817779268f / tau, 1e-44f), 3e38f), hm = -0.5f * m;
  float s = 0.f;
  if (!greedy && finite) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      auto power = [&](float y) { return ex2(fmaxf(fmaf(0.5f, y, hm) * c, -200.f)); };  // NaN counts as -inf
      x[k] = make_float4(power(x[k].x), power(x[k].y), power(x[k].z), power(x[k].w));
      s += (x[k].x + x[k].y) + (x[k].z + x[k].w);
    }
  }
  s = warp_sum(s);
  if (lane == 0) reds[warp] = s;
  __syncthreads();
  s = reds[lane & (kProbWarps - 1)];
#pragma unroll
  for (int o = kProbWarps / 2; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  float M = m, S = s;
  int best = at;
  if (a.cs > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (tid == 0) mbar_arrive_expect_tx(&told_bar, 16 * a.cs);
    if (tid < a.cs) tell_remote(&told[rank], make_float4(m, s, __int_as_float(at), 0.f), &told_bar, tid);
    if (!mbar_wait(&told_bar, 0)) atomicOr(&g_qg_status_draft, QG_STATUS_BIT_TIMEOUT);
    // a lane per CTA
    const float4 other = told[lane & (a.cs - 1)];
    const float om = other.x, os = other.y;
    M = om;
    best = __float_as_int(other.z);
    for (int o = a.cs / 2; o; o >>= 1) {
      const float y = __shfl_xor_sync(0xFFFFFFFFu, M, o);
      const int j = __shfl_xor_sync(0xFFFFFFFFu, best, o);
      if (y > M || (y == M && j < best)) M = y, best = j;
    }
    S = om > -INFINITY && M < INFINITY ? os * ex2(fmaxf((0.5f * om - 0.5f * M) * c, -200.f)) : 0.f;
    for (int o = a.cs / 2; o; o >>= 1) S += __shfl_xor_sync(0xFFFFFFFFu, S, o);
  }
  const bool none = !(M > -INFINITY && M < INFINITY);
  const float f = none || greedy || !finite ? 0.f : ex2(fmaxf((0.5f * m - 0.5f * M) * c, -200.f)) / S;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = 4 * (tid + k * kProbThreads);
    const long long g = g0 + i;
    if (i < count) {
      float4 y;
      if (f == 0.f) {
        const int v = greedy && !none ? best - static_cast<int>(g - r0) : -1;
        y = make_float4(v == 0 ? 1.f : 0.f, v == 1 ? 1.f : 0.f, v == 2 ? 1.f : 0.f, v == 3 ? 1.f : 0.f);
      } else {
        y = make_float4(x[k].x * f, x[k].y * f, x[k].z * f, x[k].w * f);
      }
      if (g >= r0 && g + 4 <= r1) {
        *reinterpret_cast<float4 *>(a.probs + g) = y;
      } else {
        if (g >= r0) a.probs[g] = y.x;
        if (g + 1 >= r0 && g + 1 < r1) a.probs[g + 1] = y.y;
        if (g + 2 >= r0 && g + 2 < r1) a.probs[g + 2] = y.z;
        if (g + 3 >= r0 && g + 3 < r1) a.probs[g + 3] = y.w;
      }
    }
  }
}

// The same for many rows that start at 16-byte boundaries: clusters stay on their SMs and take every so many-th row, and a CTA's slice
// of the next row is copied to shared memory while this one's, in registers, is worked on and written, so that reads, exchanges and writes
// of different rows overlap (200 rows of 151936, 243 MB: 44.7 us, 5.4 TB/s, 0.81 of the copy; the kernel above 59.8; with a cluster
// barrier for the exchange, which waits for the writes of the row before, 59.4).
template <int NV>
__global__ void __launch_bounds__(kProbThreads, 2) probs_stream_kernel(const ProbArgs a, int clusters) {
  extern __shared__ __align__(128) float4 slice[];
  __shared__ float red[kProbWarps], reds[kProbWarps];
  __shared__ int redi[kProbWarps];
  __shared__ __align__(16) float4 told[2][8];  // (maximum, sum, index) of each CTA, by the row's parity
  __shared__ uint64_t full, told_bar[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x) % a.cs, first = static_cast<int>(blockIdx.x) / a.cs;
  const int lo = rank * a.slice, n = max(0, min(a.slice, a.V - lo)) / 4;  // vectors
  if (tid == 0) {
    mbar_init(&full, 1);
    mbar_init(&told_bar[0], 1);
    mbar_init(&told_bar[1], 1);
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  cluster_sync();  // the barriers stand
  auto ask = [&](int row) {
    mbar_arrive_expect_tx(&full, 16 * n);
    bulk_g2s<true>(slice, a.logits + static_cast<long long>(row) * a.V + lo, 16 * n, &full);
  };
  if (tid == 0 && n && first < a.T) ask(first);
  int k = 0;
  for (int row = first; row < a.T; row += clusters, ++k) {
    const int buf = k & 1;
    const float tau = a.temperature ? __ldg(a.temperature + row) : 1.f;
    const bool greedy = !(tau > 0.f);
    if (n && !mbar_wait(&full, k & 1)) atomicOr(&g_qg_status_draft, QG_STATUS_BIT_TIMEOUT);
    float4 x[NV];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * kProbThreads;
      x[i] = v < n ? slice[v] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      m = fmaxf(m, fmaxf(fmaxf(x[i].x, x[i].y), fmaxf(x[i].z, x[i].w)));
    }
    int at = 0x7FFFFFFF;
    if (greedy) {
#pragma unroll
      for (int i = NV - 1; i >= 0; --i) {
        const int e = lo + 4 * (tid + i * kProbThreads);
        if (x[i].w == m) at = e + 3;
        if (x[i].z == m) at = e + 2;
        if (x[i].y == m) at = e + 1;
        if (x[i].x == m) at = e;
      }
    }
    best_of(m, at, red, redi);  // everyone has read the slice
    if (tid == 0 && n && row + clusters < a.T) ask(row + clusters);
    const bool finite = m > -INFINITY && m < INFINITY;
    const float c = fminf(fmaxf(2.8853900817779268f / tau, 1e-44f), 3e38f), hm = -0.5f * m;
    float s = 0.f;
    if (!greedy && finite) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        auto power = [&](float y) { return ex2(fmaxf(fmaf(0.5f, y, hm) * c, -200.f)); };
        x[i] = make_float4(power(x[i].x), power(x[i].y), power(x[i].z), power(x[i].w));
        s += (x[i].x + x[i].y) + (x[i].z + x[i].w);
      }
    }
    s = warp_sum(s);
    if (lane == 0) reds[warp] = s;
    __syncthreads();
    s = reds[lane & (kProbWarps - 1)];
#pragma unroll
    for (int o = kProbWarps / 2; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    // told to every CTA's shared memory, with its barrier: a cluster barrier would wait for the row before to be written.  Two
    // places in turn: who is a row ahead has heard from everyone about the row before, after they left this place
    if (tid == 0) mbar_arrive_expect_tx(&told_bar[buf], 16 * a.cs);
    if (tid < a.cs) tell_remote(&told[buf][rank], make_float4(m, s, __int_as_float(at), 0.f), &told_bar[buf], tid);
    if (!mbar_wait(&told_bar[buf], (k >> 1) & 1)) atomicOr(&g_qg_status_draft, QG_STATUS_BIT_TIMEOUT);
    const float4 other = told[buf][lane & (a.cs - 1)];
    const float om = other.x, os = other.y;
    float M = om;
    int best = __float_as_int(other.z);
    for (int o = a.cs / 2; o; o >>= 1) {
      const float y = __shfl_xor_sync(0xFFFFFFFFu, M, o);
      const int j = __shfl_xor_sync(0xFFFFFFFFu, best, o);
      if (y > M || (y == M && j < best)) M = y, best = j;
    }
    float S = om > -INFINITY && M < INFINITY ? os * ex2(fmaxf((0.5f * om - 0.5f * M) * c, -200.f)) : 0.f;
    for (int o = a.cs / 2; o; o >>= 1) S += __shfl_xor_sync(0xFFFFFFFFu, S, o);
    const bool none = !(M > -INFINITY && M < INFINITY);
    const float f = none || greedy || !finite ? 0.f : ex2(fmaxf((0.5f * m - 0.5f * M) * c, -200.f)) / S;
    float4 *dst = reinterpret_cast<float4 *>(a.probs + static_cast<long long>(row) * a.V + lo);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = tid + i * kProbThreads;
      if (v >= n) continue;
      if (f == 0.f) {
        const int e = greedy && !none ? best - lo - 4 * v : -1;
        dst[v] = make_float4(e == 0 ? 1.f : 0.f, e == 1 ? 1.f : 0.f, e == 2 ? 1.f : 0.f, e == 3 ? 1.f : 0.f);
      } else {
        dst[v] = make_float4(x[i].x * f, x[i].y * f, x[i].z * f, x[i].w * f);
      }
    }
  }
}

// Vocabularies that eight CTAs' registers do not hold: slices in shared memory, what does not fit is read again.
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
// The draw must not depend on how the sum is split, so sums are kept in two f32 terms (the error of every addition
// is kept: 2^-40 of the sum at the least; f64 additions would cost more than the reads here, at two a clock and SM).
// The CTA and then the warp whose range holds the threshold are found from their sums, by one warp of each CTA
// with the same additions, and the threads of that CTA search that warp's range.

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

// a sum and the rounding errors of its additions; s + e with |e| at most half a step of s
struct Sum {
  float s, e;
};
QG_DEVICE void add_kept(Sum &a, float x) {  // not brought to normal form: for many additions in a row
  const float t = __fadd_rn(a.s, x);
  const float b = __fadd_rn(t, -a.s);
  a.e = __fadd_rn(a.e, __fadd_rn(__fadd_rn(a.s, -__fadd_rn(t, -b)), __fadd_rn(x, -b)));
  a.s = t;
}
QG_DEVICE Sum normal(float s, float e) {
  const float t = __fadd_rn(s, e);
  return {t, __fadd_rn(e, -__fadd_rn(t, -s))};
}
QG_DEVICE Sum operator+(Sum a, Sum b) {
  const float e = __fadd_rn(a.e, b.e);
  a.e = 0.f;
  add_kept(a, b.s);
  return normal(a.s, __fadd_rn(a.e, e));
}
QG_DEVICE bool operator<(Sum a, Sum b) { return a.s < b.s || (a.s == b.s && a.e < b.e); }
QG_DEVICE Sum times(Sum a, float u) {
  const float p = __fmul_rn(a.s, u);
  return normal(p, __fmaf_rn(a.e, u, __fmaf_rn(a.s, u, -p)));
}
QG_DEVICE Sum shfl_up(Sum a, int o) {
  return {__shfl_up_sync(0xFFFFFFFFu, a.s, o), __shfl_up_sync(0xFFFFFFFFu, a.e, o)};
}
QG_DEVICE Sum shfl_xor(Sum a, int o) {
  return {__shfl_xor_sync(0xFFFFFFFFu, a.s, o), __shfl_xor_sync(0xFFFFFFFFu, a.e, o)};
}
QG_DEVICE Sum shfl(Sum a, int i) { return {__shfl_sync(0xFFFFFFFFu, a.s, i), __shfl_sync(0xFFFFFFFFu, a.e, i)}; }
// running sums over the first N lanes
template <int N>
QG_DEVICE Sum scan(Sum a) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < N; o <<= 1) {
    const Sum y = shfl_up(a, o);
    if (lane >= o) a = y + a;
  }
  return a;
}

// NT threads a CTA: 256 keep 64 sequences' CTAs on the SMs all at once (20 us; 35 with 512), 1024 read a slice in one round of
// loads where there are few sequences
template <int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) draft_verify_kernel(const VerifyArgs a) {
  constexpr int kVerThreads = NT, kVerWarps = NT / 32;
  __shared__ Sum wsum[kVerWarps], s_rest;
  __shared__ int wlast[kVerWarps], stop, found, tail, s_pick;  // s_pick: the warp whose range is searched
  __shared__ __align__(16) float4 told[2][8];  // (sum, its error, last element with mass) of each CTA, for both passes
  __shared__ uint64_t told_bar[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = static_cast<int>(blockIdx.x) / a.cs, rank = static_cast<int>(blockIdx.x) % a.cs;
  if (a.cs > 1) {
    if (tid == 0) {
      mbar_init(&told_bar[0], 1);
      mbar_init(&told_bar[1], 1);
      fence_mbar_init();
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // its other half is where it is needed
  }
  pdl_wait();
  pdl_launch_dependents();
  auto start = [&](int i) { return a.q_start ? max(0, min(a.T, __ldg(a.q_start + i))) : min(i, a.T); };
  const int t0 = start(b), t1 = start(b + 1);
  if (t1 <= t0) {  // the whole cluster leaves
    if (a.cs > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (rank == 0 && tid == 0) {
      a.accepted[b] = 0;
      a.next_token[b] = -1;
      if (a.kept_len) a.kept_len[b] = a.kv_len[b];
    }
    return;
  }
  const float u = fmaxf(__ldg(a.u_next + b), 0.f);
  int t = t1 - 1;
  if (t > t0) {
    if (tid == 0) stop = t;
    __syncthreads();
    for (int i = t0 + tid; i < t1 - 1; i += kVerThreads) {
      const int x = __ldg(a.tokens + i + 1);
      bool ok = false;
      if (x < 0 || x >= a.V) {
        if (rank == 0) atomicOr(&g_qg_status_draft, QG_STATUS_BIT_ID);
      } else {
        const size_t at = static_cast<size_t>(i) * a.V + x;
        const float un = fmaxf(__ldg(a.u + i), 0.f);
        const float q = a.draft ? as_prob(__ldg(a.draft + at)) : 1.f;
        ok = static_cast<double>(un) * q < static_cast<double>(as_prob(__ldg(a.probs + at)));  // exact products
      }
      if (!ok) atomicMin(&stop, i);
    }
    __syncthreads();
    t = stop;
  }
  const bool refused = t < t1 - 1;
  const size_t row = static_cast<size_t>(t) * a.V;
  Residual r{a.probs + row, nullptr, -1};
  if (refused) {
    if (a.draft) r.q = a.draft + row;
    else r.x = __ldg(a.tokens + t + 1);
  }

  // element v sits at a 16-byte boundary when (row + v) % 4 == 0; slices and warps' ranges start at such places
  const int skew = static_cast<int>((4 - (row & 3)) & 3);
  auto edge = [&](int v) { return v <= 0 ? 0 : min(a.V, v + skew); };
  auto range = [&](int w) { return edge(rank * a.slice + min(a.slice, w * a.sub)); };
  const int wlo = range(warp), whi = range(warp + 1);
  for (int pass = 0; pass < 2; ++pass) {
    // this warp's sum, in two chains, and its last element with mass
    Sum s{0.f, 0.f}, s2{0.f, 0.f};
    int last = -1;
    auto take = [&](float x, int v) {
      add_kept(v & 1 ? s2 : s, x);
      if (x > 0.f) last = v;
    };
    const int head = min(whi - wlo, wlo == 0 ? skew : 0);
    const int body = (whi - wlo - head) >> 2, from = wlo + head;
    if (lane < head) take(r.at(wlo + lane), wlo + lane);
#pragma unroll 5
    for (int i = lane; i < body; i += 32) {
      const float4 x = r.at4(from + 4 * i);
      add_kept(s, x.x);
      add_kept(s2, x.y);
      add_kept(s, x.z);
      add_kept(s2, x.w);
      const int v = from + 4 * i;
      if (x.x > 0.f) last = v;
      if (x.y > 0.f) last = v + 1;
      if (x.z > 0.f) last = v + 2;
      if (x.w > 0.f) last = v + 3;
    }
    for (int v = from + 4 * body + lane; v < whi; v += 32) take(r.at(v), v);
    s = normal(s.s, s.e) + normal(s2.s, s2.e);
#pragma unroll
    for (int o = 16; o; o >>= 1) s = s + shfl_xor(s, o);
    last = __reduce_max_sync(0xFFFFFFFFu, last);
    if (lane == 0) {
      wsum[warp] = s;
      wlast[warp] = last;
    }
    __syncthreads();
    // running sums of the CTA's warps, in every warp alike
    Sum run = scan<kVerWarps>(lane < kVerWarps ? wsum[lane] : Sum{0.f, 0.f});
    const Sum own = shfl(run, kVerWarps - 1);
    const int own_last = __reduce_max_sync(0xFFFFFFFFu, lane < kVerWarps ? wlast[lane] : -1);
    Sum total = own, before{0.f, 0.f};
    int all_last = own_last, pick = 0;
    Sum want = times(total, u);
    if (a.cs > 1) {
      // every CTA tells every other
      if (pass == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      if (tid == 0) mbar_arrive_expect_tx(&told_bar[pass], 16 * a.cs);
      if (tid < a.cs)
        tell_remote(&told[pass][rank], make_float4(own.s, own.e, __int_as_float(own_last), 0.f), &told_bar[pass], tid);
      if (!mbar_wait(&told_bar[pass], 0)) atomicOr(&g_qg_status_draft, QG_STATUS_BIT_TIMEOUT);
      Sum x{0.f, 0.f};
      int l = -1;
      if (lane < a.cs) {
        const float4 other = told[pass][lane];
        x = {other.x, other.y};
        l = __float_as_int(other.z);
      }
      const Sum upto = scan<8>(x);
      total = shfl(upto, a.cs - 1);
      all_last = __reduce_max_sync(0xFFFFFFFFu, l);
      // the first CTA whose running sum passes the threshold: every CTA finds the same
      want = times(total, u);
      const unsigned over = __ballot_sync(0xFFFFFFFFu, lane < a.cs && want < upto);
      pick = over ? __ffs(over) - 1 : a.cs;
      if (pick > 0) before = shfl(upto, pick - 1);
    }
    if (!(total.s > 0.f) && pass == 0 && refused) {  // nothing is left of the difference: the row itself
      r.q = nullptr;
      r.x = -1;
      __syncthreads();
      continue;
    }
    if (!(want < total)) {  // no mass at all; a random number of 1 or more, or rounding: the last one with mass
      if (rank == 0 && tid == 0) a.next_token[b] = total.s > 0.f ? all_last : -1;
    } else if (pick == rank) {
      if (warp == 0) {
        // the first warp's range that passes it; by rounding none may: then the last with mass, and in it the last element
        const Sum here = want + Sum{-before.s, -before.e};
        const unsigned over = __ballot_sync(0xFFFFFFFFu, lane < kVerWarps && here < run);
        const unsigned some = __ballot_sync(0xFFFFFFFFu, lane < kVerWarps && wsum[lane & (kVerWarps - 1)].s > 0.f);
        const int w = over ? __ffs(over) - 1 : 31 - __clz(some);
        const Sum upto = shfl(run, max(w - 1, 0));
        if (lane == 0) {
          s_pick = w;
          s_rest = !over ? Sum{INFINITY, 0.f} : w > 0 ? here + Sum{-upto.s, -upto.e} : here;
          found = 0x7FFFFFFF;
          tail = -1;
        }
      }
      __syncthreads();
      const int lo = range(s_pick), hi = range(s_pick + 1);
      const Sum rest = s_rest;
      const int each = (hi - lo + kVerThreads - 1) / kVerThreads;
      const int v0 = min(hi, lo + tid * each), v1 = min(hi, v0 + each);
      Sum c{0.f, 0.f};
      for (int v = v0; v < v1; ++v) add_kept(c, r.at(v));
      const Sum incl = scan<32>(normal(c.s, c.e));
      if (lane == 31) wsum[warp] = incl;  // warp 0 has read the ranges' sums
      __syncthreads();
      const Sum warps = scan<kVerWarps>(lane < kVerWarps ? wsum[lane] : Sum{0.f, 0.f});
      Sum sum = shfl_up(incl, 1);
      if (lane == 0) sum = {0.f, 0.f};
      const Sum w0 = shfl(warps, max(warp - 1, 0));
      if (warp > 0) sum = w0 + sum;
      for (int v = v0; v < v1; ++v) {
        const float x = r.at(v);
        if (!(x > 0.f)) continue;
        sum = sum + Sum{x, 0.f};
        atomicMax(&tail, v);
        if (rest < sum) {
          atomicMin(&found, v);
          break;
        }
      }
      __syncthreads();
      if (tid == 0) a.next_token[b] = found != 0x7FFFFFFF ? found : tail;
    }
    break;
  }
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
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // CTAs per row: as many as hold the row in registers, and more to occupy the SMs when there are few rows
  g_launched = true;
  constexpr int kHold = 4 * kProbThreads;  // elements a CTA holds in one vector a thread
  int cs = 1;
  while (cs < 8 && (V + 3 > int64_t(cs) * 10 * kHold || (int64_t(T) * cs < 2 * dev.sms && V > int64_t(cs) * kHold))) cs *= 2;
  ProbArgs a{logits, temperature, probs, T, static_cast<int>(V), cs, 0};
  // slices of whole vectors, from the boundary at or below a row's start
  a.slice = static_cast<int>((V + 3 + 4 * cs - 1) / (4 * cs)) * 4;
  const int nv = (a.slice + kHold - 1) / kHold;
  const unsigned blocks = static_cast<unsigned>(T) * cs;
  cudaError_t e;
  // many rows of whole vectors, not in place (the next row is read early, but that is another row): clusters that stay
  int clusters = 0;
  if (V % 4 == 0 && cs == 8 && nv > 5 && nv <= 10 && T >= 4 * (dev.sms / cs)) {
    constexpr size_t most = sizeof(float) * 10 * kHold;
    if (!qg::set_smem_attr(reinterpret_cast<const void *>(probs_stream_kernel<10>), static_cast<uint32_t>(most))) return QG_ECUDA;
    clusters = clusters_at_once(reinterpret_cast<const void *>(probs_stream_kernel<10>), kProbThreads, most, cs);
  }
  if (clusters > 0) {
    e = launch_cluster(probs_stream_kernel<10>, static_cast<unsigned>(std::min(clusters, T)) * cs, kProbThreads, sizeof(float) * a.slice, cs, st, a, std::min(clusters, T));
  } else if (nv <= 2) e = launch_cluster(probs_kernel<2>, blocks, kProbThreads, 0, cs, st, a);
  else if (nv <= 5) e = launch_cluster(probs_kernel<5>, blocks, kProbThreads, 0, cs, st, a);
  else if (nv <= 10) e = launch_cluster(probs_kernel<10>, blocks, kProbThreads, 0, cs, st, a);
  else if (nv <= 17) e = launch_cluster(probs_kernel<17>, blocks, kProbThreads, 0, cs, st, a);
  else {
    a.slice = static_cast<int>((V + cs - 1) / cs + 3) & ~3;
    const size_t smem = (static_cast<size_t>(std::min(a.slice, kKeep - 4)) + 4) * sizeof(float);
    if (!qg::set_smem_attr(reinterpret_cast<const void *>(token_probs_kernel), static_cast<uint32_t>(smem))) return QG_ECUDA;
    e = launch_cluster(token_probs_kernel, blocks, kProbThreads, smem, cs, st, a);
  }
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
  const bool few = int64_t(n_seqs) * cs <= dev.sms;
  const int warps = few ? 32 : 8;
  a.sub = ((a.slice + warps - 1) / warps + 3) & ~3;
  g_launched = true;
  const unsigned blocks = static_cast<unsigned>(n_seqs) * cs;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = few ? launch_cluster(draft_verify_kernel<1024>, blocks, 1024, 0, cs, st, a)
                            : launch_cluster(draft_verify_kernel<256>, blocks, 256, 0, cs, st, a);
  if (e != cudaSuccess) return QG_ECUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ECUDA;
}

}  // extern "C"
