// qg_delta.cu -- the gated delta rule: token after token, for decode steps and drafts.
#include <algorithm>
#include <atomic>

#include "qg_delta.cuh"

__device__ unsigned int g_qg_status_delta;   // this translation unit's device status word
static std::atomic<bool> g_launched{false};  // whether a kernel that may set it has been launched

namespace {

using qg::DeltaArgs;

// ---- token after token ----------------------------------------------------------------------
// The columns of a state are independent, so a CTA takes JC of a value head's columns: thread (row group,
// column group) holds NR rows of four columns in registers, which are read once and written once a call (and once a
// token that is kept): HBM bounds a batch of single tokens.  Both products with the old state,
// S^T k and S^T q, are summed in one pass over the registers (the output is e^g S^T q + (q . k) u), so a token
// costs one exchange between warps, and the wait for its values and its state's slot, which are loaded when it is its turn (0.6 us in
// all where one sequence is alone; of 16 sequences of 2 to 7 kept tokens the warps wait for loads most).  Queries, keys and gates of up to TG tokens are made ready at a time, a warp per
// token.
constexpr int TG = 16;

template <int DK, int JC, int NT>
__global__ void __launch_bounds__(NT, NT == 128 ? 5 : 2) delta_tokens_kernel(const DeltaArgs a, int first_len) {
  constexpr int kWarps = NT / 32;
  constexpr int CG = JC / 4;            // lanes side by side in a row
  constexpr int RPW = 32 / CG;          // row groups of a warp
  constexpr int NR = DK / (kWarps * RPW);  // rows of a thread
  static_assert(NR >= 1, "rows");
  __shared__ __align__(16) float sk[TG][DK], sq[TG][DK];
  __shared__ float s_alpha[TG], s_beta[TG], s_qk[TG];
  __shared__ __align__(16) float4 red_k[2][kWarps][CG], red_q[2][kWarps][CG];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cg = lane % CG, rg = warp * RPW + lane / CG;
  const int parts = a.Dv / JC;
  const int part = static_cast<int>(blockIdx.x) % parts;
  const int bh = static_cast<int>(blockIdx.x) / parts;
  const int h = bh % a.Hv, b = bh / a.Hv;
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = qg::delta_tok(a, b), n = qg::delta_tok(a, b + 1) - t0;
  if (n <= 0 || n >= first_len) return;  // longer sequences are another kernel's
  const int hk = qg::delta_key_head(a, h), col = part * JC + 4 * cg, row0 = rg * NR;

  const int in = a.state_in ? __ldg(a.state_in + b) : -1;
  const bool teller = tid == 0 && part == 0 && h == 0;
  if (teller && (in < -1 || in >= a.n_slots)) atomicOr(&g_qg_status_delta, QG_STATUS_BIT_ID);
  float4 S[NR];
  {
    const bool have = in >= 0 && in < a.n_slots;
    const float *p = a.states + (have ? in : 0) * a.slot_stride + (static_cast<long long>(h) * DK + row0) * a.Dv + col;
#pragma unroll
    for (int i = 0; i < NR; ++i)
      S[i] = have ? *reinterpret_cast<const float4 *>(p + static_cast<long long>(i) * a.Dv) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  auto leave = [&](int slot) {
    if (slot == -1) return;
    if (slot < 0 || slot >= a.n_slots) {
      if (teller) atomicOr(&g_qg_status_delta, QG_STATUS_BIT_ID);
      return;
    }
    float *p = a.states + slot * a.slot_stride + (static_cast<long long>(h) * DK + row0) * a.Dv + col;
#pragma unroll
    for (int i = 0; i < NR; ++i) *reinterpret_cast<float4 *>(p + static_cast<long long>(i) * a.Dv) = S[i];
  };

  int buf = 0;
  for (int g0 = 0; g0 < n; g0 += TG) {
    const int m = min(TG, n - g0);
    __syncthreads();
    for (int j = warp; j < m; j += kWarps) {
      const int t = t0 + g0 + j;
      constexpr int E = DK / 32;
      float qv[E], kv[E], qq = 0.f, kk = 0.f, qk = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        qv[i] = __ldg(a.q + t * a.q_stride + hk * DK + lane + 32 * i);
        kv[i] = __ldg(a.k + t * a.k_stride + hk * DK + lane + 32 * i);
        qq = fmaf(qv[i], qv[i], qq);
        kk = fmaf(kv[i], kv[i], kk);
      }
      float qs = a.scale, ks = 1.f;
      if (a.l2norm) {
        qs *= 1.f / sqrtf(warp_sum(qq) + a.eps);
        ks = 1.f / sqrtf(warp_sum(kk) + a.eps);
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        qv[i] *= qs;
        kv[i] *= ks;
        qk = fmaf(qv[i], kv[i], qk);
        sq[j][lane + 32 * i] = qv[i];
        sk[j][lane + 32 * i] = kv[i];
      }
      qk = warp_sum(qk);
      if (lane == 0) {
        const float2 ga = qg::delta_gates(a, t, h);
        s_alpha[j] = expf(ga.x);
        s_beta[j] = ga.y;
        s_qk[j] = qk;
      }
    }
    __syncthreads();
    for (int j = 0; j < m; ++j) {
      const int t = t0 + g0 + j;
      const float4 v = __ldg(reinterpret_cast<const float4 *>(a.v + t * a.v_stride + static_cast<long long>(h) * a.Dv + col));
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      float kr[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float k = sk[j][row0 + i], q = sq[j][row0 + i];
        kr[i] = k;
        x.x = fmaf(S[i].x, k, x.x);
        x.y = fmaf(S[i].y, k, x.y);
        x.z = fmaf(S[i].z, k, x.z);
        x.w = fmaf(S[i].w, k, x.w);
        y.x = fmaf(S[i].x, q, y.x);
        y.y = fmaf(S[i].y, q, y.y);
        y.z = fmaf(S[i].z, q, y.z);
        y.w = fmaf(S[i].w, q, y.w);
      }
#pragma unroll
      for (int o = CG; o < 32; o <<= 1) {
        x.x += __shfl_xor_sync(0xFFFFFFFFu, x.x, o);
        x.y += __shfl_xor_sync(0xFFFFFFFFu, x.y, o);
        x.z += __shfl_xor_sync(0xFFFFFFFFu, x.z, o);
        x.w += __shfl_xor_sync(0xFFFFFFFFu, x.w, o);
        y.x += __shfl_xor_sync(0xFFFFFFFFu, y.x, o);
        y.y += __shfl_xor_sync(0xFFFFFFFFu, y.y, o);
        y.z += __shfl_xor_sync(0xFFFFFFFFu, y.z, o);
        y.w += __shfl_xor_sync(0xFFFFFFFFu, y.w, o);
      }
      if (lane < CG) {
        red_k[buf][warp][lane] = x;
        red_q[buf][warp][lane] = y;
      }
      __syncthreads();
      x = red_k[buf][0][cg];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 z = red_k[buf][w][cg];
        x = make_float4(x.x + z.x, x.y + z.y, x.z + z.z, x.w + z.w);
      }
      const float al = s_alpha[j], be = s_beta[j];
      const float4 u = make_float4(be * (v.x - al * x.x), be * (v.y - al * x.y), be * (v.z - al * x.z), be * (v.w - al * x.w));
      if (rg == 0) {
        y = red_q[buf][0][cg];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          const float4 z = red_q[buf][w][cg];
          y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
        }
        const float qk = s_qk[j];
        *reinterpret_cast<float4 *>(a.out + t * a.out_stride + static_cast<long long>(h) * a.Dv + col) =
            make_float4(fmaf(qk, u.x, al * y.x), fmaf(qk, u.y, al * y.y), fmaf(qk, u.z, al * y.z), fmaf(qk, u.w, al * y.w));
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        S[i].x = fmaf(kr[i], u.x, al * S[i].x);
        S[i].y = fmaf(kr[i], u.y, al * S[i].y);
        S[i].z = fmaf(kr[i], u.z, al * S[i].z);
        S[i].w = fmaf(kr[i], u.w, al * S[i].w);
      }
      buf ^= 1;
      if (a.state_each) leave(__ldg(a.state_each + t));
    }
  }
  if (a.state_out) leave(__ldg(a.state_out + b));
}

template <int DK>
cudaError_t tokens_launch(const DeltaArgs &a, int first_len, int sms, cudaStream_t s) {
  // 64 columns to a CTA of four warps, five of which share an SM, so that some read while others exchange or write (64 sequences of
  // 32 heads of 128 x 128, 268 MB: 49.4 us, 5.4 TB/s; with eight warps 60, with 128 columns and eight warps 57.7, six CTAs an SM
  // spill more than two registers: 62.7); 32 columns to one of eight where that does not give two CTAs an SM (one sequence: 3.8 us)
  const int jc = a.Dv % 64 == 0 && static_cast<long long>(a.B) * a.Hv * (a.Dv / 64) >= 2 * sms ? 64 : 32;
  const dim3 grid(static_cast<unsigned>(a.B) * a.Hv * (a.Dv / jc));
  if (jc == 64) return qg::launch_pdl(delta_tokens_kernel<DK, 64, 128>, grid, dim3(128), 0, s, a, first_len);
  return qg::launch_pdl(delta_tokens_kernel<DK, 32, 256>, grid, dim3(256), 0, s, a, first_len);
}

qg_status check(const qg_delta_args *g, DeltaArgs *a) {
  if (!g) return QG_EINVAL_PTR;
  if (g->n_seqs < 0 || g->n_seqs > 65535 || g->n_tokens < 0 || g->n_tokens > (1 << 24) || g->max_new < 0)
    return QG_EINVAL_SHAPE;
  if (!g->q_start && g->n_tokens != g->n_seqs) return QG_EINVAL_SHAPE;
  if (g->Hk < 1 || g->Hv < g->Hk || g->Hv > 1024 || g->Hv % g->Hk) return QG_EINVAL_SHAPE;
  if (g->Dk != 64 && g->Dk != 128) return QG_EUNSUPPORTED;
  if (g->Dv < 32 || g->Dv > 1024 || g->Dv % 32) return QG_EUNSUPPORTED;
  if ((g->head_order & ~1) || (g->l2norm & ~1) || g->n_slots < 0 || !(g->eps >= 0.f)) return QG_EINVAL_SHAPE;
  if (!g->a_scale != !g->a_bias) return QG_EINVAL_PTR;
  const int64_t lim = int64_t(1) << 38;
  const int64_t qk = int64_t(g->Hk) * g->Dk, vo = int64_t(g->Hv) * g->Dv;
  if (g->q_stride < qk || g->k_stride < qk || g->v_stride < vo || g->out_stride < vo || g->a_stride < g->Hv ||
      g->b_stride < g->Hv || g->q_stride > lim || g->k_stride > lim || g->v_stride > lim || g->out_stride > lim ||
      g->a_stride > lim || g->b_stride > lim)
    return QG_EINVAL_SHAPE;
  if (g->n_slots > 0 && (g->slot_stride < vo * g->Dk || g->slot_stride > lim)) return QG_EINVAL_SHAPE;
  auto odd = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
  if (!qg::aligned16(g->q) || !qg::aligned16(g->k) || !qg::aligned16(g->v) || !qg::aligned16(g->out) ||
      !qg::aligned16(g->states) || g->q_stride % 4 || g->k_stride % 4 || g->v_stride % 4 || g->out_stride % 4 ||
      (g->n_slots > 0 && g->slot_stride % 4) || odd(g->a) || odd(g->b) || odd(g->a_scale) || odd(g->a_bias) ||
      odd(g->q_start) || odd(g->state_in) || odd(g->state_out) || odd(g->state_each))
    return QG_EALIGN;
  *a = DeltaArgs{g->n_seqs, g->n_tokens, g->Hk, g->Hv, g->Dk, g->Dv, g->head_order, g->l2norm, g->n_slots, g->eps, g->scale,
                 g->q_start, g->state_in, g->state_out, g->state_each, g->q, g->k, g->v, g->a, g->b, g->a_scale, g->a_bias,
                 g->q_stride, g->k_stride, g->v_stride, g->a_stride, g->b_stride, g->slot_stride, g->out_stride,
                 g->states, g->out};
  return QG_OK;
}

// whether the call's longer sequences go in chunks: single tokens, calls said to be short, and those that keep each
// token's state go token after token
bool in_chunks(const qg_delta_args &g) {
  const int most = g.max_new > 0 ? std::min(g.max_new, g.n_tokens) : g.n_tokens;
  return g.q_start && !g.state_each && most >= qg::kDeltaFirstLen;
}

}  // namespace

namespace qg {

unsigned int read_status_delta(bool clear) {
  unsigned int v = 0;
  if (!g_launched) return v;
  if (cudaMemcpyFromSymbol(&v, g_qg_status_delta, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (clear) {
    const unsigned int z = 0;
    cudaMemcpyToSymbol(g_qg_status_delta, &z, sizeof(z));
  }
  return v;
}

}  // namespace qg

extern "C" {

size_t qg_delta_workspace_size(const qg_delta_args *args) {
  DeltaArgs a;
  if (check(args, &a) != QG_OK || !in_chunks(*args)) return 0;
  return qg::delta_chunk_workspace(a);
}

qg_status qg_delta_rule(const qg_delta_args *args, void *workspace, size_t workspace_bytes, qg_stream_t stream) {
  DeltaArgs a;
  const qg_status st = check(args, &a);
  if (st != QG_OK) return st;
  if (a.B == 0 || a.T == 0) return QG_OK;
  if (!a.q || !a.k || !a.v || !a.a || !a.b || !a.out) return QG_EINVAL_PTR;
  // slots that may be named need states
  if ((a.state_in || a.state_out || a.state_each) && (!a.states || a.n_slots < 1)) return QG_EINVAL_PTR;
  const size_t need = qg_delta_workspace_size(args);
  if (need && (!workspace || workspace_bytes < need)) return QG_EWORKSPACE;
  if (need && !qg::aligned16(workspace)) return QG_EALIGN;
  const qg::DeviceInfo &dev = qg::device_info();
  if (!dev.ok) return QG_ECUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  g_launched = true;
  const int first_len = in_chunks(*args) ? qg::kDeltaFirstLen : 0x7FFFFFFF;
  cudaError_t e = a.Dk == 64 ? tokens_launch<64>(a, first_len, dev.sms, s) : tokens_launch<128>(a, first_len, dev.sms, s);
  if (e == cudaSuccess && in_chunks(*args)) e = qg::delta_chunks(a, first_len, workspace, s);
  if (e != cudaSuccess) return QG_ECUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ECUDA;
}

}  // extern "C"
