// qg_delta.cuh -- the gated delta rule's call as its kernels see it.
#pragma once

#include "qg_common.cuh"
#include "qg_host.h"

namespace qg {

struct DeltaArgs {
  int B, T, Hk, Hv, Dk, Dv, tiled, l2norm, n_slots;
  float eps, scale;
  const int32_t *q_start, *state_in, *state_out, *state_each;
  const float *q, *k, *v, *a, *b, *a_scale, *a_bias;
  long long q_stride, k_stride, v_stride, a_stride, b_stride, slot_stride, out_stride;
  float *states, *out;
};

constexpr int kDeltaChunk = 32;  // tokens of a chunk
// sequences from this many tokens on go in chunks.  Where the two meet (32 heads of 128, token by token / in chunks): 8 sequences of
// 20 tokens 36 / 27 us and of 24 tokens 42 / 27, 32 of 20 tokens 116 / 96 and of 24 tokens 134 / 97 (of 16 tokens token by
// token 97).  One sequence alone would rather wait: of 20 tokens 13.5 / 16.8, of 24 tokens 15.3 / 16.8, of 28 tokens 17.8 / 17.0 and of
// 48 tokens 28 / 20
constexpr int kDeltaFirstLen = 20;

// the chunk kernels (qg_delta_chunk.cu), for sequences of first_len tokens and more
size_t delta_chunk_workspace(const DeltaArgs &a);
cudaError_t delta_chunks(const DeltaArgs &a, int first_len, void *ws, cudaStream_t s);

// first token row of sequence b (b = B: the end)
QG_DEVICE int delta_tok(const DeltaArgs &a, int b) {
  return a.q_start ? max(0, min(a.T, __ldg(a.q_start + b))) : min(b, a.T);
}
QG_DEVICE int delta_key_head(const DeltaArgs &a, int h) { return a.tiled ? h % a.Hk : h / (a.Hv / a.Hk); }

constexpr float kDeltaForgets = -110.f;  // a log decay of which nothing is left: e^g is 0 in f32

// log decay and step of value head h at token t.  Log decays below kDeltaForgets count as that: sums of them stay finite (fmaxf
// would turn NaN into it).
QG_DEVICE float2 delta_gates(const DeltaArgs &a, int t, int h) {
  float g = __ldg(a.a + t * a.a_stride + h), beta = __ldg(a.b + t * a.b_stride + h);
  if (a.a_scale) {
    const float x = g + __ldg(a.a_bias + h);
    g = __ldg(a.a_scale + h) * (x > 0.f ? x + log1pf(expf(-x)) : log1pf(expf(x)));
    beta = 1.f / (1.f + expf(-beta));
  }
  return make_float2(g < kDeltaForgets ? kDeltaForgets : g, beta);
}

}  // namespace qg
