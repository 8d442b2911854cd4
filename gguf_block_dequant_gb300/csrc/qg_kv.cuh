// qg_kv.cuh -- the paged cache and its batch as the kernels see them, with the look-ups every
// kernel shares: a sequence's token range and length, the sequence of a token, the group of a
// sequence.  Every index read from device memory is clamped before it is used.
#pragma once

#include "qg_common.cuh"
#include "qg_host.h"

namespace qg {

struct KvPool {
  uint16_t *k, *v;
  long long page_stride, token_stride, head_stride;  // elements
  int n_pages, page_shift, Hkv, D;
};

struct KvBatch {
  int B, T, G, max_pages, max_prefix_pages;
  const int32_t *q_start, *kv_len, *group_start, *prefix_len, *prefix_pages;
  int32_t *pages;
};

QG_DEVICE int kv_clamp(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// first token row of sequence b (b = B: the end)
QG_DEVICE int kv_tok(const KvBatch &a, int b) {
  return a.q_start ? kv_clamp(__ldg(a.q_start + b), 0, a.T) : min(b, a.T);
}

// the page lists' capacity in tokens (at most 2^30 - 1, so that sums of two stay in 32 bits)
QG_DEVICE int kv_cap(int pages, int shift) {
  const long long c = static_cast<long long>(pages) << shift;
  return c > 0x3FFFFFFFLL ? 0x3FFFFFFF : static_cast<int>(c);
}
QG_DEVICE int kv_own_len(const KvBatch &a, int shift, int b) {
  return kv_clamp(__ldg(a.kv_len + b), 0, kv_cap(a.max_pages, shift));
}

// the largest i in [lo, hi) with f(i) <= x (f rising), or lo - 1 when there is none
template <typename F>
QG_DEVICE int kv_search(int lo, int hi, int x, F f) {
  int a = lo - 1, b = hi;
  while (b - a > 1) {
    const int m = a + (b - a) / 2;
    if (f(m) <= x) a = m;
    else b = m;
  }
  return a;
}
// sequence of token t, -1 when no sequence holds it
QG_DEVICE int kv_seq_of(const KvBatch &a, int t) {
  if (!a.q_start) return t < a.B ? t : -1;
  const int b = kv_search(0, a.B, t, [&](int i) { return __ldg(a.q_start + i); });
  return b >= 0 && t < __ldg(a.q_start + b + 1) ? b : -1;
}
// group of sequence b, -1 when it has none
QG_DEVICE int kv_group_of(const KvBatch &a, int b) {
  if (a.G == 0) return -1;
  const int g = kv_search(0, a.G, b, [&](int i) { return __ldg(a.group_start + i); });
  return g >= 0 && b < __ldg(a.group_start + g + 1) ? g : -1;
}

// host checks shared by the calls; on QG_OK *pool and *kb are filled.  prefix: the call reads
// the prefix page lists.  tokens: the call has token rows (q_start, n_tokens).
qg_status kv_check_cache(const qg_kv_cache *c, KvPool *pool);
qg_status kv_check_batch(const qg_kv_batch *b, bool tokens, bool prefix, KvBatch *kb);

}  // namespace qg
