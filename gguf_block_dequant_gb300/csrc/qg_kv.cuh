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

// the i < n with start[i] <= x < start[i + 1] (start rising, n + 1 entries), -1 when there is none.
// Each round loads seven places at once: the search costs load latencies, one per factor of
// eight.
QG_DEVICE int kv_search(const int32_t *start, int n, int x) {
  int lo = -1, hi = n + 1;  // start[lo] <= x < start[hi], as far as is known
  while (hi - lo > 1) {
    const int step = (hi - lo + 7) / 8;
    int v[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      const int at = lo + (i + 1) * step;
      v[i] = at < hi ? __ldg(start + at) : 0x7FFFFFFF;
    }
    int below = 0;  // places up to the first one above x
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (below == i && v[i] <= x && lo + (i + 1) * step < hi) below = i + 1;
    const int base = lo;
    lo = base + below * step;
    hi = min(hi, base + (below + 1) * step);
  }
  return lo < n ? lo : -1;
}
// sequence of token t, -1 when no sequence holds it
QG_DEVICE int kv_seq_of(const KvBatch &a, int t) {
  if (!a.q_start) return t < a.B ? t : -1;
  return kv_search(a.q_start, a.B, t);
}
// group of sequence b, -1 when it has none
QG_DEVICE int kv_group_of(const KvBatch &a, int b) { return a.G ? kv_search(a.group_start, a.G, b) : -1; }

// host checks shared by the calls; on QG_OK *pool and *kb are filled.  prefix: the call reads
// the prefix page lists.  tokens: the call has token rows (q_start, n_tokens).
qg_status kv_check_cache(const qg_kv_cache *c, KvPool *pool);
qg_status kv_check_batch(const qg_kv_batch *b, bool tokens, bool prefix, KvBatch *kb);

}  // namespace qg
