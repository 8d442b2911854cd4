// qg_mma.cuh -- warp-level pieces of the attention kernels: 16-bit packing, powers of two,
// cp.async groups, ldmatrix and the m16n8k16 product.
#pragma once

#include "qg_common.cuh"

// two f32 rounded to the 16-bit type, `lo` in the low half
template <bool BF16>
QG_DEVICE uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if constexpr (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool BF16>
QG_DEVICE float lo16(uint32_t v) {
  return BF16 ? __uint_as_float(v << 16) : h2f(v);
}
template <bool BF16>
QG_DEVICE float hi16(uint32_t v) {
  return BF16 ? __uint_as_float(v & 0xFFFF0000u) : h2f(v >> 16);
}

// whether the low 16-bit value is infinite or NaN: its exponent is all ones
template <bool BF16>
QG_DEVICE bool nonfinite16(uint32_t v) {
  constexpr uint32_t E = BF16 ? 0x7F80u : 0x7C00u;
  return (v & E) == E;
}
// not zero if there are such values among eight: adding one to an exponent of ones carries into the
// sign's place
template <bool BF16>
QG_DEVICE uint32_t any_nonfinite(uint4 v) {
  constexpr uint32_t E = BF16 ? 0x7F807F80u : 0x7C007C00u, ONE = BF16 ? 0x00800080u : 0x04000400u;
  return (((v.x & E) + ONE) | ((v.y & E) + ONE) | ((v.z & E) + ONE) | ((v.w & E) + ONE)) & 0x80008000u;
}
// eight values with zeros in the places of such
template <bool BF16>
QG_DEVICE uint4 make_finite(uint4 v) {
  auto fin = [](uint32_t x) {
    return (nonfinite16<BF16>(x) ? 0u : x & 0xFFFFu) | (nonfinite16<BF16>(x >> 16) ? 0u : x & 0xFFFF0000u);
  };
  return make_uint4(fin(v.x), fin(v.y), fin(v.z), fin(v.w));
}

// 2^x on the special function unit (relative error about 2^-22; 2^-inf = 0)
QG_DEVICE float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 16-byte asynchronous copy of which the first n (0 or 16) bytes are read, the rest zeros
QG_DEVICE void cp_async16_zfill(uint32_t dst_smem, const void *src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst_smem), "l"(src), "r"(n) : "memory");
}
QG_DEVICE void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
QG_DEVICE void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

QG_DEVICE void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
QG_DEVICE void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool BF16>
QG_DEVICE void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
