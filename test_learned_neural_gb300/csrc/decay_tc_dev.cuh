// Device helpers of the tensor-core decay attention: tensor maps over either
// layout, TMA, MMAs with A in TMEM, splits into bf16 terms.
#pragma once
#include "decay_common.cuh"
#include "decay_tc.cuh"
#include "tc2.cuh"

namespace decay {

constexpr int C = 128, SL = 64;               // tokens per chunk, columns per slice
constexpr int TILE = C * 128;                 // 128 rows of 64 bf16 values

// 4-D map over [row][head][token][d] in either layout: boxes of 64 bf16 or 32
// fp32 values x 128 tokens, 128-byte swizzled
inline bool map_4d(CUtensorMap* map, const void* base, bool is_bf16, int d, int T, int heads, int B, size_t st, size_t sh,
            size_t sb) {
  auto fn = tc::tensor_map_encoder();
  if (!fn) return false;
  const size_t es = is_bf16 ? 2 : 4;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)heads, (cuuint64_t)B};
  const cuuint64_t strides[3] = {st * es, sh * es, sb * es};
  const cuuint32_t box[4] = {is_bf16 ? 64u : 32u, (cuuint32_t)C, 1, 1}, estr[4] = {1, 1, 1, 1};
  return fn(map, is_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap* map, int c, int t, int h, int b, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(t), "r"(h), "r"(b), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void store_4d(const CUtensorMap* map, int c, int t, int h, int b, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c), "r"(t), "r"(h), "r"(b), "r"(src)
               : "memory");
}
// D (+)= A B^T with A (16-bit, two values of K per column) in TMEM
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 packed columns of this warp's lanes
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t* w) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr)
               : "memory");
}
// byte offset of 16-byte chunk j of row r in a 128-byte swizzled tile
__device__ __forceinline__ uint32_t swz(int r, int j) { return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)); }

// Packed pairs of fp32 values: one instruction for two.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Two fp32 values as N packed bf16 pairs whose sums are the values to 8 N
// bits: each term but the last is the remainder's leading bits cut off, so the
// subtraction is exact; the last is rounded.
template <int N>
__device__ __forceinline__ void split_pair(uint64_t v, uint32_t* w) {
#pragma unroll
  for (int i = 0; i + 1 < N; ++i) {
    float a, b;
    unpair(v, a, b);
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    w[i] = __byte_perm(ua, ub, 0x7632);
    v = fma_pair(pair(__uint_as_float(ua & 0xffff0000u), __uint_as_float(ub & 0xffff0000u)), pair(-1.f, -1.f), v);
  }
  float a, b;
  unpair(v, a, b);
  w[N - 1] = layer::pack_bf16(a, b);
}
template <int N>
__device__ __forceinline__ void split2(float a, float b, uint32_t* w) {
  split_pair<N>(pair(a, b), w);
}
// two packed bf16 values as an fp32 pair
__device__ __forceinline__ uint64_t widen(uint32_t x) {
  return pair(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

}  // namespace decay
