// The 4-bit cache format and the pieces the kernels that read it share.
//
// A cache element is (code - 8) * scale: codes are 4 bits, one fp16 scale per group of 32
// dims of a slot (6 groups of a key, 4 of a value).  A block (one KV head of a page, or of a
// sequence's ring) holds the codes of all its slots, then their scales: keys 96 + 12 bytes
// per slot, values 64 + 8.  Byte i of a row of codes holds dims 2i (low bits) and 2i + 1; a
// key row's 32-bit words are stored as word w at (w % 4) * 6 + w / 4, so that the six words a
// lane of an mma fragment needs (word 4 j + lane % 4 of each group j) are 24 consecutive
// bytes, and the warp's 8-byte shared loads of 8 key rows meet no bank twice.
//
// Fragments without arithmetic: bits 0..3 of a 16-bit half, alone, are the fp16 subnormal
// code * 2^-24, bits 4..7 are code * 2^-20.  One shift and four ANDs turn a word into four
// fp16x2 operands; the powers of two are moved into the query (low field * 4, high field / 4)
// or the final scale, and the offset 8 into one more product (of the scales and the query's
// group sums for keys, of the probabilities and a constant for values).
#pragma once
#include <cstdint>

#include "common.cuh"

namespace mimo {

constexpr int kI4Group = 32;
constexpr int kI4KCodes = kDqk / 2, kI4VCodes = kDv / 2;                // bytes of codes per slot
constexpr int kI4KGroups = kDqk / kI4Group, kI4VGroups = kDv / kI4Group;
constexpr int kI4KSlot = kI4KCodes + 2 * kI4KGroups;                    // 108
constexpr int kI4VSlot = kI4VCodes + 2 * kI4VGroups;                    // 72
// Largest value scale an append stores: the decode's probability * scale products (fp16,
// probabilities biased by 2^6) stay finite.
constexpr float kI4VScaleMax = 1023.f;
constexpr uint32_t kI4Lo = 0x000F000Fu, kI4Hi = 0x00F000F0u;

// D = A B + C on m16n8k16, fp16 operands, fp32 accumulation.
__device__ __forceinline__ void mma_f16_c(float* d, const uint32_t* a, uint32_t b0, uint32_t b1, const float* c) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ float2 f32x2_of_f16x2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Query rows of an mma block as fragments for 4-bit keys.  x0 / x1: the 8 dims of group j
// that this lane covers (dims 32 j + 8 (lane % 4) + i) of rows lane / 4 and lane / 4 + 8,
// rotated, in fp32.  The k order within a step is the order the fields come out of a word:
// step 2 j takes dims (0, 4 | 1, 5) of the eight, step 2 j + 1 dims (2, 6 | 3, 7).
// rest: the same of what fp16 leaves over (the rotated dims' second term).
__device__ __forceinline__ void int4_query_group(const float* x0, const float* x1, uint32_t (*qa)[4],
                                                 uint32_t (*rest)[4], float& amax) {
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float* x = r ? x1 : x0;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const float u = (f & 1) ? 0.25f : 4.f;
      const uint32_t h = pack2_f16_sat(x[f] * u, x[f + 4] * u, amax);
      const float2 v = f32x2_of_f16x2(h);
      qa[f >> 1][(f & 1) * 2 + r] = h;
      rest[f >> 1][(f & 1) * 2 + r] = pack2_f16(x[f] * u - v.x, x[f + 4] * u - v.y);
    }
  }
}

constexpr float kI4KeyUnit = 0x1p22f;  // 2^24 / 4: what a key product has to be multiplied with

// The offset -8 of every code adds, per key, the sum over groups of scale * (-8 * group sum of
// the query): one more product, whose scales are the stored fp16 pairs and whose other side
// is -8 * sum / 128 (no query in range overflows) as two fp16 terms: groups 0..5 are k 0..5,
// the remainders k 8..13, and both halves meet the same scales.
constexpr float kI4OffsetUnit = 0x1p-15f;  // 128 * 2^-22: from that product to the key products' unit
__device__ __forceinline__ void int4_offset_group(uint32_t* a, int j, int q4, float s0, float s1) {
  if ((j >> 1) != q4) return;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float c = (r ? s1 : s0) * -0.0625f;
    const __half hi = __float2half_rn(c), lo = __float2half_rn(c - __half2float(hi));
    const int sh = (j & 1) * 16;
    a[r] |= uint32_t(__half_as_ushort(hi)) << sh;
    a[2 + r] |= uint32_t(__half_as_ushort(lo)) << sh;
  }
}

}  // namespace mimo
