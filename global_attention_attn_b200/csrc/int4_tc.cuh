// What the tcgen05 kernels over 4-bit keys share (decode_int4_tc.cu, weights_int4.cu): S^T = K Q^T
// of 128 keys (the rows of A, in tensor memory, a key's words unpacked by int4.cuh's masks) against
// N query rows of a KV head (columns of B, in shared memory), 6 sums per key and row.
#pragma once
#include "common.cuh"
#include "int4.cuh"
#include "ptx.cuh"

namespace mimo {

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t* r) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t a;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a) : "r"(addr) : "memory");
  return a;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t* r) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// Registers whose load a wait before has covered.
template <int C>
__device__ __forceinline__ void tied(uint32_t* d) {
#pragma unroll
  for (int i = 0; i < C; ++i) asm volatile("" : "+r"(d[i]));
}

// The query operand at `at`, by THREADS threads: four chunks of N rows of 64 elements (128-byte
// swizzle, CHUNK bytes): dims 0..63 rotated, 64..127, 128..191, and the second terms of dims 0..63,
// which enter as two fp16 terms (no 16-bit type holds them to the digits of an fp32 log-sum-exp);
// then a 32-byte row (32-byte swizzle) of the code offset for each of the 6 N columns of sums.
// q: draft 0's first head of the KV head; row n is head n % 2^g_log of draft n >> g_log, rows from
// `rows` on are 0, and so are those for which counts(n), asked after prepare(), is false.  prepare():
// called once the rows' loads are under way; after it `at` is free and cs[draft * 32 + i] holds
// (cos, sin).  Returns the largest magnitude that this thread stored.
// 8 threads a row: thread r dims 4 r .. 4 r + 3, their rotary partners, and 64 + 16 r .. 64 + 16 r + 15.
template <int N, int THREADS, int CHUNK, class F, class C>
__device__ __forceinline__ float int4_query_operand(const uint16_t* q, int rows, int g_log, uint32_t at, int tid,
                                                    const float2* cs, F&& prepare, C&& counts) {
  constexpr int kRows = THREADS / 8, kPasses = (N + kRows - 1) / kRows;
  const int r = tid & 7, G = 1 << g_log;
  uint2 ra[kPasses], rb[kPasses];
  uint4 rc[kPasses][2];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int n = i * kRows + (tid >> 3);
    ra[i] = rb[i] = make_uint2(0, 0);
    rc[i][0] = rc[i][1] = make_uint4(0, 0, 0, 0);
    if (n < rows) {
      const uint16_t* const src = q + ((n >> g_log) * kHq + (n & (G - 1))) * kDqk;
      ra[i] = __ldg(reinterpret_cast<const uint2*>(src + 4 * r));
      rb[i] = __ldg(reinterpret_cast<const uint2*>(src + 32 + 4 * r));
      rc[i][0] = __ldg(reinterpret_cast<const uint4*>(src + 64 + 16 * r));
      rc[i][1] = __ldg(reinterpret_cast<const uint4*>(src + 64 + 16 * r) + 1);
    }
  }
  prepare();
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int n = i * kRows + (tid >> 3);
    if (n >= N) break;  // (warp-uniform)
    if (!counts(n)) {
      ra[i] = rb[i] = make_uint2(0, 0);
      rc[i][0] = rc[i][1] = make_uint4(0, 0, 0, 0);
    }
    // 8 dims: fields come out of a word as (0, 4), (1, 5), (2, 6), (3, 7), the odd ones times 16 (* 4, / 4)
    auto put = [&](const float* v, int chunk, int unit, bool two) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = (e & 1) ? 0.25f : 4.f;
        hi[e] = pack2_f16_sat(v[e] * f, v[e + 4] * f, amax);
        if (two) {
          const float2 t = f32x2_of_f16x2(hi[e]);
          lo[e] = f16x2_of(v[e] * f - t.x, v[e + 4] * f - t.y);
        }
      }
      const uint32_t to = at + n * 128 + ((unit ^ (n & 7)) << 4);
      sts128(to + chunk * CHUNK, hi);
      if (two) sts128(to + 3 * CHUNK, lo);
    };
    float s0 = 0.f, s1 = 0.f, s2 = 0.f;
    {
      // rotated: even threads end up with 8 dims of the first half, odd ones with 8 of the second
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t wa = e < 2 ? ra[i].x : ra[i].y, wb = e < 2 ? rb[i].x : rb[i].y;
        const float xa = (e & 1) ? hi_bf16(wa) : lo_bf16(wa), xb = (e & 1) ? hi_bf16(wb) : lo_bf16(wb);
        const float2 t = cs[(n < rows ? n >> g_log : 0) * kHalf + 4 * r + e];
        const float a0 = xa * t.x - xb * t.y, b0 = xb * t.x + xa * t.y;
        s0 += a0;
        s1 += b0;
        const float other = __shfl_xor_sync(0xffffffffu, (r & 1) ? a0 : b0, 1);
        v[e] = (r & 1) ? other : a0;
        v[4 + e] = (r & 1) ? b0 : other;
      }
      put(v, 0, (r >> 1) + 4 * (r & 1), true);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w4[4] = {rc[i][h].x, rc[i][h].y, rc[i][h].z, rc[i][h].w};
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = lo_bf16(w4[e]);
        v[2 * e + 1] = hi_bf16(w4[e]);
        s2 += v[2 * e] + v[2 * e + 1];
      }
      put(v, 1 + (r >> 2), 2 * (r & 3) + h, false);
    }
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
      s0 += __shfl_xor_sync(0xffffffffu, s0, d);
      s1 += __shfl_xor_sync(0xffffffffu, s1, d);
      if (d == 1) s2 += __shfl_xor_sync(0xffffffffu, s2, d);
    }
    auto offset = [&](int j, float sum) {
      // -8 sum in the sums' unit 2^-22, over the constant 2^-14, as two terms
      const float o = sum * -0.03125f;
      const uint32_t hi = f16x2_of(o, 0.f), lo = f16x2_of(o - f32x2_of_f16x2(hi).x, 0.f);
      const int col = j * N + n;
      const uint32_t to = at + 4 * CHUNK + col * 32, swz = ((col >> 2) & 1) << 4;
      const uint32_t first[4] = {hi | (lo << 16), 0, 0, 0}, none[4] = {0, 0, 0, 0};
      sts128(to + swz, first);
      sts128(to + (swz ^ 16), none);
    };
    if (r == 0) offset(0, s0);
    if (r == 1) offset(1, s1);
    if ((r & 1) == 0) offset(2 + (r >> 1), s2);
  }
  return amax;
}

}  // namespace mimo
