// KV append: rotate the first 64 dims of each new key at its position and
// store key and value into the ring or paged cache.  Cache rows hold the key
// as dims 0..63 rotated in IEEE fp16 and dims 64..191 in bf16 (the input
// format), and the value in bf16; or, for an E4M3 cache, every element as one
// E4M3 byte scaled by 1 / (its KV head's dequantisation scale); or, for a 4-bit cache, codes
// with a scale per 32 dims.
//
// Cache layout follows the serving pages: window-sized KV for the sliding
// layers (gaudi-cookbook "MiMo-V2.6-Flash-RL", "Launch": window-sized KV for
// the 39 sliding layers) kept here as a 128-slot ring per sequence, and paged
// KV with block size 128 for the global layers (same page, "--block-size 128").
#include "common.cuh"
#include "int4.cuh"
#include "../../include/mimoattn.h"

namespace mimo {

namespace {
// The cache entry (slot of the whole pool, in units of one KV row set) of token t; -1 and a
// status bit if its sequence, position, slot or page lies outside the cache.
__device__ __forceinline__ long append_entry(const AppendParams& p, int t, int pos, int lane) {
  const int s = p.seq_idx[t], at = p.slots ? p.slots[t] : pos;
  bool ok = s >= 0 && s < p.num_seqs && pos >= 0 && at >= 0;
  long entry = -1;
  if (ok && p.cache_kind == MIMO_CACHE_RING) {
    entry = long(s) * p.ring_slots + (at % p.ring_slots);
  } else if (ok) {
    const int pi = at / kPage;
    const int page = pi < p.max_pages ? p.block_table[long(s) * p.max_pages + pi] : -1;
    ok = page >= 0 && page < p.num_pages;
    if (ok) entry = long(page) * kPage + (at % kPage);
  }
  if (!ok && lane == 0) atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
  return entry;
}
}  // namespace

// One warp per (token, kv head).  Lanes 0..3 rotate the chunk pairs (u, u+4) of
// dims 0..63; lanes 8..23 copy chunks 8..23 (dims 64..191); lanes 0..15 copy V.
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendParams p) {
  const int warp = int((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
  const int lane = threadIdx.x & 31;
  if (warp >= p.num_tokens * p.hkv) return;
  const int t = warp / p.hkv, g = warp % p.hkv;
  const int pos = p.pos[t];
  const long entry = append_entry(p, t, pos, lane);
  if (entry < 0) return;
  const uint4* ks = reinterpret_cast<const uint4*>(p.k_new + (long(t) * p.hkv + g) * kDqk);
  if (p.fp8) {
    // E4M3 rows: each element divided by its KV head's dequantisation scale, rounded to
    // nearest even and saturated (the rotation itself in fp32).  A scale that is not finite
    // and positive would store inf / NaN or sign-flipped codes: skip the row and report it.
    const float kdq = p.k_dequant[g], vdq = p.v_dequant[g];
    if (!(kdq > 0.f && kdq < INFINITY && vdq > 0.f && vdq < INFINITY)) {
      if (lane == 0) atomicOr(p.status, MIMO_STATUS_BAD_SCALE);
      return;
    }
    const float kq = 1.f / kdq, vq = 1.f / vdq;
    uint8_t* k8 = reinterpret_cast<uint8_t*>(p.k_cache) + (entry * p.hkv + g) * kDqk;
    uint8_t* v8 = reinterpret_cast<uint8_t*>(p.v_cache) + (entry * p.hkv + g) * kDv;
    auto pack8 = [](const float* x, float sc) {
      return make_uint2(uint32_t(e4m3x2_from_f32(x[0] * sc, x[1] * sc)) | (uint32_t(e4m3x2_from_f32(x[2] * sc, x[3] * sc)) << 16),
                        uint32_t(e4m3x2_from_f32(x[4] * sc, x[5] * sc)) | (uint32_t(e4m3x2_from_f32(x[6] * sc, x[7] * sc)) << 16));
    };
    auto widen8 = [](const uint4& c, float* x) {
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = lo_bf16(w[i]);
        x[2 * i + 1] = hi_bf16(w[i]);
      }
    };
    if (lane < 4) {
      // dims 8u..8u+7 pair with 8u+32..8u+39 (frequency index 8u + i)
      float x[8], y[8], xr[8], yr[8];
      widen8(__ldg(ks + lane), x);
      widen8(__ldg(ks + lane + 4), y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float c, sn;
        rope_cos_sin(pos, p.rope.inv_freq[8 * lane + i], &c, &sn);
        xr[i] = x[i] * c - y[i] * sn;
        yr[i] = y[i] * c + x[i] * sn;
      }
      *reinterpret_cast<uint2*>(k8 + 8 * lane) = pack8(xr, kq);
      *reinterpret_cast<uint2*>(k8 + 32 + 8 * lane) = pack8(yr, kq);
    } else if (lane >= 8 && lane < 24) {
      float x[8];
      widen8(__ldg(ks + lane), x);
      *reinterpret_cast<uint2*>(k8 + 8 * lane) = pack8(x, kq);
    }
    if (lane < 16) {
      float x[8];
      widen8(__ldg(reinterpret_cast<const uint4*>(p.v_new + (long(t) * p.hkv + g) * kDv) + lane), x);
      *reinterpret_cast<uint2*>(v8 + 8 * lane) = pack8(x, vq);
    }
    return;
  }
  uint4* kd = reinterpret_cast<uint4*>(p.k_cache + (entry * p.hkv + g) * kDqk);
  if (lane < 4) {
    uint4 lo = __ldg(ks + lane), hi = __ldg(ks + lane + 4);
    float amax = 0.f;
    rope_chunk_pair(lo, hi, lane, pos, p.rope, amax);
    if (amax > kF16Max) atomicOr(p.status, MIMO_STATUS_RANGE);
    kd[lane] = lo;
    kd[lane + 4] = hi;
  } else if (lane >= 8 && lane < 24) {
    kd[lane] = __ldg(ks + lane);
  }
  if (lane < 16) {
    const uint4* vs = reinterpret_cast<const uint4*>(p.v_new + (long(t) * p.hkv + g) * kDv);
    uint4* vd = reinterpret_cast<uint4*>(p.v_cache + (entry * p.hkv + g) * kDv);
    vd[lane] = __ldg(vs + lane);
  }
}

// 4-bit rows (int4.cuh): one warp per token and HPW of its KV heads, 640 bytes read and 180
// written per head (6700 tokens of 4 heads: 14.1 us, 1.6 TB/s; bound by the quantising, 30 thread
// instructions an element, half of the ALU pipe and 59 % of the issue slots).  A lane takes 8 dims at a time, so a group of 32 dims is four
// neighbouring lanes, its largest magnitude two shuffles, and a lane's codes one word; the words of
// four heads lie side by side (a head at a time left a quarter of the lanes idle in its key and
// half in its value: 21 us).  Per group: scale = fp16(amax / 7), code = rint(x /
// scale) + 8; 7 of amax keeps zero exact and both signs alike.  The rounding is the addition of
// 1.5 * 2^23 + 8, whose low four bits are the code.  One bf16 element in 600 lies exactly between
// two codes, where x * (1 / scale) may end on the wrong side: the remainder x - n * scale, which
// is exact, says so (a division per element instead took twice the time); only words with a remainder
// near half a step look at each of theirs.
// All heads of a token turn by the same angles: with many tokens a warp takes four of them and
// computes the angles once.
// The rotated dims are fp32 sums, off by up to kSlip times the largest magnitude of their two groups.
// Where that could move a scale (its fp16 rounding) or a code (its border), for one (token, four heads) in
// some fifty, the warp does the word again with the rotation in 64 bits or two fp32 terms: codes and scales
// are those of the exact one (of 5.4 M codes some tens were not; 0.3 us of the call above, 0.8 us of one with
// 48 tokens where it happens).
constexpr float kRound = 12582920.f;
// x' = x c - y s: cos and sin are off by 1.25 x 2^-23 (sincosf by two units in the last place), the product
// and the sum round by 2^-24 of themselves, and |x| + |y| is at most twice the larger of |x'|, |y'|:
// 2 x 2.25 x 2^-23, of which this leaves a tenth.
constexpr float kSlip = 0x1.4p-21f;

// A word of a key (8 dims; a group of 32 is four neighbouring lanes) quantised from the exact rotation, by
// the whole warp.  `turn`: this lane's dims are rotated ones; the partners' are four lanes away.  `angle`: that
// of frequency `lane`, in [-pi, pi].  was: the word and the scale's bits, which stay in groups with an element
// that is not finite.
// (Two fp32 terms a value: with all of it in fp64 it took 1.4 us.)
__device__ __noinline__ uint2 quantise_exact(uint4 raw, bool turn, double angle, float cap, int lane, uint2 was) {
  // cos and sin by their Taylor series on [-pi/4, pi/4] (to 2^-41; fp64 steps take some 60 cycles each, so
  // the sums are short chains)
  const float turns = rintf(float(angle) * 0.636619772f);
  const double r = fma(double(-turns), 1.5707963267948966, angle), q = r * r, q2 = q * q;
  const double s5 = fma(q, 1.0 / 6227020800, -1.0 / 39916800), s3 = fma(q, 1.0 / 362880, -1.0 / 5040), s1 = fma(q, 1.0 / 120, -1.0 / 6);
  const double c5 = fma(q, 1.0 / 479001600, -1.0 / 3628800), c3 = fma(q, 1.0 / 40320, -1.0 / 720), c1 = fma(q, 1.0 / 24, -0.5);
  const double s = fma(r * q, fma(q2, fma(q2, s5, s3), s1), r), c = fma(q, fma(q2, fma(q2, c5, c3), c1), 1.0);
  float sh = float(s), ch = float(c), sl = float(s - double(sh)), cl = float(c - double(ch));
  const int quarter = int(turns) & 3;
  if (quarter & 1) {
    const float h = sh, l = sl;
    sh = ch, sl = cl, ch = h, cl = l;
  }
  if (quarter >= 2) sh = -sh, sl = -sl;
  if (quarter == 1 || quarter == 2) ch = -ch, cl = -cl;
  float x[8], xl[8], amax = 0.f;  // values and what they leave over
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 2 ? raw.x : (i < 4 ? raw.y : (i < 6 ? raw.z : raw.w));
    const float u = (i & 1) ? hi_bf16(w) : lo_bf16(w), v0 = __shfl_xor_sync(0xffffffffu, u, 4), v = (lane & 4) ? v0 : -v0;
    const int from = 8 * (lane & 3) + i;
    const float cih = __shfl_sync(0xffffffffu, ch, from), cil = __shfl_sync(0xffffffffu, cl, from);
    const float sih = __shfl_sync(0xffffffffu, sh, from), sil = __shfl_sync(0xffffffffu, sl, from);
    const float a = __fmul_rn(u, cih), b = __fmul_rn(v, sih), sum = __fadd_rn(a, b), part = __fsub_rn(sum, a);
    const float rest = __fadd_rn(__fsub_rn(a, __fsub_rn(sum, part)), __fsub_rn(b, part)) + (fmaf(u, cih, -a) + fmaf(v, sih, -b)) +
                       fmaf(u, cil, v * sil);
    x[i] = turn ? __fadd_rn(sum, rest) : u;
    xl[i] = turn ? __fsub_rn(rest, __fsub_rn(x[i], sum)) : 0.f;
    amax = fmaxf(amax, fabsf(x[i]));
    bad = bad || !(fabsf(x[i]) < INFINITY);
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  float more = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) more = fabsf(x[i]) == amax ? fmaxf(more, x[i] > 0.f ? xl[i] : -xl[i]) : more;
  more = fmaxf(more, __shfl_xor_sync(0xffffffffu, more, 1));
  more = fmaxf(more, __shfl_xor_sync(0xffffffffu, more, 2));
  const bool keep = (__ballot_sync(0xffffffffu, bad) >> (lane & 28)) & 15u;
  const float want = float((double(amax) + double(more)) * (1.0 / 7.0));
  const __half scale_h = __float2half_rn(fminf(want, cap));
  const float scale = __half2float(scale_h), half = 0.5f * scale, inv = scale > 0.f ? __fdividef(1.f, scale) : 0.f;
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float n = rintf(fminf(fmaxf(x[i] * inv, -7.f), 7.f));
    const float d = fmaf(-n, scale, x[i]), over = (fabsf(d) - half) + (d > 0.f ? xl[i] : -xl[i]);
    if (inv > 0.f && (over > 0.f || (over == 0.f && (int(n) & 1)))) n += d > 0.f ? 1.f : -1.f;
    word |= uint32_t(int(fminf(fmaxf(n, -7.f), 7.f)) + 8) << (4 * i);
  }
  return keep ? was : make_uint2(word, __float_as_uint(scale));
}

template <int HPW>
__global__ void __launch_bounds__(256, 3) kv_append_int4_kernel(const AppendParams p) {
  const int warp = int((blockIdx.x * blockDim.x + threadIdx.x) >> 5);
  const int lane = threadIdx.x & 31;
  const int parts = p.hkv / HPW;
  if (warp >= p.num_tokens * parts) return;
  const int t = warp / parts, g0 = warp % parts * HPW;
  const int pos = p.pos[t];
  const long entry = append_entry(p, t, pos, lane);
  if (entry < 0) return;
  const int slots = p.cache_kind == MIMO_CACHE_RING ? p.ring_slots : kPage;
  const int slot = int(entry % slots);
  auto widen = [](const uint4& c, float* x) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = lo_bf16(w[i]);
      x[2 * i + 1] = hi_bf16(w[i]);
    }
  };
  bool range = false;
  // 8 dims of a group -> their word of codes; every lane of the warp takes part.  turned: the dims are
  // rotated, and `near` tells whether what that is off by could matter.
  auto quantise = [&](float* x, float cap, float& scale, bool turned, bool& near) -> uint32_t {
    float amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      amax = fmaxf(amax, fabsf(x[i]));
      bad = bad || !(fabsf(x[i]) < INFINITY);  // (a NaN does not show in amax)
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const float want = float(double(amax) * (1.0 / 7.0));  // (a float divided by 7, rounded once but for one case in 2^28)
    scale = __half2float(__float2half_rn(fminf(want, cap)));
    range = range || bad || want > cap;
    const float slip = turned ? kSlip * fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 4)) : 0.f;
    if (turned) {
      // (a seventh of it, and a step of `want` itself)
      const float e = 0.15f * slip + 0x1p-23f * want;
      near = __half_as_ushort(__float2half_rn(want - e)) != __half_as_ushort(__float2half_rn(want + e));
    }
    if (bad || want > 1.05f * scale) {  // (a scale cut to its range, or a subnormal one: quotients beyond 7.5)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -7.f * scale), 7.f * scale);
    }
    const float inv = scale > 0.f ? __fdividef(1.f, scale) : 0.f, half = 0.5f * scale;
    uint32_t w = 0;
    float dmax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sum = x[i] * inv + kRound;
      dmax = fmaxf(dmax, fabsf(fmaf(kRound - sum, scale, x[i])));
      w |= (__float_as_uint(sum) & 15u) << (4 * i);
    }
    if (dmax >= 0.99999f * half) {
      w = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float sum = x[i] * inv + kRound, d = fmaf(kRound - sum, scale, x[i]);
        const bool off = fabsf(d) > half || (fabsf(d) == half && (__float_as_uint(sum) & 1u));
        const uint32_t code = __float_as_uint(sum) + (off ? (d > 0.f ? 1u : ~0u) : 0u);
        w |= (code & 15u) << (4 * i);
      }
    }
    if (turned) near = near || (scale > 0.f && dmax + slip >= 0.999999f * half);  // (no scale, no codes)
    return w;
  };
  // the heads' words of 8 dims side by side, 32 at a time: word m is word m % 24 of key m / 24, or
  // m % 16 of value m / 16
  constexpr int kK = (24 * HPW + 31) / 32, kV = (16 * HPW + 31) / 32;
  const uint16_t* const k_row = p.k_new + (long(t) * p.hkv + g0) * kDqk;
  const uint16_t* const v_row = p.v_new + (long(t) * p.hkv + g0) * kDv;
  uint4 kr[kK], vr[kV];
#pragma unroll
  for (int i = 0; i < kK; ++i) {
    const int m = 32 * i + lane;
    kr[i] = m < 24 * HPW ? __ldg(reinterpret_cast<const uint4*>(k_row) + m) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int m = 32 * i + lane;
    vr[i] = m < 16 * HPW ? __ldg(reinterpret_cast<const uint4*>(v_row) + m) : make_uint4(0, 0, 0, 0);
  }
  // words 0..3 of a key hold dims 8 w + i, words 4..7 their partners + 32: x' = x c -+ y s.  24 and 32
  // are multiples of 8, so partners are four lanes apart whatever the head
  float c, sn, ci[8], si[8];
  const double angle = rope_cos_sin_fine(pos, p.rope.inv_freq[lane], &c, &sn);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    ci[i] = __shfl_sync(0xffffffffu, c, 8 * (lane & 3) + i);
    si[i] = __shfl_sync(0xffffffffu, sn, 8 * (lane & 3) + i);
    if (!(lane & 4)) si[i] = -si[i];
  }
  const long block0 = entry / slots * p.hkv + g0;
#pragma unroll
  for (int i = 0; i < kK; ++i) {
    const int m = 32 * i + lane, h = m / 24, w = m - 24 * h;
    float x[8], scale;
    widen(kr[i], x);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = __shfl_xor_sync(0xffffffffu, x[e], 4);
      if (w < 8) x[e] = x[e] * ci[e] + y * si[e];
    }
    bool near = false;
    uint32_t word = quantise(x, kF16Max, scale, true, near);
    near = near && w < 8 && m < 24 * HPW;
    if (__any_sync(0xffffffffu, near)) {
      const uint2 e = quantise_exact(kr[i], w < 8, angle, kF16Max, lane, make_uint2(word, __float_as_uint(scale)));
      word = e.x;
      scale = __uint_as_float(e.y);
    }
    if (m < 24 * HPW) {
      uint8_t* const kb = reinterpret_cast<uint8_t*>(p.k_cache) + (block0 + h) * (long(slots) * kI4KSlot);
      reinterpret_cast<uint32_t*>(kb + long(slot) * kI4KCodes)[(w & 3) * 6 + (w >> 2)] = word;
      if ((w & 3) == 0)
        reinterpret_cast<__half*>(kb + long(slots) * kI4KCodes)[slot * kI4KGroups + (w >> 2)] = __float2half_rn(scale);
    }
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int m = 32 * i + lane, h = m / 16, w = m % 16;
    float x[8], scale;
    widen(vr[i], x);
    bool near;
    const uint32_t word = quantise(x, kI4VScaleMax, scale, false, near);
    if (m < 16 * HPW) {
      uint8_t* const vb = reinterpret_cast<uint8_t*>(p.v_cache) + (block0 + h) * (long(slots) * kI4VSlot);
      reinterpret_cast<uint32_t*>(vb + long(slot) * kI4VCodes)[w] = word;
      if ((w & 3) == 0)
        reinterpret_cast<__half*>(vb + long(slots) * kI4VCodes)[slot * kI4VGroups + (w >> 2)] = __float2half_rn(scale);
    }
  }
  if (range) atomicOr(p.status, MIMO_STATUS_RANGE);
}

// (token, head) pairs up to which each has a warp of its own: a few to every scheduler.
constexpr long kAppendWarps = 2048;

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t s) {
  const long warps = long(p.num_tokens) * p.hkv;
  if (warps == 0) return cudaSuccess;
  const int block = 256;
  const long grid = (warps * 32 + block - 1) / block;
  if (!p.int4) {
    kv_append_kernel<<<unsigned(grid), block, 0, s>>>(p);
  } else if (warps <= kAppendWarps) {
    kv_append_int4_kernel<1><<<unsigned(grid), block, 0, s>>>(p);  // few tokens: a warp per head is sooner done
  } else {
    const unsigned g4 = unsigned((warps / 4 * 32 + block - 1) / block);
    kv_append_int4_kernel<4><<<g4, block, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace mimo
