// Attention weights per cached slot: scores[s][g][t] += sum over the draft rows i and the query
// heads h of KV head g of exp(z_iht - lse_ih), the probabilities that the attention call whose
// log-sum-exp is given assigned to slot t.  Their running sum over steps is what eviction by
// accumulated weight ranks slots by.
//
// (4-bit keys: weights_int4.cu.)
//
// The keys are read once (384 or 192 bytes per slot and KV head) and 8 bytes of scores:
// no second pass for the normalisation (it is given), no exchange between tiles, no atomics (a
// score belongs to one lane of one tile).  S^T = K Q^T on mma.sync m16n8k16: 16 keys are the
// rows, the heads of a KV group the columns (two blocks of 8 on 4-head layers, one on 8-head
// layers: no padding), so a key's sum over heads is four values of a thread and two shuffles.
// A probability is compared in fp32, so the logits are kept to fp32's digits: the rotated query
// dims, which no 16-bit type holds, enter as two fp16 terms (4 of 16 k-steps).
//
// One CTA takes a contiguous piece of the line of 32-key tiles of all (sequence, KV head) units;
// its warps take the piece's tiles in turn, each with its own two stages of TMA copies, and share
// the unit's query fragments (shared memory, up to 8 drafts).
//
// 32 sequences of 1000..16384 slots, 4 heads, bf16, one token: 91 us, 4.3 TB/s, 0.66 of a copy's rate;
// 8 sequences of 4099..65536: one token 89 us (E4M3 63), 4 drafts 152 (133).  With one token bound by
// latency: two warps a scheduler, all that the stages leave room for, issue in 17 % of the cycles
// (tensor pipe 21 %) and wait for scores, tiles and each other's query fragments.  With drafts each
// one loads the key fragments again from shared memory and multiplies on its own.
#include "common.cuh"
#include "ptx.cuh"
#include "tiles.cuh"
#include "../../include/mimoattn.h"

namespace mimo {

namespace {

constexpr int kTile = 32, kMaxWarps = 8, kStages = 2;
constexpr int kMaxSmem = 232448;  // of a CTA
constexpr float kLog2e = 1.4426950408889634f;

template <int FMT>
struct Fmt {  // bytes of a stage: 32 key rows
  static constexpr int kRow = FMT == MIMO_DTYPE_BF16 ? 384 : 192;
  static constexpr int kStage = (kTile * kRow + 1023) / 1024 * 1024;
};
// query fragments of a draft: 12 steps, and 4 of the rotated dims' second terms
constexpr int kSteps = 16;

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16_acc(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_acc(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float2 f32x2_of(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }

// A fragments of 16 keys for step kk.
template <int FMT>
__device__ __forceinline__ void key_frag(uint32_t kb, int k0, int kk, int lane, uint32_t* a) {
  const int row = k0 + (lane & 7) + ((lane >> 3) & 1) * 8;
  if constexpr (FMT == MIMO_DTYPE_BF16) {
    ldsm_x4(kb + (kk >> 2) * (kTile * 128) + row * 128 + ((((kk & 3) * 2 + (lane >> 4)) ^ (row & 7)) << 4), a);
  } else {
    // two steps at once: bytes in pairs, 4 consecutive dims of a key per lane
    uint32_t m[4];
    ldsm_x4(kb + (kk >> 2) * (kTile * 64) + row * 64 + (((2 * ((kk >> 1) & 1) + (lane >> 4)) ^ ((row >> 1) & 3)) << 4), m);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      a[4 * i] = f16x2_from_e4m3x2(uint16_t(m[2 * i]));
      a[4 * i + 1] = f16x2_from_e4m3x2(uint16_t(m[2 * i + 1]));
      a[4 * i + 2] = f16x2_from_e4m3x2(uint16_t(m[2 * i] >> 16));
      a[4 * i + 3] = f16x2_from_e4m3x2(uint16_t(m[2 * i + 1] >> 16));
    }
  }
}

}  // namespace

template <int FMT, int NB>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) weights_kernel(const __grid_constant__ WeightsParams p) {
  using F = Fmt<FMT>;
  constexpr int G = 8 * NB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q4 = lane & 3, r0 = lane >> 2;
  const int warps = blockDim.x >> 5;
  // stages | query fragments | cos, sin | lse | barriers | tile table
  const uint32_t ring0 = sbase + warp * kStages * F::kStage;
  uint32_t at = warps * kStages * F::kStage;
  const uint32_t qf = sbase + at;
  uint4* const qf_p = reinterpret_cast<uint4*>(smem + at);
  at += p.q_len * kSteps * 512;
  float2* const cs = reinterpret_cast<float2*>(smem + at);
  at += p.q_len * kHalf * 8;
  float* const lse2 = reinterpret_cast<float*>(smem + at);
  at += p.q_len * G * 4;
  const uint32_t bar = sbase + at + warp * kStages * 8;
  at += kMaxWarps * kStages * 8;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + at);
  long long* const tbl = reinterpret_cast<long long*>(smem + at + 16);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bar + 8 * i, 1);
    if (warp == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tile_table(tbl, p.batch, lane, [&](int s) {
      const int ctx = p.seq_lens[s];
      if ((ctx < p.q_len || ctx > p.max_seq_len) && blockIdx.x == 0) atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
      return ctx < p.q_len ? 0 : (min(ctx, p.max_seq_len) + kTile - 1) / kTile;
    });
  }
  __syncthreads();
  const long long total = tbl[p.batch] * p.hkv;
  const long long a = blockIdx.x * total / gridDim.x, b = (blockIdx.x + 1) * total / gridDim.x;
  if (a >= b) return;

  // ---- this warp's tiles: a + warp, a + warp + warps, ...
  auto step = [&](TileCursor& c, int n) {
    c.t += n;
    while (c.t >= c.nt) {
      const int over = c.t - c.nt;
      next_unit(tbl, p.hkv, c);
      c.t = over;
    }
  };
  TileCursor ic;
  long long nxt = a + warp;
  if (nxt < b) ic = cursor_at(tbl, p.batch, p.hkv, nxt);
  int ist = 0, pg_s = -1, pg_base = 0, pg = 0;
  auto issue = [&]() {
    if (nxt >= b) return;
    const int key = ic.t * kTile, pi = key / kPage;
    if (ic.s != pg_s || pi < pg_base || pi >= pg_base + 32) {
      pg_s = ic.s;
      pg_base = pi;
      const int last = (ic.nt - 1) * kTile / kPage, mine = pi + lane;
      pg = 0;
      if (mine <= last) {
        pg = mine < p.max_pages ? p.block_table[long(ic.s) * p.max_pages + mine] : -1;
        if (pg < 0 || pg >= p.num_pages) {
          atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
          pg = 0;
        }
      }
    }
    const int page = __shfl_sync(0xffffffffu, pg, pi - pg_base), slot = key % kPage;
    const uint32_t dst = ring0 + ist * F::kStage, br = bar + 8 * ist;
    if (lane == 0) {
      mbar_expect_tx(br, kTile * F::kRow);
      const int row = page * kPage + slot;
#pragma unroll
      for (int i = 0; i < 3; ++i) tma_load_3d(dst + i * (F::kRow / 3) * kTile, &p.tm_k, br, 64 * i, ic.g, row);
    }
    __syncwarp();
    if (++ist == kStages) ist = 0;
    nxt += warps;
    if (nxt < b) step(ic, warps);
  };
  for (int i = 0; i < kStages; ++i) issue();

  int st = 0, ph = 0;
  bool ok = true;
  TileCursor c = cursor_at(tbl, p.batch, p.hkv, a);  // the whole CTA's: the unit's first tile of the piece
  long long x = a;
  int mine = warp;  // this warp's next tile, counted from x
  while (x < b) {
    if (c.t >= c.nt) next_unit(tbl, p.hkv, c);
    const int s = c.s, g = c.g, ctx = p.seq_lens[s], end = min(ctx, p.max_seq_len);
    const int n = int(min((long long)(c.nt - c.t), b - x));  // tiles of this unit in the piece
    // ---- the unit's query fragments
    __syncthreads();  // (the last unit's are read)
    const int pos0 = (p.positions ? p.positions[s] + 1 : ctx) - p.q_len;
    for (int i = threadIdx.x; i < p.q_len * kHalf; i += blockDim.x)
      rope_cos_sin(pos0 + i / kHalf, p.rope.inv_freq[i % kHalf], &cs[i].x, &cs[i].y);
    for (int i = threadIdx.x; i < p.q_len * G; i += blockDim.x) {
      // a row that attended nothing (or whose log-sum-exp is no number) adds nothing
      const float l = p.lse[(long(s) * p.q_len + i / G) * kHq + g * G + i % G];
      lse2[i] = fabsf(l) < INFINITY ? l * kLog2e : INFINITY;
    }
    __syncthreads();
    const uint16_t* qg = p.q + (long(s) * p.q_len * kHq + g * G) * kDqk;
    auto qval = [&](int i, int h, int d) {  // rotated component d of head h of draft i
      const uint16_t* r = qg + (long(i) * kHq + h) * kDqk;
      const float v = bf16_to_f32(r[d]);
      if (d >= kRope) return v;
      const float w = bf16_to_f32(r[d ^ kHalf]);
      const float2 t = cs[i * kHalf + (d & (kHalf - 1))];
      return d < kHalf ? v * t.x - w * t.y : v * t.x + w * t.y;
    };
    float amax = 0.f;
    for (int it = warp; it < p.q_len * kSteps; it += warps) {
      const int i = it / kSteps, kq = it % kSteps;
      uint32_t r[4] = {0, 0, 0, 0};  // (b0, b1) of heads r0, then of heads 8 + r0
      const bool rest = kq >= 12 && kq < 16;
      const int kk = rest ? kq - 12 : kq;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int h = 8 * nb + r0;
        // (a row that adds nothing may hold NaN or infinities, which no log-sum-exp would cancel: 0)
        const float on = lse2[i * G + h];
#pragma unroll
        for (int bb = 0; bb < 2; ++bb) {
          float v[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // (E4M3 keys come out of ldmatrix as 4 consecutive dims a lane)
            const float x = qval(i, h, FMT == MIMO_DTYPE_BF16 ? 16 * kk + 8 * bb + 2 * q4 + e : 16 * kk + 4 * q4 + 2 * bb + e);
            v[e] = on < INFINITY ? x : 0.f;
          }
          if (FMT == MIMO_DTYPE_BF16 && kk >= 4) {
            r[2 * nb + bb] = pack2_bf16(v[0], v[1]);
          } else {
            r[2 * nb + bb] = pack2_f16_sat(v[0], v[1], amax);
            if (rest) {
              const float2 t = f32x2_of(r[2 * nb + bb]);
              r[2 * nb + bb] = pack2_f16(v[0] - t.x, v[1] - t.y);
            }
          }
        }
      }
      qf_p[it * 32 + lane] = make_uint4(r[0], r[1], r[2], r[3]);
    }
    if (amax > kF16Max) atomicOr(p.status, MIMO_STATUS_RANGE);
    __syncthreads();

    const float c_log2 = p.scale_log2 * (FMT == MIMO_DTYPE_FP8_E4M3 ? p.k_dequant[g] : 1.f);
    float* const row_out = p.scores + (long(s) * p.hkv + g) * p.score_stride;
    for (; mine < n && ok; mine += warps) {
      const int key0 = (c.t + mine) * kTile;
      // lane q4 < 2 adds to keys r0 + 8 q4 (+ 16): fetched before the tile is waited for
      float old[2];
      int slot[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        slot[m] = key0 + 16 * m + r0 + 8 * (q4 & 1);
        old[m] = q4 < 2 && slot[m] < end ? row_out[slot[m]] : 0.f;
      }
      if (!__all_sync(0xffffffffu, mbar_wait(bar + 8 * st, ph & 1, abort_flag, p.status, MIMO_STATUS_TIMEOUT))) {
        ok = false;
        break;
      }
      const uint32_t kb = ring0 + st * F::kStage;
      float add[2][2] = {{0.f, 0.f}, {0.f, 0.f}};  // keys r0, r0 + 8 of either half
      for (int i = 0; i < p.q_len; ++i) {
        const uint32_t qi = qf + i * kSteps * 512 + lane * 16;
        float S[2][NB][4];
        auto q_frag = [&](int kq, uint32_t* r) {
          asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                       : "r"(qi + kq * 512)
                       : "memory");
        };
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) S[m][nb][0] = S[m][nb][1] = S[m][nb][2] = S[m][nb][3] = 0.f;
        constexpr int kPer = FMT == MIMO_DTYPE_BF16 ? 1 : 2;  // steps a key fragment load covers
#pragma unroll
        for (int k2 = 0; k2 < 12; k2 += kPer) {
          uint32_t ka[2][4 * kPer];
#pragma unroll
          for (int m = 0; m < 2; ++m) key_frag<FMT>(kb, 16 * m, k2, lane, ka[m]);
#pragma unroll
          for (int t = 0; t < kPer; ++t) {
            const int kk = k2 + t;
            uint32_t r[4], rr[4];
            q_frag(kk, r);
            if (kk < 4) q_frag(12 + kk, rr);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                if (FMT == MIMO_DTYPE_BF16 && kk >= 4) mma_bf16_acc(S[m][nb], ka[m] + 4 * t, r[2 * nb], r[2 * nb + 1]);
                else mma_f16_acc(S[m][nb], ka[m] + 4 * t, r[2 * nb], r[2 * nb + 1]);
                if (kk < 4) mma_f16_acc(S[m][nb], ka[m] + 4 * t, rr[2 * nb], rr[2 * nb + 1]);
              }
          }
        }
        // heads 8 nb + 2 q4, + 1
        const int last = min(end - 1, ctx - p.q_len + i);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const float2 l = *reinterpret_cast<const float2*>(lse2 + i * G + 8 * nb + 2 * q4);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const float v0 = ex2(fmaf(S[m][nb][0], c_log2, -l.x)) + ex2(fmaf(S[m][nb][1], c_log2, -l.y));
            const float v1 = ex2(fmaf(S[m][nb][2], c_log2, -l.x)) + ex2(fmaf(S[m][nb][3], c_log2, -l.y));
            if (key0 + 16 * m + r0 <= last) add[m][0] += v0;
            if (key0 + 16 * m + r0 + 8 <= last) add[m][1] += v1;
          }
        }
      }
      __syncwarp();
      issue();  // the stage is read
#pragma unroll
      for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          add[m][e] += __shfl_xor_sync(0xffffffffu, add[m][e], 1);
          add[m][e] += __shfl_xor_sync(0xffffffffu, add[m][e], 2);
        }
        if (q4 < 2 && slot[m] < end) row_out[slot[m]] = old[m] + (q4 ? add[m][1] : add[m][0]);
      }
      if (++st == kStages) st = 0, ++ph;
    }
    // (a wait that ran out: the warp goes on to the next barriers with nothing to do)
    mine -= n;
    if (!ok) mine = 0x3fffffff;
    c.t += n;
    x += n;
  }
  if (!ok && lane == 0) {
    // the copies under way land before the warp leaves: the stage waited for, and the one after it
    int dummy = 0;
    const long long done = nxt - warps;  // the last tile that was issued
    mbar_wait(bar + 8 * st, ph & 1, &dummy, nullptr, 0, 50000000ull);
    if (done >= a + warp + warps) mbar_wait(bar + 8 * (st ^ 1), (ph + (st == 1 ? 1 : 0)) & 1, &dummy, nullptr, 0, 50000000ull);
  }
}

namespace {
template <int FMT>
int smem_of(int warps, int q_len, int hkv) {
  const int G = kHq / hkv;
  return 1024 + warps * kStages * Fmt<FMT>::kStage + q_len * (kSteps * 512 + kHalf * 8 + G * 4) +
         kMaxWarps * kStages * 8 + 16 + (kMaxTableBatch + 1) * 8;
}
template <int FMT, int NB>
cudaError_t launch_weights_fmt(const WeightsParams& p, int sms, cudaStream_t s) {
  int warps = kMaxWarps;  // as many as their stages fit beside the drafts' fragments
  while (smem_of<FMT>(warps, p.q_len, p.hkv) > kMaxSmem) --warps;
  const int bytes = smem_of<FMT>(warps, p.q_len, p.hkv);
  // (the attribute is the kernel's, not the launch's: always the same value, as another host thread may be
  // between its own two calls)
  cudaError_t e = cudaFuncSetAttribute(weights_kernel<FMT, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e != cudaSuccess) return e;
  const long long tiles = ((long long)p.max_seq_len + kTile - 1) / kTile * p.batch * p.hkv;
  weights_kernel<FMT, NB><<<int(tiles < sms ? tiles : sms), warps * 32, bytes, s>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_weights(const WeightsParams& p, int sms, cudaStream_t s) {
  switch (p.cache_dtype * 2 + (p.hkv == 8)) {
    case MIMO_DTYPE_BF16 * 2: return launch_weights_fmt<MIMO_DTYPE_BF16, 2>(p, sms, s);
    case MIMO_DTYPE_BF16 * 2 + 1: return launch_weights_fmt<MIMO_DTYPE_BF16, 1>(p, sms, s);
    case MIMO_DTYPE_FP8_E4M3 * 2: return launch_weights_fmt<MIMO_DTYPE_FP8_E4M3, 2>(p, sms, s);
    case MIMO_DTYPE_FP8_E4M3 * 2 + 1: return launch_weights_fmt<MIMO_DTYPE_FP8_E4M3, 1>(p, sms, s);
    default: return launch_weights_int4(p, sms, s);
  }
}

}  // namespace mimo
