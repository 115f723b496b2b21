// Attention weights per cached slot (weights.cu) over 4-bit keys, the logits on tcgen05.
//
// On mma.sync this operator is bound by the products: 17 steps of 16 x 8 x 16 per 16 keys and
// draft, at 8.9 cycles of a scheduler each, and the keys unpacked again for every draft (235 us
// for 8 sequences of 4099..65536 keys and 4 drafts, 130 MB).  A tcgen05.mma of 128 keys and 64
// columns costs 34 cycles of a unit of its own, so all drafts of a KV head (up to 64 rows: 4
// drafts of 16 heads, 8 of 8) are one product's columns, and a key is unpacked once: 88 us, and
// 60 us with one token.
//
// One CTA per SM takes a contiguous piece of the line of 128-key tiles (a tile is a page).  Two
// threads share a key: they unpack half of its words each into the A operand in tensor memory,
// and each applies the key's 6 scales to its half of the columns' 6 group sums and adds up the
// exponentials; one of the two updates the score.  (Four threads a key: 98 us for the call above.)
// The tensor memory is 96 columns of keys, 8 of a constant (the code offset's factor) and 6 x 64
// of sums, all single: groups 0..2 and 3..5 run as two parts, so that the products of one run
// behind the arithmetic on the other (three parts were a tenth slower, six two fifths).  What
// bounds the kernel is the chain of the parts' handshakes, which eight warps do not cover: no pipe is
// above 36 % (1.5 TB/s).  A ninth warp issues copies and products.
#include "int4_tc.cuh"
#include "tiles.cuh"
#include "../../include/mimoattn.h"

namespace mimo {

namespace {

constexpr int kTile = kPage, kStages = 6;
constexpr int kStage = kTile * kI4KSlot;  // codes, then scales, as a page holds them
constexpr int kOffKs = kTile * kI4KCodes;
constexpr int kMaxCols = 64, kMaxDrafts = 8;
constexpr int kShare = 2, kWork = 128 * kShare;  // threads per key, of a tile
constexpr int kParts = 2, kPer = kI4KGroups / kParts;  // parts of a tile, groups of a part
// query operand: 128-byte rows of 64 elements (128-byte swizzle) of up to 64 query rows: dims 0..63,
// 64..127, 128..191, the second terms of dims 0..63; then a 32-byte row (32-byte swizzle) of the
// offset per column of sums
constexpr int kQChunk = kMaxCols * 128, kQOffset = 4 * kQChunk, kQBytes = kQOffset + 6 * kMaxCols * 32;
constexpr int kOffStage = kQBytes;
constexpr int kOffCs = kOffStage + kStages * kStage;     // cos, sin of each draft
constexpr int kOffLse = kOffCs + kMaxDrafts * kHalf * 8;
constexpr int kOffPart = kOffLse + kMaxCols * 4;         // the other threads' sums, two buffers
constexpr int kOffBar = kOffPart + 2 * (kShare - 1) * kTile * 4;
constexpr int kOffTbl = kOffBar + 288;
constexpr int kSmem = kOffTbl + (kMaxTableBatch + 1) * 8 + 1024;
static_assert(kSmem <= 232448 && kOffStage % 128 == 0 && kOffBar % 8 == 0, "shared memory budget");
constexpr uint32_t kColA = 0, kColOne = 96, kColD = 128;
constexpr float kLog2e = 1.4426950408889634f;

// Steps KK .. of part PT of a tile's products, N columns a group (two terms for groups 0, 1).
template <int N, int PT, int KK>
__device__ __forceinline__ void product_steps(uint32_t tmem, uint32_t lo, uint32_t hi) {
  if constexpr (KK < 2 * kPer * (PT + 1)) {
    constexpr uint32_t idesc = idesc_f32acc(128, N, 0, 0, 0), d = kColD + (KK >> 1) * N, a = kColA + 8 * KK;
    tc_mma_ts_at<d, a, (((KK >> 2) * kQChunk + (KK & 3) * 32) >> 4)>(tmem, lo, hi, idesc);
    if constexpr (KK < 4) tc_mma_ts_at<d, a, ((3 * kQChunk + KK * 32) >> 4)>(tmem, lo, hi, idesc);
    product_steps<N, PT, KK + 1>(tmem, lo, hi);
  }
}
// The part: the offset over its groups, then their steps.
template <int N, int PT>
__device__ __forceinline__ void products(uint32_t tmem, uint64_t qd, uint64_t qo) {
  tc_fence_after();
  tc_mma_ts(tmem + kColD + kPer * PT * N, tmem + kColOne, qo + ((kPer * PT * N * 32) >> 4),
            idesc_f32acc(128, kPer * N, 0, 0, 0), 0u);
  product_steps<N, PT, 2 * kPer * PT>(tmem, uint32_t(qd), uint32_t(qd >> 32));
}

// Parts PT .. of a tile: each once its keys stand in A and its old sums are read.
template <int N, int PT, class W>
__device__ __forceinline__ bool issue_part(W&& ready, uint32_t tmem, uint64_t qd, uint64_t qo, uint32_t done0) {
  if constexpr (PT < kParts) {
    if (!ready(PT)) return false;
    if (elect_one()) {
      products<N, PT>(tmem, qd, qo);
      tc_commit(done0 + 8 * PT);
    }
    __syncwarp();
    return issue_part<N, PT + 1>(ready, tmem, qd, qo, done0);
  }
  return true;
}

}  // namespace

template <int NC>  // columns of a thread
__global__ void __launch_bounds__(kWork + 32, 1) weights_int4_kernel(const __grid_constant__ WeightsParams p) {
  constexpr int N = kShare * NC;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool issuer = warp == kWork / 32;
  const int gq = warp & 3, hw = warp >> 2;  // the quarter of the tile's keys, and which of a key's two threads
  const uint32_t bar0 = sbase + kOffBar;
  auto full = [&](int i) { return bar0 + 8 * i; };
  auto empty = [&](int i) { return bar0 + 8 * (kStages + i); };
  auto a_ready = [&](int h) { return bar0 + 16 * kStages + 8 * h; };
  auto done = [&](int h) { return bar0 + 16 * kStages + 8 * kParts + 8 * h; };
  volatile int* const bad_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 240);  // [2]
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 248);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + 256);
  float2* const cs = reinterpret_cast<float2*>(smem + kOffCs);
  float* const lse2 = reinterpret_cast<float*>(smem + kOffLse);
  float* const part = reinterpret_cast<float*>(smem + kOffPart);
  long long* const tbl = reinterpret_cast<long long*>(smem + kOffTbl);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), kWork / 32);
    }
    for (int h = 0; h < kParts; ++h) {
      mbar_init(a_ready(h), kWork / 32);
      mbar_init(done(h), 1);
    }
    bad_flag[0] = bad_flag[1] = 0;
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 1)
    tile_table(tbl, p.batch, lane, [&](int s) {
      const int ctx = p.seq_lens[s];
      if ((ctx < p.q_total || ctx > p.max_seq_len) && blockIdx.x == 0) atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
      return ctx < p.q_total ? 0 : (min(ctx, p.max_seq_len) + kTile - 1) / kTile;
    });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);  // (known uniform)
  const long long total = tbl[p.batch] * p.hkv;
  const long long a = blockIdx.x * total / gridDim.x, b = (blockIdx.x + 1) * total / gridDim.x;
  const int n_all = int(b - a);
  auto wait_w = [&](uint32_t bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;  // (a branch of the whole warp)
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, MIMO_STATUS_TIMEOUT));
  };

  if (issuer) {
    if (n_all > 0) {
      TileCursor ic = cursor_at(tbl, p.batch, p.hkv, a);
      int pg_s = -1, pg_base = 0, pg = 0;  // lane i: page id of page pg_base + i of sequence pg_s
      auto copy = [&](int n) {             // tile n of the piece
        if (ic.t == ic.nt) next_unit(tbl, p.hkv, ic);
        const int pi = ic.t;
        if (ic.s != pg_s || pi < pg_base || pi >= pg_base + 32) {
          pg_s = ic.s;
          pg_base = pi;
          const int mine = pi + lane;
          pg = 0;
          if (mine < ic.nt) {
            pg = mine < p.max_pages ? p.block_table[long(ic.s) * p.max_pages + mine] : -1;
            if (pg < 0 || pg >= p.num_pages) {
              atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
              pg = 0;
            }
          }
        }
        const long block = long(__shfl_sync(0xffffffffu, pg, pi - pg_base)) * p.hkv + ic.g;
        if (lane == 0) {
          mbar_expect_tx(full(n % kStages), kStage);
          bulk_load(sbase + kOffStage + n % kStages * kStage, p.k_cache + block * kStage, kStage, full(n % kStages));
        }
        __syncwarp();
        ++ic.t;
      };
      const uint64_t qd = sdesc_sw128(sbase, 16, 1024), qo = sdesc_sw32(sbase + kQOffset, 256);
      int copied = 0, n = 0;
      bool ok = true;
      for (; copied < n_all && copied < kStages; ++copied) copy(copied);
      for (; n < n_all && ok; ++n) {
        ok = issue_part<N, 0>([&](int h) { return wait_w(a_ready(h), n & 1); }, tmem, qd, qo, done(0));
        if (!ok) break;
        if (n >= 2 && copied < n_all) {
          if (!(ok = wait_w(empty(copied % kStages), (copied / kStages - 1) & 1))) break;
          copy(copied++);
        }
      }
      if (!ok && elect_one()) {
        // a wait ran out: the copies and products under way end before the block does
        int dummy = 0;
        for (int i = copied > kStages ? copied - kStages : 0; i < copied; ++i)
          mbar_wait(full(i % kStages), (i / kStages) & 1, &dummy, nullptr, 0, 50000000ull);
        tc_commit(done(kParts - 1));
        for (int i = 1; i >= 0; --i) mbar_wait(done(kParts - 1), (n + i) & 1, &dummy, nullptr, 0, 50000000ull);
      }
    }
    tc_fence_before();
    __syncthreads();
    return;
  }

  const uint32_t t_lane = tmem + (uint32_t(gq * 32) << 16);
  auto all_sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(kWork) : "memory"); };
  // A barrier at which a warp whose wait ran out takes the others with it (alternating flags: a warp
  // ahead of the others writes the other one).
  int tick = 0;
  auto all_sync_ok = [&](bool good) -> bool {
    if (!good && lane == 0) bad_flag[tick & 1] = 1;
    all_sync();
    const bool ok = bad_flag[tick & 1] == 0;
    ++tick;
    return ok;
  };
  if (hw == 0) {
    uint32_t one[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) one[i] = 0x04000400u;  // 2^-14
    tmem_st8(t_lane + kColOne, one);
    tmem_wait_st();
  }
  // This thread's half of its key's words: word 4 j + 2 hw + q of group j at 6 q + j.
  auto fetch = [&](uint32_t stage, uint32_t* W) {
    const uint32_t ka = stage + (gq * 32 + lane) * kI4KCodes + 48 * hw;
#pragma unroll
    for (int i = 0; i < 3; ++i) lds128(ka + 16 * i, W + 4 * i);
  };
  // The groups of part h of them into the key's row of A.
  auto unpack = [&](const uint32_t* W, int h) {
#pragma unroll
    for (int j = kPer * h; j < kPer * (h + 1); ++j) {
      uint32_t r[8];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t x = W[6 * q + j], y = x >> 8;
        r[4 * q] = x & kI4Lo;
        r[4 * q + 1] = x & kI4Hi;
        r[4 * q + 2] = y & kI4Lo;
        r[4 * q + 3] = y & kI4Hi;
      }
      tmem_st8(t_lane + kColA + 16 * j + 8 * hw, r);
    }
    tmem_wait_st();
  };
  auto hand_over = [&](int h) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(a_ready(h));
  };
  const int G = kHq / p.hkv, rows = p.q_len * G;
  const float c_log2 = p.scale_log2 * kI4KeyUnit;
  const uint64_t c2 = pack_f32x2(c_log2, c_log2);
  int st = 0, ph = 0;
  bool ok = true;
  TileCursor c;
  if (n_all > 0) c = cursor_at(tbl, p.batch, p.hkv, a);
  for (int x = 0; x < n_all && ok;) {
    if (c.t == c.nt) next_unit(tbl, p.hkv, c);
    const int s = c.s, g = c.g, ctx = p.seq_lens[s], end = min(ctx, p.max_seq_len);
    const int t_end = min(c.nt, c.t + (n_all - x));
    // ---- the unit's query operand
    const float amax = int4_query_operand<N, kWork, kQChunk>(
        p.q + ((long(s) * p.q_total + p.q_first) * kHq + g * G) * kDqk, rows, G == 16 ? 4 : 3, sbase, threadIdx.x, cs, [&]() {
          const int pos0 = (p.positions ? p.positions[s] + 1 : ctx) - p.q_total + p.q_first;
          for (int i = threadIdx.x; i < p.q_len * kHalf; i += kWork)
            rope_cos_sin(pos0 + i / kHalf, p.rope.inv_freq[i % kHalf], &cs[i].x, &cs[i].y);
          if (threadIdx.x < N) {
            // a row that attended nothing (or whose log-sum-exp is no number) adds nothing, nor does a padding column
            float l = INFINITY;
            if (threadIdx.x < rows) {
              l = p.lse[(long(s) * p.q_total + p.q_first + threadIdx.x / G) * kHq + g * G + threadIdx.x % G];
              l = fabsf(l) < INFINITY ? l * kLog2e : INFINITY;
            }
            lse2[threadIdx.x] = -l;  // (added to the logits)
          }
          all_sync();
        },
        // (a row that adds nothing may hold NaN or infinities, which no log-sum-exp would cancel)
        [&](int n) { return lse2[n] != -INFINITY; });
    if (amax > kF16Max) atomicOr(p.status, MIMO_STATUS_RANGE);
    fence_proxy_async_smem();
    all_sync();
    bool good = wait_w(full(st), ph & 1);
    uint32_t W[12];
    if (good) {
      fetch(sbase + kOffStage + st * kStage, W);
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        unpack(W, h);
        hand_over(h);
      }
    }
    float* const row_out = p.scores + (long(s) * p.hkv + g) * p.score_stride;
    for (; c.t < t_end; ++c.t, ++x) {
      const uint32_t stage = sbase + kOffStage + st * kStage;
      const int key = c.t * kTile + gq * 32 + lane;
      const float old = hw == 0 && key < end ? row_out[key] : 0.f;
      int nst = st + 1, nph = ph;
      if (nst == kStages) nst = 0, ++nph;
      uint64_t S[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) S[i] = 0;
      uint32_t z[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) z[i] = lds32(stage + kOffKs + (gq * 32 + lane) * 2 * kI4KGroups + 4 * i);
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        if (good) good = wait_w(done(h), x & 1);
        if (good) {
          tc_fence_after();
          constexpr int kC = NC % 16 ? 8 : 16;  // columns at a time
#pragma unroll
          for (int c0 = 0; c0 < NC; c0 += kC) {
            uint32_t d[kPer][kC];
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
              const uint32_t at = t_lane + kColD + (kPer * h + j) * N + hw * NC + c0;
              if constexpr (kC == 16) tmem_ld16(at, d[j]);
              else tmem_ld8(at, d[j]);
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
              if (j > 0) tied<kC>(d[j]);  // (one wait is for all)
              else if constexpr (kC == 16) tmem_wait_ld_r16(d[j]);
              else tmem_wait_ld_r8(d[j]);
              const float2 zz = f32x2_of_f16x2(z[(kPer * h + j) >> 1]);
              const float sc = ((kPer * h + j) & 1) ? zz.y : zz.x;
              const uint64_t s2 = pack_f32x2(sc, sc);
#pragma unroll
              for (int i = 0; i < kC / 2; ++i)
                S[c0 / 2 + i] = fma_f32x2(pack_f32x2(__uint_as_float(d[j][2 * i]), __uint_as_float(d[j][2 * i + 1])), s2, S[c0 / 2 + i]);
            }
          }
          if (c.t + 1 < t_end) {
            if (h == 0) {
              good = wait_w(full(nst), nph & 1);
              fetch(sbase + kOffStage + nst * kStage, W);
            }
            if (good) {
              unpack(W, h);
              hand_over(h);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(st));
      // ---- probabilities: 4 columns at a time are of one draft
      float add = 0.f;
#pragma unroll
      for (int i = 0; i < NC / 4; ++i) {
        const int col = hw * NC + 4 * i;
        uint32_t l[4];
        lds128(sbase + kOffLse + col * 4, l);
        uint64_t v = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint64_t e = fma_f32x2(S[2 * i + k], c2, pack_f32x2(__uint_as_float(l[2 * k]), __uint_as_float(l[2 * k + 1])));
          v = add_f32x2(v, pack_f32x2(ex2(lo_f32(e)), ex2(hi_f32(e))));
        }
        if (key <= ctx - p.q_total + p.q_first + col / G) add += lo_f32(v) + hi_f32(v);
      }
      float* const buf = part + (x & 1) * (kShare - 1) * kTile + gq * 32 + lane;
      if (hw) *buf = add;
      asm volatile("bar.sync %0, %1;" ::"r"(2 + gq), "n"(32 * kShare) : "memory");
      if (hw == 0 && key < end) row_out[key] = old + (add + *buf);
      st = nst;
      ph = nph;
    }
    // a warp whose wait ran out takes the others with it here
    ok = all_sync_ok(good);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

namespace {
template <int NC>
cudaError_t launch_cols(const WeightsParams& p, int grid, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(weights_int4_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  weights_int4_kernel<NC><<<grid, kWork + 32, kSmem, s>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_weights_int4(WeightsParams p, int sms, cudaStream_t s) {
  const int G = kHq / p.hkv, per = kMaxCols / G;  // drafts of a launch (each adds to the scores)
  const long long tiles = ((long long)p.max_seq_len + kTile - 1) / kTile * p.batch * p.hkv;
  const int grid = int(tiles < sms ? tiles : sms);
  p.q_total = p.q_len;
  for (p.q_first = 0; p.q_first < p.q_total; p.q_first += per) {
    p.q_len = p.q_total - p.q_first < per ? p.q_total - p.q_first : per;
    cudaError_t e;
    switch ((p.q_len * G + 15) / 16) {
      case 1: e = launch_cols<8>(p, grid, s); break;
      case 2: e = launch_cols<16>(p, grid, s); break;
      case 3: e = launch_cols<24>(p, grid, s); break;
      default: e = launch_cols<32>(p, grid, s); break;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mimo
