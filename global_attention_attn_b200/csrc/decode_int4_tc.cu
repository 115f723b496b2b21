// One-token decode over a 4-bit paged cache, the logits on the 5th-generation tensor cores.
//
// The mma.sync kernel of decode_int4.cu spends most of its issue slots on the logits: an
// mma.sync m16n8k16 takes 8.9 cycles of a scheduler during which the other instructions it
// dispatches do not come for free (an mma.sync and four LOP3, 2 cycles each, measured 12.2 to
// 12.8 cycles, not 8.9).  Here S^T = K Q^T runs as tcgen05.mma: a group of four warps takes 128
// keys, each thread unpacks its own key (int4.cuh: one shift and four ANDs per 8 codes, no
// conversion) into its row of the A operand in tensor memory, and reads back 16 heads times 6
// group sums of its row, to which it applies its key's 6 scales.  Both sides of a
// thread-per-key layout are free of shuffles, and a key's scales are read and converted once.
//   - The rotated query dims enter as two fp16 terms (no 16-bit type holds them to the digits of
//     an fp32 log-sum-exp); the code offset is one more k-step, a constant row of A against -8 *
//     the query's group sums (two fp16 terms).  Both terms are columns of one product (N = 32), and the
//     offset is one product over all columns, which also starts the sums: 13 products a tile.  Tensor memory of a group: 96 columns of keys, 8 of the constant, 128 of sums.
//   - O = P V stays on mma.sync with the accumulators in registers (decode_int4.cu explains the
//     operands): P goes through shared memory, transposed by ldmatrix.  Each warp sums over its
//     own keys against its own reference; the four warps meet at the end of a unit.
// The keys of tile i + 1 are unpacked before the softmax and P V of tile i, so the tensor cores
// work behind the arithmetic.  Two groups per CTA, one CTA per SM, four 23 KB stages each; a
// ninth and a tenth warp issue the groups' copies and products (by one of the four warps, the
// other three waited for its 22 issues every tile: 716 against 530 us with them left out), so the
// warps that compute meet only on mbarriers, and at the ends of units.
#include "common.cuh"
#include "int4.cuh"
#include "ptx.cuh"
#include "tiles.cuh"
#include "../../include/mimoattn.h"

namespace mimo {

namespace {

constexpr int kTile = kI4TcTile, kGroups = kI4TcGroups, kStages = 4;
constexpr int kThreads = (kGroups + 1) * 128;  // the groups, and a warpgroup whose first warps issue
// registers: 384 x 168 at launch = 256 x 224 + 128 x 56
constexpr int kRegsWork = 224, kRegsIssue = 56;
static_assert(kGroups * 128 * kRegsWork + 128 * kRegsIssue <= kThreads * 168, "register split");
static_assert(kTile == kPage, "a tile is a page");
// stage: value codes (64-byte swizzle), key codes, key scales, value scales
constexpr int kOffK = kTile * kI4VCodes, kOffKs = kOffK + kTile * kI4KCodes;
constexpr int kOffVs = kOffKs + kTile * 2 * kI4KGroups, kStage = kOffVs + kTile * 2 * kI4VGroups;
static_assert(kStage % 512 == 0, "64-byte swizzle alignment");
// query operand of a group, 128-byte rows of 64 elements with the 128-byte swizzle: dims 0..63 of
// 16 heads and their second terms (32 rows), dims 64..127, dims 128..191; then the offsets: a
// 32-byte row (16 elements, 32-byte swizzle) per column of sums
constexpr int kQOff1 = 32 * 128, kQOff2 = kQOff1 + 16 * 128, kQOffset = kQOff2 + 16 * 128;
constexpr int kCols = 128;  // of sums: groups 0, 1: 16 heads and their second terms, groups 2..5: 16 heads
constexpr int kQBytes = kQOffset + kCols * 32;
__host__ __device__ constexpr int col_of(int j) { return j < 2 ? 32 * j : 64 + 16 * (j - 2); }
constexpr int kPRow = 48, kPBytes = 32 * kPRow;  // a warp's P: 16 heads per key, rows apart in banks
constexpr int kOffP = kGroups * kQBytes;
constexpr int kOffStage = kOffP + kGroups * 4 * kPBytes;
static_assert(kOffStage % 512 == 0, "stage alignment");
constexpr int kOffBar = kOffStage + kGroups * kStages * kStage;
constexpr int kOffX = kOffBar + 256;  // a group's (reference, sum) of 16 heads per warp
constexpr int kOffTbl = kOffX + kGroups * 4 * 2 * 16 * 4;
constexpr int kSmem = kOffTbl + (kMaxTableBatch + 1) * 8 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");
// tensor memory of a group
constexpr uint32_t kColA = 0, kColOne = 96, kColD = 128, kColGroup = 256;
static_assert(kColD + kCols <= kColGroup && kGroups * kColGroup <= 512, "tensor memory");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Weights are 2^(z - ref): ref is a row's maximum when it was set, and moves only when a logit
// passes it by more than this many powers of two (2^6 * 1023, the largest value scale an
// append stores, is still a finite fp16).
constexpr float kSlack = 6.f;

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
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
__device__ __forceinline__ void sts16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// (x ^ flip) & mask, one LOP3: an immediate mask and `flip` in a register
__device__ __forceinline__ uint32_t field(uint32_t x, uint32_t flip, uint32_t mask) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x28;" : "=r"(d) : "r"(x), "r"(flip), "r"(mask));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ void mma_f16_acc(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  mma_f16_c(d, a, b0, b1, d);
}

// Steps KK .. 11 of a tile's products.
template <int KK>
__device__ __forceinline__ void product_steps(uint32_t tmem, uint32_t qd_lo, uint32_t qd_hi) {
  if constexpr (KK < 12) {
    constexpr int row = KK < 4 ? 0 : (KK < 8 ? kQOff1 : kQOff2);
    tc_mma_ts_at<kColD + col_of(KK >> 1), kColA + 8 * KK, ((row + (KK & 3) * 32) >> 4)>(
        tmem, qd_lo, qd_hi, idesc_f32acc(128, KK < 4 ? 32 : 16, 0, 0, 0));
    product_steps<KK + 1>(tmem, qd_lo, qd_hi);
  }
}

// Keys a sequence's unit covers: [lo, hi], and its first tile and tile count.
struct Span {
  int lo, hi, t0, nt;
};
__device__ __forceinline__ Span span_of(const Decode4Params& p, int ctx) {
  Span u;
  u.hi = min(ctx, p.max_seq_len) - 1;
  u.lo = p.window > 0 ? max(0, ctx - p.window) : 0;
  if (ctx < 1 || u.lo > u.hi) {
    u.t0 = u.nt = 0;
  } else {
    u.t0 = u.lo / kTile;
    u.nt = u.hi / kTile - u.t0 + 1;
  }
  return u;
}

}  // namespace

template <int NB>  // blocks of 8 heads per KV head: 2 (global layers) or 1
__global__ void __launch_bounds__(kThreads, 1) decode4_tc_kernel(const __grid_constant__ Decode4Params p) {
  constexpr int G = 8 * NB, H2 = G / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool issuer = warp >= kGroups * 4;
  const int grp = __shfl_sync(0xffffffffu, issuer ? warp - kGroups * 4 : warp >> 2, 0), gw = warp & 3;
  const int q4 = lane & 3, r0 = lane >> 2;
  const uint32_t qt = sbase + grp * kQBytes, pt = sbase + kOffP + warp * kPBytes;
  const uint32_t ring0 = sbase + kOffStage + grp * kStages * kStage;
  const uint32_t bar0 = sbase + kOffBar + grp * 96;
  auto full = [&](int i) { return bar0 + 8 * i; };
  auto empty = [&](int i) { return bar0 + 8 * (kStages + i); };
  const uint32_t a_ready = bar0 + 16 * kStages;   // a tile's keys stand in A, the sums before them are read
  const uint32_t mma_done = a_ready + 8;          // its sums stand in D
  volatile int* const bad_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 192 + grp * 8);  // [2]
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 208);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffBar + 224);
  float* const xch = reinterpret_cast<float*>(smem + kOffX) + grp * 128;  // [4 warps][ref 16 | sum 16]
  long long* const tbl = reinterpret_cast<long long*>(smem + kOffTbl);
  if (!issuer && gw == 0 && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 4);
    }
    mbar_init(a_ready, 4);
    mbar_init(mma_done, 1);
    bad_flag[0] = bad_flag[1] = 0;
    if (grp == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == kGroups * 4 - 1) {
    tile_table(tbl, p.batch, lane, [&](int s) {
      const int ctx = p.seq_lens[s];
      if (blockIdx.x == 0 && (ctx < 1 || ctx > p.max_seq_len))
        atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
      return span_of(p, ctx).nt;
    });
    if (blockIdx.x == 0 && p.ws_tbl)
      for (int s = lane; s <= p.batch; s += 32) p.ws_tbl[s] = tbl[s];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot + grp * kColGroup, 0);  // (known uniform)
  const uint32_t t_lane = tmem + (uint32_t(gw * 32) << 16);

  // ---- this group's piece of the line
  const long long total = tbl[p.batch] * p.hkv;
  const int w = grp * gridDim.x + blockIdx.x;
  long long a = 0, b = 0;
  if (grp >= kGroups) {
    // the issuing warpgroup's idle warps
  } else if (total > 0 && p.whole_units) {
    const long long units = (long long)p.batch * p.hkv;
    const int W = int(units < p.workers ? units : p.workers);
    auto at = [&](long long u) {
      const int s = int(u / p.hkv);
      return s >= p.batch ? total : tbl[s] * p.hkv + (u - (long long)s * p.hkv) * (tbl[s + 1] - tbl[s]);
    };
    if (w < W) {
      a = at(w * units / W);
      b = at((w + 1) * units / W);
    }
  } else if (total > 0) {
    const int W = pieces_of(total, p.min_tiles, p.workers);
    if (w < W) {
      a = w * total / W;
      b = (w + 1) * total / W;
    }
  }
  const int n_all = int(b - a);
  auto wait_w = [&](uint32_t bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, MIMO_STATUS_TIMEOUT));
  };
  auto group_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(grp + 1) : "memory"); };
  // A barrier at which a warp whose wait ran out takes the whole group with it.  The flags
  // alternate: a warp ahead of the others writes the other one.
  int tick = 0;
  auto group_sync_ok = [&](bool good) -> bool {
    if (!good && lane == 0) bad_flag[tick & 1] = 1;
    group_sync();
    const bool ok = bad_flag[tick & 1] == 0;
    ++tick;
    return ok;
  };

  if (issuer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (n_all > 0) {
      // ---- copies of the piece's tiles in order, kStages ahead, and each tile's products
      TileCursor ic = cursor_at(tbl, p.batch, p.hkv, a);
      int pg_s = -1, pg_base = 0, pg = 0, it0 = 0;  // lane i: page id of page pg_base + i of sequence pg_s
      // what lanes 0..3 copy: key codes, key scales, value scales (bulk copies), value codes (a TMA tile)
      const int lane_bytes = lane == 0 ? kI4KCodes : (lane == 1 ? 2 * kI4KGroups : 2 * kI4VGroups);
      const uint32_t lane_dst = lane == 0 ? kOffK : (lane == 1 ? kOffKs : kOffVs);
      const int lane_block = kPage * (lane < 2 ? kI4KSlot : kI4VSlot);
      const uint8_t* const lane_src =
          lane == 0 ? p.k_cache : (lane == 1 ? p.k_cache + kPage * kI4KCodes : p.v_cache + kPage * kI4VCodes);
      auto copy = [&](int n) {  // tile n of the piece
        if (ic.t == ic.nt) next_unit(tbl, p.hkv, ic);
        if (ic.s != pg_s) it0 = span_of(p, p.seq_lens[ic.s]).t0;
        const int pi = it0 + ic.t;
        if (ic.s != pg_s || pi < pg_base || pi >= pg_base + 32) {
          pg_s = ic.s;
          pg_base = pi;
          const int mine = pi + lane;
          pg = 0;
          if (mine < it0 + ic.nt) {
            pg = mine < p.max_pages ? p.block_table[long(ic.s) * p.max_pages + mine] : -1;
            if (pg < 0 || pg >= p.num_pages) {
              atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
              pg = 0;
            }
          }
        }
        const int block = __shfl_sync(0xffffffffu, pg, pi - pg_base) * p.hkv + ic.g;
        const uint32_t dst = ring0 + n % kStages * kStage, bar = full(n % kStages);
        if (lane == 0) mbar_expect_tx(bar, kStage);
        __syncwarp();
        if (lane < 3) bulk_load(dst + lane_dst, lane_src + long(block) * lane_block, kTile * lane_bytes, bar);
        else if (lane == 3) tma_load_3d(dst, &p.tm_v, bar, 0, 0, block);
        __syncwarp();
        ++ic.t;
      };
      // a tile's products: the offset over all columns, then two steps per group
      const uint64_t qd = sdesc_sw128(qt, 16, 1024), qo = sdesc_sw32(qt + kQOffset, 256);
      const uint32_t qd_lo = uint32_t(qd), qd_hi = uint32_t(qd >> 32);
      auto products = [&]() {
        tc_fence_after();
        tc_mma_ts(tmem + kColD, tmem + kColOne, qo, idesc_f32acc(128, kCols, 0, 0, 0), 0u);
        product_steps<0>(tmem, qd_lo, qd_hi);
        tc_commit(mma_done);
      };
      int copied = 0, done = 0;
      bool ok = true;
      for (; copied < n_all && copied < kStages; ++copied) copy(copied);
      for (; done < n_all && ok; ++done) {
        if (!(ok = wait_w(a_ready, done & 1))) break;
        if (elect_one()) products();
        __syncwarp();
        // the stage of tile done - 2 is read: its next copy
        if (done >= 2 && copied < n_all) {
          if (!(ok = wait_w(empty(copied % kStages), (copied / kStages - 1) & 1))) break;
          copy(copied++);
        }
      }
      if (!ok && elect_one()) {
        // a wait ran out: the copies and products under way end before the block does
        int dummy = 0;
        for (int i = copied > kStages ? copied - kStages : 0; i < copied; ++i)
          mbar_wait(full(i % kStages), (i / kStages) & 1, &dummy, nullptr, 0, 50000000ull);
        tc_commit(mma_done);
        for (int i = 0; i < 2; ++i) mbar_wait(mma_done, (done + i) & 1, &dummy, nullptr, 0, 50000000ull);
      }
    }
    tc_fence_before();
    __syncthreads();
    return;
  }
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsWork));
  TileCursor c;
  if (n_all > 0) c = cursor_at(tbl, p.batch, p.hkv, a);

  // the constant row of A: 2^-14 (times the offset operand's -8 sum / 2^8 / ... : int4.cuh)
  if (n_all > 0) {
    uint32_t one[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) one[i] = 0x04000400u;
    tmem_st8(t_lane + kColOne, one);
    tmem_wait_st();
    if (NB == 1) {  // heads 8..15 of the P rows: none
      const uint32_t z[4] = {0, 0, 0, 0};
      sts128(pt + lane * kPRow + 16, z);
    }
  }

  // Key of this thread, unpacked into its row of A.
  auto unpack = [&](uint32_t stage) {
    uint32_t W[24];
    const uint32_t ka = stage + kOffK + (gw * 32 + lane) * kI4KCodes;
#pragma unroll
    for (int i = 0; i < 6; ++i) lds128(ka + 16 * i, W + 4 * i);
#pragma unroll
    for (int j = 0; j < kI4KGroups; ++j) {
      uint32_t r[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t x = W[6 * q + j], y = x >> 8;
        r[4 * q] = x & kI4Lo;
        r[4 * q + 1] = x & kI4Hi;
        r[4 * q + 2] = y & kI4Lo;
        r[4 * q + 3] = y & kI4Hi;
      }
      tmem_st16(t_lane + kColA + 16 * j, r);
    }
    tmem_wait_st();
  };
  // ... and hands it to the issuing warp, the sums of the tile before read
  auto hand_over = [&]() {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(a_ready);
  };

  const float c_log2 = p.scale_log2 * kI4KeyUnit;
  const uint64_t c2 = pack_f32x2(c_log2, c_log2);
  uint32_t flip;
  asm volatile("mov.b32 %0, 0xFFFF0000;" : "=r"(flip));  // (opaque, or it is folded into a second instruction)
  const uint32_t sign = (lane & 1) ? 0x80008000u : 0u;  // odd keys enter as -p * (15 - code)
  uint32_t tb[kI4VGroups];  // (-8, -7) in the columns of group u, else 0
#pragma unroll
  for (int u = 0; u < kI4VGroups; ++u) tb[u] = (r0 & 3) == u ? 0xC700C800u : 0u;

  int st = 0, ph = 0;
  bool ok = true;
  for (int x = 0; x < n_all && ok;) {
    if (c.t == c.nt) next_unit(tbl, p.hkv, c);
    const int s = c.s, g = c.g, t_first = c.t;
    const int t_end = min(c.nt, c.t + (n_all - x));
    const int ctx = p.seq_lens[s];
    const Span U = span_of(p, ctx);
    // ---- the unit's query operand: 8 threads per head, thread r of them dims 4 r .. 4 r + 3, their
    // rotary partners 32 + 4 r .., and 64 + 16 r .. 64 + 16 r + 15
    {
      const int h = (threadIdx.x & 127) >> 3, r = lane & 7;
      float cs, sn;
      rope_cos_sin(p.positions ? p.positions[s] : ctx - 1, p.rope.inv_freq[lane], &cs, &sn);
      const uint16_t* row = p.q + (long(s) * kHq + g * G + h) * kDqk;
      uint2 ra = make_uint2(0, 0), rb = ra;
      uint4 rc[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (NB == 2 || h < 8) {
        ra = __ldg(reinterpret_cast<const uint2*>(row + 4 * r));
        rb = __ldg(reinterpret_cast<const uint2*>(row + 32 + 4 * r));
        rc[0] = __ldg(reinterpret_cast<const uint4*>(row + 64 + 16 * r));
        rc[1] = __ldg(reinterpret_cast<const uint4*>(row + 64 + 16 * r) + 1);
      }
      float v[24];
      {
        const uint32_t wa[2] = {ra.x, ra.y}, wb[2] = {rb.x, rb.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float xa = (i & 1) ? hi_bf16(wa[i >> 1]) : lo_bf16(wa[i >> 1]);
          const float xb = (i & 1) ? hi_bf16(wb[i >> 1]) : lo_bf16(wb[i >> 1]);
          const float ci = __shfl_sync(0xffffffffu, cs, 4 * r + i), si = __shfl_sync(0xffffffffu, sn, 4 * r + i);
          v[i] = xa * ci - xb * si;
          v[4 + i] = xb * ci + xa * si;
        }
        const uint32_t wc[8] = {rc[0].x, rc[0].y, rc[0].z, rc[0].w, rc[1].x, rc[1].y, rc[1].z, rc[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[8 + 2 * i] = lo_bf16(wc[i]);
          v[9 + 2 * i] = hi_bf16(wc[i]);
        }
      }
      // element k (the position of a dim) of row `row` of the operand part at `at`
      auto elem = [&](int at, int row, int k) {
        return qt + at + row * 128 + ((((k & 63) >> 3) ^ (row & 7)) << 4) + (k & 7) * 2;
      };
      // the offset rows: 4096 bytes of zeros, 32 a thread
      const uint32_t zero[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 2; ++i) sts128(qt + kQOffset + (threadIdx.x & 127) * 32 + 16 * i, zero);
      float amax = 0.f, s0 = 0.f, s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < 24; i += 2) {
        // dims d and d + 1: an even and an odd field (* 4, / 4)
        const int d = i < 4 ? 4 * r + i : (i < 8 ? 32 + 4 * r + i - 4 : 64 + 16 * r + i - 8);
        const uint32_t hw = pack2_f16_sat(v[i] * 4.f, v[i + 1] * 0.25f, amax);
        // k of dim d: fields come out of a word as (0, 4), (1, 5), (2, 6), (3, 7)
        const int k0 = (d & ~7) + 2 * (d & 3) + ((d >> 2) & 1), k1 = k0 + 2;
        const int at = i < 8 ? 0 : (r < 4 ? kQOff1 : kQOff2);
        sts16(elem(at, h, k0), uint16_t(hw));
        sts16(elem(at, h, k1), uint16_t(hw >> 16));
        if (i < 8) {
          const float2 t = f32x2_of_f16x2(hw);
          const uint32_t lw = f16x2_of(v[i] * 4.f - t.x, v[i + 1] * 0.25f - t.y);
          sts16(elem(0, 16 + h, k0), uint16_t(lw));
          sts16(elem(0, 16 + h, k1), uint16_t(lw >> 16));
        }
        (i < 4 ? s0 : (i < 8 ? s1 : s2)) += v[i] + v[i + 1];
      }
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        s0 += __shfl_xor_sync(0xffffffffu, s0, d);
        s1 += __shfl_xor_sync(0xffffffffu, s1, d);
        if (d == 1) s2 += __shfl_xor_sync(0xffffffffu, s2, d);
      }
      group_sync();  // (the zeros are written)
      auto offset = [&](int j, float sum) {
        // -8 sum in the sums' unit 2^-22, over the constant 2^-14: elements 0 and 1 of the column's row
        const float o = sum * -0.03125f;
        const uint32_t hi = f16x2_of(o, 0.f), lo = f16x2_of(o - f32x2_of_f16x2(hi).x, 0.f);
        const int row = col_of(j) + h;
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(qt + kQOffset + row * 32 + (((row >> 2) & 1) << 4)), "r"(hi | (lo << 16))
                     : "memory");
      };
      if (r == 0) offset(0, s0);
      if (r == 1) offset(1, s1);
      if ((r & 1) == 0) offset(2 + (r >> 1), s2);
      if (amax > kF16Max) atomicOr(p.status, MIMO_STATUS_RANGE);
      fence_proxy_async_smem();
    }
    group_sync();  // every warp's part of the operand is written
    bool good = wait_w(full(st), ph & 1);
    if (good) {
      unpack(ring0 + st * kStage);
      hand_over();
    }
    uint64_t nref[H2];    // minus this warp's references, alike in all lanes
    uint64_t l2[H2];      // this thread's sums, heads 2 i and 2 i + 1
    float o[kI4VGroups][4][4], T[4] = {0.f, 0.f, 0.f, 0.f};  // T: column n holds group n % 4's offset
#pragma unroll
    for (int i = 0; i < H2; ++i) {
      nref[i] = pack_f32x2(INFINITY, INFINITY);
      l2[i] = 0;
    }
#pragma unroll
    for (int u = 0; u < kI4VGroups; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[u][e][0] = o[u][e][1] = o[u][e][2] = o[u][e][3] = 0.f;

    for (; c.t < t_end && good; ++c.t, ++x) {
      const uint32_t stage = ring0 + st * kStage;
      const int key0 = (U.t0 + c.t) * kTile + gw * 32;  // this warp's keys
      const bool live = key0 <= U.hi && key0 + 31 >= U.lo;
      const bool edge = key0 < U.lo || key0 + 31 > U.hi;
      if (!(good = wait_w(mma_done, x & 1))) break;
      tc_fence_after();
      // ---- logits of this thread's key
      uint64_t S[H2];
#pragma unroll
      for (int i = 0; i < H2; ++i) S[i] = 0;
      if (live) {
        uint32_t z[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) z[i] = lds32(stage + kOffKs + (gw * 32 + lane) * 2 * kI4KGroups + 4 * i);
        // two blocks of columns at a time: both terms of group 0, of group 1, then groups 2..5
#pragma unroll
        for (int b2 = 0; b2 < 4; ++b2) {
          uint32_t d[2][16];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if constexpr (NB == 2) tmem_ld16(t_lane + kColD + 32 * b2 + 16 * i, d[i]);
            else tmem_ld8(t_lane + kColD + 32 * b2 + 16 * i, d[i]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if constexpr (NB == 2) tmem_wait_ld_r16(d[i]);
            else tmem_wait_ld_r8(d[i]);
            const int j = b2 < 2 ? b2 : 2 * b2 - 2 + i;
            const float2 zz = f32x2_of_f16x2(z[j >> 1]);
            const float sc = (j & 1) ? zz.y : zz.x;
            const uint64_t s2 = pack_f32x2(sc, sc);
#pragma unroll
            for (int e = 0; e < H2; ++e)
              S[e] = fma_f32x2(pack_f32x2(__uint_as_float(d[i][2 * e]), __uint_as_float(d[i][2 * e + 1])), s2, S[e]);
          }
        }
      }
      // ---- the next tile's keys: its products run behind this tile's softmax
      int nst = st + 1, nph = ph;
      if (nst == kStages) nst = 0, ++nph;
      if (c.t + 1 < t_end) {
        if (!(good = wait_w(full(nst), nph & 1))) break;
        unpack(ring0 + nst * kStage);
        hand_over();
      }
      if (live) {
        // ---- weights
        const bool valid = key0 + lane >= U.lo && key0 + lane <= U.hi;
        float xs[G];
        float top = -INFINITY;
        auto logits = [&]() {
          top = -INFINITY;
#pragma unroll
          for (int i = 0; i < H2; ++i) {
            const uint64_t v = fma_f32x2(S[i], c2, nref[i]);
            xs[2 * i] = lo_f32(v);
            xs[2 * i + 1] = hi_f32(v);
          }
          if (edge && !valid) {
#pragma unroll
            for (int i = 0; i < G; ++i) xs[i] = -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < G; ++i) top = fmaxf(top, xs[i]);
        };
        logits();
        if (__any_sync(0xffffffffu, top > kSlack)) {
          // move the references that were passed to their new maxima, and the sums with them
          float al[G];
#pragma unroll
          for (int i = 0; i < G; ++i) {
            float z = ((i & 1) ? hi_f32(S[i >> 1]) : lo_f32(S[i >> 1])) * c_log2;
            if (edge && !valid) z = -INFINITY;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, d));
            const float ref = -((i & 1) ? hi_f32(nref[i >> 1]) : lo_f32(nref[i >> 1]));
            const bool up = z > ref + kSlack;
            al[i] = up ? ex2(ref - z) : 1.f;  // (from -inf: 0, of sums that are 0)
            const float now = up ? -z : -ref;
            nref[i >> 1] = (i & 1) ? pack_f32x2(lo_f32(nref[i >> 1]), now) : pack_f32x2(now, hi_f32(nref[i >> 1]));
          }
          float* const ax = xch + gw * 32;
          if (lane == 0)
#pragma unroll
            for (int i = 0; i < G; ++i) ax[i] = al[i];
          __syncwarp();
          const float a0 = ax[r0], a1 = NB == 2 ? ax[8 + r0] : 0.f;
          __syncwarp();
#pragma unroll
          for (int i = 0; i < H2; ++i) l2[i] = mul_f32x2(l2[i], pack_f32x2(al[2 * i], al[2 * i + 1]));
#pragma unroll
          for (int u = 0; u < kI4VGroups; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[u][e][0] *= a0;
              o[u][e][1] *= a0;
              o[u][e][2] *= a1;
              o[u][e][3] *= a1;
            }
          T[0] *= a0;
          T[1] *= a0;
          T[2] *= a1;
          T[3] *= a1;
          logits();
        }
        uint32_t pk[H2];
#pragma unroll
        for (int i = 0; i < H2; ++i) {
          const float p0 = ex2(xs[2 * i]), p1 = ex2(xs[2 * i + 1]);
          l2[i] = add_f32x2(l2[i], pack_f32x2(p0, p1));
          pk[i] = f16x2_of(p0, p1) ^ sign;
        }
        sts128(pt + lane * kPRow, pk);
        if constexpr (NB == 2) sts128(pt + lane * kPRow + 16, pk + 4);
        __syncwarp();
        // ---- O += P V over this warp's 32 keys
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          uint32_t P[4];
          ldsm_x4_t(pt + (16 * kk + (lane >> 4) * 8 + (lane & 7)) * kPRow + ((lane >> 3) & 1) * 16, P);
          // value scales of keys 2 q4, 2 q4 + 1 of either 8: [group] fp16 pairs.  A slot nothing was
          // written to may hold any scale: it counts as 0
          uint32_t vs[2][kI4VGroups];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t h[4];
            const int k8 = 16 * kk + 8 * e + 2 * q4;
            lds128(stage + kOffVs + (gw * 32 + k8) * 2 * kI4VGroups, h);
            vs[e][0] = __byte_perm(h[0], h[2], 0x5410);
            vs[e][1] = __byte_perm(h[0], h[2], 0x7632);
            vs[e][2] = __byte_perm(h[1], h[3], 0x5410);
            vs[e][3] = __byte_perm(h[1], h[3], 0x7632);
            if (edge) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (key0 + k8 + i > U.hi)
#pragma unroll
                  for (int u = 0; u < kI4VGroups; ++u) vs[e][u] &= i ? 0x0000FFFFu : 0xFFFF0000u;
            }
          }
          const int row = gw * 32 + 16 * kk + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
          for (int up = 0; up < 2; ++up) {
            uint32_t m[4];
            ldsm_x4_t(stage + row * kI4VCodes + (((2 * up + (lane >> 4)) ^ ((row >> 1) & 3)) << 4), m);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int u = 2 * up + h;
              uint32_t pa[4];
              pa[0] = hmul2(P[0], vs[0][u]);
              pa[1] = hmul2(P[1], vs[0][u]);
              pa[2] = hmul2(P[2], vs[1][u]);
              pa[3] = hmul2(P[3], vs[1][u]);
              const uint32_t x0 = m[2 * h], x1 = m[2 * h + 1], y0 = x0 >> 8, y1 = x1 >> 8;
              // (the odd key's codes complemented)
              mma_f16_acc(o[u][0], pa, field(x0, flip, kI4Lo), field(x1, flip, kI4Lo));
              mma_f16_acc(o[u][1], pa, field(x0, flip, kI4Hi), field(x1, flip, kI4Hi));
              mma_f16_acc(o[u][2], pa, field(y0, flip, kI4Lo), field(y1, flip, kI4Lo));
              mma_f16_acc(o[u][3], pa, field(y0, flip, kI4Hi), field(y1, flip, kI4Hi));
              // p (n - 8) = p n - 8 p for the even key, -p (15 - n) + 7 p for the odd one
              mma_f16_acc(T, pa, tb[u], tb[u]);
            }
          }
        }
      }
      __syncwarp();  // (P is read before the next tile writes it)
      if (lane == 0) mbar_arrive(empty(st));
      st = nst;
      ph = nph;
    }
    // a warp whose wait ran out takes the group with it here
    if (!(ok = group_sync_ok(good))) break;

    // ---- the segment's rows: the four warps' sums against the largest of their references
    {
      float* const ax = xch + gw * 32;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        float v = (i & 1) ? hi_f32(l2[i >> 1]) : lo_f32(l2[i >> 1]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (lane == 0) {
          ax[i] = -((i & 1) ? hi_f32(nref[i >> 1]) : lo_f32(nref[i >> 1]));
          ax[16 + i] = v;
        }
      }
    }
    group_sync();
    float M[2], L[2], fac[2];  // heads r0 and 8 + r0
#pragma unroll
    for (int hf = 0; hf < NB; ++hf) {
      const int h = r0 + 8 * hf;
      M[hf] = fmaxf(fmaxf(xch[h], xch[32 + h]), fmaxf(xch[64 + h], xch[96 + h]));
      L[hf] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float rf = xch[32 * i + h], f = rf == -INFINITY ? 0.f : ex2(rf - M[hf]);
        L[hf] += f * xch[32 * i + 16 + h];
        if (i == gw) fac[hf] = f;
      }
    }
    const bool direct = t_first == 0 && c.t == c.nt;
    const long piece = 2L * w + (x > c.t - t_first ? 1 : 0);  // this worker's first or last segment
    // 2 KB blocks of the group's query operand and P rows (both free now): [warp][group of a round]
    auto block = [&](int i) {
      return reinterpret_cast<float4*>(i < 6 ? smem + grp * kQBytes + 2048 * i
                                             : smem + kOffP + grp * 4 * kPBytes + 2048 * (i - 6));
    };
    static_assert(4 * kPBytes >= 2 * 2048 && kQBytes >= 6 * 2048, "merge room");
#pragma unroll
    for (int round = 0; round < 2; ++round) {
#pragma unroll
      for (int ur = 0; ur < 2; ++ur) {
        const int u = 2 * round + ur;
        float4* const dst = block(gw * 2 + ur);
#pragma unroll
        for (int hf = 0; hf < NB; ++hf) {
          // T's columns 0..3 are in lanes 0 and 1 of the quad
          const float t = __shfl_sync(0xffffffffu, T[2 * hf + (u & 1)], (lane & ~3) + (u >> 1));
          float f[8];  // dims 32 u + 8 q4 + i of head r0 + 8 hf
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = fmaf(o[u][i & 3][2 * hf + (i >> 2)], (i & 1) ? 0x1p20f : 0x1p24f, t) * fac[hf];
          dst[(2 * hf) * 32 + lane] = make_float4(f[0], f[1], f[2], f[3]);
          dst[(2 * hf + 1) * 32 + lane] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
      group_sync();
      if ((gw >> 1) == round) {
        const int u = gw;
#pragma unroll
        for (int hf = 0; hf < NB; ++hf) {
          float4 v[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 t = block(2 * i + (gw & 1))[(2 * hf + e) * 32 + lane];
              v[e].x += t.x;
              v[e].y += t.y;
              v[e].z += t.z;
              v[e].w += t.w;
            }
          }
          const int rr = r0 + 8 * hf, h = g * G + rr, dim = 32 * u + 8 * q4;
          if (direct) {
            float M2 = M[hf], L2 = L[hf], f = 1.f;
            if (p.sink) {
              const float sl = p.sink[h] * kLog2e;
              M2 = fmaxf(M[hf], sl);
              f = ex2(M[hf] - M2);
              L2 = L[hf] * f + ex2(sl - M2);
            }
            const float sc = p.v_scale * f / L2;
            if (p.lse && u == 0 && q4 == 0) p.lse[long(s) * kHq + h] = (M2 + log2f(L2)) * kLn2;
            *reinterpret_cast<uint4*>(p.out + (long(s) * kHq + h) * kDv + dim) =
                make_uint4(pack2_bf16(v[0].x * sc, v[0].y * sc), pack2_bf16(v[0].z * sc, v[0].w * sc),
                           pack2_bf16(v[1].x * sc, v[1].y * sc), pack2_bf16(v[1].z * sc, v[1].w * sc));
          } else {
            if (u == 0 && q4 == 0) *reinterpret_cast<float2*>(p.ws_ml + (piece * 16 + rr) * 2) = make_float2(M[hf], L[hf]);
            float4* dst = reinterpret_cast<float4*>(p.ws_o + (piece * 16 + rr) * kDv + dim);
            dst[0] = v[0];
            dst[1] = v[1];
          }
        }
      }
      group_sync();
    }
    if (NB == 1) {  // the merge used the P rows: heads 8..15 are none again
      const uint32_t z[4] = {0, 0, 0, 0};
      sts128(pt + lane * kPRow + 16, z);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, 512);
  }
}

cudaError_t launch_decode4_tc(const Decode4Params& p, int sms, cudaStream_t s) {
  auto kernel = p.hkv == 8 ? decode4_tc_kernel<1> : decode4_tc_kernel<2>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  kernel<<<p.workers < sms ? p.workers : sms, kThreads, kSmem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace mimo
