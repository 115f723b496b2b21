// Decode and draft verification (1..8 query tokens per sequence) over a 4-bit ring: the attention
// of decode.cu on the cache format of int4.cuh.  Also the host side of decode_int4_tc.cu, which
// takes the paged caches: its tile is 128 keys, and a ring of 128 to 512 slots is one to four of
// those, a new query operand and an emptied pipeline before each ring.
//
// 180 bytes per (key, KV head) stand against 16 x 320 multiply-adds a draft (57 FLOP per byte),
// and every element has to be unpacked first: unlike the wide caches this one is bound by
// instruction issue and mma.sync, and the kernel is laid out to spend as few instructions per
// element as it can:
//   - unpacking is one shift and four ANDs per 8 elements (int4.cuh); the key offset is one
//     product per 8 keys, and a group's scale multiplies its 16 x 8 products in fp32, not its
//     32 x 8 elements;
//   - a value's scale is moved into the probabilities (fp16 pairs), its transposed fragments
//     come from ldmatrix.trans: a 16-bit element of the transposed matrix is 4 dims of a key,
//     so a register is 4 dims of a key pair, ready for the same masks;
//   - the value offset is one more product per group of dims, p against a constant in the
//     columns of that group (the groups share an accumulator).  Codes are never negative, so a sum of
//     p * code over a ring's keys would be 8 times the weights' sum whatever the result, and the
//     accumulator's rounding be relative to that; so the odd key of each pair enters as
//     -p * (15 - code) (the complement is free in the mask's LOP3) and the sum stays near zero;
//   - the rotated query dims enter as two fp16 terms: no 16-bit type holds them to the digits of
//     an fp32 log-sum-exp.
//
// Workers are groups of nc warps (one per 16-row block of query rows, sharing the tiles of 32
// keys), each of which takes whole (sequence, KV head) units and writes their rows; where that
// leaves half of the warps without a unit, two of them share one and add up their halves in shared
// memory (64 rings of 144 slots and 8 KV heads: 18.5 -> 16.5 us).  Each group's
// leader warp issues the copies of later tiles itself (one bulk copy for the codes and for the
// scales, one TMA tile with the 64-byte swizzle for the values); there are no producer warps, so
// all 8 warps multiply.
//
// 64 rings of 144 slots and 8 heads: 16.5 us, against 2.4 for the bytes.  Bound by latency: 1.8 warps
// a scheduler, which issue in a third of the cycles (tensor pipe 13 %, ALU 26 %), walk a ring's five
// tiles as two chains of dependent products.
#include <cuda_bf16.h>

#include "common.cuh"
#include "int4.cuh"
#include "ptx.cuh"
#include "tiles.cuh"
#include "../../include/mimoattn.h"

namespace mimo {

namespace {

constexpr int kWarps = 8;
constexpr int kTile = kI4Tile;
// stage: value codes (64-byte swizzle), key codes, key scales, value scales
constexpr int kOffK = kTile * kI4VCodes, kOffKs = kOffK + kTile * kI4KCodes;
constexpr int kOffVs = kOffKs + kTile * 2 * kI4KGroups;
constexpr int kStage = 6144;
static_assert(kOffVs + kTile * 2 * kI4VGroups <= kStage && kStage % 1024 == 0, "stage layout");
constexpr int kAllStages = 24;
constexpr int kOffRest = kAllStages * kStage;  // a warp's second terms of the rotated dims: 4 steps x 512 bytes
constexpr int kOffPair = kOffRest + kWarps * 2048;  // a split unit's second half: 72 floats a lane
constexpr int kOffBar = kOffPair + kWarps / 2 * 72 * 32 * 4;
constexpr int kOffTbl = kOffBar + 2 * kAllStages * 8 + 16;
constexpr int kSmem = kOffTbl + (kMaxTableBatch + 1) * 8 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// probabilities are kept as 2^kPBias * p: products with small value scales stay clear of
// fp16's subnormals (and 2^6 * 1023, the largest scale an append stores, below its limit)
constexpr float kPBias = 6.f;

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void lds64(uint32_t addr, uint32_t& a, uint32_t& b) {
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr));
}
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t* r) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t a;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(a) : "r"(addr));
  return a;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t* r) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// two floats -> fp16x2, one instruction
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

}  // namespace

__global__ void __launch_bounds__(kWarps * 32, 1) decode4_kernel(const __grid_constant__ Decode4Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nc = p.nc, stages = p.stages;
  const int grp = warp / nc, blk = warp - grp * nc;
  const uint32_t ring0 = sbase + grp * stages * kStage;
  const uint32_t bar0 = sbase + kOffBar + grp * stages * 16;
  auto full = [&](int i) { return bar0 + 16 * i; };
  auto empty = [&](int i) { return bar0 + 16 * i + 8; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + 2 * kAllStages * 8);
  long long* tbl = reinterpret_cast<long long*>(smem + kOffTbl);
  if (grp < p.groups && blk == 0 && lane == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), nc);
    }
    if (grp == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarps - 1) {
    const int ring_tiles = (p.ring_slots + kTile - 1) / kTile;
    tile_table(tbl, p.batch, lane, [&](int s) {
      const int ctx = p.seq_lens[s];
      if (blockIdx.x == 0 && (ctx < p.q_len || ctx > p.max_seq_len)) atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
      return ctx < p.q_len ? 0 : ring_tiles;
    });
  }
  __syncthreads();
  if (grp >= p.groups) return;
  const long long total = tbl[p.batch] * p.hkv;
  if (total == 0) return;
  // split: a pair of groups (of one warp) shares its units, each takes half of a unit's tiles
  const int split = p.split, half = split > 1 ? grp & 1 : 0;
  const int w = grp / split * gridDim.x + blockIdx.x;
  const int units = p.batch * p.hkv, W = min(units, p.workers);
  if (w >= W) return;
  auto at = [&](int u) {
    const int s = u / p.hkv;
    return s >= p.batch ? total : tbl[s] * p.hkv + (u - s * p.hkv) * (tbl[s + 1] - tbl[s]);
  };
  const long long a = at(w * units / W), b = at((w + 1) * units / W);
  if (a >= b) return;

  const bool leader = blk == 0;
  const int slots = p.ring_slots;  // of a block
  auto wait_w = [&](uint32_t bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;  // (a branch of the whole warp)
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, MIMO_STATUS_TIMEOUT));
  };

  const int tiles = (slots + kTile - 1) / kTile, n_units = int(b - a) / tiles;  // (every unit that has tiles has as many)
  const int t_lo = half ? (tiles + 1) / 2 : 0, t_hi = split > 1 && !half ? (tiles + 1) / 2 : tiles;

  // ---- the leader's side: copies of the units' tiles t_lo .. t_hi - 1 in order
  const TileCursor start = cursor_at(tbl, p.batch, p.hkv, a);
  TileCursor ic = start;
  ic.t = t_lo;
  int left = n_units * (t_hi - t_lo);
  int ist = 0, iph = 0;         // stage and pass of the next copy
  // what lanes 0..3 copy: key codes, key scales, value scales (bulk copies), value codes (a TMA tile)
  const int lane_bytes = lane == 0 ? kI4KCodes : (lane == 1 ? 2 * kI4KGroups : 2 * kI4VGroups);
  const uint32_t lane_dst = lane == 0 ? kOffK : (lane == 1 ? kOffKs : kOffVs);
  const int lane_block = slots * (lane < 2 ? kI4KSlot : kI4VSlot);
  const uint8_t* const lane_src =
      lane == 0 ? p.k_cache : (lane == 1 ? p.k_cache + slots * kI4KCodes : p.v_cache + slots * kI4VCodes);
  auto issue = [&]() -> bool {
    if (left == 0) return true;
    --left;
    if (ic.t == t_hi) {
      next_unit(tbl, p.hkv, ic);
      ic.t = t_lo;
    }
    const int block = int(p.block0) + ic.s * p.hkv + ic.g, slot = ic.t * kTile;
    if (nc > 1 && iph > 0 && !wait_w(empty(ist), (iph - 1) & 1)) return false;
    const int n = min(kTile, slots - slot);
    const uint32_t dst = ring0 + ist * kStage, bar = full(ist);
    if (lane == 0) mbar_expect_tx(bar, n * (kI4KSlot + 2 * kI4VGroups) + kTile * kI4VCodes);
    __syncwarp();
    if (lane < 3) bulk_load(dst + lane_dst, lane_src + (long(block) * lane_block + slot * lane_bytes), n * lane_bytes, bar);
    else if (lane == 3) tma_load_3d(dst, &p.tm_v, bar, 0, slot, block);
    __syncwarp();
    ++ic.t;
    if (++ist == stages) ist = 0, ++iph;
    return true;
  };
  // before the group leaves on a failed wait: let the copies under way land
  auto drain = [&]() {
    if (!leader || lane != 0) return;
    int dummy = 0, st = ist, ph = iph;
    for (int i = 0; i < stages && (ph > 0 || st > 0); ++i) {
      if (--st < 0) st = stages - 1, --ph;
      mbar_wait(full(st), ph & 1, &dummy, nullptr, 0, 50000000ull);
    }
  };
  bool ok = true;
  if (leader)
    for (int i = 0; i < stages && ok; ++i) ok = issue();

  // ---- every warp's side
  const int q4 = lane & 3, r0 = lane >> 2;
  const uint32_t rest0 = sbase + kOffRest + warp * 2048 + lane * 16;
  const int G = p.group;
  int st = 0, ph = 0;
  bool behind = false;  // nc > 1: a stage was released but its next copy is not issued yet
  TileCursor c = start;
  for (int u = 0; u < n_units && (ok || split > 1); ++u) {  // (a pair meets once a unit, whatever became of its waits)
    if (u) next_unit(tbl, p.hkv, c);
    const int s = c.s, g = c.g;
    const int ctx = p.seq_lens[s];
    // rows r0 and r0 + 8 of the block: row 16 blk + r is draft (16 blk + r) / G
    int lo_r[2], hi_r[2], draft[2];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      draft[hf] = (blk * 16 + 8 * hf) / G;
      const int at = ctx - p.q_len + draft[hf];
      // (a padding row sees what the row before it sees: it calls for no mask of its own)
      const bool valid = draft[hf] < p.q_len;
      lo_r[hf] = valid ? (p.window > 0 ? max(0, at - p.window + 1) : 0) : lo_r[0];
      hi_r[hf] = valid ? at : hi_r[0];
    }
    // ---- query fragments (the second terms in shared memory), and those of the key offset's product
    uint32_t qa[2 * kI4KGroups][4];
    uint32_t off[4] = {0u, 0u, 0u, 0u};
    {
      float cs[2], sn[2];
      const int pos0 = ctx - p.q_len;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (hf == 0 || draft[1] != draft[0]) {
          rope_cos_sin(pos0 + draft[hf], p.rope.inv_freq[lane], &cs[hf], &sn[hf]);
        } else {
          cs[1] = cs[0];
          sn[1] = sn[0];
        }
      }
      uint4 raw[2][kI4KGroups];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int rr = blk * 16 + r0 + 8 * hf;
        const bool valid = draft[hf] < p.q_len;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + ((long(s) * p.q_len + (valid ? draft[hf] : 0)) * kHq + g * G + rr % G) * kDqk + 8 * q4);
#pragma unroll
        for (int j = 0; j < kI4KGroups; ++j) raw[hf][j] = valid ? __ldg(src + 4 * j) : make_uint4(0, 0, 0, 0);
      }
      float amax = 0.f;
      float v[2][2][8];  // [row][group 0 / 1][dim]
      auto widen = [](const uint4& r, float* f) {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = lo_bf16(u[i]);
          f[2 * i + 1] = hi_bf16(u[i]);
        }
      };
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        widen(raw[hf][0], v[hf][0]);
        widen(raw[hf][1], v[hf][1]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // dims 8 q4 + i and 32 + 8 q4 + i turn with frequency 8 q4 + i
          const float ci = __shfl_sync(0xffffffffu, cs[hf], 8 * q4 + i), si = __shfl_sync(0xffffffffu, sn[hf], 8 * q4 + i);
          const float xx = v[hf][0][i], yy = v[hf][1][i];
          v[hf][0][i] = xx * ci - yy * si;
          v[hf][1][i] = yy * ci + xx * si;
        }
      }
      auto group = [&](int j, const float* x0, const float* x1) {
        uint32_t rest[2][4];
        int4_query_group(x0, x1, qa + 2 * j, rest, amax);
        if (j < 2) {
          sts128(rest0 + 1024 * j, rest[0]);
          sts128(rest0 + 1024 * j + 512, rest[1]);
        }
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum[0] += x0[i];
          sum[1] += x1[i];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
          sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
        }
        int4_offset_group(off, j, q4, sum[0], sum[1]);
      };
      group(0, v[0][0], v[1][0]);
      group(1, v[0][1], v[1][1]);
#pragma unroll
      for (int j = 2; j < kI4KGroups; ++j) {
        widen(raw[0][j], v[0][0]);
        widen(raw[1][j], v[1][0]);
        group(j, v[0][0], v[1][0]);
      }
      if (amax > kF16Max) atomicOr(p.status, MIMO_STATUS_RANGE);
    }
    const float c_log2 = p.scale_log2 * kI4KeyUnit;
    const int R = p.ring_slots;
    const int ring_off = ((R - ctx) % R + R) % R;  // slot j holds position ctx - R + (j + ring_off) % R
    float m_r[2] = {-INFINITY, -INFINITY}, l_r[2] = {0.f, 0.f};
    float o[kI4VGroups][4][4], T[4] = {0.f, 0.f, 0.f, 0.f};  // T: column n holds group n % 4's offset
    uint32_t tb[kI4VGroups];  // (-8, -7) in the columns of group u, else 0
#pragma unroll
    for (int u = 0; u < kI4VGroups; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[u][e][0] = o[u][e][1] = o[u][e][2] = o[u][e][3] = 0.f;
      tb[u] = (r0 & 3) == u ? 0xC700C800u : 0u;
    }

    for (int t = t_lo; t < t_hi && ok; ++t) {
      if (!(ok = wait_w(full(st), ph & 1))) break;
      {
        const uint32_t vb = ring0 + st * kStage, kb = vb + kOffK, ksb = vb + kOffKs, vsb = vb + kOffVs;
        // ---- S = Q K^T, 8 keys at a time
        float S[4][4];
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          uint32_t kw[6], kh[6];
          const uint32_t ka = kb + (8 * nb + r0) * kI4KCodes + 24 * q4;
          const uint32_t sa = ksb + (8 * nb + 2 * q4) * 2 * kI4KGroups;  // keys 2 q4 and 2 q4 + 1
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            lds64(ka + 8 * i, kw[2 * i], kw[2 * i + 1]);
            lds64(sa + 8 * i, kh[2 * i], kh[2 * i + 1]);
          }
          // groups 2 q4, 2 q4 + 1 of key r0 (lane 3 of a quad: k 6, 7, which are none)
          uint32_t ob = lds32(ksb + (8 * nb + r0) * 2 * kI4KGroups + 4 * min(q4, 2));
          ob = q4 == 3 ? 0u : ob;
          mma_f16_c(S[nb], off, ob, ob, zero);
#pragma unroll
          for (int e = 0; e < 4; ++e) S[nb][e] *= kI4OffsetUnit;
#pragma unroll
          for (int j = 0; j < kI4KGroups; ++j) {
            const uint32_t wd = kw[j], w8 = wd >> 8;
            const uint32_t f0 = wd & kI4Lo, f1 = wd & kI4Hi, f2 = w8 & kI4Lo, f3 = w8 & kI4Hi;
            float d[4];
            mma_f16_c(d, qa[2 * j], f0, f1, zero);
            mma_f16_c(d, qa[2 * j + 1], f2, f3, d);
            if (j < 2) {
              uint32_t rest[4];
              lds128(rest0 + 1024 * j, rest);
              mma_f16_c(d, rest, f0, f1, d);
              lds128(rest0 + 1024 * j + 512, rest);
              mma_f16_c(d, rest, f2, f3, d);
            }
            const float2 sA = f32x2_of_f16x2(kh[j >> 1]), sB = f32x2_of_f16x2(kh[3 + (j >> 1)]);
            const float s0 = (j & 1) ? sA.y : sA.x, s1 = (j & 1) ? sB.y : sB.x;
            S[nb][0] = fmaf(d[0], s0, S[nb][0]);
            S[nb][1] = fmaf(d[1], s1, S[nb][1]);
            S[nb][2] = fmaf(d[2], s0, S[nb][2]);
            S[nb][3] = fmaf(d[3], s1, S[nb][3]);
          }
        }
        // ---- value scales of keys 2 q4, 2 q4 + 1 of each 8: [group] fp16 pairs (even, odd key)
        uint32_t vs[4][kI4VGroups];
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          uint32_t h[4];
          lds128(vsb + (8 * nb + 2 * q4) * 2 * kI4VGroups, h);
          vs[nb][0] = __byte_perm(h[0], h[2], 0x5410);
          vs[nb][1] = __byte_perm(h[0], h[2], 0x7632);
          vs[nb][2] = __byte_perm(h[1], h[3], 0x5410);
          vs[nb][3] = __byte_perm(h[1], h[3], 0x7632);
        }
        // ---- masks.  A slot nothing was written to may hold any scale: it counts as 0
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at = t * kTile + 8 * nb + 2 * q4 + e, j = at + ring_off;
            const int kp = at < R ? ctx - R + (j >= R ? j - R : j) : -1;
            if (kp < 0)
#pragma unroll
              for (int u = 0; u < kI4VGroups; ++u) vs[nb][u] &= e ? 0x0000FFFFu : 0xFFFF0000u;
            if (!(kp >= lo_r[0] && kp <= hi_r[0])) S[nb][e] = -INFINITY;
            if (!(kp >= lo_r[1] && kp <= hi_r[1])) S[nb][2 + e] = -INFINITY;
          }
        // ---- running maximum and sum
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          mx[0] = fmaxf(mx[0], fmaxf(S[nb][0], S[nb][1]));
          mx[1] = fmaxf(mx[1], fmaxf(S[nb][2], S[nb][3]));
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 1));
          mx[hf] = fmaxf(mx[hf], __shfl_xor_sync(0xffffffffu, mx[hf], 2));
          mx[hf] = fmaxf(m_r[hf], mx[hf] * c_log2);
        }
        if (__any_sync(0xffffffffu, mx[0] > m_r[0] || mx[1] > m_r[1])) {
          // (a row that has seen no key yet: its sums are zero, whatever the factor)
          const float al0 = mx[0] == -INFINITY ? 1.f : ex2(m_r[0] - mx[0]);
          const float al1 = mx[1] == -INFINITY ? 1.f : ex2(m_r[1] - mx[1]);
          m_r[0] = mx[0];
          m_r[1] = mx[1];
          l_r[0] *= al0;
          l_r[1] *= al1;
#pragma unroll
          for (int u = 0; u < kI4VGroups; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[u][e][0] *= al0;
              o[u][e][1] *= al0;
              o[u][e][2] *= al1;
              o[u][e][3] *= al1;
            }
          T[0] *= al0;
          T[1] *= al0;
          T[2] *= al1;
          T[3] *= al1;
        }
        const float mu0 = m_r[0] == -INFINITY ? 0.f : m_r[0] - kPBias, mu1 = m_r[1] == -INFINITY ? 0.f : m_r[1] - kPBias;
        uint32_t P[4][2];  // (p of the even key, -p of the odd key) of rows r0, r0 + 8
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          const float a0 = ex2(fmaf(S[nb][0], c_log2, -mu0)), a1 = ex2(fmaf(S[nb][1], c_log2, -mu0));
          const float b0 = ex2(fmaf(S[nb][2], c_log2, -mu1)), b1 = ex2(fmaf(S[nb][3], c_log2, -mu1));
          l_r[0] += a0 + a1;
          l_r[1] += b0 + b1;
          P[nb][0] = f16x2_of(a0, -a1);
          P[nb][1] = f16x2_of(b0, -b1);
        }
        // ---- O += P V, 16 keys at a time
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const int row = 16 * kk + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
          for (int up = 0; up < 2; ++up) {
            uint32_t m[4];
            ldsm_x4_t(vb + row * kI4VCodes + (((2 * up + (lane >> 4)) ^ ((row >> 1) & 3)) << 4), m);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int u = 2 * up + h;
              uint32_t pa[4];
              pa[0] = hmul2(P[2 * kk][0], vs[2 * kk][u]);
              pa[1] = hmul2(P[2 * kk][1], vs[2 * kk][u]);
              pa[2] = hmul2(P[2 * kk + 1][0], vs[2 * kk + 1][u]);
              pa[3] = hmul2(P[2 * kk + 1][1], vs[2 * kk + 1][u]);
              const uint32_t x0 = m[2 * h], x1 = m[2 * h + 1], y0 = x0 >> 8, y1 = x1 >> 8;
              constexpr uint32_t cl = 0x000F0000u, ch = 0x00F00000u;  // the odd key's complement
              mma_f16_c(o[u][0], pa, (x0 & kI4Lo) ^ cl, (x1 & kI4Lo) ^ cl, o[u][0]);
              mma_f16_c(o[u][1], pa, (x0 & kI4Hi) ^ ch, (x1 & kI4Hi) ^ ch, o[u][1]);
              mma_f16_c(o[u][2], pa, (y0 & kI4Lo) ^ cl, (y1 & kI4Lo) ^ cl, o[u][2]);
              mma_f16_c(o[u][3], pa, (y0 & kI4Hi) ^ ch, (y1 & kI4Hi) ^ ch, o[u][3]);
              // p (n - 8) = p n - 8 p for the even key, -p (15 - n) + 7 p for the odd one
              mma_f16_c(T, pa, tb[u], tb[u], T);
            }
          }
        }
      }
      // ---- release the stage; the leader refills the one before it (other warps may still read this one)
      __syncwarp();
      if (nc > 1) {
        if (lane == 0) mbar_arrive(empty(st));
        if (leader && behind && !(ok = issue())) break;
        behind = true;
      } else if (!(ok = issue())) {
        break;
      }
      if (++st == stages) st = 0, ++ph;
    }
    if (split > 1) {
      // the second half's sums join the first's, which writes the rows
      float* const ex = reinterpret_cast<float*>(smem + kOffPair) + (grp >> 1) * 72 * 32 + lane;
      auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + (grp >> 1)) : "memory"); };
      if (half) {
#pragma unroll
        for (int i = 0; i < 64; ++i) ex[32 * i] = o[i >> 4][(i >> 2) & 3][i & 3];
#pragma unroll
        for (int i = 0; i < 4; ++i) ex[32 * (64 + i)] = T[i];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ex[32 * (68 + i)] = m_r[i];
          ex[32 * (70 + i)] = l_r[i];
        }
      }
      meet();
      if (!half) {
        float f[2], e[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float m2 = ex[32 * (68 + i)], m = fmaxf(m_r[i], m2);
          f[i] = m_r[i] == -INFINITY ? 0.f : ex2(m_r[i] - m);
          e[i] = m2 == -INFINITY ? 0.f : ex2(m2 - m);
          m_r[i] = m;
          l_r[i] = l_r[i] * f[i] + ex[32 * (70 + i)] * e[i];
        }
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          float& v = o[i >> 4][(i >> 2) & 3][i & 3];
          v = v * f[(i >> 1) & 1] + ex[32 * i] * e[(i >> 1) & 1];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) T[i] = T[i] * f[i >> 1] + ex[32 * (64 + i)] * e[i >> 1];
      }
      meet();
      if (half) continue;
    } else if (!ok) {
      break;
    }

    // ---- the unit's rows
    float t_off[2][kI4VGroups];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      // columns 0..3 are in lanes 0 and 1 of the quad
#pragma unroll
      for (int u = 0; u < kI4VGroups; ++u) t_off[hf][u] = __shfl_sync(0xffffffffu, T[2 * hf + (u & 1)], (lane & ~3) + (u >> 1));
      l_r[hf] += __shfl_xor_sync(0xffffffffu, l_r[hf], 1);
      l_r[hf] += __shfl_xor_sync(0xffffffffu, l_r[hf], 2);
    }
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      if (draft[hf] >= p.q_len) continue;
      const int rr = blk * 16 + r0 + 8 * hf, h = g * G + rr % G;
      const long qrow = long(s) * p.q_len + draft[hf];
      const float M = m_r[hf] - kPBias, L = l_r[hf];
      float M2 = M, L2 = L, f = 1.f;
      if (p.sink) {
        const float sl = p.sink[h] * kLog2e;
        M2 = fmaxf(M, sl);
        f = ex2(M - M2);
        L2 = L * f + ex2(sl - M2);
      }
      const float sc = p.v_scale * f / L2;
      if (p.lse && q4 == 0) p.lse[qrow * kHq + h] = (M2 + log2f(L2)) * kLn2;
#pragma unroll
      for (int u = 0; u < kI4VGroups; ++u) {
        float f[8];  // dims 32 u + 8 q4 + i
#pragma unroll
        for (int i = 0; i < 8; ++i)
          f[i] = fmaf(o[u][i & 3][2 * hf + (i >> 2)], (i & 1) ? 0x1p20f : 0x1p24f, t_off[hf][u]) * sc;
        *reinterpret_cast<uint4*>(p.out + (qrow * kHq + h) * kDv + 32 * u + 8 * q4) =
            make_uint4(pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7]));
      }
    }
  }
  if (!ok) drain();
}

Decode4Plan decode4_plan(int batch, int hkv, int q_len, int unit_keys, bool ring, int sms) {
  Decode4Plan d;
  d.tc = !ring;
  d.tile = ring ? kI4Tile : kI4TcTile;
  d.n_blocks = (q_len * (kHq / hkv) + 15) / 16;
  d.nc = d.n_blocks;
  d.groups = ring ? kWarps / d.nc : (d.n_blocks == 1 ? 2 : 1);
  // Rings that leave half of the warps without one are split in two.
  d.split = ring && d.nc == 1 && (long long)batch * hkv * 2 <= (long long)sms * d.groups ? 2 : 1;
  d.stages = kAllStages / d.groups;
  const int tiles = (unit_keys + d.tile - 1) / d.tile + 1;  // a window may begin inside a tile
  // A unit of up to 512 keys stays whole, one of up to 1024 where there are units for a third of the
  // workers: a second kernel would cost more than it saves (us, whole / cut, one token: 1 sequence of
  // 500 keys 13 / 12.4, but 14 / 16.4 from Python, a launch less; 48 of 100..500 17 / 22, of 100..1000
  // 23 / 27; 4 of 1000 19 / 14; 16 of 2000 30 / 25, 64 of 100..4000 62 / 58).
  const long long units = (long long)batch * hkv;
  d.no_pieces = ring || unit_keys <= 256;
  d.whole_units = ring || unit_keys <= 512 || (unit_keys <= 1024 && units * 3 >= (long long)kI4Sms * d.groups);
  const long long most = d.whole_units ? units : units * tiles;
  const long long all = (long long)sms * d.groups / d.split;
  d.workers = int(most < all ? most : all);
  // A batch that is cut has more workers than a larger one of whole units; a buffer for the larger one
  // has to serve it.  Units that no batch cuts leave the tile table alone.
  d.max_workers = unit_keys <= 512 ? 0 : int(units * tiles < all ? units * tiles : all);
  return d;
}

cudaError_t launch_decode4(const Decode4Params& p, int sms, cudaStream_t s, void* ev_begin, void* ev_end) {
  cudaError_t e;
  if (ev_begin && (e = cudaEventRecord(static_cast<cudaEvent_t>(ev_begin), s)) != cudaSuccess) return e;
  if (p.tc) {
    e = launch_decode4_tc(p, sms, s);
  } else {
    e = cudaFuncSetAttribute(decode4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    decode4_kernel<<<p.workers < sms ? p.workers : sms, kWarps * 32, kSmem, s>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  if (ev_end && (e = cudaEventRecord(static_cast<cudaEvent_t>(ev_end), s)) != cudaSuccess) return e;
  return p.whole_units ? cudaSuccess : launch_decode4_combine(p, s);
}

}  // namespace mimo
