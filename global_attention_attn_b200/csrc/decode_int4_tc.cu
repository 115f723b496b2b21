// Decode and draft verification over a 4-bit paged cache on the 5th-generation tensor cores.
//
// 180 bytes per (key, KV head), 57 FLOP per byte and draft, and every element unpacked first: on
// mma.sync (decode_int4.cu) an m16n8k16 takes 8.9 cycles of a scheduler during which the other
// instructions it dispatches do not come for free (an mma.sync and four LOP3, 2 cycles each,
// measured 12.2 to 12.8 cycles), and every draft unpacks the tile again.  Here both products are
// tcgen05.mma, so the warps only unpack and exponentiate, once for all drafts:
//   - S^T = K Q^T, 128 keys as the rows of A in tensor memory: a thread unpacks half of its own
//     key's words (int4.cuh: one shift and four ANDs per 8 codes, no conversion) and applies the
//     key's 6 scales to its half of the columns' 6 group sums.  The rotated query dims enter as
//     two fp16 terms (no 16-bit type holds them to the digits of an fp32 log-sum-exp); the code
//     offset is one more k-step, a constant row of A against -8 * the query's group sums.
//   - O^T = V^T P^T: a thread unpacks half of its key's value row to fp16, scale applied, into
//     shared memory ([key][dim], the M-major operand), and stores its weights beside it.  The
//     sums of all tiles stay in tensor memory, 128 dims x columns.
// A column is a query row of the KV head (draft, head).  Its reference is common to a tile's warps,
// which share the sums: after its logits a warp tells the others whether one has passed the
// reference by 2^6, and reads their answer after the values are unpacked; only then do all of
// them meet and move it, else nothing is rescaled.
//
// Eight warps (two threads a key) work on a tile, another issues copies and products.  One token
// of a KV head is 16 columns, whose tensor and shared memory let two such streams share an SM; more
// columns have one stream.  (Four threads a key: 4 and 8 drafts 103 and 215 us against 97 and 195
// at the time, the work that does not divide by columns done twice.)  From 64 columns on the six group
// sums do not fit beside the output's, so the logits run in two or three parts that take turns in
// the same columns; an SM's warps hide the wait between them with the next tile's keys.
// Workers are the streams: the tiles of all sequences and KV heads form one line, cut into as many
// equal pieces as there are workers, so any mix of lengths loads every SM alike.  A piece's first
// and last (sequence, head) may be partial and go through the combine kernel, the others write
// their rows directly; short contexts are cut between units only.
//
// Measured (graph replay, in brackets the same on mma.sync with the drafts' rows in warps of their
// own): 64 sequences of 4096..65536 keys, one token, 412 us (548), 3.7 TB/s, 0.57 of a copy's rate;
// one of 131001 keys 39 us (64); one of 500 13.4 us (18.5); 16 of 1001..16384 with 1, 2, 4, 8
// drafts 43, 62, 92 (160), 186 us.  Nothing is saturated (one token: the ALU pipe and the issue slots at
// half; 4 drafts: 22 % and a third): a tile's chain of sums, vote, values and hand-over sets the pace,
// 540 instructions per warp and tile of 16 columns (a third of them the unpacking) with four to five
// warps a scheduler to cover its latencies, three with more columns.  The copies alone take 260 us in
// the first call.
// Short calls are the sum of what a worker does once: 2 us to its first tile's copy, 1.5 us for the
// query operand, 3 us for the first tile (nothing overlaps yet, the references are set) and 1.5 us
// for its rows.
#include "int4_tc.cuh"
#include "tiles.cuh"
#include "../../include/mimoattn.h"

namespace mimo {

namespace {

constexpr int kTile = kI4TcTile;
static_assert(kTile == kPage, "a tile is a page");
// a tile's keys: codes, scales; its values: codes (64-byte swizzle), scales
constexpr int kKBytes = kTile * kI4KSlot, kOffKs = kTile * kI4KCodes;
constexpr int kVBytes = kTile * kI4VSlot, kOffVs = kTile * kI4VCodes;
static_assert(kVBytes % 512 == 0, "64-byte swizzle alignment");
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Weights are 2^(z - ref + kPBias): ref is a column's maximum when it was set, and moves only when a
// logit passes it by more than kSlack powers of two.  The products take them in fp16, whose smallest
// steps are 2^-24: the bias uses all of the range above (2^(kSlack + kPBias) < 65504), so that a weight
// keeps its digits down to 2^-24 of the reference and is not lost before 2^-35 (without it 2^-14 and
// 2^-25: a key that takes nearly all the weight, over 131000 others at 2^-25.2 each, took their 0.4 %
// of the sum, and with a small value of its own most of the output).  The sums of weights carry the
// same factor; -ref + kPBias is what stands for the reference everywhere.
constexpr float kSlack = 6.f, kPBias = 9.9375f;
constexpr int kW = 8, kN = 32 * kW;  // warps and threads of a stream, two threads a key

// What depends on the number of columns.
template <int N>
struct Lay {
  static constexpr int kStreams = N == 16 ? 2 : 1;
  static constexpr int kThreads = kStreams * kN + 128;  // and a warpgroup whose first warps issue
  // registers at launch, of a thread that computes and of one that issues
  static constexpr int kRegs = kStreams == 2 ? 96 : 168, kRegsWork = kStreams == 2 ? kRegs : 208, kRegsIssue = kStreams == 2 ? kRegs : 88;
  static_assert(kStreams * kN * kRegsWork + 128 * kRegsIssue <= kThreads * kRegs, "register split");
  // A tile's logits run in parts of kPer groups, in one where their columns all fit (kSep), else the
  // parts take turns in the same columns.
  static constexpr bool kSep = 7 * N + 112 <= 512;
  static constexpr int kPer = kSep ? kI4KGroups : (N <= 96 ? 3 : 2), kParts = kI4KGroups / kPer;
  static constexpr uint32_t kColA = 0, kColOne = 96, kColD = 112, kColO = kColD + (kSep ? kI4KGroups : kPer) * N;
  static constexpr uint32_t kColStream = 256;
  static_assert(kColO + N <= (kStreams == 1 ? 512 : kColStream), "tensor memory");
  __host__ __device__ static constexpr uint32_t col(int j) { return kColD + (kSep ? j : j % kPer) * N; }
  // a stream's shared memory: query operand (N rows of 64 elements, 128-byte swizzle: dims 0..63,
  // 64..127, 128..191, the second terms of 0..63; a 32-byte row of the offset per column of sums),
  // values, weights, then the rings of copied tiles
  static constexpr int kQChunk = N * 128, kQOffset = 4 * kQChunk;
  static constexpr int kOffV = (kQOffset + kI4KGroups * N * 32 + 1023) / 1024 * 1024;
  static constexpr int kVChunk = kTile * 128, kOffP = kOffV + 2 * kVChunk;
  static constexpr int kPBytes = N == 16 ? kTile * 32 : (N + 63) / 64 * kVChunk;
  static constexpr int kStagesK = N <= 64 && N > 16 ? 4 : 3, kStagesV = N <= 64 && N > 16 ? 3 : 2;
  static constexpr int kOffRingV = kOffP + kPBytes, kOffRingK = kOffRingV + kStagesV * kVBytes;
  static constexpr int kStream = (kOffRingK + kStagesK * kKBytes + 1023) / 1024 * 1024;
  // per stream: references, factors, the warps' maxima or sums, cos and sin
  static constexpr int kOffX = kStreams * kStream, kXBytes = 6 * N * 4 + (N < 64 ? N / 8 : 8) * kHalf * 8;
  static constexpr int kOffBar = kOffX + kStreams * kXBytes;
  static constexpr int kOffTbl = kOffBar + 288;
  static constexpr int kSmem = kOffTbl + (kMaxTableBatch + 1) * 8 + 1024;
  static_assert(kOffRingV % 512 == 0 && kSmem <= 232448, "shared memory budget");
};

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// two weights -> fp16x2 (saturating: beyond |z| = 2^19 the fp32 step of a logit is above what is left
// between 2^(kSlack + kPBias) and fp16's limit)
__device__ __forceinline__ uint32_t f16x2_sat_of(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
// (x & mask) | base, one LOP3 (base in a register)
__device__ __forceinline__ uint32_t field(uint32_t x, uint32_t mask, uint32_t base) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "r"(mask), "r"(base));
  return d;
}
template <int V>
struct Int {
  static constexpr int value = V;
};

// Steps KK .. of part PT of a tile's logits (two terms for groups 0, 1).
template <int N, int PT, int KK>
__device__ __forceinline__ void logit_steps(uint32_t tmem, uint32_t lo, uint32_t hi) {
  using Y = Lay<N>;
  if constexpr (KK < 2 * Y::kPer * (PT + 1)) {
    constexpr uint32_t idesc = idesc_f32acc(128, N, 0, 0, 0), d = Y::col(KK >> 1), a = Y::kColA + 8 * KK;
    tc_mma_ts_at<d, a, (((KK >> 2) * Y::kQChunk + (KK & 3) * 32) >> 4)>(tmem, lo, hi, idesc);
    if constexpr (KK < 4) tc_mma_ts_at<d, a, ((3 * Y::kQChunk + KK * 32) >> 4)>(tmem, lo, hi, idesc);
    logit_steps<N, PT, KK + 1>(tmem, lo, hi);
  }
}
// The offset over columns COL .. of part PT, which starts the sums.
template <int N, int PT, int COL>
__device__ __forceinline__ void logit_offset(uint32_t tmem, uint64_t qo) {
  using Y = Lay<N>;
  constexpr int all = Y::kPer * N;
  if constexpr (COL < all) {
    constexpr int n = all - COL > 240 ? 240 : all - COL;
    tc_mma_ts(tmem + Y::col(Y::kPer * PT) + COL, tmem + Y::kColOne, qo + (((all * PT + COL) * 32) >> 4),
              idesc_f32acc(128, n, 0, 0, 0), 0u);
    logit_offset<N, PT, COL + n>(tmem, qo);
  }
}
template <int N, int PT>
__device__ __forceinline__ void logits_part(uint32_t tmem, uint64_t qd, uint64_t qo) {
  logit_offset<N, PT, 0>(tmem, qo);
  logit_steps<N, PT, 2 * Lay<N>::kPer * PT>(tmem, uint32_t(qd), uint32_t(qd >> 32));
}

// Pieces that a line of `total` tiles is cut into: piece w is tiles w total / W .. (w + 1) total / W.
__device__ __forceinline__ int pieces_of(long long total, int workers) { return int(total < workers ? total : workers); }

// Keys a sequence's unit covers: [lo, hi], and its first tile and tile count.
struct Span {
  int lo, hi, t0, nt;
};
__device__ __forceinline__ Span span_of(const Decode4Params& p, int ctx) {
  Span u;
  u.hi = min(ctx, p.max_seq_len) - 1;
  u.lo = p.window > 0 ? max(0, ctx - p.q_len + 1 - p.window) : 0;
  if (ctx < p.q_len || u.lo > u.hi) {
    u.t0 = u.nt = 0;
  } else {
    u.t0 = u.lo / kTile;
    u.nt = u.hi / kTile - u.t0 + 1;
  }
  return u;
}

}  // namespace

template <int N>
__global__ void __launch_bounds__(Lay<N>::kThreads, 1) decode4_tc_kernel(const __grid_constant__ Decode4Params p) {
  using Y = Lay<N>;
  constexpr int NC = N / 2, kParts = Y::kParts, kPer = Y::kPer;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool issuer = warp >= Y::kStreams * kW;
  const int str = __shfl_sync(0xffffffffu, issuer ? warp - Y::kStreams * kW : warp / kW, 0);
  const int gq = warp & 3, hw = (warp >> 2) & 1;  // the quarter of the tile's keys, and which of a key's two threads
  const int tid = threadIdx.x & (kN - 1);                 // within the stream
  const uint32_t base = sbase + str * Y::kStream;
  const uint32_t vt = base + Y::kOffV, pt = base + Y::kOffP;
  const uint32_t ring_k = base + Y::kOffRingK, ring_v = base + Y::kOffRingV;
  float* const nref = reinterpret_cast<float*>(smem + Y::kOffX + str * Y::kXBytes);  // [N] kPBias minus the references
  float* const fac = nref + N;                                                       // [N] what a move multiplies with
  float* const wmax = fac + N;                                                       // [4][N]
  float2* const cs = reinterpret_cast<float2*>(wmax + 4 * N);
  const uint32_t bar0 = sbase + Y::kOffBar + str * 128;
  auto full_k = [&](int i) { return bar0 + 8 * i; };
  auto full_v = [&](int i) { return bar0 + 32 + 8 * i; };
  auto ready = [&](int h) { return bar0 + 56 + 8 * h; };  // part h of a tile's logits may run
  auto done = [&](int h) { return bar0 + 80 + 8 * h; };   // its sums stand
  const uint32_t pv_ready = bar0 + 104, pv_done = bar0 + 112, vote = bar0 + 120;
  static_assert(Y::kStagesK <= 4 && Y::kStagesV <= 3 && kParts <= 3, "barriers");
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + Y::kOffBar + 256);
  volatile int* const flag = reinterpret_cast<volatile int*>(smem + Y::kOffBar + 272 + str * 8);  // [2]
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + Y::kOffBar + 264);
  long long* const tbl = reinterpret_cast<long long*>(smem + Y::kOffTbl);
  if (!issuer && tid == 0) {
    for (int i = 0; i < Y::kStagesK; ++i) mbar_init(full_k(i), 1);
    for (int i = 0; i < Y::kStagesV; ++i) mbar_init(full_v(i), 1);
    for (int h = 0; h < kParts; ++h) {
      mbar_init(ready(h), kW);
      mbar_init(done(h), 1);
    }
    mbar_init(pv_ready, kW);
    mbar_init(pv_done, 1);
    mbar_init(vote, kW);
    flag[0] = flag[1] = 0;
    if (str == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == 1) {
    tile_table(tbl, p.batch, lane, [&](int s) {
      const int ctx = p.seq_lens[s];
      if (blockIdx.x == 0 && (ctx < p.q_len || ctx > p.max_seq_len)) atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
      return span_of(p, ctx).nt;
    });
    if (blockIdx.x == 0 && p.ws_tbl)
      for (int s = lane; s <= p.batch; s += 32) p.ws_tbl[s] = tbl[s];
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot + str * Y::kColStream, 0);  // (known uniform)

  // ---- this stream's piece of the line
  const long long total = tbl[p.batch] * p.hkv;
  const int w = str * gridDim.x + blockIdx.x;
  long long a = 0, b = 0;
  if (str >= Y::kStreams) {
    // the issuing warpgroup's idle warps
  } else if (total > 0 && p.whole_units) {
    const int units = p.batch * p.hkv, W = min(units, p.workers);
    auto at = [&](int u) {
      const int s = u / p.hkv;
      return s >= p.batch ? total : tbl[s] * p.hkv + (u - s * p.hkv) * (tbl[s + 1] - tbl[s]);
    };
    if (w < W) {
      a = at(w * units / W);
      b = at((w + 1) * units / W);
    }
  } else if (total > 0) {
    // (total fits 31 bits, W * W too: w total / W without a 64-bit division)
    const int W = pieces_of(total, p.workers);
    const unsigned each = unsigned(total) / W, rest = unsigned(total) - each * W;
    if (w < W) {
      a = (long long)w * each + w * rest / W;
      b = (long long)(w + 1) * each + (w + 1) * rest / W;
    }
  }
  const int n_all = int(b - a);
  auto wait_w = [&](uint32_t bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;  // (a branch of the whole warp)
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, MIMO_STATUS_TIMEOUT));
  };

  if (issuer) {
    if constexpr (Y::kRegsIssue != Y::kRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Y::kRegsIssue));
    if (n_all > 0) {
      // ---- copies of the piece's tiles in order, and each tile's products.  A slot of keys is free
      // when the last part of its logits may run, one of values when its product may.
      struct Copies {
        TileCursor c;
        int n, pg_s, pg_base, pg, t0;  // tiles copied; lane i: page id of page pg_base + i of sequence pg_s
      };
      Copies ck, cv;
      ck.c = cv.c = cursor_at(tbl, p.batch, p.hkv, a);
      ck.n = cv.n = ck.pg = cv.pg = ck.t0 = cv.t0 = ck.pg_base = cv.pg_base = 0;
      ck.pg_s = cv.pg_s = -1;
      auto next_block = [&](Copies& k) {  // of tile k.n of the piece
        if (k.c.t == k.c.nt) next_unit(tbl, p.hkv, k.c);
        if (k.c.s != k.pg_s) k.t0 = span_of(p, p.seq_lens[k.c.s]).t0;
        const int pi = k.t0 + k.c.t;
        if (k.c.s != k.pg_s || pi < k.pg_base || pi >= k.pg_base + 32) {
          k.pg_s = k.c.s;
          k.pg_base = pi;
          const int mine = pi + lane;
          k.pg = 0;
          if (mine < k.t0 + k.c.nt) {
            k.pg = mine < p.max_pages ? p.block_table[long(k.c.s) * p.max_pages + mine] : -1;
            if (k.pg < 0 || k.pg >= p.num_pages) {
              atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
              k.pg = 0;
            }
          }
        }
        ++k.c.t;
        ++k.n;
        return __shfl_sync(0xffffffffu, k.pg, pi - k.pg_base) * p.hkv + k.c.g;
      };
      auto copy_k = [&]() {
        if (ck.n >= n_all) return;
        const int i = ck.n % Y::kStagesK;
        const uint32_t dst = ring_k + i * kKBytes, bar = full_k(i);
        const int block = next_block(ck);
        if (elect_one()) {  // a block's codes and scales are one piece
          mbar_expect_tx(bar, kKBytes);
          bulk_load(dst, p.k_cache + long(block) * kPage * kI4KSlot, kKBytes, bar);
        }
        __syncwarp();
      };
      auto copy_v = [&]() {
        if (cv.n >= n_all) return;
        const int i = cv.n % Y::kStagesV;
        const uint32_t dst = ring_v + i * kVBytes, bar = full_v(i);
        const int block = next_block(cv);
        if (elect_one()) {
          mbar_expect_tx(bar, kVBytes);
          tma_load_3d(dst, &p.tm_v, bar, 0, 0, block);
          bulk_load(dst + kOffVs, p.v_cache + long(block) * kPage * kI4VSlot + kOffVs, kTile * 2 * kI4VGroups, bar);
        }
        __syncwarp();
      };
      const uint64_t qd = sdesc_sw128(base, 16, 1024), qo = sdesc_sw32(base + Y::kQOffset, 256);
      const uint64_t vd = sdesc_sw128(vt, Y::kVChunk, 1024);
      const uint64_t pd = N == 16 ? sdesc_sw32(pt, 256) : sdesc_sw128(pt, Y::kVChunk, 1024);
      constexpr int kPStep = N == 16 ? 16 * 32 : 16 * 128;  // bytes of a 16-key step of the weights
      bool ok = true;
      auto part = [&](auto pt_, int tile) {
        constexpr int PT = decltype(pt_)::value;
        if (!ok || !(ok = wait_w(ready(PT), tile & 1))) return;
        if (elect_one()) {
          tc_fence_after();
          logits_part<N, PT>(tmem, qd, qo);
          tc_commit(done(PT));
        }
        __syncwarp();
        if (PT == kParts - 1) copy_k();
      };
      auto first_part = [&](int tile) { part(Int<0>(), tile); };
      auto other_parts = [&](int tile) {
        if constexpr (!Y::kSep) {
          part(Int<1>(), tile);
          if constexpr (kParts == 3) part(Int<2>(), tile);
        }
      };
      for (int i = 0; i < Y::kStagesK; ++i) copy_k();
      for (int i = 0; i < Y::kStagesV; ++i) copy_v();
      TileCursor mc = cursor_at(tbl, p.batch, p.hkv, a);
      int n = 0;
      first_part(0);
      for (; n < n_all && ok; ++n) {
        if (mc.t == mc.nt) next_unit(tbl, p.hkv, mc);
        const bool first = n == 0 || mc.t == 0;  // of the unit's tiles here: the sums start
        ++mc.t;
        const bool last = mc.t == mc.nt || n + 1 == n_all;  // (the next tile waits for its unit's query)
        other_parts(n);
        if (!last) first_part(n + 1);
        if (!ok || !(ok = wait_w(pv_ready, n & 1))) break;
        if (elect_one()) {
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            tc_mma_ss(tmem + Y::kColO, vd + ((kk * 2048) >> 4), pd + ((kk * kPStep) >> 4), idesc_f32acc(128, N, 1, 1, 0),
                      first && kk == 0 ? 0u : 1u);
          tc_commit(pv_done);
        }
        __syncwarp();
        copy_v();
        if (last && n + 1 < n_all) first_part(n + 1);
      }
      if (!ok && elect_one()) {
        // a wait ran out: the copies and products under way end before the block does
        int dummy = 0;
        auto drain = [&](uint32_t bar, uint32_t parity) { mbar_wait(bar, parity, &dummy, nullptr, 0, 50000000ull); };
        for (int i = max(0, ck.n - Y::kStagesK); i < ck.n; ++i) drain(full_k(i % Y::kStagesK), (i / Y::kStagesK) & 1);
        for (int i = max(0, cv.n - Y::kStagesV); i < cv.n; ++i) drain(full_v(i % Y::kStagesV), (i / Y::kStagesV) & 1);
        tc_commit(pv_done);
        for (int i = 1; i >= 0; --i) drain(pv_done, (n + i) & 1);
      }
    }
    tc_fence_before();
    __syncthreads();
    return;
  }

  if constexpr (Y::kRegsWork != Y::kRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Y::kRegsWork));
  const uint32_t t_lane = tmem + (uint32_t(gq * 32) << 16);
  auto stream_sync = [&]() { asm volatile("bar.sync %0, %1;" ::"r"(str + 1), "n"(kN) : "memory"); };
  // A barrier that tells whether any thread of the stream brought `v`.
  auto any_of = [&](bool v) -> bool {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(v)), "r"(str + 1), "n"(kN)
        : "memory");
    return r != 0;
  };
  if (hw == 0 && n_all > 0) {
    uint32_t one[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) one[i] = 0x04000400u;  // 2^-14
    tmem_st8(t_lane + Y::kColOne, one);
    tmem_wait_st();
  }
  const int row = gq * 32 + lane;  // this thread's key of the tile
  const uint32_t v_row = vt + hw * Y::kVChunk + row * 128 + ((row & 7) << 4);
  uint32_t W[12], zs[3];           // this thread's half of the next tile's key: word 4 j + 2 hw + q of group j at 6 q + j; its scales
  int kst = 0, kph = 0, vst = 0, vph = 0;
  auto fetch = [&]() -> bool {
    if (!wait_w(full_k(kst), kph & 1)) return false;
    const uint32_t at = ring_k + kst * kKBytes, ka = at + row * kI4KCodes + 48 * hw;
#pragma unroll
    for (int i = 0; i < 3; ++i) lds128(ka + 16 * i, W + 4 * i);
#pragma unroll
    for (int i = 0; i < 3; ++i) zs[i] = lds32(at + kOffKs + row * 2 * kI4KGroups + 4 * i);
    if (++kst == Y::kStagesK) kst = 0, ++kph;
    return true;
  };
  // Part h of it into the key's row of A.
  auto unpack = [&](int h) {
#pragma unroll
    for (int j = kPer * h; j < kPer * h + kPer; ++j) {
      uint32_t r[8];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t x = W[6 * q + j], y = x >> 8;
        r[4 * q] = x & kI4Lo;
        r[4 * q + 1] = x & kI4Hi;
        r[4 * q + 2] = y & kI4Lo;
        r[4 * q + 3] = y & kI4Hi;
      }
      tmem_st8(t_lane + Y::kColA + 16 * j + 8 * hw, r);
    }
    tmem_wait_st();
  };
  auto hand_over = [&](uint32_t bar) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  uint32_t k1024, k64;
  asm volatile("mov.b32 %0, 0x64006400;\n\tmov.b32 %1, 0x54005400;" : "=r"(k1024), "=r"(k64));  // (opaque: see field)
  const int G = p.group, g_log = G == 16 ? 4 : 3, rows = p.q_len * G;
  const float c_log2 = p.scale_log2 * kI4KeyUnit;
  const uint64_t c2 = pack_f32x2(c_log2, c_log2);
  bool ok = true;
  TileCursor c;
  if (n_all > 0) c = cursor_at(tbl, p.batch, p.hkv, a);
  for (int x = 0; x < n_all && ok;) {
    if (c.t == c.nt) next_unit(tbl, p.hkv, c);
    const int s = c.s, g = c.g, t_first = c.t, ctx = p.seq_lens[s];
    const int t_end = min(c.nt, c.t + (n_all - x));
    const Span U = span_of(p, ctx);
    const int first_pos = ctx - p.q_len;  // slot of the first draft
    // ---- the unit's query operand
    const float amax = int4_query_operand<N, kN, Y::kQChunk>(
        p.q + (long(s) * p.q_len * kHq + g * G) * kDqk, rows, g_log, base, tid, cs, [&]() {
          stream_sync();  // (the unit before has read what is written here)
          const int pos0 = (p.positions ? p.positions[s] + 1 : ctx) - p.q_len;
          for (int i = tid; i < p.q_len * kHalf; i += kN)
            rope_cos_sin(pos0 + i / kHalf, p.rope.inv_freq[i % kHalf], &cs[i].x, &cs[i].y);
          if (tid < N) nref[tid] = tid < rows ? INFINITY : -INFINITY;  // (a padding column: weight 0)
          stream_sync();
        },
        [](int) { return true; });
    if (amax > kF16Max) atomicOr(p.status, MIMO_STATUS_RANGE);
    fence_proxy_async_smem();
    stream_sync();
    bool good = fetch();
    uint32_t z[3];
    if (good) {
#pragma unroll
      for (int h = 0; h < kParts; ++h) unpack(h);
      hand_over(ready(0));
    }
    constexpr bool kHold = N <= 64;  // the references in registers
    auto ref2 = [&](int i) { return *reinterpret_cast<const uint64_t*>(nref + hw * NC + 2 * i); };
    uint64_t nr[kHold ? NC / 2 : 1];
    if constexpr (kHold)
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) nr[i] = ref2(i);
    uint64_t l[NC / 2];  // this thread's sums of its columns
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) l[i] = 0;

    for (; c.t < t_end; ++c.t, ++x) {
      const int key = (U.t0 + c.t) * kTile + row, key0 = key - lane;
      // a column's draft d sees the keys first_pos + d - window + 1 .. first_pos + d of [lo, hi]
      const bool edge = key0 < U.lo + (p.window > 0 ? p.q_len - 1 : 0) || key0 + 31 > min(U.hi, first_pos);
      const bool more = c.t + 1 < t_end, start = c.t == t_first;
#pragma unroll
      for (int i = 0; i < 3; ++i) z[i] = zs[i];
      uint64_t S[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) S[i] = 0;
#pragma unroll
      for (int h = 0; h < kParts; ++h) {
        if (good) good = wait_w(done(h), x & 1);
        if (!good) continue;
        tc_fence_after();
        constexpr int kC = NC == 16 ? 16 : 8;  // columns at a time
#pragma unroll
        for (int c0 = 0; c0 < NC; c0 += kC) {
          uint32_t d[kPer][kC];
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const uint32_t at = t_lane + Y::col(kPer * h + j) + hw * NC + c0;
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
        if (h + 1 < kParts) hand_over(ready(h + 1));  // (its columns are free)
        if (more) {
          if (h == 0) good = fetch();
          if (good) unpack(h);
        }
        if (good && more && h == kParts - 1) hand_over(ready(0));
      }
      // ---- logits against the references, 8 columns at a time (of one draft)
      auto logits = [&](int i, float* xs) {
        uint64_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = kHold ? nr[kHold ? 4 * i + e : 0] : ref2(4 * i + e);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t v = fma_f32x2(S[4 * i + e], c2, r[e]);
          xs[2 * e] = lo_f32(v);
          xs[2 * e + 1] = hi_f32(v);
        }
      };
      auto hidden = [&](int i) {
        const int at = first_pos + ((hw * NC + 8 * i) >> g_log);
        return key > min(at, U.hi) || (p.window > 0 && key <= at - p.window);
      };
      float top = -INFINITY;
      // where registers allow, the weights are made here, in the hope that no reference moves
      constexpr bool kEarly = NC <= 32;
      float ws[kEarly ? NC : 8];
#pragma unroll
      for (int i = 0; i < NC / 8; ++i) {
        float* const xs = ws + (kEarly ? 8 * i : 0);
        float t8 = -INFINITY;
        logits(i, xs);
        if (edge && hidden(i)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) xs[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) t8 = fmaxf(t8, xs[e]);
        top = fmaxf(top, t8);
      }
      // (the warps tell each other which tile moves the references; the answer is read after the values)
      const bool raise = __any_sync(0xffffffffu, top > kSlack + kPBias) || !good;
      if (lane == 0) {
        if (raise) flag[x & 1] = x + 1;
        mbar_arrive(vote);
      }
      auto weights = [&](int i, float* xs) {
        logits(i, xs);
        if (edge && hidden(i)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) xs[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) xs[e] = ex2(xs[e]);
      };
      if constexpr (kEarly)
#pragma unroll
        for (int e = 0; e < NC; ++e) ws[e] = ex2(ws[e]);
      // ---- values: (code - 8) * scale in fp16, this thread's 64 dims.  1024 + n and 64 + n come out of a
      // word with one LOP3; the scale is not folded into the weights, as a row of 64 dims has two.
      // A slot nothing was written to may hold any scale: it counts as 0
      // (where the logits run in parts, the last one's sums stand after the product of the tile before)
      if (Y::kSep && good && x > 0) good = wait_w(pv_done, (x - 1) & 1);
      if (good) good = wait_w(full_v(vst), vph & 1);
      if (good) {
        const uint32_t at = ring_v + vst * kVBytes;
        uint32_t sv = lds32(at + kOffVs + row * 2 * kI4VGroups + 4 * hw);
        sv = key <= U.hi ? sv : 0u;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t s2 = __byte_perm(sv, 0, u ? 0x3232 : 0x1010);
          uint32_t vw[4];
          lds128(at + row * kI4VCodes + (((2 * hw + u) ^ ((row >> 1) & 3)) << 4), vw);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t y = vw[i] >> 8;
            uint32_t o[4];
            o[0] = hmul2(hadd2(field(vw[i], kI4Lo, k1024), 0xE408E408u), s2);  // - 1032
            o[1] = hmul2(hadd2(field(vw[i], kI4Hi, k64), 0xD480D480u), s2);    // - 72
            o[2] = hmul2(hadd2(field(y, kI4Lo, k1024), 0xE408E408u), s2);
            o[3] = hmul2(hadd2(field(y, kI4Hi, k64), 0xD480D480u), s2);
            sts128(v_row ^ ((4 * u + i) << 4), o);
          }
        }
      }
      if (++vst == Y::kStagesV) vst = 0, ++vph;
      // (every warp arrives, whatever became of its waits, and must not be left behind at the barriers
      // below: a probe takes 4 us, so this gives up after 16 s, beyond the six waits of 2 s that another
      // warp can have since the last vote; the one that ran out has set the status)
      for (int i = 0; i < 4000000 && !mbar_try_wait_hint(vote, x & 1, 20000); ++i) {
      }
      if (flag[x & 1] == x + 1) {
        // the references that were passed move to their new maxima, and the sums with them
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          float m = ((i & 1) ? hi_f32(S[i >> 1]) : lo_f32(S[i >> 1])) * c_log2;
          if (edge && hidden(i >> 3)) m = -INFINITY;
          m = warp_max(m);
          if (lane == 0) wmax[gq * N + hw * NC + i] = m;
        }
        if (any_of(!good)) {
          ok = false;
          break;
        }
        if (tid < N) {
          const float m = fmaxf(fmaxf(wmax[tid], wmax[N + tid]), fmaxf(wmax[2 * N + tid], wmax[3 * N + tid]));
          const float old = nref[tid], now = kPBias - m;
          const bool up = m + old > kSlack + kPBias;
          fac[tid] = up ? ex2(now - old) : 1.f;  // (from a reference of -inf: 0, of sums that are 0)
          if (up) nref[tid] = now;
        }
        stream_sync();
#pragma unroll
        for (int i = 0; i < NC / 2; ++i) l[i] = mul_f32x2(l[i], *reinterpret_cast<const uint64_t*>(fac + hw * NC + 2 * i));
        if constexpr (kHold)
#pragma unroll
          for (int i = 0; i < NC / 2; ++i) nr[i] = ref2(i);
        if (!start) {
#pragma unroll 1
          for (int c0 = 0; c0 < NC; c0 += 8) {
            uint32_t d[8];
            tmem_ld8(t_lane + Y::kColO + hw * NC + c0, d);
            tmem_wait_ld_r8(d);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = __float_as_uint(__uint_as_float(d[i]) * fac[hw * NC + c0 + i]);
            tmem_st8(t_lane + Y::kColO + hw * NC + c0, d);
          }
          tmem_wait_st();
        }
        if constexpr (kEarly)
#pragma unroll
          for (int i = 0; i < NC / 8; ++i) weights(i, ws + 8 * i);
      }
      // ---- weights
#pragma unroll
      for (int i = 0; i < NC / 8; ++i) {
        float* const xs = ws + (kEarly ? 8 * i : 0);
        if constexpr (!kEarly) weights(i, xs);
        uint32_t pk[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pk[e] = f16x2_sat_of(xs[2 * e], xs[2 * e + 1]);
          l[4 * i + e] = add_f32x2(l[4 * i + e], pack_f32x2(xs[2 * e], xs[2 * e + 1]));
        }
        const int c8 = hw * (NC / 8) + i;  // of 8 columns
        if constexpr (N == 16) sts128(pt + row * 32 + ((c8 ^ ((row >> 2) & 1)) << 4), pk);
        else sts128(pt + (c8 >> 3) * Y::kVChunk + row * 128 + (((c8 & 7) ^ (row & 7)) << 4), pk);
      }
      if (good) {
        fence_proxy_async_smem();
        hand_over(pv_ready);
      }
    }
    if (!ok) break;

    // ---- the segment's rows: this thread holds one dim of its columns' sums
    if (good) good = wait_w(pv_done, (x - 1) & 1);
#pragma unroll
    for (int c0 = 0; c0 < NC / 8; ++c0) {
      // 8 sums over the warp: a step halves what a lane holds, down to one column per 4 lanes
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = lo_f32(l[4 * c0 + e]);
        v[2 * e + 1] = hi_f32(l[4 * c0 + e]);
      }
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) {
        const bool up = lane & (4 * d);
#pragma unroll
        for (int e = 0; e < d; ++e) {
          const float got = __shfl_xor_sync(0xffffffffu, up ? v[e] : v[e + d], 4 * d);
          v[e] = (up ? v[e + d] : v[e]) + got;
        }
      }
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
      if ((lane & 3) == 0) wmax[gq * N + hw * NC + 8 * c0 + (lane >> 2)] = v[0];
    }
    if (any_of(!good)) {
      ok = false;
      break;
    }
    tc_fence_after();
    const bool direct = t_first == 0 && c.t == c.nt;
    const long piece = 2L * w + (x > c.t - t_first ? 1 : 0);  // this worker's first or last segment
    if (tid < rows) {
      const int n = tid, h = g * G + (n & (G - 1));
      const float M = -nref[n], L = wmax[n] + wmax[N + n] + wmax[2 * N + n] + wmax[3 * N + n];
      if (direct) {
        float M2 = M, L2 = L, f = 1.f;
        if (p.sink) {
          const float sl = p.sink[h] * kLog2e;
          M2 = fmaxf(M, sl);
          f = ex2(M - M2);
          L2 = L * f + ex2(sl - M2);
        }
        fac[n] = p.v_scale * f / L2;
        if (p.lse) p.lse[(long(s) * p.q_len + (n >> g_log)) * kHq + h] = (M2 + log2f(L2)) * kLn2;
      } else {
        *reinterpret_cast<float2*>(p.ws_ml + (piece * (p.n_blocks * 16) + n) * 2) = make_float2(M, L);
      }
    }
    stream_sync();
    const int dim = (row & ~7) + ((row & 7) >> 1) + 4 * (row & 1);
#pragma unroll 1
    for (int n0 = hw * NC; n0 < min(rows, hw * NC + NC); n0 += 8) {  // 8 heads of a draft
      uint32_t d[8];
      tmem_ld8(t_lane + Y::kColO + n0, d);
      tmem_wait_ld_r8(d);
      if (direct) {
        uint16_t* const at = p.out + ((long(s) * p.q_len + (n0 >> g_log)) * kHq + g * G + (n0 & (G - 1))) * kDv + dim;
#pragma unroll
        for (int i = 0; i < 8; ++i) at[i * kDv] = uint16_t(pack2_bf16(__uint_as_float(d[i]) * fac[n0 + i], 0.f));
      } else {
        float* const at = p.ws_o + (piece * (p.n_blocks * 16) + n0) * kDv + dim;
#pragma unroll
        for (int i = 0; i < 8; ++i) at[i * kDv] = __uint_as_float(d[i]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, 512);
  }
}

namespace {
template <int N>
cudaError_t launch_n(const Decode4Params& p, int sms, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(decode4_tc_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<N>::kSmem);
  if (e != cudaSuccess) return e;
  decode4_tc_kernel<N><<<p.workers < sms ? p.workers : sms, Lay<N>::kThreads, Lay<N>::kSmem, s>>>(p);
  return cudaGetLastError();
}
}  // namespace

cudaError_t launch_decode4_tc(const Decode4Params& p, int sms, cudaStream_t s) {
  const int rows = p.q_len * p.group;
  if (rows <= 16) return launch_n<16>(p, sms, s);
  if (rows <= 32) return launch_n<32>(p, sms, s);
  if (rows <= 48) return launch_n<48>(p, sms, s);
  if (rows <= 64) return launch_n<64>(p, sms, s);
  if (rows <= 96) return launch_n<96>(p, sms, s);
  return launch_n<128>(p, sms, s);
}

// Merges the pieces that share a (query row, head)'s unit, kRow warps a row: a long context of a
// small batch has hundreds, each a dependent load away, so the warps take turns and the first adds
// up their sums (a fixed order, whatever the timing).
template <int kRow>
__global__ void __launch_bounds__(kRow == 1 ? 128 : 32 * kRow) decode4_combine_kernel(const __grid_constant__ Decode4Params p) {
  __shared__ float4 part[kRow][32];
  __shared__ float part_m[kRow], part_l[kRow];
  const int lane = threadIdx.x & 31, warp = kRow == 1 ? 0 : threadIdx.x >> 5;
  const int at = kRow == 1 ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const int qrow = at / kHq, h = at % kHq, s = qrow / p.q_len, g = h / p.group;
  pdl_wait_prerequisites();  // (the pieces stand from here on)
  const long long total = p.ws_tbl[p.batch] * p.hkv;
  const long long nt = p.ws_tbl[s + 1] - p.ws_tbl[s];
  if (nt == 0) return;
  const long long u0 = p.ws_tbl[s] * p.hkv + g * nt;
  const int W = pieces_of(total, p.workers);
  const int w0 = int(((u0 + 1) * W - 1) / total), w1 = int(((u0 + nt) * W - 1) / total);
  if (w0 == w1) return;  // one piece holds the unit: its rows are written
  const int rows = p.n_blocks * 16, rr = (qrow - s * p.q_len) * p.group + h % p.group;
  // the first piece's unit is that piece's last segment, unless it begins with it
  const long first = 2L * w0 + (u0 > w0 * total / W ? 1 : 0);
  auto piece = [&](int i) { return (i == 0 ? first : 2L * (w0 + i)) * rows + rr; };
  const int n = w1 - w0 + 1;
  float M = -INFINITY;
  for (int i = 32 * warp + lane; i < n; i += 32 * kRow) M = fmaxf(M, p.ws_ml[2 * piece(i)]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  if constexpr (kRow > 1) {
    if (lane == 0) part_m[warp] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRow; ++i) M = fmaxf(M, part_m[i]);
  }
  float sl = -INFINITY;
  if (p.sink) {
    sl = p.sink[h] * kLog2e;
    M = fmaxf(M, sl);
  }
  float L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = warp; i < n; i += kRow) {
    const float2 ml = *reinterpret_cast<const float2*>(p.ws_ml + 2 * piece(i));
    const float f = ex2(ml.x - M);
    const float4 v = *reinterpret_cast<const float4*>(p.ws_o + piece(i) * kDv + lane * 4);
    L += f * ml.y;
    acc.x += f * v.x;
    acc.y += f * v.y;
    acc.z += f * v.z;
    acc.w += f * v.w;
  }
  if constexpr (kRow > 1) {
    part[warp][lane] = acc;
    if (lane == 0) part_l[warp] = L;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int i = 1; i < kRow; ++i) {
      const float4 v = part[i][lane];
      L += part_l[i];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
  }
  if (p.sink) L += ex2(sl - M);
  const float sc = p.v_scale / L;
  *reinterpret_cast<uint2*>(p.out + (long(qrow) * kHq + h) * kDv + lane * 4) =
      make_uint2(pack2_bf16(acc.x * sc, acc.y * sc), pack2_bf16(acc.z * sc, acc.w * sc));
  if (p.lse && lane == 0) p.lse[long(qrow) * kHq + h] = (M + log2f(L)) * kLn2;
}

// Launched with programmatic serialization: its launch overlaps the decode's last blocks (131001 keys of one
// sequence 42.5 -> 41.4 us; waiting on the SMs from the decode's start on it cost 45.3).
cudaError_t launch_decode4_combine(const Decode4Params& p, cudaStream_t s) {
  const int rows = p.batch * p.q_len * kHq, pieces = p.workers / (p.batch * p.hkv) + 1;  // a unit's, about
  cudaLaunchConfig_t cfg = {};
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(unsigned(pieces <= 4 ? rows / 4 : rows));
  cfg.blockDim = dim3(pieces <= 16 ? 128 : 512);
  auto kernel = pieces <= 4 ? decode4_combine_kernel<1> : (pieces <= 16 ? decode4_combine_kernel<4> : decode4_combine_kernel<16>);
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace mimo
