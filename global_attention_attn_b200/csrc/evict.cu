// Eviction from a paged cache: which slots of every (sequence, KV head) stay, and the move of
// the kept slots into other pages (or of a narrow cache's slots into bf16 pages).
#include <cooperative_groups.h>

#include "common.cuh"
#include "int4.cuh"
#include "ptx.cuh"
#include "../../include/mimoattn.h"

namespace cg = cooperative_groups;

namespace mimo {

namespace {

// Scores as unsigned keys of the same order, from 0x007FFFFF (-infinity) to 0xFF800000: -0 equals
// 0, NaN counts as -infinity.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

constexpr uint32_t kZeroKey = 0x80000000u, kKeepKey = 0xFFFFFFFFu;

// Whether a key tells its score's bits (not -0 or 0, NaN or -infinity, a slot kept whatever it scores), and those.
__device__ __forceinline__ bool exact_key(uint32_t k) { return k != kZeroKey && k != kKeepKey && k > 0x007FFFFFu; }
__device__ __forceinline__ float key_score(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k ^ 0x80000000u : ~k); }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The keys that a CTA's registers (8 steps of its threads) leave over of the most slots that a CTA gets:
// an eighth of the longest row, or 65536.
constexpr int kMaxRestBytes = 4 * (65536 - 8 * 4 * 1024);
static_assert(4 * (MIMO_SELECT_MAX_SLOTS / 8 - 8 * 4 * 512) <= kMaxRestBytes, "512 threads, 8 CTAs");

constexpr int kBins = 2048;  // 11, 11 and 10 bits a pass
constexpr int kBinThreads = kBins / 4;  // a thread's bins are one 16-byte read

// Sum over the warps before this one, and over all, of one value per warp (a block-wide call).
template <int W>  // warps
__device__ __forceinline__ uint2 warps_before(uint32_t* buf, uint32_t mine, int warp, int lane) {
  if (lane == 0) buf[warp] = mine;
  __syncthreads();
  const uint32_t v = lane < W ? buf[lane] : 0u;
  uint32_t incl = v;
#pragma unroll
  for (int d = 1; d < W; d <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += u;
  }
  return make_uint2(__shfl_sync(0xffffffffu, incl - v, warp), __shfl_sync(0xffffffffu, incl, W - 1));
}

}  // namespace

// One cluster per (sequence, KV head) row.  The row is read once (4 bytes a slot, the floor) by the
// cluster's 1..8 CTAs, and stays with them: 4 Q keys a thread in registers, the rest of the longest
// rows in shared memory.  A lane takes 4 neighbouring slots at a step, a warp 128.  The border is found by up to three histogram passes (a CTA adds
// its bins that hold anything to those of one of the cluster through distributed shared memory,
// and every CTA draws the same conclusion from these: at 16 sequences of 40000..131072
// slots and 4 heads a seventh faster than every CTA reading the bins of all; a pass whose bin is wanted
// whole is the last), then each CTA writes its part of
// the kept slots at the place that the counts of the parts before it give: ascending, equal
// scores lowest slot first.  Slots never attended all score 0, so zeros are counted aside and
// enter the histogram once per warp; other equal scores add up one by one.
template <int T, int Q>  // threads; steps a warp holds in registers
__global__ void __launch_bounds__(T, 1024 / T) select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kWarps = T / 32;
  extern __shared__ uint4 rest_keys[];  // the steps after them, [step][thread]
  __shared__ __align__(16) uint32_t hist[3][kBins];
  __shared__ uint32_t sums[2][kWarps];
  __shared__ uint32_t found[3][3];  // of a pass: the border's bin, how many of it are wanted, how many it holds
  __shared__ uint32_t part[2];      // this CTA's counts, for the CTAs behind it
  cg::cluster_group cl = cg::this_cluster();
  const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
  const int row = blockIdx.x / C, s = row / p.hkv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int L = p.seq_lens[s];
  if (L < 0 || L > p.max_seq_len) {
    if (rank == 0 && tid == 0) atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
    L = max(0, min(L, p.max_seq_len));
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (tid < kBinThreads) reinterpret_cast<uint4*>(hist[i])[tid] = make_uint4(0, 0, 0, 0);
  if (C > 1) cluster_arrive();
  const float* const src = p.scores + long(row) * p.score_stride;
  const bool wide = (reinterpret_cast<uintptr_t>(src) & 15) == 0;
  const int per = ((L + C - 1) / C + 127) & ~127;  // slots of a CTA
  const int lo = min(L, rank * per), end = min(L, lo + per);
  // a warp's contiguous range of slots, 128 at a step
  const int range = (((end - lo) + kWarps - 1) / kWarps + 127) & ~127, steps = range / 128;
  const int at0 = lo + warp * range + 4 * lane, at_end = min(end, lo + (warp + 1) * range);
  // Keys: of a slot that stays whatever its score (the first, the recent; every slot of a row that
  // fits) the largest there is, above any score's; where there is no slot 0, below any score's.
  const bool all = L <= p.keep;
  const int first = all ? L : p.first, tail = all ? L : L - p.recent;
  uint32_t zeros = 0;
  auto load = [&](int k) {
    const int at = at0 + 128 * k;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (wide && at + 4 <= at_end) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(src + at));
      x[0] = v.x;
      x[1] = v.y;
      x[2] = v.z;
      x[3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at + e < at_end) x[e] = __ldg(src + at + e);
    }
    uint32_t key[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) key[e] = order_key(x[e]);
    if (at < first || at + 4 > tail) {  // (tail <= L: the end of the row is in here)
#pragma unroll
      for (int e = 0; e < 4; ++e) key[e] = at + e >= at_end ? 0u : (at + e < first || at + e >= tail ? kKeepKey : key[e]);
    } else if (at + 4 > at_end) {
#pragma unroll
      for (int e = 0; e < 4; ++e) key[e] = at + e >= at_end ? 0u : key[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) zeros += key[e] == kZeroKey;
    return make_uint4(key[0], key[1], key[2], key[3]);
  };
  uint4 reg[Q];
#pragma unroll
  for (int k = 0; k < Q; ++k) reg[k] = k < steps ? load(k) : make_uint4(0, 0, 0, 0);
  for (int k = Q; k < steps; ++k) rest_keys[(k - Q) * T + tid] = load(k);
  zeros = __reduce_add_sync(0xffffffffu, zeros);
  // f(step, 4 keys) for every 128 slots of this warp, in order
  auto each = [&](auto&& f) {
#pragma unroll
    for (int k = 0; k < Q; ++k)
      if (k < steps) {
        const uint32_t key[4] = {reg[k].x, reg[k].y, reg[k].z, reg[k].w};
        f(k, key);
      }
#pragma unroll 1
    for (int k = Q; k < steps; ++k) {
      const uint4 v = rest_keys[(k - Q) * T + tid];
      const uint32_t key[4] = {v.x, v.y, v.z, v.w};
      f(k, key);
    }
  };
  int need = p.keep;
  uint32_t prefix = 0, mask = 0;  // keys & mask == prefix are still in question
  bool whole = all;               // every slot whose key matches the prefix stays
  if (C > 1) cluster_wait();      // every CTA's bins are 0
  else __syncthreads();
  for (int pass = 0; !whole && pass < 3; ++pass) {  // (cluster-uniform: all of this is the row's)
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
    uint32_t* const hs = hist[pass];
    const uint32_t low = (1u << bits) - 1;
    each([&](int, const uint32_t* key) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((key[e] & mask) == prefix && key[e] != kZeroKey) atomicAdd(hs + ((key[e] >> shift) & low), 1u);
    });
    if (lane == 0 && zeros && (kZeroKey & mask) == prefix) atomicAdd(hs + ((kZeroKey >> shift) & low), zeros);
    // the cluster's bins add up in one CTA's: few of a CTA's bins hold anything
    const int leader = pass % C;
    __syncthreads();
    if (C > 1) {
      if (rank != leader && tid < kBinThreads) {
        uint32_t* const to = cl.map_shared_rank(hs, leader);
        const uint4 v = reinterpret_cast<const uint4*>(hs)[tid];
        const uint32_t mine[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (mine[e]) atomicAdd(to + 4 * tid + e, mine[e]);
      }
      cl.sync();
    }
    // bins from the largest down, 4 a thread
    uint4 b4 = make_uint4(0, 0, 0, 0);
    if (tid < kBinThreads) b4 = *reinterpret_cast<const uint4*>(cl.map_shared_rank(hs, leader) + kBins - 4 - 4 * tid);
    const uint32_t h[4] = {b4.w, b4.z, b4.y, b4.x};
    const uint32_t sum = h[0] + h[1] + h[2] + h[3];
    uint32_t incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += u;
    }
    uint32_t before = incl - sum + warps_before<kWarps>(sums[pass & 1], __shfl_sync(0xffffffffu, incl, 31), warp, lane).x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (before < uint32_t(need) && before + h[e] >= uint32_t(need)) {
        found[pass][0] = uint32_t(kBins - 1 - 4 * tid - e);
        found[pass][1] = uint32_t(need) - before;
        found[pass][2] = h[e];
      }
      before += h[e];
    }
    __syncthreads();
    prefix |= found[pass][0] << shift;
    mask |= low << shift;
    need = int(found[pass][1]);
    whole = found[pass][2] == found[pass][1];
  }
  // What is above the prefix stays, and of the slots whose key matches it the first `take` (of a row
  // that fits: all that is above 0)
  if (all) mask = 0xFFFFFFFFu;
  const uint32_t take = all ? 0 : uint32_t(need);
  uint32_t more = 0, tie = 0;
  each([&](int, const uint32_t* key) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      more += (key[e] & mask) > prefix;
      tie += (key[e] & mask) == prefix;
    }
  });
  more = __reduce_add_sync(0xffffffffu, more);
  tie = __reduce_add_sync(0xffffffffu, tie);
  const bool ties = tie > 0 && take > 0;  // this warp may have to choose
  __syncthreads();  // (the last pass's sums are read)
  const uint2 m = warps_before<kWarps>(sums[0], more, warp, lane), t = warps_before<kWarps>(sums[1], tie, warp, lane);
  more = m.x;
  tie = t.x;
  if (C > 1) {
    if (tid == 0) {
      part[0] = m.y;
      part[1] = t.y;
    }
    cl.sync();
    for (int r = 0; r < rank; ++r) {
      const uint32_t* q = cl.map_shared_rank(part, r);
      more += q[0];
      tie += q[1];
    }
  }
  int32_t* const idx = p.idx + long(row) * p.keep;
  float* const out = p.scores_out ? p.scores_out + long(row) * p.keep : nullptr;
  each([&](int k, const uint32_t* key) {
    // places by votes: slots of lower lanes, then the lane's own
    uint32_t up[4], eq[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e) up[e] = __ballot_sync(0xffffffffu, (key[e] & mask) > prefix);
    if (ties)
#pragma unroll
      for (int e = 0; e < 4; ++e) eq[e] = __ballot_sync(0xffffffffu, (key[e] & mask) == prefix);
    if (!(up[0] | up[1] | up[2] | up[3] | eq[0] | eq[1] | eq[2] | eq[3])) return;
    const uint32_t lower = (1u << lane) - 1;
    uint32_t mo = more, ti = tie;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      mo += __popc(up[e] & lower);
      ti += __popc(eq[e] & lower);
      more += __popc(up[e]);
      tie += __popc(eq[e]);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t u = (up[e] >> lane) & 1, q = (eq[e] >> lane) & 1;
      if (u || (q && ti < take)) {
        const uint32_t j = mo + min(ti, take);
        const int slot = at0 + 128 * k + e;
        idx[j] = slot;
        if (out) out[j] = exact_key(key[e]) ? key_score(key[e]) : __ldg(src + slot);
      }
      mo += u;
      ti += q;
    }
  });
  const int count = min(L, p.keep);
  for (int j = count + rank * T + tid; j < p.keep; j += C * T) {
    idx[j] = -1;
    if (out) out[j] = 0.f;
  }
  if (rank == 0 && tid == 0 && row % p.hkv == 0) p.counts[s] = count;
  if (C > 1) cl.sync();  // no CTA leaves while another reads its bins or counts
}

cudaError_t launch_select(const SelectParams& p, int sms, cudaStream_t s) {
  const long rows = long(p.num_seqs) * p.hkv;
  int c = 1, threads = 512;  // CTAs per row: 4096 slots each at least, 8 at most
  while (c < 8 && c * 4096 < p.max_seq_len) c *= 2;
  // Where an SM cannot hold two of them, or all the rows' CTAs are more than one round, fewer CTAs of
  // twice the threads and at most 65536 slots: fewer barriers across CTAs, and no second round
  // (us, with / without: 16 sequences of 40000..131072 slots and 4 heads 47 / 56, 32 of 20000..32768
  // 27 / 65, 64 of 4000..16384 29 / 46, 8 of 300000..390000 113 / 123; but one of 30000, a single
  // round, 18.6 / 16.4, and 4 of 100000..131072 45 / 30).
  const int resident = (p.max_seq_len + c - 1) / c > 19 * 2048 ? 1 : 2;
  if (c > 1 && rows * c > resident * sms) {
    threads = 1024;
    for (c = 1; c < 8 && c * 65536 < p.max_seq_len;) c *= 2;
  }
  const int per = ((p.max_seq_len + c - 1) / c + 127) & ~127;
  const int steps = (per + 4 * threads - 1) / (4 * threads);
  auto kernel = threads == 1024 ? select_kernel<1024, 8> : (steps <= 2 ? select_kernel<512, 2> : select_kernel<512, 8>);
  const size_t bytes = steps <= 8 ? 0 : size_t(steps - 8) * 16 * threads;
  if (bytes > 0) {
    // (the attribute is the kernel's, not the launch's: always the same value, as another host thread may
    // be between its own two calls)
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRestBytes);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(rows * c));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

namespace {
constexpr int kMoveThreads = 256, kMoveSlots = 32;
static_assert(kPage % kMoveSlots == 0, "a block stays within a page");

__device__ __forceinline__ void widen_e4m3(const uint2& r, float sc, float* x) {
  const uint32_t w[2] = {r.x, r.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = f32x2_of_f16x2(f16x2_from_e4m3x2(uint16_t(w[i >> 1] >> (16 * (i & 1)))));
    x[2 * i] = t.x * sc;
    x[2 * i + 1] = t.y * sc;
  }
}
}  // namespace

// A block moves 32 slots of one destination page and KV head (128 left an SM one or two blocks
// and their latencies at a few thousand slots: 13.8 us for 6750 of 4 heads widened), bound by the
// bytes read and written: 16-byte pieces, neighbouring threads on neighbouring pieces of a row, several in
// flight per thread (16 x 4000 bf16 slots of 4 heads: 65 us, 5.0 TB/s, the warps waiting for their loads
// alone).  SRC is the source's format; WIDE: the destination is bf16 (dims 0..63 of
// a key fp16), and a thread makes 8 dims of it.
template <int SRC, bool WIDE>
__global__ void __launch_bounds__(kMoveThreads) gather_kernel(const __grid_constant__ GatherParams p) {
  __shared__ long from[kMoveSlots];  // source entry (page * 128 + slot) of each destination slot, or -1
  const int s = blockIdx.z, g = blockIdx.y, j0 = blockIdx.x * kMoveSlots, tid = threadIdx.x;
  int count = p.counts[s];
  if (count < 0 || count > p.max_count) {
    if (g == 0 && blockIdx.x == 0 && tid == 0) atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
    count = min(count, p.max_count);  // (below 0: nothing to move)
  }
  const int n = min(kMoveSlots, count - j0);
  if (n <= 0) return;
  const int dst_at = j0 / kPage, slot0 = j0 % kPage;
  const int dst_page = dst_at < p.max_pages_dst ? p.table_dst[long(s) * p.max_pages_dst + dst_at] : -1;
  if (dst_page < 0 || dst_page >= p.num_pages_dst) {
    if (tid == 0) atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
    return;
  }
  if (tid < n) {
    const int at = p.idx ? p.idx[(long(s) * p.hkv + g) * p.idx_stride + j0 + tid] : j0 + tid;
    const int pi = at / kPage;
    const int page = at >= 0 && pi < p.max_pages_src ? p.table_src[long(s) * p.max_pages_src + pi] : -1;
    const bool ok = page >= 0 && page < p.num_pages_src;
    if (!ok) atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
    from[tid] = ok ? long(page) * kPage + at % kPage : -1;
  }
  __syncthreads();
  constexpr bool kI4 = SRC == MIMO_DTYPE_INT4;
  // row `entry` of KV head g of a wide or E4M3 cache, row bytes b; of a 4-bit block: its codes
  auto row_of = [&](auto* base, long entry, int b) { return base + (entry * p.hkv + g) * b; };
  auto block_of = [&](auto* base, long page, int b) { return base + (page * p.hkv + g) * (long(kPage) * b); };
  const long to0 = long(dst_page) * kPage + slot0;

  auto move = [&](const uint8_t* src, uint8_t* dst, int slot_bytes, int code_bytes) {
    // 16-byte pieces of the rows (codes)
    const int per = (kI4 ? code_bytes : slot_bytes) / 16, total = n * per;
#pragma unroll 4
    for (int i = tid; i < total; i += kMoveThreads) {
      const int r = i / per, c = i - r * per;
      const long f = from[r];
      if (f < 0) continue;
      const uint8_t* a = kI4 ? block_of(src, f / kPage, slot_bytes) + f % kPage * code_bytes : row_of(src, f, slot_bytes);
      uint8_t* b = kI4 ? block_of(dst, dst_page, slot_bytes) + (slot0 + r) * code_bytes : row_of(dst, to0 + r, slot_bytes);
      reinterpret_cast<uint4*>(b)[c] = __ldg(reinterpret_cast<const uint4*>(a) + c);
    }
    if constexpr (kI4) {  // the rows of scales, 4-byte pieces
      const int sb = slot_bytes - code_bytes, pw = sb / 4;
      for (int i = tid; i < n * pw; i += kMoveThreads) {
        const int r = i / pw, c = i - r * pw;
        const long f = from[r];
        if (f < 0) continue;
        const uint8_t* a = block_of(src, f / kPage, slot_bytes) + kPage * code_bytes + f % kPage * sb;
        uint8_t* b = block_of(dst, dst_page, slot_bytes) + kPage * code_bytes + (slot0 + r) * sb;
        reinterpret_cast<uint32_t*>(b)[c] = __ldg(reinterpret_cast<const uint32_t*>(a) + c);
      }
    }
  };
  // 8 dims a thread of a narrow row into bf16 (the first kRope dims of a key: fp16)
  auto widen = [&](const uint8_t* src, uint8_t* dst, int dims, bool key, float sc) {
    const int per = dims / 8, total = n * per;
    float amax = 0.f;
#pragma unroll 4
    for (int i = tid; i < total; i += kMoveThreads) {
      const int r = i / per, c = i - r * per;
      const long f = from[r];
      if (f < 0) continue;
      float x[8];
      if constexpr (kI4) {
        const int codes = dims / 2, slot_bytes = codes + dims / 16;
        const uint8_t* blk = block_of(src, f / kPage, slot_bytes);
        const int slot = int(f % kPage), word = key ? (c & 3) * 6 + (c >> 2) : c;
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(blk + slot * codes) + word);
        const float z = __half2float(reinterpret_cast<const __half*>(blk + kPage * codes)[slot * (dims / kI4Group) + (c >> 2)]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = float(int((w >> (4 * e)) & 15u) - 8) * z;
      } else {
        widen_e4m3(__ldg(reinterpret_cast<const uint2*>(row_of(src, f, dims)) + c), sc, x);
      }
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = key && c < kRope / 8 ? pack2_f16_sat(x[2 * e], x[2 * e + 1], amax) : pack2_bf16(x[2 * e], x[2 * e + 1]);
      reinterpret_cast<uint4*>(row_of(dst, to0 + r, 2 * dims))[c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (amax > kF16Max) atomicOr(p.status, MIMO_STATUS_RANGE);
  };
  if constexpr (WIDE) {
    widen(p.k_src, p.k_dst, kDqk, true, SRC == MIMO_DTYPE_FP8_E4M3 ? p.k_dequant[g] : 1.f);
    widen(p.v_src, p.v_dst, kDv, false, SRC == MIMO_DTYPE_FP8_E4M3 ? p.v_dequant[g] : 1.f);
  } else if constexpr (kI4) {
    move(p.k_src, p.k_dst, kI4KSlot, kI4KCodes);
    move(p.v_src, p.v_dst, kI4VSlot, kI4VCodes);
  } else {
    constexpr int e = SRC == MIMO_DTYPE_BF16 ? 2 : 1;
    move(p.k_src, p.k_dst, kDqk * e, 0);
    move(p.v_src, p.v_dst, kDv * e, 0);
  }
}

cudaError_t launch_gather(const GatherParams& p, cudaStream_t s) {
  const dim3 grid((p.max_count + kMoveSlots - 1) / kMoveSlots, p.hkv, p.num_seqs);
  if (p.out_dtype == p.cache_dtype) {
    if (p.cache_dtype == MIMO_DTYPE_BF16) gather_kernel<MIMO_DTYPE_BF16, false><<<grid, kMoveThreads, 0, s>>>(p);
    else if (p.cache_dtype == MIMO_DTYPE_FP8_E4M3) gather_kernel<MIMO_DTYPE_FP8_E4M3, false><<<grid, kMoveThreads, 0, s>>>(p);
    else gather_kernel<MIMO_DTYPE_INT4, false><<<grid, kMoveThreads, 0, s>>>(p);
  } else if (p.cache_dtype == MIMO_DTYPE_FP8_E4M3) {
    gather_kernel<MIMO_DTYPE_FP8_E4M3, true><<<grid, kMoveThreads, 0, s>>>(p);
  } else {
    gather_kernel<MIMO_DTYPE_INT4, true><<<grid, kMoveThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace mimo
