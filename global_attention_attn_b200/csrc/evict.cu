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

// Scores as unsigned keys of the same order: -0 equals 0, NaN counts as -infinity.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;  // 11, 11 and 10 bits a pass

}  // namespace

// One cluster per (sequence, KV head) row.  The row is read once (4 bytes a slot, the floor) into
// the shared memory of the cluster's 1..8 CTAs; the need-th largest score is found by three
// histogram passes over it (bins summed over the cluster through distributed shared memory,
// every CTA drawing the same conclusion), then each CTA writes its part of the kept slots at the
// place that the counts of the parts before it give: ascending, equal scores lowest slot first.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ uint32_t keys[];  // this CTA's part of the row
  __shared__ __align__(16) uint32_t hist[kBins];
  __shared__ uint32_t warp_sum[kSelWarps + 1];
  __shared__ uint32_t found[2];               // bin and how many of it are wanted
  __shared__ uint32_t w_more[kSelWarps + 1], w_tie[kSelWarps + 1];
  __shared__ uint32_t part[2];                // this CTA's counts, for the CTAs behind it
  cg::cluster_group cl = cg::this_cluster();
  const int C = int(cl.num_blocks()), rank = int(cl.block_rank());
  const int row = blockIdx.x / C, s = row / p.hkv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int L = p.seq_lens[s];
  if (L < 0 || L > p.max_seq_len) {
    if (rank == 0 && tid == 0) atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
    L = max(0, min(L, p.max_seq_len));
  }
  const float* const src = p.scores + long(row) * p.score_stride;
  const int per = ((L + C - 1) / C + 31) & ~31;  // slots of a CTA
  const int lo = min(L, rank * per), n = min(L, lo + per) - lo;
  // the slots that stay whatever their score; all of a row that fits
  const bool all = L <= p.keep;
  const int first = all ? L : p.first, tail = all ? L : L - p.recent;  // candidates: [first, tail)
  int need = all ? 0 : p.keep - p.first - p.recent;
  for (int i = tid; i < n; i += kSelThreads) keys[i] = order_key(src[lo + i]);
  uint32_t prefix = 0, mask = 0;  // keys & mask == prefix are still in question
  const bool search = need > 0;   // (cluster-uniform: need and L are the row's)
  if (search) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i0 = warp * 32; i0 < n; i0 += kSelThreads) {
        const int i = i0 + lane, slot = lo + i;
        const bool in = i < n && slot >= first && slot < tail && (keys[i] & mask) == prefix;
        const uint32_t who = __ballot_sync(0xffffffffu, in);
        if (in) {
          const uint32_t bin = (keys[i] >> shift) & ((1u << bits) - 1);
          // equal bins of a warp (unattended slots all score 0) are added once
          const uint32_t same = __match_any_sync(who, bin);
          if (lane == __ffs(same) - 1) atomicAdd(&hist[bin], uint32_t(__popc(same)));
        }
      }
      cl.sync();
      // bins from the largest down, 4 a thread, summed over the cluster
      uint32_t h[4], sum = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = 0;
      for (int r = 0; r < C; ++r) {
        const uint4 v = *reinterpret_cast<const uint4*>(cl.map_shared_rank(hist, r) + kBins - 4 - 4 * tid);
        h[0] += v.w;
        h[1] += v.z;
        h[2] += v.y;
        h[3] += v.x;
      }
      sum = h[0] + h[1] + h[2] + h[3];
      uint32_t incl = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += u;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      uint32_t before = incl - sum;
      for (int w = 0; w < warp; ++w) before += warp_sum[w];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (before < uint32_t(need) && before + h[e] >= uint32_t(need)) {
          found[0] = uint32_t(kBins - 1 - 4 * tid - e);
          found[1] = uint32_t(need) - before;
        }
        before += h[e];
      }
      cl.sync();  // every CTA has read the bins before they are cleared
      prefix |= found[0] << shift;
      mask |= ((1u << bits) - 1) << shift;
      need = int(found[1]);
    }
  }
  __syncthreads();
  // prefix: the smallest score kept; need: how many of those that equal it, the first ones
  auto kind = [&](int i) {  // 2: stays, 1: equals the border, 0: goes
    const int slot = lo + i;
    if (slot < first || slot >= tail) return 2;
    if (!search) return 0;
    return keys[i] > prefix ? 2 : (keys[i] == prefix ? 1 : 0);
  };
  // a warp's contiguous range
  const int range = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int i_lo = min(n, warp * range), i_hi = min(n, i_lo + range);
  uint32_t more = 0, tie = 0;
  for (int i0 = i_lo; i0 < i_hi; i0 += 32) {
    const int k = i0 + lane < i_hi ? kind(i0 + lane) : 0;
    more += __popc(__ballot_sync(0xffffffffu, k == 2));
    tie += __popc(__ballot_sync(0xffffffffu, k == 1));
  }
  if (lane == 0) {
    w_more[warp] = more;
    w_tie[warp] = tie;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t m = 0, t = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      m += w_more[w];
      t += w_tie[w];
    }
    part[0] = m;
    part[1] = t;
  }
  cl.sync();
  more = tie = 0;
  for (int r = 0; r < rank; ++r) {
    const uint32_t* q = cl.map_shared_rank(part, r);
    more += q[0];
    tie += q[1];
  }
  for (int w = 0; w < warp; ++w) {
    more += w_more[w];
    tie += w_tie[w];
  }
  int32_t* const idx = p.idx + long(row) * p.keep;
  float* const out = p.scores_out ? p.scores_out + long(row) * p.keep : nullptr;
  const uint32_t below = (1u << lane) - 1;
  for (int i0 = i_lo; i0 < i_hi; i0 += 32) {
    const int k = i0 + lane < i_hi ? kind(i0 + lane) : 0;
    const uint32_t bm = __ballot_sync(0xffffffffu, k == 2), bt = __ballot_sync(0xffffffffu, k == 1);
    const uint32_t t = tie + __popc(bt & below);
    if (k == 2 || (k == 1 && t < uint32_t(need))) {
      const uint32_t j = more + __popc(bm & below) + min(t, uint32_t(need));
      idx[j] = lo + i0 + lane;
      if (out) out[j] = src[lo + i0 + lane];
    }
    more += __popc(bm);
    tie += __popc(bt);
  }
  const int count = min(L, p.keep);
  for (int j = count + rank * kSelThreads + tid; j < p.keep; j += C * kSelThreads) {
    idx[j] = -1;
    if (out) out[j] = 0.f;
  }
  if (rank == 0 && tid == 0 && row % p.hkv == 0) p.counts[s] = count;
  cl.sync();  // no CTA leaves while another reads its counts
}

cudaError_t launch_select(const SelectParams& p, cudaStream_t s) {
  int c = 1;  // CTAs per row: 4096 slots each at least, 8 at most
  while (c < 8 && c * 4096 < p.max_seq_len) c *= 2;
  const size_t bytes = size_t((((p.max_seq_len + c - 1) / c + 31) & ~31)) * 4;
  cudaError_t e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.num_seqs) * p.hkv * c);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, select_kernel, p);
}

namespace {
constexpr int kMoveThreads = 256;

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

// A block moves the slots of one destination page and KV head, bound by the bytes read and
// written: 16-byte pieces, neighbouring threads on neighbouring pieces of a row, several in
// flight per thread.  SRC is the source's format; WIDE: the destination is bf16 (dims 0..63 of
// a key fp16), and a thread makes 8 dims of it.
template <int SRC, bool WIDE>
__global__ void __launch_bounds__(kMoveThreads) gather_kernel(const __grid_constant__ GatherParams p) {
  __shared__ long from[kPage];  // source entry (page * 128 + slot) of each destination slot, or -1
  const int s = blockIdx.z, g = blockIdx.y, j0 = blockIdx.x * kPage, tid = threadIdx.x;
  int count = p.counts[s];
  if (count > p.max_count) {
    if (g == 0 && blockIdx.x == 0 && tid == 0) atomicOr(p.status, MIMO_STATUS_BAD_INDEX);
    count = p.max_count;
  }
  const int n = min(kPage, count - j0);
  if (n <= 0) return;
  const int dst_page = blockIdx.x < p.max_pages_dst ? p.table_dst[long(s) * p.max_pages_dst + blockIdx.x] : -1;
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
  const long to0 = long(dst_page) * kPage;

  auto move = [&](const uint8_t* src, uint8_t* dst, int slot_bytes, int code_bytes) {
    // 16-byte pieces of the rows (codes)
    const int per = (kI4 ? code_bytes : slot_bytes) / 16, total = n * per;
#pragma unroll 4
    for (int i = tid; i < total; i += kMoveThreads) {
      const int r = i / per, c = i - r * per;
      const long f = from[r];
      if (f < 0) continue;
      const uint8_t* a = kI4 ? block_of(src, f / kPage, slot_bytes) + f % kPage * code_bytes : row_of(src, f, slot_bytes);
      uint8_t* b = kI4 ? block_of(dst, dst_page, slot_bytes) + r * code_bytes : row_of(dst, to0 + r, slot_bytes);
      reinterpret_cast<uint4*>(b)[c] = __ldg(reinterpret_cast<const uint4*>(a) + c);
    }
    if constexpr (kI4) {  // the rows of scales, 4-byte pieces
      const int sb = slot_bytes - code_bytes, pw = sb / 4;
      for (int i = tid; i < n * pw; i += kMoveThreads) {
        const int r = i / pw, c = i - r * pw;
        const long f = from[r];
        if (f < 0) continue;
        const uint8_t* a = block_of(src, f / kPage, slot_bytes) + kPage * code_bytes + f % kPage * sb;
        uint8_t* b = block_of(dst, dst_page, slot_bytes) + kPage * code_bytes + r * sb;
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
  const dim3 grid((p.max_count + kPage - 1) / kPage, p.hkv, p.num_seqs);
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
