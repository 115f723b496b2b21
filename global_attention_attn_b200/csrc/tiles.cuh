// The line of key tiles of all (sequence, KV head) units, which persistent kernels cut into
// equal pieces whatever the mix of lengths, and the bulk copy its readers use.
#pragma once
#include <cstdint>

#include "internal.h"

namespace mimo {

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

// One warp: tbl[s] = tiles per KV head before sequence s (tbl[batch]: of all); tiles(s) of each.
template <class F>
__device__ __forceinline__ void tile_table(long long* tbl, int batch, int lane, F tiles) {
  long long carry = 0;
  if (lane == 0) tbl[0] = 0;
  for (int base = 0; base < batch; base += 32) {
    const int s = base + lane;
    long long n = s < batch ? tiles(s) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += u;
    }
    if (s < batch) tbl[s + 1] = carry + n;
    carry += __shfl_sync(0xffffffffu, n, 31);
  }
  __syncwarp();
}

// A position on the line: sequence s's heads hold hkv * (tbl[s + 1] - tbl[s]) tiles.
struct TileCursor {
  int s, g, t, nt;
};
__device__ __forceinline__ TileCursor cursor_at(const long long* tbl, int batch, int hkv, long long x) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tbl[mid] * hkv <= x) lo = mid;
    else hi = mid;
  }
  TileCursor c;
  c.s = lo;
  c.nt = int(tbl[lo + 1] - tbl[lo]);
  const unsigned rem = unsigned(x - tbl[lo] * hkv);  // (at most hkv * nt)
  c.g = int(rem / unsigned(c.nt));
  c.t = int(rem - c.g * unsigned(c.nt));
  return c;
}
// The next unit that has tiles (the caller knows there is one).
__device__ __forceinline__ void next_unit(const long long* tbl, int hkv, TileCursor& c) {
  c.t = 0;
  if (++c.g < hkv) return;
  c.g = 0;
  do {
    ++c.s;
    c.nt = int(tbl[c.s + 1] - tbl[c.s]);
  } while (c.nt == 0);
}

}  // namespace mimo
