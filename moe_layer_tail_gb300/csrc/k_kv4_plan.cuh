// k_kv4_plan.cuh -- how the attention over the MXFP4 cache cuts its work: items, ranges, parts.
// Internal to libmoe_tail.so.
//
// A work item is one request's query rows of one kv head, RN rows at a time; its tiles of 16
// tokens, laid end to end over all items, are cut into equal ranges, one per CTA.  A part is what
// an item and a range have in common.  In front of each item lie kItemTiles places that stand for
// the time it takes to open and close one, so that a CTA of many short items gets fewer tiles; a
// range that ends among them leaves the item to the next.
#pragma once

#include "k_kv4.cuh"

namespace kv4 {

constexpr int kMinTiles = 8;    // of a range
constexpr int kItemTiles = 36;  // (32 requests up to 32768 tokens: 184 us without, 172 with 12, 163 with 36, 164 with 60)

struct Req {
  int L, nq, rt;   // cache length, query rows, items per kv head
  int ns, off, T;  // tiles of first tokens, then off further; tiles of the whole length
  int n;           // tiles of an item
};

// A request's work; nq = 0 (and *bits) when its row starts are not usable.
__device__ __forceinline__ Req req_of(const AttnArgs& a, int rn, int L, int rs, int re, int* bits) {
  Req q;
  if (L < 0 || L > a.max_len) *bits |= kStatusBadLength;
  q.L = max(0, min(L, a.max_len));
  if (rs < 0 || re < rs || re > a.rows) *bits |= kStatusBadLength, re = rs;
  q.nq = re - rs;
  q.rt = (int)(((int64_t)q.nq * a.G + rn - 1) / rn);
  q.T = (int)(((uint32_t)q.L + 15u) >> 4);
  q.ns = q.off = 0;
  int fw = 0;
  if (a.window > 0) {
    const int64_t f = (int64_t)q.L - q.nq - a.window + 1;  // first token of the first row's window
    fw = f > 0 ? (int)(f >> 4) : 0;
    q.ns = (int)min((int64_t)fw, ((int64_t)a.sinks + 15) >> 4);
    q.off = fw - q.ns;
  }
  q.n = max(1, q.ns + q.T - fw);
  return q;
}

// Sums the work of all requests: pre[r] = places before request r (shared), the lengths and row
// starts beside it.  One warp does it, 32 requests at a time; `first` are the lengths and starts of
// the first 32, loaded ahead.  The caller synchronises before the results are read.
struct PlanLoad {
  int L, rs, re;
};
__device__ __forceinline__ PlanLoad plan_load(const AttnArgs& a, int r) {
  PlanLoad p = {0, 0, 0};
  if (r < a.reqs) p.L = a.kv_lens[r], p.rs = a.row_starts[r], p.re = a.row_starts[r + 1];
  return p;
}
__device__ __forceinline__ uint64_t plan(const AttnArgs& a, int rn, PlanLoad next, uint32_t* pre, int* lens,
                                         int* starts, int* bits) {
  const int lane = threadIdx.x & 31;
  uint64_t base = 0;
  for (int r0 = 0; r0 < a.reqs; r0 += 32) {
    const int r = r0 + lane;
    const PlanLoad p = next;
    next = plan_load(a, r + 32);
    uint64_t v = 0;
    if (r < a.reqs) {
      const Req q = req_of(a, rn, p.L, p.rs, p.re, bits);
      v = (uint64_t)q.rt * (uint32_t)a.heads * (uint32_t)(q.n + kItemTiles);
      lens[r] = p.L;
      starts[r] = p.rs;
      if (r == a.reqs - 1) starts[a.reqs] = p.re;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t w = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v += w;
    }
    if (r < a.reqs) pre[r + 1] = (uint32_t)(base + v);
    base += __shfl_sync(~0u, v, 31);
  }
  if (lane == 0) pre[0] = 0;
  return base;
}
__device__ __forceinline__ uint32_t range_tiles(uint64_t total, int ctas) {
  return max((uint32_t)((total + ctas - 1) / ctas), (uint32_t)kMinTiles);
}
__device__ __forceinline__ int find_req(const uint32_t* pre, int reqs, uint32_t u) {
  int lo = 0, hi = reqs - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (pre[m] <= u) lo = m; else hi = m - 1;
  }
  while (lo < reqs - 1 && pre[lo + 1] <= u) ++lo;  // (requests without work)
  return lo;
}

// The part of the range [u, u1) that lies in its first item.
struct Seg {
  int r, h, j;      // request, kv head, block of RN rows
  int k0, k1;       // its tiles of the item's q.n
  uint32_t places;  // how far it reaches
  uint32_t item;    // the item's first place
  Req q;
};
__device__ __forceinline__ Seg open_seg(const AttnArgs& a, int rn, const uint32_t* pre,
                                        const int* lens, const int* starts, int r, uint32_t u,
                                        uint32_t u1) {
  Seg s;
  while (r < a.reqs - 1 && pre[r + 1] <= u) ++r;
  int bits = 0;
  s.r = r;
  s.q = req_of(a, rn, lens[r], starts[r], starts[r + 1], &bits);
  const uint32_t local = u - pre[r], n = (uint32_t)(s.q.n + kItemTiles), item = local / n, at = local - item * n;
  s.item = u - at;
  s.h = (int)(item / (uint32_t)s.q.rt);
  s.j = (int)(item - (uint32_t)s.h * (uint32_t)s.q.rt);
  s.places = min(n - at, u1 - u);
  s.k0 = max((int)at - kItemTiles, 0);
  s.k1 = max((int)(at + s.places) - kItemTiles, 0);
  return s;
}
// The end of a range [u0, u1) without an item that it would only open.
__device__ __forceinline__ uint32_t range_end(const AttnArgs& a, int rn, const uint32_t* pre, const int* lens,
                                              const int* starts, uint32_t u0, uint32_t u1) {
  if (u0 == u1) return u1;
  const int r = find_req(pre, a.reqs, u1 - 1);
  int bits = 0;
  const Req q = req_of(a, rn, lens[r], starts[r], starts[r + 1], &bits);
  const uint32_t at = (u1 - 1 - pre[r]) % (uint32_t)(q.n + kItemTiles);
  return at < (uint32_t)kItemTiles ? (uint32_t)max((int64_t)u0, (int64_t)u1 - 1 - at) : u1;
}

}  // namespace kv4
