// k_kv4_attn.cu -- attention of a step's query rows over the paged MXFP4 cache (kv4_attn.h).
//
//   out[i] = sum_j p_j V_j / sum_j p_j,  p_j = 2^(scale log2(e) q_i . K_j - m_i)
//
// in one pass over the cache.  A work item is one request's query rows of one kv head (RN rows
// at a time; the query heads that share a kv head are rows of the same item, so the cache is read
// once for all of them); its tiles of 16 tokens, laid end to end over all items, are cut into
// equal ranges, one per resident CTA, so that ragged lengths, one long request and many short
// ones all load every SM the same.  An item that lies in one range is written by its CTA; the
// others leave an average and (max, sum) per row and part in the workspace, which a second
// launch joins (started early by programmatic dependent launch, it waits only for the first).
//
// Each of a CTA's four warps walks its own tiles (every fourth of the range) without any barrier:
// a ring of tiles per warp in shared memory, filled by bulk copies (a tile is one contiguous
// piece of the cache), each on its own mbarrier.  Per tile (tokens as M, query rows as N):
//   S^T [16 x RN] = K Q^T: a block of 32 channels at a time, mma.m16n8k16 on the E2M1 codes
//       converted to f16 (exact) and q as f16; the block's product times the key scale, fp32;
//   P^T = 2^(S - m), fp32, packed to f16 (2^11 times the numerator, so that the small ones keep
//       their bits); a row's reference m moves only when a score passes it by 3 (a warp vote),
//       which leaves the running sums to be rescaled rarely instead of at every tile;
//   O^T [D x RN] += V^T P^T: P^T transposed in registers (movmatrix), times the value scale of
//       each block of 32 channels (a power of two, exact in f16 while the block's scales lie in a
//       window of 16 octaves; a tile outside goes through as many windows as it takes), the codes
//       of two neighbouring tokens merged to one E2M1 pair before their conversion.
// The cache stores codes and scales in the order in which the lanes use them: every shared-memory
// read is 16 bytes wide (8 or 4 for the scales of small heads) and free of bank conflicts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "k_kv4.cuh"
#include "k_stream_common.cuh"

namespace kv4 {

using mtail::bulk_load;
using mtail::mbar_arrive;
using mtail::mbar_expect_tx;
using mtail::mbar_init;
using mtail::mbar_try_wait;
using mtail::mma_f16;
using mtail::mma_f16_z;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMinTiles = 8;               // of a CTA's range
constexpr int64_t kBudgetClocks = 200000000;  // of a wait for a tile, about 0.1 s
constexpr float kLow = -3.0e38f;           // a row's reference before its first score

template <int D, int NT>
struct Geo {
  static constexpr int RN = 8 * NT;
  static constexpr int NB = D / 32;
  static constexpr int kTile = 17 * D;
  static constexpr int kStages = D == 256 ? 3 : 4;
  static constexpr int kQRow = 2 * D + 64;  // bytes: odd rows 64 bytes further, no conflicts
  static constexpr bool kQReg = D * NT <= 128;
  static constexpr int kORegs = NB * 2 * NT * 4;
  static constexpr int kBlocks = kORegs >= 128 ? 2 : kORegs >= 64 ? 3 : 4;  // CTAs per SM
  // shared memory: ring, two merge buffers, queries, then the small arrays
  static constexpr int kRing = kWarps * kStages * kTile;
  static constexpr int kMerge = 2 * kORegs * 32 * 4;
  static constexpr int kQ = RN * kQRow;
  static constexpr int kSmall = RN * 8 /* rowpos, qs */ + kWarps * RN * 8 /* m, l */ +
                                kWarps * NB * 4 /* windows */ + kWarps * kStages * 8 +
                                kWarps * 36 * 8 /* queues and walks */ + 64 /* notes */;
  static constexpr size_t smem(int reqs) {
    return (size_t)kRing + kMerge + kQ + kSmall + (size_t)(3 * reqs + 2) * 4;
  }
};

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

// Sums the work of all requests: pre[r] = tiles before request r (shared), the lengths and row
// starts beside it.  Returns all tiles (the same in every thread).
__device__ __forceinline__ uint64_t plan(const AttnArgs& a, int rn, uint32_t* pre, int* lens,
                                         int* starts, uint64_t* wsum, int* bits) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t base = 0;
  for (int r0 = 0; r0 < a.reqs; r0 += kThreads) {
    const int r = r0 + tid;
    uint64_t v = 0;
    if (r < a.reqs) {
      const int L = a.kv_lens[r], rs = a.row_starts[r], re = a.row_starts[r + 1];
      const Req q = req_of(a, rn, L, rs, re, bits);
      v = (uint64_t)q.rt * (uint32_t)a.heads * (uint32_t)q.n;
      lens[r] = L;
      starts[r] = rs;
      if (r == a.reqs - 1) starts[a.reqs] = re;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t w = __shfl_up_sync(~0u, v, o);
      if (lane >= o) v += w;
    }
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    uint64_t all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) v += wsum[w];
      all += wsum[w];
    }
    if (r < a.reqs) pre[r + 1] = (uint32_t)(base + v);
    base += all;
    __syncthreads();
  }
  if (tid == 0) pre[0] = 0;
  __syncthreads();
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

// One item's part of a CTA's range.
struct Seg {
  int r, h, j;      // request, kv head, block of RN rows
  int k0, k1;       // its tiles of the item's q.n
  uint32_t item;    // the range-wide number of the item's first tile
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
  const uint32_t local = u - pre[r], item = local / (uint32_t)s.q.n;
  s.k0 = (int)(local - item * (uint32_t)s.q.n);
  s.item = u - (uint32_t)s.k0;
  s.h = (int)(item / (uint32_t)s.q.rt);
  s.j = (int)(item - (uint32_t)s.h * (uint32_t)s.q.rt);
  s.k1 = (int)min((uint32_t)s.q.n, (uint32_t)s.k0 + (u1 - u));
  return s;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// bits of y where the mask has ones, of x elsewhere
__device__ __forceinline__ uint32_t select_bits(uint32_t m, uint32_t x, uint32_t y) {
  return (x & ~m) | (y & m);
}
// nonzero where a byte of w is 255
__device__ __forceinline__ uint32_t has_ff(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & w & 0x80808080u;
}

// Bounded wait for a tile: false when the budget ran out.
__device__ __forceinline__ bool tile_wait(uint64_t* b, uint32_t parity) {
  if (mbar_try_wait(b, parity)) return true;
  const int64_t t0 = clock64();
  do {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(b, parity)) return true;
  } while (clock64() - t0 < kBudgetClocks);
  return false;
}

// What a warp keeps of the item it works on.
template <int D, int NT>
struct State {
  float o[D / 32][2][NT][4];  // [block][16 channels][8 rows]: channels 4 g + 2 mt + {0, 0, 1, 1}
                              // of the block, rows 8 nt + 2 c + {0, 1, 0, 1}
  float m[NT][2], l[NT][2];   // reference (less 11) and this lane's share of the sum
  uint32_t lo4[D / 32];       // window [lo, lo + 15] of the block's value scales, lo in each byte:
                              // o = sum * 2^(127 - 14 - lo)
  bool placed;                // the windows stand where the item's scales are
};

template <int D, int NT>
__device__ __forceinline__ void scale_block(State<D, NT>& st, int b, float f) {
#pragma unroll
  for (int mt = 0; mt < 2; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[b][mt][nt][e] *= f;
}

// One tile of 16 tokens in shared memory.  partial: some of its (token, row) pairs are not seen.
template <int D, int NT>
__device__ __forceinline__ void tile_step(State<D, NT>& st, const uint8_t* tp, const uint8_t* sq,
                                          const uint32_t (&qr)[Geo<D, NT>::kQReg ? D / 32 : 1][NT][4],
                                          const float (&qs)[NT][2], const int* rowpos, bool partial,
                                          int t0, int pmax, int window, int sinks) {
  constexpr int NB = D / 32;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint32_t kw[2 * NB], ks[NB / 2], vs[NB];
#pragma unroll
  for (int v = 0; v < D / 64; ++v) {
    const uint4 u = *reinterpret_cast<const uint4*>(tp + v * 512 + lane * 16);
    kw[4 * v] = u.x, kw[4 * v + 1] = u.y, kw[4 * v + 2] = u.z, kw[4 * v + 3] = u.w;
  }
  // key scales of tokens g and g + 8: byte hh NB + b; value scales of tokens 2c, 2c+1, 2c+8, 2c+9
  const uint8_t* kp = tp + 16 * D + g * (D / 16);
  const uint8_t* vp = tp + 16 * D + D / 2 + c * (D / 8);
  if constexpr (NB == 2) {
    ks[0] = *reinterpret_cast<const uint32_t*>(kp);
    const uint2 u = *reinterpret_cast<const uint2*>(vp);
    vs[0] = u.x, vs[1] = u.y;
  } else if constexpr (NB == 4) {
    const uint2 k2 = *reinterpret_cast<const uint2*>(kp);
    ks[0] = k2.x, ks[1] = k2.y;
    const uint4 u = *reinterpret_cast<const uint4*>(vp);
    vs[0] = u.x, vs[1] = u.y, vs[2] = u.z, vs[3] = u.w;
  } else {
    const uint4 k4 = *reinterpret_cast<const uint4*>(kp);
    ks[0] = k4.x, ks[1] = k4.y, ks[2] = k4.z, ks[3] = k4.w;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint4 u = *reinterpret_cast<const uint4*>(vp + 16 * v);
      vs[4 * v] = u.x, vs[4 * v + 1] = u.y, vs[4 * v + 2] = u.z, vs[4 * v + 3] = u.w;
    }
  }
  // slots past the last row's position may hold anything: their value scales are put in the window
  uint32_t past = 0;
  if (partial) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t0 + 2 * c + (i & 1) + 8 * (i >> 1) > pmax) past |= 0xFFu << (8 * i);
#pragma unroll
    for (int b = 0; b < NB; ++b) vs[b] = select_bits(past, vs[b], st.lo4[b]);
  }
  // a NaN scale, or a value scale outside its block's window [lo, lo + 15] (lo <= 239, so that
  // 255 is always outside; a byte below lo borrows from the next one, but is itself outside)
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < NB / 2; ++i) bad |= has_ff(ks[i]);
#pragma unroll
  for (int b = 0; b < NB; ++b) bad |= (vs[b] - st.lo4[b]) & 0xF0F0F0F0u;
  bool nan_key = false, outside = false;
  if (!st.placed || __any_sync(~0u, bad != 0)) {
    bad = 0;
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) bad |= has_ff(ks[i]);
    nan_key = __any_sync(~0u, bad != 0);
    // place the windows anew: the first tile of an item, or scales far above all so far
    bad = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      int hi = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = (int)(vs[b] >> (8 * i) & 255);
        if (v != 255 && !(past >> (8 * i) & 1)) hi = max(hi, v);
      }
      hi = __reduce_max_sync(~0u, hi);
      const int old = (int)(st.lo4[b] & 255);
      if (!st.placed || hi > old + 15) {
        const int lo = min(max(hi - 10, 0), 239);
        if (st.placed) scale_block(st, b, exp2f((float)(old - lo)));
        st.lo4[b] = (uint32_t)lo * 0x01010101u;
      }
      vs[b] = select_bits(past, vs[b], st.lo4[b]);
      bad |= (vs[b] - st.lo4[b]) & 0xF0F0F0F0u;
    }
    st.placed = true;
    outside = __any_sync(~0u, bad != 0);
  }

  // ---- S^T = K Q^T
  float s[NT][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    uint32_t x[4], y[4];
    mtail::e2m1x8_to_f16x2(kw[b], x[0], x[1], x[2], x[3]);
    mtail::e2m1x8_to_f16x2(kw[NB + b], y[0], y[1], y[2], y[3]);
    const float f0 = mtail::e8m0_byte(ks[b / 4], b % 4);
    const float f1 = mtail::e8m0_byte(ks[(NB + b) / 4], (NB + b) % 4);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t q0, q1, q2, q3;
      if constexpr (Geo<D, NT>::kQReg) {
        q0 = qr[b][nt][0], q1 = qr[b][nt][1], q2 = qr[b][nt][2], q3 = qr[b][nt][3];
      } else {
        const uint4 u = *reinterpret_cast<const uint4*>(sq + (8 * nt + g) * Geo<D, NT>::kQRow +
                                                        64 * b + 16 * c);
        q0 = u.x, q1 = u.y, q2 = u.z, q3 = u.w;
      }
      float acc[4];
      mma_f16_z(acc, x[0], y[0], x[1], y[1], q0, q1);
      mma_f16(acc, x[2], y[2], x[3], y[3], q2, q3);
      s[nt][0] = b ? fmaf(acc[0], f0, s[nt][0]) : acc[0] * f0;
      s[nt][1] = b ? fmaf(acc[1], f0, s[nt][1]) : acc[1] * f0;
      s[nt][2] = b ? fmaf(acc[2], f1, s[nt][2]) : acc[2] * f1;
      s[nt][3] = b ? fmaf(acc[3], f1, s[nt][3]) : acc[3] * f1;
    }
  }
  if (nan_key) {  // (the scale byte 255 came in as an infinity)
    bool n0 = false, n1 = false;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      n0 = n0 || (ks[b / 4] >> (8 * (b % 4)) & 255) == 255;
      n1 = n1 || (ks[(NB + b) / 4] >> (8 * ((NB + b) % 4)) & 255) == 255;
    }
    const float nan = __uint_as_float(0x7FC00000u);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (n0) s[nt][0] = s[nt][1] = nan;
      if (n1) s[nt][2] = s[nt][3] = nan;
    }
  }

  // ---- P^T = 2^(S - m)
  uint32_t hidden = 0;  // bit nt * 4 + e: the pair is masked
  if (partial) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int p = rowpos[8 * nt + 2 * c + (e & 1)], t = t0 + g + 8 * (e >> 1);
        const bool see = t <= p && (window == 0 || t > p - window || t < sinks);
        if (!see) hidden |= 1u << (nt * 4 + e), s[nt][e] = -INFINITY;
      }
  }
  float x[NT][4], top = -INFINITY;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[nt][e] = fmaf(s[nt][e], qs[nt][e & 1], -st.m[nt][e & 1]);
      top = fmaxf(top, x[nt][e]);
    }
  if (__any_sync(~0u, top > 14.f)) {  // 2^14 * 2^(15 + 1 - 15) stays below the f16 maximum
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float y0 = s[nt][e] * qs[nt][e], y1 = s[nt][e + 2] * qs[nt][e];
        float t = fmaxf(y0, y1);
        t = fmaxf(t, __shfl_xor_sync(~0u, t, 4));
        t = fmaxf(t, __shfl_xor_sync(~0u, t, 8));
        t = fmaxf(t, __shfl_xor_sync(~0u, t, 16));
        const float m = fmaxf(st.m[nt][e], t - 11.f);
        const float f = ex2(st.m[nt][e] - m);
        st.m[nt][e] = m;
        st.l[nt][e] *= f;
        x[nt][e] = y0 - m;
        x[nt][e + 2] = y1 - m;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            st.o[b][mt][nt][e] *= f;
            st.o[b][mt][nt][e + 2] *= f;
          }
      }
  }
  uint32_t pb[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[e] = ex2(x[nt][e]);
      st.l[nt][e & 1] += p[e];
    }
    if (partial) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (hidden >> (nt * 4 + e) & 1) p[e] = -0.f;  // marks a masked pair
    }
    pb[nt][0] = transpose8(pack_f16(p[0], p[1]));
    pb[nt][1] = transpose8(pack_f16(p[2], p[3]));
  }

  // ---- O^T += V^T P^T
  uint32_t vw[D / 16];  // words of (h, o): [2 h + o][D / 64]
#pragma unroll
  for (int v = 0; v < D / 64; ++v) {
    const uint4 u = *reinterpret_cast<const uint4*>(tp + 8 * D + v * 512 + lane * 16);
    vw[4 * v] = u.x, vw[4 * v + 1] = u.y, vw[4 * v + 2] = u.z, vw[4 * v + 3] = u.w;
  }
#pragma unroll
  for (int bp = 0; bp < D / 64; ++bp) {
    // X: channels j = 0, 2 of blocks 2 bp, 2 bp + 1 for the token pair, Y: channels j = 1, 3
    uint32_t X[2][4], Y[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w0 = vw[(2 * h) * (D / 64) + bp], w1 = vw[(2 * h + 1) * (D / 64) + bp];
      mtail::e2m1x8_to_f16x2(select_bits(0xF0F0F0F0u, w0, w1 << 4), X[h][0], X[h][1], X[h][2], X[h][3]);
      mtail::e2m1x8_to_f16x2(select_bits(0xF0F0F0F0u, w0 >> 4, w1), Y[h][0], Y[h][1], Y[h][2], Y[h][3]);
    }
#pragma unroll
    for (int bb = 0; bb < 2; ++bb) {
      const int b = 2 * bp + bb, i = 2 * bb;
      const uint32_t s0 = __byte_perm(vs[b], 0, 0x4140), s1 = __byte_perm(vs[b], 0, 0x4342);
      if (!outside) {
        // f16 with the exponent field s - lo + 1: 2^(s - lo - 14)
        const uint32_t add = 0x04000400u - (st.lo4[b] & 0x00FF00FFu) * 1024u;
        const uint32_t f0 = s0 * 1024u + add, f1 = s1 * 1024u + add;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = mul_f16x2(pb[nt][0], f0), b1 = mul_f16x2(pb[nt][1], f1);
          mma_f16(st.o[b][0][nt], X[0][i], Y[0][i], X[1][i], Y[1][i], b0, b1);
          mma_f16(st.o[b][1][nt], X[0][i + 1], Y[0][i + 1], X[1][i + 1], Y[1][i + 1], b0, b1);
        }
      } else {
        // window after window, from the largest scale down; NaN scales with the first
        const int sv[4] = {(int)(s0 & 255), (int)(s0 >> 16), (int)(s1 & 255), (int)(s1 >> 16)};
        bool first = true;
        int below = 255;
#pragma unroll 1
        for (int pass = 0; pass < 17; ++pass) {  // 255 / 16 windows at most
          int hi = -1;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (sv[k] < below) hi = max(hi, sv[k]);
          hi = __reduce_max_sync(~0u, hi);
          if (hi < 0 && !first) break;
          const int lo = hi - 15;  // (hi = -1: only NaN scales)
          uint32_t f[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            f[k] = first && sv[k] == 255 ? 0x7E00u
                   : sv[k] < below && sv[k] >= lo ? (uint32_t)(sv[k] - lo + 1) << 10 : 0u;
          const float back = exp2f((float)(lo - (int)(st.lo4[b] & 255)));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t pp[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t r = mul_f16x2(pb[nt][k], f[2 * k] | f[2 * k + 1] << 16);
              // a masked pair stays out even where the scale is NaN
              if ((pb[nt][k] & 0xFFFFu) == 0x8000u) r &= 0xFFFF0000u;
              if ((pb[nt][k] >> 16) == 0x8000u) r &= 0x0000FFFFu;
              pp[k] = r;
            }
            float t0v[4], t1v[4];
            mma_f16_z(t0v, X[0][i], Y[0][i], X[1][i], Y[1][i], pp[0], pp[1]);
            mma_f16_z(t1v, X[0][i + 1], Y[0][i + 1], X[1][i + 1], Y[1][i + 1], pp[0], pp[1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              st.o[b][0][nt][e] = fmaf(t0v[e], back, st.o[b][0][nt][e]);
              st.o[b][1][nt][e] = fmaf(t1v[e], back, st.o[b][1][nt][e]);
            }
          }
          first = false;
          below = lo;
        }
      }
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, (Geo<D, NT>::kBlocks))
k_kv4_attn(const __grid_constant__ AttnArgs a) {
  using G = Geo<D, NT>;
  constexpr int RN = G::RN, NB = G::NB;
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ uint64_t wsum[kWarps];
  uint8_t* ring = sm;
  float* merge = reinterpret_cast<float*>(sm + G::kRing);
  uint8_t* sq = sm + G::kRing + G::kMerge;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sq + G::kQ);
  int64_t* queues = reinterpret_cast<int64_t*>(bars + kWarps * G::kStages);
  int* notes = reinterpret_cast<int*>(queues + kWarps * 36);
  int* rowpos = notes + 16;
  float* sqs = reinterpret_cast<float*>(rowpos + RN);
  float* xm = sqs + RN;                  // [warp][RN]
  float* xl = xm + kWarps * RN;          // [warp][RN]
  int* xlo = reinterpret_cast<int*>(xl + kWarps * RN);  // [warp][NB]
  uint32_t* pre = reinterpret_cast<uint32_t*>(xlo + kWarps * NB);
  int* lens = reinterpret_cast<int*>(pre + a.reqs + 1);
  int* starts = lens + a.reqs;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  mtail::pdl_trigger();  // the joining launch may line up; it waits for this one to end

  int bits = 0;
  const uint64_t total64 = plan(a, RN, pre, lens, starts, wsum, &bits);
  if (total64 > 0x7FFFFFFFull) bits |= kStatusBadLength;
  if (blockIdx.x == 0 && bits && a.status) atomicOr(a.status, bits);
  if (total64 > 0x7FFFFFFFull) return;
  const uint32_t total = (uint32_t)total64, per = range_tiles(total64, a.ctas);
  const uint64_t u0w = (uint64_t)blockIdx.x * per;
  if (u0w >= total) return;
  const uint32_t u0 = (uint32_t)u0w, u1 = min(total, u0 + per);

  uint64_t* bar = bars + warp * G::kStages;
  uint8_t* wring = ring + warp * G::kStages * G::kTile;
  if (lane == 0) {
    for (int i = 0; i < G::kStages; ++i) mbar_init(bar + i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  __syncwarp();

  // ---- the copies of this warp's tiles, running ahead of the arithmetic by up to kStages tiles.
  // A queue holds where the next (up to 32) tiles of the warp stand in the cache, one lane having
  // looked up each; it is filled again, from the same or the range's next part, when it is empty.
  // The walk itself (where its part begins in the range, the part's next tile of this warp or -1,
  // the request) waits in shared memory: registers that the arithmetic needs.
  int64_t* queue = queues + warp * 36;
  int* walk = reinterpret_cast<int*>(queue + 32);
  const int r0 = find_req(pre, a.reqs, u0);
  if (lane == 0) walk[0] = (int)u0, walk[1] = -1, walk[2] = r0;
  __syncwarp();
  int qn = 0, qi = 0;
  uint32_t badmask = 0;  // stages whose tile has no page
  auto refill = [&]() {
    qn = qi = 0;
    uint32_t pu = (uint32_t)walk[0];
    int pk = walk[1], r = walk[2];
    while (pu < u1) {
      const Seg s = open_seg(a, RN, pre, lens, starts, r, pu, u1);
      r = s.r;
      const int k = pk < 0 ? s.k0 + warp : pk;
      const int n = k < s.k1 ? min(32, (s.k1 - k + kWarps - 1) / kWarps) : 0;
      if (lane < n) {
        const int kk = k + kWarps * lane, tile = kk < s.q.ns ? kk : kk + s.q.off;
        int64_t at = -1;
        if (tile < s.q.T) {
          const int e = (int)(((uint64_t)(uint32_t)tile * a.page_magic) >> 34);
          const int page = a.table[s.r * a.stride + e];
          if ((uint64_t)(int64_t)page < (uint64_t)a.n_pages)
            at = (((int64_t)page * a.heads + s.h) * a.page_tiles + (tile - e * a.page_tiles)) * G::kTile;
          else if (a.status)
            atomicOr(a.status, kStatusBadPage);
        }
        queue[lane] = at;
      }
      pk = k + kWarps * n;
      if (pk >= s.k1) pu += (uint32_t)(s.k1 - s.k0), pk = -1;
      if (n) {
        qn = n;
        break;
      }
    }
    __syncwarp();
    if (lane == 0) walk[0] = (int)pu, walk[1] = pk, walk[2] = r;
    __syncwarp();
  };
  auto issue = [&](int stage) {
    if (qi == qn) refill();
    if (qn == 0) return;
    const int64_t at = queue[qi++];
    badmask = at >= 0 ? badmask & ~(1u << stage) : badmask | 1u << stage;
    if (lane == 0) {
      if (at >= 0) {
        mbar_expect_tx(bar + stage, G::kTile);
        bulk_load(wring + stage * G::kTile, a.cache + at, G::kTile, bar + stage);
      } else {
        mbar_arrive(bar + stage);
      }
    }
    __syncwarp();
  };
  for (int i = 0; i < G::kStages; ++i) issue(i);

  int stage = 0;
  uint32_t phase = 0;
  bool dead = false;

  State<D, NT> st;
  uint32_t qr[G::kQReg ? NB : 1][NT][4];
  float qs[NT][2];

  int r = r0;
  int* part = notes;
  for (uint32_t u = u0; u < u1;) {
    const Seg s = open_seg(a, RN, pre, lens, starts, r, u, u1);
    const int row0 = starts[s.r];
    const int nrow = min(RN, s.q.nq * a.G - s.j * RN);  // rows of this item
    const int first = s.j * RN;
    if (tid == 0) {  // for the end of the part
      part[0] = row0, part[1] = nrow, part[2] = first, part[3] = s.h;
      part[4] = s.k0 == 0 ? 1 : 0, part[5] = s.k0 == 0 && s.k1 == s.q.n ? 1 : 0;
      part[6] = (int)(u + (uint32_t)(s.k1 - s.k0)), part[7] = s.r;
    }

    // ---- the item's queries: f16 times a power of two for each row
#pragma unroll 1
    for (int i = warp; i < RN; i += kWarps) {
      constexpr int E = D / 32;  // channels of a lane
      float x[E];
      const int rho = first + i, tok = rho / a.G;
#pragma unroll
      for (int k = 0; k < E; ++k) x[k] = 0.f;
      if (i < nrow) {
        const uint16_t* p = a.q + (row0 + tok) * a.ldq + (int64_t)(s.h * a.G + rho - tok * a.G) * D + lane * E;
        uint32_t w[E / 2];
        if constexpr (E == 2) {
          w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (E == 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(p);
          w[0] = v.x, w[1] = v.y;
        } else {
          const uint4 v = *reinterpret_cast<const uint4*>(p);
          w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < E / 2; ++k) x[2 * k] = mtail::bf16_lo(w[k]), x[2 * k + 1] = mtail::bf16_hi(w[k]);
      }
      uint32_t ab = 0;
#pragma unroll
      for (int k = 0; k < E; ++k) ab = max(ab, __float_as_uint(x[k]) & 0x7FFFFFFFu);
      ab = __reduce_max_sync(~0u, ab);
      // largest magnitude to [2^14, 2^15); rows with an infinity or a NaN are left as they are
      const int ex = ab >= 0x7F800000u ? 14 : max((int)(ab >> 23), 1) - 127;
      const int up = min(14 - ex, 110), up1 = up / 2;
      const float f1 = mtail::exp2_int(up1), f2 = mtail::exp2_int(up - up1);
      uint8_t* dst = sq + i * G::kQRow + lane * E * 2;
#pragma unroll
      for (int k = 0; k < E / 2; ++k)
        reinterpret_cast<uint32_t*>(dst)[k] = pack_f16(x[2 * k] * f1 * f2, x[2 * k + 1] * f1 * f2);
      if (lane == 0) {
        rowpos[i] = i < nrow ? s.q.L - s.q.nq + tok : INT32_MIN / 2;
        sqs[i] = fmaxf(a.scale_log2 * mtail::exp2_int(-up), 1.4e-45f);  // (0 * -inf is a NaN)
      }
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qs[nt][e] = sqs[8 * nt + 2 * c + e];
        st.m[nt][e] = kLow;
        st.l[nt][e] = 0.f;
      }
      if constexpr (G::kQReg) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint4 v = *reinterpret_cast<const uint4*>(sq + (8 * nt + g) * G::kQRow + 64 * b + 16 * c);
          qr[b][nt][0] = v.x, qr[b][nt][1] = v.y, qr[b][nt][2] = v.z, qr[b][nt][3] = v.w;
        }
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      st.lo4[b] = 0;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) st.o[b][mt][nt][e] = 0.f;
    }
    st.placed = false;
    const int pmin = s.q.L - s.q.nq + first / a.G, pmax = s.q.L - s.q.nq + (first + nrow - 1) / a.G;

    // ---- this warp's tiles of the part
    const int k1 = s.k1, ns = s.q.ns, off = s.q.off;
    for (int k = s.k0 + warp; k < k1; k += kWarps) {
      if (!dead && !__all_sync(~0u, tile_wait(bar + stage, phase))) {
        if (lane == 0 && a.status) atomicOr(a.status, kStatusTimeout);
        dead = true;
      }
      const int t0 = (k < ns ? k : k + off) * 16;
      if (!dead) {
        const uint8_t* tp = wring + stage * G::kTile;
        if (!(badmask >> stage & 1) && t0 <= pmax) {
          const bool full = t0 + 15 <= pmin && (a.window == 0 || t0 > pmax - a.window || t0 + 15 < a.sinks);
          tile_step<D, NT>(st, tp, sq, qr, qs, rowpos, !full, t0, pmax, a.window, a.sinks);
        }
        __syncwarp();
        issue(stage);
      }
      if (++stage == G::kStages) stage = 0, phase ^= 1;
    }

    // ---- the warps' sums become one
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = st.l[nt][e];
        l += __shfl_xor_sync(~0u, l, 4);
        l += __shfl_xor_sync(~0u, l, 8);
        l += __shfl_xor_sync(~0u, l, 16);
        if (g == 0) {
          xm[warp * RN + 8 * nt + 2 * c + e] = st.m[nt][e];
          xl[warp * RN + 8 * nt + 2 * c + e] = l;
        }
      }
    if (lane == 0) {
#pragma unroll
      for (int b = 0; b < NB; ++b) xlo[warp * NB + b] = st.placed ? (int)(st.lo4[b] & 255) : -1;
    }
    __syncthreads();
    float lsum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 8 * nt + 2 * c + e;
        float m = xm[i];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) m = fmaxf(m, xm[w * RN + i]);
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) l += xl[w * RN + i] * ex2(xm[w * RN + i] - m);
        const float f = ex2(st.m[nt][e] - m);
        lsum[nt][e] = l;
        st.m[nt][e] = m;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            st.o[b][mt][nt][e] *= f;
            st.o[b][mt][nt][e + 2] *= f;
          }
      }
    int lomax[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      lomax[b] = xlo[b];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) lomax[b] = max(lomax[b], xlo[w * NB + b]);
      if (st.placed) scale_block(st, b, exp2f((float)((int)(st.lo4[b] & 255) - lomax[b])));
    }
    float* of = &st.o[0][0][0][0];
    if (warp >= 2) {
#pragma unroll
      for (int i = 0; i < G::kORegs; ++i) merge[((warp - 2) * G::kORegs + i) * 32 + lane] = of[i];
    }
    __syncthreads();
    if (warp < 2) {
#pragma unroll
      for (int i = 0; i < G::kORegs; ++i) of[i] += merge[(warp * G::kORegs + i) * 32 + lane];
      if (warp == 1) {
#pragma unroll
        for (int i = 0; i < G::kORegs; ++i) merge[(G::kORegs + i) * 32 + lane] = of[i];
      }
    }
    __syncthreads();
    if (warp == 0) {
      const int row0 = part[0], nrow = part[1], first = part[2], h = part[3];
      const bool whole = part[5] != 0;
      const int64_t slot = 2 * (int64_t)blockIdx.x + part[4];
      float* po = a.part + slot * RN * D;
      float* pml = a.part + 2 * (int64_t)a.ctas * RN * D + slot * RN * 2;
#pragma unroll
      for (int i = 0; i < G::kORegs; ++i) of[i] += merge[(G::kORegs + i) * 32 + lane];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 8 * nt + 2 * c + e;
          const float inv = lsum[nt][e] == 0.f ? 0.f : 1.f / lsum[nt][e];
          if (i >= nrow) continue;
          const int rho = first + i, tok = rho / a.G;
          uint16_t* orow = a.out + (row0 + tok) * a.ldo + (int64_t)(h * a.G + rho - tok * a.G) * D;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const float f = inv * mtail::exp2_int(max(lomax[b], 0) + 14 - 127);
            const float4 v = make_float4(st.o[b][0][nt][e] * f, st.o[b][0][nt][e + 2] * f,
                                         st.o[b][1][nt][e] * f, st.o[b][1][nt][e + 2] * f);
            if (whole) {
              const __nv_bfloat162 lo2 = __floats2bfloat162_rn(v.x, v.y), hi2 = __floats2bfloat162_rn(v.z, v.w);
              *reinterpret_cast<uint2*>(orow + 32 * b + 4 * g) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&lo2), *reinterpret_cast<const uint32_t*>(&hi2));
            } else {
              *reinterpret_cast<float4*>(po + i * D + 32 * b + 4 * g) = v;
            }
          }
          if (!whole && g == 0) *reinterpret_cast<float2*>(pml + 2 * i) = make_float2(st.m[nt][e], lsum[nt][e]);
        }
    }
    u = (uint32_t)part[6];
    r = part[7];
    part = part == notes ? notes + 8 : notes;  // (a warp may still be reading these)
  }

  if (dead) {  // let the copies in flight land before the shared memory goes
    for (int i = 0; i < G::kStages; ++i) {
      tile_wait(bar + stage, phase);
      if (++stage == G::kStages) stage = 0, phase ^= 1;
    }
  }
}

// Joins the parts of the items that several ranges share.  CTA (x, y): the item that crosses the
// end of range x, if this is its first crossing, rows 4 y .. 4 y + 3, one per warp:
//   out = sum_k w_k o_k / sum_k w_k,  w_k = l_k 2^(m_k - max m), in range order.
template <int D>
__global__ void __launch_bounds__(kThreads) k_kv4_join(const __grid_constant__ AttnArgs a, int rn) {
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ uint64_t wsum[kWarps];
  uint32_t* pre = reinterpret_cast<uint32_t*>(sm);
  int* lens = reinterpret_cast<int*>(pre + a.reqs + 1);
  int* starts = lens + a.reqs;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int bits = 0;
  const uint64_t total64 = plan(a, rn, pre, lens, starts, wsum, &bits);
  if (total64 <= 0x7FFFFFFFull) {
    const uint32_t total = (uint32_t)total64, per = range_tiles(total64, a.ctas);
    const uint64_t u = ((uint64_t)blockIdx.x + 1) * per;
    if (u < total) {
      const Seg s = open_seg(a, rn, pre, lens, starts, find_req(pre, a.reqs, (uint32_t)u), (uint32_t)u, total);
      const uint32_t c0 = s.item / per, c1 = (s.item + (uint32_t)s.q.n - 1) / per;
      const int i = blockIdx.y * 4 + warp, rho = s.j * rn + i;
      if (s.k0 > 0 && c0 == blockIdx.x && rho < s.q.nq * a.G) {
        mtail::pdl_wait();
        const float* po = a.part + (int64_t)i * D;
        const float2* ml = reinterpret_cast<const float2*>(a.part + 2 * (int64_t)a.ctas * rn * D) + i;
        auto slot = [&](uint32_t k) { return 2 * (int64_t)k + (k == c0 ? 1 : 0); };
        float m = kLow;
        for (uint32_t k = c0 + lane; k <= c1; k += 32) m = fmaxf(m, ml[slot(k) * rn].x);
        m = mtail::warp_max(m);
        constexpr int E = D / 32;
        float o[E], sum = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
        for (uint32_t k = c0; k <= c1; ++k) {
          const float2 v = ml[slot(k) * rn];
          const float w = v.y * ex2(v.x - m);
          const float* p = po + slot(k) * rn * D + lane * E;
          sum += w;
          if constexpr (E == 2) {
            const float2 x = *reinterpret_cast<const float2*>(p);
            o[0] = fmaf(w, x.x, o[0]), o[1] = fmaf(w, x.y, o[1]);
          } else {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
              const float4 x = *reinterpret_cast<const float4*>(p + e);
              o[e] = fmaf(w, x.x, o[e]), o[e + 1] = fmaf(w, x.y, o[e + 1]);
              o[e + 2] = fmaf(w, x.z, o[e + 2]), o[e + 3] = fmaf(w, x.w, o[e + 3]);
            }
          }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int tok = rho / a.G;
        uint16_t* orow = a.out + (starts[s.r] + tok) * a.ldo + (int64_t)(s.h * a.G + rho - tok * a.G) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(o[e] * inv, o[e + 1] * inv);
          reinterpret_cast<uint32_t*>(orow)[e / 2] = *reinterpret_cast<const uint32_t*>(&v);
        }
        return;
      }
    }
  }
  mtail::pdl_wait();  // every CTA: the launch ends after the one it joins
}

template <int D, int NT>
cudaError_t prepare(int* blocks) {
  using G = Geo<D, NT>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // CTAs resident per SM with room for the largest request count, looked up once per device
  // (racing threads store the same value)
  static std::atomic<int> known[64];
  int n = dev < 64 ? known[dev].load(std::memory_order_acquire) : 0;
  if (!n) {
    e = cudaFuncSetAttribute(k_kv4_attn<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)G::smem(kMaxReqs));
    if (e != cudaSuccess) return e;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_kv4_attn<D, NT>, kThreads, G::smem(kMaxReqs));
    if (e != cudaSuccess) return e;
    if (n < 1) return cudaErrorInvalidConfiguration;
    if (dev < 64) known[dev].store(n, std::memory_order_release);
  }
  *blocks = n;
  return cudaSuccess;
}

template <int D, int NT>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  int blocks = 0;
  cudaError_t e = prepare<D, NT>(&blocks);
  if (e != cudaSuccess) return e;
  k_kv4_attn<D, NT><<<a.ctas, kThreads, Geo<D, NT>::smem(a.reqs), st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.ctas < 2) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas - 1, 2 * NT);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)(3 * a.reqs + 2) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_kv4_join<D>, a, 8 * NT);
}

template <typename F>
cudaError_t dispatch(int D, int rn, F&& f) {
  const int key = D * 100 + rn;
  switch (key) {
    case 6408: return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
    case 6416: return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
    case 6432: return f(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
    case 12808: return f(std::integral_constant<int, 128>(), std::integral_constant<int, 1>());
    case 12816: return f(std::integral_constant<int, 128>(), std::integral_constant<int, 2>());
    case 12832: return f(std::integral_constant<int, 128>(), std::integral_constant<int, 4>());
    case 25608: return f(std::integral_constant<int, 256>(), std::integral_constant<int, 1>());
    case 25616: return f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int attn_rows_per_item(int D, int G, int max_new) {
  const int64_t rows = (int64_t)G * max_new;
  return rows <= 8 ? 8 : (rows <= 16 || D == 256) ? 16 : 32;
}

int attn_ctas(int D, int rn, cudaError_t* err) {
  int blocks = 0, dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = dispatch(D, rn, [&](auto d, auto n) { return prepare<decltype(d)::value, decltype(n)::value>(&blocks); });
  *err = e;
  return e == cudaSuccess ? blocks * sms : 0;
}

size_t attn_workspace_bytes(int D, int rn, int ctas) {
  return (size_t)2 * ctas * rn * (D + 2) * sizeof(float);
}

cudaError_t launch_kv4_attention(const AttnArgs& a, int rn, cudaStream_t st) {
  return dispatch(a.D, rn, [&](auto d, auto n) { return launch<decltype(d)::value, decltype(n)::value>(a, st); });
}

}  // namespace kv4
