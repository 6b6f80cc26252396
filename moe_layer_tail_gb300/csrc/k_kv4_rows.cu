// k_kv4_rows.cu -- the row-wise kernels of the decode step's attention block (kv4_attn.h):
// step tables, query/key norm with rotation, cache rows in and out.  Each launch is a programmatic
// dependent launch of the kernel before it: its CTAs line up while that one ends and touch no
// memory until it has completed.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "k_kv4.cuh"
#include "moe_tail_internal.cuh"

namespace kv4 {

using mtail::bf16_hi;
using mtail::bf16_lo;

namespace {

__device__ __forceinline__ void report(int32_t* status, int32_t bits) {
  if (status && bits) atomicOr(status, bits);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
  f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z); f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
// two floats side by side: one instruction for both
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  return (uint64_t)__float_as_uint(lo) | (uint64_t)__float_as_uint(hi) << 32;
}
__device__ __forceinline__ float lower(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float upper(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ void unpack8(const uint4& u, uint64_t (&f)[4]) {
  f[0] = pair(bf16_lo(u.x), bf16_hi(u.x)), f[1] = pair(bf16_lo(u.y), bf16_hi(u.y));
  f[2] = pair(bf16_lo(u.z), bf16_hi(u.z)), f[3] = pair(bf16_lo(u.w), bf16_hi(u.w));
}
int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    return 1;
  return n;
}

// ------------------------------------------------------------------------ step tables ----
//
// Two exclusive sums over the requests (rows, pages), then every row and every fresh table
// entry finds its request by bisection.  Each CTA sums the (at most 1024) lengths for itself:
// 8 KB from L2, so that the launch needs no second pass.  1024 prompts of 262144 rows in all take 6.2
// us (3.3 MB at 0.5 TB/s): the chain of loads, sums and searches bounds it, not the bytes; 32
// decoding requests take 2.3 us, a launch.  The sums saturate at INT_MAX, which is
// associative and above anything that is asked of them (max_rows, the entries of all tables).
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return min(a + b, (uint32_t)INT32_MAX); }

// the last of n ascending starts (the first is 0) that is at most i
__device__ __forceinline__ int find_start(const int* start, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (start[m] <= i) lo = m; else hi = m - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kMaxReqs) k_step_tables(const TablesArgs a) {
  __shared__ int s_row[kMaxReqs + 1];   // first row of each request, cut to max_rows
  __shared__ int s_page[kMaxReqs + 1];  // its first fresh page
  __shared__ int s_len[kMaxReqs], s_held[kMaxReqs];  // its cached tokens, the pages that hold them
  __shared__ uint32_t s_wr[32], s_wp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int R = a.reqs;
  int bits = 0;
  mtail::pdl_trigger();
  mtail::pdl_wait();

  auto over_page = [&](int x) { return (int)__umul64hi((uint64_t)x, a.page_magic); };  // x / page, x >= 0
  auto pages = [&](int x) { return x ? over_page(x - 1) + 1 : 0; };
  int c = 0, n = 0, have = 0, want = 0;
  if (tid < R) {
    c = a.cached[tid];
    n = a.fresh[tid];
    const int64_t len = (int64_t)c + n;
    if (!(c >= 0 && n >= 0 && len <= INT32_MAX && len <= (int64_t)a.width * a.page))
      bits |= kStatusBadLength, c = n = 0;
    have = pages(c);
    want = n ? pages(c + n) : have;  // (c + n <= INT_MAX)
    s_len[tid] = c, s_held[tid] = have;
  }
  uint32_t r = n, p = want - have;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t r1 = __shfl_up_sync(~0u, r, o), p1 = __shfl_up_sync(~0u, p, o);
    if (lane >= o) r = add_sat(r, r1), p = add_sat(p, p1);
  }
  if (lane == 31) s_wr[warp] = r, s_wp[warp] = p;
  __syncthreads();
  uint32_t wr = lane < nw ? s_wr[lane] : 0, wp = lane < nw ? s_wp[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t r1 = __shfl_up_sync(~0u, wr, o), p1 = __shfl_up_sync(~0u, wp, o);
    if (lane >= o) wr = add_sat(wr, r1), wp = add_sat(wp, p1);
  }
  const uint32_t all_rows = __shfl_sync(~0u, wr, 31);
  uint32_t all_pages = __shfl_sync(~0u, wp, 31);
  const uint32_t r0 = __shfl_sync(~0u, wr, max(warp - 1, 0)), p0 = __shfl_sync(~0u, wp, max(warp - 1, 0));
  if (warp) r = add_sat(r, r0), p = add_sat(p, p0);
  if (tid < R) {
    s_row[tid + 1] = min((int)r, a.max_rows);
    s_page[tid + 1] = (int)p;
  }
  if (tid == 0) s_row[0] = s_page[0] = 0;
  __syncthreads();
  if ((int)all_rows > a.max_rows) {  // (the same in every thread)
    // a cut step: lengths and pages go by the rows that are kept
    if (tid < R) n = s_row[tid + 1] - s_row[tid], want = n ? pages(c + n) : have;
    p = want - have;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t p1 = __shfl_up_sync(~0u, p, o);
      if (lane >= o) p = add_sat(p, p1);
    }
    if (lane == 31) s_wp[warp] = p;
    __syncthreads();
    all_pages = 0;
    for (int w = 0; w < nw; ++w) {
      if (w == warp) p = add_sat(p, all_pages);
      all_pages = add_sat(all_pages, s_wp[w]);
    }
    if (tid < R) s_page[tid + 1] = (int)p;
    __syncthreads();
  }

  if (blockIdx.x == 0) {
    if (tid < R) {
      a.row_starts[tid + 1] = s_row[tid + 1];
      a.kv_lens[tid] = c + n;
    }
    if (tid == 0) {
      a.row_starts[0] = 0;
      a.used[0] = min((int)all_pages, a.n_free);
      if ((int)all_pages > a.n_free) bits |= kStatusNoPages;
      if ((int)all_rows > a.max_rows) bits |= kStatusRows;
    }
    report(a.status, bits);
  }

  const int step = gridDim.x * blockDim.x, at = blockIdx.x * blockDim.x + tid;  // (max_rows is at most 2^24)
  const int T = s_row[R];
  for (int i = at; i < a.max_rows; i += step) {
    int pos = 0;
    int64_t slot = -1;
    if (i < T) {
      const int q = find_start(s_row, R, i);
      pos = s_len[q] + (i - s_row[q]);
      const int e = over_page(pos), f = e - s_held[q];
      int page;
      if (f < 0) {
        page = a.table[q * a.stride + e];
      } else {
        const int64_t g = (int64_t)s_page[q] + f;
        page = g < a.n_free ? a.free_pages[g] : -1;
      }
      if (page >= 0) slot = (int64_t)page * a.page + (pos - e * a.page);
    }
    a.positions[i] = pos;
    a.slots[i] = slot;
  }
  for (int64_t i = at; i < (int)all_pages; i += step) {
    const int q = find_start(s_page, R, (int)i);
    a.table[q * a.stride + s_held[q] + (i - s_page[q])] = i < a.n_free ? a.free_pages[i] : -1;
  }
}

// ------------------------------------------------------- query/key norm and rotation ----
//
// L lanes hold one head, eight channels (16 bytes) each; the mean square is an L-lane butterfly, the
// partner of a channel comes from the same lane (interleaved) or by a shuffle of the packed values
// from the lane rot/16 further on (halves).  A warp takes up to `per` heads of one row, all queries'
// or all keys', so that what a lane multiplies with stays in its registers: out = y cos' + y' sin',
// y the scaled channel, y' its partner, cos' = gain cos, sin' = partner's gain times +-sin.  The
// heads come through a ring in shared memory, kDepth asynchronous copies of 512 bytes ahead of
// their use and the first of them while the angles are formed: in registers as many would leave
// room for half the warps (three of them: 68 us, the ring then 60).  8192 rows of 64 + 8 heads of 128
// take 50 us (302 MB, 6.05 TB/s, 0.89 of the measured copy rate), of 128 + 8 heads 88 us (0.95):
// memory, and below some 30 heads a row the angles' instructions.  CTAs of one row each, which form
// its angles together, take 69 us there, but are what serves a few rows (2.4 us for one row, 2.9 for
// 32 of D 256: launches).
//
// Angles: positions reach 2^31, where a product in 32 bits has lost the fraction of a turn and one
// in fp64 is slow on this part.  So the frequency is taken in turns as a 64-bit binary fraction,
// inv_freq / (2 pi) = M 2^E C with M the 24-bit significand and C = 1 / (2 pi) to 64 bits; the
// position times that, modulo 2^64, is the angle's fraction of a turn, exact to 2^-33 of one.
__device__ __forceinline__ float half_turns(int pos, float freq) {  // angle / pi, in [-1, 1)
  const uint32_t u = __float_as_uint(freq);
  const int e = (int)(u >> 23 & 255);
  if (e > 127 + 20 || (u >> 31)) {  // (large, negative or not a number)
    double turn = (double)pos * (double)freq * 0.15915494309189533577;
    turn -= rint(turn);
    return 2.f * (float)turn;
  }
  const uint64_t C = 0x28BE60DB9391054Aull, M = (u & 0x7FFFFFu) | 0x800000u;  // freq = M 2^(e - 150)
  const uint64_t lo = M * C, hi = __umul64hi(M, C);
  const int s = 150 - e;  // 3 .. 150; subnormal frequencies turn nothing
  const uint64_t f = s >= 128 ? 0 : s >= 64 ? hi >> (s - 64) : (hi << (64 - s)) | (lo >> s);
  const int64_t t = (int64_t)((uint64_t)(int64_t)pos * f);
  return (float)(int32_t)(t >> 32) * 4.656612873077392578125e-10f;  // 2^-31
}

template <int L>
__global__ void __launch_bounds__(256, 4) k_qk_norm_rope(const RopeArgs a, int qparts, int kparts, int perq,
                                                         int perk, int blocks) {
  constexpr int G = 32 / L, kDepth = 8;
  __shared__ __align__(16) float s_cos[8][128], s_sin[8][128];  // [warp][rot / 2], or one for all
  __shared__ uint4 s_ring[8][kDepth][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, li = lane % L, gi = lane / L;
  // `blocks` CTAs to a row, which form its angles together, or (0) each warp for itself
  const int parts = qparts + kparts, w = blockIdx.x * 8 + warp;
  // (there the queries' parts come first, the keys' shorter ones fill up at the end)
  const int keys = w - a.rows * qparts;
  const int row = blocks ? blockIdx.x / blocks : keys < 0 ? w / qparts : keys / max(kparts, 1);
  const int part = blocks ? w - row * blocks * 8 : keys < 0 ? w - row * qparts : qparts + keys - row * kparts;
  mtail::pdl_trigger();
  mtail::pdl_wait();
  if (row >= a.rows) return;  // (the whole CTA where it works together)
  const bool isq = part < qparts, act = li < a.D / 8;
  const int per = isq ? perq : perk, h0 = (isq ? part : part - qparts) * per;
  const int n = part < parts ? min(per, (isq ? a.hq : a.hk) - h0) : 0;
  const uint16_t* in = (isq ? a.q + row * a.ldq : a.k + row * a.ldk) + (int64_t)h0 * a.D + 8 * li;
  uint16_t* out = (isq ? a.qo + row * a.ldqo : a.ko + row * a.ldko) + (int64_t)h0 * a.D + 8 * li;
  const uint16_t* gain = isq ? a.gq : a.gk;

  const int half = a.rot / 2, hv = a.rot / 16;  // vectors of one half
  const bool low = li < hv, turns = a.interleaved ? 8 * li < a.rot : li < 2 * hv;
  const int other = a.interleaved ? li : low ? li + hv : li < 2 * hv ? li - hv : li;
  const float inv_d = 1.f / (float)a.D;
  // All loads set out before anything waits for one.
  const int pos = half ? a.pos[row] : 0;  // (without a rotation there may be no positions)
  const int first = blocks ? threadIdx.x : lane, step = blocks ? 256 : 32;
  float* const cosines = s_cos[blocks ? 0 : warp];
  float* const sines = s_sin[blocks ? 0 : warp];
  float freq[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) freq[j] = first + j * step < half ? a.freq[first + j * step] : 0.f;
  const uint32_t one2 = 0x3F803F80;
  uint4 ug = make_uint4(one2, one2, one2, one2), ugo = ug;
  if (gain && act && n > 0) {
    ug = *(reinterpret_cast<const uint4*>(gain) + li);
    ugo = *(reinterpret_cast<const uint4*>(gain) + other);
  }
  uint4* const ring = &s_ring[warp][0][lane];
  const uint16_t* next = in + gi * a.D;  // of this lane group's next head
  const int step_d = G * a.D, left0 = act ? (n - gi + G - 1) / G : 0;  // its heads
  int ahead = 0;
  auto fetch = [&]() {  // (a group of copies each time, empty behind the last)
    if (ahead < left0) cp_async16(ring + (ahead % kDepth) * 32, next);
    asm volatile("cp.async.commit_group;" ::: "memory");
    ++ahead, next += step_d;
  };
#pragma unroll
  for (int v = 0; v < kDepth; ++v) fetch();

  uint64_t c[4], s[4];  // cos', sin'
  {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int x = first + j * step;
      if (x < half) sincospif(half_turns(pos, freq[j]), &sines[x], &cosines[x]);
    }
    float g[8], go[8];
    unpack8(ug, g);
    unpack8(ugo, go);
    if (blocks) __syncthreads();
    else __syncwarp();
    float cf[8], sf[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) cf[e] = g[e], sf[e] = 0.f;
    if (turns && a.interleaved) {
      const float4 co = *reinterpret_cast<const float4*>(cosines + 4 * li), si = *reinterpret_cast<const float4*>(sines + 4 * li);
      const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        cf[e] = g[e] * cc[e / 2], cf[e + 1] = g[e + 1] * cc[e / 2];
        sf[e] = g[e + 1] * -ss[e / 2], sf[e + 1] = g[e] * ss[e / 2];
      }
    } else if (turns) {
      const int f = 8 * (low ? li : other);
      const float sign = low ? -1.f : 1.f;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 co = *reinterpret_cast<const float4*>(cosines + f + e), si = *reinterpret_cast<const float4*>(sines + f + e);
        cf[e] = g[e] * co.x, cf[e + 1] = g[e + 1] * co.y, cf[e + 2] = g[e + 2] * co.z, cf[e + 3] = g[e + 3] * co.w;
        sf[e] = go[e] * (sign * si.x), sf[e + 1] = go[e + 1] * (sign * si.y);
        sf[e + 2] = go[e + 2] * (sign * si.z), sf[e + 3] = go[e + 3] * (sign * si.w);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = pair(cf[2 * e], cf[2 * e + 1]), s[e] = pair(sf[2 * e], sf[2 * e + 1]);
  }
  uint16_t* to = out + gi * a.D;
  const int partner = other - li;
  for (int v = 0; v * G < n; ++v, to += step_d) {  // (uniform over the warp)
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
    __syncwarp();
    const uint4* at = ring + (v % kDepth) * 32;
    const uint4 u = v < left0 ? *at : make_uint4(0, 0, 0, 0);
    uint64_t x[4], y[4];
    unpack8(u, x);
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = pair(upper(x[e]), lower(x[e]));
    } else {
      unpack8(at[partner], y);  // (used where it turns)
    }
    __syncwarp();
    fetch();
    float rs = 1.f;
    if (gain) {
      uint64_t s2 = mul2(x[0], x[0]);
#pragma unroll
      for (int e = 1; e < 4; ++e) s2 = fma2(x[e], x[e], s2);
      float ss = lower(s2) + upper(s2);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
      rs = rsqrtf(fmaf(ss, inv_d, a.eps));
    }
    const uint64_t rs2 = pair(rs, rs);
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint64_t t = mul2(x[e], c[e]);
      if (turns) t = fma2(y[e], s[e], t);  // (else nothing of the partner: it may be infinite)
      t = mul2(t, rs2);
      r[e] = pack2(lower(t), upper(t));
    }
    if (v < left0) *reinterpret_cast<uint4*>(to) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

// ------------------------------------------------------------------------- cache rows ----
//
// D/8 lanes hold one token's head, eight channels each, of its keys and of its values, so that a
// block of 32 channels is four neighbouring lanes: its largest magnitude is two shuffles, and a
// lane's eight codes are one word.  65537 rows of 8 heads of 128: in 57 us (5.9 TB/s over 340 MB, 0.87
// of the measured copy rate; with a look-up for each head it took 68, instructions), out 61 us (5.6
// TB/s, 0.82); 32 rows in and out 3.3 us, two launches.  A token's bytes lie in 8- and 1-byte pieces all
// over its tile, so partial sectors reach the L2; tiles put together in shared memory first took 103 us
// (75 then), as the two more barriers cost more than the sectors.

template <int D>
__device__ __forceinline__ uint8_t* tile_of(const RowsArgs& a, int64_t slot, int h) {
  // slot / page by the multiplier 2^64 / page, rounded up: exact while slot * page < 2^64
  const int64_t page = (int64_t)__umul64hi((uint64_t)slot, a.page_magic);
  const int off = (int)(slot - page * a.page);
  return a.cache + ((page * a.heads + h) * (a.page / 16) + off / 16) * (17 * D);
}
// A group of lanes takes `units` a row: heads h, h + units, .. of kPairs, whose loads overlap and which
// share the row's look-up.
__device__ __forceinline__ uint32_t row_of(const RowsArgs& a, uint32_t id) {  // id / units
  return a.units == 1 ? id : (uint32_t)__umul64hi(id, a.unit_magic);
}
template <int D>
__device__ __forceinline__ int64_t next_tile(const RowsArgs& a) { return (int64_t)a.units * (a.page / 16) * (17 * D); }
// byte n of lane l of a tile's codes
__device__ __forceinline__ int lane_byte(int n, int l) { return (n >> 4) * 512 + l * 16 + (n & 15); }

// Eight bf16 of a block's four lanes -> this lane's codes and the block's scale byte.
__device__ __forceinline__ uint32_t quantize8(const uint4& u, uint32_t* scale) {
  // the block's largest magnitude as bf16 bits: an infinity or a NaN (exponent 255) is larger
  // than every number
  const uint32_t mask = 0x7FFF7FFFu;
  const uint32_t a2 = __vmaxu2(__vmaxu2(u.x & mask, u.y & mask), __vmaxu2(u.z & mask, u.w & mask));
  uint32_t am = __vmaxu2(a2, __shfl_xor_sync(~0u, a2, 1));
  am = __vmaxu2(am, __shfl_xor_sync(~0u, am, 2));
  am = max(am & 0xFFFFu, am >> 16);
  if (am >= 0x7F80u) {
    *scale = 255;
    return 0;
  }
  // smallest e in [-126, 125] with amax <= 6 * 2^e: amax = 1.m * 2^E, 6 = 1.5 * 2^2
  const int e = min(max((int)(am >> 7) - 129 + ((am & 0x7Fu) > 0x40u ? 1 : 0), -126), 125);
  *scale = (uint32_t)(e + 127);
  const float inv = mtail::exp2_int(-e);
  uint64_t x2[4];
  unpack8(u, x2);
  float x[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t t = mul2(x2[j], pair(inv, inv));
    x[2 * j] = lower(t), x[2 * j + 1] = upper(t);
  }
  return mtail::e2m1x8_pack(x);
}

template <int D, int kPairs>
__global__ void __launch_bounds__(256) k_kv4_append(const RowsArgs a) {
  constexpr int L = D / 8, NB = D / 32;
  const uint32_t id = blockIdx.x * (256 / L) + threadIdx.x / L;  // (row, unit); at most 2^32
  const int i = threadIdx.x % L, b = i >> 2, c = i & 3;
  mtail::pdl_trigger();
  mtail::pdl_wait();
  const uint32_t row = row_of(a, id), h = id - row * (uint32_t)a.units;
  int64_t slot = -1;
  uint4 ku[kPairs], vu[kPairs];
#pragma unroll
  for (int p = 0; p < kPairs; ++p) ku[p] = vu[p] = make_uint4(0, 0, 0, 0);
  if (row < (uint32_t)a.rows) {  // (the loads need not wait for the slot)
    slot = a.slots[row];
    const uint16_t* k = a.k + row * a.ldk + h * D + 8 * i;
    const uint16_t* v = a.v + row * a.ldv + h * D + 8 * i;
#pragma unroll
    for (int p = 0; p < kPairs; ++p)
      if (p == 0 || h + p * a.units < (uint32_t)a.heads) {
        ku[p] = *reinterpret_cast<const uint4*>(k + p * a.units * D);
        vu[p] = *reinterpret_cast<const uint4*>(v + p * a.units * D);
      }
  }
  if (slot >= a.n_slots) {
    if (h == 0 && i == 0) report(a.status, kStatusBadSlot);
    slot = -1;
  }
  const int t = (int)(slot & 15);  // (a page is a multiple of 16 tokens)
  uint8_t* tile = slot >= 0 ? tile_of<D>(a, slot, (int)h) : a.cache;
  // this lane's places in the tile: its key codes, the key scales of up to four blocks, the value codes
  // of lanes (b, c), b = 0, 1 and the value scale
  const int kc = lane_byte((t >> 3) * (D / 8) + 4 * b, (t & 7) * 4 + c);
  const int ksc = 16 * D + (t & 7) * (D / 16) + (t >> 3) * NB + (NB == 2 ? 0 : b);
  const int vc = 8 * D + lane_byte(((t >> 3) * 2 + (t & 1)) * (D / 16), (2 * c + b) * 4 + ((t & 7) >> 1));
  const int vsc = 16 * D + D / 2 + ((t & 7) >> 1) * (D / 8) + 4 * b + (t >> 3) * 2 + (t & 1);
#pragma unroll
  for (int p = 0; p < kPairs; ++p) {
    uint32_t ks, vs;
    const uint32_t kw = quantize8(ku[p], &ks), vw = quantize8(vu[p], &vs);
    uint32_t sw = ks << (8 * (b & 3));
    sw |= __shfl_xor_sync(~0u, sw, 4);
    if (NB > 2) sw |= __shfl_xor_sync(~0u, sw, 8);
    // the 16-bit pieces of every block of the values for g = 2c + b
    uint32_t vv[4];
#pragma unroll
    for (int k = 0; k < NB / 2; ++k) {
      const uint32_t w0 = __shfl_sync(~0u, vw, 8 * k + c, L), w1 = __shfl_sync(~0u, vw, 8 * k + 4 + c, L);
      vv[k] = b == 0 ? __byte_perm(w0, w1, 0x5410) : __byte_perm(w0, w1, 0x7632);
    }
    if (slot >= 0 && (p == 0 || h + p * a.units < (uint32_t)a.heads)) {
      uint8_t* to = tile + p * next_tile<D>(a);
      *reinterpret_cast<uint32_t*>(to + kc) = kw;
      if (c == 0 && (b & 3) == 0) {
        if (NB == 2) *reinterpret_cast<uint16_t*>(to + ksc) = (uint16_t)sw;
        else *reinterpret_cast<uint32_t*>(to + ksc) = sw;
      }
      if (b < 2) {
        if constexpr (NB == 2) *reinterpret_cast<uint32_t*>(to + vc) = vv[0];
        else if constexpr (NB == 4) *reinterpret_cast<uint2*>(to + vc) = make_uint2(vv[0], vv[1]);
        else *reinterpret_cast<uint4*>(to + vc) = make_uint4(vv[0], vv[1], vv[2], vv[3]);
      }
      if (c == 0) to[vsc] = (uint8_t)vs;
    }
  }
}

__device__ __forceinline__ uint4 dequantize8(uint32_t w, uint32_t s) {
  const float f = s == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(s << 23);  // (0: 0)
  uint32_t hh[4];
  mtail::e2m1x8_to_f16x2(w, hh[0], hh[1], hh[2], hh[3]);
  float x[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hh[j]));
    x[2 * j] = v.x * f;
    x[2 * j + 1] = v.y * f;
  }
  return pack8(x);
}

template <int D, int kPairs>
__global__ void __launch_bounds__(256) k_kv4_read(const RowsArgs a) {
  constexpr int L = D / 8, NB = D / 32;
  const uint32_t id = blockIdx.x * (256 / L) + threadIdx.x / L;
  const int i = threadIdx.x % L, b = i >> 2, c = i & 3;
  mtail::pdl_trigger();
  mtail::pdl_wait();
  const uint32_t row = row_of(a, id), h = id - row * (uint32_t)a.units;
  if (row >= (uint32_t)a.rows) return;
  const int64_t slot = a.slots[row];
  if (slot >= a.n_slots && h == 0 && i == 0) report(a.status, kStatusBadSlot);
  if (slot < 0 || slot >= a.n_slots) return;
  const int t = (int)(slot & 15);
  const uint8_t* tile = tile_of<D>(a, slot, (int)h);
  const int kc = lane_byte((t >> 3) * (D / 8) + 4 * b, (t & 7) * 4 + c);
  const int ksc = 16 * D + (t & 7) * (D / 16) + (t >> 3) * NB + b;
  const int n = ((t >> 3) * 2 + (t & 1)) * (D / 16) + 2 * b;
  const int vc0 = 8 * D + lane_byte(n, 8 * c + ((t & 7) >> 1)), vc1 = 8 * D + lane_byte(n, 8 * c + 4 + ((t & 7) >> 1));
  const int vsc = 16 * D + D / 2 + ((t & 7) >> 1) * (D / 8) + 4 * b + (t >> 3) * 2 + (t & 1);
  uint32_t kw[kPairs], vw[kPairs], ks[kPairs], vs[kPairs];
#pragma unroll
  for (int p = 0; p < kPairs; ++p) {
    if (p > 0 && h + p * a.units >= (uint32_t)a.heads) continue;
    const uint8_t* at = tile + p * next_tile<D>(a);
    kw[p] = *reinterpret_cast<const uint32_t*>(at + kc);
    ks[p] = at[ksc];
    vw[p] = *reinterpret_cast<const uint16_t*>(at + vc0) | (uint32_t)*reinterpret_cast<const uint16_t*>(at + vc1) << 16;
    vs[p] = at[vsc];
  }
  uint16_t* k = a.k + row * a.ldk + h * D + 8 * i;
  uint16_t* v = a.v + row * a.ldv + h * D + 8 * i;
#pragma unroll
  for (int p = 0; p < kPairs; ++p) {
    if (p > 0 && h + p * a.units >= (uint32_t)a.heads) continue;
    *reinterpret_cast<uint4*>(k + p * a.units * D) = dequantize8(kw[p], ks[p]);
    *reinterpret_cast<uint4*>(v + p * a.units * D) = dequantize8(vw[p], vs[p]);
  }
}

}  // namespace

cudaError_t launch_step_tables(const TablesArgs& a, cudaStream_t st) {
  const int threads = std::max(128, (a.reqs + 31) / 32 * 32);
  // One row a thread while that fills the GPU once: the rows' loads are what takes time.
  const int want = (a.max_rows + threads - 1) / threads;
  const int grid = std::min(want, num_sms() * std::max(1, 2048 / threads));
  return mtail::launch_k(k_step_tables, dim3(grid), dim3(threads), 0, st, true, a);
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st) {
  const int L = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32, G = 32 / L;
  // One head per lane group and warp until every SM has 48 warps, then up to 32, in equal parts: the
  // angles are formed once per warp, and a ring is better used by a longer run (8192 rows of 64 + 8
  // heads: 61 us with 8, 53 with 16, 50 with 32 and with 64; of 128 + 8: 93, 88 and 92 with 16, 32, 64).
  const int64_t groups = (int64_t)a.rows * ((a.hq + a.hk + G - 1) / G), fill = (int64_t)num_sms() * 48;
  const int most = G * (int)std::min<int64_t>(std::max<int64_t>(groups / fill, 1), 32);
  auto split = [&](int heads, int& parts) {
    parts = (heads + most - 1) / most;
    return parts ? ((heads + parts - 1) / parts + G - 1) / G * G : G;
  };
  int qparts, kparts;
  const int perq = split(a.hq, qparts), perk = split(a.hk, kparts);
  // With one head to a lane group the angles are a warp's longest work: there the CTAs take whole
  // rows and form them together (32 rows, D 256: 2.9 us against 3.3).
  const int blocks = most == G ? (qparts + kparts + 7) / 8 : 0;
  const int64_t grid = blocks ? (int64_t)a.rows * blocks : ((int64_t)a.rows * (qparts + kparts) + 7) / 8;
  if (grid > INT32_MAX / 8) return cudaErrorInvalidConfiguration;
  auto* kernel = L == 8 ? k_qk_norm_rope<8> : L == 16 ? k_qk_norm_rope<16> : k_qk_norm_rope<32>;
  return mtail::launch_k(kernel, dim3((unsigned)grid), dim3(256), 0, st, true, a, qparts, kparts, perq, perk, blocks);
}

namespace {
template <bool kAppend, int kPairs>
cudaError_t launch_rows(RowsArgs a, cudaStream_t st) {
  a.units = (a.heads + kPairs - 1) / kPairs;
  a.unit_magic = ~0ull / (uint64_t)a.units + 1;
  const int per = 256 / (a.D / 8);                                // units of a CTA
  const int64_t n = ((int64_t)a.rows * a.units + per - 1) / per;  // <= 2^24 * 256 / 8
  auto* kernel = a.D == 64    ? (kAppend ? k_kv4_append<64, kPairs> : k_kv4_read<64, kPairs>)
                 : a.D == 128 ? (kAppend ? k_kv4_append<128, kPairs> : k_kv4_read<128, kPairs>)
                              : (kAppend ? k_kv4_append<256, kPairs> : k_kv4_read<256, kPairs>);
  return mtail::launch_k(kernel, dim3((unsigned)n), dim3(256), 0, st, true, a);
}
template <bool kAppend>
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t st) {
  // One head a group of lanes until the GPU is filled several times over (32 rows of 8 heads, in and
  // out: 3.3 us, with two 4.5), then more where a row has them (65537 rows of 8 heads: in 60 us with two
  // and 57 with four, out 61 and 64).
  const int64_t threads = (int64_t)a.rows * a.heads * (a.D / 8);
  if (threads < (int64_t)num_sms() * 2048 * 4 || a.heads < 2) return launch_rows<kAppend, 1>(a, st);
  return kAppend && a.heads % 4 == 0 ? launch_rows<kAppend, 4>(a, st) : launch_rows<kAppend, 2>(a, st);
}
}  // namespace

cudaError_t launch_kv4_append(const RowsArgs& a, cudaStream_t st) { return launch_rows<true>(a, st); }
cudaError_t launch_kv4_read(const RowsArgs& a, cudaStream_t st) { return launch_rows<false>(a, st); }

}  // namespace kv4
