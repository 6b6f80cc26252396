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
// 8 KB from L2, so that the launch needs no second pass.
__global__ void __launch_bounds__(kMaxReqs) k_step_tables(const TablesArgs a) {
  __shared__ int s_row[kMaxReqs + 1];    // first row of each request, cut to max_rows
  __shared__ int s_page[kMaxReqs + 1];   // its first free page, cut to INT_MAX
  __shared__ int64_t s_wr[32], s_wp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int R = a.reqs;
  const bool first = blockIdx.x == 0;
  int bits = 0;
  mtail::pdl_trigger();
  mtail::pdl_wait();

  int c = 0, n = 0, have = 0, want = 0;
  bool ok = true;
  if (tid < R) {
    c = a.cached[tid];
    n = a.fresh[tid];
    const int64_t len = (int64_t)c + n;
    ok = c >= 0 && n >= 0 && len <= INT32_MAX && len <= (int64_t)a.width * a.page;
    if (!ok) bits |= kStatusBadLength, c = n = 0;
    have = c / a.page + (c % a.page != 0);
    want = n ? (c + n - 1) / a.page + 1 : have;  // (c + n <= INT_MAX)
  }
  int64_t r = n, p = want - have;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t r1 = __shfl_up_sync(~0u, r, o), p1 = __shfl_up_sync(~0u, p, o);
    if (lane >= o) r += r1, p += p1;
  }
  if (lane == 31) s_wr[warp] = r, s_wp[warp] = p;
  __syncthreads();
  for (int w = 0; w < warp; ++w) r += s_wr[w], p += s_wp[w];
  if (tid < R) {
    s_row[tid + 1] = (int)min(r, (int64_t)a.max_rows);
    s_page[tid + 1] = (int)min(p, (int64_t)INT32_MAX);
  }
  if (tid == 0) s_row[0] = s_page[0] = 0;
  int64_t all_rows = 0, all_pages = 0;
  for (int w = 0; w < nw; ++w) all_rows += s_wr[w], all_pages += s_wp[w];
  __syncthreads();

  if (first) {
    if (tid < R) {
      a.row_starts[tid + 1] = s_row[tid + 1];
      a.kv_lens[tid] = c + n;
    }
    if (tid == 0) {
      a.row_starts[0] = 0;
      a.used[0] = (int)min(all_pages, (int64_t)a.n_free);
      if (all_pages > a.n_free) bits |= kStatusNoPages;
      if (all_rows > a.max_rows) bits |= kStatusRows;
    }
    report(a.status, bits);
  }

  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + tid;
  const int T = s_row[R];
  for (int64_t i = at; i < a.max_rows; i += step) {
    int pos = 0;
    int64_t slot = -1;
    if (i < T) {
      int lo = 0, hi = R - 1;  // the last request that starts at or before row i
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (s_row[m] <= i) lo = m; else hi = m - 1;
      }
      const int cl = a.cached[lo];  // (valid: the request has rows)
      pos = cl + (int)(i - s_row[lo]);
      const int e = pos / a.page, held = cl / a.page + (cl % a.page != 0);
      int page;
      if (e < held) {
        page = a.table[lo * a.stride + e];
      } else {
        const int64_t f = (int64_t)s_page[lo] + (e - held);
        page = f < a.n_free ? a.free_pages[f] : -1;
      }
      if (page >= 0) slot = (int64_t)page * a.page + pos % a.page;
    }
    a.positions[i] = pos;
    a.slots[i] = slot;
  }
  const int64_t P = min(all_pages, (int64_t)INT32_MAX);
  for (int64_t i = at; i < P; i += step) {
    int lo = 0, hi = R - 1;
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (s_page[m] <= i) lo = m; else hi = m - 1;
    }
    const int cl = a.cached[lo], held = cl / a.page + (cl % a.page != 0);
    a.table[lo * a.stride + held + (i - s_page[lo])] = i < a.n_free ? a.free_pages[i] : -1;
  }
}

// ------------------------------------------------------- query/key norm and rotation ----
//
// L lanes hold one head, eight channels (16 bytes) each; the mean square is an L-lane butterfly,
// the partner of a channel pair comes from the same lane (interleaved) or by a shuffle from the
// lane rot/16 further on (halves).  The row's angles are formed once per CTA (fp64 product and
// reduction to one turn, then sincospi in fp32) while the first heads are in flight.
template <int L>
__global__ void __launch_bounds__(256) k_qk_norm_rope(const RopeArgs a, int chunks, int per) {
  __shared__ float s_cos[128], s_sin[128];
  const int tid = threadIdx.x, li = tid % L, gi = tid / L;
  constexpr int kHeads = 256 / L;
  const int t = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int heads = a.hq + a.hk;
  const int h0 = chunk * per * kHeads, h1 = min(heads, h0 + per * kHeads);
  const bool act = li < a.D / 8;
  const int half = a.rot / 2;
  mtail::pdl_trigger();
  mtail::pdl_wait();

  auto src = [&](int h) -> const uint4* {
    return reinterpret_cast<const uint4*>(h < a.hq ? a.q + t * a.ldq + (int64_t)h * a.D
                                                   : a.k + t * a.ldk + (int64_t)(h - a.hq) * a.D) + li;
  };
  int h = h0 + gi;
  uint4 u = make_uint4(0, 0, 0, 0);
  if (h < h1 && act) u = *src(h);

  if (tid < half) {
    double turn = (double)a.pos[t] * (double)a.freq[tid] * 0.15915494309189533577;
    turn -= rint(turn);
    sincospif(2.f * (float)turn, &s_sin[tid], &s_cos[tid]);
  }
  __syncthreads();

  for (int i = 0; i < per; ++i) {
    if (h0 + i * kHeads >= h1) break;  // (uniform over the CTA)
    const int hn = h + kHeads;
    uint4 un = make_uint4(0, 0, 0, 0);
    if (i + 1 < per && hn < h1 && act) un = *src(hn);
    float x[8];
    unpack8(u, x);
    const bool isq = h < a.hq;
    const uint16_t* gp = isq ? a.gq : a.gk;
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o, L);
    if (gp && act) {
      float g[8];
      unpack8(*(reinterpret_cast<const uint4*>(gp) + li), g);
      const float rs = rsqrtf(ss / (float)a.D + a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = x[e] * rs * g[e];
    }
    if (a.interleaved) {
      if (8 * li < a.rot) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float c = s_cos[4 * li + e / 2], s = s_sin[4 * li + e / 2];
          const float lo = x[e], hi = x[e + 1];
          x[e] = lo * c - hi * s;
          x[e + 1] = hi * c + lo * s;
        }
      }
    } else if (a.rot) {
      const int hv = a.rot / 16;  // vectors of one half
      const bool low = li < hv;
      const int other = low ? li + hv : li < 2 * hv ? li - hv : li;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = __shfl_sync(0xffffffffu, x[e], other, L);
        if (li < 2 * hv) {
          const int f = 8 * (low ? li : other) + e;
          const float c = s_cos[f], s = s_sin[f];
          x[e] = low ? x[e] * c - y * s : x[e] * c + y * s;
        }
      }
    }
    if (h < h1 && act) {
      uint16_t* o = isq ? a.qo + t * a.ldqo + (int64_t)h * a.D
                        : a.ko + t * a.ldko + (int64_t)(h - a.hq) * a.D;
      reinterpret_cast<uint4*>(o)[li] = pack8(x);
    }
    u = un;
    h = hn;
  }
}

// ------------------------------------------------------------------------- cache rows ----
//
// D/8 lanes hold one token's head, eight channels each, so that a block of 32 channels is four
// neighbouring lanes: its largest magnitude is two shuffles, and a lane's eight codes are one
// word.  blockIdx.y = 0: keys, 1: values.

template <int D>
__device__ __forceinline__ uint8_t* tile_of(const RowsArgs& a, int64_t slot, int h) {
  const int64_t page = slot / a.page;
  const int off = (int)(slot - page * a.page);
  return a.cache + ((page * a.heads + h) * (a.page / 16) + off / 16) * (17 * D);
}
// byte n of lane l of a tile's codes
__device__ __forceinline__ int lane_byte(int n, int l) { return (n >> 4) * 512 + l * 16 + (n & 15); }

template <int D>
__global__ void __launch_bounds__(256) k_kv4_append(const RowsArgs a) {
  constexpr int L = D / 8, NB = D / 32;
  const bool val = blockIdx.y != 0;
  const int64_t id = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;  // (row, head)
  const int i = threadIdx.x % L, b = i >> 2, c = i & 3;
  const bool in = id < (int64_t)a.rows * a.heads;
  const int row = in ? (int)(id / a.heads) : 0, h = in ? (int)(id % a.heads) : 0;
  mtail::pdl_trigger();
  mtail::pdl_wait();
  int64_t slot = in ? a.slots[row] : -1;
  if (slot >= a.n_slots) {
    if (h == 0 && i == 0 && !val) report(a.status, kStatusBadSlot);
    slot = -1;
  }
  uint4 u = make_uint4(0, 0, 0, 0);
  if (slot >= 0) {
    const uint16_t* p = val ? a.v + row * a.ldv : a.k + row * a.ldk;
    u = *(reinterpret_cast<const uint4*>(p + h * D) + i);
  }
  float x[8];
  unpack8(u, x);
  // the block's largest magnitude as bf16 bits: an infinity or a NaN (exponent 255) is larger
  // than every number
  uint32_t am = 0;
  am = max(max(u.x & 0x7FFFu, (u.x >> 16) & 0x7FFFu), max(u.y & 0x7FFFu, (u.y >> 16) & 0x7FFFu));
  am = max(am, max(max(u.z & 0x7FFFu, (u.z >> 16) & 0x7FFFu),
                   max(u.w & 0x7FFFu, (u.w >> 16) & 0x7FFFu)));
  am = max(am, __shfl_xor_sync(~0u, am, 1));
  am = max(am, __shfl_xor_sync(~0u, am, 2));
  uint32_t sc, w;
  if (am >= 0x7F80u) {
    sc = 255;
    w = 0;
  } else {
    // smallest e in [-126, 125] with amax <= 6 * 2^e: amax = 1.m * 2^E, 6 = 1.5 * 2^2
    const int e = min(max((int)(am >> 7) - 129 + ((am & 0x7Fu) > 0x40u ? 1 : 0), -126), 125);
    sc = (uint32_t)(e + 127);
    const float inv = mtail::exp2_int(-e);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= inv;
    w = mtail::e2m1x8_pack(x);
  }
  const int t = (int)(slot & 15);  // (a page is a multiple of 16 tokens)
  uint8_t* tile = slot >= 0 ? tile_of<D>(a, slot, h) : nullptr;
  if (!val) {
    if (slot >= 0)
      *reinterpret_cast<uint32_t*>(tile + lane_byte((t >> 3) * (D / 8) + 4 * b, (t & 7) * 4 + c)) = w;
    // the scale bytes of up to four blocks in one store
    uint32_t sw = sc << (8 * (b & 3));
    sw |= __shfl_xor_sync(~0u, sw, 4);
    if (NB > 2) sw |= __shfl_xor_sync(~0u, sw, 8);
    uint8_t* s = tile + 16 * D + (t & 7) * (D / 16) + (t >> 3) * NB;
    if (slot >= 0 && c == 0 && (b & 3) == 0) {
      if (NB == 2)
        *reinterpret_cast<uint16_t*>(s) = (uint16_t)sw;
      else
        *reinterpret_cast<uint32_t*>(s + b) = sw;
    }
  } else {
    // lanes (b, c), b = 0, 1 collect the 16-bit pieces of every block for g = 2c + b
    uint32_t vv[NB / 2];
#pragma unroll
    for (int k = 0; k < NB / 2; ++k) {
      const uint32_t w0 = __shfl_sync(~0u, w, 8 * k + c, L), w1 = __shfl_sync(~0u, w, 8 * k + 4 + c, L);
      vv[k] = b == 0 ? __byte_perm(w0, w1, 0x5410) : __byte_perm(w0, w1, 0x7632);
    }
    if (slot >= 0 && b < 2) {
      uint8_t* p = tile + 8 * D +
                   lane_byte(((t >> 3) * 2 + (t & 1)) * (D / 16), (2 * c + b) * 4 + ((t & 7) >> 1));
      if (NB == 2) *reinterpret_cast<uint32_t*>(p) = vv[0];
      else if (NB == 4) *reinterpret_cast<uint2*>(p) = make_uint2(vv[0], vv[NB / 2 - 1]);
      else *reinterpret_cast<uint4*>(p) = make_uint4(vv[0], vv[1 % (NB / 2)], vv[2 % (NB / 2)], vv[3 % (NB / 2)]);
    }
    if (slot >= 0 && c == 0)
      tile[16 * D + D / 2 + ((t & 7) >> 1) * (D / 8) + 4 * b + (t >> 3) * 2 + (t & 1)] = (uint8_t)sc;
  }
}

template <int D>
__global__ void __launch_bounds__(256) k_kv4_read(const RowsArgs a) {
  constexpr int L = D / 8, NB = D / 32;
  const bool val = blockIdx.y != 0;
  const int64_t id = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
  const int i = threadIdx.x % L, b = i >> 2, c = i & 3;
  mtail::pdl_trigger();
  mtail::pdl_wait();
  if (id >= (int64_t)a.rows * a.heads) return;
  const int row = (int)(id / a.heads), h = (int)(id % a.heads);
  const int64_t slot = a.slots[row];
  if (slot < 0 || slot >= a.n_slots) {
    if (slot >= 0 && h == 0 && i == 0 && !val) report(a.status, kStatusBadSlot);
    return;
  }
  const int t = (int)(slot & 15);
  const uint8_t* tile = tile_of<D>(a, slot, h);
  uint32_t w, s;
  if (!val) {
    w = *reinterpret_cast<const uint32_t*>(tile + lane_byte((t >> 3) * (D / 8) + 4 * b, (t & 7) * 4 + c));
    s = tile[16 * D + (t & 7) * (D / 16) + (t >> 3) * NB + b];
  } else {
    const uint8_t* p = tile + 8 * D;
    const int n = ((t >> 3) * 2 + (t & 1)) * (D / 16) + 2 * b;
    w = *reinterpret_cast<const uint16_t*>(p + lane_byte(n, 8 * c + ((t & 7) >> 1)));
    w |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + lane_byte(n, 8 * c + 4 + ((t & 7) >> 1))) << 16;
    s = tile[16 * D + D / 2 + ((t & 7) >> 1) * (D / 8) + 4 * b + (t >> 3) * 2 + (t & 1)];
  }
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
  uint16_t* o = val ? a.v + row * a.ldv : a.k + row * a.ldk;
  *(reinterpret_cast<uint4*>(o + h * D) + i) = pack8(x);
}

}  // namespace

cudaError_t launch_step_tables(const TablesArgs& a, cudaStream_t st) {
  const int threads = std::max(128, (a.reqs + 31) / 32 * 32);
  // four rows a thread, at most two CTAs' worth of threads on every SM
  const int64_t want = ((int64_t)a.max_rows + 4 * threads - 1) / (4 * threads);
  const int grid = (int)std::min<int64_t>(want, 2 * num_sms());
  return mtail::launch_k(k_step_tables, dim3(grid), dim3(threads), 0, st, true, a);
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st) {
  const int L = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
  const int kHeads = 256 / L, groups = (a.hq + a.hk + kHeads - 1) / kHeads;
  // one group of heads per CTA until the rows alone fill the GPU several times over
  int per = (int)std::min<int64_t>(groups, std::max<int64_t>(1, (int64_t)a.rows * groups / (num_sms() * 16)));
  const int chunks = (groups + per - 1) / per;
  const int64_t grid = (int64_t)a.rows * chunks;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  auto* kernel = L == 8 ? k_qk_norm_rope<8> : L == 16 ? k_qk_norm_rope<16> : k_qk_norm_rope<32>;
  return mtail::launch_k(kernel, dim3((unsigned)grid), dim3(256), 0, st, true, a, chunks, per);
}

namespace {
template <bool kAppend>
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t st) {
  const int per = 256 / (a.D / 8);
  const int64_t n = ((int64_t)a.rows * a.heads + per - 1) / per;  // <= 2^24 * 256 / 8
  const dim3 grid((unsigned)n, 2);
  auto* kernel = a.D == 64    ? (kAppend ? k_kv4_append<64> : k_kv4_read<64>)
                 : a.D == 128 ? (kAppend ? k_kv4_append<128> : k_kv4_read<128>)
                              : (kAppend ? k_kv4_append<256> : k_kv4_read<256>);
  return mtail::launch_k(kernel, grid, dim3(256), 0, st, true, a);
}
}  // namespace

cudaError_t launch_kv4_append(const RowsArgs& a, cudaStream_t st) { return launch_rows<true>(a, st); }
cudaError_t launch_kv4_read(const RowsArgs& a, cudaStream_t st) { return launch_rows<false>(a, st); }

}  // namespace kv4
