// k_kv4_tc.cu -- attention of a step's query rows over the paged MXFP4 cache (kv4_attn.h) on the
// tcgen05 tensor cores.
//
//   out[i] = sum_j p_j V_j / sum_j p_j,  p_j = 2^(scale log2(e) q_i . K_j - m_i)
//
// in one pass over the cache.  The query heads that share a kv head, and the rows of a request,
// are rows of one work item (RN at a time), so the cache is read once for all of them; the items'
// tiles of 16 tokens, laid end to end, are cut into equal ranges, one per SM (k_kv4_plan.cuh), so
// that ragged lengths, one long request and many short ones all load every SM the same (32 requests
// of up to 32768 tokens run at the rate of one of 524287).  An item that lies in one range is
// written by its CTA; the others leave an average and (max, sum) per row and part in the workspace,
// which a second launch joins (programmatic dependent launch).
//
// The CUDA cores never see a key or a value.  A step is 8 tiles (128 tokens) of one kv head:
//   K' [128 tokens x D] = K I      tcgen05 kind::mxf4 block-scaled, the codes and scales as they
//                                  are cached times an E2M1 identity: the dequantised keys, exact
//                                  fp32, in tensor memory;
//   S^T [128 x RN] = K' Q^T        kind::tf32, K' read from tensor memory as operand A, the bf16
//                                  queries exact as tf32 in shared memory;
//   P^T = 2^(S - m)                fp32 on the CUDA cores, a token per thread, rounded to tf32 for
//                                  the product (half a step, 2^-11 of each term: the least that a
//                                  tensor-core operand of this range costs; the row's sum takes them
//                                  unrounded); m is the row's maximum over the part's first step
//                                  and moves only when a score passes it by 40 octaves, since a
//                                  move rescales O and holds the products up;
//   V' [D x 128 tokens] = I V^T    the dequantised values, transposed by the product itself;
//   O^T [D x RN] += V' P^T         kind::tf32, V' from tensor memory, accumulating there.
// Conversions on the CUDA cores into mma.sync had taken 490 warp instructions per tile and stayed
// at 2.5 TB/s.
//
// What bounds it (524287 tokens, 8 kv heads of 128, 16 query heads each: 570 MB in 139 us, 4.1 TB/s,
// 0.61 of the measured copy rate): not the tensor cores (about 550 cycles of products a step), not
// the memory (740 cycles for a step's 17 KB) but two chains of hand-overs of about 1100 cycles a
// step each, K' -> S -> K' of the next step (each product is seen complete about 300 cycles after
// its last instruction has issued, and K' has room for one step only) and S -> P -> S of the
// softmax.  Tensor memory has no room for K' twice at D 128 (K' 128 columns, V' 2 x 128, S twice, O and
// the scales are 456 of 512 with up to 16 rows an item, 504 with 32), so neither can run further ahead.
// Tried and slower at this size (against 135 us at the time): K' in a ring of three blocks of 64
// channels with a warp of its own (163 us: six runs of products a step instead of four, and each
// costs the pipe some 150 cycles beside its products); both dequantisations in one run (160); a warp
// of its own for V' (141: its products get in front of the scores' in the pipe), V' before the output
// product (140); V' and K' in halves (234); waits that poll (185; a dozen polling warps take the
// shared-memory pipe from the others); one group of four softmax warps (190).  D 64 has the same
// chains for half the bytes (K' twice there changed nothing); D 256 twice the products for its two
// halves of channels: four rows of eight requests of up to 16384 tokens, 64 rows a kv head, take 73
// us in two items of 32 rows (71 at the time, and 103 in four of 16).
//
// Warps: 0 looks up pages and copies tiles (bulk copies into a ring, 32 look-ups at a time);
// 6..13 (one per tile of a step) bring a tile's bytes, which the cache holds in the order of
// register fragments, into the swizzled rows and scale-factor atoms of the tensor cores' operands;
// 1 issues K' and S, 14 V' and O (an elected thread each: a divergent issuer costs 45 cycles an
// instruction, an elected one 9 at these sizes); 2..5 and 15..18 are the softmax and the output of
// the lower and the upper half of the rows.  They hand over through mbarriers; every wait is bounded
// and reports MOE_TAIL_STATUS_TIMEOUT; a CTA in which one has given up leaves NaN in the rows that it
// had a part of.  Spills must stay out of the steps: local memory shares what little L1 the 150..210 KB
// of shared memory leave, and versions that spilled took 2.5 times as long.
//
// Tensor memory is taken whole (512 columns), once the kernels before this one in the stream have
// ended: CTAs of this launch may be resident while a kernel of the caller's several launches back still
// runs, and that one could otherwise wait for the columns that these hold while these wait for it.
// The allocation runs beside the plan and costs nothing (1000 and 524287 tokens took the same before and
// behind).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "k_kv4_plan.cuh"
#include "k_stream_common.cuh"

namespace kv4 {

using mtail::bulk_load;
using mtail::mbar_arrive;
using mtail::mbar_expect_tx;
using mtail::mbar_init;
using mtail::smem_u32;

namespace {

// warps: 0 copies, 1 key products, 2..5 and 15..18 softmax (rows of the lower and the upper half;
// warp mod 4 = the tensor-memory lanes it reaches), 6..13 layout, 14 value products
constexpr int kWarps = 19, kThreads = 32 * kWarps;
constexpr int kLayWarp = 6, kValWarp = 14, kSoft2Warp = 15;
constexpr int kStepTiles = 8;
constexpr int kInfos = 8;                     // steps whose notes are kept
constexpr uint32_t kBudgetClocks = 200000000;  // of a wait, about 0.1 s
constexpr float kLow = -3.0e38f;              // a row's reference before its first score
constexpr float kOver = 40.f;                 // octaves above the reference that move it

// A position in a ring of N buffers and the parity of its pass.
template <int N>
struct Ring {
  uint32_t i = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++i == N) i = 0, ph ^= 1;
  }
};

// What the softmax needs to know of a step's tokens.
struct Info {
  uint64_t plain;         // byte j is 1: every row sees all of tile j, no scale of it is a NaN
  // of the other tiles:
  int t0[kStepTiles];     // their first token, negative: the tile has no page
  uint16_t flags[128];    // of a token: bit 15 a NaN among its key scales, bit b one at value block b
};

template <int D, int RN>
struct Geo {
  static constexpr int NM = RN < 16 ? 16 : RN;  // columns of the products
  static constexpr int NB = D / 32;
  static constexpr int CH = D < 128 ? D : 128;  // channels of one half
  static constexpr int kHalves = D / CH;
  static constexpr int kTile = 17 * D;
  static constexpr int kStep = kStepTiles * kTile;
  static constexpr int kRaw = D == 256 ? 2 : D == 128 ? 4 : 6;
  static constexpr int kOps = D == 256 ? 2 : 3;
  static constexpr int kQs = D == 256 ? 1 : 2;
  static constexpr int kOp = D == 256 ? 32768 : 16384;  // codes of a step: rows of 128 bytes
  static constexpr int kAtoms = D == 256 ? 2 : 1;
  static constexpr int kSf = 2 * kAtoms * 512;           // key atoms, then value atoms
  static constexpr int kP = NM * 512, kQ = NM * D * 4;
  // tensor-memory columns: K' once, V' twice (32 rows of D 256 leave room for one), S twice, O
  static constexpr int kVs = D == 256 && RN == 32 ? 1 : 2;
  static constexpr int cK = 0, cV = 128, cS = cV + 128 * kVs, cO = cS + 2 * NM;
  static constexpr int cSfK = cO + kHalves * NM, cSfV = cSfK + 8 * kAtoms, cSfI = cSfV + 8 * kAtoms, cSfJ = cSfI + 4;
  static_assert(cSfJ + 4 <= 512, "tensor memory");
  // shared memory (from a 1024-byte boundary)
  static constexpr int oOp = 0, oI = oOp + kOps * kOp, oQ = oI + 16384, oP = oQ + kQs * kQ;
  static constexpr int oRaw = oP + 2 * kP, oSf = (oRaw + kRaw * kStep + 127) / 128 * 128;
  static constexpr int oSfI = oSf + kOps * kSf, oInfo = oSfI + 512;
  static constexpr int oSmall = oInfo + kInfos * (int)sizeof(Info);
  // raw and operand rings, info ring, q, and the single ones
  static constexpr int kBars = 2 * kRaw + 2 * kOps + kInfos + 4 + 12 + 4 + 2;
  static constexpr int kSmall = kBars * 8 + kRaw * 20 * 4 /* t0, full */ + 4 * RN * 12 /* red, l */ +
                                RN * 16 /* rowpos, nan */ + 64 /* checks */;
  static constexpr size_t smem(int reqs) {
    return 1024 + (size_t)oSmall + kSmall + (size_t)(3 * reqs + 2) * 4;
  }
  static constexpr int kReqs = D == 256 && RN == 32 ? 256 : kMaxReqs;  // that it has room for
};

// ------------------------------------------------------------------ PTX wrappers ----

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}
// shared-memory matrix descriptors: K-major rows of 128 bytes under the 128-byte swizzle (8-row
// groups 1024 bytes apart), and scale-factor atoms (no swizzle)
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t sf_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (8ull << 16) | (8ull << 32) | (1ull << 46);
}
// instruction descriptors: E2M1 x E2M1 with UE8M0 scales (the scale bytes of the K step's two
// blocks from sf_id on), and tf32 x tf32; M 128, N columns, fp32 accumulators
__device__ __forceinline__ uint32_t idesc_mxf4(int N, uint32_t sf_id) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | (8u << 24) | (sf_id << 29) |
         (sf_id << 4);
}
__device__ __forceinline__ uint32_t idesc_tf32(int N) {
  return (1u << 4) | (2u << 7) | (2u << 10) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void cp_sf(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc));
}
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb));
}
// A in tensor memory, B in shared memory
__device__ __forceinline__ void mma_tf32(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
#define KV4_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define KV4_W8(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// this warp's 32 lanes x 8 consecutive columns (lane = tensor-memory lane)
__device__ __forceinline__ void ld8(uint32_t t, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : KV4_R8(0) : "r"(t));
}
__device__ __forceinline__ void st8(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), KV4_W8(0));
}
#undef KV4_R8
#undef KV4_W8
__device__ __forceinline__ void ld4(uint32_t t, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(t));
}
__device__ __forceinline__ void st4(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]));
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t t, float (&v)[N]) {
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    if (N % 8) ld4(t + i, r + i);
    else ld8(t + i, r + i);
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t t, const float (&v)[N]) {
  uint32_t r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __float_as_uint(v[i]);
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    if (N % 8) st4(t + i, r + i);
    else st8(t + i, r + i);
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// to the nearest tf32 (a NaN may come out as a zero)
__device__ __forceinline__ float to_tf32(float x) {
  return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xFFFFE000u);
}
// bytes of w that are 255, one bit each
__device__ __forceinline__ uint32_t ff_bytes(uint32_t w) {
  const uint32_t f = ((w & 0x7F7F7F7Fu) + 0x01010101u) & w & 0x80808080u;
  return (f >> 7 & 1) | (f >> 14 & 2) | (f >> 21 & 4) | (f >> 28 & 8);
}

// The largest of each of N values over the warp: lane l returns that of value l mod N.
template <int N>
__device__ __forceinline__ float warp_max_of(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = N / 2; h >= 1; h >>= 1) {
    const bool up = (lane & h) != 0;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float send = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = fmaxf(keep, __shfl_xor_sync(~0u, send, h));
    }
  }
#pragma unroll
  for (int o = N; o < 32; o <<= 1) v[0] = fmaxf(v[0], __shfl_xor_sync(~0u, v[0], o));
  return v[0];
}
template <int N>
__device__ __forceinline__ float warp_sum_of(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = N / 2; h >= 1; h >>= 1) {
    const bool up = (lane & h) != 0;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float send = up ? v[i] : v[i + h], keep = up ? v[i + h] : v[i];
      v[i] = keep + __shfl_xor_sync(~0u, send, h);
    }
  }
#pragma unroll
  for (int o = N; o < 32; o <<= 1) v[0] += __shfl_xor_sync(~0u, v[0], o);
  return v[0];
}

// Waits in hardware for up to 20 us (without the hint a waiting warp polls, and a dozen of them take
// the shared-memory pipe from the others; once a wait has given up, the others cost as long each).
__device__ __forceinline__ bool mbar_sleep_wait(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(ok)
      : "r"(smem_u32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}

struct Bars {
  uint64_t *raw_full, *raw_empty, *op_full, *op_empty, *info, *q_full, *q_empty;
  uint64_t *k_full, *k_free, *s_full, *p_full, *v_full, *v_free, *pv, *soft, *meet;
};

// The record that tells the joining launch which item crosses the end of a range.
constexpr int kRefused = -2;
struct JoinRec {
  int last;   // the last range of the item, negative: none crosses; kRefused: the call is too large
  int row0;   // first query row of its request
  int first;  // the item's first row among the request's (row, head) pairs
  int head;   // kv head
  int rows;   // rows of the item
  int pad[3];
};

// What a CTA whose waits gave up leaves of its range, whatever it had written of it: NaN in the rows of its
// whole items, and parts that make the rows of the others NaN when they are joined.
template <int D, int RN>
__device__ __forceinline__ void forsake(const AttnArgs& a, const uint32_t* pre, const int* lens, const int* starts,
                                     uint32_t u0, uint32_t u1, uint32_t per) {
  JoinRec rec = {};
  rec.last = -1;
  int r = find_req(pre, a.reqs, u0);
  for (uint32_t u = u0; u < u1;) {
    const Seg s = open_seg(a, RN, pre, lens, starts, r, u, u1);
    r = s.r;
    const int first = s.j * RN, nrow = min(RN, s.q.nq * a.G - first);
    const bool whole = s.k0 == 0 && s.k1 == s.q.n;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (s.k0 == 0 ? 1 : 0);
    float2* ml = reinterpret_cast<float2*>(a.part + 2 * (int64_t)a.ctas * RN * D) + slot * RN;
    for (int i = threadIdx.x; i < nrow * D; i += kThreads) {
      const int k = i / D, rho = first + k, tk = rho / a.G;
      if (whole) a.out[(starts[s.r] + tk) * a.ldo + (int64_t)(s.h * a.G + rho - tk * a.G) * D + i % D] = 0x7FC0;
      else if (i % D == 0) ml[k] = make_float2(0.f, __uint_as_float(0x7FC00000u));
    }
    u += s.places;
    if (u >= u1) {
      if (s.k0 == 0 && !whole) rec.last = (int)((s.item + (uint32_t)(s.q.n + kItemTiles) - 1) / per);
      rec.row0 = starts[s.r], rec.first = first, rec.head = s.h, rec.rows = nrow;
    }
  }
  if (threadIdx.x == 0)
    reinterpret_cast<JoinRec*>(a.part + 2 * (int64_t)a.ctas * RN * (D + 2))[blockIdx.x] = rec;
}

template <int D, int RN>
__global__ void __launch_bounds__(kThreads, 1) k_kv4_attn(const __grid_constant__ AttnArgs a) {
  using G = Geo<D, RN>;
  constexpr int NM = G::NM, NB = G::NB;
  extern __shared__ uint8_t sm_raw[];
  __shared__ uint32_t s_range[3];  // of places: first, end, of each CTA
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead;
  uint8_t* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  Info* infos = reinterpret_cast<Info*>(sm + G::oInfo);
  uint64_t* bp = reinterpret_cast<uint64_t*>(sm + G::oSmall);
  Bars B;
  B.raw_full = bp;
  B.raw_empty = B.raw_full + G::kRaw;
  B.op_full = B.raw_empty + G::kRaw;
  B.op_empty = B.op_full + G::kOps;
  B.info = B.op_empty + G::kOps;
  B.q_full = B.info + kInfos;
  B.q_empty = B.q_full + 2;
  B.k_full = B.q_empty + 2;
  B.k_free = B.k_full + 1;  // (two halves only: with one, the scores are all that use the keys)
  B.s_full = B.k_free + 1;
  B.p_full = B.s_full + 2;
  B.v_full = B.p_full + 2;
  B.v_free = B.v_full + 2;  // (two halves only)
  B.pv = B.v_free + 2;
  B.soft = B.pv + 2;
  B.meet = B.soft + 4;
  int* raw_info = reinterpret_cast<int*>(bp + G::kBars);  // [kRaw][20]: t0 of the tiles, full
  float* red = reinterpret_cast<float*>(raw_info + G::kRaw * 20);  // [2][4][RN]
  float* lsum = red + 8 * RN;                                       // [4][RN]
  int* rowpos = reinterpret_cast<int*>(lsum + 4 * RN);
  uint32_t* nanrow = reinterpret_cast<uint32_t*>(rowpos + 2 * RN);  // both [2 turns][RN]
  // what the softmax warps ask for once a step, [half][turn]: a byte each, whether its scores passed
  // kOver, and a word that tells them that a wait has given up
  uint32_t* checks = nanrow + 2 * RN;
  uint32_t* pre = checks + 16;
  int* lens = reinterpret_cast<int*>(pre + a.reqs + 1);
  int* starts = lens + a.reqs;

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);
  JoinRec* recs = reinterpret_cast<JoinRec*>(a.part + 2 * (int64_t)a.ctas * RN * (D + 2));

  // ---- set-up that depends on nothing (it may run while the previous kernel ends), then the plan
  if (tid == 0) {
    s_dead = 0;
    for (int i = 0; i < 8; ++i) checks[i] = 0;
    for (int i = 0; i < G::kBars; ++i) {
      uint64_t* b = bp + i;
      const bool lay = (b >= B.raw_empty && b < B.op_empty) || (b >= B.info && b < B.q_empty);
      const uint32_t n = lay ? 8u : b >= B.op_empty && b < B.info ? 2u : b >= B.p_full && b < B.v_full ? 8u : b >= B.soft ? 4u : 1u;
      mbar_init(b, n + (blockIdx.x == 0 && i == a.stall));
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
    mtail::pdl_wait();
    int bits = 0;
    const uint64_t total64 = plan(a, RN, plan_load(a, lane), pre, lens, starts, &bits);
    if (total64 > 0x7FFFFFFFull) bits |= kStatusBadLength;
    if (blockIdx.x == 0 && bits && a.status) atomicOr(a.status, bits);
    const uint32_t total = total64 > 0x7FFFFFFFull ? 0u : (uint32_t)total64;
    const uint32_t per = total64 > 0x7FFFFFFFull ? 0u : range_tiles(total, a.ctas);
    const uint32_t u0 = (uint32_t)min((uint64_t)blockIdx.x * per, (uint64_t)total);
    __syncwarp();
    const uint32_t u1 = range_end(a, RN, pre, lens, starts, u0, min(total, u0 + per));
    if (lane == 0) s_range[0] = u0, s_range[1] = u1, s_range[2] = per;
  } else {
    // the identity (E2M1 code 2 is 1.0) in rows of 128 bytes, and its scales
    for (int i = tid < 64 ? tid : tid - 32; i < 128 * 8; i += kThreads - 32) {
      const int r = i >> 3, ch = i & 7;
      const uint32_t one = ch == r >> 5 ? 2u << (4 * (r & 7)) : 0u;
      const int w = (r >> 3) & 3;
      *reinterpret_cast<uint4*>(sm + G::oI + r * 128 + ((ch ^ (r & 7)) << 4)) =
          make_uint4(w == 0 ? one : 0u, w == 1 ? one : 0u, w == 2 ? one : 0u, w == 3 ? one : 0u);
    }
    if (warp == 3) *reinterpret_cast<uint4*>(sm + G::oSfI + lane * 16) = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    fence_proxy();
    mtail::pdl_wait();
    if (warp == 1) {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem)) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t u0 = s_range[0], u1 = s_range[1], per = s_range[2];
  const uint32_t tm = __shfl_sync(~0u, s_tmem, 0);
  if (u0 == u1 && tid == 0) recs[blockIdx.x].last = per ? -1 : kRefused;

  // A wait gave up, here or elsewhere in the CTA (of each lane: a warp asks for it by a vote).  From then
  // on a wait takes one sleep at most and every role leaves its loops where it next asks; the
  // softmax and the layout ask in what they read anyway, which warp 0 marks as it leaves.  What a warp
  // still does then may differ from the others', so none waits for another but at these barriers, and
  // all reach the kernel's last.  (Small code: a variable that lives through the steps of all
  // roles, or a longer way out of each wait, cost 4 to 25 % of a long call; this 2 to 3 %.)
  bool gone = false;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (mbar_test(b, parity & 1)) return;  // (quicker than the waiting form where it has completed)
    const uint32_t t0 = clock();
    while (!mbar_sleep_wait(b, parity & 1)) {
      if (*reinterpret_cast<volatile int*>(&s_dead) || (uint32_t)clock() - t0 > kBudgetClocks) {
        *reinterpret_cast<volatile int*>(&s_dead) = 1;
        gone = true;
        return;
      }
    }
  };
  // both, asked for together
  auto wait2 = [&](uint64_t* b0, uint32_t p0, uint64_t* b1, uint32_t p1) {
    const bool d0 = mbar_test(b0, p0 & 1), d1 = mbar_test(b1, p1 & 1);
    if (!d0) wait(b0, p0);
    if (!d1) wait(b1, p1);
    __syncwarp();
  };
  // in front of what a warp does together
  auto wait1 = [&](uint64_t* b, uint32_t parity) {
    wait(b, parity);
    __syncwarp();
  };
  auto dead = [&]() { return __any_sync(~0u, *reinterpret_cast<volatile int*>(&s_dead)) != 0; };
  const int r0 = u0 < u1 ? find_req(pre, a.reqs, u0) : 0;

  if (warp == 0) {
    // ------------------------------------------------------------------ the tiles' copies ----
    Ring<G::kRaw> raw;
    int r = r0;
    for (uint32_t u = u0; u < u1;) {
      const Seg s = open_seg(a, RN, pre, lens, starts, r, u, u1);
      r = s.r;
      const int first = s.j * RN, nrow = min(RN, s.q.nq * a.G - first);
      const int pmin = s.q.L - s.q.nq + first / a.G, pmax = s.q.L - s.q.nq + (first + nrow - 1) / a.G;
      for (int k = s.k0; k < s.k1 && !dead(); k += 32) {
        // a lane looks up one of 32 tiles, the copies of four steps
        const int kk = k + lane, tile = kk < s.q.ns ? kk : kk + s.q.off;
        int64_t at = -1;
        if (kk < s.k1 && tile < s.q.T) {
          const int e = (int)(((uint64_t)(uint32_t)tile * a.page_magic) >> 34);
          const int page = a.table[s.r * a.stride + e];
          if ((uint64_t)(int64_t)page < (uint64_t)a.n_pages)
            at = (((int64_t)page * a.heads + s.h) * a.page_tiles + (tile - e * a.page_tiles)) * G::kTile;
          else if (a.status)
            atomicOr(a.status, kStatusBadPage);
        }
        const int t0 = tile * 16;
        const bool full = at >= 0 && t0 + 15 <= pmin && (a.window == 0 || t0 > pmax - a.window || t0 + 15 < a.sinks);
        const uint32_t have = __ballot_sync(~0u, at >= 0);
        const int steps = (min(32, s.k1 - k) + kStepTiles - 1) / kStepTiles;
        for (int q = 0; q < steps; ++q, raw.next()) {
          const uint32_t st = raw.i;
          wait(B.raw_empty + st, raw.ph ^ 1);
          uint8_t* dst = sm + G::oRaw + st * G::kStep;
          const uint32_t mine = have >> (8 * q) & 255;
          if (lane >> 3 == q) raw_info[st * 20 + (lane & 7)] = at >= 0 ? t0 : -1, raw_info[st * 20 + 8 + (lane & 7)] = full;
          __syncwarp();
          if (__any_sync(~0u, gone)) break;
          if (lane == 0) {
            if (mine) mbar_expect_tx(B.raw_full + st, __popc(mine) * G::kTile);
            else mbar_arrive(B.raw_full + st);
          }
          __syncwarp();
          if (lane >> 3 == q && at >= 0)
            bulk_load(dst + (lane & 7) * G::kTile, a.cache + at, G::kTile, B.raw_full + st);
        }
      }
      u += s.places;
      if (dead()) break;
    }
    if (dead() && lane == 0) {  // (the softmax's checks, the tiles' full marks)
      for (int i = 1; i < 8; i += 2) *reinterpret_cast<volatile uint32_t*>(checks + i) = 1;
      for (int i = 0; i < G::kRaw * 8; ++i) *reinterpret_cast<volatile int*>(raw_info + (i >> 3) * 20 + 8 + (i & 7)) = 0;
    }
  } else if (warp == 1) {
    // --------------------------------------- the tensor cores: K' = K I, S^T = K' Q^T ----
    // The warp stays together; each run of products is one elected thread's (the same every time),
    // whose operands the compiler then keeps in uniform registers: 9 cycles an instruction instead
    // of 46 from a divergent thread.  Sub-step n is half n % kHalves (of the channels) of step n /
    // kHalves.
    const uint32_t base = smem_u32(sm);
    const uint64_t dI = sw128_desc(base + G::oI);
    if (elect_one()) cp_sf(tm + G::cSfI, sf_desc(base + G::oSfI));
    __syncwarp();
    Ring<G::kOps> op;  // of the keys asked for next
    auto k_ident = [&](uint32_t n) {
      const uint32_t h = n % G::kHalves;
      const uint32_t ob = base + G::oOp + op.i * G::kOp, sb = base + G::oSf + op.i * G::kSf;
      const uint32_t sf = tm + G::cSfK + (n / G::kHalves & 1) * 4 * G::kAtoms;
      // the operands, and the scores of the sub-step before: the keys are used up
      if (G::kHalves > 1) {
        if (h == 0) wait(B.op_full + op.i, op.ph);
        wait1(B.k_free, n + 1);
      } else if (n > 0) {
        wait2(B.op_full + op.i, op.ph, B.s_full + ((n - 1) & 1), (n - 1) >> 1);
      } else {
        wait1(B.op_full + op.i, op.ph);
      }
      fence_after();
      if (elect_one()) {
        if (h == 0) {
#pragma unroll
          for (int at = 0; at < G::kAtoms; ++at) cp_sf(sf + 4 * at, sf_desc(sb + 512 * at));
        }
        const uint64_t dK = sw128_desc(ob + 64 * h);
#pragma unroll
        for (int k = 0; k < G::CH / 64; ++k)
          mma_mxf4(tm + G::cK, dK + (uint64_t)(2 * k), dI + (uint64_t)(2 * k), idesc_mxf4(G::CH, 2 * k), sf + 4 * h,
                   tm + G::cSfI, k > 0);
        commit(B.k_full);
        if (h + 1 == G::kHalves) commit(B.op_empty + op.i);
      }
      __syncwarp();
      if (h + 1 == G::kHalves) op.next();
    };
    uint32_t n = 0;
    Ring<G::kQs> qr;
    int r = r0;
    if (u0 < u1) k_ident(0);
    for (uint32_t u = u0; u < u1; qr.next()) {
      const Seg s = open_seg(a, RN, pre, lens, starts, r, u, u1);
      r = s.r;
      u += s.places;
      const int subs = (s.k1 - s.k0 + kStepTiles - 1) / kStepTiles * G::kHalves;
      const uint32_t q0 = base + G::oQ + qr.i * G::kQ;
      wait(B.q_full + qr.i, qr.ph);
      for (int st = 0; st < subs; ++st, ++n) {
        if (__any_sync(~0u, gone)) break;
        const uint32_t i = n / G::kHalves, h = n % G::kHalves, ib = i & 1;
        // the keys are there, the scores two steps ago are read
        wait2(B.k_full, n, B.p_full + ib, (i >> 1) + 1);
        fence_after();
        if (elect_one()) {
          const uint64_t dQ = sw128_desc(q0 + h * (NM * 512));
          const uint32_t d = tm + G::cS + ib * NM;
#pragma unroll
          for (int k = 0; k < G::CH / 8; ++k)
            mma_tf32(d, tm + G::cK + 8 * k, dQ + (uint64_t)(((k >> 2) * NM * 128 + (k & 3) * 32) >> 4),
                     idesc_tf32(NM), k > 0 ? 1u : h);
          if (G::kHalves > 1) commit(B.k_free);
          if (h + 1 == G::kHalves) commit(B.s_full + ib);
          if (st + 1 == subs) commit(B.q_empty + qr.i);
        }
        __syncwarp();
        if (st + 1 < subs || u < u1) k_ident(n + 1);
      }
      if (__any_sync(~0u, gone)) break;
    }
  } else if (warp == kValWarp) {
    // ------------------------------------- the tensor cores: V' = I V^T, O^T += V' P^T ----
    const uint32_t base = smem_u32(sm);
    const uint64_t dI = sw128_desc(base + G::oI);
    if (elect_one()) cp_sf(tm + G::cSfJ, sf_desc(base + G::oSfI));
    __syncwarp();
    Ring<G::kOps> op;  // of the values asked for next
    auto v_ident = [&](uint32_t n) {
      const uint32_t h = n % G::kHalves, nb = n % G::kVs;
      const uint32_t ob = base + G::oOp + op.i * G::kOp, sb = base + G::oSf + op.i * G::kSf + 512 * G::kAtoms;
      const uint32_t sf = tm + G::cSfV + (n / G::kHalves & 1) * 4 * G::kAtoms;
      // the operands, and the last product that read the values in this place
      wait2(B.op_full + op.i, op.ph, (G::kHalves > 1 ? B.v_free : B.pv) + nb, n / G::kVs + 1);
      fence_after();
      if (elect_one()) {
        if (h == 0) {
#pragma unroll
          for (int at = 0; at < G::kAtoms; ++at) cp_sf(sf + 4 * at, sf_desc(sb + 512 * at));
        }
        const uint64_t dV = sw128_desc(ob + (D == 256 ? 16384 + 64 * h : 64));
        const uint32_t d = tm + G::cV + 128 * nb;
#pragma unroll
        for (int k = 0; k < G::CH / 64; ++k)
          mma_mxf4(d, dI + (uint64_t)(2 * k), dV + (uint64_t)(2 * k), idesc_mxf4(128, 2 * k), tm + G::cSfJ,
                   sf + 4 * h, k > 0);
        commit(B.v_full + nb);
        if (h + 1 == G::kHalves) commit(B.op_empty + op.i);
      }
      __syncwarp();
      if (h + 1 == G::kHalves) op.next();
    };
    uint32_t n = 0;
    int r = r0;
    if (u0 < u1) v_ident(0);
    for (uint32_t u = u0; u < u1;) {
      const Seg s = open_seg(a, RN, pre, lens, starts, r, u, u1);
      r = s.r;
      u += s.places;
      const int subs = (s.k1 - s.k0 + kStepTiles - 1) / kStepTiles * G::kHalves;
      for (int st = 0; st < subs; ++st, ++n) {
        if (__any_sync(~0u, gone)) break;
        const uint32_t i = n / G::kHalves, h = n % G::kHalves, ib = i & 1, nb = n % G::kVs;
        // (with two halves the next values would come too late behind this product, with one this
        // product behind the next values)
        bool next = st + 1 < subs || u < u1;
        if (G::kHalves > 1 && G::kVs > 1 && next && __all_sync(~0u, mbar_test(B.op_full + op.i, op.ph))) {
          v_ident(n + 1);
          next = false;
        }
        wait2(B.v_full + nb, n / G::kVs, B.p_full + ib, i >> 1);
        fence_after();
        if (elect_one()) {
          const uint64_t dP = sw128_desc(base + G::oP + ib * G::kP);
          const uint32_t d = tm + G::cO + h * NM, av = tm + G::cV + 128 * nb, keep = st < G::kHalves ? 0u : 1u;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            mma_tf32(d, av + 8 * k, dP + (uint64_t)(((k >> 2) * NM * 128 + (k & 3) * 32) >> 4), idesc_tf32(NM),
                     k > 0 ? 1u : keep);
          if (G::kHalves > 1) commit(B.v_free + nb);
          if (h + 1 == G::kHalves) commit(B.pv + ib);
        }
        __syncwarp();
        if (next) v_ident(n + 1);
      }
      if (__any_sync(~0u, gone)) break;
    }
  } else if (warp < kLayWarp || warp >= kSoft2Warp) {
    // -------------------------------------------------------------- the softmax, the output ----
    constexpr int RH = RN / 2;                       // rows of this warp: half of the item's
    const int half = warp < kLayWarp ? 0 : 1, k0 = half * RH;
    const int quad = warp & 3;                       // tensor-memory lanes 32 quad ..
    const uint32_t tl = tm + ((uint32_t)quad << 21);  // (lane in bits 16..)
    const int tok = 32 * quad + lane;                // this thread's token of a step
    uint32_t* check = checks + 4 * half;
    // where this token's numerators of rows k0 + k go (k and k + 8 lie 1024 bytes apart)
    uint8_t* ps[RH < 8 ? RH : 8];
#pragma unroll
    for (int k = 0; k < (RH < 8 ? RH : 8); ++k)
      ps[k] = sm + G::oP + quad * (NM * 128) + (k0 + k) * 128 + (((lane >> 2) ^ ((k0 + k) & 7)) << 4) + (lane & 3) * 4;
    float* hred = red + half * 4 * RH;  // [2 turns][2 halves][4][RH]
    float* hsum = lsum + half * 4 * RH;
    int turn = 0, part = 0;
    uint32_t i = 0, nchecks = 0, meets = 0;
    Seg s;
    int first = 0, nrow = 0;
    auto open = [&](int r, uint32_t u) {  // the part from u on, its rows' positions
      s = open_seg(a, RN, pre, lens, starts, r, u, u1);
      first = s.j * RN, nrow = min(RN, s.q.nq * a.G - first);
      if (quad == 0 && lane < RH) {
        const int k = k0 + lane;
        rowpos[(part & 1) * RN + k] = s.q.L - s.q.nq + (first + min(k, nrow - 1)) / a.G;
        nanrow[(part & 1) * RN + k] = 0;
      }
    };
    auto meet = [&]() {  // the four warps of this half: each sees what the others have stored
      __syncwarp();
      if (lane == 0) mbar_arrive(B.meet + half);
      wait1(B.meet + half, meets++);
    };
    if (u0 < u1) open(r0, u0);
    meet();
    for (uint32_t u = u0; u < u1 && !dead(); ++part) {
      const int* rowp = rowpos + (part & 1) * RN + k0;
      uint32_t* nanr = nanrow + (part & 1) * RN + k0;
      const int steps = (s.k1 - s.k0 + kStepTiles - 1) / kStepTiles;
      float l[RH], m[RH];
#pragma unroll
      for (int k = 0; k < RH; ++k) l[k] = 0.f, m[k] = kLow;
      for (int st = 0; st < steps; ++st, ++i) {
        const uint32_t b = i & 1;
        const Info& inf = infos[i % kInfos];
        const uint32_t sa = tl + G::cS + b * NM + k0;
        wait1(B.s_full + b, i >> 1);
        fence_after();
        // the notes of the step, and the product that read the numerators before these (both are
        // there by now as a rule: their tests run beside the load)
        const bool d0 = mbar_test(B.info + i % kInfos, i / kInfos & 1), d1 = mbar_test(B.pv + b, ((i >> 1) + 1) & 1);
        float x[RH];
        tmem_ld<RH>(sa, x);
        if (!d0) wait(B.info + i % kInfos, i / kInfos);
        uint32_t seen = ~0u, fl = 0;
        if (inf.plain != 0x0101010101010101ull) {
          int t0 = inf.t0[tok >> 4], t = t0 < 0 ? INT32_MAX : t0 + (tok & 15);
          fl = inf.flags[tok];
          if (inf.plain >> (8 * (tok >> 4)) & 1) t = INT32_MIN, fl = 0;
          // the rows' positions ascend: most tokens are seen by all of them or by none
          const int p0 = rowp[0], p1 = rowp[RH - 1];
          const bool out = a.window != 0 && t >= a.sinks;  // (only a window shows it)
          if (t == INT32_MIN || (t <= p0 && !(out && t <= p1 - a.window))) {
          } else if (t > p1 || (out && p0 >= 0 && t <= p0 - a.window)) {
            seen = 0;
          } else {
            seen = 0;
#pragma unroll
            for (int k = 0; k < RH; ++k) {
              const int p = rowp[k];
              if (t <= p && !(out && t <= p - a.window)) seen |= 1u << k;
            }
          }
          if (__any_sync(~0u, fl != 0 || seen != ~0u)) {
#pragma unroll
            for (int k = 0; k < RH; ++k) {
              if (fl >> 15) x[k] = __uint_as_float(0x7FC00000u);  // a NaN among the key scales
              if (!(seen >> k & 1)) x[k] = -INFINITY;
              else if (fl & 255u) atomicOr(nanr + k, fl & 255u);  // value scales
            }
          }
        }
        bool move = st == 0;  // the rows' references move
        const uint32_t cb = nchecks & 1;
        if (!move) {
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < RH; ++k) {
            x[k] = fmaf(x[k], a.scale_log2, -m[k]);
            top = fmaxf(top, x[k]);
          }
          const bool mine = __any_sync(~0u, top > kOver);
          if (lane == 0) {
            reinterpret_cast<uint8_t*>(check + 2 * cb)[quad] = mine;
            mbar_arrive(B.soft + 2 * half + cb);
          }
        }
        if (!d1) wait(B.pv + b, (i >> 1) + 1);
        const uint32_t pb = b * G::kP;
        float p[RH];
        auto numerators = [&]() {
#pragma unroll
          for (int k = 0; k < RH; ++k) {
            p[k] = ex2(x[k]);
            *reinterpret_cast<float*>(ps[k & 7] + pb + (k >> 3) * 1024) = to_tf32(p[k]);
          }
        };
        if (!move) {
          numerators();
          wait1(B.soft + 2 * half + cb, nchecks++ >> 1);
          const uint64_t c = *reinterpret_cast<volatile uint64_t*>(check + 2 * cb);
          move = c != 0;
          if (move) {  // from the scores themselves
            if (c >> 32) break;
            tmem_ld<RH>(sa, x);
#pragma unroll
            for (int k = 0; k < RH; ++k) {
              if (fl >> 15) x[k] = __uint_as_float(0x7FC00000u);
              if (!(seen >> k & 1)) x[k] = -INFINITY;
            }
          }
        }
        if (move) {
          // to the maxima over this step's 128 tokens (eight rows at a time: with 16 a warp is short
          // of registers)
          constexpr int C = RH < 8 ? RH : 8;
          float* hr = hred + (turn ^= 1) * 8 * RH;  // (the turn before may still be read)
#pragma unroll
          for (int c = 0; c < RH; c += C) {
            float y[C];
#pragma unroll
            for (int k = 0; k < C; ++k) y[k] = x[c + k] = x[c + k] * a.scale_log2;
            const float w = warp_max_of<C>(y);
            if (lane < C) hr[quad * RH + c + lane] = w;
          }
          meet();
          if (st > 0) {  // the sums so far, once no product adds to them
            wait1(B.pv + ((i - 1) & 1), (i - 1) >> 1);
            fence_after();
          }
#pragma unroll
          for (int c = 0; c < RH; c += C) {
            float f[C];
#pragma unroll
            for (int k = 0; k < C; ++k) {
              const float d = fmaxf(fmaxf(hr[c + k], hr[RH + c + k]), fmaxf(hr[2 * RH + c + k], hr[3 * RH + c + k]));
              const float old = m[c + k];
              m[c + k] = fmaxf(old, d);
              x[c + k] -= m[c + k];
              f[k] = ex2(old - m[c + k]);
              l[c + k] *= f[k];
            }
            if (st > 0) {
#pragma unroll
              for (int h = 0; h < G::kHalves; ++h) {
                float o[C];
                tmem_ld<C>(tl + G::cO + h * NM + k0 + c, o);
#pragma unroll
                for (int k = 0; k < C; ++k) o[k] *= f[k];
                tmem_st<C>(tl + G::cO + h * NM + k0 + c, o);
              }
            }
          }
          numerators();
        }
#pragma unroll
        for (int k = 0; k < RH; ++k) l[k] += p[k];
        fence_proxy();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(B.p_full + b);
      }

      // ---- the part's sums and averages; what need not wait for the last product, the next part's
      // opening among it, comes first
      const float lw = warp_sum_of<RH>(l);
      if (lane < RH) hsum[quad * RH + lane] = lw;
      const bool whole = s.k0 == 0 && s.k1 == s.q.n;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (s.k0 == 0 ? 1 : 0);
      const int rows = nrow;
      // lane k of each warp: where row k0 + k goes
      const int kl = k0 + (lane < RH ? lane : 0);
      int64_t at_l = (slot * RN + kl) * D;
      if (whole) {
        const int rho = first + kl, tk = rho / a.G;
        at_l = (starts[s.r] + tk) * a.ldo + (int64_t)(s.h * a.G + rho - tk * a.G) * D;
      }
      u += s.places;
      if (u >= u1) {
        if (warp == 4 && lane == 0) {
          JoinRec rec;
          rec.last = s.k0 == 0 && !whole ? (int)((s.item + (uint32_t)(s.q.n + kItemTiles) - 1) / per) : -1;
          rec.row0 = starts[s.r], rec.first = first, rec.head = s.h, rec.rows = nrow;
          rec.pad[0] = rec.pad[1] = rec.pad[2] = 0;
          recs[blockIdx.x] = rec;
        }
      } else {
        ++part;
        open(s.r, u);
        --part;
      }
      meet();
      // ... its 1 / sum and its NaN blocks
      const float sum = (hsum[kl - k0] + hsum[RH + kl - k0]) + (hsum[2 * RH + kl - k0] + hsum[3 * RH + kl - k0]);
      const float inv_l = sum == 0.f ? 0.f : 1.f / sum;
      const uint32_t nan_l = nanr[kl - k0];
      const bool nans = __any_sync(~0u, nan_l != 0);
      if (!whole) {
        float* pml = a.part + 2 * (int64_t)a.ctas * RN * D + slot * RN * 2;
        float mk = m[0];
#pragma unroll
        for (int k = 1; k < RH; ++k) mk = lane == k ? m[k] : mk;
        if (quad == 0 && lane < RH && kl < rows) *reinterpret_cast<float2*>(pml + 2 * kl) = make_float2(mk, sum);
      }
      wait1(B.pv + ((i - 1) & 1), (i - 1) >> 1);
      fence_after();
      // the joining launch may line up now (from the start on, its CTAs had cost 2 us a call)
      if (u >= u1) mtail::pdl_trigger();
#pragma unroll
      for (int h = 0; h < G::kHalves; ++h) {
        float o[RH];
        tmem_ld<RH>(tl + G::cO + h * NM + k0, o);
        const int ch = 128 * h + tok;  // (D 64: the upper lanes hold zeros)
#pragma unroll
        for (int k = 0; k < RH; ++k) {
          const int64_t at = __shfl_sync(~0u, at_l, k);
          float v = o[k] * __shfl_sync(~0u, inv_l, k);
          if (nans && (__shfl_sync(~0u, nan_l, k) >> (ch >> 5) & 1)) v = __uint_as_float(0x7FC00000u);
          if (k0 + k < rows && tok < G::CH) {
            if (whole) a.out[at + ch] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
            else a.part[at + ch] = v;
          }
        }
      }
      fence_before();
    }
  } else {
    // ----------------------------------------- cached bytes into the tensor cores' operands ----
    const int j = warp - kLayWarp, g = lane >> 2, c = lane & 3, t = lane & 15;
    // where this lane's words go in a step's operands: keys, word w = 4 v + x is block w mod NB of
    // token 8 (w / NB) + g; values, the four words of a transposing load are block (8 v + g) mod NB of
    // token 8 (ho / 2) + 2 c + ho mod 2, ho = (8 v + g) / NB; scales, a word of the token's row
    uint32_t ko[NB], vo;
#pragma unroll
    for (int b = 0; b < NB; ++b) ko[b] = (16 * j + g) * 128 + ((b ^ g) << 4) + 4 * c;
    {
      const int ho = g / NB, b = g % NB;
      const int tt = 8 * (ho >> 1) + 2 * c + (ho & 1);
      vo = (D == 256 ? 16384 : 0) + (16 * j + tt) * 128 + (((D == 256 ? b : 4 + b) ^ (tt & 7)) << 4);
    }
    const uint32_t so = (lane < 16 ? 0 : 512 * G::kAtoms) + 16 * ((16 * j + t) & 31) + 4 * ((16 * j + t) >> 5);
    // of the transposing loads: matrix x takes rows (c, g) for g = 2 x, 2 x + 1, 128 bytes side by side
    const uint32_t va = ((2 * (lane >> 3) + (lane & 1)) * 4 + ((lane & 7) >> 1)) * 16;
    const uint32_t vsel = (2 * (t >> 3) + (t & 1)) * 0x11u + 0x40u;  // this token's byte of two words
    Ring<G::kRaw> raw;
    Ring<G::kOps> op;
    Ring<G::kQs> qr;
    uint32_t i = 0;
    int r = r0;
    for (uint32_t u = u0; u < u1; qr.next()) {
      if (dead()) break;
      const Seg s = open_seg(a, RN, pre, lens, starts, r, u, u1);
      r = s.r;
      const int first = s.j * RN, nrow = min(RN, s.q.nq * a.G - first), row0 = starts[s.r];
      const int pmax = s.q.L - s.q.nq + (first + nrow - 1) / a.G;
      const int steps = (s.k1 - s.k0 + kStepTiles - 1) / kStepTiles;
      // the item's queries: bf16 to tf32, rows of 32 channels
      {
        uint8_t* dst = sm + G::oQ + qr.i * G::kQ;
        constexpr int E = (D + 127) / 128, R8 = NM / 8;
        uint2 qv[R8][E];
#pragma unroll
        for (int rr = 0; rr < R8; ++rr) {
          const int k = j + 8 * rr, rho = first + k, tk = rho / a.G;
          const uint16_t* p = a.q + (row0 + tk) * a.ldq + (int64_t)(s.h * a.G + rho - tk * a.G) * D;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int ch = 128 * e + 4 * lane;
            qv[rr][e] = k < nrow && ch < D ? *reinterpret_cast<const uint2*>(p + ch) : make_uint2(0, 0);
          }
        }
        wait(B.q_empty + qr.i, qr.ph ^ 1);
#pragma unroll
        for (int rr = 0; rr < R8; ++rr)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int k = j + 8 * rr, ch = 128 * e + 4 * lane;
            const uint2 v = qv[rr][e];
            if (ch < D)
              *reinterpret_cast<uint4*>(dst + (ch >> 5) * (NM * 128) + k * 128 + ((((ch & 31) >> 2) ^ (k & 7)) << 4)) =
                  make_uint4(v.x << 16, v.x & 0xFFFF0000u, v.y << 16, v.y & 0xFFFF0000u);
          }
        fence_proxy();
        __syncwarp();
        if (lane == 0) mbar_arrive(B.q_full + qr.i);
      }
      for (int st = 0; st < steps; ++st, ++i, raw.next(), op.next()) {
        wait1(B.raw_full + raw.i, raw.ph);
        const uint8_t* tp = sm + G::oRaw + raw.i * G::kStep + j * G::kTile;
        // keys: lane (g, c) holds 8 channels of each block of tokens g and g + 8
        uint32_t kw[D / 16], vw[D / 16];
#pragma unroll
        for (int v = 0; v < D / 64; ++v) {
          const uint4 x = *reinterpret_cast<const uint4*>(tp + v * 512 + lane * 16);
          kw[4 * v] = x.x, kw[4 * v + 1] = x.y, kw[4 * v + 2] = x.z, kw[4 * v + 3] = x.w;
        }
        // values: a transposing load brings the pieces of lanes g = 0..7 (4 bytes from each two) of one
        // token and block together: 16 bytes of its row
#pragma unroll
        for (int v = 0; v < D / 64; ++v)
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                       : "=r"(vw[4 * v]), "=r"(vw[4 * v + 1]), "=r"(vw[4 * v + 2]), "=r"(vw[4 * v + 3])
                       : "r"(smem_u32(tp) + 8 * D + v * 512 + va));
        // scales of token t: lanes 0..15 of its keys, lanes 16..31 of its values (a byte of each word)
        uint32_t sw[G::kAtoms];
        {
          const uint8_t* kp = tp + 16 * D + (t & 7) * (D / 16) + (t >> 3) * NB;
          const uint32_t* vp = reinterpret_cast<const uint32_t*>(tp + 16 * D + D / 2 + ((t & 7) >> 1) * (D / 8));
#pragma unroll
          for (int at = 0; at < G::kAtoms; ++at) {
            uint32_t k4, w[4] = {0, 0, 0, 0};
            if constexpr (NB == 2) {
              k4 = *reinterpret_cast<const uint16_t*>(kp);
              const uint2 x = *reinterpret_cast<const uint2*>(vp);
              w[0] = x.x, w[1] = x.y;
            } else {
              k4 = reinterpret_cast<const uint32_t*>(kp)[at];
              const uint4 x = reinterpret_cast<const uint4*>(vp)[at];
              w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            }
            uint32_t v4 = __byte_perm(w[0], w[1], vsel);
            v4 = NB == 2 ? v4 & 0xFFFFu : __byte_perm(v4, __byte_perm(w[2], w[3], vsel), 0x5410);
            sw[at] = lane < 16 ? k4 : v4;
          }
        }
        const int t0 = raw_info[raw.i * 20 + j], full = raw_info[raw.i * 20 + 8 + j];
        uint32_t nan = 0;
#pragma unroll
        for (int at = 0; at < G::kAtoms; ++at) nan |= ((sw[at] & 0x7F7F7F7Fu) + 0x01010101u) & sw[at] & 0x80808080u;
        Info& inf = infos[i % kInfos];
        const bool plain = full && !__any_sync(~0u, nan != 0);
        if (!plain) {
          if (dead()) break;
          // zero scales for tokens that no row sees, and for NaN scales, which the flags report
          const bool unseen = t0 < 0 || t0 + t > pmax;
          uint32_t fl = 0;
#pragma unroll
          for (int at = 0; at < G::kAtoms; ++at) {
            const uint32_t f = unseen ? 0u : ff_bytes(sw[at]);
            fl |= f << (4 * at);
#pragma unroll
            for (int b = 0; b < 4; ++b)
              if (unseen || (f >> b & 1)) sw[at] &= ~(0xFFu << (8 * b));
          }
          const uint32_t vfl = __shfl_sync(~0u, fl, 16 + t);
          if (lane < 16) inf.flags[16 * j + t] = (uint16_t)((fl ? 0x8000u : 0u) | vfl);
          if (lane == 16) inf.t0[j] = t0;
        }
        if (lane == 16) reinterpret_cast<uint8_t*>(&inf.plain)[j] = plain;
        wait(B.op_empty + op.i, op.ph ^ 1);
        uint8_t* ob = sm + G::oOp + op.i * G::kOp;
#pragma unroll
        for (int w = 0; w < D / 16; ++w) *reinterpret_cast<uint32_t*>(ob + ko[w % NB] + (w / NB) * 1024) = kw[w];
        // (a vector v further is 8 / NB values of ho: D 64 has one, D 128 8 tokens, D 256 one of the two
        // tokens of a pair, whose rows differ in their swizzle)
#pragma unroll
        for (int v = 0; v < D / 64; ++v) {
          uint32_t o = vo;
          if (D == 128) o += 1024 * v;
          if (D == 256) o = ((o + 128 * (v & 1)) ^ (16u * (v & 1))) + 1024 * (v >> 1);
          *reinterpret_cast<uint4*>(ob + o) = make_uint4(vw[4 * v], vw[4 * v + 1], vw[4 * v + 2], vw[4 * v + 3]);
        }
        uint8_t* sb = sm + G::oSf + op.i * G::kSf + so;
#pragma unroll
        for (int at = 0; at < G::kAtoms; ++at) *reinterpret_cast<uint32_t*>(sb + 512 * at) = sw[at];
        fence_proxy();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(B.raw_empty + raw.i);
          mbar_arrive(B.info + i % kInfos);
          mbar_arrive(B.op_full + op.i);
        }
      }
      u += s.places;
    }
  }

  if (*reinterpret_cast<volatile int*>(&s_dead)) {
    if (lane == 0 && a.status) atomicOr(a.status, kStatusTimeout);
    // let the copies and products in flight end before their memory goes
    const int64_t t0 = clock64();
    while (clock64() - t0 < 2000000) __nanosleep(1000);
  }
  fence_before();
  __syncthreads();
  if (*reinterpret_cast<volatile int*>(&s_dead)) {
    const volatile uint32_t* range = s_range;  // (read again: kept in registers it cost the steps spills)
    forsake<D, RN>(a, pre, lens, starts, range[0], range[1], range[2]);
  }
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tm));
}

// Joins the parts of the items that several ranges share.  CTA (x, y): the item that crosses the
// end of range x for the first time, rows 4 y .. 4 y + 3, one per warp:
//   out = sum_k w_k o_k / sum_k w_k,  w_k = l_k 2^(m_k - max m), in range order.
// The first parts are on their way while the weights are formed.  It reads its parts once (5 MB with
// 16 rows of 128 in 152 ranges) and costs a call about 3 us, most of it a chain of three dependent
// loads behind the main launch's end.
template <int D, int RN>
__global__ void __launch_bounds__(128) k_kv4_join(const __grid_constant__ AttnArgs a) {
  extern __shared__ float sw[];  // [4][ctas]: weights of a warp's row
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  mtail::pdl_trigger();
  mtail::pdl_wait();
  const JoinRec rec = reinterpret_cast<const JoinRec*>(a.part + 2 * (int64_t)a.ctas * RN * (D + 2))[blockIdx.x];
  const int i = blockIdx.y * 4 + warp;
  if (rec.last == kRefused) {  // NaN for every row of a request
    const int w = (blockIdx.x * gridDim.y + blockIdx.y) * 4 + warp, width = a.heads * a.G * D;
    for (int r = 0; r < a.reqs; ++r) {
      int bits = 0;
      const int rs = a.row_starts[r], n = req_of(a, RN, a.kv_lens[r], rs, a.row_starts[r + 1], &bits).nq;
      for (int t = w; t < n; t += gridDim.x * gridDim.y * 4)
        for (int c = lane; c < width; c += 32) a.out[(int64_t)(rs + t) * a.ldo + c] = 0x7FC0;
    }
    return;
  }
  if (rec.last < 0 || i >= rec.rows) return;
  const int c0 = blockIdx.x, n = rec.last - c0 + 1;
  // part k's slot: the item begins in the second one of its first range, then takes the first ones
  auto slot = [&](int k) { return 2 * (int64_t)(c0 + k) + (k == 0 ? 1 : 0); };
  const float2* ml = reinterpret_cast<const float2*>(a.part + 2 * (int64_t)a.ctas * RN * D) + i;
  const float* po = a.part + (int64_t)i * D;
  float* w = sw + warp * a.ctas;
  constexpr int E = D / 32, kAhead = 8;  // channels of a lane (2 or 4 side by side), parts on their way
  constexpr int V = E == 2 ? 2 : 4, C = E / V;
  float x[kAhead][E];
  auto load = [&](int k, float* v) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float* p = po + slot(k) * RN * D + (c * 32 + lane) * V;
      if constexpr (V == 2) {
        const float2 t = *reinterpret_cast<const float2*>(p);
        v[0] = t.x, v[1] = t.y;
      } else {
        const float4 t = *reinterpret_cast<const float4*>(p);
        v[4 * c] = t.x, v[4 * c + 1] = t.y, v[4 * c + 2] = t.z, v[4 * c + 3] = t.w;
      }
    }
  };
  float2 mine = make_float2(kLow, 0.f);
  if (lane < n) mine = ml[slot(lane) * RN];
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (k < n) load(k, x[k]);
  float m = mine.x, sum = 0.f;
  for (int k = 32 + lane; k < n; k += 32) m = fmaxf(m, ml[slot(k) * RN].x);
  m = __shfl_sync(~0u, mtail::warp_max(m), 0);
  for (int k = lane; k < n; k += 32) {
    const float2 v = k < 32 ? mine : ml[slot(k) * RN];
    const float wk = v.y * ex2(v.x - m);
    w[k] = wk;
    sum += wk;
  }
  sum = __shfl_sync(~0u, mtail::warp_sum(sum), 0);
  __syncwarp();
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int k0 = 0; k0 < n; k0 += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (k0 + k < n) {
        const float wk = w[k0 + k];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(wk, x[k][e], o[e]);
        if (k0 + k + kAhead < n) load(k0 + k + kAhead, x[k]);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int rho = rec.first + i, tok = rho / a.G;
  uint16_t* orow = a.out + (rec.row0 + tok) * a.ldo + (int64_t)(rec.head * a.G + rho - tok * a.G) * D;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(o[V * c + e] * inv, o[V * c + e + 1] * inv);
      *reinterpret_cast<uint32_t*>(orow + (c * 32 + lane) * V + e) = *reinterpret_cast<const uint32_t*>(&v);
    }
}

template <int D, int RN>
cudaError_t prepare() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  // once per device (racing threads do the same)
  static std::atomic<int> known[64];
  if (dev < 64 && known[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(k_kv4_attn<D, RN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)Geo<D, RN>::smem(Geo<D, RN>::kReqs));
  if (e == cudaSuccess && dev < 64) known[dev].store(1, std::memory_order_release);
  return e;
}

template <int D, int RN>
cudaError_t launch(const AttnArgs& a, cudaStream_t st) {
  static_assert(Geo<D, RN>::smem(Geo<D, RN>::kReqs) <= 232448 - 256, "shared memory");
  cudaError_t e = prepare<D, RN>();
  if (e != cudaSuccess) return e;
  e = mtail::launch_k(k_kv4_attn<D, RN>, dim3(a.ctas), dim3(kThreads), Geo<D, RN>::smem(a.reqs), st, true, a);
  if (e != cudaSuccess || a.ctas < 2) return e;
  return mtail::launch_k(k_kv4_join<D, RN>, dim3(a.ctas - 1, RN / 4), dim3(128), (size_t)a.ctas * 4 * sizeof(float), st, true, a);
}

template <typename F>
cudaError_t dispatch(int D, int rn, F&& f) {
  switch (D * 100 + rn) {
    case 6408: return f(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
    case 6416: return f(std::integral_constant<int, 64>(), std::integral_constant<int, 16>());
    case 6432: return f(std::integral_constant<int, 64>(), std::integral_constant<int, 32>());
    case 12808: return f(std::integral_constant<int, 128>(), std::integral_constant<int, 8>());
    case 12816: return f(std::integral_constant<int, 128>(), std::integral_constant<int, 16>());
    case 12832: return f(std::integral_constant<int, 128>(), std::integral_constant<int, 32>());
    case 25608: return f(std::integral_constant<int, 256>(), std::integral_constant<int, 8>());
    case 25616: return f(std::integral_constant<int, 256>(), std::integral_constant<int, 16>());
    case 25632: return f(std::integral_constant<int, 256>(), std::integral_constant<int, 32>());
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int attn_rows_per_item(int G, int max_new) {
  const int64_t rows = (int64_t)G * max_new;
  return rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

int attn_ctas(cudaError_t* err) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  *err = e;
  return e == cudaSuccess ? sms : 0;
}

size_t attn_workspace_bytes(int D, int rn, int ctas) {
  return (size_t)2 * ctas * rn * (D + 2) * sizeof(float) + (size_t)ctas * sizeof(JoinRec);
}

cudaError_t launch_kv4_attention(const AttnArgs& a, int rn, cudaStream_t st) {
  if (a.D == 256 && a.reqs > Geo<256, 32>::kReqs) rn = std::min(rn, 16);
  return dispatch(a.D, rn, [&](auto d, auto n) { return launch<decltype(d)::value, decltype(n)::value>(a, st); });
}

}  // namespace kv4
