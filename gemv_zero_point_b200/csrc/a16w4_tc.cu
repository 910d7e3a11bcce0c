// Weight-only int4 products on the 5th-generation tensor cores, for many rows
// per expert: the forward product and the gradient with respect to its input.
//
//   forward   y[p,n]  = sum_k x[p,k] * w[n,k] + bias[n]     features n, reduction k
//   gradient  dx[p,k] = sum_n dy[p,n] * w[n,k]              features k, reduction n
//
// One tile is 256 features on a pair of CTAs (cta_group::2: 128 features, MMA
// M, TMEM lanes, in each) x up to 256 rows (MMA N, TMEM columns): the rows are
// the side of free size, so the ragged row counts of experts waste little.
// The weights are expanded to bf16 on the way into shared memory: w is formed
// as the real value and rounded to bf16 once (half a step, 2^-8 of w), the
// price of one MMA per weight; the sums stay in f32 (TMEM) and the output is
// rounded once.  An MMA adds 16 products to a sum and cuts it off towards zero
// (a reduction of 2^24 came out 1 to 2 % short, the exact sums of whole numbers
// exact); a shared reduction has shorter sums.
//
// In a pair each CTA stages half of the rows, so 64 k of 256 rows x 256
// features move 72 KB through a CTA's shared memory for 512 cycles of MMAs (a
// CTA on its own with 256 rows: 104 KB).  A single CTA with 128 rows remains
// for calls with few tiles, where pairs would leave SMs without work.
//
// What bounds it otherwise are the hand-offs between the roles: with no
// copy, expansion or MMA left in it, a 64-wide stage still took 500 to 600
// cycles.  So a stage is 128 wide (two sub-tiles of one swizzle row each), has
// one barrier for rows and weights together, and all of its MMAs are issued
// by an elected thread of a converged warp (from a lane picked by number the
// operands go through slower registers: 415 against 352 us at
// 4096x14336x4096).  Per stage of a full tile 64 KB of weights and 64 KB of
// rows go in and out of shared memory, 1024 cycles at its rate, as long as the
// MMAs: 4096x14336x4096 with bf16 scales takes 318 us in a burst at 1965 MHz
// (1510 TFLOP/s, tensor pipe 92 % of the busy cycles) and 370 us back to back
// for seconds, where the power limit holds the clock at 1340 MHz (1300 TFLOP/s);
// 64x14336x4096 takes 21 us (about 1000 cycles a stage, half of them the
// weights' way through shared memory).
//
// Both directions read the same 128 rows n x 128 k of the packed matrix per
// stage.  Forward the bf16 sub-tiles are K-major; for the gradient the
// features (k) run along the rows, so the same row-wise expansion writes an
// MN-major operand: no transpose anywhere.
//
// Roles (768 threads, one CTA per SM, persistent over tiles):
//   warp 0      rows: tensor copies of 64-wide slices (128-byte swizzle)
//   warp 1      TMEM; MMA issue by one thread (of the pair's first CTA), one
//               commit per stage and one per tile
//   warp 2      nibbles: tensor copies, a ring of their own
//   warps 4-7   epilogue: TMEM -> bf16 -> global, overlapping the next tile
//   warps 8-23  expansion of the nibbles into the swizzled bf16 stage, two
//               groups of eight warps that take the stages in turn (one stage
//               takes a group about 700 cycles, mostly latencies)
// Indirect rows are first brought into sorted order in the workspace (24 us
// for 32768 rows of 2048, 215 us in all with 64 experts of 1536 features):
// gathering them here took 963 us in all with tensor-map row
// gathers of four rows, 534 with cp.async.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "a16w4.cuh"

namespace qg {

namespace {

constexpr int TF = 128;                    // features per CTA and tile
constexpr int KS = 64;                     // reduction per sub-tile: one 128-byte swizzle row
constexpr int SUBS = 2;                    // sub-tiles per stage
constexpr int KST = KS * SUBS;             // reduction per stage
constexpr int XR = 128;                    // rows per CTA and tile at most
// Rows per tensor copy: the smallest of these that holds a CTA's rows.  One
// copy takes the copy engine some 350 cycles whatever its size, so a stage is
// one copy: both sub-tiles of all rows.
constexpr int kBoxes = 3;
__host__ __device__ constexpr int box_rows(int i) { return 32 << i; }
__device__ __forceinline__ int box_of(int rows) { return rows <= 32 ? 0 : rows <= 64 ? 1 : 2; }
constexpr int STAGES = 3;
constexpr int NRING = 3;
// Signals that the two expansion groups wait for have a barrier per stage mod
// 6, not per slot: a group sees every other stage, so with three barriers it
// would see every other phase of each, and a wait by parity passes when the
// phase before the skipped one is the last to have ended (the copies of two
// slots may land out of order).  With six, every phase of a barrier is waited
// for by the one group that uses it.
constexpr int NBAR = 6;
static_assert(STAGES == 3 && NRING == 3, "stages mod 6 give the slot and the group");
constexpr int kBarriers = STAGES + 2 * NBAR + NRING + 5;
constexpr int X_BYTES = XR * KS * 2;       // 16 KiB per sub-tile
constexpr int W_BYTES = TF * KS * 2;       // 16 KiB per sub-tile
constexpr int NIB_BYTES = TF * KST / 2;    // 8 KiB per stage
static_assert(kBarriers + 1 + kBoxes <= 32, "one warp sets them up");
constexpr int kFewRows = 64;               // rows of a tile up to which its weights' bytes count
constexpr int THREADS = 768;
constexpr int EPI_WARP0 = 4, CONV_WARP0 = 8, CONV_WARPS = 8;  // CONV_WARPS per group
constexpr int row_tile(bool pair) { return pair ? 2 * XR : XR; }  // rows per tile at most

constexpr size_t OFF_W = (size_t)STAGES * SUBS * X_BYTES;
constexpr size_t OFF_N = OFF_W + (size_t)STAGES * SUBS * W_BYTES;
constexpr size_t OFF_BAR = OFF_N + (size_t)NRING * NIB_BYTES;
constexpr size_t OFF_PRE = OFF_BAR + 512;
constexpr int PART_LD = TF + 4;            // floats per row of a partial tile
static_assert((size_t)XR * PART_LD * 4 <= OFF_N, "partial tiles reuse the stages");
size_t tc_smem(int E) { return 1024 + OFF_PRE + (size_t)(E + 1) * 4; }

struct TcMaps {
  CUtensorMap nib, rows[kBoxes];
};

struct TcArgs {
  A16W4Call c;
  int F, R;        // features and reduction length
  int ftiles, stages, subs;  // subs: sub-tiles of the reduction
  int splits;        // kShared: CTAs of a cluster
  int whole;         // the reduction is whole sub-tiles: rows as [64-wide block][row][64]
  int stall;         // test hook: no rows are asked for for a CTA's second stage
  // Limit of the waits that run out when rows are missing: for a stage's rows,
  // for its MMAs, for a tile.  (Read by every wait it cost 0.5 us at
  // 64x14336x4096, 22.05 against 21.5.)
  uint32_t spin;
};

struct Tile {
  int e, f0, p0, np;  // expert, first feature, first sorted row, rows
};

__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  // MN-major, 128-byte swizzle: 64 features x 8 reduction rows per 1 KiB
  // atom; 1 KiB to the next 8 reduction rows, 8 KiB to the next 64 features
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(8192 >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

template <bool PAIR>
__device__ __forceinline__ void mma_f16(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
// Arrive on `bar` (in both CTAs of a pair) once the MMAs issued so far end.
template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (PAIR) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)0x3)
        : "memory");
  } else {
    mma_commit(bar);
  }
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
// Tensor loads of rows; in a pair they complete on the barrier at cluster
// address `bar`, which may be the other CTA's (no multicast).
template <bool PAIR>
__device__ __forceinline__ void load_rows_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void load_rows_3d(uint32_t dst, const void* tmap, int y, int block,
                                             uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(tmap), "r"(0), "r"(y), "r"(block), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(tmap), "r"(0), "r"(y), "r"(block), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Every lane waits; the warp takes its decision together.  The limit counts
// the pipeline's own time: a role waits for the work before this call first.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status, uint32_t limit) {
  // a phase that is complete is seen at once; a parked wait costs about 180
  // cycles even then
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_park(bar, parity, status, limit));
}

// A group scale (and zero) as the expansion uses it.
template <int FMT>
struct Scale;
// bf16 scales: code * s in bf16 is one rounding of the exact product
template <>
struct Scale<QG_W4_BF16> {
  uint32_t s;
};
// f32 scales: s = hi + lo in bf16; fma(code, hi, code * lo) rounds the sum
// once (the roundings of lo and of code * lo are below 2^-15 of the weight)
template <>
struct Scale<QG_W4_F32> {
  uint32_t hi, lo;
};
// f32 scales and zeros: fma(s, code, z) in f32, rounded to bf16.  The code
// itself is the factor: with 128 + u as it is unpacked, the rounding of z - 136 s
// would stay where s * code and z cancel.
template <>
struct Scale<QG_W4_ASYM> {
  float s, z;
};

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

__device__ __forceinline__ uint64_t pair_bits(float2 a) {
  return (uint64_t)__float_as_uint(a.y) << 32 | __float_as_uint(a.x);
}
__device__ __forceinline__ float2 pair_of(uint64_t a) {
  return make_float2(__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)(a >> 32)));
}
__device__ __forceinline__ float2 f32x2_add(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_bits(a)), "l"(pair_bits(b)));
  return pair_of(d);
}
__device__ __forceinline__ float2 f32x2_fma(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(pair_bits(a)), "l"(pair_bits(b)), "l"(pair_bits(c)));
  return pair_of(d);
}

// Raw stored scales (and zeros, zoff bytes further) of two neighbouring
// groups: loaded ahead, turned into a Scale at use.
struct RawScales {
  uint2 s, z;  // bf16: both in s.x
};
template <int FMT>
__device__ __forceinline__ RawScales load_scales(const uint8_t* p, int64_t zoff, bool in) {
  RawScales v;
  v.s = v.z = make_uint2(0, 0);
  if (in) {
    if constexpr (FMT == QG_W4_BF16) {
      v.s.x = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      v.s = __ldg(reinterpret_cast<const uint2*>(p));
      if constexpr (FMT == QG_W4_ASYM) v.z = __ldg(reinterpret_cast<const uint2*>(p + zoff));
    }
  }
  return v;
}
template <int FMT>
__device__ __forceinline__ Scale<FMT> make_scale(const RawScales& v, int i) {
  Scale<FMT> s;
  const uint32_t raw = i ? v.s.y : v.s.x;
  if constexpr (FMT == QG_W4_BF16) {
    s.s = prmt(v.s.x, 0u, i ? 0x3232u : 0x1010u);
  } else if constexpr (FMT == QG_W4_F32) {
    const float f = __uint_as_float(raw);
    const uint32_t hi = __bfloat16_as_ushort(__float2bfloat16_rn(f));
    const float rest = f - __uint_as_float(hi << 16);
    const uint32_t lo = __bfloat16_as_ushort(__float2bfloat16_rn(rest));
    s.hi = hi | (hi << 16);
    s.lo = lo | (lo << 16);
  } else {
    s.s = __uint_as_float(raw);
    s.z = __uint_as_float(i ? v.z.y : v.z.x);
  }
  return s;
}

// The 8 weights of one nibble word, in their order, as bf16 pairs.
template <int FMT>
__device__ __forceinline__ void expand8(uint32_t w, const Scale<FMT>& s, uint32_t (&o)[4]) {
  const uint32_t L = w & 0x0F0F0F0Fu, H = (w >> 4) & 0x0F0F0F0Fu;
  if constexpr (FMT == QG_W4_ASYM) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = i < 2 ? L : H;
      // 0x43uu0000 is 128 + u; two weights at a time, code = 128 + u - 136
      float2 v = make_float2(__uint_as_float(prmt(b, 0x43000000u, (i & 1) ? 0x7244u : 0x7044u)),
                             __uint_as_float(prmt(b, 0x43000000u, (i & 1) ? 0x7344u : 0x7144u)));
      v = f32x2_fma(f32x2_add(v, make_float2(-136.0f, -136.0f)), make_float2(s.s, s.s), make_float2(s.z, s.z));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(v.y), "f"(v.x));
    }
  } else {
    o[0] = bf16x2_minus136(prmt(L, 0x43434343u, 0x5140u));
    o[1] = bf16x2_minus136(prmt(L, 0x43434343u, 0x5342u));
    o[2] = bf16x2_minus136(prmt(H, 0x43434343u, 0x5140u));
    o[3] = bf16x2_minus136(prmt(H, 0x43434343u, 0x5342u));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (FMT == QG_W4_BF16) o[i] = bf16x2_mul(o[i], s.s);
      else o[i] = bf16x2_fma(o[i], s.hi, bf16x2_mul(o[i], s.lo));
    }
  }
}

// How CTAs share a tile: on its own, a pair (256 features, cta_group::2), or a
// cluster of `splits` CTAs that share its reduction.
enum TcMode { kSingle = 0, kPair = 1, kShared = 2 };

template <int FMT, bool GRAD, int MODE>
__global__ void __launch_bounds__(THREADS, 1)
    a16w4_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs a,
                    int* status) {
  constexpr bool PAIR = MODE == kPair, SHARED = MODE == kShared;
  constexpr int TT = row_tile(PAIR);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sX = smem_u32(smem), sW = smem_u32(smem + OFF_W);
  const uint32_t sN = smem_u32(smem + OFF_N);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);  // rows and weights of a stage
  uint64_t* empty = full + STAGES;  // [NBAR] by stage: its MMAs have ended
  uint64_t* n_full = empty + NBAR;  // [NBAR] by stage
  uint64_t* n_empty = n_full + NBAR;
  uint64_t* t_full = n_empty + NRING;
  uint64_t* t_empty = t_full + 2;
  uint64_t* drain = t_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* pre = reinterpret_cast<int*>(smem + OFF_PRE);  // [E + 1] row tiles before expert e
  float* part = reinterpret_cast<float*>(smem);        // shared reduction: [row][PART_LD]

  const A16W4Call& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0;  // rank 0 issues the pair's MMAs
  const int splits = SHARED ? a.splits : 1, split = SHARED ? (int)cluster_rank() : 0;
  const int first = PAIR ? blockIdx.x >> 1 : SHARED ? blockIdx.x / splits : blockIdx.x;
  const int step = PAIR ? gridDim.x >> 1 : gridDim.x;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0) {  // a barrier per lane
    constexpr uint32_t kConv = PAIR ? 2 * CONV_WARPS : CONV_WARPS;
    if (lane < kBarriers) {
      uint64_t* bar = full + lane;
      mbar_init(bar, bar < empty ? 1 + kConv : bar < n_empty ? 1 : bar < t_full ? CONV_WARPS
                     : bar < t_empty ? 1 : bar < drain ? (PAIR ? 8 : 4) : 1);
    } else if (lane - kBarriers < 1 + kBoxes) {
      prefetch_tmap(lane == kBarriers ? &maps.nib : &maps.rows[lane - kBarriers - 1]);
    }
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(512)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(tmem_slot)),
                   "r"(512)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  // the offsets come from the work before this call
  if (c.offsets) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 3) {  // the experts' tiles
    int carry = 0;
    for (int b = 0; b < c.E; b += 32) {
      const int e = b + lane;
      const int own =
          e < c.E ? (expert_range(c.offsets, e, c.S, blockIdx.x == 0 ? status : nullptr).y + TT - 1) / TT
                  : 0;
      int x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (e < c.E) pre[e] = carry + x - own;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) pre[c.E] = carry;
  }
  __syncwarp();
  tc_fence_before();
  // in a pair, both CTAs' barriers exist before any signal between them
  if constexpr (PAIR) cluster_sync_all(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int64_t total = (int64_t)pre[c.E] * a.ftiles;
  // this CTA's part of the reduction, in stages
  const int all_stages = a.stages;
  const int s_first = SHARED ? all_stages * split / splits : 0;
  const int stages = SHARED ? all_stages * (split + 1) / splits - s_first : all_stages;

  constexpr int kRowStep = PAIR ? 32 : 16;  // MMA N in steps of 16 per CTA
  // tile t: features fastest, so concurrent CTAs share the rows' tiles
  auto tile_at = [&](int64_t t) {
    Tile r;
    const int u = (int)(t / a.ftiles);
    r.f0 = (int)(t - (int64_t)u * a.ftiles) * (PAIR ? 2 * TF : TF) + (int)rank * TF;
    int lo = 0, hi = c.E - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= u) lo = mid; else hi = mid - 1;
    }
    r.e = lo;
    const int2 range = expert_range(c.offsets, lo, c.S, nullptr);
    // an expert's rows in equal tiles
    const int nt = pre[lo + 1] - pre[lo];
    const int per = ((range.y + nt - 1) / nt + kRowStep - 1) & ~(kRowStep - 1);
    const int from = min((u - pre[lo]) * per, range.y);
    r.p0 = range.x + from;
    r.np = min(per, range.y - from);
    return r;
  };

  if (warp == 0) {
    // ---------------- rows: this CTA's half, or all ----------------
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // `free`: the barrier of the stage that had the slot before
    uint32_t it = 0, slot = 0, free = NBAR - STAGES, par = 1;
    const uint32_t skip = a.stall ? 1u : 0xFFFFFFFFu;
    bool ok = true;
    for (int64_t t = first; t < total && ok; t += step) {
      const Tile tl = tile_at(t);
      const int n = (tl.np + kRowStep - 1) & ~(kRowStep - 1);
      const int mine = PAIR ? n / 2 : n;
      const int y = tl.p0 + (int)rank * mine;
      const int box = box_of(mine);
      const uint32_t sub_b = (uint32_t)box_rows(box) * (KS * 2);  // bytes of a sub-tile
      const void* map = &maps.rows[box];
      for (int s = 0; s < stages; ++s, ++it) {
        ok = warp_wait(&empty[free], par, status, a.spin);  // the first round passes
        if (!ok) break;
        const int subs = a.whole ? SUBS : min(SUBS, a.subs - SUBS * (s_first + s));
        if (it != skip && elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[slot], sub_b * (uint32_t)(PAIR ? 2 * subs : subs));
          const uint32_t dst = sX + slot * (SUBS * X_BYTES);
          const uint32_t bar = PAIR ? mapa(smem_u32(&full[slot]), 0) : smem_u32(&full[slot]);
          if (a.whole) {
            load_rows_3d<PAIR>(dst, map, y, SUBS * (s_first + s), bar);
          } else {
            for (int u = 0; u < subs; ++u)
              load_rows_2d<PAIR>(dst + u * sub_b, map, (s_first + s) * KST + u * KS, y, bar);
          }
        }
        __syncwarp();
        if (++slot == STAGES) slot = 0;
        if (++free == NBAR) {
          free = 0;
          par ^= 1;
        }
      }
    }
    // Every copy has landed (in a pair the first CTA waits for both, and the
    // CTAs end together) and every commit has arrived before the CTA may exit.
    for (uint32_t k = it > STAGES ? it - STAGES : 0; k < it; ++k) {
      if (rank == 0 && k != skip) warp_wait(&full[k % STAGES], (k / STAGES) & 1, status, kSpinLimit);
      if (ok) warp_wait(&empty[k % NBAR], (k / NBAR) & 1, status, a.spin);
    }
  } else if (warp == 2) {
    // ---------------- nibbles (inputs of the call alone) ----------------
    uint32_t it = 0, slot = 0, bar = 0, par = 1;
    bool ok = true;
    for (int64_t t = first; t < total && ok; t += step) {
      const Tile tl = tile_at(t);
      // With few rows the weights' bytes count: the next tile's into L2 (its
      // 128 rows lie together; the gradient's tiles are columns).
      if (!GRAD && t + step < total) {
        const Tile nx = tile_at(t + step);
        if (nx.np <= kFewRows && elect_one()) {
          const int rows = min(TF, c.N - nx.f0), G = c.K >> 5;
          const uint8_t* w = c.packed + (int64_t)nx.e * c.expert_bytes;
          constexpr int sb = FMT == QG_W4_BF16 ? 2 : 4;
          if (rows > 0) {
            prefetch_l2(w + (int64_t)nx.f0 * (c.K >> 1), (int64_t)rows * (c.K >> 1));
            w += (int64_t)c.N * (c.K >> 1) + (int64_t)nx.f0 * G * sb;
            prefetch_l2(w, (int64_t)rows * G * sb);
            if (FMT == QG_W4_ASYM) prefetch_l2(w + (int64_t)c.N * G * 4, (int64_t)rows * G * sb);
          }
        }
        __syncwarp();
      }
      for (int s = 0; s < stages; ++s, ++it) {
        if (it == NRING) asm volatile("griddepcontrol.wait;" ::: "memory");  // from here on a wait can block
        ok = warp_wait(&n_empty[slot], par, status, kSpinLimit);  // the first round passes
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&n_full[bar], NIB_BYTES);
          if (GRAD) tma_load_3d(sN + slot * NIB_BYTES, &maps.nib, tl.f0 / 8, (s_first + s) * KST, tl.e, &n_full[bar]);
          else tma_load_3d(sN + slot * NIB_BYTES, &maps.nib, (s_first + s) * (KST / 8), tl.f0, tl.e, &n_full[bar]);
        }
        __syncwarp();
        if (++bar == NBAR) bar = 0;
        if (++slot == NRING) {
          slot = 0;
          par ^= 1;
        }
      }
    }
    for (uint32_t k = it > NRING ? it - NRING : 0; k < it; ++k)
      warp_wait(&n_full[k % NBAR], (k / NBAR) & 1, status, kSpinLimit);
  } else if (warp == 1) {
    // ---------------- MMA issue ----------------
    // One thread, and every stage passes through it: with divisions by the
    // ring's size, two barriers a stage and polled waits it took 1050 cycles a
    // stage, twice the MMAs' own time.
    if (rank == 0) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      uint32_t use = 0, slot = 0, bar = 0, par = 0;
      bool ok = true;
      for (int64_t t = first; t < total && ok; t += step, ++use) {
        const Tile tl = tile_at(t);
        const int n = (tl.np + kRowStep - 1) & ~(kRowStep - 1);
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (GRAD ? 1u << 15 : 0u) |
                               ((uint32_t)(n >> 3) << 17) |
                               ((uint32_t)((PAIR ? 2 * TF : TF) >> 4) << 24);
        const uint32_t buf = use & 1;
        const uint32_t next_x = (uint32_t)box_rows(box_of(PAIR ? n / 2 : n)) * (KS * 2) >> 4;
        ok = warp_wait(&t_empty[buf], ((use >> 1) & 1) ^ 1, status, kSpinLimit);
        const uint32_t d = tmem_base + buf * TT;
        for (int s = 0; s < stages && ok; ++s) {
          ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], par, status, a.spin));
          if (!ok) break;
          tc_fence_after();
          const int subs = min(SUBS, a.subs - SUBS * (s_first + s));
          if (elect_one()) {
            // descriptor addresses count 16 bytes: 16 k further is 32 bytes
            // of a K-major row, or 16 rows of 128 bytes of the MN-major tile
            uint64_t dx = sdesc_sw128(sX + slot * (SUBS * X_BYTES));
            const uint32_t w0 = sW + slot * (SUBS * W_BYTES);
            uint64_t dw = GRAD ? sdesc_mn_sw128(w0) : sdesc_sw128(w0);
#pragma unroll
            for (int u = 0; u < SUBS; ++u) {
              if (u >= subs) break;
#pragma unroll
              for (int k = 0; k < KS / 16; ++k)
                mma_f16<PAIR>(d, dw + (GRAD ? 128 : 2) * k, dx + 2 * k, idesc, s > 0 || u > 0 || k > 0);
              dx += next_x;
              dw += W_BYTES >> 4;
            }
            commit<PAIR>(&empty[bar]);
            if (s == stages - 1) commit<PAIR>(&t_full[buf]);
          }
          __syncwarp();
          if (++bar == NBAR) bar = 0;
          if (++slot == STAGES) {
            slot = 0;
            par ^= 1;
          }
        }
      }
      if (ok) {  // the epilogues' last signals have arrived, the other CTA's among them
        for (uint32_t k = use > 2 ? use - 2 : 0; k < use; ++k)
          warp_wait(&t_empty[k & 1], (k >> 1) & 1, status, kSpinLimit);
      } else {  // MMAs in flight end before their operands or TMEM go away
        if (elect_one()) commit<PAIR>(drain);
        __syncwarp();
        warp_wait(drain, 0, status, kSpinLimit);
      }
    }
  } else if (warp >= CONV_WARP0) {
    // ---------------- expansion ----------------
    const uint32_t group = (uint32_t)(warp - CONV_WARP0) / CONV_WARPS;
    const int tid = (threadIdx.x - CONV_WARP0 * 32) % (CONV_WARPS * 32);
    // row n of the stage's 128, and half of its 128 k: 64 weights, two groups,
    // 32 nibble bytes.  Forward, the halves are the stage's sub-tiles (K-major
    // rows); for the gradient the rows' halves are, and this half of k is a
    // block of 64 features (MN-major).
    const int row = tid >> 1, half = tid & 1;
    const uint32_t nib_at = (uint32_t)(tid * 32);
    const int G = c.K >> 5;
    constexpr int SB = FMT == QG_W4_BF16 ? 2 : 4;
    const int64_t zoff = (int64_t)c.N * G * 4;
    const uint32_t w_at = sW + (GRAD ? (row >> 6) * W_BYTES + half * 8192 + (row & 63) * 128
                                     : half * W_BYTES + row * 128);
    const uint32_t turn = (uint32_t)((row & 7) ^ (half << 2));  // swizzle, and the groups' order
    const uint32_t step_b = GRAD ? (uint32_t)(KST * G * SB) : 4u * SB;  // scales: stage to stage
    uint32_t it = 0, slot = group;                 // of the stage and of its nibbles
    uint32_t nib = group, free = group + NBAR - STAGES;  // barriers
    uint32_t npar = 0, par = 1;                    // and the parities to wait for
    bool ok = true, early = true;
    for (int64_t t = first; t < total && ok; t += step) {
      const Tile tl = tile_at(t);
      const uint8_t* scl = c.packed + (int64_t)tl.e * c.expert_bytes + (int64_t)c.N * (c.K >> 1);
      const int g = (GRAD ? tl.f0 >> 5 : 0) + 2 * half;  // forward: 4 further with every stage
      const int n0 = GRAD ? row : tl.f0 + row;           // gradient: 128 further
      scl += ((int64_t)n0 * G + g) * SB;
      // stages of this tile in which the thread's weights exist
      const int live = GRAD ? (g < G ? (c.N - n0 + KST - 1) / KST : 0) : (n0 < c.N ? (G - g + 3) / 4 : 0);
      auto fetch = [&](int s) {
        return load_scales<FMT>(scl + (int64_t)(s_first + s) * step_b, zoff, s_first + s < live);
      };
      int s = (it & 1) == group ? 0 : 1;  // this group's stages: every other one
      RawScales now = fetch(s), next = fetch(s + 2);
      for (; s < stages; s += 2) {
        // The first copies leave ahead of the work before this call and find
        // free slots; every later one follows it, and so must the count of a
        // bounded wait for it or for its slot.
        if (early && it + s >= NRING) {
          asm volatile("griddepcontrol.wait;" ::: "memory");
          early = false;
        }
        ok = warp_wait(&n_full[nib], npar, status, kSpinLimit);
        if (!ok) break;
        uint32_t wd[8];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(wd[0]), "=r"(wd[1]), "=r"(wd[2]), "=r"(wd[3])
                     : "r"(sN + slot * NIB_BYTES + nib_at)
                     : "memory");
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(wd[4]), "=r"(wd[5]), "=r"(wd[6]), "=r"(wd[7])
                     : "r"(sN + slot * NIB_BYTES + nib_at + 16)
                     : "memory");
        // Once they are in registers the next copy into the slot may leave.
        // The signal depends on the values themselves: behind the loads in
        // program order alone it went ahead of them.
        const uint32_t seen = (wd[0] | wd[1] | wd[2]) | (wd[3] | wd[4] | wd[5]) | (wd[6] | wd[7]);
        const int signaller = __any_sync(0xffffffffu, seen != 0) ? 0 : 1;
        if (lane == signaller) mbar_arrive(&n_empty[slot]);
        // the halves' 16-byte parts lie in the same banks: the second half
        // stores its second group first
        const Scale<FMT> sc[2] = {make_scale<FMT>(now, half), make_scale<FMT>(now, half ^ 1)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a0 = wd[i], a1 = wd[4 + i];
          wd[i] = half ? a1 : a0;
          wd[4 + i] = half ? a0 : a1;
        }
        now = next;
        next = fetch(s + 4);
        ok = warp_wait(&empty[free], par, status, a.spin);  // the first round passes
        if (!ok) break;
        const uint32_t dst = w_at + slot * (SUBS * W_BYTES);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t o[4];
          expand8<FMT>(wd[i], sc[i >> 2], o);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + ((i ^ turn) << 4)),
                       "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                       : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR) mbar_arrive_cluster(mapa(smem_u32(&full[slot]), 0));
          else mbar_arrive(&full[slot]);
        }
        if ((slot += 2) >= STAGES) slot -= STAGES;
        if ((nib += 2) >= NBAR) {
          nib -= NBAR;
          npar ^= 1;
        }
        if ((free += 2) >= NBAR) {
          free -= NBAR;
          par ^= 1;
        }
      }
      it += (uint32_t)stages;
    }
  } else if (warp >= EPI_WARP0) {
    // ---------------- epilogue ----------------
    const int q = warp & 3;  // TMEM lane quarter
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool even = (lane & 1) == 0;
    const bool vec = ((reinterpret_cast<uintptr_t>(c.out) & 3) == 0) && ((c.ld_out & 1) == 0);
    const bool vec4 = ((reinterpret_cast<uintptr_t>(c.out) & 7) == 0) && ((c.ld_out & 3) == 0);
    uint32_t use = 0;
    for (int64_t t = first; t < total; t += step, ++use) {
      const Tile tl = tile_at(t);
      const uint32_t buf = use & 1;
      // a whole reduction, of 2^24 at most
      if (!warp_wait(&t_full[buf], (use >> 1) & 1, status, a.spin << 4)) break;
      tc_fence_after();
      const int f = tl.f0 + 32 * q + lane;
      float b = 0.0f;
      if (c.bias && f < a.F) b = __ldg(c.bias + (int64_t)tl.e * a.F + f);
      for (int j0 = 0; j0 < tl.np; j0 += 32) {
        uint32_t v[32];
        __syncwarp();  // converged again after the stores, as the load asks
        tmem_ld32(tmem_base + ((uint32_t)(32 * q) << 16) + buf * TT + j0, v);
        tmem_wait_ld();
        if constexpr (SHARED) {
          // partial sums over the stages' memory: every MMA has ended
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j0 + j < tl.np) part[(j0 + j) * PART_LD + 32 * q + lane] = __uint_as_float(v[j]);
        } else if (vec4 && tl.f0 + 32 * q + 32 <= a.F) {
          // A quad's lanes hold 4 rows j .. j + 3 of 4 features; two swaps
          // give each lane one row of all four.
          const int jl = j0 + (lane & 1) + (lane & 2);  // this lane's row of the four
          uint16_t* dst = c.out + (int64_t)(tl.p0 + jl) * c.ld_out + (f & ~3);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            if (j0 + j >= tl.np) break;
            uint32_t lo, hi;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                : "=r"(lo)
                : "f"(__uint_as_float(v[j + 1]) + b), "f"(__uint_as_float(v[j]) + b));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                : "=r"(hi)
                : "f"(__uint_as_float(v[j + 3]) + b), "f"(__uint_as_float(v[j + 2]) + b));
            // features f, f + 1 of rows j (even lanes) or j + 1 (odd), and 2 further
            const uint32_t lo2 = __shfl_xor_sync(0xffffffffu, lo, 1);
            const uint32_t hi2 = __shfl_xor_sync(0xffffffffu, hi, 1);
            const uint32_t x = even ? prmt(lo, lo2, 0x5410) : prmt(lo2, lo, 0x7632);
            const uint32_t y = even ? prmt(hi, hi2, 0x5410) : prmt(hi2, hi, 0x7632);
            const bool first_pair = (lane & 2) == 0;
            const uint32_t other = __shfl_xor_sync(0xffffffffu, first_pair ? y : x, 2);
            if (jl + j < tl.np)
              *reinterpret_cast<uint2*>(dst) = first_pair ? make_uint2(x, other) : make_uint2(other, y);
            dst += 4 * c.ld_out;
          }
        } else if (vec) {
          // lanes f, f + 1 swap halves: the even one stores both features of
          // row j, the odd one those of row j + 1
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            if (j0 + j >= tl.np) break;
            uint32_t mine;
            const float v0 = __uint_as_float(v[j]) + b, v1 = __uint_as_float(v[j + 1]) + b;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(mine) : "f"(v1), "f"(v0));
            const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
            const uint32_t o = even ? prmt(mine, other, 0x5410) : prmt(other, mine, 0x7632);
            const int jj = j0 + j + (even ? 0 : 1), ff = even ? f : f - 1;
            uint16_t* dst = c.out + (int64_t)(tl.p0 + jj) * c.ld_out + ff;
            if (jj < tl.np) {
              if (ff + 1 < a.F) *reinterpret_cast<uint32_t*>(dst) = o;
              else if (ff < a.F) *dst = (uint16_t)o;
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j0 + j < tl.np && f < a.F)
              c.out[(int64_t)(tl.p0 + j0 + j) * c.ld_out + f] =
                  __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[j]) + b));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(mapa(smem_u32(&t_empty[buf]), 0));
        else mbar_arrive(&t_empty[buf]);
      }
    }
  }

  if constexpr (SHARED) {
    // Sum the cluster's partial tiles, each CTA its part of the rows, in the
    // order of the ranks.
    __syncwarp();
    cluster_sync_all();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Tile tl = tile_at(first);
    const uint32_t base = smem_u32(part);
    const int j0 = tl.np * split / splits, j1 = tl.np * (split + 1) / splits;
    const int f = (int)(threadIdx.x & 63) * 2;  // two features
    const bool two = tl.f0 + f + 1 < a.F;
    float b0 = 0.0f, b1 = 0.0f;
    if (c.bias && tl.f0 + f < a.F) b0 = __ldg(c.bias + tl.f0 + f);
    if (c.bias && two) b1 = __ldg(c.bias + tl.f0 + f + 1);
    const bool vec = ((reinterpret_cast<uintptr_t>(c.out) & 3) == 0) && ((c.ld_out & 1) == 0);
    for (int j = j0 + (int)(threadIdx.x >> 6); j < j1; j += THREADS / 64) {
      float s0 = b0, s1 = b1;
      for (int k = 0; k < splits; ++k) {
        float x, y;
        asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];"
                     : "=f"(x), "=f"(y)
                     : "r"(mapa(base + (uint32_t)(j * PART_LD + f) * 4, (uint32_t)k))
                     : "memory");
        s0 += x;
        s1 += y;
      }
      uint16_t* dst = c.out + (int64_t)(tl.p0 + j) * c.ld_out + tl.f0 + f;
      const uint16_t h0 = __bfloat16_as_ushort(__float2bfloat16_rn(s0));
      const uint16_t h1 = __bfloat16_as_ushort(__float2bfloat16_rn(s1));
      if (vec && two) {
        *reinterpret_cast<uint32_t*>(dst) = h0 | ((uint32_t)h1 << 16);
      } else {
        if (tl.f0 + f < a.F) dst[0] = h0;
        if (two) dst[1] = h1;
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA ends while another may read its sums
  }
  // no CTA of a pair leaves while the other may still signal its barriers or
  // read its shared memory
  __syncwarp();
  tc_fence_before();
  if constexpr (PAIR) cluster_sync_all(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512)
                   : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512)
                   : "memory");
  }
}

// Does row p lie in a range of offsets that expert_range takes?  One warp asks.
__device__ __forceinline__ bool in_some_range(const A16W4Call& c, int p, int lane) {
  // the ranges of sorted offsets cover [offsets[0], offsets[E]); with unsorted
  // ones that may hold rows of nobody, which nobody reads
  if (p >= c.offsets[0] && p < min(c.offsets[c.E], c.S)) return true;
  // behind the last row in ordinary calls; with unsorted offsets a range may
  // lie there all the same
  bool in = false;
  for (int e = lane; e < c.E; e += 32) {
    const int2 r = expert_range(c.offsets, e, c.S, nullptr);
    in |= p >= r.x && p - r.x < r.y;
  }
  return __any_sync(0xffffffffu, in);
}

// Rows into sorted order: xs[p] = x[src[p] / topk] for the rows that belong
// to an expert, a warp per row.  The work before the call may write them while
// this kernel is resident, so they are read by ordinary loads, not as constants.
__global__ void __launch_bounds__(256) a16w4_gather_kernel(const __grid_constant__ A16W4Call c,
                                                           uint16_t* __restrict__ xs, int* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (at >= c.S || !in_some_range(c, (int)at, lane)) return;
  const int p = (int)at;
  const int s = c.src[p];
  const int row = s < 0 ? c.in_rows : s / c.topk;
  const int nv = c.K / 8;  // K % 64 == 0 and 16-byte aligned rows
  uint4* dst = reinterpret_cast<uint4*>(xs + (int64_t)p * c.K);
  if (row >= c.in_rows) {  // outside x: zeros
    record_error(status, QG_ERR_INVALID_ARG);
    for (int i = lane; i < nv; i += 32) dst[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  const uint4* from = reinterpret_cast<const uint4*>(c.in + row * c.ld_in);
  int i = lane;
  for (; i + 96 < nv; i += 128) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = from[i + 32 * k];
#pragma unroll
    for (int k = 0; k < 4; ++k) dst[i + 32 * k] = v[k];
  }
  for (; i < nv; i += 32) dst[i] = from[i];
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 g_tc_encode = nullptr;

template <int FMT, bool GRAD>
const void* kernel_of(int mode) {
  if (mode == kPair) return (const void*)a16w4_tc_kernel<FMT, GRAD, kPair>;
  if (mode == kShared) return (const void*)a16w4_tc_kernel<FMT, GRAD, kShared>;
  return (const void*)a16w4_tc_kernel<FMT, GRAD, kSingle>;
}
const void* kernel_of(int fmt, bool grad, int mode) {
  if (fmt == QG_W4_F32)
    return grad ? kernel_of<QG_W4_F32, true>(mode) : kernel_of<QG_W4_F32, false>(mode);
  if (fmt == QG_W4_BF16)
    return grad ? kernel_of<QG_W4_BF16, true>(mode) : kernel_of<QG_W4_BF16, false>(mode);
  return grad ? kernel_of<QG_W4_ASYM, true>(mode) : kernel_of<QG_W4_ASYM, false>(mode);
}

constexpr int kMaxDevices = 64;
// What can be resident at once: CTA pairs, and clusters of 2 << i that share a
// tile's reduction (a cluster lies within one GPC, so fewer than SMs / size).
int g_tc_pairs[kMaxDevices], g_tc_clusters[kMaxDevices][3];

}  // namespace

int a16w4_tc_setup() {
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult qr;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                       &qr) != cudaSuccess ||
      qr != cudaDriverEntryPointSuccess || !fn)
    return QG_ERR_CUDA;
  g_tc_encode = (PFN_cuTensorMapEncodeTiled_v12000)fn;
  for (int fmt = 0; fmt < 3; ++fmt)
    for (int v = 0; v < 6; ++v)
      if (cudaFuncSetAttribute(kernel_of(fmt, v >= 3, v % 3), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)tc_smem(kA16W4MaxExperts)) != cudaSuccess)
        return QG_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return QG_ERR_CUDA;
  auto resident = [](int size, const void* kernel, int& count) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = tc_smem(kA16W4MaxExperts);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(&count, kernel, &cfg) == cudaSuccess;
  };
  bool ok = resident(2, kernel_of(QG_W4_F32, false, kPair), g_tc_pairs[dev]);
  for (int i = 0; i < 3; ++i)
    ok = ok && resident(2 << i, kernel_of(QG_W4_F32, false, kShared), g_tc_clusters[dev][i]);
  return ok && g_tc_pairs[dev] >= 1 ? QG_OK : QG_ERR_CUDA;
}

size_t a16w4_tc_workspace(int S, int K, bool gather) {
  return gather ? (size_t)S * K * 2 : 0;
}

int launch_a16w4_tc(const A16W4Call& call, bool grad, void* ws, cudaStream_t st) {
  A16W4Call c = call;
  int* status = status_word();
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (c.src) {
    cfg.gridDim = dim3((unsigned)cdiv(c.S, 8));
    cfg.blockDim = dim3(256);
    if (cudaLaunchKernelEx(&cfg, a16w4_gather_kernel, c, (uint16_t*)ws, status) != cudaSuccess)
      return QG_ERR_CUDA;
    c.in = (const uint16_t*)ws;
    c.ld_in = c.K;
    c.in_rows = c.S;
    c.src = nullptr;
  }
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return QG_ERR_CUDA;
  TcArgs a{};
  a.c = c;
  a.stall = take_stall(kStallA16W4TC);
  a.spin = a.stall ? kStallSpinLimit : kSpinLimit;
  a.F = grad ? c.K : c.N;
  a.R = grad ? c.N : c.K;
  a.subs = (int)cdiv(a.R, KS);
  a.stages = (int)cdiv(a.subs, SUBS);
  // pairs, unless their tiles leave half of the SMs without work
  const int64_t likely = c.offsets ? max64(cdiv(c.S, row_tile(true)), min64(c.E, c.S)) : cdiv(c.S, row_tile(true));
  const bool pair = likely * cdiv(a.F, 2 * TF) * 4 > num_sms();
  // at most this many tiles of rows: every expert's last one may be partial
  const int64_t row_tiles = cdiv(c.S, row_tile(pair)) + (c.offsets ? min64(c.E, c.S) : 0);
  a.ftiles = (int)cdiv(a.F, pair ? 2 * TF : TF);
  TcMaps m;
  {
    cuuint64_t dims[3] = {(cuuint64_t)c.K / 8, (cuuint64_t)c.N, (cuuint64_t)c.E};
    cuuint64_t strides[2] = {(cuuint64_t)c.K / 2,
                             (cuuint64_t)(c.E > 1 ? c.expert_bytes : (int64_t)c.N * (c.K / 2))};
    cuuint32_t box[3] = {KST / 8, TF, 1};  // 128 k of 128 rows in both directions
    cuuint32_t es[3] = {1, 1, 1};
    if (g_tc_encode(&m.nib, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, (void*)c.packed, dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return QG_ERR_CUDA;
  }
  // Rows as [64-wide block of the reduction][row][64], or plainly [row][R]
  // where the last block is a partial one, which only this form ends in zeros.
  a.whole = a.R % KS == 0;
  for (int b = 0; b < kBoxes; ++b) {
    const cuuint32_t rows = (cuuint32_t)box_rows(b);
    cuuint64_t dims3[3] = {KS, (cuuint64_t)c.in_rows, (cuuint64_t)a.subs};
    cuuint64_t strides3[2] = {(cuuint64_t)c.ld_in * 2, KS * 2};
    cuuint32_t box3[3] = {KS, rows, SUBS};
    cuuint64_t dims2[2] = {(cuuint64_t)a.R, (cuuint64_t)c.in_rows};
    cuuint32_t box2[2] = {KS, rows};
    cuuint32_t es[3] = {1, 1, 1};
    if (g_tc_encode(&m.rows[b], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.whole ? 3 : 2, (void*)c.in,
                    a.whole ? dims3 : dims2, strides3, a.whole ? box3 : box2, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return QG_ERR_CUDA;
  }
  const int64_t most = row_tiles * a.ftiles;
  // A dense call whose tiles leave SMs without work: clusters share each
  // tile's reduction, two stages or more per CTA, all of them resident at once
  // (17x2048x2048, 16 tiles: clusters of 8, which take two turns, 13.0 us, of 4
  // 6.5; 33x512x8192, 4 tiles: 9.1 and 12.9).
  a.splits = 1;
  if (!pair && !c.offsets)
    for (int i = 0; i < 3 && most <= g_tc_clusters[dev][i] && a.stages >= 4 * a.splits; ++i)
      a.splits *= 2;
  cfg.gridDim = dim3(pair ? 2 * (unsigned)min64(g_tc_pairs[dev], most) : (unsigned)(a.splits > 1 ? most * a.splits : min64(num_sms(), most)));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = tc_smem(c.E);
  if (pair || a.splits > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = pair ? 2 : (unsigned)a.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  void* args[] = {&m, &a, &status};
  return cudaLaunchKernelExC(&cfg, kernel_of(c.format, grad, pair ? kPair : a.splits > 1 ? kShared : kSingle), args) == cudaSuccess ? QG_OK
                                                                                        : QG_ERR_CUDA;
}

}  // namespace qg
