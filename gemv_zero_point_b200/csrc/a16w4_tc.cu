// Weight-only int4 products on the 5th-generation tensor cores, for many rows
// per expert: the forward product and the gradient with respect to its input.
//
//   forward   y[p,n]  = sum_k x[p,k] * w[n,k] + bias[n]     features n, reduction k
//   gradient  dx[p,k] = sum_n dy[p,n] * w[n,k]              features k, reduction n
//
// One tile is 128 features (MMA M, TMEM lanes) x up to 256 rows (MMA N, TMEM
// columns): the rows are the side of free size, in steps of 16, so the
// ragged row counts of experts waste little.  The weights are expanded to
// bf16 on the way into shared memory: w is formed as the real value and
// rounded to bf16 once (half a step, 2^-8 of w), the price of one MMA per
// weight; the sums stay in f32 (TMEM) and the output is rounded once.  With
// 256 rows a stage's four MMAs take 256 cycles, and the expansion of its 8192
// weights about 150 issue cycles, so the expansion hides behind the MMAs.
//
// Both directions read the same packed matrix.  Forward, a stage is 128 rows
// n x 64 k of it and the bf16 tile is K-major; for the gradient it is 64 rows
// n x 128 k and the tile's features (k) run along the rows, so the same
// row-wise expansion writes an MN-major operand: no transpose anywhere.
//
// Roles (512 threads, one CTA per SM, persistent over tiles):
//   warp 0      rows: tensor copies of 64-wide slices (128-byte swizzle), or
//               row gathers of four rows each when the rows are indirect
//   warp 1      TMEM; MMA issue, one commit per stage and one per tile
//   warp 2      nibbles: tensor copies, a ring of their own
//   warps 4-7   epilogue: TMEM -> bf16 -> global, overlapping the next tile
//   warps 8-15  expansion of the nibbles into the swizzled bf16 stage
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "a16w4.cuh"

namespace qg {

namespace {

constexpr int TF = 128;                    // features per tile
constexpr int TT = 256;                    // rows per tile at most
constexpr int KS = 64;                     // reduction per stage: one 128-byte swizzle row
constexpr int XBOX = 64;                   // rows per tensor copy
constexpr int STAGES = 4;
constexpr int NRING = 6;
constexpr int X_BYTES = TT * KS * 2;       // 32 KiB
constexpr int W_BYTES = TF * KS * 2;       // 16 KiB
constexpr int NIB_BYTES = TF * KS / 2;     // 4 KiB
constexpr int THREADS = 512;
constexpr int EPI_WARP0 = 4, CONV_WARP0 = 8, CONV_WARPS = 8;

constexpr size_t OFF_X = 0;
constexpr size_t OFF_W = OFF_X + (size_t)STAGES * X_BYTES;
constexpr size_t OFF_N = OFF_W + (size_t)STAGES * W_BYTES;
constexpr size_t OFF_BAR = OFF_N + (size_t)NRING * NIB_BYTES;
constexpr size_t OFF_PRE = OFF_BAR + 512;
size_t tc_smem(int E) { return 1024 + OFF_PRE + (size_t)(E + 1) * 4; }

struct TcMaps {
  CUtensorMap nib, rows;
};

struct TcArgs {
  A16W4Call c;
  int F, R;        // features and reduction length
  int ftiles, stages;
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

__device__ __forceinline__ void mma_f16(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
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

// Four rows r.x .. r.w of a one-row box; rows outside the tensor read as zeros.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const void* tmap, int x, int4 r,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(smem_u32(bar))
      : "memory");
}

// Every lane waits; the warp takes its decision together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* status) {
  return __all_sync(0xffffffffu, mbar_park(bar, parity, status));
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
// once (lo's own rounding is 2^-17 of s)
template <>
struct Scale<QG_W4_F32> {
  uint32_t hi, lo;
};
// f32 scales and zeros: s * code + z in f32, rounded to bf16
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

// Raw stored values of group `at`: loaded ahead, turned into a Scale at use.
template <int FMT>
__device__ __forceinline__ uint2 load_scale(const uint8_t* scl, const uint8_t* zer, int64_t at,
                                            bool in) {
  uint2 v = make_uint2(0, 0);
  if (in) {
    if constexpr (FMT == QG_W4_BF16) {
      v.x = __ldg(reinterpret_cast<const unsigned short*>(scl) + at);
    } else {
      v.x = __ldg(reinterpret_cast<const uint32_t*>(scl) + at);
      if constexpr (FMT == QG_W4_ASYM) v.y = __ldg(reinterpret_cast<const uint32_t*>(zer) + at);
    }
  }
  return v;
}
template <int FMT>
__device__ __forceinline__ Scale<FMT> make_scale(uint2 v) {
  Scale<FMT> s;
  if constexpr (FMT == QG_W4_BF16) {
    s.s = v.x | (v.x << 16);
  } else if constexpr (FMT == QG_W4_F32) {
    const float f = __uint_as_float(v.x);
    const uint32_t hi = __bfloat16_as_ushort(__float2bfloat16_rn(f));
    const float rest = f - __uint_as_float(hi << 16);
    const uint32_t lo = __bfloat16_as_ushort(__float2bfloat16_rn(rest));
    s.hi = hi | (hi << 16);
    s.lo = lo | (lo << 16);
  } else {
    s.s = __uint_as_float(v.x);
    s.z = __uint_as_float(v.y);
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
      // 0x4B0000uu is 2^23 + u
      const float c0 = __uint_as_float(prmt(b, 0x4B000000u, 0x7440u + (i & 1) * 2)) - 8388616.0f;
      const float c1 = __uint_as_float(prmt(b, 0x4B000000u, 0x7441u + (i & 1) * 2)) - 8388616.0f;
      const float w0 = fmaf(s.s, c0, s.z), w1 = fmaf(s.s, c1, s.z);
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(w1), "f"(w0));
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

template <int FMT, bool GRAD, bool GATHER>
__global__ void __launch_bounds__(THREADS, 1)
    a16w4_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ TcArgs a,
                    int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t sX = smem_u32(smem + OFF_X), sW = smem_u32(smem + OFF_W);
  const uint32_t sN = smem_u32(smem + OFF_N);
  uint64_t* x_full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* w_full = x_full + STAGES;
  uint64_t* empty = w_full + STAGES;
  uint64_t* n_full = empty + STAGES;
  uint64_t* n_empty = n_full + NRING;
  uint64_t* t_full = n_empty + NRING;
  uint64_t* t_empty = t_full + 2;
  uint64_t* drain = t_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* pre = reinterpret_cast<int*>(smem + OFF_PRE);  // [E + 1] row tiles before expert e

  const A16W4Call& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&x_full[s], 1);
      mbar_init(&w_full[s], CONV_WARPS);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < NRING; ++s) {
      mbar_init(&n_full[s], 1);
      mbar_init(&n_empty[s], CONV_WARPS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&t_full[b], 1);
      mbar_init(&t_empty[b], 4);
    }
    mbar_init(drain, 1);
    fence_mbar_init();
    prefetch_tmap(&maps.nib);
    prefetch_tmap(&maps.rows);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int64_t total = (int64_t)pre[c.E] * a.ftiles;
  const int stages = a.stages;

  // tile t: features fastest, so concurrent CTAs share the rows' tiles
  auto tile_at = [&](int64_t t) {
    Tile r;
    const int u = (int)(t / a.ftiles);
    r.f0 = (int)(t - (int64_t)u * a.ftiles) * TF;
    int lo = 0, hi = c.E - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= u) lo = mid; else hi = mid - 1;
    }
    r.e = lo;
    const int2 range = expert_range(c.offsets, lo, c.S, nullptr);
    // an expert's rows in equal tiles
    const int nt = pre[lo + 1] - pre[lo];
    const int per = ((range.y + nt - 1) / nt + 15) & ~15;
    const int from = min((u - pre[lo]) * per, range.y);
    r.p0 = range.x + from;
    r.np = min(per, range.y - from);
    return r;
  };

  if (warp == 0) {
    // ---------------- rows ----------------
    asm volatile("griddepcontrol.wait;" ::: "memory");
    uint32_t it = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const Tile tl = tile_at(t);
      int4 r0, r1;  // GATHER: input rows of tile rows 8*lane .. 8*lane + 7
      uint32_t bytes = (uint32_t)((tl.np + XBOX - 1) / XBOX) * (XBOX * KS * 2);
      if constexpr (GATHER) {
        int rr[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int j = 8 * lane + i;
          rr[i] = c.in_rows;  // outside: zeros
          if (j < tl.np) {
            const int s = c.src[tl.p0 + j];
            const int q = s < 0 ? c.in_rows : s / c.topk;
            if (q >= c.in_rows) record_error(status, QG_ERR_INVALID_ARG);
            else rr[i] = q;
          }
        }
        r0 = make_int4(rr[0], rr[1], rr[2], rr[3]);
        r1 = make_int4(rr[4], rr[5], rr[6], rr[7]);
        bytes = (uint32_t)((tl.np + 3) / 4) * (4 * KS * 2);
      }
      for (int s = 0; s < stages; ++s, ++it) {
        const int slot = it % STAGES;
        if (it >= STAGES) ok = warp_wait(&empty[slot], ((it / STAGES) - 1) & 1, status);
        if (!ok) break;
        const uint32_t dst = sX + slot * X_BYTES;
        if (lane == 0) mbar_arrive_expect_tx(&x_full[slot], bytes);
        __syncwarp();
        if constexpr (GATHER) {
          if (8 * lane < tl.np) tma_gather4(dst + lane * 1024, &maps.rows, s * KS, r0, &x_full[slot]);
          if (8 * lane + 4 < tl.np)
            tma_gather4(dst + lane * 1024 + 512, &maps.rows, s * KS, r1, &x_full[slot]);
        } else {
          if (lane * XBOX < tl.np)
            tma_load_2d(smem + OFF_X + slot * X_BYTES + lane * (XBOX * KS * 2), &maps.rows, s * KS,
                        tl.p0 + lane * XBOX, &x_full[slot]);
        }
      }
    }
    // every copy has landed before the CTA may exit
    for (uint32_t k = it > STAGES ? it - STAGES : 0; k < it; ++k)
      warp_wait(&x_full[k % STAGES], (k / STAGES) & 1, status);
  } else if (warp == 2) {
    // ---------------- nibbles (inputs of the call alone) ----------------
    uint32_t it = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const Tile tl = tile_at(t);
      for (int s = 0; s < stages; ++s, ++it) {
        const int slot = it % NRING;
        if (it >= NRING) ok = warp_wait(&n_empty[slot], ((it / NRING) - 1) & 1, status);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&n_full[slot], NIB_BYTES);
          if (GRAD) tma_load_3d(sN + slot * NIB_BYTES, &maps.nib, tl.f0 / 8, s * KS, tl.e, &n_full[slot]);
          else tma_load_3d(sN + slot * NIB_BYTES, &maps.nib, s * (KS / 8), tl.f0, tl.e, &n_full[slot]);
        }
        __syncwarp();
      }
    }
    for (uint32_t k = it > NRING ? it - NRING : 0; k < it; ++k)
      warp_wait(&n_full[k % NRING], (k / NRING) & 1, status);
  } else if (warp == 1) {
    // ---------------- MMA issue ----------------
    uint32_t it = 0, use = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < total && ok; t += gridDim.x, ++use) {
      const Tile tl = tile_at(t);
      const int n = (tl.np + 15) & ~15;
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (GRAD ? 1u << 15 : 0u) |
                             ((uint32_t)(n >> 3) << 17) | ((uint32_t)(TF >> 4) << 24);
      const uint32_t buf = use & 1;
      ok = warp_wait(&t_empty[buf], ((use >> 1) & 1) ^ 1, status);
      if (!ok) break;
      const uint32_t d = tmem_base + buf * TT;
      for (int s = 0; s < stages; ++s, ++it) {
        const int slot = it % STAGES;
        const uint32_t par = (it / STAGES) & 1;
        ok = warp_wait(&x_full[slot], par, status) && warp_wait(&w_full[slot], par, status);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t dx = sdesc_sw128(sX + slot * X_BYTES);
          const uint64_t dw = GRAD ? sdesc_mn_sw128(sW + slot * W_BYTES) : sdesc_sw128(sW + slot * W_BYTES);
          // descriptor addresses count 16 bytes: 16 k further is 32 bytes of
          // a K-major row, or 16 rows of 128 bytes of the MN-major tile
#pragma unroll
          for (int k = 0; k < KS / 16; ++k)
            mma_f16(d, dw + (GRAD ? 128 : 2) * k, dx + 2 * k, idesc, s > 0 || k > 0);
          mma_commit(&empty[slot]);
          if (s == stages - 1) mma_commit(&t_full[buf]);
        }
        __syncwarp();
      }
    }
    if (!ok) {  // MMAs in flight end before their operands or TMEM go away
      if (lane == 0) mma_commit(drain);
      __syncwarp();
      warp_wait(drain, 0, status);
    }
  } else if (warp >= CONV_WARP0) {
    // ---------------- expansion ----------------
    const int tid = threadIdx.x - CONV_WARP0 * 32;
    // forward: row n (of 128), half of its 64 k; gradient: row n (of 64),
    // quarter of its 128 k.  32 weights, one group, 16 nibble bytes each.
    const int row = GRAD ? tid >> 2 : tid >> 1, part = GRAD ? tid & 3 : tid & 1;
    const uint32_t nib_at = (uint32_t)(tid * 16);
    const int G = c.K >> 5;
    uint32_t it = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const Tile tl = tile_at(t);
      const uint8_t* scl = c.packed + (int64_t)tl.e * c.expert_bytes + (int64_t)c.N * (c.K >> 1);
      const uint8_t* zer = scl + (int64_t)c.N * G * 4;
      auto fetch = [&](int s) {
        const int n = GRAD ? s * KS + row : tl.f0 + row;
        const int g = GRAD ? (tl.f0 >> 5) + part : 2 * s + part;
        return load_scale<FMT>(scl, zer, (int64_t)n * G + g, s < stages && n < c.N && g < G);
      };
      uint2 s0 = fetch(0), s1 = fetch(1);
      for (int s = 0; s < stages; ++s, ++it) {
        const int slot = it % STAGES, ns = it % NRING;
        const uint2 s2 = fetch(s + 2);  // two stages ahead
        ok = warp_wait(&n_full[ns], (it / NRING) & 1, status);
        if (!ok) break;
        uint4 q;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                     : "r"(sN + ns * NIB_BYTES + nib_at)
                     : "memory");
        const Scale<FMT> sc = make_scale<FMT>(s0);
        if (it >= STAGES) ok = warp_wait(&empty[slot], ((it / STAGES) - 1) & 1, status);
        if (!ok) break;
        // gradient: parts 2 and 3 go 8 KiB behind 0 and 1, to the same banks,
        // so they store their words in the order 2, 3, 0, 1
        const bool turn = GRAD && part >= 2;
        const uint32_t wd[4] = {turn ? q.z : q.x, turn ? q.w : q.y, turn ? q.x : q.z, turn ? q.y : q.w};
        const uint32_t dst = GRAD ? sW + slot * W_BYTES + (part >> 1) * 8192 + row * 128
                                  : sW + slot * W_BYTES + row * 128;
        const int c0 = GRAD ? (part & 1) * 4 + (turn ? 2 : 0) : part * 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
          expand8<FMT>(wd[i], sc, o);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + (((c0 ^ i) ^ (row & 7)) << 4)),
                       "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                       : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&n_empty[ns]);
          mbar_arrive(&w_full[slot]);
        }
        s0 = s1;
        s1 = s2;
      }
    }
  } else if (warp >= EPI_WARP0) {
    // ---------------- epilogue ----------------
    const int q = warp & 3;  // TMEM lane quarter
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const bool even = (lane & 1) == 0;
    const bool vec = ((reinterpret_cast<uintptr_t>(c.out) & 3) == 0) && ((c.ld_out & 1) == 0);
    uint32_t use = 0;
    for (int64_t t = blockIdx.x; t < total; t += gridDim.x, ++use) {
      const Tile tl = tile_at(t);
      const uint32_t buf = use & 1;
      if (!warp_wait(&t_full[buf], (use >> 1) & 1, status)) break;
      tc_fence_after();
      const int f = tl.f0 + 32 * q + lane;
      float b = 0.0f;
      if (c.bias && f < a.F) b = __ldg(c.bias + (int64_t)tl.e * a.F + f);
      for (int j0 = 0; j0 < tl.np; j0 += 32) {
        uint32_t v[32];
        tmem_ld32(tmem_base + ((uint32_t)(32 * q) << 16) + buf * TT + j0, v);
        tmem_wait_ld();
        if (vec) {
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
      if (lane == 0) mbar_arrive(&t_empty[buf]);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512)
                 : "memory");
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 g_tc_encode = nullptr;

template <int FMT>
const void* kernel_of(bool grad, bool gather) {
  if (grad) return (const void*)a16w4_tc_kernel<FMT, true, false>;
  return gather ? (const void*)a16w4_tc_kernel<FMT, false, true>
                : (const void*)a16w4_tc_kernel<FMT, false, false>;
}
const void* kernel_of(int fmt, bool grad, bool gather) {
  if (fmt == QG_W4_F32) return kernel_of<QG_W4_F32>(grad, gather);
  if (fmt == QG_W4_BF16) return kernel_of<QG_W4_BF16>(grad, gather);
  return kernel_of<QG_W4_ASYM>(grad, gather);
}

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
    for (int v = 0; v < 3; ++v)
      if (cudaFuncSetAttribute(kernel_of(fmt, v == 2, v == 1),
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)tc_smem(kA16W4MaxExperts)) != cudaSuccess)
        return QG_ERR_CUDA;
  return QG_OK;
}

int launch_a16w4_tc(const A16W4Call& c, bool grad, cudaStream_t st) {
  TcArgs a{};
  a.c = c;
  a.F = grad ? c.K : c.N;
  a.R = grad ? c.N : c.K;
  a.ftiles = (int)cdiv(a.F, TF);
  a.stages = (int)cdiv(a.R, KS);
  const bool gather = c.src != nullptr;
  TcMaps m;
  {
    cuuint64_t dims[3] = {(cuuint64_t)c.K / 8, (cuuint64_t)c.N, (cuuint64_t)c.E};
    cuuint64_t strides[2] = {(cuuint64_t)c.K / 2,
                             (cuuint64_t)(c.E > 1 ? c.expert_bytes : (int64_t)c.N * (c.K / 2))};
    cuuint32_t box[3] = {grad ? (cuuint32_t)TF / 8 : (cuuint32_t)KS / 8,
                         grad ? (cuuint32_t)KS : (cuuint32_t)TF, 1};
    cuuint32_t es[3] = {1, 1, 1};
    if (g_tc_encode(&m.nib, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, (void*)c.packed, dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return QG_ERR_CUDA;
  }
  {
    cuuint64_t dims[2] = {(cuuint64_t)a.R, (cuuint64_t)c.in_rows};
    cuuint64_t strides[1] = {(cuuint64_t)c.ld_in * 2};
    cuuint32_t box[2] = {KS, gather ? 1u : (cuuint32_t)XBOX};
    cuuint32_t es[2] = {1, 1};
    if (g_tc_encode(&m.rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (void*)c.in, dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return QG_ERR_CUDA;
  }
  // at most this many tiles: every expert's last tile may be a partial one
  const int64_t most = (cdiv(c.S, TT) + min64(c.E, c.S)) * a.ftiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)min64(num_sms(), c.offsets ? most : cdiv(c.S, TT) * a.ftiles));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = tc_smem(c.E);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int* status = status_word();
  void* args[] = {&m, &a, &status};
  return cudaLaunchKernelExC(&cfg, kernel_of(c.format, grad, gather), args) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

}  // namespace qg
