// Weight-only int4 products: bf16 rows, not quantized, times int4 weights
// with group scales, dense or per expert.  This file: the entry points and
// the kernel for few rows per expert.
//
//   y[p,n] = sum_g sw[n,g] * I[p,n,g] (+ zw[n,g] * X[p,g]) + bias[n]
//   I[p,n,g] = sum_{k in g} x[p,k] * c[n,k],  X[p,g] = sum_{k in g} x[p,k]
// with c the int4 codes, exact in bf16.
//
// With few rows the weights' bytes bound the call, so the kernel is a stream
// over the packed weights that must not run out of issue slots: at the
// measured copy bandwidth an SM receives about 37 weights per cycle, which
// leaves 3.4 issue slots per weight, and logic, shifts and packed bf16
// arithmetic take two each.  Warp MMAs (m16n8k16, 8 cycles a sub-partition)
// take 16 weight rows x 8 token rows at once, so the cost per weight is the
// unpacking, whatever the number of tokens up to 8.
//   - A code c goes in as 128 + u, u = c + 8: two nibbles become a pair of
//     bf16 values with one logic and one byte permute instruction.
//   - 128 + u = c + 136, so a group's sums start at -136 X, X = sum x, formed
//     by MMAs with the constant once per chunk for all weight rows.
//   - The group scale is applied to the f32 sums of the group: nothing is
//     rounded below f32 before y (the 136 costs the sums 5 of their 24 bits).
// 1x14336x4096 takes 12.4 us (2.96 TB/s), 12x4096x14336 19.0 us, 8 tokens x 8
// of 64 experts of 2048x2048 35 to 40 us, by how many of them the tokens reach.
// 42 to 49 % of the issue slots are used; the chains of a chunk (ldmatrix,
// unpacking, MMAs, scales) leave the rest.  At the 128 registers that two CTAs
// an SM allow, the forms for 8 tokens spill 24 to 184 bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "a16w4.cuh"

namespace qg {

int device_setup_status();
int a16w4_tc_setup();

namespace {

constexpr int W = 8;              // warps per CTA
constexpr int KC = 128;           // K per chunk: 4 groups, 64 nibble bytes a row
constexpr int RT = 4;             // 16-row tiles of a run and row warp
constexpr int WROWS = 16 * RT;
constexpr int D = 2;              // chunks in a warp's ring
constexpr int kDenseRows = 16;    // tokens that a dense call's only pass can hold
constexpr int kMinRows = 8;       // fewest weight rows that a CTA takes
constexpr int kXParts = 16;       // CTAs that prefetch a dense call's rows

// Bytes of one chunk in a warp's ring: nibbles (their 16-byte parts turned by
// row / 2, so eight rows of a part lie in eight bank groups), then scales
// (and zeros) of WROWS rows x 4 groups.
template <int FMT>
struct Slot {
  static constexpr int SCL = FMT == QG_W4_BF16 ? 8 : 16;  // scale bytes per row
  static constexpr int OFF_SCL = WROWS * 64;
  static constexpr int OFF_ZERO = OFF_SCL + WROWS * SCL;
  static constexpr int BYTES = OFF_ZERO + (FMT == QG_W4_ASYM ? WROWS * 16 : 0);
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 lds128f(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
// Four 8 x 16-byte blocks: register m of lane (g, t) is word t of row g of block m.
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

// d = a * b + {c0, c1, c0, c1} (m16n8k16)
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8 codes of nibble word w in their order as bf16 pairs 128 + u, u = code + 8.
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&p)[4]) {
  const uint32_t L = w & 0x0F0F0F0Fu, H = (w >> 4) & 0x0F0F0F0Fu;
  p[0] = prmt(L, 0x43434343u, 0x5140u);
  p[1] = prmt(L, 0x43434343u, 0x5342u);
  p[2] = prmt(H, 0x43434343u, 0x5140u);
  p[3] = prmt(H, 0x43434343u, 0x5342u);
}

// q = v / d and the rest r, by 32-bit division where v allows it.
__device__ __forceinline__ void divide(int64_t v, int d, int64_t& q, int64_t& r) {
  if (v <= 0x7FFFFFFF) {
    q = (uint32_t)v / (uint32_t)d;
    r = (uint32_t)v - (uint32_t)q * (uint32_t)d;
  } else {
    q = v / d;
    r = v - q * d;
  }
}

// What the CTAs of one launch share out: the weight rows of every pass over
// an expert's tokens, one after another ("virtual rows").  A pass takes up
// to 8*NT tokens.
struct RowsArgs {
  A16W4Call c;
  int chunks;        // ceil(K / KC)
  int wk;            // warps that split K; W / wk warps split the rows
  int per_sm;        // CTAs an SM
  int share, more;   // dense: 8-row blocks of a CTA, and how many CTAs take one more
};

// A run: consecutive weight rows of one pass, at most WROWS per row warp.
struct Run {
  int e, pass, r0, rows;  // expert, its pass, first weight row, rows
  int64_t left;           // virtual rows of this CTA from r0 on
  int base, nrows;        // this warp's rows of the run
};

// The runs of one CTA.  DENSE: one matrix and at most one pass, so they
// follow from the CTA's number alone and the first loads leave at once.
// Otherwise the passes (of `per` tokens) of every expert are counted first,
// from the offsets that the work before this call has written.
template <bool DENSE>
struct Shares {
  const RowsArgs& a;
  const int* pre;    // [E + 1] passes before expert e
  const int* start;  // [E] first sorted row
  const int* count;  // [E] rows
  const int per, wr, rw;
  int64_t v0, v1;    // this CTA's virtual rows

  __device__ __forceinline__ Shares(const RowsArgs& a_, int per_, int* pre_, int* start_, int* count_,
                                    int* status)
      : a(a_), pre(pre_), start(start_), count(count_), per(per_), wr(W / a_.wk),
        rw((int)(threadIdx.x >> 5) / a_.wk) {
    const A16W4Call& c = a.c;
    if (DENSE) {
      const int b = (int)blockIdx.x;
      v0 = 8 * ((int64_t)a.share * b + min(a.more, b));
      v1 = min64(v0 + 8 * (a.share + (b < a.more ? 1 : 0)), c.N);
      return;
    }
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int e = threadIdx.x; e < c.E; e += W * 32) {
      const int2 r = expert_range(c.offsets, e, c.S, status);
      start_[e] = r.x;
      count_[e] = r.y;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      int carry = 0;
      for (int b = 0; b < c.E; b += 32) {
        const int e = b + lane;
        const int own = e < c.E ? (count_[e] + per - 1) / per : 0;
        int x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (e < c.E) pre_[e] = carry + x - own;
        carry += __shfl_sync(0xffffffffu, x, 31);
      }
      if (lane == 0) pre_[c.E] = carry;
    }
    __syncthreads();
    const int64_t total = (int64_t)pre[c.E] * c.N;
    if (total < (int64_t)gridDim.x * kMinRows) {
      v0 = min64(total, (int64_t)blockIdx.x * kMinRows);
      v1 = min64(total, v0 + kMinRows);
    } else {
      // shares differ by one row at most
      int64_t q, r;
      divide(total, (int)gridDim.x, q, r);
      v0 = q * blockIdx.x + min64(r, blockIdx.x);
      v1 = v0 + q + (blockIdx.x < r ? 1 : 0);
    }
  }

  // the rest of a run, its start known
  __device__ __forceinline__ void shape(Run& r) const {
    r.rows = (int)min64(min64(a.c.N - r.r0, r.left), (int64_t)WROWS * wr);
    const int share = wr == 1 ? r.rows : ((r.rows + wr - 1) / wr + 15) & ~15;
    r.base = rw * share;
    r.nrows = max(0, min(r.rows - r.base, share));
  }
  __device__ __forceinline__ Run first() const {
    Run r;
    r.e = r.pass = r.r0 = r.rows = r.base = r.nrows = 0;
    r.left = v1 - v0;
    if (r.left <= 0) return r;
    if (DENSE) {
      r.r0 = (int)v0;
    } else {
      int64_t u64, r064;
      divide(v0, a.c.N, u64, r064);
      const int u = (int)u64;
      int lo = 0, hi = a.c.E - 1;  // last expert with pre[e] <= u: the one that has pass u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= u) lo = mid; else hi = mid - 1;
      }
      r.e = lo;
      r.pass = u - pre[lo];
      r.r0 = (int)r064;
    }
    shape(r);
    return r;
  }
  __device__ __forceinline__ void next(Run& r) const {
    r.left -= r.rows;
    if (r.left <= 0) {
      r.nrows = 0;
      return;
    }
    r.r0 += r.rows;
    if (!DENSE && r.r0 == a.c.N) {
      r.r0 = 0;
      if (++r.pass == pre[r.e + 1] - pre[r.e]) {
        r.pass = 0;
        do ++r.e; while (pre[r.e + 1] == pre[r.e]);  // left > 0: one follows
      }
    }
    shape(r);
  }
  __device__ __forceinline__ int tokens_from(const Run& r) const {
    return DENSE ? 0 : start[r.e] + r.pass * per;
  }
  __device__ __forceinline__ int tokens(const Run& r) const {
    return DENSE ? a.c.S : min(count[r.e] - r.pass * per, per);
  }
  // row of x that sorted row p reads, -1 (read as zeros) for one outside x
  __device__ __forceinline__ int input_row(int p, int* status) const {
    if (DENSE) return p;
    int row = p;
    if (a.c.src) {
      const int s = a.c.src[p];
      row = s < 0 ? -1 : s / a.c.topk;
    }
    if (row < 0 || row >= a.c.in_rows) {
      record_error(status, QG_ERR_INVALID_ARG);
      return -1;
    }
    return row;
  }
  // One whole run into L2, and on to the next (few and large requests: each
  // costs the copy engine some 100 ns).
  __device__ __forceinline__ void prefetch(Run& r, int sb, int64_t zoff, bool zeros) const {
    if (r.left <= 0) return;
    const int rowb = a.c.K >> 1, G = a.c.K >> 5;
    const uint8_t* wq = a.c.packed + (int64_t)r.e * a.c.expert_bytes;
    prefetch_l2(wq + (int64_t)r.r0 * rowb, (int64_t)r.rows * rowb);
    const uint8_t* s = wq + (int64_t)a.c.N * rowb + (int64_t)r.r0 * G * sb;
    prefetch_l2(s, (int64_t)r.rows * G * sb);
    if (zeros) prefetch_l2(s + zoff, (int64_t)r.rows * G * sb);
    next(r);
  }
};

// Dense: x into L2 while the work before this call ends (a prefetch cannot
// return stale data), one part of one row from each of the first CTAs.
__device__ __forceinline__ void prefetch_x(const A16W4Call& c) {
  if ((int)threadIdx.x < c.S && blockIdx.x < kXParts) {
    const int64_t k0 = (int64_t)c.K * blockIdx.x / kXParts, k1 = (int64_t)c.K * (blockIdx.x + 1) / kXParts;
    prefetch_l2(c.in + (int64_t)threadIdx.x * c.ld_in + k0, (k1 - k0) * 2);
  }
}

// y of one run from the partial sums [K warp][token of `per`][row].
__device__ __forceinline__ void sum_and_store(const A16W4Call& c, const Run& at, int p0, int np,
                                              int per, int wk, const float* part, int prows) {
  for (int o = threadIdx.x; o < at.rows * np; o += W * 32) {
    const int tok = np == 1 ? 0 : o / at.rows, r = o - tok * at.rows;
    const float* d = part + (size_t)tok * prows + r;
    float s = 0.0f;
    for (int k = 0; k < wk; ++k) s += d[(size_t)k * per * prows];
    const int n = at.r0 + r;
    if (c.bias) s += __ldg(c.bias + (int64_t)at.e * c.N + n);
    c.out[(int64_t)(p0 + tok) * c.ld_out + n] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
  }
}

// ---------------------------------------------------------------------------
// The kernel.  Nibbles and scales come through a ring in shared
// memory that each warp keeps for itself (cp.async, no barriers), and
// ldmatrix hands every lane the nibble words of its fragment rows.  The warps
// of a CTA split K; their sums meet in shared memory at the end of a run.
// ---------------------------------------------------------------------------
// NT: MMA column blocks (8 tokens) per pass.
template <int FMT, int NT, bool DENSE>
__global__ void __launch_bounds__(W * 32, NT == 1 ? 2 : 1)
    a16w4_rows_kernel(const __grid_constant__ RowsArgs a, int* status) {
  using Sl = Slot<FMT>;
  extern __shared__ __align__(128) uint8_t sm[];
  const A16W4Call& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;  // MMA fragment coordinates
  const int K = c.K, N = c.N, G = K >> 5, rowb = K >> 1;
  const int wk = a.wk, wr = W / wk;
  const int kw = warp % wk, rw = warp / wk;
  constexpr int SB = FMT == QG_W4_BF16 ? 2 : 4;
  // shared memory: rings, partial sums, expert tables
  const int prows = WROWS * wr + 4;  // pitch of a token's partial sums; +4 spreads the banks
  const uint32_t ring = smem_u32(sm) + (uint32_t)(warp * D * Sl::BYTES);
  float* part = reinterpret_cast<float*>(sm + W * D * Sl::BYTES);
  int* pre = reinterpret_cast<int*>(part + (size_t)wk * 8 * NT * prows);  // [E + 1] passes before e
  int* start = pre + c.E + 1;
  int* count = start + c.E;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Shares<DENSE> sh(a, 8 * NT, pre, start, count, status);
  Run at = sh.first();
  const int ch0 = (int)((int64_t)kw * a.chunks / wk), ch1 = (int)((int64_t)(kw + 1) * a.chunks / wk);

  // ---- copies into the ring, D - 1 chunks ahead of their use ----
  Run put = at;
  int put_chunk = ch0;
  const uint8_t* nib = nullptr;   // this lane's 16 bytes of rows lane / 4, + 8, ...
  const uint8_t* scl = nullptr;   // scales of row `lane` (and lane + 32)
  const int64_t nib8 = (int64_t)8 * rowb, scl32 = (int64_t)32 * G * SB;
  const int64_t zoff = (int64_t)N * G * 4;  // zeros follow the scales
  const bool wide = (G & 3) == 0;  // a chunk's scales start on their whole size
  const uint32_t nib_to = ring + (uint32_t)((lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4));
  const uint32_t scl_to = ring + Sl::OFF_SCL + (uint32_t)(lane * Sl::SCL);
  auto open_put = [&]() {
    while (put.left > 0 && put.nrows == 0) sh.next(put);
    if (put.left <= 0) return;
    const uint8_t* wq = c.packed + (int64_t)put.e * c.expert_bytes;
    const int64_t row = put.r0 + put.base;
    nib = wq + (row + (lane >> 2)) * rowb + ch0 * (KC / 2) + (lane & 3) * 16;
    scl = wq + (int64_t)N * rowb + ((row + lane) * G + 4 * ch0) * SB;
    put_chunk = ch0;
  };
  // scales of one row and chunk: 4 groups, or 2 at the end of K
  auto copy_scales = [&](uint32_t d, const uint8_t* s, bool half) {
    if constexpr (FMT == QG_W4_BF16) {
      if (wide) {
        cp8(d, s);
      } else {
        cp4(d, s);
        if (!half) cp4(d + 4, s + 4);
      }
    } else {
      if (wide) {
        cp16(d, s);
      } else {
        cp8(d, s);
        if (!half) cp8(d + 8, s + 8);
      }
    }
  };
  auto issue = [&](int slot) {
    if (put.left > 0) {
      const uint32_t so = (uint32_t)(slot * Sl::BYTES);
      const bool half = 4 * put_chunk + 4 > G;  // the last 64 of K
      if (!half || (lane & 3) < 2) {
        const uint8_t* p = nib;
#pragma unroll
        for (int i = 0; i < WROWS / 8; ++i) {
          if ((lane >> 2) + 8 * i < put.nrows) cp16(nib_to + so + i * 512, p);
          p += nib8;
        }
      }
#pragma unroll
      for (int i = 0; i < WROWS / 32; ++i) {
        if (lane + 32 * i < put.nrows) {
          copy_scales(scl_to + so + i * 32 * Sl::SCL, scl + i * scl32, half);
          if constexpr (FMT == QG_W4_ASYM)
            copy_scales(scl_to + so + WROWS * 16 + i * 32 * Sl::SCL, scl + i * scl32 + zoff, half);
        }
      }
      nib += KC / 2;
      scl += 4 * SB;
      if (++put_chunk == ch1) {
        sh.next(put);
        open_put();
      }
    }
    cp_commit();
  };
  // Thread 0 asks for whole runs in L2, two runs ahead of their use, so that
  // the ring's loads only have L2's latency to cover.
  Run ahead = at;
  bool cold = true;

  if (DENSE) prefetch_x(c);
  open_put();
#pragma unroll
  for (int d = 0; d < D - 1; ++d) issue(d);
  if (DENSE) asm volatile("griddepcontrol.wait;" ::: "memory");

  // ldmatrix source of this lane: blocks (rows 0-7, q), (8-15, q), (0-7, q+1), (8-15, q+1)
  const uint32_t a_at = ring + (uint32_t)(((lane & 15) * 64) + (((lane >> 4) ^ ((lane >> 1) & 3)) << 4));
  const uint32_t s_at = ring + Sl::OFF_SCL + (uint32_t)(g * Sl::SCL);

  // this lane's token rows (MMA column g); columns past the last token repeat
  // it, and are not stored
  const uint16_t* xr[NT];
  auto point_x = [&](const Run& r) {
    const int p0 = sh.tokens_from(r), np = sh.tokens(r);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = sh.input_row(p0 + min(8 * n + g, np - 1), status);
      xr[n] = row < 0 ? nullptr : c.in + row * c.ld_in + t * 8;
    }
  };
  // B fragments: lane t gives x[8t .. 8t+7] of its group, as A's words do.
  uint4 xb[NT][4], xn[NT][4];  // this chunk, and the next one read ahead
  auto load_x = [&](uint4 (&x)[NT][4], int ch) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[n][q] = make_uint4(0, 0, 0, 0);
        if (xr[n] && 4 * ch + q < G)
          x[n][q] = *reinterpret_cast<const uint4*>(xr[n] + (int64_t)ch * KC + q * 32);
      }
  };
  if (at.nrows > 0) {
    point_x(at);
    load_x(xn, ch0);
  }

  // every warp walks every run: its chunks, then the sum over the K warps
  int slot = 0;
  while (at.left > 0) {
    const int p0 = sh.tokens_from(at), np = sh.tokens(at);
    float acc[RT][NT][4];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][n][k] = 0.0f;
    if (at.nrows > 0) {
      for (int ch = ch0; ch < ch1; ++ch) {
        const bool half = 4 * ch + 4 > G;  // x is 0 for groups 2 and 3
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) xb[n][q] = xn[n][q];
        if (ch + 1 < ch1) load_x(xn, ch + 1);
        // -136 X of this lane's tokens 2t, 2t + 1
        float z[NT][4][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            constexpr uint32_t m = 0xC308C308u;  // -136, -136
            float d[4];
            mma16816(d, m, m, m, m, xb[n][q].x, xb[n][q].y, 0.0f, 0.0f);
            mma16816(d, m, m, m, m, xb[n][q].z, xb[n][q].w);
            z[n][q][0] = d[0];
            z[n][q][1] = d[1];
          }
        // The run and the next one into L2, once x has landed (its sums are
        // finite or not: the test only makes thread 0 wait for them); asked
        // for earlier, they keep x waiting behind them.
        if (cold && threadIdx.x == 0 && z[0][0][0] != 12345.678f) {
          sh.prefetch(ahead, SB, zoff, FMT == QG_W4_ASYM);
          sh.prefetch(ahead, SB, zoff, FMT == QG_W4_ASYM);
        }
        cold = false;
        issue(slot ^ 1);
        cp_wait<D - 1>();
        __syncwarp();
        const uint32_t so = (uint32_t)(slot * Sl::BYTES);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          if (16 * i >= at.nrows) break;
          uint32_t w01[4], w23[4];  // words of groups 0, 1 and 2, 3: rows g, g + 8 each
          ldsm4(a_at + so + i * 1024, w01);
          ldsm4((a_at ^ 32u) + so + i * 1024, w23);
          float sa[4], sb[4], za[4], zb[4];
          const uint32_t sc = s_at + so + i * 16 * Sl::SCL;
          if constexpr (FMT == QG_W4_BF16) {
            const uint2 u = lds64(sc), v = lds64(sc + 8 * Sl::SCL);
            sa[0] = __uint_as_float(u.x << 16); sa[1] = __uint_as_float(u.x & 0xFFFF0000u);
            sa[2] = __uint_as_float(u.y << 16); sa[3] = __uint_as_float(u.y & 0xFFFF0000u);
            sb[0] = __uint_as_float(v.x << 16); sb[1] = __uint_as_float(v.x & 0xFFFF0000u);
            sb[2] = __uint_as_float(v.y << 16); sb[3] = __uint_as_float(v.y & 0xFFFF0000u);
          } else {
            const float4 u = lds128f(sc), v = lds128f(sc + 8 * Sl::SCL);
            sa[0] = u.x; sa[1] = u.y; sa[2] = u.z; sa[3] = u.w;
            sb[0] = v.x; sb[1] = v.y; sb[2] = v.z; sb[3] = v.w;
          }
          if constexpr (FMT == QG_W4_ASYM) {
            const float4 u = lds128f(sc + WROWS * 16), v = lds128f(sc + WROWS * 16 + 8 * 16);
            const float f = -1.0f / 136.0f;
            za[0] = f * u.x; za[1] = f * u.y; za[2] = f * u.z; za[3] = f * u.w;
            zb[0] = f * v.x; zb[1] = f * v.y; zb[2] = f * v.z; zb[3] = f * v.w;
          }
          if (half) {  // nothing was copied there
            sa[2] = sa[3] = sb[2] = sb[3] = 0.0f;
            if constexpr (FMT == QG_W4_ASYM) za[2] = za[3] = zb[2] = zb[3] = 0.0f;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pa[4], pb[4];
            codes8(q < 2 ? w01[2 * q] : w23[2 * q - 4], pa);
            codes8(q < 2 ? w01[2 * q + 1] : w23[2 * q - 3], pb);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float d[4];
              mma16816(d, pa[0], pb[0], pa[1], pb[1], xb[n][q].x, xb[n][q].y, z[n][q][0], z[n][q][1]);
              mma16816(d, pa[2], pb[2], pa[3], pb[3], xb[n][q].z, xb[n][q].w);
              float* ac = acc[i][n];
              ac[0] = fmaf(sa[q], d[0], ac[0]);
              ac[1] = fmaf(sa[q], d[1], ac[1]);
              ac[2] = fmaf(sb[q], d[2], ac[2]);
              ac[3] = fmaf(sb[q], d[3], ac[3]);
              if constexpr (FMT == QG_W4_ASYM) {
                ac[0] = fmaf(za[q], z[n][q][0], ac[0]);
                ac[1] = fmaf(za[q], z[n][q][1], ac[1]);
                ac[2] = fmaf(zb[q], z[n][q][0], ac[2]);
                ac[3] = fmaf(zb[q], z[n][q][1], ac[3]);
              }
            }
          }
        }
        __syncwarp();  // the slot may be filled again
        slot ^= 1;
      }
      // partial sums [K warp][token][row]; a lane holds rows g, g + 8 and
      // columns 2t, 2t + 1 of each tile
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if (16 * i >= at.nrows) break;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float* d = part + ((size_t)kw * 8 * NT + 8 * n + 2 * t) * prows + at.base + 16 * i + g;
          d[0] = acc[i][n][0];
          d[prows] = acc[i][n][1];
          d[8] = acc[i][n][2];
          d[prows + 8] = acc[i][n][3];
        }
      }
    }
    // the next run's first x, before the sums of this one
    Run nx = at;
    sh.next(nx);
    if (nx.nrows > 0) {
      if (!DENSE && (nx.e != at.e || nx.pass != at.pass)) point_x(nx);
      load_x(xn, ch0);
    }
    if (threadIdx.x == 0) sh.prefetch(ahead, SB, zoff, FMT == QG_W4_ASYM);
    __syncthreads();
    sum_and_store(c, at, p0, np, 8 * NT, wk, part, prows);
    __syncthreads();
    at = nx;
  }
  cp_wait<0>();
}

size_t rows_smem(int fmt, int nt, int wk, int E) {
  const int slot = fmt == QG_W4_BF16 ? Slot<QG_W4_BF16>::BYTES
                   : fmt == QG_W4_F32 ? Slot<QG_W4_F32>::BYTES : Slot<QG_W4_ASYM>::BYTES;
  return (size_t)W * D * slot + (size_t)wk * 8 * nt * (WROWS * (W / wk) + 4) * 4 +
         (size_t)(3 * E + 1) * 4;
}

template <int FMT, int NT, bool DENSE>
int run_rows(RowsArgs a, cudaStream_t st) {
  const size_t smem = rows_smem(FMT, NT, a.wk, a.c.E);
  int ctas = num_sms() * (a.per_sm == 2 && NT == 1 && smem <= 113 * 1024 ? 2 : 1);
  if (DENSE) {  // in blocks of 8 rows, half an MMA tile
    const int blocks = (int)cdiv(a.c.N, 8);
    ctas = (int)min64(ctas, blocks);
    a.share = blocks / ctas;
    a.more = blocks % ctas;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, a16w4_rows_kernel<FMT, NT, DENSE>, a, status_word()) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

template <int FMT>
int run_rows_nt(int nt, const RowsArgs& a, cudaStream_t st) {
  if (!a.c.offsets) return nt == 1 ? run_rows<FMT, 1, true>(a, st) : run_rows<FMT, 2, true>(a, st);
  return nt == 1 ? run_rows<FMT, 1, false>(a, st) : run_rows<FMT, 2, false>(a, st);
}

template <int FMT, int NT, bool DENSE>
int set_rows_smem() {
  size_t most = 0;
  for (int wk = 1; wk <= W; wk *= 2) {
    const size_t b = rows_smem(FMT, NT, wk, kA16W4MaxExperts);
    most = b > most ? b : most;
  }
  return cudaFuncSetAttribute((const void*)a16w4_rows_kernel<FMT, NT, DENSE>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) ==
                 cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

template <int FMT>
int set_rows_smem_nt() {
  int rc = set_rows_smem<FMT, 1, true>();
  if (rc == QG_OK) rc = set_rows_smem<FMT, 2, true>();
  if (rc == QG_OK) rc = set_rows_smem<FMT, 1, false>();
  if (rc == QG_OK) rc = set_rows_smem<FMT, 2, false>();
  return rc;
}

}  // namespace

int a16w4_setup() {
  int rc = set_rows_smem_nt<QG_W4_F32>();
  if (rc == QG_OK) rc = set_rows_smem_nt<QG_W4_BF16>();
  if (rc == QG_OK) rc = set_rows_smem_nt<QG_W4_ASYM>();
  if (rc == QG_OK) rc = a16w4_tc_setup();
  return rc;
}

int launch_a16w4_rows(const A16W4Call& c, cudaStream_t st) {
  RowsArgs a{};
  a.c = c;
  a.chunks = (int)cdiv(c.K, KC);
  // tokens per pass: what one expert has, as far as the host knows
  const int64_t each = cdiv(c.S, c.E);
  const int nt = each <= 8 ? 1 : 2;
  // weight rows of an SM, as far as the host knows
  const int64_t share = min64(c.E, c.S) * c.N / num_sms();
  // Two CTAs an SM hide each other's start and sums, but each reads all of x:
  // one where an SM has no more than a run's rows.
  a.per_sm = share > WROWS ? 2 : 1;
  // All warps split K, except where a CTA has rows for two row warps and K
  // would leave each warp less than four chunks between two sums.
  a.wk = 1;
  while (a.wk * 2 <= W && a.wk * 2 <= a.chunks) a.wk *= 2;
  while (a.wk > 1 && a.chunks < 4 * a.wk && share >= 4 * WROWS * (W / a.wk)) a.wk /= 2;
  if (c.format == QG_W4_F32) return run_rows_nt<QG_W4_F32>(nt, a, st);
  if (c.format == QG_W4_BF16) return run_rows_nt<QG_W4_BF16>(nt, a, st);
  return run_rows_nt<QG_W4_ASYM>(nt, a, st);
}

}  // namespace qg

using namespace qg;

// ---------------------------------------------------------------------------
// Entry points
// ---------------------------------------------------------------------------
namespace {

int64_t packed_bytes(int N, int K, int format) {
  const int64_t group = format == QG_W4_BF16 ? 2 : format == QG_W4_F32 ? 4 : 8;
  return (int64_t)N * (K / 2) + (int64_t)N * (K / 32) * group;
}

// Few rows per expert stream the weights past warp MMAs, more go to the
// tensor cores.  One matrix, at N = 14336, K = 4096: 16 rows take 19 us here
// and 22 there, 32 rows 34 and 22 (12 rows at 2048 x 2048: 4.6 and 12.7).
// Experts (64 of 2048 x 2048): 3 rows each take 54 and 75 us, 4 rows 63 and 76,
// 16 rows 122 and 83.  The host knows the average alone: 512 rows of 128
// experts take 116 us here and 152 there when they are spread evenly, 60 and 18
// when one expert has them all.
bool few_rows(int E, int S) { return cdiv(S, E) <= (E > 1 ? 4 : kDenseRows); }

// Checks of every product: QG_OK when the call can run (S may be 0).
int product_args(int E, int S, int N, int K, const void* in, int64_t ld_in, int in_cols,
                 const void* packed, int64_t expert_bytes, int format, const float* bias,
                 const void* out, int64_t ld_out, int out_cols) {
  if (E <= 0 || S < 0 || N <= 0 || K <= 0 || ld_in < in_cols || ld_out < out_cols)
    return QG_ERR_INVALID_ARG;
  if (format != QG_W4_F32 && format != QG_W4_BF16 && format != QG_W4_ASYM)
    return QG_ERR_INVALID_ARG;
  if (K % 64 || E > kA16W4MaxExperts || N > kA16W4MaxSide || K > kA16W4MaxSide)
    return QG_ERR_UNSUPPORTED;
  if (S == 0) return QG_OK;
  if (!in || !packed || !out) return QG_ERR_INVALID_ARG;
  if (((uintptr_t)packed & 15) || ((uintptr_t)in & 15) || ld_in % 8 || ((uintptr_t)out & 1) ||
      ((uintptr_t)bias & 3))
    return QG_ERR_MISALIGNED;
  if (E > 1) {
    if (expert_bytes < packed_bytes(N, K, format)) return QG_ERR_INVALID_ARG;
    if (expert_bytes % 16) return QG_ERR_MISALIGNED;
  }
  return QG_OK;
}

}  // namespace

extern "C" int qgemm_a16w4_bf16(int M, int N, int K, const void* x, int64_t ldx,
                                const void* packed_w, int format, const float* bias, void* y,
                                int64_t ldy, void* stream) {
  int rc = product_args(1, M, N, K, x, ldx, K, packed_w, 0, format, bias, y, ldy, N);
  if (rc != QG_OK || M == 0) return rc;
  rc = device_setup_status();
  if (rc != QG_OK) return rc;
  A16W4Call c{};
  c.E = 1; c.S = M; c.N = N; c.K = K;
  c.in = (const uint16_t*)x; c.ld_in = ldx; c.in_rows = M; c.topk = 1;
  c.packed = (const uint8_t*)packed_w; c.format = format; c.bias = bias;
  c.out = (uint16_t*)y; c.ld_out = ldy;
  return few_rows(1, M) ? launch_a16w4_rows(c, (cudaStream_t)stream)
                        : launch_a16w4_tc(c, false, nullptr, (cudaStream_t)stream);
}

extern "C" int qgemm_a16w4_bf16_grad_x(int M, int N, int K, const void* dy, int64_t lddy,
                                       const void* packed_w, int format, void* dx, int64_t lddx,
                                       void* stream) {
  int rc = product_args(1, M, N, K, dy, lddy, N, packed_w, 0, format, nullptr, dx, lddx, K);
  if (rc != QG_OK || M == 0) return rc;
  rc = device_setup_status();
  if (rc != QG_OK) return rc;
  A16W4Call c{};
  c.E = 1; c.S = M; c.N = N; c.K = K;
  c.in = (const uint16_t*)dy; c.ld_in = lddy; c.in_rows = M; c.topk = 1;
  c.packed = (const uint8_t*)packed_w; c.format = format;
  c.out = (uint16_t*)dx; c.ld_out = lddx;
  return launch_a16w4_tc(c, true, nullptr, (cudaStream_t)stream);
}

extern "C" int qgemm_a16w4_bf16_experts_grad_x(int E, int S, int N, int K, const void* dy,
                                               int64_t lddy, const int32_t* offsets,
                                               const void* packed_w, int64_t expert_bytes,
                                               int format, void* dx, int64_t lddx,
                                               void* stream) {
  int rc = product_args(E, S, N, K, dy, lddy, N, packed_w, expert_bytes, format, nullptr, dx, lddx, K);
  if (rc != QG_OK || S == 0) return rc;
  if (!offsets) return QG_ERR_INVALID_ARG;
  if ((uintptr_t)offsets & 3) return QG_ERR_MISALIGNED;
  rc = device_setup_status();
  if (rc != QG_OK) return rc;
  A16W4Call c{};
  c.E = E; c.S = S; c.N = N; c.K = K;
  c.in = (const uint16_t*)dy; c.ld_in = lddy; c.in_rows = S; c.topk = 1;
  c.offsets = offsets; c.packed = (const uint8_t*)packed_w; c.expert_bytes = expert_bytes;
  c.format = format; c.out = (uint16_t*)dx; c.ld_out = lddx;
  return launch_a16w4_tc(c, true, nullptr, (cudaStream_t)stream);
}

extern "C" size_t qgemm_a16w4_bf16_experts_workspace_bytes(int E, int S, int K, int indirect) {
  if (E <= 0 || S <= 0 || K <= 0 || K % 64) return 0;
  return few_rows(E, S) ? 0 : a16w4_tc_workspace(S, K, indirect != 0);
}

extern "C" int qgemm_a16w4_bf16_experts(int E, int S, int N, int K, const void* x, int64_t ldx,
                                        int x_rows, const int32_t* src, int topk,
                                        const int32_t* offsets, const void* packed_w,
                                        int64_t expert_bytes, int format, const float* bias,
                                        void* y, int64_t ldy, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  int rc = product_args(E, S, N, K, x, ldx, K, packed_w, expert_bytes, format, bias, y, ldy, N);
  if (rc != QG_OK) return rc;
  if (topk <= 0 || x_rows < 0) return QG_ERR_INVALID_ARG;
  if (S == 0) return QG_OK;
  if (!offsets || x_rows == 0 || (!src && x_rows < S)) return QG_ERR_INVALID_ARG;
  if (((uintptr_t)offsets | (uintptr_t)src) & 3) return QG_ERR_MISALIGNED;
  const size_t need = qgemm_a16w4_bf16_experts_workspace_bytes(E, S, K, src != nullptr);
  if (need && (!workspace || workspace_bytes < need)) return QG_ERR_WORKSPACE;
  if (need && ((uintptr_t)workspace & 255)) return QG_ERR_MISALIGNED;
  rc = device_setup_status();
  if (rc != QG_OK) return rc;
  A16W4Call c{};
  c.E = E; c.S = S; c.N = N; c.K = K;
  c.in = (const uint16_t*)x; c.ld_in = ldx; c.in_rows = x_rows; c.src = src; c.topk = topk;
  c.offsets = offsets; c.packed = (const uint8_t*)packed_w; c.expert_bytes = expert_bytes;
  c.format = format; c.bias = bias; c.out = (uint16_t*)y; c.ld_out = ldy;
  return few_rows(E, S) ? launch_a16w4_rows(c, (cudaStream_t)stream)
                        : launch_a16w4_tc(c, false, workspace, (cudaStream_t)stream);
}
