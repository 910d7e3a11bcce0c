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
// leaves 3.4 lane instructions per weight.  A scalar form (unpack, convert,
// multiply) takes most of them for one row and grows with the rows.  Warp
// MMAs (m16n8k16) take 16 weight rows x 8 token rows at once: the cost per
// weight is the unpacking (about 1.4 instructions), whatever the number of
// tokens up to 8.  The MMAs see the exact codes, each group's two MMAs start
// from zero, and the group scale is applied to their f32 result, so nothing
// is rounded below f32 before y.
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
constexpr int SR = 32;            // weight rows per step (two MMA row tiles)
constexpr int RP = 2;             // steps per chunk at most: 64 rows per warp
constexpr int WROWS = SR * RP;
constexpr int NIB_PITCH = 80;     // 64 bytes of nibbles; the pitch spreads 8 rows over all banks

// Bytes of one step in a warp's ring: nibbles, then scales (and zeros) of SR
// rows x 4 groups.
template <int FMT>
struct Step {
  static constexpr int SCL = FMT == QG_W4_BF16 ? 8 : 16;  // scale bytes per row
  static constexpr int OFF_SCL = SR * NIB_PITCH;
  static constexpr int OFF_ZERO = OFF_SCL + SR * SCL;
  static constexpr int BYTES = OFF_ZERO + (FMT == QG_W4_ASYM ? SR * 16 : 0);
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

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
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

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8 codes of nibble word w as four bf16 pairs, exact: 0x4300 | u is
// 128 + u, less 136 is u - 8.  Pair order: codes (0,2), (4,6), (1,3), (5,7).
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&p)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(p[i]) : "r"(m), "r"(0x43084308u));
  }
}

// What the CTAs of one launch share out: the weight rows of every pass over
// an expert's tokens, one after another ("virtual rows").  A pass takes up
// to 8*NT tokens.
struct RowsArgs {
  A16W4Call c;
  int chunks;        // ceil(K / KC)
  int wk;            // warps that split K; W / wk warps split the rows
  int min_rows;      // fewest rows a CTA takes
};

// A run: consecutive weight rows of one pass, at most WROWS per row warp.
struct Run {
  int e, r0, rows, p0, np;  // expert, first weight row, rows, first sorted row, token rows
};

// Position of a warp in its steps: run, chunk, step within the chunk.
struct Cursor {
  int64_t v;   // virtual row where the run starts
  Run run;
  int base, nrows, steps;  // this warp's rows of the run and its steps per chunk
  int chunk, step;
  bool done;
};

template <int FMT, int NT, int D>
__global__ void __launch_bounds__(W * 32, NT <= 2 ? 2 : 1)
    a16w4_rows_kernel(const RowsArgs a, int* status) {
  using St = Step<FMT>;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ int64_t s_total;
  const A16W4Call& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;  // MMA fragment coordinates
  const int K = c.K, N = c.N, G = K >> 5;
  const int wk = a.wk, wr = W / wk;
  const int kw = warp % wk, rw = warp / wk;
  // shared memory: rings, partial sums, expert tables
  const int prows = WROWS * wr + 4;  // pitch of a token's partial sums; +4 spreads the banks
  const uint32_t ring = smem_u32(sm) + (uint32_t)(warp * D * St::BYTES);
  float* part = reinterpret_cast<float*>(sm + W * D * St::BYTES);
  int* pre = reinterpret_cast<int*>(part + (size_t)wk * 8 * NT * prows);  // [E + 1] passes before e
  int* start = pre + c.E + 1;
  int* count = start + c.E;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (c.offsets) asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int e = threadIdx.x; e < c.E; e += W * 32) {
    const int2 r = expert_range(c.offsets, e, c.S, status);
    start[e] = r.x;
    count[e] = r.y;
  }
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    for (int b = 0; b < c.E; b += 32) {
      const int e = b + lane;
      const int own = e < c.E ? (count[e] + 8 * NT - 1) / (8 * NT) : 0;
      int x = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (e < c.E) pre[e] = carry + x - own;
      carry += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      pre[c.E] = carry;
      s_total = (int64_t)carry * N;
    }
  }
  __syncthreads();
  const int64_t total = s_total;
  int64_t per = (total + gridDim.x - 1) / gridDim.x;
  int64_t v0, v1;
  if (per < a.min_rows) {
    v0 = min64(total, (int64_t)blockIdx.x * a.min_rows);
    v1 = min64(total, v0 + a.min_rows);
  } else {
    // shares differ by one row at most
    const int64_t q = total / gridDim.x, r = total - q * gridDim.x;
    v0 = q * blockIdx.x + min64(r, blockIdx.x);
    v1 = v0 + q + (blockIdx.x < r ? 1 : 0);
  }

  const int ch0 = (int)((int64_t)kw * a.chunks / wk), ch1 = (int)((int64_t)(kw + 1) * a.chunks / wk);

  auto open_run = [&](Cursor& cu) {
    if (cu.v >= v1) {
      cu.done = true;
      return;
    }
    const int u = (int)(cu.v / N);
    int lo = 0, hi = c.E - 1;  // last expert with pre[e] <= u that has passes
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] <= u) lo = mid; else hi = mid - 1;
    }
    cu.run.e = lo;
    const int pass = u - pre[lo];
    cu.run.r0 = (int)(cu.v - (int64_t)u * N);
    cu.run.rows = (int)min64(min64(N - cu.run.r0, v1 - cu.v), (int64_t)WROWS * wr);
    cu.run.p0 = start[lo] + pass * 8 * NT;
    cu.run.np = min(count[lo] - pass * 8 * NT, 8 * NT);
    const int share = ((cu.run.rows + wr - 1) / wr + 15) & ~15;  // rows per row warp
    cu.base = rw * share;
    cu.nrows = max(0, min(cu.run.rows - cu.base, share));
    cu.steps = (cu.nrows + SR - 1) / SR;
    cu.chunk = ch0;
    cu.step = 0;
  };
  // to the first run at or after the cursor's place where this warp has steps
  auto settle = [&](Cursor& cu) {
    while (!cu.done && (cu.steps == 0 || ch0 == ch1)) {
      cu.v += cu.run.rows;
      open_run(cu);
    }
  };
  auto advance = [&](Cursor& cu) {
    if (++cu.step < cu.steps) return;
    cu.step = 0;
    if (++cu.chunk < ch1) return;
    cu.v += cu.run.rows;
    open_run(cu);
    settle(cu);
  };

  auto issue = [&](const Cursor& cu, int slot) {
    if (!cu.done) {
      const uint8_t* wq = c.packed + (int64_t)cu.run.e * c.expert_bytes;
      const int row0 = cu.run.r0 + cu.base + SR * cu.step;  // weight row of the step's first
      const int nr = min(SR, cu.nrows - SR * cu.step);
      const int groups = min(4, G - 4 * cu.chunk);          // 4, or 2 at the end of K
      const uint32_t dst = ring + (uint32_t)(slot * St::BYTES);
      const uint8_t* nib = wq + (int64_t)row0 * (K >> 1) + (int64_t)cu.chunk * (KC / 2);
#pragma unroll
      for (int i = 0; i < SR * 4 / 32; ++i) {
        const int r = (lane >> 2) + 8 * i, q = lane & 3;
        if (r < nr && q < groups) cp16(dst + r * NIB_PITCH + q * 16, nib + (int64_t)r * (K >> 1) + q * 16);
      }
      const uint8_t* scl = wq + (int64_t)N * (K >> 1);
      if (lane < nr) {
        const int64_t at = (int64_t)(row0 + lane) * G + 4 * cu.chunk;
        const uint32_t d = dst + St::OFF_SCL + lane * St::SCL;
        if constexpr (FMT == QG_W4_BF16) {
          cp4(d, scl + 2 * at);
          if (groups == 4) cp4(d + 4, scl + 2 * at + 4);
        } else {
          cp8(d, scl + 4 * at);
          if (groups == 4) cp8(d + 8, scl + 4 * at + 8);
        }
        if constexpr (FMT == QG_W4_ASYM) {
          const uint8_t* zer = scl + (int64_t)N * G * 4;
          cp8(dst + St::OFF_ZERO + lane * 16, zer + 4 * at);
          if (groups == 4) cp8(dst + St::OFF_ZERO + lane * 16 + 8, zer + 4 * at + 8);
        }
      }
    }
    cp_commit();
  };

  Cursor put;
  put.v = v0;
  put.done = false;
  open_run(put);
  settle(put);
#pragma unroll
  for (int d = 0; d < D - 1; ++d) {
    issue(put, d);
    if (!put.done) advance(put);
  }
  if (!c.offsets) asm volatile("griddepcontrol.wait;" ::: "memory");

  // every warp walks every run: its steps, then the sum over the K warps
  Cursor at;
  at.v = v0;
  at.done = false;
  open_run(at);
  int slot = 0;
  while (!at.done) {
    float acc[2 * RP][NT][4];
#pragma unroll
    for (int i = 0; i < 2 * RP; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][n][k] = 0.0f;
    // this lane's token rows (MMA column g); columns past the last token
    // repeat it, and are not stored
    const uint16_t* xr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int p = at.run.p0 + min(8 * n + g, at.run.np - 1);
      int64_t row = p;
      if (c.src) {
        const int s = c.src[p];
        row = s < 0 ? -1 : s / c.topk;
      }
      if (row < 0 || row >= c.in_rows) {  // read as zeros
        record_error(status, QG_ERR_INVALID_ARG);
        xr[n] = nullptr;
      } else {
        xr[n] = c.in + row * c.ld_in;
      }
    }
    if (at.steps > 0) {
      for (int ch = ch0; ch < ch1; ++ch) {
        const int groups = min(4, G - 4 * ch);
        uint4 xb[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            xb[n][q] = make_uint4(0, 0, 0, 0);
            if (xr[n] && q < groups)
              xb[n][q] = *reinterpret_cast<const uint4*>(xr[n] + (int64_t)ch * KC + q * 32 + t * 8);
          }
        // pairs in the order of codes8
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint4 v = xb[n][q];
            xb[n][q] = make_uint4(prmt(v.x, v.y, 0x5410), prmt(v.z, v.w, 0x5410),
                                  prmt(v.x, v.y, 0x7632), prmt(v.z, v.w, 0x7632));
          }
#pragma unroll
        for (int s = 0; s < RP; ++s) {
          if (s >= at.steps) break;
          issue(put, slot == 0 ? D - 1 : slot - 1);
          if (!put.done) advance(put);
          cp_wait<D - 1>();
          __syncwarp();
          const uint32_t st = ring + (uint32_t)(slot * St::BYTES);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (SR * s + 16 * i >= at.nrows) break;
            const uint32_t ra = st + (16 * i + g) * NIB_PITCH + t * 4;
            float sa[4], sb[4], za[4], zb[4];
            const uint32_t sc = st + St::OFF_SCL + (16 * i + g) * St::SCL;
            if constexpr (FMT == QG_W4_BF16) {
              const uint2 u = lds64(sc), v = lds64(sc + 8 * St::SCL);
              sa[0] = __uint_as_float(u.x << 16); sa[1] = __uint_as_float(u.x & 0xFFFF0000u);
              sa[2] = __uint_as_float(u.y << 16); sa[3] = __uint_as_float(u.y & 0xFFFF0000u);
              sb[0] = __uint_as_float(v.x << 16); sb[1] = __uint_as_float(v.x & 0xFFFF0000u);
              sb[2] = __uint_as_float(v.y << 16); sb[3] = __uint_as_float(v.y & 0xFFFF0000u);
            } else {
              const float4 u = lds128f(sc), v = lds128f(sc + 8 * St::SCL);
              sa[0] = u.x; sa[1] = u.y; sa[2] = u.z; sa[3] = u.w;
              sb[0] = v.x; sb[1] = v.y; sb[2] = v.z; sb[3] = v.w;
            }
            if constexpr (FMT == QG_W4_ASYM) {
              const uint32_t zc = st + St::OFF_ZERO + (16 * i + g) * 16;
              const float4 u = lds128f(zc), v = lds128f(zc + 8 * 16);
              za[0] = u.x; za[1] = u.y; za[2] = u.z; za[3] = u.w;
              zb[0] = v.x; zb[1] = v.y; zb[2] = v.z; zb[3] = v.w;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (q >= groups) break;
              uint32_t pa[4], pb[4];
              codes8(lds32(ra + q * 16), pa);
              codes8(lds32(ra + 8 * NIB_PITCH + q * 16), pb);
              const uint32_t a0[4] = {pa[0], pb[0], pa[1], pb[1]};
              const uint32_t a1[4] = {pa[2], pb[2], pa[3], pb[3]};
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma16816(d, a0, xb[n][q].x, xb[n][q].y);
                mma16816(d, a1, xb[n][q].z, xb[n][q].w);
                float* ac = acc[2 * s + i][n];
                ac[0] = fmaf(sa[q], d[0], ac[0]);
                ac[1] = fmaf(sa[q], d[1], ac[1]);
                ac[2] = fmaf(sb[q], d[2], ac[2]);
                ac[3] = fmaf(sb[q], d[3], ac[3]);
                if constexpr (FMT == QG_W4_ASYM) {
                  // X[p,g] in every row: MMAs with ones
                  const uint32_t one[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
                  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                  mma16816(x, one, xb[n][q].x, xb[n][q].y);
                  mma16816(x, one, xb[n][q].z, xb[n][q].w);
                  ac[0] = fmaf(za[q], x[0], ac[0]);
                  ac[1] = fmaf(za[q], x[1], ac[1]);
                  ac[2] = fmaf(zb[q], x[2], ac[2]);
                  ac[3] = fmaf(zb[q], x[3], ac[3]);
                }
              }
            }
          }
          __syncwarp();  // the slot may be filled again
          slot = slot + 1 == D ? 0 : slot + 1;
        }
      }
    }
    // partial sums [K warp][token][row]; a lane holds rows g, g + 8 and
    // columns 2t, 2t + 1 of each tile
    if (at.steps > 0) {
#pragma unroll
      for (int i = 0; i < 2 * RP; ++i) {
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
    __syncthreads();
    for (int o = threadIdx.x; o < at.run.rows * at.run.np; o += W * 32) {
      const int tok = o / at.run.rows, r = o - tok * at.run.rows;
      float s = 0.0f;
      for (int k = 0; k < wk; ++k) s += part[((size_t)k * 8 * NT + tok) * prows + r];
      const int n = at.run.r0 + r;
      if (c.bias) s += __ldg(c.bias + (int64_t)at.run.e * N + n);
      c.out[(int64_t)(at.run.p0 + tok) * c.ld_out + n] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
    }
    __syncthreads();
    at.v += at.run.rows;
    open_run(at);
  }
  cp_wait<0>();
}

template <int FMT, int NT>
struct Ring {
  static constexpr int D = 3;
};

size_t rows_smem(int fmt, int nt, int d, int wk, int E) {
  const int step = fmt == QG_W4_BF16 ? Step<QG_W4_BF16>::BYTES
                   : fmt == QG_W4_F32 ? Step<QG_W4_F32>::BYTES : Step<QG_W4_ASYM>::BYTES;
  return (size_t)W * d * step + (size_t)wk * 8 * nt * (WROWS * (W / wk) + 4) * 4 +
         (size_t)(3 * E + 1) * 4;
}

template <int FMT, int NT>
int run_rows(const RowsArgs& a, cudaStream_t st) {
  constexpr int D = Ring<FMT, NT>::D;
  const size_t smem = rows_smem(FMT, NT, D, a.wk, a.c.E);
  const int per_sm = smem <= 112 * 1024 ? 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_sms() * per_sm));
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, a16w4_rows_kernel<FMT, NT, D>, a, status_word()) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

template <int FMT>
int run_rows_nt(int nt, const RowsArgs& a, cudaStream_t st) {
  if (nt == 1) return run_rows<FMT, 1>(a, st);
  if (nt == 2) return run_rows<FMT, 2>(a, st);
  return run_rows<FMT, 4>(a, st);
}

template <int FMT, int NT>
int set_rows_smem() {
  const size_t most = rows_smem(FMT, NT, Ring<FMT, NT>::D, W, kA16W4MaxExperts);
  return cudaFuncSetAttribute((const void*)a16w4_rows_kernel<FMT, NT, Ring<FMT, NT>::D>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)most) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

template <int FMT>
int set_rows_smem_nt() {
  int rc = set_rows_smem<FMT, 1>();
  if (rc == QG_OK) rc = set_rows_smem<FMT, 2>();
  if (rc == QG_OK) rc = set_rows_smem<FMT, 4>();
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
  a.wk = 1;
  while (a.wk * 2 <= W && a.wk * 2 <= a.chunks) a.wk *= 2;
  a.min_rows = 8;
  // token rows per pass: what one expert has, as far as the host knows
  const int64_t each = cdiv(c.S, c.E);
  const int nt = each <= 8 ? 1 : each <= 16 ? 2 : 4;
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
// tensor cores.
int launch_product(const A16W4Call& c, cudaStream_t st) {
  if (cdiv(c.S, c.E) <= 32) return launch_a16w4_rows(c, st);
  return launch_a16w4_tc(c, false, st);
}

// Checks of every product: QG_OK when the call can run (S may be 0).
int product_args(int E, int S, int N, int K, const void* in, int64_t ld_in, int in_cols,
                 const void* packed, int64_t expert_bytes, int format, const float* bias,
                 const void* out, int64_t ld_out, int out_cols) {
  if (E <= 0 || S < 0 || N <= 0 || K <= 0 || ld_in < in_cols || ld_out < out_cols)
    return QG_ERR_INVALID_ARG;
  if (format != QG_W4_F32 && format != QG_W4_BF16 && format != QG_W4_ASYM)
    return QG_ERR_INVALID_ARG;
  if (K % 64 || E > kA16W4MaxExperts) return QG_ERR_UNSUPPORTED;
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
  return launch_product(c, (cudaStream_t)stream);
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
  return launch_a16w4_tc(c, true, (cudaStream_t)stream);
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
  return launch_a16w4_tc(c, true, (cudaStream_t)stream);
}

extern "C" int qgemm_a16w4_bf16_experts(int E, int S, int N, int K, const void* x, int64_t ldx,
                                        int x_rows, const int32_t* src, int topk,
                                        const int32_t* offsets, const void* packed_w,
                                        int64_t expert_bytes, int format, const float* bias,
                                        void* y, int64_t ldy, void* stream) {
  int rc = product_args(E, S, N, K, x, ldx, K, packed_w, expert_bytes, format, bias, y, ldy, N);
  if (rc != QG_OK) return rc;
  if (topk <= 0 || x_rows < 0) return QG_ERR_INVALID_ARG;
  if (S == 0) return QG_OK;
  if (!offsets || x_rows == 0 || (!src && x_rows < S)) return QG_ERR_INVALID_ARG;
  if (((uintptr_t)offsets | (uintptr_t)src) & 3) return QG_ERR_MISALIGNED;
  rc = device_setup_status();
  if (rc != QG_OK) return rc;
  A16W4Call c{};
  c.E = E; c.S = S; c.N = N; c.K = K;
  c.in = (const uint16_t*)x; c.ld_in = ldx; c.in_rows = x_rows; c.src = src; c.topk = topk;
  c.offsets = offsets; c.packed = (const uint8_t*)packed_w; c.expert_bytes = expert_bytes;
  c.format = format; c.bias = bias; c.out = (uint16_t*)y; c.ld_out = ldy;
  return launch_product(c, (cudaStream_t)stream);
}
