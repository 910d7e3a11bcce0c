// Tokens in the order of their experts, and back: the stable order by expert
// id, token rows spread to their sorted positions, the weighted sum of the
// sorted rows per token, and the gradients of both.
//
//   order    sorted position p of entry i = t*topk + j with expert id e:
//            p = #{entries of smaller ids} + #{entries of id e before i}
//   spread   xs[pos[t,j]] = x[t]            (gradient: the sum below, weights 1)
//   combine  y[t] = sum_j w[t,j] * ys[pos[t,j]]
//   its gradient  dys[pos[t,j]] = w[t,j] * dy[t],  dw[t,j] = <dy[t], ys[pos[t,j]]>
//
// The row kernels are bound by HBM: each moves every row it needs once, in
// 16-byte accesses where the rows allow it.  Walking the tokens (not the
// sorted rows) lets a token's row be read once for its topk copies, and lets
// combine's gradient read dy once for all of a token's experts.  Sums are
// held in f32 and rounded once.
//
// Every kernel becomes resident while the work before it may still be writing
// its inputs.  They are not constant over the kernel's life, so they are read by
// ordinary loads behind griddepcontrol.wait: no __ldg and no __restrict__ on
// an input, either of which lets a load go through the path for constants, or
// ahead of the wait.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include <type_traits>

#include "qg_internal.cuh"

namespace qg {

int device_setup_status();

namespace {

// ---------------------------------------------------------------------------
// Order by expert
// ---------------------------------------------------------------------------
// A warp owns a contiguous run of at most 32 * EPL entries, whose ids it loads
// at once, and takes them 32 at a time: one ballot per bit of the ids groups
// the lanes of one expert (a match instruction per 32 took 280 cycles, 19 us
// for 8192 entries), the lanes below a lane in its group give its rank, and
// the warp's own counters in shared memory carry the rank from one 32 to the
// next.  No atomics, so the order is the stable one by construction.
constexpr int kSortMaxE = 1024;
constexpr int EPL = 8;                   // entries per lane
constexpr int kSortOneWarps = 32;        // one CTA sorts everything
constexpr int64_t kSortOneMax = 2048;    // most entries of that form (it could hold 8192)
constexpr int64_t kSortMax = 1 << 22;    // each CTA reads every chunk's counts
constexpr int kSortWarps = 16;           // several CTAs
// Entries per CTA then: small chunks while there are few of them, since each CTA
// reads the counts of all.  E = 64: 8192 entries 5.3 us by chunks of 1024, 6.8
// of 2048, 11.6 in one CTA; E = 128, 65536 entries: 9.9, 8.3 (4096: 9.9); 262144:
// 23, 16.4 and, of 4096, 15.4.  2048 entries take 5.7 us in one CTA and 4.9 in two
// launches, of which the second costs the host 2 us.
int sort_chunk(int64_t n) { return n <= 32768 ? 1024 : n <= 131072 ? 2048 : kSortWarps * 32 * EPL; }

// Expert of entry i (of n), -1 for none.  n < 2^31, so 32-bit divisions.
__device__ __forceinline__ int expert_of(const int32_t* ids, int64_t ld, int topk, int64_t i,
                                         int64_t n, int E) {
  if (i >= n) return -1;
  int64_t at = i;
  if (ld != topk) {
    const uint32_t t = (uint32_t)i / (uint32_t)topk;
    at = t * ld + ((uint32_t)i - t * (uint32_t)topk);
  }
  const int e = ids[at];
  return (unsigned)e < (unsigned)E ? e : -1;
}

// Exclusive prefix sum over v[0, E) in place by the whole CTA; v[E] = total.
__device__ __forceinline__ void scan_experts(int* v, int E, int* part /* [33] */) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int carry = 0;
  for (int b = 0; b < E; b += blockDim.x) {
    const int i = b + threadIdx.x;
    const int own = i < E ? v[i] : 0;
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    int before = carry, total = 0;
    for (int w = 0; w < nw; ++w) {
      const int s = part[w];
      if (w < warp) before += s;
      total += s;
    }
    if (i < E) v[i] = before + x - own;
    carry += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) v[E] = carry;
  __syncthreads();
}

// Lanes with this lane's expert (of an id below 2^bits; -1 counts as one).
__device__ __forceinline__ uint32_t peers_of(int e, int bits) {
  uint32_t m = __ballot_sync(0xffffffffu, e >= 0);
  if (e < 0) m = ~m;
  for (int b = 0; b < bits; ++b) {
    const bool one = (e >> b) & 1;
    const uint32_t v = __ballot_sync(0xffffffffu, one);
    m &= one ? v : ~v;
  }
  return m;
}

// Dynamic shared memory: base[E + 1], then cnt[warps][E].
// hist == NULL: one CTA holds every entry.  Otherwise hist[chunks][E] holds
// each chunk's counts and this CTA places chunk blockIdx.x.
__global__ void __launch_bounds__(kSortOneWarps * 32)
    sort_place_kernel(int64_t n, int topk, int E, const int32_t* ids, int64_t ld,
                      const int32_t* hist, int64_t per_cta,
                      int32_t* __restrict__ offsets, int32_t* __restrict__ src,
                      int32_t* __restrict__ pos) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ int sort_smem[];
  __shared__ int part[33];
  int* base = sort_smem;
  int* cnt = sort_smem + E + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  for (int i = threadIdx.x; i < nw * E; i += blockDim.x) cnt[i] = 0;
  const int64_t c0 = (int64_t)blockIdx.x * per_cta;
  const int64_t c1 = min64(n, c0 + per_cta);
  const int rounds = (int)((c1 - c0 + nw * 32 - 1) / (nw * 32));  // at most EPL
  const int64_t i0 = c0 + (int64_t)warp * rounds * 32 + lane;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int e[EPL];
#pragma unroll
  for (int r = 0; r < EPL; ++r) e[r] = r < rounds ? expert_of(ids, ld, topk, i0 + 32 * r, c1, E) : -1;
  int* mine = cnt + warp * E;
  const int bits = 32 - __clz(E - 1 | 1);
#pragma unroll
  for (int r = 0; r < EPL; ++r) {
    if (r >= rounds) break;
    const uint32_t m = peers_of(e[r], bits);
    if (e[r] >= 0 && lane == __ffs(m) - 1) mine[e[r]] += __popc(m);
    __syncwarp();
  }
  __syncthreads();
  // base[e]: entries of e in all chunks; the earlier chunks' part is added
  // to the warps' starts
  for (int x = threadIdx.x; x < E; x += blockDim.x) {
    int all = 0, before = 0;
    if (hist) {
#pragma unroll 8
      for (int c = 0; c < (int)gridDim.x; ++c) {
        const int h = hist[(int64_t)c * E + x];
        all += h;
        if (c < (int)blockIdx.x) before += h;
      }
    }
    int here = before;
    for (int w = 0; w < nw; ++w) {
      const int k = cnt[w * E + x];
      cnt[w * E + x] = here;
      here += k;
    }
    base[x] = hist ? all : here;
  }
  __syncthreads();
  scan_experts(base, E, part);
  if (blockIdx.x == 0)
    for (int x = threadIdx.x; x <= E; x += blockDim.x) offsets[x] = base[x];
  // mine[e]: how many entries of e lie before this warp's next one
#pragma unroll
  for (int r = 0; r < EPL; ++r) {
    if (r >= rounds) break;
    const uint32_t m = peers_of(e[r], bits);
    int p = -1;
    if (e[r] >= 0) p = base[e[r]] + mine[e[r]] + __popc(m & ((1u << lane) - 1u));
    __syncwarp();
    if (e[r] >= 0 && lane == __ffs(m) - 1) mine[e[r]] += __popc(m);
    __syncwarp();
    const int64_t i = i0 + 32 * r;
    if (i < c1) {
      pos[i] = p;
      if (p >= 0) src[p] = (int32_t)i;
    }
  }
}

// Counts of each chunk, for the form with several CTAs.
__global__ void __launch_bounds__(kSortWarps * 32)
    sort_count_kernel(int64_t n, int topk, int E, const int32_t* ids, int64_t ld,
                      int64_t per_cta, int32_t* __restrict__ hist) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ int sort_smem[];
  for (int i = threadIdx.x; i < E; i += blockDim.x) sort_smem[i] = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t c0 = (int64_t)blockIdx.x * per_cta, c1 = min64(n, c0 + per_cta);
  int e[EPL];
#pragma unroll
  for (int r = 0; r < EPL; ++r)
    e[r] = expert_of(ids, ld, topk, c0 + r * (kSortWarps * 32) + threadIdx.x, c1, E);
#pragma unroll
  for (int r = 0; r < EPL; ++r)
    if (e[r] >= 0) atomicAdd(&sort_smem[e[r]], 1);  // integers: any order gives the same count
  __syncthreads();
  for (int x = threadIdx.x; x < E; x += blockDim.x)
    hist[(int64_t)blockIdx.x * E + x] = sort_smem[x];
}

// ---------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------
// V values of type T as one access of V * sizeof(T) bytes, kept as raw words
// until they are used (as arrays of 16-bit values the compiler widens them on
// arrival and runs out of registers).
template <typename T, int V, typename W = uint32_t, int N = (int)(sizeof(T) * V / sizeof(W))>
struct alignas(sizeof(T) * V) Words {
  W w[N];
};
template <typename T, int V>
struct Pack : Words<T, V> {};
template <typename T>
struct Pack<T, 1> : Words<T, 1, T, 1> {};  // a value on its own

template <int V>
__device__ __forceinline__ void unpack(const Words<float, V>& p, float (&f)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) f[k] = __uint_as_float(p.w[k]);
}
template <int V>
__device__ __forceinline__ void unpack(const Words<__nv_bfloat16, V>& p, float (&f)[V]) {
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    f[2 * k] = __uint_as_float(p.w[k] << 16);
    f[2 * k + 1] = __uint_as_float(p.w[k] & 0xFFFF0000u);
  }
}
template <int V>
__device__ __forceinline__ void unpack(const Words<__half, V>& p, float (&f)[V]) {
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&p.w[k]));
    f[2 * k] = v.x;
    f[2 * k + 1] = v.y;
  }
}
__device__ __forceinline__ void unpack(const Pack<float, 1>& p, float (&f)[1]) { f[0] = p.w[0]; }
__device__ __forceinline__ void unpack(const Pack<__half, 1>& p, float (&f)[1]) {
  f[0] = __half2float(p.w[0]);
}
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, 1>& p, float (&f)[1]) {
  f[0] = __bfloat162float(p.w[0]);
}

template <int V>
__device__ __forceinline__ void pack(const float (&f)[V], Words<float, V>& p) {
#pragma unroll
  for (int k = 0; k < V; ++k) p.w[k] = __float_as_uint(f[k]);
}
template <int V>
__device__ __forceinline__ void pack(const float (&f)[V], Words<__nv_bfloat16, V>& p) {
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
    p.w[k] = *reinterpret_cast<const uint32_t*>(&v);
  }
}
template <int V>
__device__ __forceinline__ void pack(const float (&f)[V], Words<__half, V>& p) {
#pragma unroll
  for (int k = 0; k < V / 2; ++k) {
    const __half2 v = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
    p.w[k] = *reinterpret_cast<const uint32_t*>(&v);
  }
}
__device__ __forceinline__ void pack(const float (&f)[1], Pack<float, 1>& p) { p.w[0] = f[0]; }
__device__ __forceinline__ void pack(const float (&f)[1], Pack<__half, 1>& p) {
  p.w[0] = __float2half_rn(f[0]);
}
__device__ __forceinline__ void pack(const float (&f)[1], Pack<__nv_bfloat16, 1>& p) {
  p.w[0] = __float2bfloat16_rn(f[0]);
}

// Sorted positions of J entries from pos on, of which there are n; negative
// ones have no expert.  A position outside [0, S) is an error of the caller's:
// recorded, then treated as -1.  All loads come before the checks: a load
// behind one check and ahead of the next would wait for it.
template <int J>
__device__ __forceinline__ void places_of(const int32_t* pos, int n, int64_t S, int* status, int (&p)[J]) {
#pragma unroll
  for (int j = 0; j < J; ++j) p[j] = j < n ? pos[j] : -1;
#pragma unroll
  for (int j = 0; j < J; ++j)
    if (p[j] >= S) {
      record_error(status, QG_ERR_INVALID_ARG);
      p[j] = -1;
    }
}

// J experts of a token are taken together: 8, or 4 or 2 where topk is no more.
// A thread has U accesses per row in flight: narrow ones (rows whose start or
// length is no multiple of 16 bytes) come in several, and so do the rows of
// few experts, so that about as much is on its way in every case.
constexpr int in_flight(int bytes, int J) {
  return (bytes >= 16 ? 1 : bytes == 8 ? 2 : 4) * (8 / J);
}

template <typename W, int U, int J>
__global__ void __launch_bounds__(256, 4)
    spread_rows_kernel(int topk, int64_t S, int64_t nv, const W* x, int64_t ldx,
                       const int32_t* pos, W* __restrict__ xs, int64_t ldxs,
                       int* status) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t t = blockIdx.x;
  const W* xr = x + t * ldx;
  const int64_t i0 = (int64_t)blockIdx.y * blockDim.x * U + threadIdx.x;
  const int64_t step = (int64_t)gridDim.y * blockDim.x * U;
  for (int jb = 0; jb < topk; jb += J) {
    int p[J];
    places_of(pos + t * topk + jb, topk - jb, S, status, p);
    for (int64_t i = i0; i < nv; i += step) {
      W a[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * (int)blockDim.x < nv) a[u] = xr[i + u * (int)blockDim.x];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (p[j] < 0) continue;
        W* d = xs + (int64_t)p[j] * ldxs;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (i + u * (int)blockDim.x < nv) d[i + u * (int)blockDim.x] = a[u];
      }
    }
  }
}

// Positions (and weights) first, then the loads of all J rows, then the sums:
// a row's load between two checks of positions waited for the one before it
// (8192 tokens x 8 rows of 4096 bf16: 282 us).
template <typename T, int V, int U, int J>
__global__ void __launch_bounds__(256, U == 1 ? 3 : 2)
    combine_rows_kernel(int topk, int64_t S, int64_t nv, const T* ys, int64_t ldys,
                        const int32_t* pos, const float* w,
                        T* __restrict__ y, int64_t ldy, int* status) {
  using P = Pack<T, V>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t t = blockIdx.x;
  const int64_t step = (int64_t)gridDim.y * blockDim.x * U;
  int p[J];
  float wj[J];
  auto places = [&](int jb) {
#pragma unroll
    for (int j = 0; j < J; ++j) wj[j] = w && jb + j < topk ? w[t * topk + jb + j] : 1.0f;
    places_of(pos + t * topk + jb, topk - jb, S, status, p);
  };
  if (topk <= J) places(0);
  for (int64_t i = (int64_t)blockIdx.y * blockDim.x * U + threadIdx.x; i < nv; i += step) {
    float acc[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < V; ++k) acc[u][k] = 0.0f;
    for (int jb = 0; jb < topk; jb += J) {
      if (topk > J) places(jb);
      P r[J][U];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (p[j] < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u == 0 || i + u * (int)blockDim.x < nv) 
            r[j][u] = reinterpret_cast<const P*>(ys + (int64_t)p[j] * ldys)[i + u * (int)blockDim.x];
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (p[j] < 0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float v[V];
          unpack(r[j][u], v);
#pragma unroll
          for (int k = 0; k < V; ++k) acc[u][k] = fmaf(wj[j], v[k], acc[u][k]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      P out;
      pack(acc[u], out);
      if (u == 0 || i + u * (int)blockDim.x < nv)
        reinterpret_cast<P*>(y + t * ldy)[i + u * (int)blockDim.x] = out;
    }
  }
}

// One CTA per token: the dot products of its experts' rows with dy[t] need
// the whole row, and dy is read once for J of them.
template <typename T, int V, int U, int J>
__global__ void __launch_bounds__(512)
    combine_grad_kernel(int topk, int64_t S, int64_t nv, const T* dy,
                                    int64_t lddy, const T* ys, int64_t ldys,
                                    const int32_t* pos, const float* w,
                                    T* __restrict__ dys, int64_t lddys, float* __restrict__ dw,
                                    int* status) {
  using P = Pack<T, V>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float red[J][32];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  for (int jb = 0; jb < topk; jb += J) {
    int p[J];
    float wj[J], dot[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      wj[j] = w && jb + j < topk ? w[t * topk + jb + j] : 1.0f;
      dot[j] = 0.0f;
    }
    places_of(pos + t * topk + jb, topk - jb, S, status, p);
    for (int64_t i = threadIdx.x; i < nv; i += blockDim.x * U) {
      P g[U], r[J][U];
      const P* from = reinterpret_cast<const P*>(dy + t * lddy) + i;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u == 0 || i + u * (int)blockDim.x < nv) g[u] = from[u * (int)blockDim.x];
      if (dw) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (p[j] < 0) continue;
          const P* row = reinterpret_cast<const P*>(ys + (int64_t)p[j] * ldys) + i;
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (u == 0 || i + u * (int)blockDim.x < nv) r[j][u] = row[u * (int)blockDim.x];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u > 0 && i + u * (int)blockDim.x >= nv) break;
        float gf[V];
        unpack(g[u], gf);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (p[j] < 0) continue;
          float v[V];
          if (dw) {
            unpack(r[j][u], v);
#pragma unroll
            for (int k = 0; k < V; ++k) dot[j] = fmaf(gf[k], v[k], dot[j]);
          }
          if (dys) {
            P out;
#pragma unroll
            for (int k = 0; k < V; ++k) v[k] = wj[j] * gf[k];
            pack(v, out);
            reinterpret_cast<P*>(dys + (int64_t)p[j] * lddys)[i + u * (int)blockDim.x] = out;
          }
        }
      }
    }
    if (dw) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        if (lane == 0) red[j][warp] = dot[j];
      }
      __syncthreads();
      if (threadIdx.x < J && jb + (int)threadIdx.x < topk) {
        float s = 0.0f;
        for (int k = 0; k < nw; ++k) s += red[threadIdx.x][k];
        dw[t * topk + jb + threadIdx.x] = s;  // 0 for an entry without an expert
      }
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
// Programmatic dependents of the work before them: they may become resident
// while it drains and wait for it on the device.
template <typename F, typename... A>
int launch_pdl(F kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

int elem_bytes(int dtype) {
  return dtype == QG_F32 ? 4 : (dtype == QG_BF16 || dtype == QG_F16) ? 2 : 0;
}

bool all_aligned(uintptr_t bits, int a) { return (bits & (uintptr_t)(a - 1)) == 0; }

// Threads of a row of nv accesses: enough to cover it, at most `most`.
int row_threads(int64_t nv, int most) {
  return (int)min64(most, max64(32, round_up(nv, 32)));
}

template <typename T, int V, int J>
int run_combine_as(int T_, int topk, int64_t S, int N, const void* ys, int64_t ldys,
                   const int32_t* pos, const float* w, void* y, int64_t ldy, cudaStream_t st) {
  constexpr int U = in_flight(V * (int)sizeof(T), J);
  const int64_t nv = N / V;
  const int th = row_threads(cdiv(nv, U), 256);
  // a few tokens: several CTAs share a token's row
  const int parts = (int)max64(1, min64(cdiv(nv, th * U), cdiv(2 * num_sms(), T_)));
  return launch_pdl(combine_rows_kernel<T, V, U, J>, dim3((unsigned)T_, (unsigned)parts), th, 0, st,
                    topk, S, nv, (const T*)ys, ldys, pos, w, (T*)y, ldy, status_word());
}

template <typename T, int V, int J>
int run_combine_grad_as(int T_, int topk, int64_t S, int N, const void* dy, int64_t lddy,
                        const void* ys, int64_t ldys, const int32_t* pos, const float* w, void* dys,
                        int64_t lddys, float* dw, cudaStream_t st) {
  constexpr int U = in_flight(V * (int)sizeof(T), J);
  const int64_t nv = N / V;
  const int th = row_threads(cdiv(nv, U), T_ >= 8 * num_sms() ? 128 : 512);
  return launch_pdl(combine_grad_kernel<T, V, U, J>, dim3((unsigned)T_), th, 0, st, topk, S, nv,
                    (const T*)dy, lddy, (const T*)ys, ldys, pos, w, (T*)dys, lddys, dw,
                    status_word());
}

// go(V, J), both as types, for `vec` values per access and the experts per
// step.  4096 tokens of 4096 bf16: topk 4 summed 8 at a time 41.6 us, 4 at a
// time 32.6; topk 2 36.5 and, 2 at a time, 18.4 (rows of 4091: 68 and 46).
// With few tokens and narrow accesses a thread with 8 to 16 of them only lasts
// longer than several threads with 4 (1 token, 2 x 2001: 2.2 and 1.7 us).
template <typename T, typename F>
int by_shape(int vec, int T_, int topk, F go) {
  constexpr int B = (int)sizeof(T);
  if (T_ < num_sms() && vec * B < 16) topk = 8;
  auto with = [&](auto v) {
    if (topk <= 2) return go(v, std::integral_constant<int, 2>());
    if (topk <= 4) return go(v, std::integral_constant<int, 4>());
    return go(v, std::integral_constant<int, 8>());
  };
  if (vec * B == 16) return with(std::integral_constant<int, 16 / B>());
  if (vec * B == 8) return with(std::integral_constant<int, 8 / B>());
  if (vec * B == 4) return with(std::integral_constant<int, 4 / B>());
  return with(std::integral_constant<int, 1>());
}

template <typename T>
int run_combine(int vec, int T_, int topk, int64_t S, int N, const void* ys, int64_t ldys,
                const int32_t* pos, const float* w, void* y, int64_t ldy, cudaStream_t st) {
  return by_shape<T>(vec, T_, topk, [&](auto v, auto j) {
    return run_combine_as<T, decltype(v)::value, decltype(j)::value>(T_, topk, S, N, ys, ldys, pos, w,
                                                                     y, ldy, st);
  });
}

template <typename T>
int run_combine_grad(int vec, int T_, int topk, int64_t S, int N, const void* dy, int64_t lddy,
                     const void* ys, int64_t ldys, const int32_t* pos, const float* w, void* dys,
                     int64_t lddys, float* dw, cudaStream_t st) {
  return by_shape<T>(vec, T_, topk, [&](auto v, auto j) {
    return run_combine_grad_as<T, decltype(v)::value, decltype(j)::value>(
        T_, topk, S, N, dy, lddy, ys, ldys, pos, w, dys, lddys, dw, st);
  });
}

// Values per access that every pointer, stride and the row length allow.
int vector_of(int esz, uintptr_t bits) {
  for (int b = 16; b > esz; b /= 2)
    if (all_aligned(bits, b)) return b / esz;
  return 1;
}

// Sizes common to the row entry points: QG_OK, or what the call returns.
int row_args(int T, int topk, int S, int N, int dtype) {
  if (T < 0 || topk <= 0 || S < 0 || N <= 0) return QG_ERR_INVALID_ARG;
  if (!elem_bytes(dtype)) return QG_ERR_INVALID_ARG;
  if ((int64_t)T * topk > INT32_MAX) return QG_ERR_UNSUPPORTED;
  return QG_OK;
}

}  // namespace

int expert_rows_setup() {
  const int most = (kSortOneWarps * kSortMaxE + kSortMaxE + 1) * 4;
  return cudaFuncSetAttribute((const void*)sort_place_kernel,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              most) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

}  // namespace qg

using namespace qg;

// ---------------------------------------------------------------------------
// Entry points
// ---------------------------------------------------------------------------
extern "C" size_t qg_sort_by_expert_workspace_bytes(int T, int topk, int E) {
  if (T <= 0 || topk <= 0 || E <= 0 || E > kSortMaxE) return 0;
  const int64_t n = (int64_t)T * topk;
  if (n > kSortMax || n <= kSortOneMax) return 0;
  return (size_t)(cdiv(n, sort_chunk(n)) * E * 4);
}

extern "C" int qg_sort_by_expert(int T, int topk, int E, const int32_t* ids, int64_t ld_ids,
                                 int32_t* offsets, int32_t* src, int32_t* pos, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (T < 0 || topk <= 0 || E <= 0 || ld_ids < topk) return QG_ERR_INVALID_ARG;
  if (E > kSortMaxE || (int64_t)T * topk > kSortMax) return QG_ERR_UNSUPPORTED;
  if (!offsets || (T > 0 && (!ids || !src || !pos))) return QG_ERR_INVALID_ARG;
  if (((uintptr_t)ids | (uintptr_t)offsets | (uintptr_t)src | (uintptr_t)pos) & 3)
    return QG_ERR_MISALIGNED;
  const size_t need = qg_sort_by_expert_workspace_bytes(T, topk, E);
  if (need && (!workspace || workspace_bytes < need)) return QG_ERR_WORKSPACE;
  if (need && ((uintptr_t)workspace & 3)) return QG_ERR_MISALIGNED;
  const int rc = device_setup_status();
  if (rc != QG_OK) return rc;
  cudaStream_t st = (cudaStream_t)stream;
  const int64_t n = (int64_t)T * topk;
  if (!need) {
    // one CTA; fewer warps for few entries (each costs E counters to clear)
    const int warps = (int)min64(kSortOneWarps, max64(8, cdiv(n, 64)));
    return launch_pdl(sort_place_kernel, dim3(1), warps * 32,
                      (size_t)(warps * E + E + 1) * 4, st, n, topk, E, ids, ld_ids,
                      (const int32_t*)nullptr, n, offsets, src, pos);
  }
  const int64_t per_cta = sort_chunk(n);
  const unsigned chunks = (unsigned)cdiv(n, per_cta);
  const int rc2 = launch_pdl(sort_count_kernel, dim3(chunks), kSortWarps * 32, (size_t)E * 4, st,
                             n, topk, E, ids, ld_ids, per_cta, (int32_t*)workspace);
  if (rc2 != QG_OK) return rc2;
  return launch_pdl(sort_place_kernel, dim3(chunks), kSortWarps * 32,
                    (size_t)(kSortWarps * E + E + 1) * 4, st, n, topk, E, ids, ld_ids,
                    (const int32_t*)workspace, per_cta, offsets, src, pos);
}

extern "C" int qg_spread_rows(int T, int topk, int S, int N, int dtype, const void* x,
                              int64_t ldx, const int32_t* pos, void* xs, int64_t ldxs,
                              void* stream) {
  int rc = row_args(T, topk, S, N, dtype);
  if (rc != QG_OK) return rc;
  if (ldx < N || ldxs < N) return QG_ERR_INVALID_ARG;
  if (T == 0 || S == 0) return QG_OK;
  if (!x || !pos || !xs) return QG_ERR_INVALID_ARG;
  const int esz = elem_bytes(dtype);
  if (((uintptr_t)x | (uintptr_t)xs) % esz || ((uintptr_t)pos & 3)) return QG_ERR_MISALIGNED;
  rc = device_setup_status();
  if (rc != QG_OK) return rc;
  const int64_t rb = (int64_t)N * esz, xb = ldx * esz, sb = ldxs * esz;
  const uintptr_t bits = (uintptr_t)x | (uintptr_t)xs | (uintptr_t)rb | (uintptr_t)xb | (uintptr_t)sb;
  cudaStream_t st = (cudaStream_t)stream;
  auto go = [&](auto word, auto j) {
    using W = decltype(word);
    constexpr int J = decltype(j)::value, U = sizeof(W) == 16 && J == 8 ? 2 : 4;
    const int64_t nv = rb / (int64_t)sizeof(W);
    const int th = row_threads(cdiv(nv, U), 256);
    // a few tokens: several CTAs share a token's row
    const int parts = (int)max64(1, min64(cdiv(nv, U * th), cdiv(2 * num_sms(), T)));
    return launch_pdl(spread_rows_kernel<W, U, J>, dim3((unsigned)T, (unsigned)parts), th, 0, st, topk, (int64_t)S, nv,
                      (const W*)x, xb / (int64_t)sizeof(W), pos, (W*)xs, sb / (int64_t)sizeof(W),
                      status_word());
  };
  auto with = [&](auto word) {
    return topk <= 4 && T >= num_sms() ? go(word, std::integral_constant<int, 4>())
                     : go(word, std::integral_constant<int, 8>());
  };
  if (all_aligned(bits, 16)) return with(uint4());
  if (all_aligned(bits, 8)) return with(uint2());
  if (all_aligned(bits, 4)) return with(uint32_t());
  return with(uint16_t());
}

extern "C" int qg_combine_rows(int T, int topk, int S, int N, int dtype, const void* ys,
                               int64_t ldys, const int32_t* pos, const float* weights, void* y,
                               int64_t ldy, void* stream) {
  int rc = row_args(T, topk, S, N, dtype);
  if (rc != QG_OK) return rc;
  if (ldys < N || ldy < N) return QG_ERR_INVALID_ARG;
  if (T == 0) return QG_OK;
  if (!pos || !y || (S > 0 && !ys)) return QG_ERR_INVALID_ARG;
  const int esz = elem_bytes(dtype);
  if (((uintptr_t)ys | (uintptr_t)y) % esz || (((uintptr_t)pos | (uintptr_t)weights) & 3))
    return QG_ERR_MISALIGNED;
  rc = device_setup_status();
  if (rc != QG_OK) return rc;
  const uintptr_t bits = (uintptr_t)ys | (uintptr_t)y | (uintptr_t)((int64_t)N * esz) |
                         (uintptr_t)(ldys * esz) | (uintptr_t)(ldy * esz);
  const int vec = vector_of(esz, bits);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == QG_F32)
    return run_combine<float>(vec, T, topk, S, N, ys, ldys, pos, weights, y, ldy, st);
  if (dtype == QG_F16)
    return run_combine<__half>(vec, T, topk, S, N, ys, ldys, pos, weights, y, ldy, st);
  return run_combine<__nv_bfloat16>(vec, T, topk, S, N, ys, ldys, pos, weights, y, ldy, st);
}

extern "C" int qg_combine_rows_grad(int T, int topk, int S, int N, int dtype, const void* dy,
                                    int64_t lddy, const void* ys, int64_t ldys,
                                    const int32_t* pos, const float* weights, void* dys,
                                    int64_t lddys, float* dw, void* stream) {
  int rc = row_args(T, topk, S, N, dtype);
  if (rc != QG_OK) return rc;
  if (lddy < N || (dw && ldys < N) || (dys && lddys < N)) return QG_ERR_INVALID_ARG;
  if (!dys && !dw) return QG_ERR_INVALID_ARG;
  if (T == 0) return QG_OK;
  if (!dy || !pos || (dw && S > 0 && !ys)) return QG_ERR_INVALID_ARG;
  const int esz = elem_bytes(dtype);
  if (((uintptr_t)dy | (uintptr_t)(dw ? ys : nullptr) | (uintptr_t)dys) % esz ||
      (((uintptr_t)pos | (uintptr_t)weights | (uintptr_t)dw) & 3))
    return QG_ERR_MISALIGNED;
  rc = device_setup_status();
  if (rc != QG_OK) return rc;
  uintptr_t bits = (uintptr_t)dy | (uintptr_t)((int64_t)N * esz) | (uintptr_t)(lddy * esz);
  if (dw) bits |= (uintptr_t)ys | (uintptr_t)(ldys * esz);
  if (dys) bits |= (uintptr_t)dys | (uintptr_t)(lddys * esz);
  const int vec = vector_of(esz, bits);
  cudaStream_t st = (cudaStream_t)stream;
  if (dtype == QG_F32)
    return run_combine_grad<float>(vec, T, topk, S, N, dy, lddy, ys, ldys, pos, weights, dys,
                                   lddys, dw, st);
  if (dtype == QG_F16)
    return run_combine_grad<__half>(vec, T, topk, S, N, dy, lddy, ys, ldys, pos, weights, dys,
                                    lddys, dw, st);
  return run_combine_grad<__nv_bfloat16>(vec, T, topk, S, N, dy, lddy, ys, ldys, pos, weights,
                                         dys, lddys, dw, st);
}
