// The weight-only int4 products (bf16 rows): what their kernels share, and
// the inline-PTX wrappers of the tensor-core one.
#pragma once

#include "qg_internal.cuh"

namespace qg {

// ---------------------------------------------------------------------------
// One call of the weight-only products (bf16 rows x int4 weights), dense
// (offsets NULL: E = 1, every row is expert 0's) or per expert.  Forward:
// in [rows][K], out [S][N]; gradient with respect to x: in [S][N], out [S][K].
// ---------------------------------------------------------------------------
struct A16W4Call {
  int E, S, N, K;
  const uint16_t* in;      // bf16
  int64_t ld_in;
  int in_rows;             // rows of `in` (src reaches no further)
  const int32_t* src;      // sorted row p reads input row src[p] / topk; NULL: row p
  int topk;
  const int32_t* offsets;  // [E + 1] or NULL
  const uint8_t* packed;
  int64_t expert_bytes;    // from one expert's packed matrix to the next
  int format;              // QG_W4_*
  const float* bias;       // [E][N] or NULL
  uint16_t* out;           // bf16
  int64_t ld_out;
};
constexpr int kA16W4MaxExperts = 1024;
constexpr int kStallA16W4TC = 3;  // the kernel for many rows, beside StallTarget's
constexpr int kA16W4MaxSide = 1 << 24;  // N and K, either of which is a reduction
int launch_a16w4_rows(const A16W4Call& c, cudaStream_t st);           // few rows (a16w4.cu)
// many rows (a16w4_tc.cu); indirect rows need a workspace to be sorted in
int launch_a16w4_tc(const A16W4Call& c, bool grad, void* ws, cudaStream_t st);
size_t a16w4_tc_workspace(int S, int K, bool gather);

// Rows [start, start + count) of expert e; a range that is not inside [0, S)
// is an error of the caller's: recorded, then no rows.
__device__ __forceinline__ int2 expert_range(const int32_t* offsets, int e, int S, int* status) {
  if (!offsets) return make_int2(0, S);
  const int a = offsets[e], b = offsets[e + 1];
  if (a < 0 || b < a || b > S) {
    record_error(status, QG_ERR_INVALID_ARG);
    return make_int2(0, 0);
  }
  return make_int2(a, b - a);
}

// ---------------------------------------------------------------------------
// PTX wrappers
// ---------------------------------------------------------------------------

// Shared-memory descriptor of a K-major operand in 128-byte swizzled rows.
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;            // leading byte offset (unused with 128B swizzle)
  d |= (uint64_t)(1024 >> 4) << 32;  // stride byte offset between 8-row groups
  d |= (uint64_t)1 << 46;            // descriptor version
  d |= (uint64_t)2 << 61;            // SWIZZLE_128B
  return d;
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
constexpr uintptr_t kMaxPrefetch = 1u << 26;  // more would only displace itself
// L2 prefetch of the 16-byte-aligned interior of [p, p + bytes).
__device__ __forceinline__ void prefetch_l2(const void* p, int64_t bytes) {
  const uintptr_t b = ((uintptr_t)p + 15) & ~(uintptr_t)15;
  const uintptr_t e = ((uintptr_t)p + (uintptr_t)bytes) & ~(uintptr_t)15;
  if (e > b) bulk_prefetch_l2((const void*)b, (uint32_t)(e - b < kMaxPrefetch ? e - b : kMaxPrefetch));
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
// bf16x2 (0x4300 | u) - 136 = u - 8, exact.
__device__ __forceinline__ uint32_t bf16x2_minus136(uint32_t v) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x43084308u));
  return d;
}
// Wait for phase `parity` of `bar` with mbarrier.try_wait and a suspend-time
// hint: the hardware parks the thread until the phase completes (or the
// 20 us hint runs out, after which it asks again), so a waiting warp takes no
// issue slots from the other warps on its sub-partition.  At most
// limit / 256 + 1 tries: about 82 ms at kSpinLimit.
__device__ __forceinline__ bool mbar_park(uint64_t* bar, uint32_t parity, int* status,
                                          uint32_t limit = kSpinLimit) {
  const uint32_t tries = (limit >> 8) + 1;
  for (uint32_t i = 0; i < tries; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
  }
  record_error(status, QG_ERR_TIMEOUT);
  return false;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t mapa(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}

}  // namespace qg
