// Inline-PTX wrappers for the sm_103a pipeline pieces: mbarriers with bounded
// waits, 1-D bulk copies (global -> shared, mbarrier completion), tcgen05
// tensor-memory allocation, loads/stores, MMA issue and commit.
#pragma once

#include <stdint.h>

// Upper bound (ns) a waiting thread lets the hardware suspend it per try_wait.
#ifndef CSA2_WAIT_SLEEP_NS
#define CSA2_WAIT_SLEEP_NS 20000u
#endif

namespace csa2 {
namespace ptx {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// ------------------------------------------------------------------ mbarrier
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}
__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}
// kCluster: what threads of the cluster's other CTAs released at cluster scope is seen too.
#define CSA2_TRY_WAIT(SCOPE)                                                                   \
  asm volatile(                                                                                \
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire." SCOPE                          \
      ".shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"                            \
      : "=r"(ok)                                                                               \
      : "r"(smem_u32(bar)), "r"(parity)                                                        \
      : "memory")
#define CSA2_TRY_WAIT_NS(SCOPE)                                                                \
  asm volatile(                                                                                \
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire." SCOPE                          \
      ".shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"                        \
      : "=r"(ok)                                                                               \
      : "r"(smem_u32(bar)), "r"(parity), "r"(ns)                                               \
      : "memory")
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (kCluster) CSA2_TRY_WAIT("cluster");
  else CSA2_TRY_WAIT("cta");
  return ok != 0;
}

// try_wait that lets the hardware suspend the thread for up to `ns` nanoseconds
// (or until the phase completes) instead of returning at once, so waiting warps
// do not spend issue slots polling.
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_try_wait_sleep(uint64_t* bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  if constexpr (kCluster) CSA2_TRY_WAIT_NS("cluster");
  else CSA2_TRY_WAIT_NS("cta");
  return ok != 0;
}
#undef CSA2_TRY_WAIT
#undef CSA2_TRY_WAIT_NS

// Waits for the phase of `parity` to complete.  Gives up (returns false) when
// *abort becomes nonzero or after `budget` clock cycles.
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          long long budget) {
  if (mbar_try_wait<kCluster>(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
#if CSA2_WAIT_SLEEP_NS > 0
    if (mbar_try_wait_sleep<kCluster>(bar, parity, CSA2_WAIT_SLEEP_NS)) return true;
#else
    if (mbar_try_wait<kCluster>(bar, parity)) return true;
#endif
    if (*abort) return false;
    if (clock64() - t0 > budget) return false;
  }
}

// Warp-uniform form for warps that go on to issue .sync.aligned instructions:
// every lane waits, and the warp gives up together if any lane gave up.
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort,
                                               long long budget) {
  const bool ok = mbar_wait<kCluster>(bar, parity, abort, budget);
  return __all_sync(0xffffffffu, ok);
}

// ------------------------------------------------------------------ bulk copy
// global -> shared (this CTA), completion counted in bytes on `bar`.
// Both addresses 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_g2s(void* dst_smem, const void* src_gmem, uint32_t bytes,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst_smem)),
      "l"(src_gmem), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// 2-D tensor tile load (TMA) global -> shared, completion counted on `bar`.
// `map` is the address of a __grid_constant__ CUtensorMap kernel parameter.
__device__ __forceinline__ void tma_load_2d(void* dst_smem, const void* map, int c0, int c1,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(smem_u32(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// L2 policy for data read once: first in line for eviction, so that it does
// not push out what later kernels read back
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}
// bulk_g2s / tma_load_2d with an L2 cache policy
__device__ __forceinline__ void bulk_g2s_hint(void* dst_smem, const void* src_gmem, uint32_t bytes,
                                              uint64_t* bar, uint64_t pol) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::
          "r"(smem_u32(dst_smem)),
      "l"(src_gmem), "r"(bytes), "r"(smem_u32(bar)), "l"(pol)
      : "memory");
}
__device__ __forceinline__ void tma_load_2d_hint(void* dst_smem, const void* map, int c0, int c1, uint64_t* bar,
                                                 uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
      "{%2, %3}], [%4], %5;" ::"r"(smem_u32(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar)), "l"(pol)
      : "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Waits until the grids this one depends on (programmatic dependent launch)
// have completed and their memory is visible; a no-op without such a launch.
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the grid that depends on this one (programmatic dependent launch) be scheduled once every CTA has
// called this or left; what this grid writes is still seen only after its completion (griddep_wait).
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// 2^x by the hardware approximation (ex2.approx: relative error about 2^-22;
// 2^-inf = 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ------------------------------------------------------------------ tcgen05
__device__ __forceinline__ void tmem_alloc(uint32_t* slot_smem, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(slot_smem)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 32 lanes x 32 columns (this warp's lane quarter): thread i <-> lane i
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]),
      "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]),
      "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// 16 lanes x 32 columns twice: threads 0-15 <-> lanes 0-15 at columns taddr ..,
// threads 16-31 <-> the same lanes at columns taddr + kSplit .. (the rows of an
// M = 64 accumulator lie in lanes 0-15 of each quarter)
template <int kSplit>
__device__ __forceinline__ void tmem_ld_16x32bx2_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32], %33;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr), "n"(kSplit)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// D[tmem] (+)= A[smem desc] * B[smem desc]^T, kind::f16, issued by one thread.
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same MMA issued from a whole warp in uniform control flow: every lane
// executes the instruction stream and elect.sync picks the one lane (always the
// same: the lowest) that issues.  A warp that branches to lane 0 for the issue
// loses most of its issue slots to busy warps on the same scheduler (measured
// on sm_103a: M128 N64 K16 every ~150 cycles with one ALU-bound neighbour
// warp, against ~61 in this form).
__device__ __forceinline__ void mma_f16_ss_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kN (2, 4 or 8) MMAs of one accumulator, operands kA and kB descriptor units (16 bytes) apart, issued by the
// lane one elect.sync picks: next to busy warps every instruction of the issuing warp counts (32 S MMAs of
// M = N = 64, 1,024 cycles by themselves, took 2,300 issued one by one; in runs the paged attention of 48
// queries of up to 65,536 entries fell from 234 to 221 us).  The low words of the descriptors hold the addresses.
#define CSA2_MMA_FIRST(G)                                                                         \
  "{\n\t.reg .pred p, e, t;\n\t.reg .b32 r, a, b;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %6, 0;\n\t" \
  "setp.eq.b32 t, 0, 0;\n\telect.sync r|e, 0xffffffff;\n\t"                                       \
  "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"                                            \
  "@e tcgen05.mma.cta_group::" G ".kind::f16 [%0], da, db, %5, p;\n\t"
#define CSA2_MMA_NEXT(G, I)                                                                       \
  "add.u32 a, %1, " I " * %7;\n\tadd.u32 b, %3, " I " * %8;\n\t"                                    \
  "mov.b64 da, {a, %2};\n\tmov.b64 db, {b, %4};\n\t"                                              \
  "@e tcgen05.mma.cta_group::" G ".kind::f16 [%0], da, db, %5, t;\n\t"
#define CSA2_MMA_RUN(G)                                                                           \
  do {                                                                                            \
    const uint32_t al = (uint32_t)a_desc, ah = (uint32_t)(a_desc >> 32);                          \
    const uint32_t bl = (uint32_t)b_desc, bh = (uint32_t)(b_desc >> 32);                          \
    if constexpr (kN == 2)                                                                        \
      asm volatile(CSA2_MMA_FIRST(G) CSA2_MMA_NEXT(G, "1") "}" ::"r"(d_tmem), "r"(al), "r"(ah), "r"(bl), "r"(bh), \
                   "r"(idesc), "r"(accumulate), "n"(kA), "n"(kB)                                  \
                   : "memory");                                                                   \
    else if constexpr (kN == 4)                                                                   \
      asm volatile(CSA2_MMA_FIRST(G) CSA2_MMA_NEXT(G, "1") CSA2_MMA_NEXT(G, "2") CSA2_MMA_NEXT(G, "3") "}" ::"r"( \
                       d_tmem),                                                                   \
                   "r"(al), "r"(ah), "r"(bl), "r"(bh), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kB) \
                   : "memory");                                                                   \
    else                                                                                          \
      asm volatile(CSA2_MMA_FIRST(G) CSA2_MMA_NEXT(G, "1") CSA2_MMA_NEXT(G, "2") CSA2_MMA_NEXT(G, "3") \
                       CSA2_MMA_NEXT(G, "4") CSA2_MMA_NEXT(G, "5") CSA2_MMA_NEXT(G, "6") CSA2_MMA_NEXT(G, "7") "}" ::"r"( \
                           d_tmem),                                                               \
                   "r"(al), "r"(ah), "r"(bl), "r"(bh), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kB) \
                   : "memory");                                                                   \
  } while (0)
template <int kN, int kA, int kB>
__device__ __forceinline__ void mma_f16_ss_run_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                     uint32_t idesc, uint32_t accumulate) {
  static_assert(kN == 2 || kN == 4 || kN == 8, "MMAs of a run");
  CSA2_MMA_RUN("1");
}
// The same over a CTA pair, issued by the even CTA: each CTA's shared memory holds half of A's rows and half of
// B's rows (N) at the same offsets.  At M = 128 each CTA's tensor memory holds 64 rows of D: lanes 0-63 the
// columns of the even CTA's half of N, lanes 64-127 those of the odd's (checked against a CPU product on the
// GPU, B K-major and N-major, N = 64 .. 256).
template <int kN, int kA, int kB>
__device__ __forceinline__ void mma_f16_ss_pair_run_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                          uint32_t idesc, uint32_t accumulate) {
  static_assert(kN == 2 || kN == 4 || kN == 8, "MMAs of a run");
  CSA2_MMA_RUN("2");
}
#undef CSA2_MMA_FIRST
#undef CSA2_MMA_NEXT
#undef CSA2_MMA_RUN
// mma_f16_ts issued by the lane elect.sync picks (the warp runs the loop together)
__device__ __forceinline__ void mma_f16_ts_elect(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// tcgen05.commit from the lane elect.sync picks (the lane that issued the MMAs above)
__device__ __forceinline__ void mma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= (A[smem desc] * 2^sfA) * (B[smem desc] * 2^sfB)^T, block-scaled
// kind::mxf8f6f4 with one UE8M0 scale per row and per 32-element K step
// (scale_vec::1X), issued by one thread.  For an E2M1 A the shared-memory layout
// is the one the tensor-memory-access unit writes for its packed 4-bit type: 16
// codes (8 bytes, element 2i in the low nibble) per 16-byte slot.  Scale layouts
// in tensor memory (measured on sm_103a): the scale of A row m at lane m, column
// sfa + m/32, byte a_sf_id; the scale of B column n at lane 32 q + n%32 of every
// lane quarter q (replicated), column sfb + n/32, byte b_sf_id.
__device__ __forceinline__ void mma_mxf8f6f4_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], "
      "p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
      : "memory");
}

// mma_mxf8f6f4_ss issued by the lane elect.sync picks (the warp runs the loop together)
__device__ __forceinline__ void mma_mxf8f6f4_ss_elect(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                                      uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                                      uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b32 r;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "elect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], "
      "p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa_tmem), "r"(sfb_tmem), "r"(accumulate)
      : "memory");
}

// Copies a 32-row x 16-byte shared-memory matrix (descriptor `src`) into
// tensor memory at columns taddr..taddr+3 of all four lane quarters: lane
// 32 q + l, column taddr + j receives bytes 4j..4j+3 of row l.  Asynchronous,
// ordered with the MMAs the same thread issues afterwards.
__device__ __forceinline__ void tmem_cp_32x128b_warpx4(uint32_t taddr, uint64_t src) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(src) : "memory");
}

// tmem_cp_32x128b_warpx4 issued by the lane elect.sync picks
__device__ __forceinline__ void tmem_cp_32x128b_warpx4_elect(uint32_t taddr, uint64_t src) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
      "l"(src)
      : "memory");
}

// Element types of the block-scaled kinds (A/B format fields).
constexpr uint32_t kFmtE4M3 = 0, kFmtE2M1 = 5;

// Instruction descriptor of a block-scaled MMA with UE8M0 scales, both
// operands K-major, fp32 accumulate; sf ids pick the scale byte of A and B.
__host__ __device__ constexpr uint32_t idesc_block_scaled(uint32_t M, uint32_t N, uint32_t a_fmt,
                                                          uint32_t b_fmt, uint32_t a_sf_id,
                                                          uint32_t b_sf_id) {
  return (b_sf_id << 4) | (a_fmt << 7) | (b_fmt << 10) | ((N >> 3) << 17) | (1u << 23) |
         ((M >> 4) << 24) | (a_sf_id << 29);
}

// one 32-bit column of this warp's lane quarter: thread i <-> lane i
// 32 lanes x 8 columns (this warp's lane quarter): thread i <-> lane i
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Registers of this warpgroup's threads from here on; every warp of it calls it.  The increase waits for
// what other warpgroups of the CTA have given back, so the shares must not exceed the launch's total.
template <int kRegs>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// asks for the line of global memory that holds p
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}
__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p) : "memory");
}
// fetches a tensor map (a kernel parameter) ahead of its first copy
__device__ __forceinline__ void prefetch_tensormap(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ------------------------------------------------------- CTA pairs (clusters)
__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// a store to the same place of CTA `rank`'s shared memory (seen after the next cluster_sync)
__device__ __forceinline__ void st_cluster_f32(const float* p, uint32_t rank, float v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.f32 [a], %2;\n\t}" ::"r"(smem_u32(p)),
      "r"(rank), "f"(v)
      : "memory");
}
// every thread, but those that have left, of every CTA of the cluster; memory before it is seen after it
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// tma_load_2d into this CTA of a pair, whose bytes are counted by the barrier at the same offset of CTA `rank`.
__device__ __forceinline__ void tma_load_2d_pair(void* dst_smem, const void* map, int c0, int c1, uint64_t* bar,
                                                 uint32_t rank) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
      "%3}], [a];\n\t}" ::"r"(smem_u32(dst_smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar)), "r"(rank)
      : "memory");
}
// Arrives on the barrier at the same shared-memory offset of the cluster's CTA `rank`, whose waiter takes it with
// mbar_wait_warp<true>: what this thread has seen or written before is seen after the wait.  The release waits some
// 1,400 cycles, so a pair's barriers get few of these, from warps that have nothing else to do.
__device__ __forceinline__ void mbar_arrive_peer(uint64_t* bar, uint32_t rank) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar)),
      "r"(rank)
      : "memory");
}
// Tensor memory of a CTA pair: one warp of each CTA calls each of these.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot_smem, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot_smem)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
// Arrive on `bar` of both CTAs of the pair once the MMAs issued above have completed.
__device__ __forceinline__ void mma_commit_pair_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b32 r;\n\telect.sync r|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::
          "r"(smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// Arrive on `bar` once all previously issued tcgen05.mma of this thread completed.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
      : "memory");
}

// Shared-memory matrix descriptor, no swizzle, K-major: core matrices of 8 rows
// x 16 bytes stored as 128 contiguous bytes; `lbo` = byte step between core
// matrices along K, `sbo` = byte step between 8-row groups along M/N.
__device__ __forceinline__ uint64_t smem_desc_noswizzle(const void* base, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_u32(base) >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version for tcgen05
  return d;
}

// K-major operand in 128-byte swizzled rows (the layout a tensor load with
// 128-byte swizzle writes): row r at 128 r, its 16-byte slot c at c ^ (r % 8),
// 8-row groups `sbo` bytes apart; `base` must be 1024-byte aligned up to the
// K offset added for later K steps (0, 32, 64 or 96 bytes).
__device__ __forceinline__ uint64_t smem_desc_sw128(const void* base, uint32_t sbo) {
  uint64_t d = smem_desc_noswizzle(base, 16, sbo);
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}

// N-major (MN-major) operand in 128-byte swizzled rows: row k (one K index) at
// 128 k holds 64 consecutive N elements, 16-byte slot c at c ^ (k % 8); blocks
// of 64 N columns `lbo` bytes apart, 8-row K groups `sbo` bytes apart (checked
// against a CPU product on the GPU: lbo = N-block stride, sbo = K-group stride).
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(const void* base, uint32_t lbo, uint32_t sbo) {
  uint64_t d = smem_desc_noswizzle(base, lbo, sbo);
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}
constexpr uint32_t kIdescBMajorMN = 1u << 16;  // instruction descriptor: B operand N-major

// Instruction descriptor of kind::f16: fp32 accumulate, A/B type (0 = f16,
// 1 = bf16), both K-major, shape M x N.
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t M, uint32_t N, uint32_t ab_bf16) {
  return (1u << 4) | (ab_bf16 << 7) | (ab_bf16 << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

}  // namespace ptx
}  // namespace csa2
