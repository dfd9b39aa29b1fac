// Fifth-generation tensor core products and tensor memory: descriptors, issue, loads and stores, and the
// bounded waits of the kernels that use them.
#pragma once

#include "sv_common.cuh"

namespace sv {
namespace tmem {

constexpr int kColumns = 512;              // tensor memory columns: a CTA of these kernels takes all

// Descriptor of a matrix in shared memory whose rows of 128 bytes are swizzled, in two words; an offset of
// n bytes adds n / 16 to the low one. Rows along the result: `stride` is the distance of eight rows. Rows
// along the contraction: `lead` is the distance of 64 columns.
struct Matrix {
  uint32_t lo, hi;
  __device__ __forceinline__ Matrix at(uint32_t bytes) const { return {lo + (bytes >> 4), hi}; }
};
__device__ __forceinline__ Matrix matrix(uint32_t addr, uint32_t lead, uint32_t stride) {
  return {((addr & 0x3ffffu) >> 4) | ((lead >> 4) << 16), (stride >> 4) | (1u << 14) | (2u << 29)};
}

// fp32 accumulators, operands of one 16-bit type; M = 128; b_rows: B's rows are its contraction index.
template <bool F16>
__device__ __forceinline__ constexpr uint32_t product_desc(int n, bool b_rows) {
  return (1u << 4) | (F16 ? 0u : (1u << 7) | (1u << 10)) | (b_rows ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | ((128 >> 4) << 24);
}

__device__ __forceinline__ void product_ss(uint32_t d, Matrix a, Matrix b, uint32_t desc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}"
      ::"r"(d), "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(desc), "r"(add ? 1u : 0u) : "memory");
}
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, Matrix b, uint32_t desc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
      ::"r"(d), "r"(a), "r"(b.lo), "r"(b.hi), "r"(desc), "r"(add ? 1u : 0u) : "memory");
}
// The barrier gets an arrival when every product issued so far is done.
__device__ __forceinline__ void products_done(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define SV_R8(x, o) "=r"(x[o]), "=r"(x[o + 1]), "=r"(x[o + 2]), "=r"(x[o + 3]), "=r"(x[o + 4]), "=r"(x[o + 5]), "=r"(x[o + 6]), "=r"(x[o + 7])
#define SV_W8(x, o) "r"(x[o]), "r"(x[o + 1]), "r"(x[o + 2]), "r"(x[o + 3]), "r"(x[o + 4]), "r"(x[o + 5]), "r"(x[o + 6]), "r"(x[o + 7])
// 16, 32 or 64 columns of this thread's lane of tensor memory, loaded when the call returns (the wait
// is part of the statement, so that no use of the registers can move before it).
__device__ __forceinline__ void tm_load64(uint32_t* r, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,"
      "%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SV_R8(r, 0), SV_R8(r, 8), SV_R8(r, 16), SV_R8(r, 24), SV_R8(r, 32), SV_R8(r, 40), SV_R8(r, 48), SV_R8(r, 56)
      : "r"(at) : "memory");
}
__device__ __forceinline__ void tm_load16(uint32_t* r, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SV_R8(r, 0), SV_R8(r, 8) : "r"(at) : "memory");
}
__device__ __forceinline__ void tm_store16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(at), SV_W8(r, 0), SV_W8(r, 8) : "memory");
}
__device__ __forceinline__ void tm_store32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(at), SV_W8(r, 0), SV_W8(r, 8), SV_W8(r, 16), SV_W8(r, 24) : "memory");
}
__device__ __forceinline__ void tm_load32(uint32_t* r, uint32_t at) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SV_R8(r, 0), SV_R8(r, 8), SV_R8(r, 16), SV_R8(r, 24) : "r"(at) : "memory");
}
template <int N>
__device__ __forceinline__ void tm_load(uint32_t* r, uint32_t at) {
  static_assert(N == 32 || N == 64, "columns");
  if (N == 32) tm_load32(r, at);
  else tm_load64(r, at);
}
template <int N>
__device__ __forceinline__ void tm_store(uint32_t at, const uint32_t* r) {
  static_assert(N == 16 || N == 32, "columns");
  if (N == 16) tm_store16(at, r);
  else tm_store32(at, r);
}
__device__ __forceinline__ void tm_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A bounded wait; the first that gives up makes every later one return at once.
__device__ __forceinline__ bool wait_unless_lost(uint32_t bar, uint32_t parity, volatile int* lost) {
  if (sv::mbar_try_wait(bar, parity)) return true;
  if (*lost) return false;
  if (sv::mbar_wait(bar, parity)) return true;
  *lost = 1;
  return false;
}

__device__ __forceinline__ void tm_alloc(uint32_t* at) {       // one full warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
               ::"r"(sv::smem_addr(at)), "r"(static_cast<uint32_t>(kColumns)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  fence_before();
}
__device__ __forceinline__ void tm_free(uint32_t tm) {         // the same warp
  fence_after();
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
               ::"r"(tm), "r"(static_cast<uint32_t>(kColumns)) : "memory");
}

}  // namespace tmem
}  // namespace sv
