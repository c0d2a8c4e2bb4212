// tensor_core.cuh — the PTX of sm_103a's fifth-generation tensor cores that the
// products of 4-bit operands use (gemm.cu): tensor memory, block-scaled
// tcgen05.mma, the bulk copies that feed them and the barriers between.
#pragma once

#include <cstdint>

namespace mxfp4 {
namespace tc {

__device__ __forceinline__ uint32_t shared_address(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// One thread of a converged warp; what it alone runs may use uniform registers,
// which the instructions below take their operands from.
__device__ __forceinline__ bool elected() {
  uint32_t yes = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 lane;\n\t"
      "elect.sync lane|p, 0xFFFFFFFF;\n\t"
      "@p mov.u32 %0, 1;\n\t}"
      : "+r"(yes));
  return yes != 0;
}

// ---------------------------------------------------------------- barriers
__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t arrivals) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(arrivals) : "memory");
}
__device__ __forceinline__ void barrier_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// A word of shared memory that says that a wait was given up.
__device__ __forceinline__ bool raised(uint32_t flag) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(flag) : "memory");
  return v != 0;
}
__device__ __forceinline__ void raise(uint32_t flag) {
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(flag), "r"(1) : "memory");
}
// The word of another CTA of the cluster.
__device__ __forceinline__ bool raised_there(uint32_t flag, uint32_t rank) {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.u32 %0, [a];\n\t}"
      : "=r"(v)
      : "r"(flag), "r"(rank)
      : "memory");
  return v != 0;
}
// Waits for the phase of `parity`; gives up after 2^32 cycles (about two seconds).
__device__ __forceinline__ bool barrier_wait_alone(uint32_t bar, uint32_t parity) {
  for (const long long start = clock64(); !barrier_try(bar, parity);)
    if (clock64() - start > (1ll << 32)) return false;
  return true;
}
// The same, and says so by `gave_up`; or when another thread has.
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity, uint32_t gave_up) {
  long long start = 0;
  for (uint32_t i = 0;; ++i) {
    if (barrier_try(bar, parity)) return true;
    if ((i & 63u) == 63u) {
      const long long now = clock64();
      if (i == 63u) start = now;
      if (raised(gave_up) || now - start > (1ll << 32)) break;
    }
  }
  raise(gave_up);
  return false;
}

// ------------------------------------------------------------------- copies
// A box of a tensor map's rows to shared memory; x in elements of the map.
__device__ __forceinline__ void copy_box(uint32_t dst, const void* map, int32_t x, int32_t y,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// Consecutive bytes (16-byte aligned, a multiple of 16).
__device__ __forceinline__ void copy_bytes(uint32_t dst, const void* src, uint32_t bytes,
                                           uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// What this thread wrote to shared memory is seen by copies and tensor cores.
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ----------------------------------------------------------- tensor memory
// A whole warp allocates, and frees, `columns` columns of 128 lanes by 32 bits.
__device__ __forceinline__ void allocate(uint32_t address_at, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(address_at),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void release(uint32_t address, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(address), "r"(columns) : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 32 columns from each of two on, of the warp's quarter of the lanes: a lane's 64 words.
// One statement with the wait, so that nothing uses a word before it has come (and the
// second address shares no register with the first words).
__device__ __forceinline__ void load_sums(uint32_t first, uint32_t second, float (&v)[64]) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]),
        "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]),
        "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]),
        "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]), "=&r"(r[28]), "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31]),
        "=&r"(r[32]), "=&r"(r[33]), "=&r"(r[34]), "=&r"(r[35]), "=&r"(r[36]), "=&r"(r[37]), "=&r"(r[38]), "=&r"(r[39]),
        "=&r"(r[40]), "=&r"(r[41]), "=&r"(r[42]), "=&r"(r[43]), "=&r"(r[44]), "=&r"(r[45]), "=&r"(r[46]), "=&r"(r[47]),
        "=&r"(r[48]), "=&r"(r[49]), "=&r"(r[50]), "=&r"(r[51]), "=&r"(r[52]), "=&r"(r[53]), "=&r"(r[54]), "=&r"(r[55]),
        "=&r"(r[56]), "=&r"(r[57]), "=&r"(r[58]), "=&r"(r[59]), "=&r"(r[60]), "=&r"(r[61]), "=&r"(r[62]), "=&r"(r[63])
      : "r"(first), "r"(second)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// ------------------------------------------------------------- descriptors
// The low words of shared memory descriptors, which step with the address (in
// units of 16 bytes), and the constant high words.
// Operands: rows of 128 bytes (256 E2M1 codes) as a copy with the 128-byte
// swizzle lays them, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint32_t operand_low(uint32_t address) { return (address >> 4) | (1u << 16); }
constexpr uint32_t kOperandHigh = 64u | (1u << 14) | (2u << 29);
// Scales: 512 bytes, 32 rows of 16, groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint32_t scales_low(uint32_t address) { return address >> 4; }
constexpr uint32_t kScalesHigh = 8u | (1u << 14);
__device__ __forceinline__ uint64_t descriptor(uint32_t low, uint32_t high) {
  return static_cast<uint64_t>(high) << 32 | low;
}
// E2M1 by E2M1 with float32 sums, both along K; M = 128, N columns; E8M0 or
// E4M3 scales.
__device__ __forceinline__ uint32_t instruction(uint32_t columns, bool e4m3) {
  return (1u << 7) | (1u << 10) | ((columns >> 3) << 17) | (e4m3 ? 0u : 1u << 23) | ((128u >> 4) << 24);
}
// ... with the scales that begin at byte `id` of their words.
__device__ __forceinline__ uint32_t with_scale_byte(uint32_t instruction, uint32_t id) {
  return instruction | (id << 4) | (id << 29);
}

// 128 rows' scales (512 bytes) to four columns of all four lane quarters.
__device__ __forceinline__ void copy_scales(uint32_t address, uint64_t from) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(address), "l"(from) : "memory");
}
// 64 elements of K.  One thread issues these and copy_scales; they take effect
// in its order.
template <bool kE4m3>
__device__ __forceinline__ void multiply(uint32_t sums, uint64_t a, uint64_t b, uint32_t instruction,
                                         uint32_t a_scales, uint32_t b_scales, bool add) {
  if constexpr (kE4m3)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(sums), "l"(a), "l"(b), "r"(instruction),
        "r"(a_scales), "r"(b_scales), "r"(static_cast<uint32_t>(add))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(sums), "l"(a), "l"(b), "r"(instruction),
        "r"(a_scales), "r"(b_scales), "r"(static_cast<uint32_t>(add))
        : "memory");
}
// Arrives at `bar` when all that this thread issued before has been done.
__device__ __forceinline__ void arrive_when_done(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

}  // namespace tc
}  // namespace mxfp4
