// bl_sm100.cuh -- mbarrier, TMA and bulk-copy helpers for sm_100a kernels.
// Every wait here is bounded: callers pass an SM-cycle limit and get false
// back when it runs out (or when another role of the CTA has given up).
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace bl {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---- mbarrier ----------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Single-thread bounded wait.  False if the limit ran out or another role aborted.
__device__ __forceinline__ bool wait1(uint64_t* bar, uint32_t parity, long long limit,
                                      volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > limit) return false;
  }
}

// Bounded wait that ignores the abort flag (used to drain work already issued).
__device__ __forceinline__ bool wait_drain(uint64_t* bar, uint32_t parity, long long limit) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > limit) return false;
  return true;
}

// Warp-uniform bounded wait: every lane returns the same answer.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, long long limit,
                                          volatile int* abort_flag) {
  const long long t0 = clock64();
  for (;;) {
    const bool done = mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    const bool give_up = (*abort_flag != 0) || (clock64() - t0 > limit);
    if (__any_sync(0xffffffffu, give_up)) return false;
  }
}

// ---- TMA --------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// TMA tensor store (shared -> global), tracked by the issuing thread's bulk
// group; the coordinates must be non-negative, the inner one x element size a
// multiple of 16 bytes
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// ---- clusters -----------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// shared::cluster address of the same shared variable in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t mapa_shared(uint32_t local_addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local_addr), "r"(rank));
  return r;
}
// arrive (count 1) on an mbarrier given by its shared::cluster address (the
// writer's shared-memory results were made visible to the tensor cores with
// fence.proxy.async before the arrive)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// TMA load whose completion is counted on an mbarrier of either CTA of the pair
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar_cluster_addr,
                                                 int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster_addr), "r"(c0), "r"(c1)
      : "memory");
}

// ---- tcgen05 --------------------------------------------------------------------
// arrive on the barrier at this offset in each CTA of `mask` when the MMAs issued
// so far complete
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 16 two-bit digits (q + 1) -> 16 signed int8 weights q, in K order.  The
// digits are spread into nibbles, which select bytes of 0x000100FF
// (digit 0 -> 0xFF = -1, 1 -> 0, 2 -> +1, 3 -> 0).
__device__ __forceinline__ uint32_t spread8(uint32_t h) {  // 8 digits in bits 0..15 -> 8 nibbles
  uint32_t x = h & 0xffffu;
  x = (x | (x << 8)) & 0x00ff00ffu;
  x = (x | (x << 4)) & 0x0f0f0f0fu;
  x = (x | (x << 2)) & 0x33333333u;
  return x;
}
__device__ __forceinline__ uint4 expand16(uint32_t w) {
  const uint32_t lo = spread8(w), hi = spread8(w >> 16);
  uint4 o;
  o.x = __byte_perm(0x000100ffu, 0u, lo & 0xffffu);
  o.y = __byte_perm(0x000100ffu, 0u, lo >> 16);
  o.z = __byte_perm(0x000100ffu, 0u, hi & 0xffffu);
  o.w = __byte_perm(0x000100ffu, 0u, hi >> 16);
  return o;
}

// 16 bits -> 16 int8 in {-1, 1}: four bits at a time to the low bits of four bytes
__device__ __forceinline__ uint4 expand16_bits(uint32_t h) {
  auto four = [](uint32_t b) { return ~(((b & 0xfu) * 0x00204081u & 0x01010101u) * 0xfeu); };
  return make_uint4(four(h), four(h >> 4), four(h >> 8), four(h >> 12));
}

// A base-3 segment (16 bytes, 80 weights) as five words of 2-bit codes (a base-3
// digit is the 2-bit code of the same weight).  With q_i = floor(b / 3^i) the
// digits of a byte b are d_i = q_i - 3 q_{i+1}, so its ten bits are sum d_i 4^i =
// b + q_1 + 4 q_2 + 16 q_3 + 64 q_4.  floor(x / 3) = floor(85 (x + 1) / 256) for x
// <= 255 (85 / 256 is 1/3 - 1/768: x = 3 k gives k + 1/3 - (3 k + 1) / 768 >= k, x =
// 3 k + 2 less than k + 1), two bytes at a time in the 16-bit halves of a register:
// a multiply-add, and one byte permute that takes the quotients from the halves'
// upper bytes.  The integer ALU bounds its caller's kernel on large matrices (28672
// x 8192), so shifts and masks are left to permutes and multiply-adds.
__device__ __forceinline__ uint32_t t5_pair(uint32_t x) {  // two bytes at bits 0 and 16 -> two 10-bit fields there
  const uint32_t over = __byte_perm(x + 0x000d000du, 0u, 0x4341) * 0xffu;  // bytes 243..255: five weight-0 digits (121)
  x = (x & ~over) | (0x00790079u & over);
  auto third = [](uint32_t v) { return __byte_perm(v * 85u + 0x00550055u, 0u, 0x4341); };
  const uint32_t q1 = third(x), q2 = third(q1), q3 = third(q2), q4 = third(q3);
  return x + q1 + 4u * q2 + 16u * q3 + 64u * q4;
}
__device__ __forceinline__ void t5_segment(const uint4& v, uint32_t* out) {
  const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
  uint32_t lo[4], hi[4];  // 40 bits of each packed word: 32 and 8
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // bytes 0, 2 and 1, 3: the upper field moves from bit 16 to bit 20
    const uint32_t a = t5_pair(__byte_perm(wd[i], 0u, 0x4240)), c = t5_pair(__byte_perm(wd[i], 0u, 0x4341));
    lo[i] = a + (a >> 16) * 0xf0000u + (c + (c >> 16) * 0xf0000u) * 1024u;
    hi[i] = c >> 18;
  }
  out[0] = lo[0];
  out[1] = __byte_perm(hi[0], lo[1], 0x6540);
  out[2] = __byte_perm(__byte_perm(lo[1], hi[1], 0x0043), lo[2], 0x5410);
  out[3] = __byte_perm(__byte_perm(lo[2], hi[2], 0x0432), lo[3], 0x4210);
  out[4] = __byte_perm(lo[3], hi[3], 0x4321);
}

// ---- bulk copies (no tensor map) and bulk-group waits --------------------------------
// global -> shared, completion counted on an mbarrier (size: a multiple of 16 B,
// both addresses 16-byte aligned)
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// wait until the sources of all but the newest N committed groups have been read
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void fence_proxy_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

}  // namespace bl
