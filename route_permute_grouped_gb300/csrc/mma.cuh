// Warp-level bf16 matrix products (mma.sync m16n8k16), their shared-memory
// loads (ldmatrix) and asynchronous 16-byte copies (cp.async), for products
// whose tiles are gathered row by row and whose time goes to memory.
#pragma once
#include "common.cuh"

namespace moe {

// 16 bytes global -> shared; zeros instead when !ok (nothing is read then)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// one of the barrier's expected arrivals, made when this thread's copies so far
// have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// four 8x8 matrices of 16-bit values; lane l gives the address of row l % 8 of
// matrix l / 8; register j holds, of matrix j, row lane / 4, columns
// 2 (lane % 4) and + 1 (transposed form: the same of its transpose)
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// d += a b: a 16x16 (rows lane / 4 and + 8, columns 2 (lane % 4) .. and + 8),
// b 16x8, d 16x8 fp32 (d[0], d[1]: row lane / 4, columns 2 (lane % 4) and + 1;
// d[2], d[3]: row + 8)
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// v = a + b + c in three bf16 parts: a alone is off by 2^-8 v at most, a + b by
// 2^-17 v, all three by 2^-25 v. b and c are 0 where a is not finite, so that an
// infinity stays one.
__device__ __forceinline__ void split_bf16(float v, __nv_bfloat16& a, __nv_bfloat16& b, __nv_bfloat16& c) {
  a = __float2bfloat16_rn(v);
  const float fa = __bfloat162float(a), rest = isfinite(fa) ? v - fa : 0.0f;
  b = __float2bfloat16_rn(rest);
  c = __float2bfloat16_rn(rest - __bfloat162float(b));
}

}  // namespace moe
