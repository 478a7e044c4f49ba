// seq_mma.cuh -- warp-level matrix products of the chunked sequence kernels at fp32 accuracy.
//
// A fp32 operand is split into bf16 terms, x = x0 + x1 + x2 (8 bits each, 24 together), and a
// product is the sum of the terms' products, fp32 accumulated: an exact bf16 operand (q, k, v, do)
// times a split one takes 3 products; two split ones take 6 (terms below 2^-24 are left out).  The leading
// product and the small ones have accumulators of their own: the tensor core truncates
// each addition at the accumulator's size, and the long chain of small terms would add its
// truncations at the large one's.
#pragma once

#include <cuda_bf16.h>

#include "sm100.cuh"

namespace gdn {
namespace mma {

using bf16 = __nv_bfloat16;

// Shared memory is addressed by 32-bit byte addresses: a lane's part of an address is worked out once and every
// fragment is that register and an immediate (address arithmetic between the products cost more than they did).
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint2 lds2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts(uint32_t addr, uint32_t x) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

// c[16 x 8] += a[16 x 16] b[16 x 8].  A result is ready about 21 clocks later and an SM quarter takes one in 8, so
// the callers put two products or more between two of one accumulator.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a b: `first` is known at compile time and saves the zeros.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool first) {
    if (first)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                     : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        mma(c, a, b0, b1);
}

// Lane parts of fragment addresses (bytes).
// A operand held [k][m] (m contiguous), for ldsm4_t.
__device__ __forceinline__ uint32_t at_lane(int pitch, int lane) {
    return (((lane >> 4) * 8 + (lane & 7)) * pitch + ((lane >> 3) & 1) * 8) * 2;
}
// Rows of 64 columns in the tensor maps' 128-byte swizzle: the 16-byte piece of (row, col) lies at piece
// (col / 8 % 8) ^ (row % 8) of its 128-byte line; slabs of 64 columns, `rows` lines each, follow one another.
__host__ __device__ constexpr uint32_t sw_byte(int rows, int row, int col) {
    return (col >> 6) * rows * 128 + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4);
}
// A operand of 16 rows held row-major in swizzled rows: lanes 0-15 give the rows of the left 8 columns of a 16 x 16
// tile, 16-31 those of the right 8; the tile at column 16 x (of 64).
__device__ __forceinline__ uint32_t a_lane(int x, int lane) { return sw_byte(0, lane & 15, 16 * x + (lane >> 4) * 8); }
// Two n-tiles (8 rows from n0, 8 from n1, multiples of 8) of a B operand held [n][k] in swizzled rows: r[0], r[1]
// are the first tile's fragment, r[2], r[3] the second's.  The lane part for a k step at column 16 x (of 64).
__device__ __forceinline__ uint32_t b_lane(int n0, int n1, int x, int lane) {
    return sw_byte(0, (lane < 16 ? n0 : n1) + (lane & 7), 16 * x + ((lane >> 3) & 1) * 8);
}
// Two adjacent n-tiles (16 columns from n0) of a B operand held [k][n] in swizzled rows, for ldsm4_t.
__device__ __forceinline__ uint32_t bt_lane(int rows, int n0, int lane) {
    return sw_byte(rows, ((lane >> 3) & 1) * 8 + (lane & 7), n0 + (lane >> 4) * 8);
}

// The warp's number, as a value that the compiler knows to be the same in all lanes: a branch on threadIdx.x / 32 around
// products costs a reconvergence each.
__device__ __forceinline__ int warp_number() { return __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0); }

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float low_of(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high_of(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// The first N bf16 terms of a pair of values.
template <int N> __device__ __forceinline__ void split(float x, float y, uint32_t (&t)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = pack(x, y);
        x -= low_of(t[i]);
        y -= high_of(t[i]);
    }
}

}  // namespace mma
}  // namespace gdn
