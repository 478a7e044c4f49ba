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

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void *row) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(sm100::smem_u32(row))
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], const void *row) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(sm100::smem_u32(row))
                 : "memory");
}

// c[16 x 8] += a[16 x 16] b[16 x 8].  Registers only, so the compiler may move it between the
// fragments' loads; a result is ready about 21 clocks later and an SM quarter takes one in 8, so the callers
// put two products or more between two of one accumulator.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Row address of an A operand held row-major (k contiguous): rows 16, k step of 16.
// Lanes 0-15 give the rows of the left 8 columns, 16-31 those of the right 8.
__device__ __forceinline__ const bf16 *a_row(const bf16 *base, int pitch, int row0, int k0, int lane) {
    return base + (row0 + (lane & 15)) * pitch + k0 + (lane >> 4) * 8;
}
// A operand held with its rows along the columns ([k][m], m contiguous), for ldsm4_t.
__device__ __forceinline__ const bf16 *at_row(const bf16 *base, int pitch, int k0, int m0, int lane) {
    return base + (k0 + (lane >> 4) * 8 + (lane & 7)) * pitch + m0 + ((lane >> 3) & 1) * 8;
}
// Rows of 64 columns (slabs of `rows` rows each) in the tensor maps' 128-byte swizzle: the 16-byte piece
// of (row, col) lies at piece (col / 8 % 8) ^ (row % 8) of its 128-byte line.
__device__ __forceinline__ const bf16 *sw_piece(const bf16 *base, int rows, int row, int col) {
    return base + (col >> 6) * rows * 64 + row * 64 + ((((col >> 3) & 7) ^ (row & 7)) << 3);
}
// Two n-tiles (8 rows from n0, 8 from n1) of a B operand held [n][k] in swizzled rows, k step of 16:
// r[0], r[1] are the first tile's fragment, r[2], r[3] the second's.
__device__ __forceinline__ const bf16 *b_row(const bf16 *base, int rows, int n0, int n1, int k0, int lane) {
    return sw_piece(base, rows, (lane < 16 ? n0 : n1) + (lane & 7), k0 + ((lane >> 3) & 1) * 8);
}
// Two adjacent n-tiles (16 columns from n0) of a B operand held [k][n] in swizzled rows, for ldsm4_t.
__device__ __forceinline__ const bf16 *bt_row(const bf16 *base, int rows, int k0, int n0, int lane) {
    return sw_piece(base, rows, k0 + ((lane >> 3) & 1) * 8 + (lane & 7), n0 + (lane >> 4) * 8);
}

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
