// pdssm_mma.h -- matrix products of fp32 values on the bf16 matrix cores.
//
// An fp32 value is the sum of three bf16 values (8 + 8 + 8 bits), so a
// product of two fp32 matrices is the sum of the products of their parts;
// the terms of order i + j <= 2 hold it to about 2^-24, and six bf16
// products (three when one side is bf16 by nature) still run 2.7 times
// (5.3 times) the rate of the fp32 matrix instruction.
//
// Lane layouts of the 16 x 16 x 32 product (g = lane / 16, i = lane % 16):
//   A: row i, k = 8 g + 0..7      B: column i, k = 8 g + 0..7
//   C: column i, rows 4 g + 0..3
// The k order is free as long as A and B agree.  Two C tiles of 16 rows
// stacked are a B operand with k = (4 g + 0..3 of the first, 4 g + 0..3 of
// the second), so a result feeds the next product from its registers; A is
// then read in that order ("stacked" order) from memory.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "pdssm_device.h"

namespace pdssm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// N bf16 parts of eight values, the largest first.
template <int N>
struct Frag {
    bf16x8 p[N];
};

// One part of two values as a word, leaving the rest in them: one packed
// conversion, and one two-term dot product for each rest, a + w . (-1, 0),
// which is exact and spares the unpacking of the word.  The factors are kept
// from the compiler's sight: as literals it writes them in a 32-bit form whose
// upper half the instruction takes for both.
__device__ __forceinline__ uint32_t take_part(float &a, float &b, bool rest)
{
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const uint32_t w = f32x2_to_bf16x2_rne(a, b);
    if (rest) {
        uint32_t first = 0x0000BF80u, second = 0xBF800000u;
        asm("" : "+s"(first));
        asm("" : "+s"(second));
        bf16x2_t h, f, s;
        __builtin_memcpy(&h, &w, 4);
        __builtin_memcpy(&f, &first, 4);
        __builtin_memcpy(&s, &second, 4);
        a = __builtin_amdgcn_fdot2_f32_bf16(h, f, a, false);
        b = __builtin_amdgcn_fdot2_f32_bf16(h, s, b, false);
    }
    return w;
}

template <int N>
__device__ __forceinline__ Frag<N> split(f32x8 v)
{
    Frag<N> f;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        x[j] = v[j];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = take_part(x[2 * j], x[2 * j + 1], n + 1 < N);
        __builtin_memcpy(&f.p[n], w, 16);
    }
    return f;
}

// The B operand of two stacked C tiles.
template <int N>
__device__ __forceinline__ Frag<N> split(f32x4 a, f32x4 b)
{
    return split<N>(__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// c + A B over the parts' products of order below ORD, the small ones first.
template <int ORD, int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Frag<NA> &a, const Frag<NB> &b, f32x4 c)
{
#pragma unroll
    for (int o = ORD - 1; o >= 0; --o) {
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = o - i;
            if (j >= 0 && j < NB)
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[j], c, 0, 0, 0);
        }
    }
    return c;
}

// c + A B of 16 x 16 fp32 blocks on the fp32 matrix instruction: a = row
// lane % 16, columns 4 g + 0..3 of A; b = a C tile.
__device__ __forceinline__ f32x4 mma_f32(f32x4 a, f32x4 b, f32x4 c)
{
#pragma unroll
    for (int r = 0; r < 4; ++r)
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
    return c;
}

// Eight consecutive values from LDS.
__device__ __forceinline__ bf16x8 lds_row8(const uint16_t *p) { return *reinterpret_cast<const bf16x8 *>(p); }

// Two runs of four values from LDS (the stacked order of a row-major A).
__device__ __forceinline__ bf16x8 lds_rows4(const uint16_t *p, const uint16_t *q)
{
    const bf16x4 a = *reinterpret_cast<const bf16x4 *>(p), b = *reinterpret_cast<const bf16x4 *>(q);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Transposed read: the 16 lanes of a group read a block of 4 rows x 16
// columns (lane i its row i / 4, columns 4 (i % 4) + 0..3, at p), and lane i
// gets column i, rows 0..3.
__device__ __forceinline__ bf16x4 lds_column4(const uint16_t *p)
{
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p));
    bf16x4 r;
    __builtin_memcpy(&r, &v, 8);
    return r;
}

// Eight rows of column i, as two transposed reads at p and q.
__device__ __forceinline__ bf16x8 lds_columns4(const uint16_t *p, const uint16_t *q)
{
    const bf16x4 a = lds_column4(p), b = lds_column4(q);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// A flag in LDS: `set` comes after the wave's LDS writes before it, `await`
// returns once the flag is at least v and before the LDS reads after it.  (LDS
// instructions of a wave take effect in order; through a generic pointer the
// flag would also wait for the loads from memory in flight.)
struct LdsFlag {
    typedef __attribute__((address_space(3))) int lds_int;
    static __device__ __forceinline__ void set(int *p, int v)
    {
        asm volatile("" ::: "memory");
        *(volatile lds_int *)(lds_int *)p = v;
        asm volatile("" ::: "memory");
    }
    static __device__ __forceinline__ void await(int *p, int v)
    {
        while (*(volatile lds_int *)(lds_int *)p < v)
            __builtin_amdgcn_s_sleep(1);
        asm volatile("" ::: "memory");
    }
};

// A workgroup barrier that orders LDS only: loads from memory stay in flight
// across it (__syncthreads waits for them).
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace pdssm
