// pdssm_chunk.h -- chunks of 64 steps in LDS and in registers, shared by the
// recurrences over chunks (the gated delta rule, linear attention): rows from
// memory as bf16 parts, triangular matrices, states and their gradients, and
// the sums of what crosses a step.
#pragma once

#include "pdssm_device.h"
#include "pdssm_host.h"
#include "pdssm_layers.h"
#include "pdssm_mma.h"

namespace pdssm {

constexpr int kC = 64;          // steps of a chunk

// Lower blocks of 16 x 16 of a chunk's 64 x 64 matrices: block (a,b), b <= a,
// is number a (a + 1) / 2 + b.
constexpr int kTriBlocks = 10;
constexpr int kTriBlock = 256;     // values of a block
__host__ __device__ constexpr int block_of(int a, int b) { return a * (a + 1) / 2 + b; }
__host__ __device__ constexpr int row_of(int t) { return t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0; }

struct Rows {           // rows [B,H,L,(D)] of a call
    const void *p;
    pdssm_strides s;
};

// ---------------------------------------------------------------------------
// Rows of a chunk from memory into LDS, as bf16 parts.
// ---------------------------------------------------------------------------
template <bool BF16>
struct Unit;            // eight consecutive values of a row
template <>
struct Unit<true> {
    uint4 v;
};
template <>
struct Unit<false> {
    f32x8 v;
};

// Rows of one chunk as a buffer: a wave-uniform base and 32-bit offsets inside
// the chunk (strides along l are below kMaxStride, checked on the host).
// Places outside the sequence or the row get an offset beyond the buffer, so
// loads give zero and stores write nothing, without a branch.
constexpr uint32_t kOutside = 0x80000000u;
constexpr int64_t kMaxStride = 1 << 23;     // 64 rows of 4-byte values stay below 2^31 bytes

//
// VEC: rows of 16-byte units that do not overlap (see units() on the host).
// Rows past the sequence then lie past the buffer by themselves, and only the
// columns need a look.
template <bool BF16, bool VEC>
struct Chunk {
    __amdgpu_buffer_rsrc_t r;
    uint32_t stride;        // bytes between rows
    int rows, D;            // rows of the chunk inside the sequence
    static constexpr uint32_t kSize = BF16 ? 2 : 4;

    // Rows t0 .. of L of the sequence that begins at element e0.
    // `none`: as if it had no rows.
    __device__ __forceinline__ Chunk(const void *base, int64_t e0, int64_t s, int t0, int L, int D_, bool none = false)
    {
        rows = none ? 0 : min(L - t0, kC);
        D = D_;
        stride = (uint32_t)s * kSize;
        r = make_rsrc(static_cast<const char *>(base) + (e0 + t0 * s) * kSize,
                      none ? 0 : (uint64_t)(rows - 1) * stride + D * kSize);
    }
    __device__ __forceinline__ Chunk(__amdgpu_buffer_rsrc_t r_, uint32_t stride_, int rows_, int D_)
        : r(r_), stride(stride_), rows(rows_), D(D_)
    {
    }
    // A lane's own part of an offset.  Opaque, so that the offsets of a loop's
    // many rows are formed where they are used (an addition of a scalar each)
    // and not held in registers across the loop.
    __device__ __forceinline__ uint32_t lane_at(int row, int col) const
    {
        return (uint32_t)opaque(VEC && col >= D ? (int)kOutside : (int)(row * stride + col * kSize));
    }
    // The offset of lane row + `up`, `up` the same for all lanes.
    __device__ __forceinline__ uint32_t at(uint32_t lane, int row, int up, int col) const
    {
        return VEC || (row + up < rows && col < D) ? lane + up * stride : kOutside;
    }
    // Values col .. col + 7 of a row; VEC: rows begin on 16 bytes and hold
    // whole units.
    __device__ __forceinline__ Unit<BF16> unit(uint32_t lane, int row, int up, int col) const
    {
        Unit<BF16> u;
        if constexpr (VEC) {
            const uint32_t e = at(lane, row, up, col);
            const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, e, 0, 0);
            __builtin_memcpy(&u.v, &v, 16);
            if constexpr (!BF16) {
                const auto w = __builtin_amdgcn_raw_buffer_load_b128(r, e + 16, 0, 0);
                __builtin_memcpy(reinterpret_cast<char *>(&u.v) + 16, &w, 16);
            }
        } else if constexpr (BF16) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j] = bload<uint16_t>(r, at(lane + j * kSize, row, up, col + j), 0);
            u.v = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                u.v[j] = bload<float>(r, at(lane + j * kSize, row, up, col + j), 0);
        }
        return u;
    }
    __device__ __forceinline__ Unit<BF16> unit(int row, int col) const { return unit(lane_at(row, col), row, 0, col); }
    __device__ __forceinline__ uint32_t raw(uint32_t lane, int row, int up, int col) const
    {
        if constexpr (BF16)
            return bload<uint16_t>(r, at(lane, row, up, col), 0);
        else
            return bload<uint32_t>(r, at(lane, row, up, col), 0);
    }
    // Values col .. col + 3 of a row (VEC: col a multiple of 4).
    __device__ __forceinline__ f32x4 four(uint32_t lane, int row, int up, int col) const
    {
        f32x4 v;
        if constexpr (!VEC) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w = raw(lane + j * kSize, row, up, col + j);
                v[j] = BF16 ? bf16_lo(w) : __uint_as_float(w);
            }
        } else if constexpr (BF16) {
            const auto w = __builtin_amdgcn_raw_buffer_load_b64(r, at(lane, row, up, col), 0, 0);
            v = f32x4{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
        } else {
            const auto w = __builtin_amdgcn_raw_buffer_load_b128(r, at(lane, row, up, col), 0, 0);
            __builtin_memcpy(&v, &w, 16);
        }
        return v;
    }
    __device__ __forceinline__ void put4(uint32_t lane, int row, int up, int col, f32x4 v) const
    {
        if constexpr (!VEC) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                put(lane + j * kSize, row, up, col + j, v[j]);
        } else if constexpr (BF16) {
            typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
            const u32x2 w = {f32x2_to_bf16x2_rne(v[0], v[1]), f32x2_to_bf16x2_rne(v[2], v[3])};
            __builtin_amdgcn_raw_buffer_store_b64(w, r, at(lane, row, up, col), 0, 0);
        } else {
            typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
            u32x4 w;
            __builtin_memcpy(&w, &v, 16);
            __builtin_amdgcn_raw_buffer_store_b128(w, r, at(lane, row, up, col), 0, 0);
        }
    }
    __device__ __forceinline__ void put(uint32_t lane, int row, int up, int col, float v) const
    {
        if constexpr (BF16)
            __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16_rne(v), r, at(lane, row, up, col), 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, at(lane, row, up, col), 0, 0);
    }
};

// The chunks of a sequence one after another: the place of the next one and the
// way to the one behind it, formed once (the address of a chunk from its number
// costs scalar loads and products that a walk waits for).
struct Stream {
    const char *at;
    int64_t step;           // bytes
    uint32_t stride, width; // bytes between rows, of a row

    __device__ __forceinline__ Stream(const void *base, int64_t e0, int64_t s, int c, bool back, int D, int size)
    {
        at = static_cast<const char *>(base) + (e0 + (int64_t)c * kC * s) * size;
        step = (back ? -kC : kC) * s * size;
        stride = (uint32_t)s * (uint32_t)size;
        width = (uint32_t)(D * size);
    }
    // The chunk here, of `rows` rows (none: 0).
    template <bool BF16, bool VEC>
    __device__ __forceinline__ Chunk<BF16, VEC> chunk(int rows, int D) const
    {
        const uint32_t bytes = rows > 0 ? (uint32_t)(rows - 1) * stride + width : 0;
        return Chunk<BF16, VEC>(__builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(at), (short)0, (int)bytes, 0x00020000), stride,
                                rows, D);
    }
    __device__ __forceinline__ void next(bool move) { at += move ? step : 0; }
};

template <bool BF16>
__device__ __forceinline__ Frag<BF16 ? 1 : 3> unit_frag(const Unit<BF16> &u)
{
    if constexpr (BF16) {
        Frag<1> f;
        __builtin_memcpy(&f.p[0], &u.v, 16);
        return f;
    } else {
        return split<3>(u.v);
    }
}

// A tile of 64 rows of KD values in LDS: NK parts, rows of KD + 8 values (the
// padding spreads the rows over the banks).
// APART: what is not finite in fp32 rows stays in its place.
template <int KD, bool BF16, int NT = 256, bool APART = false>
struct Tile {
    static constexpr int NK = BF16 ? 1 : 3;
    static constexpr int kRow = KD + 8;
    static constexpr int kPart = kC * kRow;
    static constexpr int kSize = NK * kPart;                  // uint16_t
    static constexpr int kUnits = kC * (KD / 8) / NT;         // units of a thread

    Unit<BF16> u[kUnits];

    // `tid`: the thread's number among the NT that share the tile.
    template <bool VEC>
    __device__ __forceinline__ void load(const Chunk<BF16, VEC> &c, int tid)
    {
        const int row = tid / (KD / 8), col = tid % (KD / 8) * 8;
        const uint32_t lane = c.lane_at(row, col);
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            u[i] = c.unit(lane, row, i * (NT * 8 / KD), col);
    }
    __device__ __forceinline__ void store(uint16_t *lds, int tid) const
    {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int x = tid + i * NT, row = x / (KD / 8), col = x % (KD / 8) * 8;
            Frag<NK> f;
            if constexpr (APART && !BF16)
                f = split_apart(u[i].v);
            else
                f = unit_frag<BF16>(u[i]);
#pragma unroll
            for (int n = 0; n < NK; ++n)
                *reinterpret_cast<bf16x8 *>(lds + n * kPart + row * kRow + col) = f.p[n];
        }
    }

    // Values col .. col + 3 of a row (col a multiple of 4), and one value.
    static __device__ __forceinline__ f32x4 four(const uint16_t *lds, int row, int col)
    {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = NK - 1; n >= 0; --n)
            v += __builtin_convertvector(*reinterpret_cast<const bf16x4 *>(lds + n * kPart + row * kRow + col), f32x4);
        return v;
    }
    static __device__ __forceinline__ float one(const uint16_t *lds, int row, int col)
    {
        float v = 0.f;
#pragma unroll
        for (int n = NK - 1; n >= 0; --n)
            v += bf16_lo(lds[n * kPart + row * kRow + col]);
        return v;
    }

    // Row tile `a`, k = 32 s + 8 g + 0..7 (plain order).
    static __device__ __forceinline__ Frag<NK> rows(const uint16_t *lds, int a, int s, int lane)
    {
        Frag<NK> f;
#pragma unroll
        for (int n = 0; n < NK; ++n)
            f.p[n] = lds_row8(lds + n * kPart + (16 * a + (lane & 15)) * kRow + 32 * s + 8 * (lane >> 4));
        return f;
    }
    // Row tile `a`, k = 32 s + (4 g + 0..3, 16 + 4 g + 0..3) (stacked order).
    static __device__ __forceinline__ Frag<NK> rows_stacked(const uint16_t *lds, int a, int s, int lane)
    {
        Frag<NK> f;
#pragma unroll
        for (int n = 0; n < NK; ++n) {
            const uint16_t *p = lds + n * kPart + (16 * a + (lane & 15)) * kRow + 32 * s + 4 * (lane >> 4);
            f.p[n] = lds_rows4(p, p + 16);
        }
        return f;
    }
    // Columns 16 m + 0..15, k = rows 32 s + (4 g + 0..3, 16 + 4 g + 0..3).
    static __device__ __forceinline__ Frag<NK> columns_stacked(const uint16_t *lds, int m, int s, int lane)
    {
        Frag<NK> f;
        const int i = lane & 15, g = lane >> 4;
#pragma unroll
        for (int n = 0; n < NK; ++n) {
            const uint16_t *p = lds + n * kPart + (32 * s + 4 * g + (i >> 2)) * kRow + 16 * m + 4 * (i & 3);
            f.p[n] = lds_columns4(p, p + 16 * kRow);
        }
        return f;
    }
    // Columns 16 m + 0..15, k = rows 32 s + 8 g + 0..7.
    static __device__ __forceinline__ Frag<NK> columns(const uint16_t *lds, int m, int s, int lane)
    {
        Frag<NK> f;
        const int i = lane & 15, g = lane >> 4;
#pragma unroll
        for (int n = 0; n < NK; ++n) {
            const uint16_t *p = lds + n * kPart + (32 * s + 8 * g + (i >> 2)) * kRow + 16 * m + 4 * (i & 3);
            f.p[n] = lds_columns4(p, p + 4 * kRow);
        }
        return f;
    }
};

__device__ __forceinline__ f32x8 load8(const float *p)
{
    const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

__device__ __forceinline__ float dot8(f32x8 a, f32x8 b, float v)
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v += a[j] * b[j];
    return v;
}

// N parts of eight values, part n at p + n * part.
template <int N>
__device__ __forceinline__ void put_parts(uint16_t *p, int part, f32x8 v)
{
    const Frag<N> f = split<N>(v);
#pragma unroll
    for (int n = 0; n < N; ++n)
        *reinterpret_cast<bf16x8 *>(p + n * part) = f.p[n];
}

// Steps whose e^g rounds to zero in fp32 (half its smallest value is e^-103.97)
// empty the state.  They are counted and stay out of the running sum, where one
// of -1e12 would take the bits of every later gate of the chunk.
constexpr float kEmpties = -104.f;

// e^(G_i - G_j) from G log2(e) as a pair of floats, zero across a step that
// empties the state.
__device__ __forceinline__ float decay_of(float hi_i, float lo_i, float n_i, float hi_j, float lo_j, float n_j)
{
    return n_i == n_j ? __builtin_amdgcn_exp2f((hi_i - hi_j) + (lo_i - lo_j)) : 0.f;
}

__device__ __forceinline__ bool finite(float v) { return __builtin_fabsf(v) <= __FLT_MAX__; }

// ---------------------------------------------------------------------------
// A chunk's lower triangular matrix (or its transpose) in LDS as A operands in
// stacked order: fragment f of row tile a and k step s, part n, at
// ((f * 3 + n) * 64 + lane) * 8 values.  Six fragments hold the triangle; the
// halves of them that it leaves out are zero.
// ---------------------------------------------------------------------------
template <bool TRANS, int NT = 256>
struct Tri {
    static constexpr int kFrags = 6;
    static constexpr int kSize = kFrags * 3 * 64 * 8;    // uint16_t
    static constexpr int kUnits = (kTriBlocks * 64 + NT - 1) / NT;
    f32x4 u[kUnits];

    // Row tile a of the matrix has k step s (of the transpose: from a / 2 on).
    static __host__ __device__ constexpr bool has(int a, int s) { return TRANS ? s >= a / 2 : s <= a / 2; }
    static __host__ __device__ constexpr int frag(int a, int s) { return TRANS ? (a < 2 ? 2 * a + s : a + 2) : (a < 2 ? a : 2 * a - 2 + s); }

    // blocks: row format, or column format for the transpose.
    __device__ __forceinline__ void load(const float *blocks, int tid)
    {
#pragma unroll
        for (int i = 0; i < kUnits; ++i)    // (without a branch: see pipe_walk)
            u[i] = *reinterpret_cast<const f32x4 *>(blocks + 4 * min(tid + i * NT, kTriBlocks * 64 - 1));
    }
    __device__ __forceinline__ void store(uint16_t *lds, int tid) const
    {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int x = tid + i * NT;
            if (x < kTriBlocks * 64) {
                const int t = x >> 6, ta = row_of(t), tb = t - block_of(ta, 0);
                put(lds, TRANS ? tb : ta, TRANS ? ta : tb, x & 63, u[i]);
            }
        }
    }
    // Block (row, col) of the matrix: lane (g, i) gives row i, columns 4 g + 0..3.
    static __device__ __forceinline__ void put(uint16_t *lds, int row, int col, int lane, f32x4 block)
    {
        uint16_t *p = lds + ((frag(row, col >> 1) * 3) * 64 + lane) * 8 + 4 * (col & 1);
        float v[4] = {block[0], block[1], block[2], block[3]};
#pragma unroll
        for (int n = 0; n < 3; ++n)
            *reinterpret_cast<uint2 *>(p + n * 512) =
                make_uint2(take_part(v[0], v[1], n < 2), take_part(v[2], v[3], n < 2));
    }
    // The halves that no block fills.
    static __device__ __forceinline__ void clear(uint16_t *lds, int tid)
    {
        for (int x = tid; x < 2 * 3 * 64; x += NT) {
            const int f = TRANS ? (x < 192 ? frag(1, 0) : frag(3, 1)) : (x < 192 ? frag(0, 0) : frag(2, 1));
            const int half = TRANS ? 0 : 1;
            *reinterpret_cast<uint2 *>(lds + (f * 192 + x % 192) * 8 + 4 * half) = make_uint2(0, 0);
        }
    }
    template <int N>
    static __device__ __forceinline__ Frag<N> get(const uint16_t *lds, int a, int s, int lane)
    {
        Frag<N> f;
#pragma unroll
        for (int n = 0; n < N; ++n)
            f.p[n] = lds_row8(lds + ((frag(a, s) * 3 + n) * 64 + lane) * 8);
        return f;
    }
};

// A wave's 16 columns of the 64 rows of a chunk in the C layout (lane: column
// lane % 16, rows 16 a + 4 g + r).
template <bool BF16>
struct Cols {
    uint32_t raw[4][4];

    template <bool VEC>
    __device__ __forceinline__ void load(const Chunk<BF16, VEC> &c, int col, int lane)
    {
        const int row = 4 * (lane >> 4);
        const uint32_t e = c.lane_at(row, col);
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                raw[a][r] = c.raw(e, row, 16 * a + r, col);
    }
    __device__ __forceinline__ f32x4 get(int a) const
    {
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            v[r] = BF16 ? bf16_lo(raw[a][r]) : __uint_as_float(raw[a][r]);
        return v;
    }
};

template <bool BF16, bool VEC>
__device__ __forceinline__ void store_cols(const Chunk<BF16, VEC> &c, int col, int lane, int a, f32x4 v)
{
    const int row = 4 * (lane >> 4);
    const uint32_t e = c.lane_at(row, col);
#pragma unroll
    for (int r = 0; r < 4; ++r)
        c.put(e, row, 16 * a + r, col, v[r]);
}

// Values of a wave's 16 columns (lane: column col, rows 4 g + r of a tile) of
// a [rows][DV] fp32 array; rows and columns outside it read as zero and are
// not written.
struct Sheet {
    __amdgpu_buffer_rsrc_t r;
    uint32_t lane, pitch;
    __device__ __forceinline__ Sheet(const float *p, int rows, int DV, int col, int lane_, bool none = false)
    {
        pitch = DV * 4;
        r = make_rsrc(p, (uint64_t)rows * pitch);
        lane = col < DV && !none ? (uint32_t)opaque((lane_ >> 4) * 4 * (int)pitch + col * 4) : kOutside;
    }
    __device__ __forceinline__ f32x4 get(int tile) const
    {
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = bload<float>(r, lane + (16 * tile + i) * pitch, 0);
        return v;
    }
    __device__ __forceinline__ void put(int tile, f32x4 v) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[i]), r, lane + (16 * tile + i) * pitch, 0, 0);
    }
};

// A state (or its gradient): KD / 16 tiles in the C layout.
template <int KD>
struct State {
    f32x4 s[KD / 16];

    // [Dk][Dv] values from memory; NULL: zero.
    __device__ __forceinline__ void load(const float *p, int Dk, int Dv, int col, int lane)
    {
        const Sheet from(p, p ? Dk : 0, Dv, col, lane);
#pragma unroll
        for (int m = 0; m < KD / 16; ++m)
            s[m] = from.get(m);
    }
    __device__ __forceinline__ void store(float *p, int Dk, int Dv, int col, int lane) const
    {
        const Sheet to(p, Dk, Dv, col, lane);
#pragma unroll
        for (int m = 0; m < KD / 16; ++m)
            to.put(m, s[m]);
    }
};

// Values 16 a + 4 g + 0..3 of vector `which` among vectors of 64 in LDS.
__device__ __forceinline__ f32x4 row_vec(const float *s_vec, int which, int a, int lane)
{
    return *reinterpret_cast<const f32x4 *>(s_vec + which * kC + 16 * a + 4 * (lane >> 4));
}

// Over the lanes of a group of 16, in all of them: row rotations, which need
// no trip through LDS.
template <int N>
__device__ __forceinline__ float add_rotated(float v)
{
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xF, 0xF, true));
}
__device__ __forceinline__ float sum16(float v)
{
    return add_rotated<1>(add_rotated<2>(add_rotated<4>(add_rotated<8>(v))));
}

// The parts of dg that lie inside a chunk, from M = P . dP + N . dN (strictly
// below the diagonal): its sum over rows i >= t and columns j < t, for every t.
// Sixteen vectors of 16 values: the row sums and the column sums of the six
// blocks below the diagonal ones, and the diagonal blocks' own sums.
struct Cuts {
    static constexpr int kSize = 16 * 16;
    static __device__ __forceinline__ int below(int ta, int tb) { return ta * (ta - 1) / 2 + tb; }

    // Block (ta, tb), lane: column lane % 16, rows 4 g + r.
    static __device__ __forceinline__ void put(float *cuts, int ta, int tb, f32x4 m, int lane)
    {
        const int g = lane >> 4, i16 = lane & 15;
        float col[4];               // sums over the rows from 4 g + r on
        col[3] = m[3], col[2] = m[2] + col[3], col[1] = m[1] + col[2], col[0] = m[0] + col[1];
        float rest = col[0];        // over the rows of all lanes from this one on
#pragma unroll
        for (int n = 16; n <= 32; n <<= 1) {
            const float x = __shfl_down(rest, n, 64);
            rest += lane + n < 64 ? x : 0.f;
        }
        if (ta == tb) {
            float later = __shfl_down(rest, 16, 64);
            later = g < 3 ? later : 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float v = sum16(i16 < 4 * g + r ? later + col[r] : 0.f);
                if (i16 == 0)
                    cuts[(12 + ta) * 16 + 4 * g + r] = v;
            }
        } else {
            if (g == 0)
                cuts[(6 + below(ta, tb)) * 16 + i16] = rest;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float v = sum16(m[r]);
                if (i16 == 0)
                    cuts[below(ta, tb) * 16 + 4 * g + r] = v;
            }
        }
    }

    // Of step t = lane (one wave).
    static __device__ __forceinline__ float get(const float *cuts, int lane)
    {
        const int T = lane >> 4, l = lane & 15;
        float rows = 0.f, cols = 0.f, far = 0.f;
#pragma unroll
        for (int ta = 1; ta < 4; ++ta)
#pragma unroll
            for (int tb = 0; tb < ta; ++tb) {
                const float row = cuts[below(ta, tb) * 16 + l];
                rows += ta == T ? row : 0.f;
                cols += tb == T ? cuts[(6 + below(ta, tb)) * 16 + l] : 0.f;
                far += tb < T && T < ta ? row : 0.f;
            }
#pragma unroll
        for (int n = 1; n < 16; n <<= 1) {
            const float x = __shfl_down(rows, n, 16), y = __shfl_up(cols, n, 16);
            rows += l + n < 16 ? x : 0.f;
            cols += l >= n ? y : 0.f;
        }
        const float before = __shfl_up(cols, 1, 16);
        return cuts[(12 + T) * 16 + l] + rows + (l ? before : 0.f) + sum16(far);
    }
};

// dg of step t = lane of a chunk (one wave), from the chunk's whole <S, dS>, what
// the lane's step adds as a reader of S and as a writer of the state behind
// the chunk, and the parts inside it.
__device__ __forceinline__ float crossing(float whole, float reads, float writes, const float *cuts, int lane)
{
#pragma unroll
    for (int n = 1; n < 64; n <<= 1) {
        const float x = __shfl_down(reads, n, 64), y = __shfl_up(writes, n, 64);
        reads += lane + n < 64 ? x : 0.f;
        writes += lane >= n ? y : 0.f;
    }
    const float before = __shfl_up(writes, 1, 64);
    return whole + reads + (lane ? before : 0.f) + Cuts::get(cuts, lane);
}

// Every row begins on 16 bytes, ends with a whole unit of eight values and
// before the next one.
inline bool units(const void *p, const pdssm_strides &s, int D, int esize)
{
    const int e = 16 / esize;
    return aligned16(p) && s.b % e == 0 && s.h % e == 0 && s.l % e == 0 && D % 8 == 0 && s.l >= D;
}

// Strides along l that a chunk's 32-bit offsets can follow.
inline bool strides_ok(const pdssm_strides *s, int n)
{
    for (int i = 0; i < n; ++i)
        if (s[i].l < 0 || s[i].l >= kMaxStride)
            return false;
    return true;
}

inline bool element_aligned(const void *p, int esize) { return ((uintptr_t)p & (uintptr_t)(esize - 1)) == 0; }

}  // namespace pdssm
