// The gated delta rule (include/pdssm_layers.h): forward, gradients, step.
//
// A chunk of 64 steps at once, from the state S before it.  With G the running
// sum of g inside the chunk, rise = e^G, left = e^(G_last - G), whole =
// e^G_last, decay[i,j] = e^(G_i - G_j) for j <= i, and
//     N = strictly lower part of (K K^T . decay)
//     P = scale * lower part of (Q K^T . decay)
// the steps' u solve u = beta (V - rise K S) - beta N u.  With the unscaled
// u~ = u / beta and Z = (I + N beta)^-1 N, which depends on keys and gates
// only,
//     R  = V - rise K S,    u~ = R - Z (beta R),    u = beta u~
//     O  = scale rise Q S + P u
//     S <- whole S + K^T (left u).
// Gradients, from dS of the state after the chunk:
//     dU = P^T dO + left K dS,   w = dU - Z^T (beta dU),   dV = beta w
//     dbeta = u~ . w (row by row)
//     dS <- whole dS + Q^T (scale rise dO) - K^T (rise dV)
//     X = lower part of (dO u^T . decay) scale,  Y = -strictly lower (dV u^T . decay)
//     dQ = X K + scale rise dO S^T
//     dK = X^T Q + (Y + Y^T) K + left u dS^T - rise dV S^T
//     dg_t = sum over what crosses step t: <whole S, dS>,
//            q_i . (scale rise dO S^T)_i - k_i . (rise dV S^T)_i   for i >= t,
//            k_j . (left u dS^T)_j                                 for j < t,
//            P_ij dP_ij + N_ij dN_ij                               for j < t <= i
// with dP = dO u^T and dN = -dV u^T: e^g_t is a factor of exactly these terms.
// (Shorter forms, as sums of q . dq - v . dv from t on, hold the terms that do
// not cross t twice with unlike signs: under strong decays dg is a small rest
// of them and loses its bits.)
//
// Kernels.  prep_kernel makes Z, P and the gates' vectors of every chunk, all
// chunks side by side.  The walks take the chunks of a head in order: a wave
// owns 16 columns of the state, whose recurrences are independent, and keeps
// them in registers in the matrix cores' result layout, so states and u feed
// the next product without leaving the wave.  pipe_kernel walks forward,
// back_kernel in both directions at once for the gradients (the walk forward
// then keeps the states and u~, the walk back the states' gradients and w),
// and grads_kernel forms what sums over the columns (dQ, dK, dg, dbeta), all
// chunks side by side.  Long sequences of few heads are cut into segments that
// walk side by side (cut_of, join_kernel).  chain_kernel, reverse_kernel and
// grad_kernel are the same steps for fp32 data, whose three parts of q, k and
// dO fill LDS, with all of a workgroup's waves doing the same.
//
// What bounds them: a walk takes its chunks one after another, and each is a
// chain of three products and two splits into parts that no other work of the
// head can overtake; see cut_of for its time.  The preparation and grads_kernel
// wait for memory between their phases more than they compute.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pdssm_device.h"
#include "pdssm_host.h"
#include "pdssm_layers.h"
#include "pdssm_mma.h"

namespace pdssm {
namespace {

constexpr int kC = 64;          // steps of a chunk
constexpr int kThreads = 256;
constexpr int kMaxDim = 128;

// Lower blocks of 16 x 16 of a chunk's 64 x 64 matrices: block (a,b), b <= a,
// is number a (a + 1) / 2 + b.
constexpr int kBlocks = 10;
constexpr int kBlock = 256;     // values of a block
__host__ __device__ constexpr int block_of(int a, int b) { return a * (a + 1) / 2 + b; }
__host__ __device__ constexpr int row_of(int t) { return t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0; }

// What prep_kernel leaves for a chunk, in floats.  In row format a block's
// lane (g, i) holds row i, columns 4 g + 0..3; in column format column i,
// rows 4 g + 0..3.
enum Vec { kRise, kLeft, kBeta, kWhole, kGhi, kGlo, kResets, kVecs };
struct Record {
    // forward: Z and P in row format; backward: Z in both, P in column format
    static constexpr int kZ = 0;
    static constexpr int kP = kBlocks * kBlock;
    static constexpr int kVec = 2 * kBlocks * kBlock;
    static constexpr int kZt = kVec + 8 * kC;
    static constexpr int kFwd = kZt;
    static constexpr int kBwd = kZt + kBlocks * kBlock;
};

struct Rows {           // rows [B,H,L,(D)] of a call
    const void *p;
    pdssm_strides s;
};

struct DeltaArgs {
    Rows q, k, v, g, beta, o, d_o;   // o, d_o: what the direction has
    Rows dq, dk, dv, dg, dbeta;
    const float *s0;        // NULL for zero
    float *s_final;         // NULL when not wanted
    const float *ds_final;
    float *ds0;
    float *records;         // [B*Hv][NC][record]
    float *states;          // [B*Hv][NC][DK][DV] states before the chunks (backward)
    float *grads;           // same shape: state gradients after the chunks
    float *ut, *w;          // [B*Hv][NC][64][DV]: u~ and w
    int64_t heads;          // B*Hv
    // Few heads: the chunks cut in segments of seg_chunks, walked side by side.
    int segs, seg_chunks;
    float *seg_states;      // [B*Hv][segs][KD][DV]: states before the segments (s0 among them)
    float *trans;           // [B*Hv][segs][KD][slices*64 + KD]: their ends from zero, and transitions
    float *seg_grads;       // [B*Hv][segs][KD][DV]: state gradients after the segments (ds_final among them)
    float *rtrans;          // [B*Hv][segs][KD][slices*64]: state gradients before them, from zero
    unsigned back_blocks;   // workgroups of back_kernel that walk back
    int Hk, Hv, L, NC, Dk, Dv, DV, record;
    int slices;             // column slices of a head over workgroups
    float scale;
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
    __device__ __forceinline__ void put(uint32_t lane, int row, int up, int col, float v) const
    {
        if constexpr (BF16)
            __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16_rne(v), r, at(lane, row, up, col), 0, 0);
        else
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, at(lane, row, up, col), 0, 0);
    }
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
template <int KD, bool BF16, int NT = kThreads>
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
            const Frag<NK> f = unit_frag<BF16>(u[i]);
#pragma unroll
            for (int n = 0; n < NK; ++n)
                *reinterpret_cast<bf16x8 *>(lds + n * kPart + row * kRow + col) = f.p[n];
        }
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

// A NaN or an infinity in a column of 64 steps (C layout, the column's rows over
// the lanes of i16): it would reach the steps before it through the zeros of
// the triangular matrices, so R and beta R of the steps from the first such one
// on become zero, and their results NaN.
struct Spoiled {
    int from = kC;      // the first such step of the lane's column, kC: none

    __device__ __forceinline__ void take_out(f32x4 (&R)[4], f32x4 (&x)[4], int g)
    {
        float mark = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                mark = __builtin_fmaf(x[t][r], 0.f, mark);
        if (__any(mark != 0.f)) {
#pragma unroll
            for (int t = 3; t >= 0; --t)
#pragma unroll
                for (int r = 3; r >= 0; --r)
                    from = finite(x[t][r]) ? from : 16 * t + 4 * g + r;
            from = min(from, __shfl_xor(from, 16, 64));
            from = min(from, __shfl_xor(from, 32, 64));
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                put(R[t], t, g, from, 0.f);
                put(x[t], t, g, from, 0.f);
            }
        }
    }
    // v in the place of a tile's steps from `from` on.
    static __device__ __forceinline__ void put(f32x4 &x, int tile, int g, int from, float v)
    {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            x[r] = 16 * tile + 4 * g + r < from ? x[r] : v;
    }
    __device__ __forceinline__ float whole(float v) const { return from < kC ? __builtin_nanf("") : v; }
};

__device__ __forceinline__ int64_t kv_head(const DeltaArgs &a, int64_t head, int64_t &b, int &h)
{
    b = head / a.Hv;
    h = (int)(head - b * a.Hv);
    return h / (a.Hv / a.Hk);
}

// ---------------------------------------------------------------------------
// prep_kernel: Z, P and the gates' vectors of one chunk of one value head.
// Wave a forms row tile a of N and P (bf16 products are exact, fp32 data goes
// in three parts).  Z = N - N beta Z by forward substitution over 16 x 16
// blocks: the diagonal blocks row by row with a column in each lane, the
// others by fp32 matrix instructions, a block column in each wave.  138 to
// 176 us for the 16384 chunks of the LM layer (8 x 32 heads of 64, 4096 steps),
// 3.7 to 4.7 TB/s of the 642 MB that the counters show: five workgroups of 32 KB
// LDS a compute unit, each waiting at the ends of its phases.
// ---------------------------------------------------------------------------
constexpr int kMat = 20;        // row of a 16 x 16 fp32 block in LDS
__device__ __forceinline__ constexpr int lds_block(int a, int b) { return block_of(a, b) * 16 * kMat; }

template <int KD, bool BF16, bool VEC, bool BWD>
__global__ void __launch_bounds__(kThreads) prep_kernel(DeltaArgs a)
{
    using T = Tile<KD, BF16>;
    constexpr int kMatrix = kBlocks * 16 * kMat;
    static_assert(kMatrix * 4 <= T::kSize * 4, "Z takes the place of k and q");
    __shared__ __attribute__((aligned(16))) char s_mem[T::kSize * 4 + kMatrix * 4];
    __shared__ float s_hi[kC], s_lo[kC], s_n[kC], s_beta[kC];
    __shared__ int s_odd[kC];
    uint16_t *s_k = reinterpret_cast<uint16_t *>(s_mem);
    uint16_t *s_q = reinterpret_cast<uint16_t *>(s_mem + T::kSize * 2);
    float *s_z = reinterpret_cast<float *>(s_mem);      // after N and P, in the place of k and q
    float *s_N = reinterpret_cast<float *>(s_mem + T::kSize * 4);

    const int64_t head = blockIdx.x / (unsigned)a.NC;
    const int c = blockIdx.x % (unsigned)a.NC;
    int64_t b;
    int h;
    const int64_t hk = kv_head(a, head, b, h);
    const int t0 = c * kC, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = lane >> 4, i16 = lane & 15;
    float *rec = a.records + (int64_t)blockIdx.x * a.record;
    float rise = 0.f;   // of step t0 + lane (wave 0)

    {
        T q, k;
        k.load(Chunk<BF16, VEC>(a.k.p, b * a.k.s.b + hk * a.k.s.h, a.k.s.l, t0, a.L, a.Dk), threadIdx.x);
        q.load(Chunk<BF16, VEC>(a.q.p, b * a.q.s.b + hk * a.q.s.h, a.q.s.l, t0, a.L, a.Dk), threadIdx.x);
        if (wave == 0) {
            // G log2(e) in 64 bits (differences of neighbours stay exact to
            // 32), steps that empty the state counted apart.
            const int t = t0 + lane;
            float gate = 0.f, bt = 0.f;
            if (t < a.L) {
                gate = static_cast<const float *>(a.g.p)[b * a.g.s.b + h * a.g.s.h + t * a.g.s.l];
                bt = static_cast<const float *>(a.beta.p)[b * a.beta.s.b + h * a.beta.s.h + t * a.beta.s.l];
            }
            const bool empty = gate < kEmpties;
            double G = empty ? 0.0 : (double)gate * 1.4426950408889634;
            float n = empty ? 1.f : 0.f;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double x = __shfl_up(G, m, 64);
                const float y = __shfl_up(n, m, 64);
                if (lane >= m) {
                    G += x;
                    n += y;
                }
            }
            const float hi = (float)G, lo = (float)(G - (double)hi);
            const float hi1 = __shfl(hi, 63, 64), lo1 = __shfl(lo, 63, 64), n1 = __shfl(n, 63, 64);
            s_hi[lane] = hi;
            s_lo[lane] = lo;
            s_n[lane] = n;
            s_beta[lane] = finite(bt) ? bt : 0.f;
            rise = finite(bt) ? decay_of(hi, lo, n, 0.f, 0.f, 0.f) : __builtin_nanf("");
            float *vec = rec + Record::kVec;
            vec[kBeta * kC + lane] = BWD ? bt : s_beta[lane];
            vec[kLeft * kC + lane] = decay_of(hi1, lo1, n1, hi, lo, n);
            vec[kWhole * kC + lane] = decay_of(hi1, lo1, n1, 0.f, 0.f, 0.f);
            vec[kGhi * kC + lane] = hi;
            vec[kGlo * kC + lane] = lo;
            vec[kResets * kC + lane] = n;
        }
        k.store(s_k, threadIdx.x);
        q.store(s_q, threadIdx.x);
    }
    __syncthreads();

    // Row tile `wave` of N and P, results as rows i = lane % 16 (columns in
    // the registers), P in column format for the backward.
    {
        Frag<T::NK> ka[KD / 32], qa[KD / 32];
#pragma unroll
        for (int s = 0; s < KD / 32; ++s) {
            ka[s] = T::rows(s_k, wave, s, lane);
            qa[s] = T::rows(s_q, wave, s, lane);
        }
        const int row = 16 * wave + i16;
        const float hi = s_hi[row], lo = s_lo[row], n = s_n[row];
        int odd = 0;
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
            if (tb > wave)
                continue;
            f32x4 kk = {0.f, 0.f, 0.f, 0.f}, qk = kk;
#pragma unroll
            for (int s = 0; s < KD / 32; ++s) {
                const Frag<T::NK> kb = T::rows(s_k, tb, s, lane);
                kk = mma<3>(kb, ka[s], kk);
                qk = BWD ? mma<3>(qa[s], kb, qk) : mma<3>(kb, qa[s], qk);
            }
            f32x4 nn, pp;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int col = 16 * tb + 4 * g + r;
                const float d = decay_of(hi, lo, n, s_hi[col], s_lo[col], s_n[col]);
                nn[r] = col < row ? kk[r] * d : 0.f;
                odd |= !finite(nn[r]);
                nn[r] = finite(nn[r]) ? nn[r] : 0.f;
                if constexpr (BWD) {
                    const int pi = 16 * wave + 4 * g + r, pj = 16 * tb + i16;
                    const float e = decay_of(s_hi[pi], s_lo[pi], s_n[pi], s_hi[pj], s_lo[pj], s_n[pj]);
                    pp[r] = pj <= pi ? a.scale * qk[r] * e : 0.f;
                } else {
                    pp[r] = col <= row ? a.scale * qk[r] * d : 0.f;
                }
            }
            *reinterpret_cast<f32x4 *>(s_N + lds_block(wave, tb) + i16 * kMat + 4 * g) = nn;
            *reinterpret_cast<f32x4 *>(rec + Record::kP + block_of(wave, tb) * kBlock + 4 * lane) = pp;
        }
        odd |= __shfl_xor(odd, 16, 64);
        odd |= __shfl_xor(odd, 32, 64);
        if (g == 0)
            s_odd[row] = odd;
    }
    __syncthreads();    // N whole; q's place is free for Z
    // What is not finite stays out of Z, whose products would carry it, times
    // zero, to the steps before; its own step is spoiled through rise.
    if (wave == 0)
        rec[Record::kVec + kRise * kC + lane] = s_odd[lane] ? __builtin_nanf("") : rise;

    // Diagonal block `wave`, a column in each lane, four rows at a time: what
    // the rows above take from all four, then the four among themselves.
    {
        const float *N = s_N + lds_block(wave, wave);
        float y[16], z[16];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            float v[4];
            f32x4 tri[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = N[(4 * p + i) * kMat + i16];
                tri[i] = *reinterpret_cast<const f32x4 *>(N + (4 * p + i) * kMat + 4 * p);
            }
#pragma unroll
            for (int m = 0; m < p; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 row = *reinterpret_cast<const f32x4 *>(N + (4 * p + i) * kMat + 4 * m);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        v[i] -= row[r] * y[4 * m + r];
                }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int r = 0; r < i; ++r)
                    v[i] -= tri[i][r] * y[4 * p + r];
                z[4 * p + i] = v[i];
                y[4 * p + i] = v[i] * s_beta[16 * wave + 4 * p + i];
            }
        }
        if (g == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                s_z[lds_block(wave, wave) + i * kMat + i16] = z[i];
        }
    }
    __syncthreads();

    // Block column `wave` below the diagonal: Z_aj = X - Z_aa beta X with
    // X = N_aj - sum over m of N_am (beta Z)_mj.
    {
        f32x4 y[4];
        f32x4 beta[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            beta[m] = *reinterpret_cast<const f32x4 *>(s_beta + 16 * m + 4 * g);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                y[m][r] = m == wave ? s_z[lds_block(m, m) + (4 * g + r) * kMat + i16] * beta[m][r] : 0.f;
        }
#pragma unroll
        for (int ta = 1; ta < 4; ++ta) {
            if (ta <= wave)
                continue;
            f32x4 x;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                x[r] = s_N[lds_block(ta, wave) + (4 * g + r) * kMat + i16];
#pragma unroll
            for (int m = 0; m < ta; ++m)
                if (m >= wave)
                    x = mma_f32(-*reinterpret_cast<const f32x4 *>(s_N + lds_block(ta, m) + i16 * kMat + 4 * g), y[m], x);
            const f32x4 zd = *reinterpret_cast<const f32x4 *>(s_z + lds_block(ta, ta) + i16 * kMat + 4 * g);
            x = mma_f32(-zd, x * beta[ta], x);
            y[ta] = x * beta[ta];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                s_z[lds_block(ta, wave) + (4 * g + r) * kMat + i16] = x[r];
        }
    }
    __syncthreads();

    // Z out: row format, and column format for the backward.
    for (int t = wave; t < kBlocks; t += kThreads / 64) {
        const float *z = s_z + t * 16 * kMat;
        *reinterpret_cast<f32x4 *>(rec + Record::kZ + t * kBlock + 4 * lane) =
            *reinterpret_cast<const f32x4 *>(z + i16 * kMat + 4 * g);
        if constexpr (BWD) {
            f32x4 v;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                v[r] = z[(4 * g + r) * kMat + i16];
            *reinterpret_cast<f32x4 *>(rec + Record::kZt + t * kBlock + 4 * lane) = v;
        }
    }
}

// ---------------------------------------------------------------------------
// A chunk's lower triangular matrix (or its transpose) in LDS as A operands in
// stacked order: fragment f of row tile a and k step s, part n, at
// ((f * 3 + n) * 64 + lane) * 8 values.  Six fragments hold the triangle; the
// halves of them that it leaves out are zero.
// ---------------------------------------------------------------------------
template <bool TRANS, int NT = kThreads>
struct Tri {
    static constexpr int kFrags = 6;
    static constexpr int kSize = kFrags * 3 * 64 * 8;    // uint16_t
    static constexpr int kUnits = (kBlocks * 64 + NT - 1) / NT;
    f32x4 u[kUnits];

    // Row tile a of the matrix has k step s (of the transpose: from a / 2 on).
    static __host__ __device__ constexpr bool has(int a, int s) { return TRANS ? s >= a / 2 : s <= a / 2; }
    static __host__ __device__ constexpr int frag(int a, int s) { return TRANS ? (a < 2 ? 2 * a + s : a + 2) : (a < 2 ? a : 2 * a - 2 + s); }

    // blocks: row format, or column format for the transpose.
    __device__ __forceinline__ void load(const float *blocks, int tid)
    {
#pragma unroll
        for (int i = 0; i < kUnits; ++i)    // (without a branch: see pipe_walk)
            u[i] = *reinterpret_cast<const f32x4 *>(blocks + 4 * min(tid + i * NT, kBlocks * 64 - 1));
    }
    __device__ __forceinline__ void store(uint16_t *lds, int tid) const
    {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int x = tid + i * NT;
            if (x < kBlocks * 64) {
                const int t = x >> 6, lane = x & 63;
                const int ta = row_of(t), tb = t - block_of(ta, 0);
                const int row = TRANS ? tb : ta, col = TRANS ? ta : tb;
                uint16_t *p = lds + ((frag(row, col >> 1) * 3) * 64 + lane) * 8 + 4 * (col & 1);
                float v[4] = {u[i][0], u[i][1], u[i][2], u[i][3]};
#pragma unroll
                for (int n = 0; n < 3; ++n)
                    *reinterpret_cast<uint2 *>(p + n * 512) =
                        make_uint2(take_part(v[0], v[1], n < 2), take_part(v[2], v[3], n < 2));
            }
        }
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

// Four vectors of the record in LDS (rise, left, beta, whole).
__device__ __forceinline__ f32x4 load_vecs(const float *vec, int tid)
{
    return *reinterpret_cast<const f32x4 *>(vec + 4 * (tid % kC));
}
__device__ __forceinline__ f32x4 row_vec(const float *s_vec, int which, int a, int lane)
{
    return *reinterpret_cast<const f32x4 *>(s_vec + which * kC + 16 * a + 4 * (lane >> 4));
}

// ---------------------------------------------------------------------------
// chain_kernel: the chunks of a head in order, fp32 data.  KEEP: the
// backward's pass, which keeps the states before the chunks and u~ and forms
// no outputs.  About 4 us a chunk (keys of 64): the next chunk's rows load
// while this one's products run, but every wave stages, walks and stores in
// turn.
// ---------------------------------------------------------------------------
template <int KD, bool VEC, bool KEEP>
__global__ void __launch_bounds__(kThreads) chain_kernel(DeltaArgs a)
{
    constexpr bool BF16 = false;
    using T = Tile<KD, BF16>;
    using L_ = Tri<false>;
    constexpr int NO = 3;
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    uint16_t *s_k = reinterpret_cast<uint16_t *>(s_dyn);
    uint16_t *s_z = s_k + T::kSize;
    float *s_vec = reinterpret_cast<float *>(s_z + L_::kSize);
    uint16_t *s_q = reinterpret_cast<uint16_t *>(s_vec + 4 * kC);     // with outputs only
    uint16_t *s_p = s_q + T::kSize;

    const int64_t head = blockIdx.x / (unsigned)a.slices;
    const int slice = blockIdx.x % (unsigned)a.slices;
    int64_t b;
    int h;
    const int64_t hk = kv_head(a, head, b, h);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = (slice * (kThreads / 64) + wave) * 16 + (lane & 15);
    const int64_t ek = b * a.k.s.b + hk * a.k.s.h, eq = b * a.q.s.b + hk * a.q.s.h, ev = b * a.v.s.b + h * a.v.s.h;
    const float *rec = a.records + head * a.NC * (int64_t)a.record;

    T tk, tq;
    L_ tz, tp;
    Cols<BF16> v;
    f32x4 tv;
    auto fetch = [&](int c) {
        const float *r = rec + (int64_t)c * a.record;
        tk.load(Chunk<BF16, VEC>(a.k.p, ek, a.k.s.l, c * kC, a.L, a.Dk), threadIdx.x);
        tz.load(r + Record::kZ, threadIdx.x);
        tv = load_vecs(r + Record::kVec, threadIdx.x);
        v.load(Chunk<BF16, VEC>(a.v.p, ev, a.v.s.l, c * kC, a.L, a.Dv), col, lane);
        if constexpr (!KEEP) {
            tq.load(Chunk<BF16, VEC>(a.q.p, eq, a.q.s.l, c * kC, a.L, a.Dk), threadIdx.x);
            tp.load(r + Record::kP, threadIdx.x);
        }
    };
    State<KD> S;
    S.load(a.s0 ? a.s0 + head * a.Dk * a.Dv : nullptr, a.Dk, a.Dv, col, lane);
    L_::clear(s_z, threadIdx.x);
    if constexpr (!KEEP)
        L_::clear(s_p, threadIdx.x);
    fetch(0);
    for (int c = 0; c < a.NC; ++c) {
        tk.store(s_k, threadIdx.x);
        tz.store(s_z, threadIdx.x);
        if (threadIdx.x < kC)
            *reinterpret_cast<f32x4 *>(s_vec + 4 * threadIdx.x) = tv;
        if constexpr (!KEEP) {
            tq.store(s_q, threadIdx.x);
            tp.store(s_p, threadIdx.x);
        }
        f32x4 R[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            R[t] = v.get(t);
        lds_barrier();
        if (c + 1 < a.NC)
            fetch(c + 1);

        if constexpr (KEEP) {
            const Sheet out(a.states + (head * a.NC + c) * KD * a.DV, KD, a.DV, col, lane);
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
                out.put(m, S.s[m]);
        }
        f32x4 ks[4], qs[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            ks[t] = qs[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KD / 32; ++s) {
            const Frag<3> f = split<3>(S.s[2 * s], S.s[2 * s + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                ks[t] = mma<3>(T::rows_stacked(s_k, t, s, lane), f, ks[t]);
                if constexpr (!KEEP)
                    qs[t] = mma<NO>(T::rows_stacked(s_q, t, s, lane), f, qs[t]);
            }
        }
        f32x4 x[4], u[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            R[t] -= row_vec(s_vec, kRise, t, lane) * ks[t];
            x[t] = row_vec(s_vec, kBeta, t, lane) * R[t];
            u[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        Spoiled bad;
        if constexpr (!KEEP)
            bad.take_out(R, x, lane >> 4);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Frag<3> f = split<3>(x[2 * s], x[2 * s + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (L_::has(t, s))
                    u[t] = mma<3>(L_::template get<3>(s_z, t, s, lane), f, u[t]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            u[t] = R[t] - u[t];      // u~
            if constexpr (KEEP)
                Sheet(a.ut + (head * a.NC + c) * kC * a.DV, kC, a.DV, col, lane).put(t, u[t]);
            u[t] *= row_vec(s_vec, kBeta, t, lane);
        }
        if constexpr (!KEEP) {
            f32x4 o[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                o[t] = a.scale * row_vec(s_vec, kRise, t, lane) * qs[t];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag<NO> f = split<NO>(u[2 * s], u[2 * s + 1]);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (L_::has(t, s))
                        o[t] = mma<NO>(L_::template get<NO>(s_p, t, s, lane), f, o[t]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                Spoiled::put(o[t], t, lane >> 4, bad.from, __builtin_nanf(""));
                store_cols(Chunk<BF16, VEC>(a.o.p, b * a.o.s.b + h * a.o.s.h, a.o.s.l, c * kC, a.L, a.Dv), col, lane, t, o[t]);
            }
        }
        const float whole = bad.whole(s_vec[kWhole * kC]);
#pragma unroll
        for (int m = 0; m < KD / 16; ++m)
            S.s[m] *= whole;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Frag<3> f = split<3>(row_vec(s_vec, kLeft, 2 * s, lane) * u[2 * s],
                                       row_vec(s_vec, kLeft, 2 * s + 1, lane) * u[2 * s + 1]);
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
                S.s[m] = mma<3>(T::columns_stacked(s_k, m, s, lane), f, S.s[m]);
        }
        lds_barrier();
    }
    if (!KEEP && a.s_final)
        S.store(a.s_final + head * a.Dk * a.Dv, a.Dk, a.Dv, col, lane);
}

// ---------------------------------------------------------------------------
// pipe_walk: the walk for bf16 data, a workgroup of twelve waves.  Waves 0..3
// ("chain") own 16 columns of the state each and do only what the next chunk
// waits for: u from S, then S.  Waves 4..11 ("help") stage the next chunk's K,
// V, Z and vectors in the other half of LDS, and form the outputs of the chunk
// before: two of them share the columns of a chain wave, whose S and u they
// get as fp32 through LDS and split again (the chain's own three parts of S do
// not fit for keys of 128).  One barrier a chunk; a flag says when S is there.
// The LM layer's walk takes 227 to 288 us, 3.5 us a chunk on every compute unit: the
// chain alone needs 2.4 us (84 products of 16 cycles, 370 other instructions,
// reads from LDS between them), the help waves' loads, products and stores on
// the same four SIMDs the rest.  (S, u and P in two parts for the outputs, whose
// terms then hold 16 bits: 203 to 247 us.)
// ---------------------------------------------------------------------------
enum Mode { kOut, kKeep, kScan };   // outputs; states and u~ kept; the last state alone

constexpr int kHelpThreads = 512, kPipeThreads = 256 + kHelpThreads;

template <int KD>
struct PipeLds {
    using K = Tile<KD, true, kHelpThreads>;
    using V = Tile<kC, true, kHelpThreads>;
    using Z = Tri<false, kHelpThreads>;
    static constexpr int kSRow = KD + 4, kURow = kC + 4;    // S and u: fp32, a wave's columns as rows
    static constexpr int kSWave = 16 * kSRow, kUWave = 16 * kURow;
    // in uint16_t
    static constexpr int kK = 0;
    static constexpr int kZ = kK + 2 * K::kSize;
    static constexpr int kV = kZ + 2 * Z::kSize;
    static constexpr int kVec = kV + 2 * V::kSize;
    static constexpr int kFlag = kVec + 2 * 4 * kC * 2;
    static constexpr int kS = kFlag + 16;                   // with outputs only
    static constexpr int kU = kS + 2 * 4 * kSWave;
    static constexpr int kFrom = kU + 2 * 2 * 4 * kUWave;   // [2][4 waves][16 columns]: the first spoiled step
    static constexpr size_t bytes(bool out) { return (out ? kFrom + 2 * 2 * 4 * 16 : kS) * 2; }
};

template <int KD, bool VEC, int MODE, bool CAREFUL>
__device__ __forceinline__ bool pipe_pass(const DeltaArgs &a, unsigned block, int thread)
{
    using LDS = PipeLds<KD>;
    using TK = typename LDS::K;
    using TV = typename LDS::V;
    using L_ = typename LDS::Z;
    constexpr int NS = KD / 32;     // k steps over the key dimensions
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    uint16_t *lds = reinterpret_cast<uint16_t *>(s_dyn);
    int *s_flag = reinterpret_cast<int *>(lds + LDS::kFlag), *s_spoiled = s_flag + 4;

    // What this workgroup walks: chunks c0 .. c1 - 1 of 64 columns of a head's
    // state, or (kScan) of 64 columns of the segment's transition, the state
    // that the unit matrix becomes without any v.
    // A scan leaves out what no joining asks for: the last segment's end and
    // transition, and the first one's transition.
    const int parts = a.slices + (MODE == kScan ? KD / 64 : 0);
    const int64_t head = block / (unsigned)(a.segs * parts);
    const int rest = block % (unsigned)(a.segs * parts), seg = rest / parts, slice = rest % parts;
    const bool unit = slice >= a.slices;
    if (MODE == kScan && (seg == a.segs - 1 || (unit && seg == 0)))
        return false;
    const int c0 = seg * a.seg_chunks, c1 = min(a.NC, c0 + a.seg_chunks);
    int64_t b;
    int h;
    const int64_t hk = kv_head(a, head, b, h);
    const int lane = thread & 63, wave = thread >> 6, g = lane >> 4, i16 = lane & 15;
    const int mine = wave & 3;      // the chain wave, or the one that this wave helps
    const int col = (slice * 4 + mine) * 16 + i16;
    bool again = false;

    if (wave < 4) {
        State<KD> S;
        if (unit) {
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    S.s[m][r] = 16 * m + 4 * g + r == col - a.slices * 64 ? 1.f : 0.f;
        } else if (a.segs > 1 && MODE != kScan) {
            S.load(a.seg_states + (head * a.segs + seg) * KD * a.DV, KD, a.DV, col, lane);
        } else {
            S.load(a.s0 && seg == 0 ? a.s0 + head * a.Dk * a.Dv : nullptr, a.Dk, a.Dv, col, lane);
        }
        if (lane == 0)
            s_flag[mine] = c0;
        Frag<3> sf[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s)
            sf[s] = split<3>(S.s[2 * s], S.s[2 * s + 1]);
        lds_barrier();
        for (int c = c0; c < c1; ++c) {
            const int half = (c - c0) & 1;
            const uint16_t *s_k = lds + LDS::kK + half * TK::kSize, *s_z = lds + LDS::kZ + half * L_::kSize;
            const uint16_t *s_v = lds + LDS::kV + half * TV::kSize;
            const float *s_vec = reinterpret_cast<const float *>(lds + LDS::kVec) + half * 4 * kC;
            Frag<1> kr[2][4];       // two k steps at a time
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    kr[s][t] = TK::rows_stacked(s_k, t, s, lane);
            if constexpr (MODE == kOut) {
                float *x = reinterpret_cast<float *>(lds + LDS::kS) + mine * LDS::kSWave + i16 * LDS::kSRow + 4 * g;
#pragma unroll
                for (int m = 0; m < KD / 16; ++m)
                    *reinterpret_cast<f32x4 *>(x + 16 * m) = S.s[m];
                if (lane == 0)
                    LdsFlag::set(&s_flag[mine], c + 1);
            }
            if constexpr (MODE == kKeep) {
                const Sheet out(a.states + (head * a.NC + c) * KD * a.DV, KD, a.DV, col, lane);
#pragma unroll
                for (int m = 0; m < KD / 16; ++m)
                    out.put(m, S.s[m]);
            }
            __builtin_amdgcn_sched_barrier(0);

            // k S, while V and the first half of Z arrive
            f32x4 R[4];
            bf16x4 v4[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                R[t] = f32x4{0.f, 0.f, 0.f, 0.f};
                v4[t] = lds_column4(s_v + (16 * t + 4 * g + (i16 >> 2)) * TV::kRow + 16 * mine + 4 * (i16 & 3));
            }
            Frag<3> z0[4], z1[2];
            auto load_z0 = [&]() {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    z0[t] = L_::template get<3>(s_z, t, 0, lane);
                __builtin_amdgcn_sched_barrier(0);
            };
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                if (s == NS - 1 && !CAREFUL)
                    load_z0();
#pragma unroll
                for (int n = 2; n >= 0; --n)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        R[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kr[s & 1][t].p[0], sf[s].p[n], R[t], 0, 0, 0);
                if (s + 2 < NS) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        kr[s & 1][t] = TK::rows_stacked(s_k, t, s + 2, lane);
                }
            }
            f32x4 x[4], u[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f32x4 v = unit ? f32x4{0.f, 0.f, 0.f, 0.f} : __builtin_convertvector(v4[t], f32x4);
                R[t] = v - row_vec(s_vec, kRise, t, lane) * R[t];
                x[t] = row_vec(s_vec, kBeta, t, lane) * R[t];
                u[t] = f32x4{0.f, 0.f, 0.f, 0.f};
            }
            Spoiled bad;
            if constexpr (CAREFUL) {
                bad.take_out(R, x, g);
                load_z0();      // (before, its registers would spill)
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
                z1[t] = L_::template get<3>(s_z, t + 2, 1, lane);
            __builtin_amdgcn_sched_barrier(0);
            const Frag<3> f0 = split<3>(x[0], x[1]), f1 = split<3>(x[2], x[3]);
#pragma unroll
            for (int o = 2; o >= 0; --o)
#pragma unroll
                for (int i = 0; i <= o; ++i) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        u[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(z0[t].p[i], f0.p[o - i], u[t], 0, 0, 0);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        u[t + 2] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(z1[t].p[i], f1.p[o - i], u[t + 2], 0, 0, 0);
                }
            // two tiles of the state at a time, the next two's k on its way
            Frag<1> kc[2][2][2];
            auto load_kc = [&](int s) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        kc[s & 1][m][i] = TK::columns_stacked(s_k, 2 * s + m, i, lane);
            };
            load_kc(0);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u[t] = R[t] - u[t];      // u~
                if constexpr (MODE == kKeep)
                    Sheet(a.ut + (head * a.NC + c) * kC * a.DV, kC, a.DV, col, lane).put(t, u[t]);
                u[t] *= row_vec(s_vec, kBeta, t, lane);
            }
            if constexpr (CAREFUL) {
                if (g == 0)
                    reinterpret_cast<int *>(lds + LDS::kFrom)[(half * 4 + mine) * 16 + i16] = bad.from;
            }
            if constexpr (MODE == kOut) {
                float *y = reinterpret_cast<float *>(lds + LDS::kU) + (half * 4 + mine) * LDS::kUWave + i16 * LDS::kURow + 4 * g;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    *reinterpret_cast<f32x4 *>(y + 16 * t) = u[t];
            }
            const float whole = bad.whole(s_vec[kWhole * kC]);
            Frag<3> w0, w1;
            w0 = split<3>(row_vec(s_vec, kLeft, 0, lane) * u[0], row_vec(s_vec, kLeft, 1, lane) * u[1]);
            w1 = split<3>(row_vec(s_vec, kLeft, 2, lane) * u[2], row_vec(s_vec, kLeft, 3, lane) * u[3]);
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
                S.s[m] *= whole;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                if (s + 1 < NS)
                    load_kc(s + 1);
#pragma unroll
                for (int n = 2; n >= 0; --n)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            S.s[2 * s + m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                kc[s & 1][m][i].p[0], i ? w1.p[n] : w0.p[n], S.s[2 * s + m], 0, 0, 0);
                sf[s] = split<3>(S.s[2 * s], S.s[2 * s + 1]);
            }
            lds_barrier();
        }
        if constexpr (MODE == kScan) {
            S.store(a.trans + (head * a.segs + seg) * KD * (a.slices * 64 + KD), KD, a.slices * 64 + KD, col, lane);
        } else if constexpr (MODE == kOut) {
            float mark = 0.f;
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    mark = __builtin_fmaf(S.s[m][r], 0.f, mark);
            const bool spoiled = !CAREFUL && __any(mark != 0.f);
            if (lane == 0)
                s_spoiled[mine] = spoiled;
            lds_barrier();
            again = s_spoiled[0] | s_spoiled[1] | s_spoiled[2] | s_spoiled[3];
            // (s_final may be s0, from which a second pass begins)
            if (a.s_final && c1 == a.NC && !again)
                S.store(a.s_final + head * a.Dk * a.Dv, a.Dk, a.Dv, col, lane);
        }
    } else {
        // The help waves have more to do than the chain and share its SIMDs:
        // going first they cut the LM layer's forward from 405 to 380 us (the
        // chain going first: 404).
        __builtin_amdgcn_s_setprio(2);
        const int tid = thread - 256;
        const int64_t ek = b * a.k.s.b + hk * a.k.s.h, eq = b * a.q.s.b + hk * a.q.s.h;
        const int64_t ev = b * a.v.s.b + h * a.v.s.h + (unit ? 0 : slice * 64);
        const int vcols = unit ? a.Dv : a.Dv - slice * 64;
        const float *rec = a.records + head * a.NC * (int64_t)a.record;
        TK tk;
        TV tv;
        L_ tz;
        f32x4 vecs;
        auto fetch = [&](int c) {
            const float *r = rec + (int64_t)c * a.record;
            tk.load(Chunk<true, VEC>(a.k.p, ek, a.k.s.l, c * kC, a.L, a.Dk), tid);
            tz.load(r + Record::kZ, tid);
            tv.load(Chunk<true, VEC>(a.v.p, ev, a.v.s.l, c * kC, a.L, vcols), tid);
            vecs = load_vecs(r + Record::kVec, tid);
        };
        auto stage = [&](int half) {
            tk.store(lds + LDS::kK + half * TK::kSize, tid);
            tz.store(lds + LDS::kZ + half * L_::kSize, tid);
            tv.store(lds + LDS::kV + half * TV::kSize, tid);
            if (tid < kC)
                *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(lds + LDS::kVec) + half * 4 * kC + 4 * tid) = vecs;
        };
        L_::clear(lds + LDS::kZ, tid);
        L_::clear(lds + LDS::kZ + L_::kSize, tid);
        fetch(c0);
        // A chain wave's outputs are shared by two help waves: row tiles 0 and
        // 3, and 1 and 2 (three fragments of P each).
        const int part = (wave - 4) >> 2, ta = part, tb = part ? 2 : 3;
        Unit<true> qf[MODE == kOut ? NS : 1][2];
        f32x4 pf[6], qs[2];
        auto fetch_q = [&](int c) {
            const Chunk<true, VEC> cq(a.q.p, eq, a.q.s.l, c * kC, a.L, a.Dk);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const uint32_t e = cq.lane_at(i16, 32 * s + 8 * g);
                qf[s][0] = cq.unit(e, i16, 16 * ta, 32 * s + 8 * g);
                qf[s][1] = cq.unit(e, i16, 16 * tb, 32 * s + 8 * g);
            }
        };
        // P's blocks (ta, 0), (ta, 1), (tb, 0..3), those right of the diagonal zero
        auto fetch_p = [&](int c) {
            const float *P = rec + (int64_t)c * a.record + Record::kP + 4 * lane;
#pragma unroll
            for (int n = 0; n < 6; ++n) {
                const int row = n < 2 ? ta : tb, cb = n < 2 ? n : n - 2;
                pf[n] = *reinterpret_cast<const f32x4 *>(P + block_of(row, min(cb, row)) * kBlock);
            }
        };
        auto output = [&](int c) {     // from qs, pf and the u of chunk c
            const float *y = reinterpret_cast<const float *>(lds + LDS::kU) + (((c - c0) & 1) * 4 + mine) * LDS::kUWave +
                             i16 * LDS::kURow + 4 * g;
            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
            Frag<3> f[2];
#pragma unroll
            for (int s = 0; s < 2; ++s)
                f[s] = split<3>(*reinterpret_cast<const f32x4 *>(y + 32 * s), *reinterpret_cast<const f32x4 *>(y + 32 * s + 16));
            qs[0] = mma<3>(split<3>(pf[0], part ? pf[1] : zero), f[0], qs[0]);
            qs[1] = mma<3>(split<3>(pf[2], pf[3]), f[0], qs[1]);
            qs[1] = mma<3>(split<3>(pf[4], part ? zero : pf[5]), f[1], qs[1]);
            if constexpr (CAREFUL) {
                const int from = reinterpret_cast<const int *>(lds + LDS::kFrom)[(((c - c0) & 1) * 4 + mine) * 16 + i16];
                Spoiled::put(qs[0], ta, g, from, __builtin_nanf(""));
                Spoiled::put(qs[1], tb, g, from, __builtin_nanf(""));
            }
            const Chunk<true, VEC> co(a.o.p, b * a.o.s.b + h * a.o.s.h, a.o.s.l, max(c, c0) * kC, a.L, a.Dv, c < c0);
            store_cols(co, col, lane, ta, qs[0]);
            store_cols(co, col, lane, tb, qs[1]);
        };
        stage(0);
        fetch(min(c0 + 1, c1 - 1));
        if constexpr (MODE == kOut) {
            fetch_q(c0);
#pragma unroll
            for (int n = 0; n < 6; ++n)
                pf[n] = f32x4{0.f, 0.f, 0.f, 0.f};
            qs[0] = qs[1] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        lds_barrier();
        for (int c = c0; c < c1; ++c) {
            const int half = (c - c0) & 1;
            // No branch on the way: where two paths with other loads in flight
            // meet, a wait for one load becomes a wait for all.  The first turn
            // writes no outputs, the last ones stage the last chunk again.
            stage(half ^ 1);
            fetch(min(c + 2, c1 - 1));
            if constexpr (MODE == kOut) {
                output(c - 1);
                fetch_p(c);
                LdsFlag::await(&s_flag[mine], c + 1);
                const float *x = reinterpret_cast<const float *>(lds + LDS::kS) + mine * LDS::kSWave + i16 * LDS::kSRow + 8 * g;
                qs[0] = qs[1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const Frag<3> f = split<3>(load8(x + 32 * s));
#pragma unroll
                    for (int n = 2; n >= 0; --n)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            qs[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(unit_frag<true>(qf[s][t]).p[0], f.p[n], qs[t], 0, 0, 0);
                }
                const float *s_vec = reinterpret_cast<const float *>(lds + LDS::kVec) + half * 4 * kC;
                qs[0] *= a.scale * row_vec(s_vec, kRise, ta, lane);
                qs[1] *= a.scale * row_vec(s_vec, kRise, tb, lane);
                fetch_q(min(c + 1, c1 - 1));
            }
            lds_barrier();
        }
        if constexpr (MODE == kOut) {
            output(c1 - 1);
            lds_barrier();
            again = s_spoiled[0] | s_spoiled[1] | s_spoiled[2] | s_spoiled[3];
        }
    }
    return again;
}

// A state that is not finite at its end: the walk again, with a look at every
// chunk (which in every walk would cost the LM layer 2 to 13 %, with heads of 128
// 23 %).
template <int KD, bool VEC, int MODE>
__device__ __forceinline__ void pipe_walk(const DeltaArgs &a, unsigned block)
{
    if (pipe_pass<KD, VEC, MODE, false>(a, block, threadIdx.x)) {
        lds_barrier();      // the flags have been read
        // (opaque: nothing formed for one pass is held through the other)
        pipe_pass<KD, VEC, MODE, true>(a, opaque_s(block), opaque(threadIdx.x));
    }
}

// ---------------------------------------------------------------------------
// The walk back, in the same form: the chain waves carry the gradient of the
// state through w, the help waves stage and form what does not depend on it,
// P^T dO before a chunk and Q^T (scale rise dO) during it, handed over as fp32
// tiles in LDS; the chain leaves w and the new gradient in the same places,
// from where the help waves write w, dV and the gradient to memory.  SCAN: the
// gradient before the segment alone, from zero after it.  Both walks of the
// backward's LM layer (4 x 16 heads of 128, 4096 steps, 1.7 GB to and from
// memory by the counters, 4.2 TB/s) take 405 us, 6.3 us a chunk; the chain by
// itself would take 2.9 us.
// ---------------------------------------------------------------------------
template <int KD>
struct BackLds {
    using K = Tile<KD, true, kHelpThreads>;
    using Z = Tri<true, kHelpThreads>;
    // in uint16_t
    static constexpr int kK = 0;
    static constexpr int kQ = kK + 2 * K::kSize;
    static constexpr int kZ = kQ + 2 * K::kSize;
    static constexpr int kVec = kZ + 2 * Z::kSize;
    static constexpr int kFlag = kVec + 4 * 4 * kC * 2;  // four chunks' vectors: the last is still read
    static constexpr int kD = kFlag + 32;               // [4 waves][4 tiles][64 lanes] of f32x4
    static constexpr int kE = kD + 4 * 4 * 64 * 8;      // [4 waves][KD / 16 tiles][64 lanes]
    static constexpr size_t kBytes = (kE + 4 * (KD / 16) * 64 * 8) * 2;
};

template <int KD, bool VEC, bool SCAN>
__device__ __forceinline__ void back_walk(const DeltaArgs &a, unsigned block)
{
    using LDS = BackLds<KD>;
    using TK = typename LDS::K;
    using U_ = typename LDS::Z;
    constexpr int NS = KD / 32, NM = KD / 16;
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    uint16_t *lds = reinterpret_cast<uint16_t *>(s_dyn);
    int *s_flag = reinterpret_cast<int *>(lds + LDS::kFlag);      // [2][2][4]: D, E ready, by either help wave

    const int64_t head = block / (unsigned)(a.segs * a.slices);
    const int rest = block % (unsigned)(a.segs * a.slices), seg = rest / a.slices, slice = rest % a.slices;
    if (SCAN && seg == 0)
        return;
    const int c0 = seg * a.seg_chunks, c1 = min(a.NC, c0 + a.seg_chunks);
    int64_t b;
    int h;
    const int64_t hk = kv_head(a, head, b, h);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15;
    const int mine = wave & 3;
    const int col = (slice * 4 + mine) * 16 + i16;
    f32x4 *s_d = reinterpret_cast<f32x4 *>(lds + LDS::kD) + mine * 4 * 64 + lane;
    f32x4 *s_e = reinterpret_cast<f32x4 *>(lds + LDS::kE) + mine * NM * 64 + lane;

    // Chunk c is step n = c1 - 1 - c of the walk.
    if (wave < 4) {
        State<KD> S;
        if (a.segs > 1 && !SCAN)
            S.load(a.seg_grads + (head * a.segs + seg) * KD * a.DV, KD, a.DV, col, lane);
        else
            S.load(a.ds_final && seg == a.segs - 1 ? a.ds_final + head * a.Dk * a.Dv : nullptr, a.Dk, a.Dv, col, lane);
        Frag<3> sf[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s)
            sf[s] = split<3>(S.s[2 * s], S.s[2 * s + 1]);
        if constexpr (!SCAN) {
#pragma unroll
            for (int m = 0; m < NM; ++m)
                s_e[m * 64] = S.s[m];
        }
        if (lane == 0)
            s_flag[mine] = s_flag[4 + mine] = s_flag[8 + mine] = s_flag[12 + mine] = 0;
        lds_barrier();
        for (int n = 0; n < c1 - c0; ++n) {
            const int half = n & 1;
            const uint16_t *s_k = lds + LDS::kK + half * TK::kSize, *s_z = lds + LDS::kZ + half * U_::kSize;
            const float *s_vec = reinterpret_cast<const float *>(lds + LDS::kVec) + (n & 3) * 4 * kC;
            Frag<1> kr[2][4];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    kr[s][t] = TK::rows_stacked(s_k, t, s, lane);
            __builtin_amdgcn_sched_barrier(0);
            f32x4 d[4], x[4], w[4];
            Frag<3> z0[2], z1[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                d[t] = w[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < NS; ++s) {
#pragma unroll
                for (int o = 2; o >= 0; --o)
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        d[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kr[s & 1][t].p[0], sf[s].p[o], d[t], 0, 0, 0);
                if (s + 2 < NS) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        kr[s & 1][t] = TK::rows_stacked(s_k, t, s + 2, lane);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                z1[t] = U_::template get<3>(s_z, t, 1, lane);
            LdsFlag::await(&s_flag[mine], n + 1);
            LdsFlag::await(&s_flag[4 + mine], n + 1);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                d[t] = s_d[t * 64] + row_vec(s_vec, kLeft, t, lane) * d[t];     // dU
                x[t] = row_vec(s_vec, kBeta, t, lane) * d[t];
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
                z0[t] = U_::template get<3>(s_z, t, 0, lane);
            __builtin_amdgcn_sched_barrier(0);
            const Frag<3> f0 = split<3>(x[0], x[1]), f1 = split<3>(x[2], x[3]);
#pragma unroll
            for (int o = 2; o >= 0; --o)
#pragma unroll
                for (int i = 0; i <= o; ++i) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        w[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(z1[t].p[i], f1.p[o - i], w[t], 0, 0, 0);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        w[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(z0[t].p[i], f0.p[o - i], w[t], 0, 0, 0);
                }
            Frag<1> kc[2][2][2];
            auto load_kc = [&](int s) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        kc[s & 1][m][i] = TK::columns_stacked(s_k, 2 * s + m, i, lane);
            };
            load_kc(0);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                w[t] = d[t] - w[t];
                if constexpr (!SCAN)
                    s_d[t * 64] = w[t];
                w[t] *= -row_vec(s_vec, kBeta, t, lane) * row_vec(s_vec, kRise, t, lane);
            }
            const float whole = s_vec[kWhole * kC];
            const Frag<3> w0 = split<3>(w[0], w[1]), w1 = split<3>(w[2], w[3]);
            LdsFlag::await(&s_flag[8 + mine], n + 1);
            LdsFlag::await(&s_flag[12 + mine], n + 1);
#pragma unroll
            for (int m = 0; m < NM; ++m)
                S.s[m] = S.s[m] * whole + s_e[m * 64];
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                if (s + 1 < NS)
                    load_kc(s + 1);
#pragma unroll
                for (int o = 2; o >= 0; --o)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            S.s[2 * s + m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                kc[s & 1][m][i].p[0], i ? w1.p[o] : w0.p[o], S.s[2 * s + m], 0, 0, 0);
                sf[s] = split<3>(S.s[2 * s], S.s[2 * s + 1]);
                if constexpr (!SCAN) {
#pragma unroll
                    for (int m = 2 * s; m < 2 * s + 2; ++m)
                        s_e[m * 64] = S.s[m];
                }
            }
            lds_barrier();
        }
        if constexpr (SCAN)
            S.store(a.rtrans + (head * a.segs + seg) * KD * (a.slices * 64), KD, a.slices * 64, col, lane);
        else if (a.ds0 && seg == 0)
            S.store(a.ds0 + head * a.Dk * a.Dv, a.Dk, a.Dv, col, lane);
    } else {
        // As in the walk forward, but worth less here: the LM layer's backward
        // takes 807 us, without it 817, with the chain going first 821.
        __builtin_amdgcn_s_setprio(2);
        const int tid = threadIdx.x - 256;
        const int64_t ek = b * a.k.s.b + hk * a.k.s.h, eq = b * a.q.s.b + hk * a.q.s.h;
        const int64_t eo = b * a.d_o.s.b + h * a.d_o.s.h;
        const float *rec = a.records + head * a.NC * (int64_t)a.record;
        TK tk, tq;
        U_ tz;
        f32x4 vecs;
        auto fetch = [&](int c) {
            const float *r = rec + (int64_t)c * a.record;
            tk.load(Chunk<true, VEC>(a.k.p, ek, a.k.s.l, c * kC, a.L, a.Dk), tid);
            tq.load(Chunk<true, VEC>(a.q.p, eq, a.q.s.l, c * kC, a.L, a.Dk), tid);
            tz.load(r + Record::kZt, tid);
            vecs = load_vecs(r + Record::kVec, tid);
        };
        auto stage = [&](int n) {
            const int half = n & 1;
            tk.store(lds + LDS::kK + half * TK::kSize, tid);
            tq.store(lds + LDS::kQ + half * TK::kSize, tid);
            tz.store(lds + LDS::kZ + half * U_::kSize, tid);
            if (tid < kC)
                *reinterpret_cast<f32x4 *>(reinterpret_cast<float *>(lds + LDS::kVec) + (n & 3) * 4 * kC + 4 * tid) = vecs;
        };
        // A chain wave has two help waves: of P^T dO and w they take row tiles 0
        // and 2, and 1 and 3, of the state's tiles the first and second half.
        const int part = (wave - 4) >> 2, ta = part, tb = 2 + part, m0 = part * (NM / 2);
        // P and dO of a chunk, and P^T dO of it
        f32x4 pf[6], pd[2];
        Cols<true> cols;
        auto fetch_o = [&](int c) {
            // blocks (0..3, ta), (2..3, tb), those above the diagonal not used
            const float *P = rec + (int64_t)c * a.record + Record::kP + 4 * lane;
#pragma unroll
            for (int n = 0; n < 6; ++n) {
                const int cb = n < 4 ? ta : tb, row = n < 4 ? n : n - 2;
                pf[n] = *reinterpret_cast<const f32x4 *>(P + block_of(max(row, cb), cb) * kBlock);
            }
            cols.load(Chunk<true, VEC>(a.d_o.p, eo, a.d_o.s.l, c * kC, a.L, a.Dv), col, lane);
        };
        auto product = [&]() {
            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
            const Frag<1> f0 = split<1>(cols.get(0), cols.get(1)), f1 = split<1>(cols.get(2), cols.get(3));
            pd[0] = mma<3>(split<3>(part ? zero : pf[0], pf[1]), f0, zero);
            pd[0] = mma<3>(split<3>(pf[2], pf[3]), f1, pd[0]);
            pd[1] = mma<3>(split<3>(part ? zero : pf[4], pf[5]), f1, zero);
        };
        // w and dV of chunk c, from the chain's w
        auto results = [&](int c, const f32x4 (&w)[2]) {
            const int at = min(c, c1 - 1);
            const Sheet out(a.w + (head * a.NC + at) * kC * a.DV, kC, a.DV, col, lane, c >= c1);
            const Chunk<true, VEC> cv(a.dv.p, b * a.dv.s.b + h * a.dv.s.h, a.dv.s.l, at * kC, a.L, a.Dv, c >= c1);
            const float *s_vec = reinterpret_cast<const float *>(lds + LDS::kVec) + ((c1 - 1 - c) & 3) * 4 * kC;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tile = t ? tb : ta;
                out.put(tile, w[t]);
                store_cols(cv, col, lane, tile, row_vec(s_vec, kBeta, tile, lane) * w[t]);
            }
        };
        U_::clear(lds + LDS::kZ, tid);
        U_::clear(lds + LDS::kZ + U_::kSize, tid);
        fetch(c1 - 1);
        fetch_o(c1 - 1);
        stage(0);
        fetch(max(c1 - 2, c0));
        product();
        lds_barrier();
        for (int n = 0; n < c1 - c0; ++n) {
            const int c = c1 - 1 - n, half = n & 1;
            const uint16_t *s_q = lds + LDS::kQ + half * TK::kSize;
            const float *s_vec = reinterpret_cast<const float *>(lds + LDS::kVec) + (n & 3) * 4 * kC;
            f32x4 w[2];
            if constexpr (!SCAN) {
                w[0] = s_d[ta * 64];    // of the chunk before; the first turn has none
                w[1] = s_d[tb * 64];
            }
            s_d[ta * 64] = pd[0];
            s_d[tb * 64] = pd[1];
            if (lane == 0)
                LdsFlag::set(&s_flag[4 * part + mine], n + 1);
            if constexpr (!SCAN) {
                const Sheet out(a.grads + (head * a.NC + c) * KD * a.DV, KD, a.DV, col, lane);
#pragma unroll
                for (int m = 0; m < NM / 2; ++m)
                    out.put(m0 + m, s_e[(m0 + m) * 64]);
            }
            // Q^T (scale rise dO)
            f32x4 e[NM / 2];
#pragma unroll
            for (int m = 0; m < NM / 2; ++m)
                e[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag<3> f = split<3>(a.scale * row_vec(s_vec, kRise, 2 * s, lane) * cols.get(2 * s),
                                           a.scale * row_vec(s_vec, kRise, 2 * s + 1, lane) * cols.get(2 * s + 1));
                Frag<1> qc[NM / 2];
#pragma unroll
                for (int m = 0; m < NM / 2; ++m)
                    qc[m] = TK::columns_stacked(s_q, m0 + m, s, lane);
#pragma unroll
                for (int o = 2; o >= 0; --o)
#pragma unroll
                    for (int m = 0; m < NM / 2; ++m)
                        e[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qc[m].p[0], f.p[o], e[m], 0, 0, 0);
            }
#pragma unroll
            for (int m = 0; m < NM / 2; ++m)
                s_e[(m0 + m) * 64] = e[m];
            if (lane == 0)
                LdsFlag::set(&s_flag[8 + 4 * part + mine], n + 1);
            // Loads wait for a turn of the walk before their use and come
            // before its stores: the counter that a load is waited for by
            // runs in order over both.
            fetch_o(max(c - 1, c0));
            stage(n + 1);
            product();
            fetch(max(c - 2, c0));
            if constexpr (!SCAN)
                results(c + 1, w);
            lds_barrier();
        }
        if constexpr (!SCAN) {
            const f32x4 w[2] = {s_d[ta * 64], s_d[tb * 64]};
            results(c0, w);
        }
    }
}

template <int KD, bool VEC, int MODE>
__global__ void __launch_bounds__(kPipeThreads, 1) pipe_kernel(DeltaArgs a)
{
    pipe_walk<KD, VEC, MODE>(a, blockIdx.x);
}

// The backward's walks: neither needs the other, so both are one launch, the
// first `back_blocks` workgroups walking back.
template <int KD, bool VEC, bool SCAN>
__global__ void __launch_bounds__(kPipeThreads, 1) back_kernel(DeltaArgs a)
{
    if (blockIdx.x < a.back_blocks)
        back_walk<KD, VEC, SCAN>(a, blockIdx.x);
    else
        pipe_walk<KD, VEC, SCAN ? kScan : kKeep>(a, blockIdx.x - a.back_blocks);
}

// ---------------------------------------------------------------------------
// join_kernel: the states before the segments of a head, from s0 and the
// segments' transitions A and ends B: S <- A S + B; behind those workgroups
// (in the backward) the state gradients after the segments, from the last to
// the first: dS <- A^T dS + C.  s0 and ds_final are copied too: the last
// launch writes s_final (or ds0) by other workgroups than those that begin
// from s0 (ds_final), and the two may be one buffer.  A workgroup owns 16 columns, each of its waves 32 rows:
// these rows of A go from memory to the wave's registers, the next two
// segments' while this one's products run, and only the state's parts pass through LDS.
// Bound by the wait for A: 49 us for 16 segments of 128 x 128 and 8 heads,
// 3.5 a segment; with one segment under way 57; a workgroup of 64 columns
// taking all of A through LDS 101.  Every workgroup splits A again, which its
// waves do side by side.
// ---------------------------------------------------------------------------
template <int KD>
struct JoinLds {
    static constexpr int kWaves = KD / 32, kThreads = 64 * kWaves;
    static constexpr size_t kBytes = 2 * kWaves * 3 * 64 * sizeof(bf16x8);     // two turns of the state's parts
};

template <int N>
struct Slot {
    static constexpr int value = N;
};

template <int KD>
__global__ void __launch_bounds__(JoinLds<KD>::kThreads, 1) join_kernel(DeltaArgs a)
{
    constexpr int kWaves = JoinLds<KD>::kWaves;
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    bf16x8 *s_f = reinterpret_cast<bf16x8 *>(s_dyn);
    const unsigned heads = (unsigned)a.heads, half = heads * (unsigned)((a.DV + 15) / 16);
    const bool back = blockIdx.x >= half;
    const unsigned block = blockIdx.x - (back ? half : 0u);
    // A head's workgroups stand a.heads apart: for a multiple of eight heads
    // on one XCD, whose L2 then serves all but the first reader of A.
    const int64_t head = block % heads;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i16 = lane & 15;
    const int col = (int)(block / heads) * 16 + i16, ends = a.slices * 64, pitch = ends + KD;
    const float *T = a.trans + head * a.segs * KD * (int64_t)pitch;
    const float *C = a.rtrans + head * a.segs * KD * (int64_t)ends;

    f32x4 u[2][2][kWaves][2], N[2][2], S[2];     // two segments on their way
    auto get = [&](f32x4 (&to)[2], const float *p, int width) {
        const Sheet from(p, KD, width, col, lane);
#pragma unroll
        for (int t = 0; t < 2; ++t)
            to[t] = from.get(2 * wave + t);
    };
    // The wave's rows of the segment's A (or of its transpose), and its end B or C.
    auto seg_of = [&](int n) { return back ? a.segs - 1 - n : n; };
    auto fetch = [&](int n, auto slot) {
        if (n + 1 >= a.segs)
            return;
        const int seg = seg_of(n);
        const float *A = T + (int64_t)seg * KD * pitch + ends;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int row = 32 * wave + 16 * t + i16;
#pragma unroll
            for (int s = 0; s < kWaves; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k = 32 * s + 16 * h + 4 * g;
                    if (back) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            u[slot.value][t][s][h][j] = A[(k + j) * pitch + row];
                    } else {
                        u[slot.value][t][s][h] = *reinterpret_cast<const f32x4 *>(A + row * pitch + k);
                    }
                }
        }
        if (back)
            get(N[slot.value], C + (int64_t)seg * KD * ends, ends);
        else
            get(N[slot.value], A - ends, pitch);
    };
    auto put = [&](int n, const f32x4 (&v)[2]) {
        const Sheet to((back ? a.seg_grads : a.seg_states) + (head * a.segs + seg_of(n)) * KD * a.DV, KD, a.DV, col, lane);
#pragma unroll
        for (int t = 0; t < 2; ++t)
            to.put(2 * wave + t, v[t]);
    };
    const float *start = back ? a.ds_final : a.s0;
    const Sheet first(start ? start + head * a.Dk * a.Dv : nullptr, start ? a.Dk : 0, a.Dv, col, lane);
#pragma unroll
    for (int t = 0; t < 2; ++t)
        S[t] = first.get(2 * wave + t);
    put(0, S);
    if (back)
        get(S, C + (int64_t)(a.segs - 1) * KD * ends, ends);
    else
        get(S, T, pitch);
    fetch(1, Slot<0>{});
    fetch(2, Slot<1>{});
    auto step = [&](int n, auto slot) {
        put(n, S);
        if (n + 1 >= a.segs)
            return false;
        bf16x8 *turn = s_f + (n & 1) * kWaves * 3 * 64 + lane;
        const Frag<3> mine = split<3>(S[0], S[1]);
#pragma unroll
        for (int i = 0; i < 3; ++i)
            turn[(wave * 3 + i) * 64] = mine.p[i];
        Frag<3> p[2][kWaves];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            S[t] = N[slot.value][t];
#pragma unroll
            for (int s = 0; s < kWaves; ++s)
                p[t][s] = split<3>(u[slot.value][t][s][0], u[slot.value][t][s][1]);
        }
        fetch(n + 2, slot);
        // The one barrier of a step: what is written two steps on has been
        // read by every wave before the next step's.
        lds_barrier();
#pragma unroll
        for (int s = 0; s < kWaves; ++s) {
            Frag<3> f;
#pragma unroll
            for (int i = 0; i < 3; ++i)
                f.p[i] = turn[(s * 3 + i) * 64];
#pragma unroll
            for (int o = 2; o >= 0; --o)
#pragma unroll
                for (int i = 0; i <= o; ++i)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        S[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p[t][s].p[i], f.p[o - i], S[t], 0, 0, 0);
        }
        return true;
    };
    for (int n = 1; step(n, Slot<0>{}) && step(n + 1, Slot<1>{}); n += 2)
        ;
}

// ---------------------------------------------------------------------------
// reverse_kernel: the chunks of a head from the last to the first, with the
// gradient of the state in registers.  Writes dV, keeps w and the gradients
// of the states after the chunks.
// ---------------------------------------------------------------------------
template <int KD, bool VEC>
__global__ void __launch_bounds__(kThreads) reverse_kernel(DeltaArgs a)
{
    constexpr bool BF16 = false;
    using T = Tile<KD, BF16>;
    using U_ = Tri<true>;
    constexpr int NK = T::NK;
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    uint16_t *s_k = reinterpret_cast<uint16_t *>(s_dyn);
    uint16_t *s_z = s_k + T::kSize;
    float *s_vec = reinterpret_cast<float *>(s_z + U_::kSize);
    uint16_t *s_q = reinterpret_cast<uint16_t *>(s_vec + 4 * kC);
    uint16_t *s_p = s_q + T::kSize;

    const int64_t head = blockIdx.x / (unsigned)a.slices;
    const int slice = blockIdx.x % (unsigned)a.slices;
    int64_t b;
    int h;
    const int64_t hk = kv_head(a, head, b, h);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = (slice * (kThreads / 64) + wave) * 16 + (lane & 15);
    const int64_t ek = b * a.k.s.b + hk * a.k.s.h, eq = b * a.q.s.b + hk * a.q.s.h;
    const int64_t eo = b * a.d_o.s.b + h * a.d_o.s.h, ev = b * a.dv.s.b + h * a.dv.s.h;
    const float *rec = a.records + head * a.NC * (int64_t)a.record;

    T tk, tq;
    U_ tz, tp;
    Cols<BF16> v;
    f32x4 tv;
    auto fetch = [&](int c) {
        const float *r = rec + (int64_t)c * a.record;
        tk.load(Chunk<BF16, VEC>(a.k.p, ek, a.k.s.l, c * kC, a.L, a.Dk), threadIdx.x);
        tq.load(Chunk<BF16, VEC>(a.q.p, eq, a.q.s.l, c * kC, a.L, a.Dk), threadIdx.x);
        tz.load(r + Record::kZt, threadIdx.x);
        tp.load(r + Record::kP, threadIdx.x);
        tv = load_vecs(r + Record::kVec, threadIdx.x);
        v.load(Chunk<BF16, VEC>(a.d_o.p, eo, a.d_o.s.l, c * kC, a.L, a.Dv), col, lane);
    };
    State<KD> S;
    S.load(a.ds_final ? a.ds_final + head * a.Dk * a.Dv : nullptr, a.Dk, a.Dv, col, lane);
    U_::clear(s_z, threadIdx.x);
    U_::clear(s_p, threadIdx.x);
    fetch(a.NC - 1);
    for (int c = a.NC - 1; c >= 0; --c) {
        tk.store(s_k, threadIdx.x);
        tq.store(s_q, threadIdx.x);
        tz.store(s_z, threadIdx.x);
        tp.store(s_p, threadIdx.x);
        if (threadIdx.x < kC)
            *reinterpret_cast<f32x4 *>(s_vec + 4 * threadIdx.x) = tv;
        f32x4 dO[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            dO[t] = v.get(t);
        lds_barrier();
        if (c > 0)
            fetch(c - 1);

        {
            const Sheet out(a.grads + (head * a.NC + c) * KD * a.DV, KD, a.DV, col, lane);
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
                out.put(m, S.s[m]);
        }
        f32x4 dU[4], x[4], w[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            dU[t] = w[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KD / 32; ++s) {
            const Frag<3> f = split<3>(S.s[2 * s], S.s[2 * s + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                dU[t] = mma<3>(T::rows_stacked(s_k, t, s, lane), f, dU[t]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
            dU[t] *= row_vec(s_vec, kLeft, t, lane);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Frag<NK> f = split<NK>(dO[2 * s], dO[2 * s + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (U_::has(t, s))
                    dU[t] = mma<3>(U_::template get<3>(s_p, t, s, lane), f, dU[t]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
            x[t] = row_vec(s_vec, kBeta, t, lane) * dU[t];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Frag<3> f = split<3>(x[2 * s], x[2 * s + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (U_::has(t, s))
                    w[t] = mma<3>(U_::template get<3>(s_z, t, s, lane), f, w[t]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            w[t] = dU[t] - w[t];
            Sheet(a.w + (head * a.NC + c) * kC * a.DV, kC, a.DV, col, lane).put(t, w[t]);
            w[t] *= row_vec(s_vec, kBeta, t, lane);     // dV
            store_cols(Chunk<BF16, VEC>(a.dv.p, ev, a.dv.s.l, c * kC, a.L, a.Dv), col, lane, t, w[t]);
            w[t] *= -row_vec(s_vec, kRise, t, lane);
            dO[t] *= a.scale * row_vec(s_vec, kRise, t, lane);
        }
        const float whole = s_vec[kWhole * kC];
#pragma unroll
        for (int m = 0; m < KD / 16; ++m)
            S.s[m] *= whole;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Frag<3> fo = split<3>(dO[2 * s], dO[2 * s + 1]), fw = split<3>(w[2 * s], w[2 * s + 1]);
#pragma unroll
            for (int m = 0; m < KD / 16; ++m) {
                S.s[m] = mma<3>(T::columns_stacked(s_q, m, s, lane), fo, S.s[m]);
                S.s[m] = mma<3>(T::columns_stacked(s_k, m, s, lane), fw, S.s[m]);
            }
        }
        lds_barrier();
    }
    if (a.ds0)
        S.store(a.ds0 + head * a.Dk * a.Dv, a.Dk, a.Dv, col, lane);
}

// ---------------------------------------------------------------------------
// grad_kernel: dQ and dK of a chunk of one key head (summed over the value
// heads of its group), and dg and dbeta of each of those.  Wave w forms row
// tile w of X and Y (sums over the state's columns), then all rows of the
// KD / 4 key dimensions that it owns.
// ---------------------------------------------------------------------------
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

template <int KD, bool VEC>
__global__ void __launch_bounds__(kThreads) grad_kernel(DeltaArgs a)
{
    constexpr bool BF16 = false;
    using T = Tile<KD, BF16>;
    using M = Tile<kC, BF16>;           // X and Y: 64 x 64
    constexpr int NK = T::NK;
    constexpr int NO = 3;
    constexpr int NM = M::NK;           // parts of X and Y
    constexpr int NTC = KD / 64;        // 16-column tiles of a wave
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    uint16_t *s_k = reinterpret_cast<uint16_t *>(s_dyn);
    uint16_t *s_q = s_k + T::kSize;
    uint16_t *s_x = s_q + T::kSize;
    uint16_t *s_y = s_x + M::kSize;
    float *s_vec = reinterpret_cast<float *>(s_y + M::kSize);         // the record's vectors
    float *s_reads = s_vec + kVecs * kC;                              // [4][64]: what the steps read of S, by wave
    float *s_cuts = s_reads + 4 * kC;
    float *s_sum = s_cuts + Cuts::kSize;                              // [4]: <S, dS> by wave
    // [64][4]: what the steps write, by wave, in the padding of k's first part
    auto s_writes = [&](int row) { return reinterpret_cast<float *>(s_k + row * T::kRow + KD); };

    const int64_t chunk = blockIdx.x % (unsigned)a.NC, bk = blockIdx.x / (unsigned)a.NC;
    const int c = (int)chunk;
    const int64_t b = bk / a.Hk;
    const int hk = (int)(bk - b * a.Hk), group = a.Hv / a.Hk;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i16 = lane & 15;
    const int t0 = c * kC;

    {
        T tk, tq;
        tk.load(Chunk<BF16, VEC>(a.k.p, b * a.k.s.b + hk * a.k.s.h, a.k.s.l, t0, a.L, a.Dk), threadIdx.x);
        tq.load(Chunk<BF16, VEC>(a.q.p, b * a.q.s.b + hk * a.q.s.h, a.q.s.l, t0, a.L, a.Dk), threadIdx.x);
        tk.store(s_k, threadIdx.x);
        tq.store(s_q, threadIdx.x);
    }
    f32x4 dq[4][NTC], dk[4][NTC];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < NTC; ++n)
            dq[t][n] = dk[t][n] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int j = 0; j < group; ++j) {
        const int h = hk * group + j;
        const int64_t head = b * a.Hv + h, at = head * a.NC + c;
        const float *rec = a.records + at * a.record;
        const float *ut = a.ut + at * kC * a.DV, *w = a.w + at * kC * a.DV;
        const float *S = a.states + at * KD * a.DV, *dS = a.grads + at * KD * a.DV;
        const Chunk<BF16, VEC> cdo(a.d_o.p, b * a.d_o.s.b + h * a.d_o.s.h, a.d_o.s.l, t0, a.L, a.Dv);

        for (int x = threadIdx.x; x < kVecs * kC; x += kThreads)
            s_vec[x] = rec[Record::kVec + x];
        __syncthreads();

        // Row tile `wave` of X and Y; rows' sums.  (Places in LDS from numbers
        // of this turn, or those of all phases are formed ahead of the loop over
        // j and held in registers that spill.)
        {
            const int ln = opaque(lane), x_at = opaque((16 * wave + 4 * g) * M::kRow + i16);
            const int row = 16 * wave + i16, t = t0 + row;
            f32x4 dp[4], dn[4];
#pragma unroll
            for (int tb = 0; tb < 4; ++tb)
                dp[tb] = dn[tb] = f32x4{0.f, 0.f, 0.f, 0.f};
            float uw = 0.f;
            for (int d0 = 0; d0 < a.DV; d0 += 32) {
                const int col = d0 + 8 * g;
                const Frag<NK> fo = unit_frag<BF16>(cdo.unit(row, col));
                const f32x8 wv = load8(w + row * a.DV + col);
                const Frag<NO> fw = split<NO>(wv);
#pragma unroll
                for (int tb = 0; tb < 4; ++tb) {
                    if (tb > wave)
                        continue;
                    const f32x8 uv = load8(ut + (16 * tb + i16) * a.DV + col);
                    if (tb == wave)
                        uw = dot8(uv, wv, uw);
                    const Frag<3> fu = split<3>(uv);
                    dp[tb] = mma<3>(fo, fu, dp[tb]);
                    dn[tb] = mma<NO>(fw, fu, dn[tb]);
                }
            }
            uw += __shfl_xor(uw, 16, 64);
            uw += __shfl_xor(uw, 32, 64);
            if (g == 0 && t < a.L)
                static_cast<float *>(const_cast<void *>(a.dbeta.p))[b * a.dbeta.s.b + h * a.dbeta.s.h + t * a.dbeta.s.l] = uw;
            // X, Y in rows 16 wave + 4 g + r, columns 16 tb + i16
#pragma unroll
            for (int tb = 0; tb < 4; ++tb) {
                const int jc = 16 * tb + i16;
                f32x4 xx = {0.f, 0.f, 0.f, 0.f}, yy = xx;
                if (tb <= wave) {
                    f32x4 kk = {0.f, 0.f, 0.f, 0.f}, m = kk;
#pragma unroll
                    for (int s = 0; s < KD / 32; ++s)
                        kk = mma<3>(T::rows(s_k, wave, s, ln), T::rows(s_k, tb, s, ln), kk);
                    const float bj = s_vec[kBeta * kC + jc];
                    const f32x4 P = *reinterpret_cast<const f32x4 *>(rec + Record::kP + block_of(wave, tb) * kBlock + 4 * lane);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int ic = 16 * wave + 4 * g + r;
                        const float d = decay_of(s_vec[kGhi * kC + ic], s_vec[kGlo * kC + ic], s_vec[kResets * kC + ic],
                                                 s_vec[kGhi * kC + jc], s_vec[kGlo * kC + jc], s_vec[kResets * kC + jc]) * bj;
                        xx[r] = jc <= ic ? a.scale * dp[tb][r] * d : 0.f;
                        yy[r] = jc < ic ? -dn[tb][r] * s_vec[kBeta * kC + ic] * d : 0.f;
                        m[r] = jc < ic ? dp[tb][r] * bj * P[r] + yy[r] * kk[r] : 0.f;
                    }
                    Cuts::put(s_cuts, wave, tb, m, ln);
                }
#pragma unroll
                for (int n = 0; n < NM; ++n) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int p = x_at + n * M::kPart + r * M::kRow + 16 * tb;
                        const uint16_t hx = f32_to_bf16_rne(xx[r]), hy = f32_to_bf16_rne(yy[r]);
                        s_x[p] = hx;
                        s_y[p] = hy;
                        xx[r] -= bf16_lo(hx);
                        yy[r] -= bf16_lo(hy);
                    }
                }
            }
        }
        __syncthreads();

        // The wave's key dimensions.
        const int ln = opaque(lane), row4 = opaque(4 * g);
        f32x4 reads[4], writes[4];
        float ss = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            reads[t] = writes[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NTC; ++n) {
            const int tile = wave * NTC + n, dim = 16 * tile + i16;
            f32x4 e[4], f[4], k2[4];        // dO S^T, w S^T, u~ dS^T
#pragma unroll
            for (int t = 0; t < 4; ++t)
                e[t] = f[t] = k2[t] = f32x4{0.f, 0.f, 0.f, 0.f};
            for (int d0 = 0; d0 < a.DV; d0 += 32) {
                const int col = d0 + 8 * g;
                const f32x8 sv = load8(S + dim * a.DV + col), dv = load8(dS + dim * a.DV + col);
                ss = dot8(sv, dv, ss);
                const Frag<3> fs = split<3>(sv), fd = split<3>(dv);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int row = 16 * t + i16;
                    const Frag<NK> fo = unit_frag<BF16>(cdo.unit(row, col));
                    e[t] = mma<3>(fo, fs, e[t]);
                    f[t] = mma<NO>(split<NO>(load8(w + row * a.DV + col)), fs, f[t]);
                    k2[t] = mma<3>(split<3>(load8(ut + row * a.DV + col)), fd, k2[t]);
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f32x4 rise = row_vec(s_vec, kRise, t, lane), beta = row_vec(s_vec, kBeta, t, lane);
                e[t] *= a.scale * rise;
                f[t] *= beta * rise;
                k2[t] *= beta * row_vec(s_vec, kLeft, t, lane);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int p = (16 * t + row4 + r) * T::kRow + dim;
                    float qv = 0.f, kv = 0.f;
#pragma unroll
                    for (int m = NK - 1; m >= 0; --m) {
                        qv += bf16_lo(s_q[m * T::kPart + p]);
                        kv += bf16_lo(s_k[m * T::kPart + p]);
                    }
                    reads[t][r] += qv * e[t][r] - kv * f[t][r];
                    writes[t][r] += kv * k2[t][r];
                }
                dq[t][n] += e[t];
                dk[t][n] += k2[t] - f[t];
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const Frag<NK> fk = T::columns(s_k, tile, s, ln), fq = T::columns(s_q, tile, s, ln);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (s <= t / 2) {
                        dq[t][n] = mma<3>(M::rows(s_x, t, s, ln), fk, dq[t][n]);
                        dk[t][n] = mma<3>(M::rows(s_y, t, s, ln), fk, dk[t][n]);
                    }
                    if (s >= t / 2) {
                        dk[t][n] = mma<3>(M::columns(s_x, t, s, ln), fq, dk[t][n]);
                        dk[t][n] = mma<3>(M::columns(s_y, t, s, ln), fk, dk[t][n]);
                    }
                }
            }
        }
        ss *= s_vec[kWhole * kC];
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1)
            ss += __shfl_xor(ss, m, 64);
        if (lane == 0)
            s_sum[wave] = ss;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float x = sum16(reads[t][r]), y = sum16(writes[t][r]);
                const int row = 16 * t + row4 + r;
                if (i16 == 0) {
                    s_reads[wave * kC + row] = x;
                    s_writes(row)[wave] = y;
                }
            }
        __syncthreads();
        if (wave == 0) {
            const float *w = s_writes(lane);
            float reads = 0.f;
#pragma unroll
            for (int m = 0; m < 4; ++m)
                reads += s_reads[m * kC + lane];
            const float v = crossing(s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3], reads, w[0] + w[1] + w[2] + w[3], s_cuts, lane);
            // the decay of an empty state does nothing
            const bool empty = s_vec[kResets * kC + lane] != (lane ? s_vec[kResets * kC + lane - 1] : 0.f) ||
                               (t0 + lane == 0 && !a.s0);
            if (t0 + lane < a.L)
                static_cast<float *>(const_cast<void *>(a.dg.p))[b * a.dg.s.b + h * a.dg.s.h + (t0 + lane) * a.dg.s.l] =
                    empty ? 0.f : v;
        }
        __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < NTC; ++n)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int dim = 16 * (wave * NTC + n) + i16;
            store_cols(Chunk<BF16, VEC>(a.dq.p, b * a.dq.s.b + hk * a.dq.s.h, a.dq.s.l, t0, a.L, a.Dk), dim, lane, t, dq[t][n]);
            store_cols(Chunk<BF16, VEC>(a.dk.p, b * a.dk.s.b + hk * a.dk.s.h, a.dk.s.l, t0, a.L, a.Dk), dim, lane, t, dk[t][n]);
        }
}

// ---------------------------------------------------------------------------
// grads_kernel: grad_kernel for bf16 data, eight waves.  u~, w (three parts
// each) and dO of the chunk go through LDS once, each row's dot products falling
// out on the way; a wave takes the 16 key dimensions it owns (with 64 of them:
// half of the rows each), reading the state and its gradient straight into the
// product's layout, two k steps ahead, then one or two 16 x 16 blocks of X and
// Y, whose three parts take the place of u~ and w.  357 to 391 us for 4096 chunks
// of 128 x 128 (2.8 to 3.0 TB/s of the 1.09 GB that the counters show): its 160 KB
// of LDS leave one workgroup to a compute unit, so loads and products of a chunk
// do not overlap with another's.
// ---------------------------------------------------------------------------
constexpr int kGradThreads = 512;

template <int KD, int KV>
struct GradLds {
    using K = Tile<KD, true, kGradThreads>;
    using V = Tile<KV, true, kGradThreads>;     // one part of 64 rows of KV values
    using M = Tile<kC, false, kGradThreads>;    // X or Y, three parts
    static constexpr int kWaves = kGradThreads / 64;
    // in uint16_t
    static constexpr int kQ = K::kSize;
    static constexpr int kU = kQ + K::kSize;
    static constexpr int kW = kU + 3 * V::kPart;
    static constexpr int kO = kW + 3 * V::kPart;
    static constexpr int kX = kU;               // once u~ and w have been read
    static constexpr int kY = kX + M::kSize;
    static_assert(kY + M::kSize <= kO, "X and Y take the place of u~ and w");
    static constexpr int kVec = kO + V::kPart;
    static constexpr int kReads = kVec + 2 * kVecs * kC;        // [KD / 16][64]: what the steps read of S
    static constexpr int kWrites = kReads + 2 * (KD / 16) * kC; // [KD / 16][64]: and write behind the chunk
    static constexpr int kCuts = kWrites + 2 * (KD / 16) * kC;
    static constexpr int kSum = kCuts + 2 * Cuts::kSize;        // [waves]: <S, dS>
    static constexpr size_t kBytes = (kSum + 2 * kWaves) * 2;
};

// Four values of a column, three parts, into rows p, p + M::kRow, ...
template <typename M>
__device__ __forceinline__ void put_rows(uint16_t *p, f32x4 v)
{
    float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
            const uint32_t w = take_part(x[r], x[r + 1], n < 2);
            p[n * M::kPart + r * M::kRow] = (uint16_t)w;
            p[n * M::kPart + (r + 1) * M::kRow] = (uint16_t)(w >> 16);
        }
}

template <int KD, int KV, bool VEC>
__global__ void __launch_bounds__(kGradThreads, 1) grads_kernel(DeltaArgs a)
{
    using LDS = GradLds<KD, KV>;
    using TK = typename LDS::K;
    using TV = typename LDS::V;
    using M = typename LDS::M;
    constexpr int kTiles = KD / 16, RG = LDS::kWaves / kTiles, NT = 4 / RG;    // row groups, row tiles of a wave
    constexpr int kUnits = kC * (KV / 8) / kGradThreads;
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    uint16_t *lds = reinterpret_cast<uint16_t *>(s_dyn);
    uint16_t *s_k = lds, *s_q = lds + LDS::kQ, *s_u = lds + LDS::kU, *s_w = lds + LDS::kW, *s_o = lds + LDS::kO;
    uint16_t *s_x = lds + LDS::kX, *s_y = lds + LDS::kY;
    float *s_vec = reinterpret_cast<float *>(lds + LDS::kVec), *s_cuts = reinterpret_cast<float *>(lds + LDS::kCuts);
    float *s_reads = reinterpret_cast<float *>(lds + LDS::kReads), *s_writes = reinterpret_cast<float *>(lds + LDS::kWrites);
    float *s_sum = reinterpret_cast<float *>(lds + LDS::kSum);

    const int c = (int)(blockIdx.x % (unsigned)a.NC);
    const int64_t bk = blockIdx.x / (unsigned)a.NC, b = bk / a.Hk;
    const int hk = (int)(bk - b * a.Hk), group = a.Hv / a.Hk, t0 = c * kC;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, i16 = lane & 15;
    const int tile = wave % kTiles, first = wave / kTiles * NT, dim = 16 * tile + i16;

    // What a value head adds: its units of u~, w, dO, and the state and its
    // gradient in the layout of the products.
    f32x8 u[kUnits], ww[kUnits], sv[2], dv[2];      // two k steps of the states at a time
    Unit<true> o[kUnits];
    float vecs;
    auto fetch = [&](int j) {
        const int h = hk * group + j;
        const int64_t at = (b * a.Hv + h) * a.NC + c;
        const float *rec = a.records + at * a.record;
        const float *ut = a.ut + at * kC * a.DV, *w = a.w + at * kC * a.DV;
        const Chunk<true, VEC> cdo(a.d_o.p, b * a.d_o.s.b + h * a.d_o.s.h, a.d_o.s.l, t0, a.L, a.Dv);
        const f32x8 zero = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int x = tid + i * kGradThreads, row = x / (KV / 8), col = x % (KV / 8) * 8;
            const int at8 = row * a.DV + min(col, a.DV - 8);
            u[i] = col < a.DV ? load8(ut + at8) : zero;
            ww[i] = col < a.DV ? load8(w + at8) : zero;
            o[i] = cdo.unit(row, col);
        }
        vecs = rec[Record::kVec + min(tid, kVecs * kC - 1)];
    };
    auto fetch_state = [&](int j, int s) {
        const int64_t at = (b * a.Hv + hk * group + j) * a.NC + c;
        const int e = dim * a.DV + min(32 * s, a.DV - 32) + 8 * g;
        sv[s & 1] = load8(a.states + at * KD * a.DV + e);
        dv[s & 1] = load8(a.grads + at * KD * a.DV + e);
    };
    {
        TK tk, tq;
        tk.load(Chunk<true, VEC>(a.k.p, b * a.k.s.b + hk * a.k.s.h, a.k.s.l, t0, a.L, a.Dk), tid);
        tq.load(Chunk<true, VEC>(a.q.p, b * a.q.s.b + hk * a.q.s.h, a.q.s.l, t0, a.L, a.Dk), tid);
        tk.store(s_k, tid);
        tq.store(s_q, tid);
    }
    f32x4 dq[NT], dk[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        dq[t] = dk[t] = f32x4{0.f, 0.f, 0.f, 0.f};

    for (int j = 0; j < group; ++j) {
        const int h = hk * group + j;
        const float *rec = a.records + ((b * a.Hv + h) * a.NC + c) * a.record;
        fetch(j);
        fetch_state(j, 0);
        fetch_state(j, 1);
        if (tid < kVecs * kC)
            s_vec[tid] = vecs;
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int x = tid + i * kGradThreads, row = x / (KV / 8), col = x % (KV / 8) * 8;
            const int p = row * TV::kRow + col;
            put_parts<3>(s_u + p, TV::kPart, u[i]);
            put_parts<3>(s_w + p, TV::kPart, ww[i]);
            *reinterpret_cast<uint4 *>(s_o + p) = o[i].v;
            float uw = dot8(u[i], ww[i], 0.f);
            if constexpr (KV == 128) {      // a row's units are a group of 16 lanes, or of 8
                uw = sum16(uw);
            } else {
#pragma unroll
                for (int m = 4; m >= 1; m >>= 1)
                    uw += __shfl_xor(uw, m, 64);
            }
            if (col == 0 && t0 + row < a.L)
                static_cast<float *>(const_cast<void *>(a.dbeta.p))[b * a.dbeta.s.b + h * a.dbeta.s.h +
                                                                    (t0 + row) * a.dbeta.s.l] = uw;
        }
        lds_barrier();

        // The wave's key dimensions.
        f32x4 e[NT], f[NT], k2[NT];     // dO S^T, w S^T, u~ dS^T
        float ss = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
            e[t] = f[t] = k2[t] = f32x4{0.f, 0.f, 0.f, 0.f};
        // (Places in LDS from a number of this turn, or those of all phases are
        // formed ahead of the loop over j and held in registers that spill.)
        const int at = opaque(i16 * TV::kRow + 8 * g);
        const int row_at = opaque(tile * kC + 16 * first + 4 * g);
        const int qk_at = opaque((4 * g + (i16 >> 2)) * TK::kRow + 16 * tile + 4 * (i16 & 3));
#pragma unroll
        for (int s = 0; s < KV / 32; ++s) {
            if (32 * s >= a.DV)
                break;
            if (first == 0)
                ss = dot8(sv[s & 1], dv[s & 1], ss);
            const Frag<3> fs = split<3>(sv[s & 1]), fd = split<3>(dv[s & 1]);
            if (s + 2 < KV / 32)
                fetch_state(j, s + 2);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int p = at + 16 * (first + t) * TV::kRow + 32 * s;
                Frag<1> fo;
                Frag<3> fw;
                Frag<3> fu;
                fo.p[0] = lds_row8(s_o + p);
#pragma unroll
                for (int n = 0; n < 3; ++n)
                    fu.p[n] = lds_row8(s_u + n * TV::kPart + p);
#pragma unroll
                for (int n = 0; n < 3; ++n)
                    fw.p[n] = lds_row8(s_w + n * TV::kPart + p);
                e[t] = mma<3>(fo, fs, e[t]);
                f[t] = mma<3>(fw, fs, f[t]);
                k2[t] = mma<3>(fu, fd, k2[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const f32x4 rise = row_vec(s_vec, kRise, first + t, lane), beta = row_vec(s_vec, kBeta, first + t, lane);
            e[t] *= a.scale * rise;
            f[t] *= beta * rise;
            k2[t] *= beta * row_vec(s_vec, kLeft, first + t, lane);
            const int p = qk_at + 16 * (first + t) * TK::kRow;
            const f32x4 qv = __builtin_convertvector(lds_column4(s_q + p), f32x4);
            const f32x4 kv = __builtin_convertvector(lds_column4(s_k + p), f32x4);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float x = sum16(qv[r] * e[t][r] - kv[r] * f[t][r]), y = sum16(kv[r] * k2[t][r]);
                if (i16 == 0) {
                    s_reads[row_at + 16 * t + r] = x;
                    s_writes[row_at + 16 * t + r] = y;
                }
            }
            dq[t] += e[t];
            dk[t] += k2[t] - f[t];
        }
        ss *= s_vec[kWhole * kC];
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1)
            ss += __shfl_xor(ss, m, 64);
        if (lane == 0)
            s_sum[wave] = ss;
        // Blocks of X and Y: one of the ten for each wave, a second for two of
        // them; after the key dimensions, whose sums hold more registers.
        __builtin_amdgcn_sched_barrier(0);
        const int ln = opaque(lane);
        f32x4 x[2], y[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int t = wave + n * LDS::kWaves;
            if (t >= kBlocks)
                break;
            const int ta = row_of(t), tb = t - block_of(ta, 0);
            const f32x4 P = *reinterpret_cast<const f32x4 *>(rec + Record::kP + t * kBlock + 4 * lane);
            f32x4 dp = {0.f, 0.f, 0.f, 0.f}, dn = dp;
            for (int d0 = 0; d0 < a.DV; d0 += 32) {
                const int pa = at + 16 * ta * TV::kRow + d0, pb = at + 16 * tb * TV::kRow + d0;
                Frag<1> fo;
                Frag<3> fw, fu;
                fo.p[0] = lds_row8(s_o + pa);
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    fu.p[i] = lds_row8(s_u + i * TV::kPart + pb);
                    fw.p[i] = lds_row8(s_w + i * TV::kPart + pa);
                }
                dp = mma<3>(fo, fu, dp);
                dn = mma<3>(fw, fu, dn);
            }
            f32x4 kk = {0.f, 0.f, 0.f, 0.f}, m;
#pragma unroll
            for (int s = 0; s < KD / 32; ++s)
                kk = mma<1>(TK::rows(s_k, ta, s, ln), TK::rows(s_k, tb, s, ln), kk);
            const int jc = 16 * tb + i16;
            const float bj = s_vec[kBeta * kC + jc];
            const float hj = s_vec[kGhi * kC + jc], lj = s_vec[kGlo * kC + jc], nj = s_vec[kResets * kC + jc];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int ic = 16 * ta + 4 * g + r;
                const float d = bj * decay_of(s_vec[kGhi * kC + ic], s_vec[kGlo * kC + ic], s_vec[kResets * kC + ic], hj, lj, nj);
                x[n][r] = jc <= ic ? a.scale * dp[r] * d : 0.f;
                y[n][r] = jc < ic ? -dn[r] * s_vec[kBeta * kC + ic] * d : 0.f;
                m[r] = jc < ic ? dp[r] * bj * P[r] + y[n][r] * kk[r] : 0.f;
            }
            Cuts::put(s_cuts, ta, tb, m, lane);
        }
        lds_barrier();      // u~, w and dO have been read
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int t = wave + n * LDS::kWaves;
            if (t >= kBlocks)
                break;
            const int ta = row_of(t), tb = t - block_of(ta, 0);
            const int p = (16 * ta + 4 * g) * M::kRow + 16 * tb + i16;
            put_rows<M>(s_x + p, x[n]);
            put_rows<M>(s_y + p, y[n]);
        }
        // the blocks right of the diagonal that share a k step with it
        if (tid < 128) {
            const int p = ((tid >> 6) * 32 + ((tid >> 2) & 15)) * M::kRow + (tid >> 6) * 32 + 16 + (tid & 3) * 4;
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                *reinterpret_cast<uint2 *>(s_x + n * M::kPart + p) = make_uint2(0, 0);
                *reinterpret_cast<uint2 *>(s_y + n * M::kPart + p) = make_uint2(0, 0);
            }
        }
        lds_barrier();

#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Frag<1> fk = TK::columns(s_k, tile, s, ln), fq = TK::columns(s_q, tile, s, ln);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int ta = first + t;
                if (s <= ta / 2) {
                    dq[t] = mma<3>(M::rows(s_x, ta, s, ln), fk, dq[t]);
                    dk[t] = mma<3>(M::rows(s_y, ta, s, ln), fk, dk[t]);
                }
                if (s >= ta / 2) {
                    dk[t] = mma<3>(M::columns(s_x, ta, s, ln), fq, dk[t]);
                    dk[t] = mma<3>(M::columns(s_y, ta, s, ln), fk, dk[t]);
                }
            }
        }
        if (wave == 0) {
            float reads = 0.f, writes = 0.f, whole = 0.f;
            for (int m = 0; m < kTiles; ++m) {
                reads += s_reads[m * kC + lane];
                writes += s_writes[m * kC + lane];
            }
            for (int m = 0; m < LDS::kWaves; ++m)
                whole += s_sum[m];
            const float v = crossing(whole, reads, writes, s_cuts, lane);
            // the decay of an empty state does nothing
            const bool empty = s_vec[kResets * kC + lane] != (lane ? s_vec[kResets * kC + lane - 1] : 0.f) ||
                               (t0 + lane == 0 && !a.s0);
            if (t0 + lane < a.L)
                static_cast<float *>(const_cast<void *>(a.dg.p))[b * a.dg.s.b + h * a.dg.s.h + (t0 + lane) * a.dg.s.l] =
                    empty ? 0.f : v;
        }
        lds_barrier();
    }
    const Chunk<true, VEC> cq(a.dq.p, b * a.dq.s.b + hk * a.dq.s.h, a.dq.s.l, t0, a.L, a.Dk);
    const Chunk<true, VEC> ck(a.dk.p, b * a.dk.s.b + hk * a.dk.s.h, a.dk.s.l, t0, a.L, a.Dk);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        store_cols(cq, dim, lane, first + t, dq[t]);
        store_cols(ck, dim, lane, first + t, dk[t]);
    }
}

// ---------------------------------------------------------------------------
// step_kernel: one step.  A workgroup takes TX x 4 columns of one head's state,
// each thread four columns of every TY-th row, all rows in registers: the
// state is read once and written once.  o needs no second pass over the new
// state: S_new^T q = (e^g S)^T q + (q . k) u, so both products over the rows
// and q . k are summed across the threads together.  4096 states of 128 x 128
// (540 MB) take 111 us, 4.9 TB/s, and 16 of them 4.6 us, a launch and a trip to
// memory and back.
// ---------------------------------------------------------------------------
struct StepArgs {
    Rows q, k, v, g, beta, o;
    const float *s;
    float *s_out;
    int64_t blocks;         // heads x slices, over both dimensions of the grid
    int Hk, Hv, Dk, Dv, slices;
    float scale;
};

template <bool BF16>
__device__ __forceinline__ float load_value(const void *p, int64_t e)
{
    if constexpr (BF16)
        return bf16_lo(static_cast<const uint16_t *>(p)[e]);
    else
        return static_cast<const float *>(p)[e];
}

template <bool BF16, int TX, bool VEC>
__global__ void __launch_bounds__(kThreads) step_kernel(StepArgs a)
{
    constexpr int TY = kThreads / TX, RP = kMaxDim / TY, WY = 64 / TX;   // rows of a wave side by side
    __shared__ float s_part[4][2][TX * 4];
    __shared__ float s_qk[4];
    const unsigned block = blockIdx.y * gridDim.x + blockIdx.x;
    if (block >= a.blocks)
        return;
    const int64_t head = block / (unsigned)a.slices;
    const int slice = block % (unsigned)a.slices;
    const int64_t b = head / a.Hv;
    const int h = (int)(head - b * a.Hv), hk = h / (a.Hv / a.Hk);
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, wave = threadIdx.x >> 6;
    const int col = slice * TX * 4 + tx * 4;
    const float *S = a.s + head * a.Dk * a.Dv;
    float *So = a.s_out + head * a.Dk * a.Dv;

    f32x4 st[RP];
    float q[RP], k[RP];
#pragma unroll
    for (int i = 0; i < RP; ++i) {
        const int row = i * TY + ty;
        st[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        q[i] = k[i] = 0.f;
        if (row < a.Dk) {
            if constexpr (VEC) {
                if (col < a.Dv)
                    st[i] = *reinterpret_cast<const f32x4 *>(S + row * a.Dv + col);
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (col + r < a.Dv)
                        st[i][r] = S[row * a.Dv + col + r];
            }
            q[i] = load_value<BF16>(a.q.p, b * a.q.s.b + hk * a.q.s.h + row);
            k[i] = load_value<BF16>(a.k.p, b * a.k.s.b + hk * a.k.s.h + row);
        }
    }
    const float decay = expf(static_cast<const float *>(a.g.p)[b * a.g.s.b + h * a.g.s.h]);
    const float beta = static_cast<const float *>(a.beta.p)[b * a.beta.s.b + h * a.beta.s.h];
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (col + r < a.Dv)
            v[r] = load_value<BF16>(a.v.p, b * a.v.s.b + h * a.v.s.h + col + r);

    f32x4 ks = {0.f, 0.f, 0.f, 0.f}, qs = ks;
    float qk = 0.f;
#pragma unroll
    for (int i = 0; i < RP; ++i) {
        st[i] *= decay;
        ks += k[i] * st[i];
        qs += q[i] * st[i];
        qk += q[i] * k[i];
    }
#pragma unroll
    for (int m = TX; m < 64; m <<= 1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            ks[r] += __shfl_xor(ks[r], m, 64);
            qs[r] += __shfl_xor(qs[r], m, 64);
        }
        qk += __shfl_xor(qk, m, 64);
    }
    if (ty % WY == 0) {
        *reinterpret_cast<f32x4 *>(&s_part[wave][0][tx * 4]) = ks;
        *reinterpret_cast<f32x4 *>(&s_part[wave][1][tx * 4]) = qs;
        if (tx == 0)
            s_qk[wave] = qk;
    }
    __syncthreads();
    ks = qs = f32x4{0.f, 0.f, 0.f, 0.f};
    qk = 0.f;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        ks += *reinterpret_cast<const f32x4 *>(&s_part[m][0][tx * 4]);
        qs += *reinterpret_cast<const f32x4 *>(&s_part[m][1][tx * 4]);
        qk += s_qk[m];
    }
    const f32x4 u = beta * (v - ks);
#pragma unroll
    for (int i = 0; i < RP; ++i) {
        const int row = i * TY + ty;
        st[i] += k[i] * u;
        if (row < a.Dk) {
            if constexpr (VEC) {
                if (col < a.Dv)
                    *reinterpret_cast<f32x4 *>(So + row * a.Dv + col) = st[i];
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (col + r < a.Dv)
                        So[row * a.Dv + col + r] = st[i][r];
            }
        }
    }
    if (ty == 0) {
        const f32x4 o = a.scale * (qs + qk * u);
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (col + r < a.Dv) {
                const int64_t e = b * a.o.s.b + h * a.o.s.h + col + r;
                if constexpr (BF16)
                    static_cast<uint16_t *>(const_cast<void *>(a.o.p))[e] = f32_to_bf16_rne(o[r]);
                else
                    static_cast<float *>(const_cast<void *>(a.o.p))[e] = o[r];
            }
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
constexpr int64_t kMaxL = (int64_t)1 << 30;
// Workgroups along x: a launch has fewer than 2^32 threads in a dimension.
constexpr int64_t kMaxGridX = (int64_t)1 << 23;

int check_delta_dims(int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk, int32_t Dv)
{
    if (B < 0 || Hk < 0 || Hv < 0 || L < 0 || L > kMaxL || Dk < 1 || Dk > kMaxDim || Dv < 1 || Dv > kMaxDim)
        return PDSSM_ERR_DIM;
    if (Hv > 0 && (Hk == 0 || Hv % Hk != 0))
        return PDSSM_ERR_DIM;
    if ((double)B * Hv > 5.0e8 || Hv > (1 << 30) || (double)B * Hv * (double)((L + kC - 1) / kC) > 2.0e9)
        return PDSSM_ERR_DIM;
    return PDSSM_OK;
}


int padded_key(int Dk) { return Dk <= 64 ? 64 : 128; }
int padded_value(int Dv) { return (Dv + 31) / 32 * 32; }

int slices_of(int Dv) { return (Dv + 63) / 64; }

// How many segments the chunks of a head are cut into.  A chunk of a forward
// walk takes 2.7 us (keys of 64) or 4.0 us (128) with few walks, 3.5 and 4.7 us
// with one on every compute unit; G segments divide that time by G, but walk twice
// (once without outputs) and are joined one after another, about 1.8 or 3.5 us
// each, so G is near the root of NC times the ratio, and no more than fills the
// device.
// In us, as one and cut.  Forward: 8 heads of 64, 512 steps 34 and 37 (not
// cut), 1024 steps 57 and 42, 16384 steps 721 and 146; 8 heads of 128, 1024 steps 78
// and 57, 16384 steps 1046 and 247; 32 heads of 128 (64 walks), 1024 steps 82 and 77
// to 87 (not cut), 2048 steps 151 and 119, 4096 steps 288 and 200; 64 heads of 128 (128
// walks), 4096 steps 319 and 369 (not cut).  Backward, two walks for each: 8 heads
// of 64, 1024 steps 77 and 65; 16 heads of 128 (64 walks), 1024 steps 103 and 104 (not cut),
// 4096 steps 372 and 336; 32 heads of 128, 4096 steps 553 and 579 (not cut).
// The factor: 8 heads of 64, 4096 steps with the root 72 us, 3/2 of it 67,
// twice 68; of 128 with the root 99, 3/2 113.
struct Cut {
    int segs, chunks;
};

Cut cut_of(int64_t heads, int64_t L, int Dk, int Dv, uint32_t flags, bool bwd)
{
    const int64_t NC = (L + kC - 1) / kC, walks = heads * slices_of(Dv) * (bwd ? 2 : 1);
    int64_t segs = 1;
    if ((flags & PDSSM_DATA_BF16) && walks > 0 && walks <= 64 && NC >= (walks > 32 ? 32 : 16)) {
        int64_t root = 1;
        while ((root + 1) * (root + 1) <= NC)
            ++root;
        segs = padded_key(Dk) == 64 ? root * 3 / 2 : root;
        const int64_t most = 256 / (heads * slices_of(Dv));
        segs = segs < most ? segs : most;
    }
    Cut c;
    c.chunks = (int)((NC + segs - 1) / segs);
    if (c.chunks < 1)
        c.chunks = 1;
    c.segs = (int)((NC + c.chunks - 1) / c.chunks);
    return c;
}

struct Layout {
    int64_t records, seg_states, trans, seg_grads, rtrans, states, grads, ut, w, total;
    Cut cut;
};

Layout layout_of(int64_t B, int64_t Hv, int64_t L, int Dk, int Dv, uint32_t flags, bool bwd)
{
    const int64_t heads = B * Hv;
    int64_t chunks = heads * ((L + kC - 1) / kC);
    chunks = chunks > 0 ? chunks : 1;
    const int64_t state = (int64_t)padded_key(Dk) * padded_value(Dv) * 4, rows = (int64_t)kC * padded_value(Dv) * 4;
    Layout l;
    l.cut = cut_of(heads, L, Dk, Dv, flags, bwd);
    const int64_t cuts = l.cut.segs > 1 ? heads * l.cut.segs : 0;
    l.records = 0;
    l.seg_states = chunks * (bwd ? Record::kBwd : Record::kFwd) * 4;
    l.trans = l.seg_states + cuts * state;
    l.seg_grads = l.trans + cuts * padded_key(Dk) * (slices_of(Dv) * 64 + padded_key(Dk)) * 4;
    l.rtrans = l.seg_grads + (bwd ? cuts * state : 0);
    l.states = l.rtrans + (bwd ? cuts * padded_key(Dk) * slices_of(Dv) * 64 * 4 : 0);
    l.grads = l.states + (bwd ? chunks * state : 0);
    l.ut = l.grads + (bwd ? chunks * state : 0);
    l.w = l.ut + (bwd ? chunks * rows : 0);
    l.total = l.w + (bwd ? chunks * rows : 0);
    return l;
}

// The parts of the workspace that both directions have.
void place_workspace(DeltaArgs &a, const Layout &l, void *workspace)
{
    char *ws = static_cast<char *>(workspace);
    a.records = reinterpret_cast<float *>(ws + l.records);
    a.seg_states = reinterpret_cast<float *>(ws + l.seg_states);
    a.trans = reinterpret_cast<float *>(ws + l.trans);
    a.seg_grads = reinterpret_cast<float *>(ws + l.seg_grads);
    a.rtrans = reinterpret_cast<float *>(ws + l.rtrans);
    a.segs = l.cut.segs;
    a.seg_chunks = l.cut.chunks;
}

// Every row begins on 16 bytes, ends with a whole unit of eight values and
// before the next one.
bool units(const void *p, const pdssm_strides &s, int D, int esize)
{
    const int e = 16 / esize;
    return aligned16(p) && s.b % e == 0 && s.h % e == 0 && s.l % e == 0 && D % 8 == 0 && s.l >= D;
}

// Strides along l that a chunk's 32-bit offsets can follow.
bool strides_ok(const pdssm_strides *s, int n)
{
    for (int i = 0; i < n; ++i)
        if (s[i].l < 0 || s[i].l >= kMaxStride)
            return false;
    return true;
}

bool element_aligned(const void *p, int esize) { return ((uintptr_t)p & (uintptr_t)(esize - 1)) == 0; }

template <typename K>
int launch(K kernel, int64_t grid, size_t lds, const DeltaArgs &a, hipStream_t stream, int threads = kThreads)
{
    // More than 64 KB of LDS has to be asked for; the device has 160 KB.
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess)
            return hip_status(e);
    }
    hipLaunchKernelGGL(kernel, dim3((unsigned)grid), dim3((unsigned)threads), lds, stream, a);
    return hip_status(hipGetLastError());
}

template <int KD>
constexpr size_t chain_lds(bool outputs)
{
    using T = Tile<KD, false>;
    const size_t one = (size_t)(T::kSize + Tri<false>::kSize) * 2;
    return one * (outputs ? 2 : 1) + 4 * kC * 4;
}

template <int KD>
constexpr size_t grad_lds()
{
    return (size_t)(2 * Tile<KD, false>::kSize + 2 * Tile<kC, false>::kSize) * 2 + (kVecs * kC + 4 * kC + Cuts::kSize + 4) * 4;
}

template <int KD, bool BF16, bool VEC>
int launch_fwd(const DeltaArgs &a, hipStream_t stream)
{
    int rc = launch(prep_kernel<KD, BF16, VEC, false>, a.heads * a.NC, 0, a, stream);
    if (rc != PDSSM_OK)
        return rc;
    const int64_t walks = a.heads * a.slices;
    if constexpr (BF16) {
        const int64_t joins = a.heads * ((a.DV + 15) / 16);
        if (a.segs > 1) {
            rc = launch(pipe_kernel<KD, VEC, kScan>, a.heads * a.segs * (a.slices + KD / 64), PipeLds<KD>::bytes(false), a,
                        stream, kPipeThreads);
            if (rc == PDSSM_OK)
                rc = launch(join_kernel<KD>, joins, JoinLds<KD>::kBytes, a, stream, JoinLds<KD>::kThreads);
        }
        if (rc == PDSSM_OK)
            rc = launch(pipe_kernel<KD, VEC, kOut>, walks * a.segs, PipeLds<KD>::bytes(true), a, stream, kPipeThreads);
        return rc;
    } else {
        return launch(chain_kernel<KD, VEC, false>, walks, chain_lds<KD>(true), a, stream);
    }
}

template <int KD, bool BF16, bool VEC>
int launch_bwd(DeltaArgs a, hipStream_t stream)
{
    int rc = launch(prep_kernel<KD, BF16, VEC, true>, a.heads * a.NC, 0, a, stream);
    if (rc != PDSSM_OK)
        return rc;
    const int64_t walks = a.heads * a.slices, chunks = a.heads / a.Hv * a.Hk * a.NC;
    if constexpr (BF16) {
        const int64_t joins = a.heads * ((a.DV + 15) / 16);
        constexpr size_t lds = BackLds<KD>::kBytes > PipeLds<KD>::bytes(false) ? BackLds<KD>::kBytes : PipeLds<KD>::bytes(false);
        a.back_blocks = (unsigned)(walks * a.segs);
        if (a.segs > 1) {
            rc = launch(back_kernel<KD, VEC, true>, (walks * 2 + a.heads * (KD / 64)) * a.segs, lds, a, stream, kPipeThreads);
            if (rc == PDSSM_OK)
                rc = launch(join_kernel<KD>, joins * 2, JoinLds<KD>::kBytes, a, stream, JoinLds<KD>::kThreads);
        }
        if (rc == PDSSM_OK)
            rc = launch(back_kernel<KD, VEC, false>, walks * 2 * a.segs, lds, a, stream, kPipeThreads);
        if (rc != PDSSM_OK)
            return rc;
        if (a.DV <= 64)
            return launch(grads_kernel<KD, 64, VEC>, chunks, GradLds<KD, 64>::kBytes, a, stream, kGradThreads);
        return launch(grads_kernel<KD, 128, VEC>, chunks, GradLds<KD, 128>::kBytes, a, stream, kGradThreads);
    } else {
        rc = launch(chain_kernel<KD, VEC, true>, walks, chain_lds<KD>(false), a, stream);
        if (rc == PDSSM_OK)
            rc = launch(reverse_kernel<KD, VEC>, walks, chain_lds<KD>(true), a, stream);
        if (rc == PDSSM_OK)
            rc = launch(grad_kernel<KD, VEC>, chunks, grad_lds<KD>(), a, stream);
        return rc;
    }
}

// The variant for these sizes, type and rows (vec: see units()).
template <bool BWD, int KD, bool BF16>
int launch_rows(const DeltaArgs &a, bool vec, hipStream_t stream)
{
    if constexpr (BWD)
        return vec ? launch_bwd<KD, BF16, true>(a, stream) : launch_bwd<KD, BF16, false>(a, stream);
    else
        return vec ? launch_fwd<KD, BF16, true>(a, stream) : launch_fwd<KD, BF16, false>(a, stream);
}

template <bool BWD>
int launch_any(const DeltaArgs &a, bool bf16, bool vec, hipStream_t stream)
{
    if (bf16)
        return a.Dk <= 64 ? launch_rows<BWD, 64, true>(a, vec, stream) : launch_rows<BWD, 128, true>(a, vec, stream);
    return a.Dk <= 64 ? launch_rows<BWD, 64, false>(a, vec, stream) : launch_rows<BWD, 128, false>(a, vec, stream);
}

}  // namespace
}  // namespace pdssm

using namespace pdssm;

extern "C" size_t pdssm_delta_workspace_bytes(int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk, int32_t Dv,
                                              uint32_t flags)
{
    if (check_delta_dims(B, Hk, Hv, L, Dk, Dv) != PDSSM_OK || (flags & ~PDSSM_DATA_BF16))
        return 0;
    return (size_t)layout_of(B, Hv, L, Dk, Dv, flags, false).total;
}

extern "C" size_t pdssm_delta_bwd_workspace_bytes(int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk,
                                                  int32_t Dv, uint32_t flags)
{
    if (check_delta_dims(B, Hk, Hv, L, Dk, Dv) != PDSSM_OK || (flags & ~PDSSM_DATA_BF16))
        return 0;
    return (size_t)layout_of(B, Hv, L, Dk, Dv, flags, true).total;
}

extern "C" int pdssm_delta_fwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                               const float *s0, void *o, float *s_final, int64_t B, int64_t Hk, int64_t Hv, int64_t L,
                               int32_t Dk, int32_t Dv, float scale, uint32_t flags, const pdssm_strides *strides,
                               void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const int rc = check_delta_dims(B, Hk, Hv, L, Dk, Dv);
    if (rc != PDSSM_OK)
        return rc;
    if (flags & ~PDSSM_DATA_BF16)
        return PDSSM_ERR_FLAGS;
    if (B == 0 || Hv == 0)
        return PDSSM_OK;
    if ((s0 && !aligned16(s0)) || (s_final && !aligned16(s_final)))
        return PDSSM_ERR_ALIGN;
    if (L == 0) {
        if (!s_final || s_final == s0)
            return PDSSM_OK;
        return launch_state_fill(s0, s_final, B * Hv * Dk * Dv, stream);
    }
    if (!q || !k || !v || !g || !beta || !o || !workspace)
        return PDSSM_ERR_NULL;
    const int esize = (flags & PDSSM_DATA_BF16) ? 2 : 4;
    for (const void *p : {q, k, v, (const void *)o})
        if (!element_aligned(p, esize))
            return PDSSM_ERR_ALIGN;
    for (const float *p : {g, beta})
        if (!element_aligned(p, 4))
            return PDSSM_ERR_ALIGN;
    if (!aligned16(workspace))
        return PDSSM_ERR_ALIGN;
    const Layout lo = layout_of(B, Hv, L, Dk, Dv, flags, false);
    if (workspace_bytes < (size_t)lo.total)
        return PDSSM_ERR_WORKSPACE;
    DeltaArgs a = {};
    const pdssm_strides keys = {Hk * L * Dk, L * Dk, Dk}, values = {Hv * L * Dv, L * Dv, Dv}, gates = {Hv * L, L, 1};
    const pdssm_strides whole[6] = {keys, keys, values, gates, gates, values};
    const pdssm_strides *s = strides ? strides : whole;
    if (!strides_ok(s, 6))
        return PDSSM_ERR_DIM;
    a.q = {q, s[0]}, a.k = {k, s[1]}, a.v = {v, s[2]}, a.g = {g, s[3]}, a.beta = {beta, s[4]}, a.o = {o, s[5]};
    a.s0 = s0, a.s_final = s_final, a.record = Record::kFwd;
    place_workspace(a, lo, workspace);
    a.heads = B * Hv, a.Hk = (int)Hk, a.Hv = (int)Hv, a.L = (int)L, a.NC = (int)((L + kC - 1) / kC);
    a.Dk = Dk, a.Dv = Dv, a.DV = padded_value(Dv), a.slices = slices_of(Dv), a.scale = scale;
    const bool vec = units(q, s[0], Dk, esize) && units(k, s[1], Dk, esize) && units(v, s[2], Dv, esize) &&
                     units(o, s[5], Dv, esize);
    return launch_any<false>(a, esize == 2, vec, stream);
}

extern "C" int pdssm_delta_bwd(const void *q, const void *k, const void *v, const float *g, const float *beta,
                               const float *s0, const void *d_o, const float *ds_final, void *dq, void *dk, void *dv,
                               float *dg, float *dbeta, float *ds0, int64_t B, int64_t Hk, int64_t Hv, int64_t L,
                               int32_t Dk, int32_t Dv, float scale, uint32_t flags, const pdssm_strides *strides,
                               void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const int rc = check_delta_dims(B, Hk, Hv, L, Dk, Dv);
    if (rc != PDSSM_OK)
        return rc;
    if (flags & ~PDSSM_DATA_BF16)
        return PDSSM_ERR_FLAGS;
    if (B == 0 || Hv == 0)
        return PDSSM_OK;
    for (const float *p : {s0, ds_final, (const float *)ds0})
        if (p && !aligned16(p))
            return PDSSM_ERR_ALIGN;
    if (L == 0) {
        if (!ds0 || ds0 == ds_final)
            return PDSSM_OK;
        return launch_state_fill(ds_final, ds0, B * Hv * Dk * Dv, stream);
    }
    if (!q || !k || !v || !g || !beta || !d_o || !dq || !dk || !dv || !dg || !dbeta || !workspace)
        return PDSSM_ERR_NULL;
    const int esize = (flags & PDSSM_DATA_BF16) ? 2 : 4;
    for (const void *p : {q, k, v, d_o, (const void *)dq, (const void *)dk, (const void *)dv})
        if (!element_aligned(p, esize))
            return PDSSM_ERR_ALIGN;
    for (const float *p : {g, beta, (const float *)dg, (const float *)dbeta})
        if (!element_aligned(p, 4))
            return PDSSM_ERR_ALIGN;
    if (!aligned16(workspace))
        return PDSSM_ERR_ALIGN;
    const Layout lo = layout_of(B, Hv, L, Dk, Dv, flags, true);
    if (workspace_bytes < (size_t)lo.total)
        return PDSSM_ERR_WORKSPACE;
    DeltaArgs a = {};
    const pdssm_strides keys = {Hk * L * Dk, L * Dk, Dk}, values = {Hv * L * Dv, L * Dv, Dv}, gates = {Hv * L, L, 1};
    const pdssm_strides whole[11] = {keys, keys, values, gates, gates, values, keys, keys, values, gates, gates};
    const pdssm_strides *s = strides ? strides : whole;
    a.q = {q, s[0]}, a.k = {k, s[1]}, a.v = {v, s[2]}, a.g = {g, s[3]}, a.beta = {beta, s[4]}, a.d_o = {d_o, s[5]};
    if (!strides_ok(s, 11))
        return PDSSM_ERR_DIM;
    a.dq = {dq, s[6]}, a.dk = {dk, s[7]}, a.dv = {dv, s[8]}, a.dg = {dg, s[9]}, a.dbeta = {dbeta, s[10]};
    a.s0 = s0, a.ds_final = ds_final, a.ds0 = ds0, a.record = Record::kBwd;
    place_workspace(a, lo, workspace);
    char *ws = static_cast<char *>(workspace);
    a.states = reinterpret_cast<float *>(ws + lo.states);
    a.grads = reinterpret_cast<float *>(ws + lo.grads);
    a.ut = reinterpret_cast<float *>(ws + lo.ut);
    a.w = reinterpret_cast<float *>(ws + lo.w);
    a.heads = B * Hv, a.Hk = (int)Hk, a.Hv = (int)Hv, a.L = (int)L, a.NC = (int)((L + kC - 1) / kC);
    a.Dk = Dk, a.Dv = Dv, a.DV = padded_value(Dv), a.slices = slices_of(Dv), a.scale = scale;
    const bool vec = units(q, s[0], Dk, esize) && units(k, s[1], Dk, esize) && units(v, s[2], Dv, esize) &&
                     units(d_o, s[5], Dv, esize) && units(dq, s[6], Dk, esize) && units(dk, s[7], Dk, esize) &&
                     units(dv, s[8], Dv, esize);
    return launch_any<true>(a, esize == 2, vec, stream);
}

extern "C" int pdssm_delta_step(const void *q, const void *k, const void *v, const float *g, const float *beta,
                                const float *s, void *o, float *s_out, int64_t B, int64_t Hk, int64_t Hv, int32_t Dk,
                                int32_t Dv, float scale, uint32_t flags, const pdssm_strides *strides,
                                hipStream_t stream)
{
    const int rc = check_delta_dims(B, Hk, Hv, 1, Dk, Dv);
    if (rc != PDSSM_OK)
        return rc;
    if (flags & ~PDSSM_DATA_BF16)
        return PDSSM_ERR_FLAGS;
    if (B == 0 || Hv == 0)
        return PDSSM_OK;
    if (!q || !k || !v || !g || !beta || !s || !o || !s_out)
        return PDSSM_ERR_NULL;
    const int esize = (flags & PDSSM_DATA_BF16) ? 2 : 4;
    for (const void *p : {q, k, v, (const void *)o})
        if (!element_aligned(p, esize))
            return PDSSM_ERR_ALIGN;
    if (!element_aligned(g, 4) || !element_aligned(beta, 4) || !aligned16(s) || !aligned16(s_out))
        return PDSSM_ERR_ALIGN;
    StepArgs a;
    const pdssm_strides keys = {Hk * Dk, Dk, 0}, values = {Hv * Dv, Dv, 0}, gates = {Hv, 1, 0};
    const pdssm_strides whole[6] = {keys, keys, values, gates, gates, values};
    const pdssm_strides *st = strides ? strides : whole;
    a.q = {q, st[0]}, a.k = {k, st[1]}, a.v = {v, st[2]}, a.g = {g, st[3]}, a.beta = {beta, st[4]}, a.o = {o, st[5]};
    a.s = s, a.s_out = s_out, a.Hk = (int)Hk, a.Hv = (int)Hv, a.Dk = Dk, a.Dv = Dv, a.scale = scale;
    a.slices = (Dv + 31) / 32;
    a.blocks = B * Hv * a.slices;       // below 2^31, by the limit on B Hv
    const dim3 grid((unsigned)std::min(a.blocks, kMaxGridX), (unsigned)((a.blocks + kMaxGridX - 1) / kMaxGridX)), block(kThreads);
    const bool vec = Dv % 4 == 0;
    if (esize == 2) {
        if (vec)
            hipLaunchKernelGGL((step_kernel<true, 8, true>), grid, block, 0, stream, a);
        else
            hipLaunchKernelGGL((step_kernel<true, 8, false>), grid, block, 0, stream, a);
    } else {
        if (vec)
            hipLaunchKernelGGL((step_kernel<false, 8, true>), grid, block, 0, stream, a);
        else
            hipLaunchKernelGGL((step_kernel<false, 8, false>), grid, block, 0, stream, a);
    }
    return hip_status(hipGetLastError());
}
