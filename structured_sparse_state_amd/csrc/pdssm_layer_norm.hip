// The layer norm of h = residual + dropout(x), its gradients, and dropout alone
// (include/pdssm_block.h):
//     y = c r w + b,   c = h - mean(h),   r = 1 / sqrt(mean(c^2) + eps)
// and, with e = w dy and c^ = r c,
//     dr = r (e - mean(e) - c^ mean(e c^)) + dh,   dx = dropout(dr)
//     dw = sum over rows of dy c^,   db = sum over rows of dy.
// The mean is taken first and the squares about it then, from registers; the sum
// of what lies about it gives the mean's own rounding (large where the mean is far
// from zero), which is taken out again: with d = mean(c), c <- c - d and
// mean(c^2) <- mean(c^2) - d^2.
//
// A row belongs to a team of 16 to 1024 lanes, which holds all of it in
// registers (up to four units of eight values a lane): every tensor is read or
// written once.  A unit's eight values take the 128 bits of one generator block,
// so a mask costs a lane one block for each 16-byte load, and is made again in
// the backward.  A team takes many rows with its weights (and the backward's sums
// of dw and db) held in registers.
//
// Bytes bound all of them at the LM layer's 8 x 4096 rows of 2048, bf16, p = 0.1, in
// calls one behind the other: forward 115 us, 537 MB at 4.7 TB/s (x and the residual
// in, y and h out); backward 144 us, layer_norm_sum_kernel's part in it, 671 MB at
// 4.6 TB/s (three rows in, two out), of which the generator's second pass costs 6 (a
// kernel trace has 152 to 161 us for the backward's and 4.5 for the sums'); dropout
// alone 47 us, 268 MB at 5.7 TB/s.  A copy reaches 4.9 TB/s here, and 6.0 with two
// rows in for one out.
// Few rows leave most of the device idle, as teams are chosen by the width alone: 32
// rows of 2048, forward, 8 workgroups, 10 us (9 without weights, 7 without residual
// too).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pdssm_block.h"
#include "pdssm_device.h"
#include "pdssm_host.h"

namespace pdssm {
namespace {

constexpr int kUnit = 8;            // values of a unit
constexpr int kMaxD = 16384;
constexpr int64_t kMaxRows = 2147483647;

// ---------------------------------------------------------------------------
// Dropout
// ---------------------------------------------------------------------------
struct Drop {
    uint64_t seed, offset;
    const uint64_t *rng;    // seed and offset in device memory, or NULL
    uint32_t least;         // a value is kept when its 16 bits are at least this; 0: no dropout
    float scale;

    __device__ __forceinline__ void begin()
    {
        if (least && rng) {
            seed = rng[0];
            offset = rng[1];
        }
    }
    // Values 8 unit .. 8 unit + 7 of a row.
    __device__ __forceinline__ void apply(float (&x)[kUnit], uint32_t row, uint32_t unit) const
    {
        uint32_t c0 = unit, c1 = row, c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
        uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
        for (int n = 0; n < 10; ++n) {
            const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
            c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
            c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
            c1 = (uint32_t)b;
            c3 = (uint32_t)a;
            k0 += 0x9E3779B9u;
            k1 += 0xBB67AE85u;
        }
        const uint32_t w[4] = {c0, c1, c2, c3};
#pragma unroll
        for (int j = 0; j < kUnit; ++j) {
            const uint32_t bits = j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xFFFFu;
            x[j] = bits >= least ? x[j] * scale : 0.f;
        }
    }
};

// ---------------------------------------------------------------------------
// Units of rows
// ---------------------------------------------------------------------------
// Rows [B,H,L,D] of a call.
struct RowsOf {
    const void *p;
    pdssm_strides s;
};

struct Place {          // of a row among them
    int64_t b, h, l;
    __device__ __forceinline__ int64_t at(const RowsOf &r) const { return b * r.s.b + h * r.s.h + l * r.s.l; }
};

template <typename T>
struct Unit;            // eight values of a row as they are stored
template <>
struct Unit<uint16_t> {
    uint4 v;
    __device__ __forceinline__ void get(float (&x)[kUnit]) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = bf16_lo(w[j]);
            x[2 * j + 1] = bf16_hi(w[j]);
        }
    }
    __device__ __forceinline__ void set(const float (&x)[kUnit])
    {
        v = make_uint4(f32x2_to_bf16x2_rne(x[0], x[1]), f32x2_to_bf16x2_rne(x[2], x[3]),
                       f32x2_to_bf16x2_rne(x[4], x[5]), f32x2_to_bf16x2_rne(x[6], x[7]));
    }
};
template <>
struct Unit<float> {
    float4 a, b;
    __device__ __forceinline__ void get(float (&x)[kUnit]) const
    {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&x)[kUnit])
    {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// Unit `unit` of the row at p.  WHOLE: rows begin on 16 bytes and hold whole
// units; else a unit inside the row is still taken as one run (of any
// alignment), and the last one value by value.  Values behind the row are zero.
template <typename T, bool WHOLE>
__device__ __forceinline__ Unit<T> load_unit(const T *p, int unit, int D)
{
    Unit<T> u;
    const int col = unit * kUnit;
    if constexpr (WHOLE) {
        if (col < D) {
            __builtin_memcpy(&u, __builtin_assume_aligned(p + col, 16), sizeof(u));
            return u;
        }
    } else {
        if (col + kUnit <= D) {
            __builtin_memcpy(&u, p + col, sizeof(u));
            return u;
        }
    }
    T v[kUnit];
#pragma unroll
    for (int j = 0; j < kUnit; ++j)
        v[j] = !WHOLE && col + j < D ? p[col + j] : T(0);
    __builtin_memcpy(&u, v, sizeof(u));
    return u;
}

template <typename T, bool WHOLE>
__device__ __forceinline__ void store_unit(T *p, int unit, int D, const float (&x)[kUnit])
{
    Unit<T> u;
    u.set(x);
    const int col = unit * kUnit;
    if constexpr (WHOLE) {
        if (col < D)
            __builtin_memcpy(__builtin_assume_aligned(p + col, 16), &u, sizeof(u));
    } else if (col + kUnit <= D) {
        __builtin_memcpy(p + col, &u, sizeof(u));
    } else {
        T v[kUnit];
        __builtin_memcpy(v, &u, sizeof(u));
#pragma unroll
        for (int j = 0; j < kUnit; ++j)
            if (col + j < D)
                p[col + j] = v[j];
    }
}

// Over the lanes of a group of 16: row rotations, which need no trip through LDS.
template <int N>
__device__ __forceinline__ float rotated(float v)
{
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + N, 0xF, 0xF, true));
}

// N sums over a team's lanes, in all of them.
template <int TEAM, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*s_sum)[16])
{
#pragma unroll
    for (int n = 0; n < N; ++n) {
        v[n] = rotated<1>(rotated<2>(rotated<4>(rotated<8>(v[n]))));
        if constexpr (TEAM >= 64) {
            v[n] += __shfl_xor(v[n], 16, 64);
            v[n] += __shfl_xor(v[n], 32, 64);
        }
    }
    if constexpr (TEAM > 64) {
        constexpr int kWaves = TEAM / 64;
        const int wave = threadIdx.x >> 6, first = wave / kWaves * kWaves;      // of the team
        __syncthreads();        // the sums before have been read
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int n = 0; n < N; ++n)
                s_sum[n][wave] = v[n];
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            v[n] = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                v[n] += s_sum[n][first + w];
        }
    }
}

// fp32 weights of a lane's units; `none` where there are no weights, 0 behind
// the row.
template <int TEAM, int UNITS>
__device__ __forceinline__ void load_weights(const float *w, float none, int lane, int D, float (&out)[UNITS][kUnit])
{
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int j = 0; j < kUnit; ++j) {
            const int col = (lane + u * TEAM) * kUnit + j;
            out[u][j] = col < D ? (w ? w[col] : none) : 0.f;
        }
}

struct NormArgs {
    RowsOf x, residual, y, h;               // forward
    RowsOf dy, dh, dr, dx;                  // backward, with h
    const float *w, *b;
    float *partial;         // backward: [workgroups][2][D] sums of dw and db, or NULL
    Drop drop;
    int64_t rows;
    int H, L, D;
    float eps;
};

__device__ __forceinline__ Place place_of(const NormArgs &a, uint32_t row)
{
    const uint32_t bh = row / (uint32_t)a.L, b = bh / (uint32_t)a.H;
    return {(int64_t)b, (int64_t)(bh - b * (uint32_t)a.H), (int64_t)(row - bh * (uint32_t)a.L)};
}

// The lanes of a workgroup: teams of TEAM lanes side by side.
template <int TEAM>
constexpr int threads_of() { return TEAM > 256 ? TEAM : 256; }

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------
template <typename T, int TEAM, int UNITS, bool WHOLE>
__global__ void __launch_bounds__(threads_of<TEAM>()) layer_norm_kernel(NormArgs a)
{
    constexpr int kTeams = threads_of<TEAM>() / TEAM;
    __shared__ float s_sum[2][16];
    const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    float w[UNITS][kUnit], bias[UNITS][kUnit];
    load_weights<TEAM, UNITS>(a.w, 1.f, lane, a.D, w);
    load_weights<TEAM, UNITS>(a.b, 0.f, lane, a.D, bias);
    Drop drop = a.drop;
    drop.begin();
    const float count = (float)a.D;
    for (int64_t first = (int64_t)blockIdx.x * kTeams; first < a.rows; first += (int64_t)gridDim.x * kTeams) {
        // (a team behind the last row stays for the barriers)
        const bool in = first + team < a.rows;
        const uint32_t row = (uint32_t)(in ? first + team : a.rows - 1);
        const Place at = place_of(a, row);
        const T *x = static_cast<const T *>(a.x.p) + at.at(a.x), *res = static_cast<const T *>(a.residual.p);
        Unit<T> xu[UNITS], ru[UNITS];
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
            xu[u] = load_unit<T, WHOLE>(x, lane + u * TEAM, a.D);
        if (res) {
            res += at.at(a.residual);
#pragma unroll
            for (int u = 0; u < UNITS; ++u)
                ru[u] = load_unit<T, WHOLE>(res, lane + u * TEAM, a.D);
        }
        float h[UNITS][kUnit], sum[1] = {0.f};
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            xu[u].get(h[u]);
            if (drop.least)
                drop.apply(h[u], row, lane + u * TEAM);
            if (res) {
                float r[kUnit];
                ru[u].get(r);
#pragma unroll
                for (int j = 0; j < kUnit; ++j)
                    h[u][j] += r[j];
            }
#pragma unroll
            for (int j = 0; j < kUnit; ++j)
                sum[0] += h[u][j];
        }
        if (a.h.p && in) {
            T *to = static_cast<T *>(const_cast<void *>(a.h.p)) + at.at(a.h);
#pragma unroll
            for (int u = 0; u < UNITS; ++u)
                store_unit<T, WHOLE>(to, lane + u * TEAM, a.D, h[u]);
        }
        team_sum<TEAM>(sum, s_sum);
        const float mean = sum[0] / count;
        float sums[2] = {0.f, 0.f};     // of c, c^2
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                h[u][j] = (lane + u * TEAM) * kUnit + j < a.D ? h[u][j] - mean : 0.f;
                sums[0] += h[u][j];
                sums[1] += h[u][j] * h[u][j];
            }
        team_sum<TEAM>(sums, s_sum);
        const float d = sums[0] / count, r = 1.f / sqrtf(fmaxf(sums[1] / count - d * d, 0.f) + a.eps);
        if (in) {
            T *to = static_cast<T *>(const_cast<void *>(a.y.p)) + at.at(a.y);
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
#pragma unroll
                for (int j = 0; j < kUnit; ++j)
                    h[u][j] = (h[u][j] - d) * r * w[u][j] + bias[u][j];
                store_unit<T, WHOLE>(to, lane + u * TEAM, a.D, h[u]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------
template <typename T, int TEAM, int UNITS, bool WHOLE>
__global__ void __launch_bounds__(threads_of<TEAM>()) layer_norm_bwd_kernel(NormArgs a)
{
    constexpr int kTeams = threads_of<TEAM>() / TEAM;
    __shared__ float s_sum[4][16];
    __shared__ float s_dw[2][kTeams > 1 ? TEAM * UNITS * kUnit : 1];
    const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    float w[UNITS][kUnit], dw[UNITS][kUnit], db[UNITS][kUnit];
    load_weights<TEAM, UNITS>(a.w, 1.f, lane, a.D, w);
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
#pragma unroll
        for (int j = 0; j < kUnit; ++j)
            dw[u][j] = db[u][j] = 0.f;
    Drop drop = a.drop;
    drop.begin();
    const float count = (float)a.D;
    for (int64_t first = (int64_t)blockIdx.x * kTeams; first < a.rows; first += (int64_t)gridDim.x * kTeams) {
        const bool in = first + team < a.rows;
        const uint32_t row = (uint32_t)(in ? first + team : a.rows - 1);
        const Place at = place_of(a, row);
        const T *hp = static_cast<const T *>(a.h.p) + at.at(a.h), *dyp = static_cast<const T *>(a.dy.p) + at.at(a.dy);
        const T *dhp = static_cast<const T *>(a.dh.p);
        Unit<T> hu[UNITS], yu[UNITS], du[UNITS];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            hu[u] = load_unit<T, WHOLE>(hp, lane + u * TEAM, a.D);
            yu[u] = load_unit<T, WHOLE>(dyp, lane + u * TEAM, a.D);
        }
        if (dhp) {
            dhp += at.at(a.dh);
#pragma unroll
            for (int u = 0; u < UNITS; ++u)
                du[u] = load_unit<T, WHOLE>(dhp, lane + u * TEAM, a.D);
        }
        float h[UNITS][kUnit], sum[1] = {0.f};
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            hu[u].get(h[u]);
#pragma unroll
            for (int j = 0; j < kUnit; ++j)
                sum[0] += h[u][j];
        }
        team_sum<TEAM>(sum, s_sum);
        const float mean = sum[0] / count;
        float sums[4] = {0.f, 0.f, 0.f, 0.f};   // of c, c^2, e, e c
        float dy[UNITS][kUnit];
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            yu[u].get(dy[u]);
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                h[u][j] = (lane + u * TEAM) * kUnit + j < a.D ? h[u][j] - mean : 0.f;
                const float e = dy[u][j] * w[u][j];
                sums[0] += h[u][j];
                sums[1] += h[u][j] * h[u][j];
                sums[2] += e;
                sums[3] += e * h[u][j];
            }
        }
        team_sum<TEAM>(sums, s_sum);
        const float d = sums[0] / count, r = 1.f / sqrtf(fmaxf(sums[1] / count - d * d, 0.f) + a.eps);
        const float mean_e = sums[2] / count, along = (sums[3] / count - d * mean_e) * r;  // mean(e), mean(e c^)
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            float out[kUnit];
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                const float unit = (h[u][j] - d) * r;
                if (in) {
                    dw[u][j] += dy[u][j] * unit;
                    db[u][j] += dy[u][j];
                }
                out[j] = r * (dy[u][j] * w[u][j] - mean_e - unit * along);
            }
            if (dhp) {
                float d[kUnit];
                du[u].get(d);
#pragma unroll
                for (int j = 0; j < kUnit; ++j)
                    out[j] += d[j];
            }
            if (in && a.dr.p)
                store_unit<T, WHOLE>(static_cast<T *>(const_cast<void *>(a.dr.p)) + at.at(a.dr), lane + u * TEAM, a.D, out);
            if (a.dx.p) {
                if (drop.least)
                    drop.apply(out, row, lane + u * TEAM);
                if (in)
                    store_unit<T, WHOLE>(static_cast<T *>(const_cast<void *>(a.dx.p)) + at.at(a.dx), lane + u * TEAM, a.D, out);
            }
        }
    }
    if (!a.partial)
        return;
    // The workgroup's sums: its teams' in their order.
    float *to = a.partial + (int64_t)blockIdx.x * 2 * a.D;
    if constexpr (kTeams > 1) {
        for (int n = 0; n < kTeams; ++n) {
            if (team == n) {
#pragma unroll
                for (int u = 0; u < UNITS; ++u)
#pragma unroll
                    for (int j = 0; j < kUnit; ++j) {
                        const int e = j * TEAM * UNITS + u * TEAM + lane;       // (lanes side by side in the banks)
                        if (n) {
                            dw[u][j] += s_dw[0][e];
                            db[u][j] += s_dw[1][e];
                        }
                        s_dw[0][e] = dw[u][j];
                        s_dw[1][e] = db[u][j];
                    }
            }
            __syncthreads();
        }
    }
    if (team == kTeams - 1) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u)
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                const int col = (lane + u * TEAM) * kUnit + j;
                if (col < a.D) {
                    to[col] = dw[u][j];
                    to[a.D + col] = db[u][j];
                }
            }
    }
}

// dw and db from the workgroups' sums.  A workgroup takes 16 columns, 64 rows at a
// time (512 rows of 2 x 2048: 4.4 us, mostly the launch's latency).
constexpr int kSumRows = 64, kSumCols = 16;
struct SumArgs {
    const float *partial;   // [rows][2][D]
    float *out[2];
    int rows, D;
};

__global__ void __launch_bounds__(kSumRows *kSumCols) layer_norm_sum_kernel(SumArgs a)
{
    __shared__ float s_part[kSumRows][kSumCols + 1];
    const int which = blockIdx.y, c = threadIdx.x % kSumCols, part = threadIdx.x / kSumCols;
    const int col = blockIdx.x * kSumCols + c;
    if (!a.out[which])
        return;
    float v = 0.f;
    if (col < a.D) {
#pragma unroll 4
        for (int i = part; i < a.rows; i += kSumRows)
            v += a.partial[((int64_t)i * 2 + which) * a.D + col];
    }
    s_part[part][c] = v;
    __syncthreads();
    if (threadIdx.x < kSumCols && col < a.D) {
        for (int i = 1; i < kSumRows; ++i)
            v += s_part[i][c];
        a.out[which][col] = v;
    }
}

// ---------------------------------------------------------------------------
// Dropout alone: a lane has one unit of a row.
// ---------------------------------------------------------------------------
template <typename T, bool WHOLE>
__global__ void __launch_bounds__(256) dropout_kernel(NormArgs a)
{
    Drop drop = a.drop;
    drop.begin();
    const uint32_t units = (uint32_t)(a.D + kUnit - 1) / kUnit;
    const int64_t all = a.rows * units;
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < all; n += (int64_t)gridDim.x * 256) {
        const uint32_t row = (uint32_t)(n / units), unit = (uint32_t)(n - (int64_t)row * units);
        const Place at = place_of(a, row);
        const Unit<T> xu = load_unit<T, WHOLE>(static_cast<const T *>(a.x.p) + at.at(a.x), unit, a.D);
        float x[kUnit];
        if (a.residual.p) {
            const Unit<T> ru = load_unit<T, WHOLE>(static_cast<const T *>(a.residual.p) + at.at(a.residual), unit, a.D);
            float r[kUnit];
            xu.get(x);
            ru.get(r);
            if (drop.least)
                drop.apply(x, row, unit);
#pragma unroll
            for (int j = 0; j < kUnit; ++j)
                x[j] += r[j];
        } else {
            xu.get(x);
            if (drop.least)
                drop.apply(x, row, unit);
        }
        store_unit<T, WHOLE>(static_cast<T *>(const_cast<void *>(a.y.p)) + at.at(a.y), unit, a.D, x);
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
int check_rows(int64_t B, int64_t H, int64_t L, int32_t D)
{
    if (B < 0 || H < 0 || L < 0 || D < 1 || D > kMaxD)
        return PDSSM_ERR_DIM;
    if ((double)B * (double)H * (double)L > (double)kMaxRows || B > kMaxRows || H > kMaxRows || L > kMaxRows)
        return PDSSM_ERR_DIM;
    return PDSSM_OK;
}

// p in [0,1) as a threshold of 16 bits.
int drop_of(Drop &d, double p, uint64_t seed, uint64_t offset, const uint64_t *rng)
{
    if (!(p >= 0.0 && p < 1.0))
        return PDSSM_ERR_DIM;
    if ((uintptr_t)rng & 7u)
        return PDSSM_ERR_ALIGN;
    d = Drop{seed, offset, rng, (uint32_t)std::min(65535.0, p * 65536.0 + 0.5), 1.f};
    d.scale = (float)(65536.0 / (65536.0 - d.least));
    return PDSSM_OK;
}

// A call's row tensors: NULL and alignment, and whether all rows are whole units
// on 16 bytes.
int take_rows(RowsOf &r, const void *p, const pdssm_strides *s, int n, const pdssm_strides &whole, bool wanted, int esize,
              bool &units)
{
    r = {p, s ? s[n] : whole};
    if (!p)
        return wanted ? PDSSM_ERR_NULL : PDSSM_OK;
    if ((uintptr_t)p & (uintptr_t)(esize - 1))
        return PDSSM_ERR_ALIGN;
    const int e = 16 / esize;
    units = units && aligned16(p) && r.s.b % e == 0 && r.s.h % e == 0 && r.s.l % e == 0;
    return PDSSM_OK;
}

// Teams, so that a lane has at most four units of a row forward and two backward
// (whose sums of dw and db take as many registers again).  8 x 4096 rows of 2048,
// bf16: forward 114 us with 64 lanes of four units, 114 with 128 of two, 117 with 256
// of one; backward (with its sums) 165, 146 and 150 (one, two and five waves to a SIMD).
int team_of(int D, bool bwd)
{
    if (D <= 128)
        return 16;
    if (D <= (bwd ? 1024 : 2048))
        return 64;
    if (bwd)
        return D <= 2048 ? 128 : D <= 4096 ? 256 : D <= 8192 ? 512 : 1024;
    return D <= 8192 ? 256 : 1024;
}

// Workgroups: no more than fill the device a few times over, so that a team's
// weights (and sums) serve many rows.  The backward above with 512, 768, 1024 and
// 1536 of them: 147, 158, 153 and 158 us.
int64_t groups_of(int64_t rows, int D, bool bwd)
{
    const int64_t teams = std::max(256 / team_of(D, bwd), 1);
    return std::min<int64_t>((rows + teams - 1) / teams, bwd ? 512 : 2048);
}

template <typename T, int TEAM, int UNITS, bool WHOLE, bool BWD>
void launch_norm(const NormArgs &a, int64_t groups, hipStream_t stream)
{
    const dim3 grid((unsigned)groups), block((unsigned)threads_of<TEAM>());
    if constexpr (BWD)
        hipLaunchKernelGGL((layer_norm_bwd_kernel<T, TEAM, UNITS, WHOLE>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((layer_norm_kernel<T, TEAM, UNITS, WHOLE>), grid, block, 0, stream, a);
}

template <typename T, bool WHOLE>
void launch_width(const NormArgs &a, bool bwd, int64_t groups, hipStream_t stream)
{
    const int units = (a.D + kUnit - 1) / kUnit, team = team_of(a.D, bwd), each = (units + team - 1) / team;
#define PDSSM_TEAM(n, u, back)                                        \
    if (team == n && each <= u && bwd == back)                        \
        return launch_norm<T, n, u, WHOLE, back>(a, groups, stream)
    PDSSM_TEAM(16, 1, false);
    PDSSM_TEAM(64, 1, false);
    PDSSM_TEAM(64, 2, false);
    PDSSM_TEAM(64, 4, false);
    PDSSM_TEAM(256, 2, false);
    PDSSM_TEAM(256, 4, false);
    PDSSM_TEAM(1024, 2, false);
    PDSSM_TEAM(16, 1, true);
    PDSSM_TEAM(64, 1, true);
    PDSSM_TEAM(64, 2, true);
    PDSSM_TEAM(128, 2, true);
    PDSSM_TEAM(256, 2, true);
    PDSSM_TEAM(512, 2, true);
    PDSSM_TEAM(1024, 2, true);
#undef PDSSM_TEAM
}

int launch_rows(const NormArgs &a, bool bf16, bool whole, bool bwd, int64_t groups, hipStream_t stream)
{
    if (bf16 && whole)
        launch_width<uint16_t, true>(a, bwd, groups, stream);
    else if (bf16)
        launch_width<uint16_t, false>(a, bwd, groups, stream);
    else if (whole)
        launch_width<float, true>(a, bwd, groups, stream);
    else
        launch_width<float, false>(a, bwd, groups, stream);
    return hip_status(hipGetLastError());
}

template <typename T>
void launch_dropout(const NormArgs &a, bool whole, dim3 grid, hipStream_t stream)
{
    if (whole)
        hipLaunchKernelGGL((dropout_kernel<T, true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((dropout_kernel<T, false>), grid, dim3(256), 0, stream, a);
}

}  // namespace
}  // namespace pdssm

using namespace pdssm;

extern "C" int pdssm_layer_norm_fwd(const void *x, const void *residual, const float *w, const float *b, void *y,
                                    void *h, int64_t B, int64_t H, int64_t L, int32_t D, float eps, double p,
                                    uint64_t seed, uint64_t offset, const uint64_t *rng, uint32_t flags,
                                    const pdssm_strides *strides, hipStream_t stream)
{
    int rc = check_rows(B, H, L, D);
    if (rc != PDSSM_OK)
        return rc;
    if (flags & ~PDSSM_DATA_BF16)
        return PDSSM_ERR_FLAGS;
    NormArgs a = {};
    rc = drop_of(a.drop, p, seed, offset, rng);
    if (rc != PDSSM_OK || B == 0 || H == 0 || L == 0)
        return rc;
    const int esize = (flags & PDSSM_DATA_BF16) ? 2 : 4;
    const pdssm_strides whole = {H * L * D, L * D, D};
    bool units = D % kUnit == 0;
    RowsOf *to[4] = {&a.x, &a.residual, &a.y, &a.h};
    const void *from[4] = {x, residual, y, h};
    for (int n = 0; n < 4; ++n) {
        rc = take_rows(*to[n], from[n], strides, n, whole, n % 2 == 0, esize, units);
        if (rc != PDSSM_OK)
            return rc;
    }
    if (((uintptr_t)w | (uintptr_t)b) & 3u)
        return PDSSM_ERR_ALIGN;
    a.w = w, a.b = b, a.rows = B * H * L, a.H = (int)H, a.L = (int)L, a.D = D, a.eps = eps;
    return launch_rows(a, esize == 2, units, false, groups_of(a.rows, D, false), stream);
}

extern "C" size_t pdssm_layer_norm_bwd_workspace_bytes(int64_t B, int64_t H, int64_t L, int32_t D)
{
    if (check_rows(B, H, L, D) != PDSSM_OK)
        return 0;
    return (size_t)(std::max<int64_t>(groups_of(B * H * L, D, true), 1) * 2 * D * 4 + 15) / 16 * 16;
}

extern "C" int pdssm_layer_norm_bwd(const void *h, const void *dy, const void *dh, const float *w, void *dr, void *dx,
                                    float *dw, float *db, int64_t B, int64_t H, int64_t L, int32_t D, float eps,
                                    double p, uint64_t seed, uint64_t offset, const uint64_t *rng, uint32_t flags,
                                    const pdssm_strides *strides, void *workspace, size_t workspace_bytes,
                                    hipStream_t stream)
{
    int rc = check_rows(B, H, L, D);
    if (rc != PDSSM_OK)
        return rc;
    if (flags & ~PDSSM_DATA_BF16)
        return PDSSM_ERR_FLAGS;
    NormArgs a = {};
    rc = drop_of(a.drop, p, seed, offset, rng);
    if (rc != PDSSM_OK)
        return rc;
    const int esize = (flags & PDSSM_DATA_BF16) ? 2 : 4;
    const pdssm_strides whole = {H * L * D, L * D, D};
    const bool any = B > 0 && H > 0 && L > 0, sums = dw || db;
    if (((uintptr_t)w | (uintptr_t)dw | (uintptr_t)db) & 3u)
        return PDSSM_ERR_ALIGN;
    a.rows = any ? B * H * L : 0;
    const int64_t groups = any ? groups_of(a.rows, D, true) : 0;
    if (any) {
        bool units = D % kUnit == 0;
        RowsOf *to[5] = {&a.h, &a.dy, &a.dh, &a.dr, &a.dx};
        const void *from[5] = {h, dy, dh, dr, dx};
        for (int n = 0; n < 5; ++n) {
            rc = take_rows(*to[n], from[n], strides, n, whole, n < 2, esize, units);
            if (rc != PDSSM_OK)
                return rc;
        }
        if (sums) {
            if (!workspace)
                return PDSSM_ERR_NULL;
            if (!aligned16(workspace))
                return PDSSM_ERR_ALIGN;
            if (workspace_bytes < pdssm_layer_norm_bwd_workspace_bytes(B, H, L, D))
                return PDSSM_ERR_WORKSPACE;
            a.partial = static_cast<float *>(workspace);
        }
        if (!dr && !dx && !sums)
            return PDSSM_OK;
        a.w = w, a.H = (int)H, a.L = (int)L, a.D = D, a.eps = eps;
        rc = launch_rows(a, esize == 2, units, true, groups, stream);
        if (rc != PDSSM_OK)
            return rc;
    }
    if (!sums)
        return PDSSM_OK;
    const SumArgs s = {a.partial, {dw, db}, (int)groups, D};
    hipLaunchKernelGGL(layer_norm_sum_kernel, dim3((unsigned)((D + kSumCols - 1) / kSumCols), 2), dim3(kSumRows * kSumCols), 0,
                       stream, s);
    return hip_status(hipGetLastError());
}

extern "C" int pdssm_dropout(const void *x, const void *residual, void *y, int64_t B, int64_t H, int64_t L, int32_t D,
                             double p, uint64_t seed, uint64_t offset, const uint64_t *rng, uint32_t flags,
                             const pdssm_strides *strides, hipStream_t stream)
{
    int rc = check_rows(B, H, L, D);
    if (rc != PDSSM_OK)
        return rc;
    if (flags & ~PDSSM_DATA_BF16)
        return PDSSM_ERR_FLAGS;
    NormArgs a = {};
    rc = drop_of(a.drop, p, seed, offset, rng);
    if (rc != PDSSM_OK || B == 0 || H == 0 || L == 0)
        return rc;
    const int esize = (flags & PDSSM_DATA_BF16) ? 2 : 4;
    const pdssm_strides whole = {H * L * D, L * D, D};
    bool units = D % kUnit == 0;
    RowsOf *to[3] = {&a.x, &a.residual, &a.y};
    const void *from[3] = {x, residual, y};
    for (int n = 0; n < 3; ++n) {
        rc = take_rows(*to[n], from[n], strides, n, whole, n != 1, esize, units);
        if (rc != PDSSM_OK)
            return rc;
    }
    a.rows = B * H * L, a.H = (int)H, a.L = (int)L, a.D = D;
    const int64_t all = a.rows * ((D + kUnit - 1) / kUnit);
    const dim3 grid((unsigned)std::min<int64_t>((all + 255) / 256, 16384));
    if (esize == 2)
        launch_dropout<uint16_t>(a, units, grid, stream);
    else
        launch_dropout<float>(a, units, grid, stream);
    return hip_status(hipGetLastError());
}
