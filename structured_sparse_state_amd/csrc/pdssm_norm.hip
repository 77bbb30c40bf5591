// Norm of query and key heads with the rotation by position, and its
// gradients (include/pdssm_layers.h):
//     r = 1 / sqrt(sum(x^2) / n + eps)   (n = D for RMS, 1 for unit length)
//     y = R(p) (w * (r x)),  R(p) turning pairs of dimensions by the angles of
//     position p
// and, with e = w * (R(p)^T dy) and the unit x^ = r x,
//     dx = r (e - x^ sum(e x^) / n),     dw = sum over rows of (R(p)^T dy) x^.
//
// Both are bound by HBM: x (and dy) read once, y (or dx) written once, with a
// few operations per value.  A row of D values belongs to a group of LPH
// lanes, and a lane holds four of the row's pairs (a, b) whole, so the
// rotation needs nothing from another lane; only the row's sum crosses lanes.
// A lane takes the same place in HP heads of one token (all their loads are
// issued before the first is used), with its weights, cosines and sines
// loaded once for them.
#include <hip/hip_runtime.h>

#include "pdssm_device.h"
#include "pdssm_host.h"
#include "pdssm_layers.h"

namespace pdssm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 256;
// Workgroups of the backward with weight gradients: each keeps its sums in
// registers over all its tokens and writes one row of partial sums.
constexpr int kBwdGroups = 2048;

// One of the two tensors (q or k) of a call.
struct NormTensor {
    const void *x, *dy;
    void *out;          // y, or dx in the backward
    const float *w;
    float *partial;     // rows of D weight gradient sums, or NULL
    pdssm_strides sx, sdy, so;
    int64_t H;
};

struct NormArgs {
    NormTensor t[2];
    const float *cs, *sn;
    const int32_t *pos;
    int64_t P;
    int tokens, L, D, half;   // half = R / 2
    int segs0;                // head segments (of HP heads) of t[0]; blockIdx.y beyond are t[1]'s
    float inv_n, eps;
    bool pairs;
};

template <typename T>
__device__ __forceinline__ float load1(const T *p)
{
    if constexpr (sizeof(T) == 2)
        return bf16_lo(*p);
    else
        return *p;
}

template <typename T>
__device__ __forceinline__ void store1(T *p, float v)
{
    if constexpr (sizeof(T) == 2)
        *p = f32_to_bf16_rne(v);
    else
        *p = v;
}

template <typename T>
__device__ __forceinline__ float4 load_quad(const T *p)
{
    if constexpr (sizeof(T) == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
    } else {
        return *reinterpret_cast<const float4 *>(p);
    }
}

template <typename T>
__device__ __forceinline__ void store_quad(T *p, float a, float b, float c, float d)
{
    if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2 *>(p) = make_uint2(f32x2_to_bf16x2_rne(a, b), f32x2_to_bf16x2_rne(c, d));
    else
        *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}

// Where a lane's four pairs lie in a row.  Pair p of the row is (p, p + half)
// when it turns in half mode, else (2p, 2p + 1); `split`: the lane's first
// elements are one quad and its second ones another, else the eight are
// consecutive.  Elements at D and beyond do not exist.
struct Place {
    int e0[4], e1[4];
    int qa, qb;      // first elements of the two quads (VEC)
    bool split;
};

__device__ __forceinline__ Place place_of(int lane, int half, bool pairs)
{
    Place q;
    q.split = !pairs && 4 * lane < half;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int p = 4 * lane + j;
        const bool turned = !pairs && p < half;
        q.e0[j] = turned ? p : 2 * p;
        q.e1[j] = turned ? p + half : 2 * p + 1;
    }
    q.qa = q.e0[0];
    q.qb = q.split ? q.e1[0] : q.e0[0] + 4;
    return q;
}

// The lane's pairs (a[j], b[j]) of one row.  VEC: two quads, each inside the
// row or outside as a whole.
template <typename T, bool VEC>
__device__ __forceinline__ void load_pairs(const T *row, const Place &q, int D, float (&a)[4], float (&b)[4])
{
    if constexpr (VEC) {
        float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
        if (q.qa < D)
            u = load_quad(row + q.qa);
        if (q.qb < D)
            v = load_quad(row + q.qb);
        if (q.split) {
            a[0] = u.x, a[1] = u.y, a[2] = u.z, a[3] = u.w;
            b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
        } else {
            a[0] = u.x, b[0] = u.y, a[1] = u.z, b[1] = u.w;
            a[2] = v.x, b[2] = v.y, a[3] = v.z, b[3] = v.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = q.e0[j] < D ? load1(row + q.e0[j]) : 0.f;
            b[j] = q.e1[j] < D ? load1(row + q.e1[j]) : 0.f;
        }
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_pairs(T *row, const Place &q, int D, const float (&a)[4], const float (&b)[4])
{
    if constexpr (VEC) {
        if (q.split) {
            if (q.qa < D)
                store_quad(row + q.qa, a[0], a[1], a[2], a[3]);
            if (q.qb < D)
                store_quad(row + q.qb, b[0], b[1], b[2], b[3]);
        } else {
            if (q.qa < D)
                store_quad(row + q.qa, a[0], b[0], a[1], b[1]);
            if (q.qb < D)
                store_quad(row + q.qb, a[2], b[2], a[3], b[3]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (q.e0[j] < D)
                store1(row + q.e0[j], a[j]);
            if (q.e1[j] < D)
                store1(row + q.e1[j], b[j]);
        }
    }
}

// The sum over the LPH lanes of a group, in every lane of it.
template <int LPH>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int m = LPH / 2; m >= 1; m >>= 1)
        v += __shfl_xor(v, m, 64);
    return v;
}

template <typename T, int LPH, int HP, bool VEC, bool BWD>
__global__ void __launch_bounds__(kThreads) norm_kernel(NormArgs g)
{
    constexpr int kGroups = kThreads / LPH;   // rows of tokens side by side
    const int lane = threadIdx.x % LPH, grp = threadIdx.x / LPH;
    const bool second = (int)blockIdx.y >= g.segs0;
    const NormTensor &t = g.t[second ? 1 : 0];
    const int64_t h0 = (int64_t)(blockIdx.y - (second ? g.segs0 : 0)) * HP;
    const int D = g.D, half = g.half;
    const int heads = (int)min((int64_t)HP, t.H - h0);
    const Place q = place_of(lane, half, g.pairs);

    float w0[4], w1[4], s0[4], s1[4];   // weights, and the sums of their gradients
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w0[j] = (t.w && q.e0[j] < D) ? t.w[q.e0[j]] : 1.f;
        w1[j] = (t.w && q.e1[j] < D) ? t.w[q.e1[j]] : 1.f;
        s0[j] = s1[j] = 0.f;
    }

    for (int64_t tok = (int64_t)blockIdx.x * kGroups + grp; tok < g.tokens; tok += (int64_t)gridDim.x * kGroups) {
        const int b = (int)((uint32_t)tok / (uint32_t)g.L), l = (int)((uint32_t)tok % (uint32_t)g.L);
        const T *x = static_cast<const T *>(t.x) + b * t.sx.b + h0 * t.sx.h + l * t.sx.l;
        float xa[HP][4], xb[HP][4];
#pragma unroll
        for (int i = 0; i < HP; ++i)
            load_pairs<T, VEC>(x + min(i, heads - 1) * t.sx.h, q, D, xa[i], xb[i]);
        float da[BWD ? HP : 1][4], db[BWD ? HP : 1][4];
        if constexpr (BWD) {
            const T *dy = static_cast<const T *>(t.dy) + b * t.sdy.b + h0 * t.sdy.h + l * t.sdy.l;
#pragma unroll
            for (int i = 0; i < HP; ++i)
                load_pairs<T, VEC>(dy + min(i, heads - 1) * t.sdy.h, q, D, da[i], db[i]);
        }
        float c[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c[j] = 1.f, s[j] = 0.f;
        if (4 * lane < half) {
            int64_t p = g.pos ? (int64_t)g.pos[tok] : (int64_t)l;
            p = p < 0 ? 0 : (p < g.P ? p : g.P - 1);
            const float *cs = g.cs + p * half + 4 * lane, *sn = g.sn + p * half + 4 * lane;
            if ((half & 3) == 0) {
                const float4 u = *reinterpret_cast<const float4 *>(cs), v = *reinterpret_cast<const float4 *>(sn);
                c[0] = u.x, c[1] = u.y, c[2] = u.z, c[3] = u.w;
                s[0] = v.x, s[1] = v.y, s[2] = v.z, s[3] = v.w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (4 * lane + j < half)
                        c[j] = cs[j], s[j] = sn[j];
            }
        }
        T *out = static_cast<T *>(t.out) + b * t.so.b + h0 * t.so.h + l * t.so.l;
#pragma unroll
        for (int i = 0; i < HP; ++i) {
            if (HP > 1 && i >= heads)
                break;
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                ss += xa[i][j] * xa[i][j] + xb[i][j] * xb[i][j];
            const float r = 1.f / sqrtf(group_sum<LPH>(ss) * g.inv_n + g.eps);
            float ya[4], yb[4];
            if constexpr (!BWD) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = xa[i][j] * r * w0[j], bb = xb[i][j] * r * w1[j];
                    ya[j] = a * c[j] - bb * s[j];
                    yb[j] = a * s[j] + bb * c[j];
                }
            } else {
                float ea[4], eb[4], dot = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float a = da[i][j] * c[j] + db[i][j] * s[j], bb = db[i][j] * c[j] - da[i][j] * s[j];
                    xa[i][j] *= r;
                    xb[i][j] *= r;
                    s0[j] += a * xa[i][j];
                    s1[j] += bb * xb[i][j];
                    ea[j] = a * w0[j];
                    eb[j] = bb * w1[j];
                    dot += ea[j] * xa[i][j] + eb[j] * xb[i][j];
                }
                const float m = group_sum<LPH>(dot) * g.inv_n;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ya[j] = r * (ea[j] - xa[i][j] * m);
                    yb[j] = r * (eb[j] - xb[i][j] * m);
                }
            }
            store_pairs<T, VEC>(out + i * t.so.h, q, D, ya, yb);
        }
    }

    if constexpr (BWD) {
        if (!t.partial)
            return;
        // The workgroup's sums: its groups' rows through LDS, in their order.
        __shared__ float s_sum[kGroups][LPH * 8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s_sum[grp][lane * 8 + j] = s0[j];
            s_sum[grp][lane * 8 + 4 + j] = s1[j];
        }
        __syncthreads();
        const int64_t row = (int64_t)(blockIdx.y - (second ? g.segs0 : 0)) * gridDim.x + blockIdx.x;
        for (int u = threadIdx.x; u < LPH * 8; u += kThreads) {
            const Place at = place_of(u / 8, half, g.pairs);
            const int e = (u & 4) ? at.e1[u & 3] : at.e0[u & 3];
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                v += s_sum[i][u];
            if (e < D)
                t.partial[row * D + e] = v;
        }
    }
}

// dw[e] = the sum of `rows` partial rows; blockIdx.y picks the tensor.
constexpr int kSumRows = 16;
struct SumArgs {
    const float *partial[2];
    float *dw[2];
    int64_t rows[2];
    int D;
};

__global__ void __launch_bounds__(64 * kSumRows) norm_sum_kernel(SumArgs a)
{
    __shared__ float s_part[kSumRows][64];
    const int which = blockIdx.y, col = blockIdx.x * 64 + (threadIdx.x & 63), part = threadIdx.x >> 6;
    if (!a.dw[which])
        return;
    float v = 0.f;
    if (col < a.D) {
#pragma unroll 8
        for (int64_t i = part; i < a.rows[which]; i += kSumRows)
            v += a.partial[which][i * a.D + col];
    }
    s_part[part][threadIdx.x & 63] = v;
    __syncthreads();
    if (part == 0 && col < a.D) {
#pragma unroll
        for (int i = 1; i < kSumRows; ++i)
            v += s_part[i][threadIdx.x];
        a.dw[which][col] = v;
    }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------

constexpr uint32_t kNormFlags = PDSSM_DATA_BF16 | PDSSM_NORM_L2 | PDSSM_ROPE_PAIRS;

int check_norm_dims(int64_t B, int64_t Hq, int64_t Hk, int64_t L, int32_t D, int32_t R, int64_t P)
{
    if (B < 0 || Hq < 0 || Hk < 0 || L < 0 || Hq > 32768 || Hk > 32768 || D < 1 || D > kMaxD || R < 0 || R > D ||
        (R & 1) || (R > 0 && P < 1))
        return PDSSM_ERR_DIM;
    if ((double)B * (double)L > 2147483647.0 || (double)P * D > 9.0e18)
        return PDSSM_ERR_DIM;
    return PDSSM_OK;
}

// Every row of the tensor can be read in quads of four elements.
bool quads(const void *p, const pdssm_strides &s, int esize)
{
    return ((uintptr_t)p % (4 * esize)) == 0 && (s.b % 4) == 0 && (s.h % 4) == 0 && (s.l % 4) == 0;
}

// Heads a lane takes of one token: four, unless the call has so few rows that
// more lanes in flight shorten it (2^16 rows are 256 workgroups at D = 128).
int heads_per_lane(int64_t rows) { return rows > (1 << 16) ? 4 : 1; }

struct Plan {
    int lph, hp;
    int64_t segs[2], blocks;
};

Plan plan_of(int64_t B, int64_t Hq, int64_t Hk, int64_t L, int32_t D, bool bwd)
{
    Plan p;
    p.lph = 1;
    while (p.lph * 8 < D)
        p.lph *= 2;
    p.lph = p.lph < 8 ? 8 : p.lph;
    p.hp = heads_per_lane(B * L * (Hq + Hk));
    p.segs[0] = (Hq + p.hp - 1) / p.hp;
    p.segs[1] = (Hk + p.hp - 1) / p.hp;
    const int64_t groups = kThreads / p.lph;
    p.blocks = (B * L + groups - 1) / groups;
    const int64_t segs = p.segs[0] + p.segs[1];
    if (bwd && segs > 0) {
        const int64_t most = (kBwdGroups + segs - 1) / segs;
        p.blocks = p.blocks < most ? p.blocks : most;
    }
    return p;
}

template <typename T, int LPH, int HP, bool BWD>
void launch_vec(const NormArgs &a, bool vec, dim3 grid, hipStream_t stream)
{
    if (vec)
        hipLaunchKernelGGL((norm_kernel<T, LPH, HP, true, BWD>), grid, dim3(kThreads), 0, stream, a);
    else
        hipLaunchKernelGGL((norm_kernel<T, LPH, HP, false, BWD>), grid, dim3(kThreads), 0, stream, a);
}

template <typename T, bool BWD>
void launch_norm(const NormArgs &a, const Plan &p, bool vec, hipStream_t stream)
{
    const dim3 grid((unsigned)p.blocks, (unsigned)(p.segs[0] + p.segs[1]));
#define PDSSM_NORM_CASE(n)                                   \
    case n:                                                  \
        if (p.hp == 4)                                       \
            launch_vec<T, n, 4, BWD>(a, vec, grid, stream);  \
        else                                                 \
            launch_vec<T, n, 1, BWD>(a, vec, grid, stream);  \
        break
    switch (p.lph) {
        PDSSM_NORM_CASE(8);
        PDSSM_NORM_CASE(16);
        PDSSM_NORM_CASE(32);
    }
#undef PDSSM_NORM_CASE
}

pdssm_strides contiguous(int64_t H, int64_t L, int64_t D) { return {H * L * D, L * D, D}; }

struct NormCall {
    const void *x[2], *dy[2];
    void *out[2];
    const float *w[2];
    float *dw[2];
    const float *cs, *sn;
    const int32_t *pos;
    int64_t B, H[2], L;
    int32_t D, R;
    int64_t P;
    float eps;
    uint32_t flags;
    const pdssm_strides *strides;
};

int norm_call(const NormCall &c, bool bwd, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    int rc = check_norm_dims(c.B, c.H[0], c.H[1], c.L, c.D, c.R, c.P);
    if (rc != PDSSM_OK)
        return rc;
    if (c.flags & ~kNormFlags)
        return PDSSM_ERR_FLAGS;
    const int64_t tokens = c.B * c.L;
    const int esize = (c.flags & PDSSM_DATA_BF16) ? 2 : 4;
    const bool has[2] = {tokens > 0 && c.H[0] > 0, tokens > 0 && c.H[1] > 0};
    const bool any = has[0] || has[1];
    if (any && c.R > 0 && (!c.cs || !c.sn))
        return PDSSM_ERR_NULL;
    if (any && c.R > 0 && (((uintptr_t)c.cs | (uintptr_t)c.sn) & 15u))
        return PDSSM_ERR_ALIGN;
    if (any && c.pos && ((uintptr_t)c.pos & 3u))
        return PDSSM_ERR_ALIGN;
    NormArgs a;
    bool vec = (c.D % 4) == 0 && ((c.flags & PDSSM_ROPE_PAIRS) || (c.R % 8) == 0);
    for (int i = 0; i < 2; ++i) {
        NormTensor &t = a.t[i];
        t.x = c.x[i], t.dy = c.dy[i], t.out = c.out[i], t.w = c.w[i], t.partial = nullptr, t.H = c.H[i];
        const pdssm_strides whole = contiguous(c.H[i], c.L, c.D);
        t.sx = c.strides ? c.strides[i] : whole;
        t.sdy = c.strides && bwd ? c.strides[2 + i] : whole;
        t.so = c.strides ? c.strides[(bwd ? 4 : 2) + i] : whole;
        if (((uintptr_t)c.w[i] | (uintptr_t)c.dw[i]) & 3u)
            return PDSSM_ERR_ALIGN;
        if (!has[i])
            continue;
        if (!t.x || !t.out || (bwd && !t.dy))
            return PDSSM_ERR_NULL;
        if (((uintptr_t)t.x | (uintptr_t)t.out | (uintptr_t)t.dy) & (uintptr_t)(esize - 1))
            return PDSSM_ERR_ALIGN;
        vec = vec && quads(t.x, t.sx, esize) && quads(t.out, t.so, esize) && (!bwd || quads(t.dy, t.sdy, esize));
    }
    const bool sums = c.dw[0] || c.dw[1];
    const Plan p = plan_of(c.B, has[0] ? c.H[0] : 0, has[1] ? c.H[1] : 0, c.L, c.D, bwd);
    if (any && sums) {
        if (!workspace)
            return PDSSM_ERR_NULL;
        if (!aligned16(workspace))
            return PDSSM_ERR_ALIGN;
        if (workspace_bytes < pdssm_qk_norm_rope_bwd_workspace_bytes(c.B, c.H[0], c.H[1], c.L, c.D))
            return PDSSM_ERR_WORKSPACE;
        float *rows = static_cast<float *>(workspace);
        a.t[0].partial = c.dw[0] ? rows : nullptr;
        a.t[1].partial = c.dw[1] ? rows + p.segs[0] * p.blocks * c.D : nullptr;
    }
    if (any) {
        a.cs = c.cs, a.sn = c.sn, a.pos = c.pos, a.P = c.P;
        a.tokens = (int)tokens, a.L = (int)c.L, a.D = c.D, a.half = c.R / 2;
        a.segs0 = (int)p.segs[0];
        a.inv_n = (c.flags & PDSSM_NORM_L2) ? 1.f : 1.f / (float)c.D;
        a.eps = c.eps;
        a.pairs = (c.flags & PDSSM_ROPE_PAIRS) != 0;
        if (esize == 2) {
            if (bwd)
                launch_norm<uint16_t, true>(a, p, vec, stream);
            else
                launch_norm<uint16_t, false>(a, p, vec, stream);
        } else {
            if (bwd)
                launch_norm<float, true>(a, p, vec, stream);
            else
                launch_norm<float, false>(a, p, vec, stream);
        }
        rc = hip_status(hipGetLastError());
        if (rc != PDSSM_OK)
            return rc;
    }
    if (!sums)
        return PDSSM_OK;
    SumArgs s;
    for (int i = 0; i < 2; ++i) {
        s.partial[i] = a.t[i].partial;
        s.dw[i] = c.dw[i];
        s.rows[i] = has[i] ? p.segs[i] * p.blocks : 0;
    }
    s.D = c.D;
    hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((c.D + 63) / 64), 2), dim3(64 * kSumRows), 0, stream, s);
    return hip_status(hipGetLastError());
}

}  // namespace
}  // namespace pdssm

using namespace pdssm;

extern "C" size_t pdssm_qk_norm_rope_bwd_workspace_bytes(int64_t B, int64_t Hq, int64_t Hk, int64_t L, int32_t D)
{
    if (check_norm_dims(B, Hq, Hk, L, D, 0, 0) != PDSSM_OK)
        return 0;
    // With or without either tensor the call has at most this many rows of sums.
    const Plan p = plan_of(B, Hq, Hk, L, D, true);
    const int64_t rows = (p.segs[0] + p.segs[1]) * p.blocks;
    return (size_t)((rows > 0 ? rows : 1) * D * (int64_t)sizeof(float) + 15) / 16 * 16;
}

extern "C" int pdssm_qk_norm_rope_fwd(const void *q, const void *k, const float *wq, const float *wk,
                                      const float *cos, const float *sin, const int32_t *pos, void *q_out,
                                      void *k_out, int64_t B, int64_t Hq, int64_t Hk, int64_t L, int32_t D,
                                      int32_t R, int64_t P, float eps, uint32_t flags,
                                      const pdssm_strides *strides, hipStream_t stream)
{
    NormCall c = {};
    c.x[0] = q, c.x[1] = k, c.out[0] = q_out, c.out[1] = k_out, c.w[0] = wq, c.w[1] = wk;
    c.cs = cos, c.sn = sin, c.pos = pos, c.B = B, c.H[0] = Hq, c.H[1] = Hk, c.L = L, c.D = D, c.R = R, c.P = P;
    c.eps = eps, c.flags = flags, c.strides = strides;
    return norm_call(c, false, nullptr, 0, stream);
}

extern "C" int pdssm_qk_norm_rope_bwd(const void *q, const void *k, const float *wq, const float *wk,
                                      const float *cos, const float *sin, const int32_t *pos, const void *dq_out,
                                      const void *dk_out, void *dq, void *dk, float *dwq, float *dwk, int64_t B,
                                      int64_t Hq, int64_t Hk, int64_t L, int32_t D, int32_t R, int64_t P, float eps,
                                      uint32_t flags, const pdssm_strides *strides, void *workspace,
                                      size_t workspace_bytes, hipStream_t stream)
{
    NormCall c = {};
    c.x[0] = q, c.x[1] = k, c.dy[0] = dq_out, c.dy[1] = dk_out, c.out[0] = dq, c.out[1] = dk;
    c.w[0] = wq, c.w[1] = wk, c.dw[0] = dwq, c.dw[1] = dwk;
    c.cs = cos, c.sn = sin, c.pos = pos, c.B = B, c.H[0] = Hq, c.H[1] = Hk, c.L = L, c.D = D, c.R = R, c.P = P;
    c.eps = eps, c.flags = flags, c.strides = strides;
    return norm_call(c, true, workspace, workspace_bytes, stream);
}
