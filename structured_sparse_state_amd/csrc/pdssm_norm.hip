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
// lanes, and a lane holds eight of the row's pairs (a, b) whole, so the
// rotation needs nothing from another lane; only the row's sum crosses lanes.
// In either pairing a lane's values are two runs of eight, one 16-byte load
// of bf16 each.  A lane takes the same place in HP heads of one token (all
// their loads are issued before the first is used), with its weights, cosines
// and sines loaded once for them.
//
// 8 x 4096 tokens of 40 heads of 128 in bf16: 127 us forward (5.3 TB/s; a copy
// of the same bytes takes 124 us) and 213 + 7 us backward (4.6 TB/s; the sum of two
// tensors into a third 168 us), whose registers leave two waves to a SIMD; in
// fp32 242 us (5.5 TB/s) and 484 us (4.2 TB/s).
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
    int segs0, segs1;         // segments of HP heads of t[0] and of t[1]
    float inv_n, eps;
    bool pairs, heads_first;
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

// Eight consecutive values as they lie in memory (bf16 ones are unpacked only
// where they are used: a lane holds several heads' rows).
template <typename T>
struct Run;
template <>
struct Run<uint16_t> {
    uint4 w;
    __device__ __forceinline__ void clear() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const uint16_t *p) { w = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void set(int j, float v)     // of a cleared run
    {
        const uint32_t h = (__float_as_uint(v) >> 16) << (16 * (j & 1));
        j / 2 == 0 ? w.x |= h : j / 2 == 1 ? w.y |= h : j / 2 == 2 ? w.z |= h : w.w |= h;
    }
    __device__ __forceinline__ float get(int j) const
    {
        const uint32_t u = j / 2 == 0 ? w.x : j / 2 == 1 ? w.y : j / 2 == 2 ? w.z : w.w;
        return (j & 1) ? bf16_hi(u) : bf16_lo(u);
    }
};
template <>
struct Run<float> {
    float4 a, b;
    __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void load(const float *p)
    {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ void set(int j, float v)
    {
        float4 &q = j < 4 ? a : b;
        (j & 3) == 0 ? q.x = v : (j & 3) == 1 ? q.y = v : (j & 3) == 2 ? q.z = v : q.w = v;
    }
    __device__ __forceinline__ float get(int j) const
    {
        const float4 &q = j < 4 ? a : b;
        return (j & 3) == 0 ? q.x : (j & 3) == 1 ? q.y : (j & 3) == 2 ? q.z : q.w;
    }
};

template <typename T>
__device__ __forceinline__ void store_run(T *p, const float (&v)[8])
{
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(f32x2_to_bf16x2_rne(v[0], v[1]), f32x2_to_bf16x2_rne(v[2], v[3]),
                                                   f32x2_to_bf16x2_rne(v[4], v[5]), f32x2_to_bf16x2_rne(v[6], v[7]));
    } else {
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
}

constexpr int kPairs = 8;       // pairs of a lane

// Where a lane's pairs lie in a row.  Pair p of the row is (p, p + half) when
// it turns in half mode, else (2p, 2p + 1); `split`: the lane's first elements
// are one run of eight and its second ones another, else the sixteen are
// consecutive.  Elements at D and beyond do not exist.
struct Place {
    int first, half;
    bool split, pairs;
    __device__ __forceinline__ Place(int lane, int half_, bool pairs_)
    {
        first = kPairs * lane, half = half_, pairs = pairs_;
        split = !pairs && first < half;
    }
    __device__ __forceinline__ int e0(int j) const { return !pairs && first + j < half ? first + j : 2 * (first + j); }
    __device__ __forceinline__ int e1(int j) const
    {
        return !pairs && first + j < half ? first + j + half : 2 * (first + j) + 1;
    }
    __device__ __forceinline__ int run0() const { return split ? first : 2 * first; }
    __device__ __forceinline__ int run1() const { return split ? first + half : 2 * first + 8; }
};

// A lane's pairs of one row.  VEC: two runs, each inside the row or outside
// as a whole; else the pairs' first and second elements one by one.
template <typename T, bool VEC>
struct Pairs {
    Run<T> u, v;
    __device__ __forceinline__ void load(const T *row, const Place &q, int D)
    {
        u.clear();
        v.clear();
        if constexpr (VEC) {
            if (q.run0() < D)
                u.load(row + q.run0());
            if (q.run1() < D)
                v.load(row + q.run1());
        } else {
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                if (q.e0(j) < D)
                    u.set(j, load1(row + q.e0(j)));
                if (q.e1(j) < D)
                    v.set(j, load1(row + q.e1(j)));
            }
        }
    }
    __device__ __forceinline__ void get(const Place &q, float (&a)[kPairs], float (&b)[kPairs]) const
    {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            a[j] = !VEC || q.split ? u.get(j) : j < 4 ? u.get((2 * j) & 7) : v.get((2 * j) & 7);
            b[j] = !VEC || q.split ? v.get(j) : j < 4 ? u.get((2 * j + 1) & 7) : v.get((2 * j + 1) & 7);
        }
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store_pairs(T *row, const Place &q, int D, const float (&a)[kPairs], const float (&b)[kPairs])
{
    if constexpr (VEC) {
        float u[8], v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u[j] = q.split ? a[j] : (j & 1) ? b[j / 2] : a[j / 2];
            v[j] = q.split ? b[j] : (j & 1) ? b[4 + j / 2] : a[4 + j / 2];
        }
        if (q.run0() < D)
            store_run(row + q.run0(), u);
        if (q.run1() < D)
            store_run(row + q.run1(), v);
    } else {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            if (q.e0(j) < D)
                store1(row + q.e0(j), a[j]);
            if (q.e1(j) < D)
                store1(row + q.e1(j), b[j]);
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
    constexpr int kGroups = kThreads / LPH;
    const int lane = threadIdx.x % LPH, grp = threadIdx.x / LPH;
    const int D = g.D, half = g.half;
    const Place q(lane, half, g.pairs);

    // A group takes one token and HP of its heads at a time: the backward a
    // segment of heads (blockIdx.y) and tokens in turn, so that the sums of
    // the weight's gradient stay in its registers; the forward any pair of the
    // two, heads first where a token's heads lie together in memory.
    const int segs = g.segs0 + g.segs1;
    const uint32_t items = BWD ? (uint32_t)g.tokens : (uint32_t)g.tokens * segs;
    float s0[kPairs], s1[kPairs];       // sums of the weights' gradients
#pragma unroll
    for (int j = 0; j < kPairs; ++j)
        s0[j] = s1[j] = 0.f;

    for (uint32_t item = blockIdx.x * kGroups + grp; item < items; item += gridDim.x * kGroups) {
        uint32_t tok, seg;
        if constexpr (BWD)
            tok = item, seg = blockIdx.y;
        else if (g.heads_first)
            tok = item / segs, seg = item - tok * segs;
        else
            seg = item / (uint32_t)g.tokens, tok = item - seg * (uint32_t)g.tokens;
        const bool second = (int)seg >= g.segs0;
        const NormTensor &t = g.t[second ? 1 : 0];
        const int64_t h0 = (int64_t)(second ? seg - g.segs0 : seg) * HP;
        const int heads = (int)min((int64_t)HP, t.H - h0);
        const int b = (int)(tok / (uint32_t)g.L), l = (int)(tok - b * (uint32_t)g.L);
        const T *x = static_cast<const T *>(t.x) + b * t.sx.b + h0 * t.sx.h + l * t.sx.l;
        Pairs<T, VEC> px[HP], pd[BWD ? HP : 1];
#pragma unroll
        for (int i = 0; i < HP; ++i)
            px[i].load(x + min(i, heads - 1) * t.sx.h, q, D);
        if constexpr (BWD) {
            const T *dy = static_cast<const T *>(t.dy) + b * t.sdy.b + h0 * t.sdy.h + l * t.sdy.l;
#pragma unroll
            for (int i = 0; i < HP; ++i)
                pd[i].load(dy + min(i, heads - 1) * t.sdy.h, q, D);
        }
        float c[kPairs], s[kPairs], w0[kPairs], w1[kPairs];
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
            c[j] = 1.f, s[j] = 0.f, w0[j] = w1[j] = 1.f;
        if (q.first < half) {
            int64_t p = g.pos ? (int64_t)g.pos[tok] : (int64_t)l;
            p = p < 0 ? 0 : (p < g.P ? p : g.P - 1);
            const float *cs = g.cs + p * half + q.first, *sn = g.sn + p * half + q.first;
            if ((half & 7) == 0) {
                Run<float> rc, rs;
                rc.load(cs);
                rs.load(sn);
#pragma unroll
                for (int j = 0; j < kPairs; ++j)
                    c[j] = rc.get(j), s[j] = rs.get(j);
            } else {
#pragma unroll
                for (int j = 0; j < kPairs; ++j)
                    if (q.first + j < half)
                        c[j] = cs[j], s[j] = sn[j];
            }
        }
        if (t.w) {
            Pairs<float, VEC> pw;
            pw.load(t.w, q, D);
            pw.get(q, w0, w1);
        }
        T *out = static_cast<T *>(t.out) + b * t.so.b + h0 * t.so.h + l * t.so.l;
#pragma unroll
        for (int i = 0; i < HP; ++i) {
            if (HP > 1 && i >= heads)
                break;
            float xa[kPairs], xb[kPairs], ss = 0.f;
            px[i].get(q, xa, xb);
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
                ss += xa[j] * xa[j] + xb[j] * xb[j];
            const float r = rsqrtf(group_sum<LPH>(ss) * g.inv_n + g.eps);
            float ya[kPairs], yb[kPairs];
            if constexpr (!BWD) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const float a = xa[j] * r * w0[j], bb = xb[j] * r * w1[j];
                    ya[j] = a * c[j] - bb * s[j];
                    yb[j] = a * s[j] + bb * c[j];
                }
            } else {
                float da[kPairs], db[kPairs], ea[kPairs], eb[kPairs], dot = 0.f;
                pd[i].get(q, da, db);
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const float a = da[j] * c[j] + db[j] * s[j], bb = db[j] * c[j] - da[j] * s[j];
                    xa[j] *= r;
                    xb[j] *= r;
                    s0[j] += a * xa[j];
                    s1[j] += bb * xb[j];
                    ea[j] = a * w0[j];
                    eb[j] = bb * w1[j];
                    dot += ea[j] * xa[j] + eb[j] * xb[j];
                }
                const float m = group_sum<LPH>(dot) * g.inv_n;
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    ya[j] = r * (ea[j] - xa[j] * m);
                    yb[j] = r * (eb[j] - xb[j] * m);
                }
            }
            store_pairs<T, VEC>(out + i * t.so.h, q, D, ya, yb);
        }
    }

    if constexpr (BWD) {
        const bool second = (int)blockIdx.y >= g.segs0;
        const NormTensor &t = g.t[second ? 1 : 0];
        if (!t.partial)
            return;
        // The workgroup's sums: its groups' rows through LDS, in their order.
        __shared__ float s_sum[kGroups][LPH * 2 * kPairs];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            s_sum[grp][lane * 2 * kPairs + j] = s0[j];
            s_sum[grp][lane * 2 * kPairs + kPairs + j] = s1[j];
        }
        __syncthreads();
        const int64_t row = (int64_t)(blockIdx.y - (second ? g.segs0 : 0)) * gridDim.x + blockIdx.x;
        for (int u = threadIdx.x; u < LPH * 2 * kPairs; u += kThreads) {
            const Place at(u / (2 * kPairs), half, g.pairs);
            const int e = (u & kPairs) ? at.e1(u % kPairs) : at.e0(u % kPairs);
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
                v += s_sum[i][u];
            if (e < D)
                t.partial[row * D + e] = v;
        }
    }
}

// dw[e] = the sum of `rows` partial rows; blockIdx.y picks the tensor.  A
// workgroup takes 16 columns, 64 rows at a time.
constexpr int kSumRows = 64, kSumCols = 16;
struct SumArgs {
    const float *partial[2];
    float *dw[2];
    int64_t rows[2];
    int D;
};

__global__ void __launch_bounds__(kSumRows *kSumCols) norm_sum_kernel(SumArgs a)
{
    __shared__ float s_part[kSumRows][kSumCols + 1];
    const int which = blockIdx.y, c = threadIdx.x % kSumCols, part = threadIdx.x / kSumCols;
    const int col = blockIdx.x * kSumCols + c;
    if (!a.dw[which])
        return;
    float v = 0.f;
    if (col < a.D) {
#pragma unroll 8
        for (int64_t i = part; i < a.rows[which]; i += kSumRows)
            v += a.partial[which][i * a.D + col];
    }
    s_part[part][c] = v;
    __syncthreads();
    if (threadIdx.x < kSumCols && col < a.D) {
        for (int i = 1; i < kSumRows; ++i)
            v += s_part[i][c];
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
    // Items (a token and a head) are counted in 32 bits.
    if ((double)B * (double)L * (double)(Hq + Hk > 1 ? Hq + Hk : 1) > 2147483647.0 || (double)P * D > 9.0e18)
        return PDSSM_ERR_DIM;
    return PDSSM_OK;
}

// Every row begins on 16 bytes.
bool runs(const void *p, const pdssm_strides &s, int esize)
{
    const int n = 16 / esize;
    return aligned16(p) && s.b % n == 0 && s.h % n == 0 && s.l % n == 0;
}

// Heads a lane takes of one token.  Four spare the loads of weights, cosines
// and sines and keep more rows in flight; with few rows, one keeps more of the
// device busy.  40 heads of 128 a token, bf16, a whole call in us with one head
// and four: forward (R = 128) 20480 rows 4.7 and 5.1, 65520 rows 9.3 and 7.6,
// 327680 rows 32.6 and 31.5, 1.3 million rows 165 and 125; backward (R = 64, adjacent
// pairs, more registers) 65520 rows 18.0 and 20.3, 327680 rows 48.4 and 52.0,
// 1.3 million rows 235 and 219.  fp32, 1.3 million rows: 246 and 242, 497 and 484.
int heads_per_lane(int64_t rows, bool bwd) { return rows > (bwd ? 1 << 19 : 1 << 15) ? 4 : 1; }

struct Plan {
    int lph, hp;
    int64_t segs[2], blocks;
};

Plan plan_of(int64_t B, int64_t Hq, int64_t Hk, int64_t L, int32_t D, bool bwd)
{
    Plan p;
    p.lph = 1;
    while (p.lph * 2 * kPairs < D)
        p.lph *= 2;
    p.lph = p.lph < 4 ? 4 : p.lph;
    p.hp = heads_per_lane(B * L * (Hq + Hk), bwd);
    p.segs[0] = (Hq + p.hp - 1) / p.hp;
    p.segs[1] = (Hk + p.hp - 1) / p.hp;
    const int64_t groups = kThreads / p.lph, segs = p.segs[0] + p.segs[1];
    // (a launch has fewer than 2^32 threads; the groups take items in turn)
    p.blocks = (B * L * (bwd ? 1 : segs) + groups - 1) / groups;
    p.blocks = p.blocks < 1 << 23 ? p.blocks : 1 << 23;
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
    const dim3 grid((unsigned)p.blocks, (unsigned)(BWD ? p.segs[0] + p.segs[1] : 1));
#define PDSSM_NORM_CASE(n)                                   \
    case n:                                                  \
        if (p.hp == 4)                                       \
            launch_vec<T, n, 4, BWD>(a, vec, grid, stream);  \
        else                                                 \
            launch_vec<T, n, 1, BWD>(a, vec, grid, stream);  \
        break
    switch (p.lph) {
        PDSSM_NORM_CASE(4);
        PDSSM_NORM_CASE(8);
        PDSSM_NORM_CASE(16);
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
    // Rows of whole runs are read as runs, others value by value: a table's
    // later rows are then no less aligned than needed.
    if (any && c.R > 0 && (((uintptr_t)c.cs | (uintptr_t)c.sn) & (c.R % 16 == 0 ? 15u : 3u)))
        return PDSSM_ERR_ALIGN;
    if (any && c.pos && ((uintptr_t)c.pos & 3u))
        return PDSSM_ERR_ALIGN;
    NormArgs a;
    bool vec = (c.D % 8) == 0 && ((c.flags & PDSSM_ROPE_PAIRS) || (c.R % 16) == 0);
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
        vec = vec && runs(t.x, t.sx, esize) && runs(t.out, t.so, esize) && (!bwd || runs(t.dy, t.sdy, esize)) &&
              aligned16(t.w);
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
        a.segs0 = (int)p.segs[0], a.segs1 = (int)p.segs[1];
        const NormTensor &most = a.t[c.H[0] >= c.H[1] ? 0 : 1];
        a.heads_first = most.sx.h <= most.sx.l;
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
    hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((c.D + kSumCols - 1) / kSumCols), 2), dim3(kSumRows * kSumCols), 0, stream, s);
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
