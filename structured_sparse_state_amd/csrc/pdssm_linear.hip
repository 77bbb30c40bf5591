// Linear attention with decays (include/pdssm_block.h): forward, gradients, step.
//
// A chunk of 64 steps at once, from the state S before it.  With G the running
// sum of g inside the chunk, rise = e^G, left = e^(G_last - G), whole =
// e^G_last, decay[i,j] = e^(G_i - G_j) for j <= i,
//     O  = scale rise Q S + P V,   P = scale * lower part of (Q K^T . decay)
//     S <- whole S + K^T (left V).
// The gradients are three walks of the same form, one forward and two back from
// the gradient dS of the state after the last chunk:
//     dQ = scale rise dO S^T + X K,   X = scale * lower part of (dO V^T . decay)
//          S^T <- whole S^T + V^T (left K)
//     dV = left K dS + P^T dO,        dS   <- whole dS   + Q^T (scale rise dO)
//     dK = left V dS^T + X^T Q,       dS^T <- whole dS^T + dO^T (scale rise Q).
// So one walk serves all:
//     Y = read X1 S + M X3,   M = scale * triangle of (X1 X2^T . decay),
//     S <- whole S + X2^T (write X3)
// with (X1, X2, X3) = (q, k, v), (dO, v, k), (k, q, dO), (v, dO, q), the lower
// triangle going forward and the upper one going back.
// The gradient of g is the sum of what crosses a step,
//     dg_t = <whole S, dS> + sum over i >= t of q_i . (scale rise dO S^T)_i
//            + sum over j < t of k_j . (left V dS^T)_j
//            + sum over j < t <= i of X_ij q_i . k_j :
// the walk of dQ keeps the states before the chunks and its share of the rows'
// products, the walk of dK, whose state has the same shape and the same owner
// for every value, adds the rest.
//
// The walk.  A workgroup takes SL = 64 or 128 columns of one head's state over the
// chunks of a segment.  Its first SL / 16 waves ("chain") own 16 columns each, whose
// recurrences are independent, and keep them in registers in the matrix cores'
// result layout, from where they feed the products without leaving the wave.  The
// four waves behind them ("help") bring the next chunk's rows to LDS, sum its gates
// and form M, all ahead of the chain; a barrier ends each chunk.  States, M and the
// weighted X3 enter the products as three bf16 parts (all 24 bits); bf16 rows are
// one part, fp32 rows three.  Parts that meet bf16 rows are cut off (24 bits in three
// parts, nothing left out); three parts against three leave out the products of
// order 3 and more, so those are rounded, which keeps them smaller.
//
// Growth.  Decays inside a chunk are e^(sum of g): sums above 88 are more than fp32
// holds, and infinity times a state, a key or a value that is zero would be NaN where
// the definition gives zero.  Where the positive gates of some chunk add up to more
// than 60 the walk is done a second time, step by step, with factors of any size as a
// float and a power of two (8 x 32 heads of 64, 4096 steps: 1.9 ms forward, 5.7 back,
// where the others take 0.15 and 0.6).
//
// What bounds it, at 64 x 64: in every chunk the chain's products, one after another
// on the state (about 3400 to 4000 clocks; 284 matrix instructions of 16 clocks each
// over the workgroup), and the help waves' way from loads through LDS to M (about
// 3500), between the same barriers.  8 x 32 heads of 64, 4096 steps, forward, one decay
// a head: 136 to 148 us by the machine, 541 MB at 3.7 to 4.0 TB/s (the rows alone,
// staged and nothing else, 75 us); 150 to 158 with gates of every step.
// At 128 x 128 a chunk takes 5.8 to 6.3 us (walks of 9 chunks 52 to 57 us).  Of that
// its matrix instructions are 1.6 us; the eight chain waves read X1, X2 and M each for
// itself, 128, 128 and 147 KB, which at the rates of such reads alone (152, 303 and 520
// bytes a ns) is 1.6 us more; the rest has not been taken apart.  The walk moves
// 170 MB at 3.0 to 3.2 TB/s meanwhile; those of dQ and dV in the backward, which keep
// the states, 979 MB at 4.5 TB/s, nearly a copy's rate.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "pdssm_block.h"
#include "pdssm_chunk.h"

namespace pdssm {
namespace {

constexpr int kMaxDim = 128;
constexpr int kHelp = 256;          // help threads
// A workgroup's columns SL of the state are 64 or 128, a chain wave for each 16.
constexpr int walk_threads(int SL) { return SL / 16 * 64 + kHelp; }

// Vectors of a chunk in LDS: what the rows read of the state and write to it,
// the state's own decay, G log2(e) as a pair of floats and the steps that
// empty the state, counted; for dg what dQ's walk left in `reads`.
enum LinVec { kRead, kWrite, kWhole, kGhi, kGlo, kResets, kReads, kVecs };

struct Walk {
    Rows x1, x2, x3, y;
    Rows x4;                // dg: the rows beside y's (q for dQ, k for dK)
    bool kv1, kv2, kv3, kvy;        // rows of the key heads
    bool wide;              // y: fp32 [B*Hv][L][pitch] whatever the type of the data
    int D1, D3, groups;     // contraction, columns, groups of 16 columns that are kept
    const float *start;     // the state before the first chunk of the walk, NULL: zero
    float *end;             // and after its last, NULL: not wanted
    int row, col;           // strides of a state's values along contraction and columns
    float *starts;          // [segs + 1]: states before the segments, see native()
    float2 *wholes;         // [segs][heads]: the segments' decays, as a float and a power of two
    int segs, seg_chunks;
};

struct LinArgs {
    Walk w[3];
    Rows g;
    Rows dg;
    float *kept;            // [NC]: the states before the chunks, see native()
    float *reads;           // [NC][heads][groups][64]: q . what dQ reads of S
    float *dg_part;         // [slices][heads][L], or NULL: dg itself
    int64_t heads;          // B*Hv
    int64_t blocks;         // below 2^32, by the limit on B Hv
    bool started;           // s0 is given
    int first, last;        // walks of this launch
    int Hk, Hv, L, NC;
    float scale;
};

enum Mode { kOut, kScan };          // outputs; the last state alone
enum Gate { kNone, kKeep, kGrad };  // what a walk does for dg
enum Pass { kFast, kCareful, kSteps };      // see walk_pass

// 16 columns of a state as a chain wave holds them: group `group` of state
// number n of a head, [KD / 16][64 lanes] four values each.
template <int KD>
__device__ __forceinline__ float *native(float *p, int64_t n, int64_t heads, int groups, int64_t head, int group, int lane)
{
    return p + (((n * heads + head) * groups + group) * (KD / 16) * 64 + lane) * 4;
}

template <int KD, bool BF16, int SL>
struct LinLds {
    static constexpr int kChain = SL / 16;
    using T1 = Tile<KD, BF16, kHelp, true>;
    using T3 = Tile<SL, BF16, kHelp, true>;
    using M = Tri<false, kHelp>;                    // (both triangles take as much)
    // bf16: the chain reads one half while the help waves fill the other.  Three
    // parts of fp32 rows leave no room for that.
    static constexpr int kHalves = BF16 ? 2 : 1;
    // in uint16_t
    static constexpr int kX1 = 0;
    static constexpr int kX2 = kX1 + kHalves * T1::kSize;
    static constexpr int kX3 = kX2 + kHalves * T1::kSize;
    static constexpr int kM = kX3 + kHalves * T3::kSize;
    // in floats
    static constexpr int kVec = (kM + kHalves * M::kSize) / 2;
    static constexpr int kCuts = kVec + 4 * kVecs * kC;             // (the gates' vectors are a chunk further ahead)
    static constexpr int kWrites = kCuts + 2 * Cuts::kSize;       // [chain waves][64]: k . what dK reads of dS
    static constexpr int kCross = kWrites + 2 * kChain * kC;        // [chain waves]: <whole S, dS>
    static constexpr int kFlag = kCross + 2 * kChain;               // [4] help waves, [chain waves] spoiled
    static constexpr size_t kBytes = (kFlag + 4 + kChain) * 4;
};

// Values of a state in memory, a lane's column and rows 16 m + 4 g + r.
template <int KD, typename F>
__device__ __forceinline__ void each_value(const Walk &w, int col, int lane, F f)
{
#pragma unroll
    for (int m = 0; m < KD / 16; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * m + 4 * (lane >> 4) + r;
            f(m, r, row < w.D1 && col < w.D3, row * w.row + col * w.col);
        }
}

// c + A B for the tiles FIRST .. LAST side by side, part products of order
// below 3, the small ones first.
template <int FIRST, int LAST, int N, int NA, int NB>
__device__ __forceinline__ void mma_tiles(const Frag<NA> &a, const Frag<NB> (&b)[N], f32x4 (&c)[N])
{
#pragma unroll
    for (int o = 2; o >= 0; --o)
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int j = o - i;
            if (j >= 0 && j < NB) {
#pragma unroll
                for (int t = FIRST; t <= LAST; ++t)
                    c[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b[t].p[j], c[t], 0, 0, 0);
            }
        }
}

// The values that parts stand for.
template <int N>
__device__ __forceinline__ f32x8 joined(const Frag<N> &f)
{
    f32x8 v = __builtin_convertvector(f.p[N - 1], f32x8);
#pragma unroll
    for (int n = N - 2; n >= 0; --n)
        v += __builtin_convertvector(f.p[n], f32x8);
    return v;
}

// Three parts of what meets rows of NK parts in a product.
template <int NK>
__device__ __forceinline__ Frag<3> parts(f32x8 v)
{
    if constexpr (NK == 1)
        return split_cut(v);
    else
        return split<3>(v);
}
template <int NK>
__device__ __forceinline__ Frag<3> parts(f32x4 a, f32x4 b)
{
    return parts<NK>(__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

__device__ __forceinline__ float sum64(float v)
{
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1)
        v += __shfl_xor(v, m, 64);
    return v;
}

// The running sum over the wave's lanes: shifts inside rows of 16, then the rows'
// last values on, without a trip through LDS.
template <int CTRL, int ROWS>
__device__ __forceinline__ float shifted(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double shifted(double v)
{
    return __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, ROWS, 0xF, false),
                            __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, ROWS, 0xF, false));
}
template <typename T>
__device__ __forceinline__ T running_sum(T v)
{
    v += shifted<0x111, 0xF>(v);    // row_shr 1, 2, 4, 8
    v += shifted<0x112, 0xF>(v);
    v += shifted<0x114, 0xF>(v);
    v += shifted<0x118, 0xF>(v);
    v += shifted<0x142, 0xA>(v);    // row_bcast 15 to rows 1 and 3
    v += shifted<0x143, 0xC>(v);    // row_bcast 31 to rows 2 and 3
    return v;
}
__device__ __forceinline__ float first_lane(float v) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(v))); }
__device__ __forceinline__ float last_lane(float v) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63)); }

// Returns once all four flags are at least v (see LdsFlag).
__device__ __forceinline__ void await_all(int *flags, int v)
{
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) i32x4 lds_i32x4;
    for (;;) {
        const i32x4 f = *(volatile lds_i32x4 *)(lds_i32x4 *)flags;
        if (min(min(f[0], f[1]), min(f[2], f[3])) >= v)
            break;
        __builtin_amdgcn_s_sleep(1);
    }
    asm volatile("" ::: "memory");
}

// Walks with a chunk whose positive gates add up to more are done step by step.  Below
// it, e^60 = 2^87 leaves 2^41 to what it multiplies.
constexpr float kGrows = 60.f;
// e^g of more leaves no number of fp32 but zero finite.
constexpr float kMostGate = 1e4f;

// e^x as a float and a power of two, of any size.
struct Growth {
    float f;
    int n;
    __device__ __forceinline__ float of(float v) const { return ldexpf(v * f, n); }
};

// As decay_of, of any size, to 2^-23 of itself.
__device__ __forceinline__ Growth growth_of(float hi_i, float lo_i, float n_i, float hi_j, float lo_j, float n_j)
{
    const float e = hi_i - hi_j, n = finite(e) ? rintf(e) : 0.f;       // (below 2^20, by kMostGate)
    return n_i == n_j ? Growth{__builtin_amdgcn_exp2f((e - n) + (lo_i - lo_j)), (int)n} : Growth{0.f, 0};
}

__device__ __forceinline__ int scalar(unsigned v) { return __builtin_amdgcn_readfirstlane((int)v); }

// A chunk step by step, from its rows in LDS: the wave's columns of the state and of
// the result.  Lane (g, i16) has rows 16 m + 4 g + r of column i16 of the state, so a
// value of Y is a sum over the four g.  The roundings are written out: the walks with
// and without dg have to give the same bits.
template <int KD, bool BF16, int SL, bool BACK, int MODE>
__device__ __forceinline__ void walk_steps(const uint16_t *s_x1, const uint16_t *s_x2, const uint16_t *s_x3, int mine, int lane,
                                           Growth own, float scale, f32x4 (&S)[KD / 16], f32x4 (&Y)[4])
{
#pragma clang fp contract(off)
    using T1 = typename LinLds<KD, BF16, SL>::T1;
    using T3 = typename LinLds<KD, BF16, SL>::T3;
    const int g = lane >> 4, i16 = lane & 15;
#pragma unroll
    for (int tile = 0; tile < 4; ++tile) {
        const int at = BACK ? 3 - tile : tile;
        if constexpr (MODE == kOut)
            Y[at] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int n = 0; n < 16; ++n) {
            const int step = BACK ? 15 - n : n, t = 16 * at + step;
            const Growth now = {__int_as_float(__builtin_amdgcn_readlane(__float_as_int(own.f), t)),
                                __builtin_amdgcn_readlane(own.n, t)};
            const float value = (BACK ? scale : 1.f) * T3::one(s_x3, t, 16 * mine + i16);
            float y = 0.f;
#pragma unroll
            for (int m = 0; m < KD / 16; ++m) {
                const f32x4 key = T1::four(s_x2, t, 16 * m + 4 * g);
                f32x4 query = {0.f, 0.f, 0.f, 0.f};
                if constexpr (MODE == kOut)
                    query = T1::four(s_x1, t, 16 * m + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    S[m][r] = __builtin_fmaf(key[r], value, BACK ? S[m][r] : now.of(S[m][r]));
                    y = __builtin_fmaf(BACK ? query[r] : scale * query[r], S[m][r], y);
                    if constexpr (BACK)
                        S[m][r] = now.of(S[m][r]);
                }
            }
            if constexpr (MODE == kOut) {
                y += __shfl_xor(y, 16, 64);
                y += __shfl_xor(y, 32, 64);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float v = bperm(y, 4 * g + r);
                    Y[at][r] = i16 == step ? v : Y[at][r];
                }
            }
        }
    }
}

// One walk over the chunks of a segment.  kFast gives the pass that is to follow:
// kSteps, every chunk step by step, where one grows by more than kGrows; kCareful,
// with a look at every chunk for values of X3 that are not finite, which would reach
// the steps on the other side of the triangle through its zeros, where the state at
// the end is not finite; or none (kFast).
template <int KD, bool BF16, bool VEC, int SL, bool BACK, int MODE, int GATE, int PASS>
__device__ __forceinline__ int walk_pass(const LinArgs &a, const Walk &w, int seg, int slice, int64_t head, int thread)
{
    using LDS = LinLds<KD, BF16, SL>;
    using T1 = typename LDS::T1;
    using T3 = typename LDS::T3;
    using M = Tri<BACK, kHelp>;
    constexpr int NK = T1::NK, NS = KD / 32, kChain = LDS::kChain;
    extern __shared__ __attribute__((aligned(16))) char s_dyn[];
    uint16_t *lds = reinterpret_cast<uint16_t *>(s_dyn);
    float *ldf = reinterpret_cast<float *>(s_dyn);
    int *s_help = reinterpret_cast<int *>(ldf + LDS::kFlag), *s_spoiled = s_help + 4;

    const int p0 = seg * w.seg_chunks, p1 = min(a.NC, p0 + w.seg_chunks);
    const int64_t b = scalar((unsigned)head / (unsigned)a.Hv);
    const int h = (int)head - (int)b * a.Hv, hk = scalar((unsigned)h / (unsigned)(a.Hv / a.Hk));
    const int lane = thread & 63, wave = scalar(thread >> 6), g = lane >> 4, i16 = lane & 15;
    const int mine = wave < kChain ? wave : wave - kChain, group = slice * kChain + mine;
    auto chunk_of = [&](int p) { return BACK ? a.NC - 1 - p : p; };
    auto turn_of = [&](int p) { return (p - p0) & 1; };     // what goes to dg is kept for a turn
    auto half_of = [&](int p) { return LDS::kHalves == 2 ? (p - p0) & 1 : 0; };
    auto begin = [&](const Rows &x, bool kv) { return b * x.s.b + (kv ? hk : h) * x.s.h; };
    auto vecs = [&](int p) { return ldf + LDS::kVec + ((p - p0) & 3) * (kVecs * kC); };
    auto rows_of = [&](int p) { return min(kC, a.L - chunk_of(p) * kC); };
    constexpr int kSize = BF16 ? 2 : 4;
    constexpr bool CAREFUL = PASS == kCareful, STEPS = PASS == kSteps;
    constexpr int kGateWave = 1;        // (a help wave with two blocks of M where others have three)

    if (wave >= kChain && lane == 0)
        s_help[mine] = 0;
    lds_barrier();
    int again = kFast;
    auto follows = [&]() {      // (behind the pass's last barrier)
        if (PASS != kFast)
            return kFast;
        if (s_help[kGateWave] < 0)
            return kSteps;
        int spoiled = 0;
        if constexpr (MODE == kOut) {
            for (int n = 0; n < kChain; ++n)
                spoiled |= s_spoiled[n];
        }
        return spoiled ? kCareful : kFast;
    };

    if (wave < kChain) {
        const int col = group * 16 + i16;
        const int col4 = group * 16 + 4 * g;    // of the lane's four values of y
        f32x4 S[KD / 16];
        if (w.segs > 1 && MODE != kScan) {
            const float *from = native<KD>(w.starts, seg, a.heads, w.groups, head, group, lane);
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
                S[m] = *reinterpret_cast<const f32x4 *>(from + m * 256);
        } else {
            const float *from = seg == 0 ? w.start : nullptr;
            each_value<KD>(w, col, lane, [&](int m, int r, bool in, int at) {
                S[m][r] = from && in ? from[head * w.D1 * w.D3 + at] : 0.f;
            });
        }
        // The first segment's start is kept too: the last one's end may go to
        // the same buffer while other workgroups still begin.
        if (MODE == kScan && seg == 0) {
            float *to = native<KD>(w.starts, 0, a.heads, w.groups, head, group, lane);
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
                *reinterpret_cast<f32x4 *>(to + m * 256) = S[m];
        }
        Frag<3> sf[NS];
        Growth product = {1.f, 0};
        if constexpr (MODE == kOut && !STEPS) {
#pragma unroll
            for (int s = 0; s < NS; ++s)
                sf[s] = parts<NK>(S[2 * s], S[2 * s + 1]);
        }
        f32x4 beside[4];       // dg: the next chunk's values of x4 beside y's
        f32x4 kept[GATE == kGrad ? KD / 16 : 1];
        const int pitch = (w.D3 + 3) / 4 * 4;
        const bool wide = BF16 && w.wide;
        Stream out(w.y.p, wide ? head * a.L * pitch : begin(w.y, w.kvy), wide ? pitch : w.y.s.l, chunk_of(p0), BACK,
                   wide ? pitch : w.D3, wide ? 4 : kSize);
        Stream x4(w.x4.p, begin(w.x4, true), w.x4.s.l, chunk_of(p0), BACK, w.D3, kSize);
        auto fetch = [&](int p) {
            const int c = chunk_of(p);
            if constexpr (GATE != kNone) {
                const Chunk<BF16, VEC> cx = x4.chunk<BF16, VEC>(rows_of(p), w.D3);
                x4.next(p + 1 < p1);
                const uint32_t e = cx.lane_at(i16, col4);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    beside[t] = cx.four(e, i16, 16 * t, col4);
            }
            if constexpr (GATE == kGrad) {
                const float *from = native<KD>(a.kept, c, a.heads, w.groups, head, group, lane);
#pragma unroll
                for (int m = 0; m < KD / 16; ++m)
                    kept[m] = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(from + m * 256));
            }
        };
        if constexpr (GATE != kNone)
            fetch(p0);
        if constexpr (BF16)
            lds_barrier();
        for (int p = p0; p < p1; ++p) {
            if constexpr (!BF16)
                lds_barrier();
            const int half = half_of(p), c = chunk_of(p);
            const uint16_t *s_x1 = lds + LDS::kX1 + half * T1::kSize, *s_x2 = lds + LDS::kX2 + half * T1::kSize;
            const uint16_t *s_x3 = lds + LDS::kX3 + half * T3::kSize, *s_m = lds + LDS::kM + half * M::kSize;
            const float *s_vec = vecs(p);
            // e^g summed from a step behind `from` to `to` (-1: before the first)
            auto grown = [&](int from, int to) {
                auto at = [&](int which, int t) { return t < 0 ? 0.f : s_vec[which * kC + t]; };
                return growth_of(at(kGhi, to), at(kGlo, to), at(kResets, to), at(kGhi, from), at(kGlo, from), at(kResets, from));
            };
            Frag<NK> x3[2];
            if constexpr (!STEPS) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    x3[s] = T3::columns_stacked(s_x3, mine, s, lane);
            }
            float gone = 1.f;       // NaN: a column of X3 that is not finite spoils its column of the state
            int from = kC;          // and its outputs from this step on (in the walk's order)
            if constexpr (CAREFUL) {
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int t = 32 * s + 16 * (j >> 2) + 4 * g + (j & 3);
                        if (!finite((float)x3[s].p[0][j]))
                            from = min(from, BACK ? kC - 1 - t : t);
                    }
                from = min(from, __shfl_xor(from, 16, 64));
                from = min(from, __shfl_xor(from, 32, 64));
                gone = from < kC ? __builtin_nanf("") : 1.f;
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int t = 32 * s + 16 * (j >> 2) + 4 * g + (j & 3);
                        if ((BACK ? kC - 1 - t : t) >= from) {
#pragma unroll
                            for (int n = 0; n < NK; ++n)
                                x3[s].p[n][j] = (__bf16)0.f;
                        }
                    }
            }
            f32x4 Y[4];    // tiles of 16 columns (rows of the result) by 16 steps
            if constexpr (MODE == kOut && !(STEPS && GATE == kNone)) {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    Y[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    if constexpr (STEPS) {      // (the scale first: what fp32 holds may be no more than the result)
                        const float first = BACK ? 1.f : a.scale;
                        sf[s] = parts<NK>(first * S[2 * s], first * S[2 * s + 1]);
                    }
                    Frag<NK> x1[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        x1[t] = T1::rows_stacked(s_x1, t, s, lane);
                    mma_tiles<0, 3>(sf[s], x1, Y);
                }
                if constexpr (!STEPS) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        Y[t] *= s_vec[kRead * kC + 16 * t + i16];
                }
                if constexpr (GATE != kNone) {
                    float *to = GATE == kKeep ? a.reads + (((int64_t)c * a.heads + head) * w.groups + group) * kC
                                              : ldf + LDS::kWrites + (turn_of(p) * kChain + mine) * kC;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        float v = Y[t][0] * beside[t][0] + Y[t][1] * beside[t][1] + Y[t][2] * beside[t][2] + Y[t][3] * beside[t][3];
                        v += __shfl_xor(v, 16, 64);
                        v += __shfl_xor(v, 32, 64);
                        if constexpr (STEPS)
                            v = (BACK ? grown(16 * t + i16, kC - 1) : grown(-1, 16 * t + i16)).of(v);
                        to[16 * t + i16] = v;     // (the four lanes of a step all write it)
                    }
                }
                if constexpr (GATE == kKeep) {
                    float *to = native<KD>(a.kept, c, a.heads, w.groups, head, group, lane);
#pragma unroll
                    for (int m = 0; m < KD / 16; ++m)
                        __builtin_nontemporal_store(S[m], reinterpret_cast<f32x4 *>(to + m * 256));
                }
                if constexpr (GATE == kGrad) {
                    float v = 0.f;
#pragma unroll
                    for (int m = 0; m < KD / 16; ++m)
                        v += kept[m][0] * S[m][0] + kept[m][1] * S[m][1] + kept[m][2] * S[m][2] + kept[m][3] * S[m][3];
                    v = sum64(v);
                    ldf[LDS::kCross + turn_of(p) * kChain + wave] = STEPS ? grown(-1, kC - 1).of(v) : v * s_vec[kWhole * kC];
                }
                if constexpr (GATE != kNone)
                    fetch(min(p + 1, p1 - 1));
            }
            auto decays = [&](Growth now) {
                product.f *= now.f;
                product.n = max(min(product.n + now.n, 1 << 20), -(1 << 20));
                if (product.f > 0x1p32f) {
                    product.f *= 0x1p-64f;
                    product.n += 64;
                }
                if (STEPS && product.f < 0x1p-32f) {
                    product.f *= 0x1p64f;
                    product.n -= 64;
                }
            };
            if constexpr (STEPS) {
                if constexpr (MODE == kScan)
                    decays(grown(-1, kC - 1));
                walk_steps<KD, BF16, SL, BACK, MODE>(s_x1, s_x2, s_x3, mine, lane, grown(lane - 1, lane), a.scale, S, Y);
            } else {
                if constexpr (MODE == kOut) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        Frag<3> m[4];
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            if (M::has(t, s))
                                m[t] = M::template get<3>(s_m, t, s, lane);
                        // (the triangle has all tiles of one k step, half of the other's)
                        if (s == (BACK ? 1 : 0))
                            mma_tiles<0, 3>(x3[s], m, Y);
                        else if (BACK)
                            mma_tiles<0, 1>(x3[s], m, Y);
                        else
                            mma_tiles<2, 3>(x3[s], m, Y);
                    }
                    if constexpr (CAREFUL) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int f = bperm(from, 4 * g + r);
#pragma unroll
                            for (int t = 0; t < 4; ++t) {
                                const int step = 16 * t + i16;
                                if ((BACK ? kC - 1 - step : step) >= f)
                                    Y[t][r] = __builtin_nanf("");
                            }
                        }
                    }
                }
                // the state
                const float whole = s_vec[kWhole * kC] * gone;
                if constexpr (MODE == kScan)
                    decays({whole, 0});
                Frag<3> wx[2];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const f32x4 lo = row_vec(s_vec, kWrite, 2 * s, lane), hi = row_vec(s_vec, kWrite, 2 * s + 1, lane);
                    wx[s] = parts<NK>(joined(x3[s]) * __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                }
#pragma unroll
                for (int m = 0; m < KD / 16; ++m)
                    S[m] *= whole;
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    Frag<NK> x2[2][2];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            x2[m][i] = T1::columns_stacked(s_x2, 2 * s + m, i, lane);
#pragma unroll
                    for (int o = 2; o >= 0; --o)
#pragma unroll
                        for (int n = 0; n < NK; ++n)
                            if (o - n >= 0) {
#pragma unroll
                                for (int i = 0; i < 2; ++i)
#pragma unroll
                                    for (int m = 0; m < 2; ++m)
                                        S[2 * s + m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x2[m][i].p[n], wx[i].p[o - n],
                                                                                              S[2 * s + m], 0, 0, 0);
                            }
                    if constexpr (MODE == kOut)
                        sf[s] = parts<NK>(S[2 * s], S[2 * s + 1]);
                }
            }
            if constexpr (MODE == kOut) {
                auto store = [&](auto cy) {
                    const uint32_t e = cy.lane_at(i16, col4);
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        cy.put4(e, i16, 16 * t, col4, Y[t]);
                };
                if (wide)
                    store(out.chunk<false, VEC>(rows_of(p), pitch));
                else
                    store(out.chunk<BF16, VEC>(rows_of(p), w.D3));
                out.next(true);
            }
            lds_barrier();
        }
        if constexpr (MODE == kScan) {
            float *to = native<KD>(w.starts, seg + 1, a.heads, w.groups, head, group, lane);
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
                *reinterpret_cast<f32x4 *>(to + m * 256) = S[m];
            if (thread == 0 && slice == 0)
                w.wholes[seg * a.heads + head] = make_float2(product.f, (float)product.n);
            lds_barrier();
            again = follows();
        } else {
            float mark = 0.f;
#pragma unroll
            for (int m = 0; m < KD / 16; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    mark = __builtin_fmaf(S[m][r], 0.f, mark);
            const bool spoiled = PASS == kFast && __any(mark != 0.f);
            if (lane == 0)
                s_spoiled[mine] = spoiled;
            lds_barrier();
            again = follows();
            // (the end may be the start, from which a second pass begins)
            if (w.end && p1 == a.NC && again == kFast) {
                each_value<KD>(w, col, lane, [&](int m, int r, bool in, int at) {
                    if (in)
                        w.end[head * w.D1 * w.D3 + at] = S[m][r];
                });
            }
        }
    } else {
        // With dg the help waves have more to do than the chain: going first they
        // cut the backward of 4 x 16 heads of 128, 4096 steps, from 554 to 512 us
        // (without it, forward, neither order gains).
        if constexpr (GATE != kNone)
            __builtin_amdgcn_s_setprio(2);
        const int tid = thread - kChain * 64;
        float most = 0.f;       // (the gates' wave) the most that the positive gates of a chunk add up to
        struct Incoming {
            T1 t1, t2;
            T3 t3;
            Unit<BF16> k[GATE == kGrad ? 4 : 1];    // the wave's rows of k
        };
        float gate, reads;
        const int c0 = chunk_of(p0);
        Stream x1(w.x1.p, begin(w.x1, w.kv1), w.x1.s.l, c0, BACK, w.D1, kSize);
        Stream x2(w.x2.p, begin(w.x2, w.kv2), w.x2.s.l, c0, BACK, w.D1, kSize);
        const int cols = w.D3 - slice * SL;
        Stream x3(w.x3.p, begin(w.x3, w.kv3) + slice * SL, w.x3.s.l, c0, BACK, cols, kSize);
        Stream x4(w.x4.p, begin(w.x4, true) + slice * SL, w.x4.s.l, c0, BACK, cols, kSize);
        Stream gates(a.g.p, b * a.g.s.b + h * a.g.s.h, a.g.s.l, c0, BACK, 1, 4);
        const bool has_gates = a.g.p != nullptr, has_steps = has_gates && a.g.s.l != 0;
        // (no branches on the way of the loads: where two paths with other loads
        // in flight meet, a wait for one becomes a wait for all)
        auto fetch = [&](Incoming &in, int p) {
            const int rows = rows_of(p);
            const bool move = p + 1 < p1;
            if constexpr (MODE == kOut) {
                in.t1.load(x1.chunk<BF16, VEC>(rows, w.D1), tid);
                x1.next(move);
            }
            in.t2.load(x2.chunk<BF16, VEC>(rows, w.D1), tid);
            x2.next(move);
            in.t3.load(x3.chunk<BF16, VEC>(rows, cols), tid);
            x3.next(move);
            if constexpr (GATE == kGrad) {
                const Chunk<BF16, VEC> ck = x4.chunk<BF16, VEC>(rows, cols);
                x4.next(move);
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    in.k[s] = ck.unit(16 * (s >= 2 && mine == 0 ? 0 : 3 - mine) + i16, 32 * (s & 1) + 8 * g);
            }
        };
        auto fetch_gate = [&](int p) {
            const Chunk<false, false> cg = gates.chunk<false, false>(has_gates ? rows_of(p) : 0, 1);
            gates.next(p + 1 < p1);
            gate = __uint_as_float(cg.raw(cg.lane_at(lane, 0), lane, 0, 0));
            if constexpr (GATE == kGrad) {
                const float *r = a.reads + (((int64_t)chunk_of(p) * a.heads + head) * w.groups + slice * kChain) * kC + lane;
                reads = r[0];
#pragma unroll
                for (int n = 1; n < kChain; ++n)
                    reads += r[n * kC];
            }
        };
        // The gates' vectors of chunk p (one wave), from the values fetched, those
        // of chunk p + 1 on their way.
        auto sum_gates = [&](int p) {
            // (the same for every whole chunk where the gates do not change from
            // step to step)
            if (mine != kGateWave || !(GATE == kGrad || has_steps || p - p0 < 4 || rows_of(p) != rows_of(p - 4)))
                return;
            // G log2(e) in 64 bits (differences of neighbours stay exact to 32),
            // steps that empty the state counted apart.
            float *s_vec = vecs(p);
            float now = has_steps ? gate : lane < rows_of(p) ? first_lane(gate) : 0.f;
            if constexpr (STEPS)
                now = finite(now) ? fminf(now, kMostGate) : now;
            const bool empty = now < kEmpties;
            const double G = running_sum(empty ? 0.0 : (double)now * 1.4426950408889634);
            const float n = running_sum(empty ? 1.f : 0.f);
            if constexpr (PASS == kFast)
                most = fmaxf(most, running_sum(now <= __FLT_MAX__ ? fmaxf(now, 0.f) : 0.f));
            const float hi = (float)G, lo = (float)(G - (double)hi);
            const float hi1 = last_lane(hi), lo1 = last_lane(lo), n1 = last_lane(n);
            const float rise = a.scale * decay_of(hi, lo, n, 0.f, 0.f, 0.f), left = decay_of(hi1, lo1, n1, hi, lo, n);
            s_vec[kRead * kC + lane] = BACK ? left : rise;
            s_vec[kWrite * kC + lane] = BACK ? rise : left;
            s_vec[kWhole * kC + lane] = decay_of(hi1, lo1, n1, 0.f, 0.f, 0.f);
            s_vec[kGhi * kC + lane] = hi;
            s_vec[kGlo * kC + lane] = lo;
            s_vec[kResets * kC + lane] = n;
            if constexpr (GATE == kGrad)
                s_vec[kReads * kC + lane] = reads;
            fetch_gate(min(p + 1, p1 - 1));
        };
        // Rows and M of chunk p into its half of LDS, the rows of chunk p + 1 on
        // their way, and the gates of chunk p + 1.
        auto prepare = [&](Incoming &in, int p) {
            const int half = half_of(p);
            uint16_t *s_x1 = lds + LDS::kX1 + half * T1::kSize, *s_x2 = lds + LDS::kX2 + half * T1::kSize;
            uint16_t *s_x3 = lds + LDS::kX3 + half * T3::kSize;
            const float *s_vec = vecs(p);
            if constexpr (MODE == kOut)
                in.t1.store(s_x1, tid);
            in.t2.store(s_x2, tid);
            in.t3.store(s_x3, tid);
            Frag<NK> kr[4];
            if constexpr (GATE == kGrad) {
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    kr[s] = unit_frag<BF16>(in.k[s]);
            }
            fetch(in, min(p + 1, p1 - 1));
            if constexpr (MODE == kOut) {
                // the other help waves' rows (and the gates, summed a turn before)
                if (lane == 0)
                    LdsFlag::set(&s_help[mine], p - p0 + 1);
                await_all(s_help, p - p0 + 1);
                uint16_t *s_m = lds + LDS::kM + half * M::kSize;
                // Three blocks for each wave in one run of code, whose waits
                // overlap: of the lower triangle (0,0) and (3,3); (1,0) and (1,1);
                // (2,0) to (2,2); (3,0) to (3,2), two of them twice; mirrored going
                // back.
                int ta[3], tb[3];
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    ta[n] = n && mine == 0 ? 3 : mine;
                    tb[n] = n && mine == 0 ? 3 : min(n, mine);
                    if constexpr (BACK) {
                        ta[n] = 3 - ta[n];
                        tb[n] = 3 - tb[n];
                    }
                }
                f32x4 v[3], kq[3];
#pragma unroll
                for (int n = 0; n < 3; ++n)
                    v[n] = kq[n] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const Frag<NK> x1[2] = {T1::rows(s_x1, ta[0], s, lane), T1::rows(s_x1, ta[1], s, lane)};
#pragma unroll
                    for (int n = 0; n < 3; ++n)
                        v[n] = mma<3>(T1::rows(s_x2, tb[n], s, lane), x1[n > 0], v[n]);
                }
                if constexpr (GATE == kGrad) {
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int n = 0; n < 3; ++n)
                            kq[n] = mma<3>(T3::rows(s_x3, tb[n], s, lane), kr[2 * (n > 0) + s], kq[n]);
                }
#pragma unroll
                for (int n = 0; n < 3; ++n) {
                    const int row = 16 * ta[n] + i16;
                    const float hi = s_vec[kGhi * kC + row], lo = s_vec[kGlo * kC + row], resets = s_vec[kResets * kC + row];
                    const f32x4 hj = row_vec(s_vec, kGhi, tb[n], lane), lj = row_vec(s_vec, kGlo, tb[n], lane),
                                nj = row_vec(s_vec, kResets, tb[n], lane);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int col = 16 * tb[n] + 4 * g + r;
                        const bool inside = BACK ? col >= row : col <= row;
                        if constexpr (STEPS) {
                            // (the growth last: a product that is zero stays zero)
                            const Growth d = BACK ? growth_of(hj[r], lj[r], nj[r], hi, lo, resets) : growth_of(hi, lo, resets, hj[r], lj[r], nj[r]);
                            kq[n][r] = GATE == kGrad && col > row ? Growth{kq[n][r], d.n}.of(a.scale * v[n][r] * d.f) : 0.f;
                        } else {
                            const float d = BACK ? decay_of(hj[r], lj[r], nj[r], hi, lo, resets) : decay_of(hi, lo, resets, hj[r], lj[r], nj[r]);
                            v[n][r] = inside ? a.scale * v[n][r] * d : 0.f;
                            kq[n][r] = GATE == kGrad && col > row ? v[n][r] * kq[n][r] : 0.f;
                        }
                    }
                    if constexpr (!STEPS)
                        M::put(s_m, ta[n], tb[n], lane, v[n]);
                }
                if constexpr (GATE == kGrad) {
#pragma unroll
                    for (int n = 0; n < 3; ++n)
                        Cuts::put(ldf + LDS::kCuts + turn_of(p) * Cuts::kSize, tb[n], ta[n], kq[n], lane);
                }
            }
        };
        // dg of a chunk that the chain has left behind (one wave).
        auto gates_of = [&](int p) {
            if constexpr (GATE == kGrad) {
                if (mine == kGateWave) {
                    const int turn = turn_of(p), t = chunk_of(p) * kC + lane;
                    const float *s_vec = vecs(p), *s_w = ldf + LDS::kWrites + turn * kChain * kC, *s_x = ldf + LDS::kCross + turn * kChain;
                    float whole = s_x[0], writes = s_w[lane];
#pragma unroll
                    for (int n = 1; n < kChain; ++n) {
                        whole += s_x[n];
                        writes += s_w[n * kC + lane];
                    }
                    const float v = crossing(whole, s_vec[kReads * kC + lane], writes, ldf + LDS::kCuts + turn * Cuts::kSize, lane);
                    // the decay of an empty state does nothing
                    const float *n = s_vec + kResets * kC;
                    const bool empty = n[lane] != (lane ? n[lane - 1] : 0.f) || (t == 0 && !a.started);
                    if (t < a.L) {
                        if (a.dg_part)
                            a.dg_part[(slice * a.heads + head) * a.L + t] = empty ? 0.f : v;
                        else
                            static_cast<float *>(const_cast<void *>(a.dg.p))[b * a.dg.s.b + h * a.dg.s.h + t * a.dg.s.l] =
                                empty ? 0.f : v;
                    }
                }
            }
        };
        if constexpr (MODE == kOut && !STEPS) {
            for (int n = 0; n < LDS::kHalves; ++n)
                M::clear(lds + LDS::kM + n * M::kSize, tid);
        }
        auto behind = [&](int p) {      // the chain has left chunk p - 1
            if (p > p0)
                gates_of(p - 1);
        };
        Incoming in;
        fetch_gate(p0);
        fetch(in, p0);
        sum_gates(p0);
        if constexpr (BF16) {
            prepare(in, p0);
            sum_gates(p0 + 1);
            lds_barrier();
            for (int p = p0; p + 1 < p1; ++p) {
                behind(p);
                prepare(in, p + 1);
                sum_gates(p + 2);
                lds_barrier();
            }
            behind(p1 - 1);
            lds_barrier();
        } else {
            for (int p = p0; p < p1; ++p) {
                prepare(in, p);
                lds_barrier();
                // while the chain is at chunk p
                sum_gates(p + 1);
                behind(p);
                lds_barrier();
            }
        }
        gates_of(p1 - 1);
        // (behind the last chunk's barrier: nobody waits for the flag any more)
        if constexpr (PASS == kFast) {
            const bool grows = last_lane(most) > kGrows;    // (with all lanes here)
            if (grows && lane == 0)
                s_help[kGateWave] = -1;
        }
        lds_barrier();
        again = follows();
    }
    return again;
}

template <int KD, bool BF16, bool VEC, int SL, bool BACK, int MODE, int GATE>
__device__ __forceinline__ void walk(const LinArgs &a, const Walk &w, int seg, int slice, int64_t head)
{
    const int again = walk_pass<KD, BF16, VEC, SL, BACK, MODE, GATE, kFast>(a, w, seg, slice, head, threadIdx.x);
    if (again == kFast)
        return;
    lds_barrier();      // the flags have been read
    // (opaque: nothing formed for one pass is held through the other)
    if (MODE == kOut && again == kCareful)
        walk_pass<KD, BF16, VEC, SL, BACK, MODE, GATE, kCareful>(a, w, seg, opaque_s(slice), head, opaque(threadIdx.x));
    else
        walk_pass<KD, BF16, VEC, SL, BACK, MODE, GATE, kSteps>(a, w, seg, opaque_s(slice), head, opaque(threadIdx.x));
}

// Workgroups by walk, segment, slice, head, the head first: those that read the
// same rows are a multiple of the heads apart, with 8 heads and their multiples
// on one die of the eight, with one L2.
enum Which { kForward, kBoth, kFirst, kLast };      // the forward's; dQ's, dV's and dK's; with dg: dQ's and dV's; dK's

template <int KD, bool BF16, bool VEC, int SL, int MODE, int WHICH>
__global__ void __launch_bounds__(walk_threads(SL), 1) walk_kernel(LinArgs)
{
    // (the arguments where they lie: of a parameter with this many uses the compiler
    // makes a copy in scratch)
    const LinArgs &a = *reinterpret_cast<const LinArgs *>((const void *)__builtin_amdgcn_kernarg_segment_ptr());
    unsigned rest = blockIdx.y * gridDim.x + blockIdx.x;
    if (rest >= a.blocks)
        return;
    const unsigned heads = (unsigned)a.heads;
    // (nothing asks for the last segment's end)
    auto slices = [&](int n) { return (unsigned)(a.w[n].D3 + SL - 1) / SL; };
    auto blocks = [&](int n) { return heads * (a.w[n].segs - (MODE == kScan)) * slices(n); };
    int n = a.first;
    if constexpr (WHICH != kForward) {
        while (n < a.last && rest >= blocks(n)) {
            rest -= blocks(n);
            ++n;
        }
    }
    const Walk &w = a.w[n];
    const unsigned of_head = rest / heads, count = slices(n);
    const int64_t head = scalar(rest - of_head * heads);
    const int seg = scalar(of_head / count), slice = scalar(of_head - seg * count);
    if constexpr (WHICH == kForward) {
        walk<KD, BF16, VEC, SL, false, MODE, kNone>(a, w, seg, slice, head);
    } else if constexpr (WHICH == kLast) {
        walk<KD, BF16, VEC, SL, true, MODE, kGrad>(a, w, seg, slice, head);
    } else {
        if (n == 0)
            walk<KD, BF16, VEC, SL, false, MODE, WHICH == kFirst ? kKeep : kNone>(a, a.w[0], seg, slice, head);
        else if constexpr (WHICH == kFirst)
            walk<KD, BF16, VEC, SL, true, MODE, kNone>(a, a.w[1], seg, slice, head);
        else
            walk<KD, BF16, VEC, SL, true, MODE, kNone>(a, w, seg, slice, head);
    }
}

// ---------------------------------------------------------------------------
// join_kernel: the states before the segments, from the segments' decays and
// ends: the first segment's end is whole, S_{n+1} = decay_n S_n + end_n.  A
// thread has four values of one state; the segments follow each other (14 us for
// 8 states of 128 x 128 and 32 segments, 4.5 for the three walks of 64 heads in two;
// each segment's values fetched a turn ahead 16).
// ---------------------------------------------------------------------------
template <int KD>
__global__ void __launch_bounds__(256) lin_join_kernel(LinArgs a)
{
    const Walk &w = a.w[blockIdx.y];
    const int64_t one = (int64_t)w.groups * KD * 16, size = a.heads * one;      // values of a state, and between segments
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= size || w.segs == 1)
        return;
    const int64_t head = at / one;
    float *p = w.starts + size + at;
    f32x4 S = *reinterpret_cast<const f32x4 *>(p);
    for (int n = 1; n + 1 < w.segs; ++n) {
        p += size;
        const float2 whole = w.wholes[n * a.heads + head];
        const f32x4 end = *reinterpret_cast<const f32x4 *>(p);
        const Growth by = {whole.x, (int)whole.y};
#pragma unroll
        for (int r = 0; r < 4; ++r)
            S[r] = by.n ? by.of(S[r]) + end[r] : __builtin_fmaf(by.f, S[r], end[r]);
        *reinterpret_cast<f32x4 *>(p) = S;
    }
}

// ---------------------------------------------------------------------------
// group_kernel: dq and dk as the sums over the value heads of their group, from
// fp32 [B*Hv][L][pitch].  A thread has four values of a row, and nothing else to do
// than move them: 58 us for 2 x 16 heads of 4 sequences of 4096 rows of 128 into 8,
// 336 MB at 5.7 TB/s.
// ---------------------------------------------------------------------------
struct GroupArgs {
    const float *part[2];
    Rows out[2];
    int64_t items;          // B*Hk*L*pitch / 4
    int Hk, group, L, D, pitch;
};

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) group_kernel(GroupArgs a)
{
    const int units = a.pitch / 4;
    const float *part = a.part[blockIdx.y];
    const Rows &out = a.out[blockIdx.y];
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < a.items; n += (int64_t)gridDim.x * 256) {
        const int col = (int)(n % units) * 4;
        const int64_t row = n / units, t = row % a.L, bk = row / a.L, hk = bk % a.Hk, b = bk / a.Hk;
        const float *p = part + (bk * a.group * a.L + t) * a.pitch + col;
        f32x4 v = *reinterpret_cast<const f32x4 *>(p);
        for (int j = 1; j < a.group; ++j)
            v += *reinterpret_cast<const f32x4 *>(p + (int64_t)j * a.L * a.pitch);
        const int64_t e = b * out.s.b + hk * out.s.h + t * out.s.l + col;
        if constexpr (VEC && BF16) {
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(const_cast<void *>(out.p)) + e) =
                make_uint2(f32x2_to_bf16x2_rne(v[0], v[1]), f32x2_to_bf16x2_rne(v[2], v[3]));
        } else if constexpr (VEC) {
            *reinterpret_cast<f32x4 *>(static_cast<float *>(const_cast<void *>(out.p)) + e) = v;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (col + r < a.D) {
                    if constexpr (BF16)
                        static_cast<uint16_t *>(const_cast<void *>(out.p))[e + r] = f32_to_bf16_rne(v[r]);
                    else
                        static_cast<float *>(const_cast<void *>(out.p))[e + r] = v[r];
                }
        }
    }
}

// ---------------------------------------------------------------------------
// dg from the slices' parts: of every step (5 us for 64 heads of 4096, a launch's
// latency), or the sum over sequences and steps, in 64 bits, by a workgroup for each
// head, 256 values after 256: 4 us for 999 values a head, but 66 for 65536 and 710
// for 524288, where few heads of many steps leave the device idle.
// ---------------------------------------------------------------------------
struct GateArgs {
    const float *part;      // [slices][B*Hv][L]
    Rows dg;
    int64_t heads;
    int Hv, L, slices;
};

__global__ void __launch_bounds__(256) gate_steps_kernel(GateArgs a)
{
    const int64_t all = a.heads * a.L;
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < all; n += (int64_t)gridDim.x * 256) {
        float v = a.part[n];
        for (int s = 1; s < a.slices; ++s)
            v += a.part[s * all + n];
        const int64_t head = n / a.L, b = head / a.Hv;
        static_cast<float *>(const_cast<void *>(a.dg.p))[b * a.dg.s.b + (head - b * a.Hv) * a.dg.s.h + n % a.L * a.dg.s.l] = v;
    }
}

__global__ void __launch_bounds__(256) gate_heads_kernel(GateArgs a)
{
    __shared__ double s_sum[4];
    const int64_t h = (int64_t)blockIdx.y * gridDim.x + blockIdx.x, B = a.heads / a.Hv;
    if (h >= a.Hv)
        return;
    double v = 0.0;
    for (int64_t n = 0; n < B * a.slices; ++n) {
        const int64_t s = n / B, b = n - s * B;
        const float *p = a.part + (s * a.heads + b * a.Hv + h) * a.L;
        for (int t = threadIdx.x; t < a.L; t += 256)
            v += p[t];
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1)
        v += __shfl_xor(v, m, 64);
    if ((threadIdx.x & 63) == 0)
        s_sum[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        static_cast<float *>(const_cast<void *>(a.dg.p))[h * a.dg.s.h] = (float)(s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3]);
}

// ---------------------------------------------------------------------------
// lin_step_kernel: one step.  A workgroup takes 32 columns of one head's state,
// each thread four columns of every 32nd row, all rows in registers: the state
// is read once and written once, and o falls out on the way.  Its bytes bound it:
// 128 x 32 states of 128 x 64 take 56 us, 270 MB at 4.8 TB/s (a copy's rate); 16
// states of 128 x 128 4.4 us, a launch's latency.
// ---------------------------------------------------------------------------
struct LinStepArgs {
    Rows q, k, v, g, o;
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

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) lin_step_kernel(LinStepArgs a)
{
    constexpr int TX = 8, TY = 256 / TX, RP = kMaxDim / TY;
    __shared__ float s_part[4][TX * 4];
    const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (block >= a.blocks)
        return;
    const int64_t head = block / a.slices;
    const int slice = (int)(block % a.slices);
    const int64_t b = head / a.Hv;
    const int h = (int)(head - b * a.Hv), hk = h / (a.Hv / a.Hk);
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX, wave = threadIdx.x >> 6;
    const int col = (slice * TX + tx) * 4;
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
    // e^g may be more than fp32 holds, and the state zero: then as a power of two
    // (rounded down, so that it leaves no finite result behind it) and the rest.
    float decay = 1.f;
    int shift = 0;
    if (a.g.p) {
        const float gate = static_cast<const float *>(a.g.p)[b * a.g.s.b + h * a.g.s.h];
        if (gate > 64.f && finite(gate)) {
            const double e = (double)fminf(gate, kMostGate) * 1.4426950408889634;
            shift = (int)e;
            decay = __builtin_amdgcn_exp2f((float)(e - shift));
        } else {
            decay = expf(gate);
        }
    }
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (col + r < a.Dv)
            v[r] = load_value<BF16>(a.v.p, b * a.v.s.b + h * a.v.s.h + col + r);

    f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < RP; ++i) {
        const int row = i * TY + ty;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            st[i][r] = ldexpf(st[i][r], shift) * decay + k[i] * v[r];
        if (row < a.Dk) {
            o += q[i] * st[i];
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
#pragma unroll
    for (int m = TX; m < 64; m <<= 1)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            o[r] += __shfl_xor(o[r], m, 64);
    if ((threadIdx.x & 63) < TX)
        *reinterpret_cast<f32x4 *>(&s_part[wave][tx * 4]) = o;
    __syncthreads();
    if (ty == 0) {
        o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < 4; ++m)
            o += *reinterpret_cast<const f32x4 *>(&s_part[m][tx * 4]);
        o *= a.scale;
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
constexpr int64_t kMaxGridX = (int64_t)1 << 22;

int check_linear_dims(int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk, int32_t Dv)
{
    if (B < 0 || Hk < 0 || Hv < 0 || L < 0 || L > kMaxL || Dk < 1 || Dk > kMaxDim || Dv < 1 || Dv > kMaxDim)
        return PDSSM_ERR_DIM;
    if (Hv > 0 && (Hk == 0 || Hv % Hk != 0))
        return PDSSM_ERR_DIM;
    if ((double)B * Hv > 5.0e8 || Hv > (1 << 30) || (double)B * Hv * (double)((L + kC - 1) / kC) > 2.0e9)
        return PDSSM_ERR_DIM;
    return PDSSM_OK;
}

int slices_of(int D, int SL) { return (D + SL - 1) / SL; }
int padded(int D) { return D <= 64 ? 64 : 128; }
// Columns of a workgroup, from the walks of a launch at 64 columns each.  128 take
// the rows through LDS and form M once in place of twice: 318 against 414 us for
// 8 x 32 heads of 128 and 4096 steps, 83 against 90 for 8 heads and 18000.  Of 64 a
// chunk is done sooner, which counts while the device is not filled: 22 against 39 us
// for 8 heads and 512 steps, 37 against 44 and 4096.  (Three parts of fp32 rows leave
// no room for 128.)
int slice_for(int D3, int64_t walks, int64_t L, uint32_t flags)
{
    const int64_t NC = (L + kC - 1) / kC;
    return !(flags & PDSSM_DATA_BF16) || D3 <= 64 || walks * std::max<int64_t>(1, NC / 4) <= 256 ? 64 : 128;
}

// How many segments the chunks of a head are cut into, walked side by side: they
// are walked twice (once without outputs, at half the cost) and joined, so walks are
// cut only where a launch's workgroups do not fill the device, no finer than fills
// it (129 to 255 workgroups stay whole, and up to half of the device idle), and where the chunks saved are worth the two launches more: about three chunks
// of a bf16 forward, whose walks begin with a chunk's wait, fewer of the others.
// Heads of 128 (fp32: 64 and 100), one sequence, us cut and whole:
//     bf16 forward, 8 heads    256 steps 19, 18      512: 22, 28     4096: 37, 173    18000: 83, 1098
//     fp32 forward, 8 heads    128: 18, 15           256: 19, 24     2048: 30, 154
//     bf16 backward, 8 heads   128: 33, 32           256: 38, 47     512: 47, 78      4096: 97, 598
//     fp32 backward, 6 heads   128: 79, 96           333: 87, 217    2048: 187, 1120
// and one chunk a segment in place of two: 28 against 25 us forward, bf16, 1024 steps;
// 19 against 24, fp32, 333; backward 87 against 119, fp32, 333.
struct Cut {
    int segs, chunks;
};

Cut cut_of(int64_t walks, int64_t L, uint32_t flags, bool bwd)
{
    const bool bf16 = flags & PDSSM_DATA_BF16;
    const int64_t NC = (L + kC - 1) / kC, launches = bwd ? bf16 : bf16 ? 3 : 1;
    const int64_t segs = walks > 0 ? std::min(256 / walks, bf16 && !bwd ? NC / 2 : NC) : 0;
    Cut c = {1, (int)std::max<int64_t>(1, NC)};
    if (segs > 1) {
        const int64_t chunks = (NC + segs - 1) / segs;
        if (3 * chunks + 2 * launches <= 2 * NC)
            c = {(int)((NC + chunks - 1) / chunks), (int)chunks};
    }
    return c;
}

// Places in the workspace.
struct Space {
    int64_t total = 0;
    int64_t take(int64_t bytes)
    {
        const int64_t at = total;
        total += (bytes + 255) / 256 * 256;
        return at;
    }
};

struct LinLayout {
    Space space;
    int SL;                 // columns of a workgroup (dK's with dg: 64)
    Cut cut[3];
    int groups[3];
    int64_t starts[3], wholes[3], kept, reads, dg_part, dq_part, dk_part, ds;
};

// Of the forward, or of dQ's, dV's and dK's walks.
LinLayout layout_of(int64_t B, int64_t Hk, int64_t Hv, int64_t L, int Dk, int Dv, uint32_t flags, bool bwd)
{
    LinLayout l = {};
    const int64_t heads = B * Hv, NC = (L + kC - 1) / kC;
    const int pitch = (Dk + 3) / 4 * 4;
    const bool grad = bwd && !(flags & PDSSM_NO_DG);
    l.space.take(256);
    if (bwd) {
        // With dg dK's walk comes after the others, its columns 64 at a time.  Cut for
        // that without dg too, so that the other gradients' bits do not depend on it
        // (432 us with dg and 304 without for 4 x 16 heads of 128, 4096 steps; cut for
        // three walks at once 656 and 263).
        auto walks = [&](int SL) { return heads * (slices_of(Dk, SL) + slices_of(Dv, SL)); };
        l.SL = slice_for(std::max(Dk, Dv), walks(64), L, flags);
        l.cut[0] = l.cut[1] = cut_of(walks(l.SL), L, flags, true);
        l.cut[2] = cut_of(heads * slices_of(Dk, 64), L, flags, true);
    } else {
        l.SL = slice_for(Dv, heads * slices_of(Dv, 64), L, flags);
        l.cut[0] = cut_of(heads * slices_of(Dv, l.SL), L, flags, false);
    }
    const int64_t rows = std::max(padded(Dk), padded(Dv));
    for (int n = 0; n < (bwd ? 3 : 1); ++n) {
        l.groups[n] = (bwd ? (int)rows : padded(Dv)) / 16;
        if (l.cut[n].segs > 1) {
            l.starts[n] = l.space.take((l.cut[n].segs + 1) * heads * l.groups[n] * rows * 64);
            l.wholes[n] = l.space.take(l.cut[n].segs * heads * 8);
        }
    }
    if (bwd) {
        l.ds = l.space.take(heads * Dk * Dv * 4);
        if (grad) {
            l.kept = l.space.take(NC * heads * l.groups[0] * rows * 64);
            l.reads = l.space.take(NC * heads * l.groups[0] * kC * 4);
            if (Dk > 64 || (flags & PDSSM_DG_HEADS))
                l.dg_part = l.space.take(heads * slices_of(Dk, 64) * L * 4);
        }
        if (Hv > Hk) {
            l.dq_part = l.space.take(heads * L * pitch * 4);
            l.dk_part = l.space.take(heads * L * pitch * 4);
        }
    }
    return l;
}

template <typename K, typename A>
int lin_launch(K kernel, dim3 grid, int threads, size_t lds, const A &a, hipStream_t stream)
{
    // More than 64 KB of LDS has to be asked for; the device has 160 KB.
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess)
            return hip_status(e);
    }
    hipLaunchKernelGGL(kernel, grid, dim3((unsigned)threads), lds, stream, a);
    return hip_status(hipGetLastError());
}

dim3 grid_of(int64_t blocks)
{
    return dim3((unsigned)std::min(blocks, kMaxGridX), (unsigned)((blocks + kMaxGridX - 1) / kMaxGridX));
}

// A call's walks; of cut sequences all scans first, and the join.
template <int KD, bool BF16, bool VEC, int SL, bool BWD>
int launch_walks(LinArgs a, bool grad, hipStream_t stream)
{
    auto launch = [&](auto kernel, int sl, size_t lds, int first, int last, bool scan) {
        a.first = first, a.last = last, a.blocks = 0;
        for (int n = first; n <= last; ++n)
            a.blocks += a.heads * (a.w[n].segs - scan) * slices_of(a.w[n].D3, sl);
        return lin_launch(kernel, grid_of(a.blocks), walk_threads(sl), lds, a, stream);
    };
    constexpr size_t lds = LinLds<KD, BF16, SL>::kBytes;
    static_assert(lds <= 163840, "LDS of a compute unit");
    constexpr int kLastWalk = BWD ? 2 : 0;
    int rc = PDSSM_OK;
    int64_t states = 0;
    for (int n = 0; n <= kLastWalk; ++n)
        if (a.w[n].segs > 1)
            states = std::max(states, a.heads * a.w[n].groups);
    if (states > 0) {
        rc = launch(walk_kernel<KD, BF16, VEC, SL, kScan, BWD ? kBoth : kForward>, SL, lds, 0, kLastWalk, true);
        if (rc == PDSSM_OK)
            rc = lin_launch(lin_join_kernel<KD>, dim3((unsigned)(states * KD / 64), kLastWalk + 1), 256, 0, a, stream);
    }
    if (rc != PDSSM_OK)
        return rc;
    if constexpr (!BWD) {
        return launch(walk_kernel<KD, BF16, VEC, SL, kOut, kForward>, SL, lds, 0, 0, false);
    } else {
        constexpr size_t lds64 = LinLds<KD, BF16, 64>::kBytes;
        if (!grad) {
            // Cut walks fill the device more than once: dK's then go behind the others
            // with columns of 64 (304 against 320 us for 4 x 16 heads of 128, 4096 steps).
            if (SL == 64 || a.w[2].segs == 1)
                return launch(walk_kernel<KD, BF16, VEC, SL, kOut, kBoth>, SL, lds, 0, 2, false);
            rc = launch(walk_kernel<KD, BF16, VEC, SL, kOut, kBoth>, SL, lds, 0, 1, false);
            return rc == PDSSM_OK ? launch(walk_kernel<KD, BF16, VEC, 64, kOut, kBoth>, 64, lds64, 2, 2, false) : rc;
        }
        // dK's walk adds up dg from what dQ's keeps
        rc = launch(walk_kernel<KD, BF16, VEC, SL, kOut, kFirst>, SL, lds, 0, 1, false);
        return rc == PDSSM_OK ? launch(walk_kernel<KD, BF16, VEC, 64, kOut, kLast>, 64, lds64, 2, 2, false) : rc;
    }
}

// The variant for these sizes, type and rows: D1 the largest contraction of the
// walks.
template <int KD, bool BF16, bool VEC>
int launch_width(const LinArgs &a, int SL, bool bwd, bool grad, hipStream_t stream)
{
    if constexpr (BF16) {
        if (SL == 128 && !bwd)
            return launch_walks<KD, BF16, VEC, 128, false>(a, false, stream);
        if constexpr (KD == 128)        // (backward, columns and contraction change places)
            if (SL == 128)
                return launch_walks<KD, BF16, VEC, 128, true>(a, grad, stream);
    }
    return bwd ? launch_walks<KD, BF16, VEC, 64, true>(a, grad, stream) : launch_walks<KD, BF16, VEC, 64, false>(a, grad, stream);
}

template <bool BF16, bool VEC>
int launch_sizes(const LinArgs &a, int D1, int SL, bool bwd, bool grad, hipStream_t stream)
{
    return D1 > 64 ? launch_width<128, BF16, VEC>(a, SL, bwd, grad, stream) : launch_width<64, BF16, VEC>(a, SL, bwd, grad, stream);
}

int launch_any(const LinArgs &a, bool bf16, bool vec, int D1, int SL, bool bwd, bool grad, hipStream_t stream)
{
    if (bf16)
        return vec ? launch_sizes<true, true>(a, D1, SL, bwd, grad, stream) : launch_sizes<true, false>(a, D1, SL, bwd, grad, stream);
    return vec ? launch_sizes<false, true>(a, D1, SL, bwd, grad, stream) : launch_sizes<false, false>(a, D1, SL, bwd, grad, stream);
}

}  // namespace
}  // namespace pdssm

using namespace pdssm;

namespace {

constexpr uint32_t kBwdFlags = PDSSM_DATA_BF16 | PDSSM_NO_DG | PDSSM_DG_HEADS;

bool bwd_flags_ok(uint32_t flags)
{
    return !(flags & ~kBwdFlags) && (flags & (PDSSM_NO_DG | PDSSM_DG_HEADS)) != (PDSSM_NO_DG | PDSSM_DG_HEADS);
}

}  // namespace

extern "C" size_t pdssm_linear_workspace_bytes(int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk, int32_t Dv,
                                               uint32_t flags)
{
    if (check_linear_dims(B, Hk, Hv, L, Dk, Dv) != PDSSM_OK || (flags & ~PDSSM_DATA_BF16))
        return 0;
    return (size_t)layout_of(B, Hk, Hv, L, Dk, Dv, flags, false).space.total;
}

extern "C" size_t pdssm_linear_bwd_workspace_bytes(int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk,
                                                   int32_t Dv, uint32_t flags)
{
    if (check_linear_dims(B, Hk, Hv, L, Dk, Dv) != PDSSM_OK || !bwd_flags_ok(flags))
        return 0;
    return (size_t)layout_of(B, Hk, Hv, L, Dk, Dv, flags, true).space.total;
}

extern "C" int pdssm_linear_fwd(const void *q, const void *k, const void *v, const float *g, const float *s0, void *o,
                                float *s_final, int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk, int32_t Dv,
                                float scale, uint32_t flags, const pdssm_strides *strides, void *workspace,
                                size_t workspace_bytes, hipStream_t stream)
{
    const int rc = check_linear_dims(B, Hk, Hv, L, Dk, Dv);
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
    if (!q || !k || !v || !o || !workspace)
        return PDSSM_ERR_NULL;
    const int esize = (flags & PDSSM_DATA_BF16) ? 2 : 4;
    for (const void *p : {q, k, v, (const void *)o})
        if (!element_aligned(p, esize))
            return PDSSM_ERR_ALIGN;
    if (!element_aligned(g, 4) || !aligned16(workspace))
        return PDSSM_ERR_ALIGN;
    const LinLayout lo = layout_of(B, Hk, Hv, L, Dk, Dv, flags, false);
    if (workspace_bytes < (size_t)lo.space.total)
        return PDSSM_ERR_WORKSPACE;
    const pdssm_strides keys = {Hk * L * Dk, L * Dk, Dk}, values = {Hv * L * Dv, L * Dv, Dv}, gates = {Hv * L, L, 1};
    const pdssm_strides contiguous[5] = {keys, keys, values, gates, values};
    const pdssm_strides *s = strides ? strides : contiguous;
    if (!strides_ok(s, 3) || (g && !strides_ok(s + 3, 1)) || !strides_ok(s + 4, 1))
        return PDSSM_ERR_DIM;
    char *ws = static_cast<char *>(workspace);
    LinArgs a = {};
    Walk &w = a.w[0];
    w.x1 = {q, s[0]}, w.x2 = {k, s[1]}, w.x3 = {v, s[2]}, w.y = {o, s[4]};
    w.kv1 = w.kv2 = true;
    w.D1 = Dk, w.D3 = Dv, w.groups = lo.groups[0], w.start = s0, w.end = s_final, w.row = Dv, w.col = 1;
    w.starts = reinterpret_cast<float *>(ws + lo.starts[0]), w.wholes = reinterpret_cast<float2 *>(ws + lo.wholes[0]);
    w.segs = lo.cut[0].segs, w.seg_chunks = lo.cut[0].chunks;
    a.g = {g, s[3]};
    a.heads = B * Hv;
    a.Hk = (int)Hk, a.Hv = (int)Hv, a.L = (int)L, a.NC = (int)((L + kC - 1) / kC), a.scale = scale;
    const bool vec = units(q, s[0], Dk, esize) && units(k, s[1], Dk, esize) && units(v, s[2], Dv, esize) &&
                     units(o, s[4], Dv, esize);
    return launch_any(a, esize == 2, vec, Dk, lo.SL, false, false, stream);
}

extern "C" int pdssm_linear_bwd(const void *q, const void *k, const void *v, const float *g, const float *s0,
                                const void *d_o, const float *ds_final, void *dq, void *dk, void *dv, float *dg,
                                float *ds0, int64_t B, int64_t Hk, int64_t Hv, int64_t L, int32_t Dk, int32_t Dv,
                                float scale, uint32_t flags, const pdssm_strides *strides, void *workspace,
                                size_t workspace_bytes, hipStream_t stream)
{
    int rc = check_linear_dims(B, Hk, Hv, L, Dk, Dv);
    if (rc != PDSSM_OK)
        return rc;
    if (!bwd_flags_ok(flags))
        return PDSSM_ERR_FLAGS;
    const bool grad = !(flags & PDSSM_NO_DG), dg_heads = flags & PDSSM_DG_HEADS;
    if (Hv == 0 || (B == 0 && !dg_heads))
        return PDSSM_OK;
    const pdssm_strides keys = {Hk * L * Dk, L * Dk, Dk}, values = {Hv * L * Dv, L * Dv, Dv}, gates = {Hv * L, L, 1};
    const pdssm_strides contiguous[9] = {keys, keys, values, gates, values, keys, keys, values, dg_heads ? pdssm_strides{0, 1, 0} : gates};
    const pdssm_strides *s = strides ? strides : contiguous;
    GateArgs ga = {};
    ga.dg = {dg, s[8]}, ga.heads = B * Hv, ga.Hv = (int)Hv, ga.L = (int)L, ga.slices = slices_of(Dk, 64);
    if (B == 0 || L == 0) {
        for (const float *p : {ds_final, (const float *)ds0})
            if (p && !aligned16(p))
                return PDSSM_ERR_ALIGN;
        if (dg_heads) {
            if (!dg)
                return PDSSM_ERR_NULL;
            if (!element_aligned(dg, 4))
                return PDSSM_ERR_ALIGN;
            rc = lin_launch(gate_heads_kernel, grid_of(Hv), 256, 0, ga, stream);
        }
        if (rc == PDSSM_OK && B > 0 && ds0 && ds0 != ds_final)
            rc = launch_state_fill(ds_final, ds0, B * Hv * Dk * Dv, stream);
        return rc;
    }
    for (const float *p : {s0, ds_final, (const float *)ds0})
        if (p && !aligned16(p))
            return PDSSM_ERR_ALIGN;
    if (!q || !k || !v || !d_o || !dq || !dk || !dv || (grad && !dg) || !workspace)
        return PDSSM_ERR_NULL;
    const int esize = (flags & PDSSM_DATA_BF16) ? 2 : 4;
    for (const void *p : {q, k, v, d_o, (const void *)dq, (const void *)dk, (const void *)dv})
        if (!element_aligned(p, esize))
            return PDSSM_ERR_ALIGN;
    if (!element_aligned(g, 4) || (grad && !element_aligned(dg, 4)) || !aligned16(workspace))
        return PDSSM_ERR_ALIGN;
    const LinLayout lo = layout_of(B, Hk, Hv, L, Dk, Dv, flags, true);
    if (workspace_bytes < (size_t)lo.space.total)
        return PDSSM_ERR_WORKSPACE;
    for (int n = 0; n < 9; ++n)
        if (!(n == 3 && !g) && !(n == 8 && (!grad || dg_heads)) && !strides_ok(s + n, 1))
            return PDSSM_ERR_DIM;
    char *ws = static_cast<char *>(workspace);
    auto place = [&](int64_t at) { return reinterpret_cast<float *>(ws + at); };
    // dV's walk writes ds0 while dK's may still begin from ds_final
    if (ds0 && ds0 == ds_final) {
        rc = launch_state_fill(ds_final, place(lo.ds), B * Hv * Dk * Dv, stream);
        if (rc != PDSSM_OK)
            return rc;
        ds_final = place(lo.ds);
    }
    const bool shared = Hv > Hk;
    const int pitch = (Dk + 3) / 4 * 4;
    LinArgs a = {};
    Walk &wq = a.w[0], &wv = a.w[1], &wk = a.w[2];
    wq.x1 = {d_o, s[4]}, wq.x2 = {v, s[2]}, wq.x3 = {k, s[1]}, wq.x4 = {q, s[0]}, wq.y = {dq, s[5]};
    wv.x1 = {k, s[1]}, wv.x2 = {q, s[0]}, wv.x3 = {d_o, s[4]}, wv.y = {dv, s[7]};
    wk.x1 = {v, s[2]}, wk.x2 = {d_o, s[4]}, wk.x3 = {q, s[0]}, wk.x4 = {k, s[1]}, wk.y = {dk, s[6]};
    wq.kv3 = wk.kv3 = wv.kv1 = wv.kv2 = true;
    wq.D1 = wk.D1 = wv.D3 = Dv, wq.D3 = wk.D3 = wv.D1 = Dk;
    wq.row = wk.row = wv.col = 1, wq.col = wk.col = wv.row = Dv;
    wq.start = s0, wv.start = wk.start = ds_final, wv.end = ds0;
    for (Walk *w : {&wq, &wk})
        w->kvy = true;
    if (shared) {
        const pdssm_strides part = {Hv * L * pitch, L * pitch, pitch};
        for (Walk *w : {&wq, &wk})
            w->wide = true, w->kvy = false;
        wq.y = {place(lo.dq_part), part}, wk.y = {place(lo.dk_part), part};
    }
    for (int n = 0; n < 3; ++n) {
        Walk &w = a.w[n];
        w.groups = lo.groups[n], w.starts = place(lo.starts[n]), w.wholes = reinterpret_cast<float2 *>(place(lo.wholes[n]));
        w.segs = lo.cut[n].segs, w.seg_chunks = lo.cut[n].chunks;
    }
    a.g = {g, s[3]}, a.dg = ga.dg, a.started = s0 != nullptr;
    a.kept = place(lo.kept), a.reads = place(lo.reads);
    a.dg_part = grad && (ga.slices > 1 || dg_heads) ? place(lo.dg_part) : nullptr;
    a.heads = B * Hv;
    a.Hk = (int)Hk, a.Hv = (int)Hv, a.L = (int)L, a.NC = (int)((L + kC - 1) / kC), a.scale = scale;
    const bool vec_keys = units(dq, s[5], Dk, esize) && units(dk, s[6], Dk, esize);
    const bool vec = units(q, s[0], Dk, esize) && units(k, s[1], Dk, esize) && units(v, s[2], Dv, esize) &&
                     units(d_o, s[4], Dv, esize) && vec_keys && units(dv, s[7], Dv, esize);
    rc = launch_any(a, esize == 2, vec, std::max(Dk, Dv), lo.SL, true, grad, stream);
    if (rc == PDSSM_OK && a.dg_part) {
        ga.part = a.dg_part;
        if (dg_heads)
            rc = lin_launch(gate_heads_kernel, grid_of(Hv), 256, 0, ga, stream);
        else
            rc = lin_launch(gate_steps_kernel, dim3((unsigned)std::min<int64_t>((a.heads * L + 255) / 256, 4096)), 256, 0, ga, stream);
    }
    if (rc == PDSSM_OK && shared) {
        GroupArgs gr = {{place(lo.dq_part), place(lo.dk_part)}, {{dq, s[5]}, {dk, s[6]}}, B * Hk * L * (pitch / 4),
                        (int)Hk, (int)(Hv / Hk), (int)L, Dk, pitch};
        const dim3 grid((unsigned)std::min<int64_t>((gr.items + 255) / 256, 8192), 2);
        if (esize == 2)
            rc = vec_keys ? lin_launch(group_kernel<true, true>, grid, 256, 0, gr, stream)
                          : lin_launch(group_kernel<true, false>, grid, 256, 0, gr, stream);
        else
            rc = vec_keys ? lin_launch(group_kernel<false, true>, grid, 256, 0, gr, stream)
                          : lin_launch(group_kernel<false, false>, grid, 256, 0, gr, stream);
    }
    return rc;
}

extern "C" int pdssm_linear_step(const void *q, const void *k, const void *v, const float *g, const float *s, void *o,
                                 float *s_out, int64_t B, int64_t Hk, int64_t Hv, int32_t Dk, int32_t Dv, float scale,
                                 uint32_t flags, const pdssm_strides *strides, hipStream_t stream)
{
    const int rc = check_linear_dims(B, Hk, Hv, 1, Dk, Dv);
    if (rc != PDSSM_OK)
        return rc;
    if (flags & ~PDSSM_DATA_BF16)
        return PDSSM_ERR_FLAGS;
    if (B == 0 || Hv == 0)
        return PDSSM_OK;
    if (!q || !k || !v || !s || !o || !s_out)
        return PDSSM_ERR_NULL;
    const int esize = (flags & PDSSM_DATA_BF16) ? 2 : 4;
    for (const void *p : {q, k, v, (const void *)o})
        if (!element_aligned(p, esize))
            return PDSSM_ERR_ALIGN;
    if (!element_aligned(g, 4) || !aligned16(s) || !aligned16(s_out))
        return PDSSM_ERR_ALIGN;
    LinStepArgs a = {};
    const pdssm_strides keys = {Hk * Dk, Dk, 0}, values = {Hv * Dv, Dv, 0}, gates = {Hv, 1, 0};
    const pdssm_strides contiguous[5] = {keys, keys, values, gates, values};
    const pdssm_strides *st = strides ? strides : contiguous;
    a.q = {q, st[0]}, a.k = {k, st[1]}, a.v = {v, st[2]}, a.g = {g, st[3]}, a.o = {o, st[4]};
    a.s = s, a.s_out = s_out, a.Hk = (int)Hk, a.Hv = (int)Hv, a.Dk = Dk, a.Dv = Dv, a.scale = scale;
    a.slices = (Dv + 31) / 32;
    a.blocks = B * Hv * a.slices;
    const dim3 grid = grid_of(a.blocks);
    if (esize == 2)
        return Dv % 4 == 0 ? lin_launch(lin_step_kernel<true, true>, grid, 256, 0, a, stream)
                           : lin_launch(lin_step_kernel<true, false>, grid, 256, 0, a, stream);
    return Dv % 4 == 0 ? lin_launch(lin_step_kernel<false, true>, grid, 256, 0, a, stream)
                       : lin_launch(lin_step_kernel<false, false>, grid, 256, 0, a, stream);
}
