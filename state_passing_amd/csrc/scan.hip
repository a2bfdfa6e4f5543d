// scan.hip -- the selective state-space scan (linrec_scan_fwd / _bwd / _step):
//   d = dt + dt_bias or its softplus,  h_t = exp(d_t A) h_{t-1} + d_t x_t b_t,
//   y_t = (c_t . h_t + D x_t) silu(z_t),
// N states a channel, b and c shared by the channels of a group.
//
// Bound by the vector units' instructions: a state and token take a product and an
// exponential for the gate, two operations for the state and one for the output,
// and no two channels share a gate, so nothing of it is a matrix product.  Per token
// and wave of 16 channels x 16 states the forward issues 30 vector instructions, the
// backward 91 (78 of them in the walk: 16 to form the states again, 36 to go back,
// 26 to add over states and channels); 8 x 2048 x 4096 bf16 runs at 79% and 93% of
// the cycles that issue them, 344 and 904 us, with 1.07 and 1.5 GB to move (3.1 and
// 1.7 TB/s, where a copy reaches 4.9).  Where a piece is split, the segments' pass
// issues 22 (from behind 24), in 83 to 92% of the cycles at 16 states.
//
// A lane owns 4 states of a channel, N / 4 lanes a channel, so a workgroup of
// four waves walks 4 * 64 / (N / 4) channels token by token with their states in
// registers.  Token rows are read 16 bytes at a time by a mapping of their own,
// a tile of tokens ahead: each value that belongs to a token and channel (the
// step d, the input d x, the gates) is formed once there and passed through LDS.
// With all 16 states of a channel in one lane, sums over states would cost nothing
// and sums over channels (db, dc) twice as much, and a quarter of the waves would
// be there to hide latencies.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ctx.hpp"
#include "device.hpp"
#include "rows.hpp"

namespace linrec {
namespace {

constexpr int NT = 256;      // threads a workgroup
constexpr int NS = 4;        // states a lane
constexpr int SEG = 32;      // tokens: segments are multiples of this, and of every tile
constexpr int BLOCK = 8;     // tokens between two saved states
constexpr float LOG2E = 1.44269504088896341f, LN2 = 0.693147180559945309f;

template <int N>
struct Geo {
    static constexpr int L = N / NS;        // lanes a channel
    static constexpr int CPW = 64 / L;      // channels a wave
    static constexpr int CW = NT / 64 * CPW;   // channels a workgroup
    static constexpr int TILE = N == 16 || N == 32 ? 32 : 16;   // tokens a tile: two workgroups' tiles fit a CU's LDS
};

template <typename T>
struct In {
    Act<const T> x, dt, b, c, z;
    const float *A, *D, *dt_bias;
    int softplus;
};

// The sequence and the channels of a workgroup.
struct Where {
    int b, g, c0, cend, n;   // sequence, group, first channel, end of the group's channels, tokens there
};

template <int N>
__device__ __forceinline__ Where where(const int* n_new, int T_, int C, int G, int blocks)
{
    const int cg = C / G;
    Where w;
    w.b = blockIdx.z;
    w.g = blockIdx.x / blocks;
    w.c0 = w.g * cg + (int)(blockIdx.x % blocks) * Geo<N>::CW;
    w.cend = (w.g + 1) * cg;
    w.n = tokens_of(n_new, w.b, T_);
    return w;
}

// log(1 + e^v) = max(v, 0) + log(w), w = 1 + e, e = exp(-|v|).  What w loses of e
// is added back, which keeps the relative precision of small steps (log(w) is c / w
// short, and w = 1 up to rounding where c counts).  v = -inf gives 0: a token whose
// step is hidden so leaves the state as it is.  slope: the derivative.
__device__ __forceinline__ float softplus(float v)
{
    const float e = __builtin_amdgcn_exp2f(-LOG2E * fabsf(v)), w = 1.f + e, c = e - (w - 1.f);
    return fmaxf(v, 0.f) + __builtin_fmaf(__builtin_amdgcn_logf(w), LN2, c);
}

__device__ __forceinline__ float softplus(float v, float& slope)
{
    const float e = __builtin_amdgcn_exp2f(-LOG2E * fabsf(v)), w = 1.f + e, c = e - (w - 1.f);
    const float r = __builtin_amdgcn_rcpf(w);
    slope = v >= 0.f ? r : e * r;
    return fmaxf(v, 0.f) + __builtin_fmaf(__builtin_amdgcn_logf(w), LN2, c);
}

// The steps of a vector of channels (and their slopes).
template <typename T, int VN>
__device__ __forceinline__ void steps(float (&d)[VN], float (&slope)[VN], const u32x4& v, const float (&bias)[VN], int sp)
{
#pragma unroll
    for (int j = 0; j < VN; ++j) {
        d[j] = vec_get<T>(v, j) + bias[j];
        slope[j] = 1.f;
    }
    if (sp)   // one branch for the vector: its channels' chains run side by side
#pragma unroll
        for (int j = 0; j < VN; ++j)
            d[j] = softplus(d[j], slope[j]);
}

template <typename T, int VN>
__device__ __forceinline__ void steps(float (&d)[VN], const u32x4& v, const float (&bias)[VN], int sp)
{
#pragma unroll
    for (int j = 0; j < VN; ++j)
        d[j] = vec_get<T>(v, j) + bias[j];
    if (sp)
#pragma unroll
        for (int j = 0; j < VN; ++j)
            d[j] = softplus(d[j]);
}

// The steps of a token that is not there are zeros; `last`: the tile may have such
// tokens (a branch for the workgroup, not a select for every value).
template <int VN>
__device__ __forceinline__ void absent(float (&d)[VN], bool last, bool gone)
{
    if (last) {
        asm volatile("");
#pragma unroll
        for (int j = 0; j < VN; ++j)
            d[j] = gone ? 0.f : d[j];
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// Sum over the L lanes of a channel, in all of them.
template <int L>
__device__ __forceinline__ float channel_sum(float v)
{
    v = dpp_add<0xb1>(v);                       // lane ^ 1
    if constexpr (L >= 4)
        v = dpp_add<0x4e>(v);                   // lane ^ 2
    if constexpr (L >= 8)
        v = dpp_add<0x141>(v);                  // the other half of 8 lanes
    if constexpr (L >= 16)
        v = dpp_add<0x140>(v);                  // the other half of 16 lanes
    return v;
}

// Sums of 4 values of every lane over the channels of a wave (the lanes of one
// state quad): a step that adds lanes 32 or 16 apart adds two values at once, one
// in each half of the lanes, so 4 values over 16 channels take 8 instructions
// where adding them one by one takes 16.  Every lane of row r of 16 lanes has the
// sum of value of(); the two sets of sums of TOKENS tokens (db's and dc's) differ
// by lane, so that a write stores 64 of them (L == 16: two writes).
template <int L>
struct WaveSums {
    static constexpr int TOKENS = L == 2 ? 4 : L == 4 ? 2 : 1, COUNT = L == 16 ? 2 : 1;
    static __device__ __forceinline__ int of() { return 2 * ((threadIdx.x >> 4) & 1) + ((threadIdx.x >> 5) & 1); }
    static __device__ __forceinline__ int set() { return L == 16 ? 0 : (threadIdx.x >> 3) & 1; }
    static __device__ __forceinline__ int token() { return L == 2 ? (threadIdx.x >> 1) & 3 : L == 4 ? (threadIdx.x >> 2) & 1 : 0; }
    static __device__ __forceinline__ void pick(float (&r)[COUNT], const float (&b)[TOKENS], const float (&c)[TOKENS])
    {
        if constexpr (L == 16) {
            r[0] = b[0];
            r[1] = c[0];
        } else {
            float v[TOKENS];
#pragma unroll
            for (int i = 0; i < TOKENS; ++i)
                v[i] = threadIdx.x & 8 ? c[i] : b[i];
            if constexpr (L == 2) {
                const bool one = threadIdx.x & 2;
                const float p = one ? v[1] : v[0], q = one ? v[3] : v[2];
                r[0] = threadIdx.x & 4 ? q : p;
            } else if constexpr (L == 4) {
                r[0] = threadIdx.x & 4 ? v[1] : v[0];
            } else {
                r[0] = v[0];
            }
        }
    }
    static __device__ __forceinline__ float halves(float a, float b)   // a in lanes 0-31, b in 32-63
    {
        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    static __device__ __forceinline__ float rows(float a, float b)     // a in even rows of 16, b in odd
    {
        const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    static __device__ __forceinline__ float row(float a)   // over the channels of a row
    {
        if constexpr (L <= 8)
            a = dpp_add<0x128>(a);                         // lanes 8 apart
        if constexpr (L <= 4)
            a = dpp_add<0x124>(a);                         // 4 apart
        if constexpr (L <= 2)
            a = dpp_add<0x122>(a);                         // 2 apart
        return a;
    }
    static __device__ __forceinline__ float sum(const floatx4& v)   // values 0-3 in the rows of 16 lanes
    {
        return row(rows(halves(v[0], v[1]), halves(v[2], v[3])));
    }
};

// Sums over the lanes of a channel of 4 values, the lane with quad q the sum of
// value q & 3 (L == 2: of values q and q + 2).
template <int L>
struct ChannelSums {
    static constexpr int COUNT = L == 2 ? 2 : 1;
    template <int CTRL>
    static __device__ __forceinline__ float pick(float a, float b, bool second)   // a's sum, or the second lane's b's
    {
        const float keep = second ? b : a, give = second ? a : b;
        return keep + __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(give), CTRL, 0xf, 0xf, true));
    }
    static __device__ __forceinline__ float both(float a)
    {
        return dpp_add<0xb1>(a);
    }
    // MANY == 3: value 2 is value 3 too; 2: only values 0 and 1 are asked for
    template <int MANY = 4>
    static __device__ __forceinline__ void sum(float (&r)[COUNT], const float (&v)[4])
    {
        const bool one = threadIdx.x & 1, two = threadIdx.x & 2;
        const float a = pick<0xb1>(v[0], v[1], one);
        const float b = MANY == 2 ? 0.f : MANY == 3 ? both(v[3]) : pick<0xb1>(v[2], v[3], one);
        if constexpr (L == 2) {
            r[0] = a;
            r[1] = b;
        } else {
            float s = MANY == 2 ? dpp_add<0x4e>(a) : pick<0x4e>(a, b, two);
            // the 4 (12) lanes beside hold other parts of the same values
            if constexpr (L == 8) {
                unsigned o = __builtin_amdgcn_update_dpp(0u, __float_as_uint(s), 0x124, 0xf, 0xa, false);   // 4 lanes before
                o = __builtin_amdgcn_update_dpp(o, __float_as_uint(s), 0x12c, 0xf, 0x5, false);             // 4 lanes behind
                s += __uint_as_float(o);
            }
            if constexpr (L == 16)
                s = dpp_add<0x124>(dpp_add<0x128>(s));
            r[0] = s;
        }
    }
};

// A walk's waves drop in priority with each quarter that they have done: of two on
// a SIMD the older issues first, and would be done long before the younger, which
// then has the SIMD to itself and cannot fill it.
__device__ __forceinline__ void pace(int done, int all)
{
    if (4 * (int64_t)done < all)
        __builtin_amdgcn_s_setprio(3);
    else if (2 * (int64_t)done < all)
        __builtin_amdgcn_s_setprio(2);
    else if (4 * (int64_t)(all - done) > all)
        __builtin_amdgcn_s_setprio(1);
    else
        __builtin_amdgcn_s_setprio(0);
}

// Waits for loads here, a walk after they were issued: the wait in front of their
// use would be one for the stores issued in between, too.
template <int K>
__device__ __forceinline__ void arrived(u32x4 (&v)[K])
{
#pragma unroll
    for (int i = 0; i < K; ++i)
        asm volatile("" : "+v"(v[i]));
}

// ---- the mapping that reads token rows ---------------------------------------
//
// A tile is TILE rows of CW channels; a thread takes PV of its 16-byte vectors,
// all of the same channels.
template <typename T, int N>
struct Rows {
    static constexpr int TILE = Geo<N>::TILE;
    static constexpr int VN = Vec<T>::N, VPR = Geo<N>::CW / VN, COUNT = TILE * VPR, PV = (COUNT + NT - 1) / NT;
    static_assert(NT % VPR == 0 && (COUNT % NT == 0 || COUNT < NT), "whole rounds of one thread's channels");
    int c, nc, row;   // first channel, channels that exist, first row
    bool whole;       // every thread has a vector of channels that exist
    __device__ __forceinline__ Rows(const Where& w)
    {
        whole = COUNT >= NT && w.c0 + Geo<N>::CW <= w.cend;
        const int v = threadIdx.x % VPR;
        c = w.c0 + v * VN;
        nc = (int)threadIdx.x < COUNT ? w.cend - c : 0;
        row = threadIdx.x / VPR;
    }
    __device__ __forceinline__ int token(int i) const { return row + i * (NT / VPR); }
    // The places of a row's channels in LDS, 16 bytes each: a thread's channels lie VN places behind those of the
    // thread beside it, so threads that write their channel j together would meet in 16 / VN groups of banks; xor-ed
    // by the thread's number among those that meet, they spread.  first(): channel 0's place, channel j's: first() ^ j.
    static __device__ __forceinline__ int place(int c) { return c ^ (c / 16 & (VN - 1)); }
    static __device__ __forceinline__ int pair(int p) { return p ^ (p / 16 & (VN / 2 - 1)); }   // likewise 2 channels in 16 bytes
    __device__ __forceinline__ int first() const { return place(col()); }
    __device__ __forceinline__ int col() const { return (threadIdx.x % VPR) * VN; }
};

// This thread's rows of one tensor, tile after tile.
template <typename T, typename R>
struct Stream {
    T* p;
    int64_t st;
    __device__ __forceinline__ Stream(const Act<T>& a, const Where& w, const R& rows, int t0)
        : p(a.ptr + w.b * a.sb + (int64_t)(t0 + rows.row) * a.st + rows.c), st(a.st)
    {
    }
    __device__ __forceinline__ void move(int tokens) { p += tokens * st; }
    __device__ __forceinline__ T* at(int i) const { return p + i * (NT / R::VPR) * st; }
    // the tile's first `left` rows; the others come as zeros
    __device__ __forceinline__ void load(u32x4 (&v)[R::PV], const R& rows, int left) const
    {
        if (rows.whole && left >= R::TILE) {
#pragma unroll
            for (int i = 0; i < R::PV; ++i)
                v[i] = *reinterpret_cast<const u32x4*>(at(i));
            return;
        }
#pragma unroll
        for (int i = 0; i < R::PV; ++i)
            v[i] = rows.token(i) < left && rows.nc > 0 ? load_vec(at(i), rows.nc) : u32x4{0u, 0u, 0u, 0u};
    }
};

// One or two projections of a tile (rows of N): a thread takes PB of the 16-byte
// vectors of all.
template <typename T, int N, int MANY>
struct Projections {
    static constexpr int TILE = Geo<N>::TILE;
    static constexpr int VN = Vec<T>::N, VPR = N / VN, ONE = TILE * VPR, COUNT = MANY * ONE, PB = (COUNT + NT - 1) / NT;
    u32x4 v[PB];
    const T* p[PB];
    int64_t step[PB];   // elements from a tile to the next
    __device__ __forceinline__ Projections(const Act<const T>& first, const Act<const T>& second, const Where& w, int t0, int dir)
    {
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int k = threadIdx.x + i * NT, r = k % ONE;
            const Act<const T>& a = k < ONE ? first : second;
            p[i] = a.head(w.b, w.g) + (int64_t)(t0 + r / VPR) * a.st + r % VPR * VN;
            step[i] = dir * TILE * a.st;
        }
    }
    // the tile's first `left` rows (the others come as zeros), and on to the next tile
    __device__ __forceinline__ void load(int left)
    {
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int k = threadIdx.x + i * NT;
            v[i] = u32x4{0u, 0u, 0u, 0u};
            if ((COUNT % NT == 0 || k < COUNT) && (left >= TILE || k % ONE / VPR < left))
                v[i] = *reinterpret_cast<const u32x4*>(p[i]);
            p[i] += step[i];
        }
    }
    __device__ __forceinline__ void store(float (*bc)[TILE][N]) const
    {
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int k = threadIdx.x + i * NT, r = k % ONE;
            if (k < COUNT) {
                float* p = &bc[k / ONE][r / VPR][r % VPR * VN];
#pragma unroll
                for (int j = 0; j < VN; j += 4)
                    *reinterpret_cast<floatx4*>(p + j) =
                        floatx4{vec_get<T>(v[i], j), vec_get<T>(v[i], j + 1), vec_get<T>(v[i], j + 2), vec_get<T>(v[i], j + 3)};
            }
        }
    }
};

// Where a lane's states lie.
template <int N>
struct Lane {
    int q, col, c;   // state quad, channel of the workgroup's, channel
    bool ok;
    __device__ __forceinline__ Lane(const Where& w)
    {
        const int lane = threadIdx.x & 63;
        q = lane % Geo<N>::L;
        col = (threadIdx.x >> 6) * Geo<N>::CPW + lane / Geo<N>::L;
        c = w.c0 + col;
        ok = c < w.cend;
    }
    __device__ __forceinline__ floatx4 load(const float* p) const   // p: [C][N]
    {
        if (!p || !ok)
            return zero4();
        p += (int64_t)c * N + q * NS;
        return floatx4{p[0], p[1], p[2], p[3]};
    }
    __device__ __forceinline__ void store(float* p, const floatx4& v) const
    {
        if (ok) {
            p += (int64_t)c * N + q * NS;
#pragma unroll
            for (int j = 0; j < NS; ++j)
                p[j] = v[j];
        }
    }
};

__device__ __forceinline__ floatx4 exp2_4(const floatx4& v)
{
    return floatx4{__builtin_amdgcn_exp2f(v[0]), __builtin_amdgcn_exp2f(v[1]), __builtin_amdgcn_exp2f(v[2]),
                   __builtin_amdgcn_exp2f(v[3])};
}

__device__ __forceinline__ float dot4(const floatx4& a, const floatx4& b)
{
    float s = a[0] * b[0];
#pragma unroll
    for (int j = 1; j < 4; ++j)
        s = __builtin_fmaf(a[j], b[j], s);
    return s;
}

// Segments of a piece: seg tokens each; state: [B][nseg][C][N], total: [B][nseg][C].
struct Segments {
    int nseg, seg;
    float *state, *total;
};

// ---- segments ----------------------------------------------------------------
//
// What a segment makes of zeros (the first in order: of the carry): the state that
// leaves it (REVERSE: the gradient that it passes on), and its sum of steps, whose
// exponential with A is what it makes of the state (gradient) that enters it.  What
// the last in order makes is not asked for: its place takes a copy of the carry,
// which the first reads (the caller's memory may be the last one's output).
template <typename T, int N, bool REVERSE>
__global__ __launch_bounds__(NT) void scan_sum_kernel(In<T> in, const float* carry, const int* n_new, Act<const T> dy,
                                                      Segments sg, int T_, int C, int G, int blocks)
{
    typedef Rows<T, N> R;
    constexpr int CW = Geo<N>::CW, TILE = Geo<N>::TILE, VN = R::VN, PV = R::PV;
    __shared__ __attribute__((aligned(16))) float2 step[TILE][CW + 2];   // d, and d x or e
    __shared__ __attribute__((aligned(16))) float bc[1][TILE][N];
    const Where w = where<N>(n_new, T_, C, G, blocks);
    const R rows(w);
    const Lane<N> lane(w);
    const int at = 2 * R::pair(lane.col / 2) + lane.col % 2;   // where this channel's step lies
    const int seg = REVERSE ? sg.nseg - 1 - blockIdx.y : blockIdx.y;
    const int begin = seg * sg.seg, end = begin + min(max(w.n - begin, 0), sg.seg);
    const int first = REVERSE ? begin + (end - 1 - begin) / TILE * TILE : begin, move = REVERSE ? -TILE : TILE;
    const floatx4 A2 = lane.load(in.A) * LOG2E;
    floatx4 h = zero4();
    if (blockIdx.y == 0) {
        h = lane.load(carry ? carry + (int64_t)w.b * C * N : nullptr);
        lane.store(sg.state + ((int64_t)w.b * sg.nseg + (REVERSE ? 0 : sg.nseg - 1)) * C * N, h);
    }
    float total = 0.f;
    float bias[VN];
    load_floats<VN>(bias, in.dt_bias ? in.dt_bias + rows.c : nullptr, rows.nc);
    u32x4 xv[PV], dv[PV], zv[PV] = {};
    Projections<T, N, 1> proj(REVERSE ? in.c : in.b, in.b, w, first, REVERSE ? -1 : 1);
    Stream<const T, R> xs(REVERSE ? dy : in.x, w, rows, first), ds(in.dt, w, rows, first), zs(in.z, w, rows, first);
    auto fetch = [&](int t0) {
        xs.load(xv, rows, end - t0);
        ds.load(dv, rows, end - t0);
        if (REVERSE && in.z.ptr)
            zs.load(zv, rows, end - t0);
        proj.load(end - t0);
        xs.move(move);
        ds.move(move);
        zs.move(move);
    };
    if (begin < end)
        fetch(first);
    for (int t0 = first; t0 >= begin && t0 < end; t0 += move) {
        pace(REVERSE ? first - t0 : t0 - first, end - begin);
#pragma unroll
        for (int i = 0; i < PV; ++i) {
            const int r = rows.token(i);
            float d[VN], u[VN];
            steps<T, VN>(d, dv[i], bias, in.softplus);
#pragma unroll
            for (int j = 0; j < VN; ++j)
                u[j] = REVERSE ? vec_get<T>(xv[i], j) : d[j] * vec_get<T>(xv[i], j);
            if (REVERSE && in.z.ptr)
#pragma unroll
                for (int j = 0; j < VN; ++j) {
                    const float z = vec_get<T>(zv[i], j);
                    u[j] *= z * sigmoid(z);
                }
            if (R::COUNT >= NT || (int)threadIdx.x < R::COUNT) {
                absent<VN>(d, t0 + TILE > end, t0 + r >= end);
#pragma unroll
                for (int j = 0; j < VN; j += 2)
                    *reinterpret_cast<floatx4*>(&step[r][2 * (R::pair(rows.col() / 2) ^ j / 2)]) = floatx4{d[j], u[j], d[j + 1], u[j + 1]};
            }
        }
        proj.store(bc);
        if (t0 + move >= begin && t0 + move < end)
            fetch(t0 + move);
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < TILE; ++k) {
            const int t = REVERSE ? TILE - 1 - k : k;
            const float2 s = step[t][at];
            const floatx4 v = *reinterpret_cast<const floatx4*>(&bc[0][t][lane.q * NS]);
            if constexpr (REVERSE)
                h = exp2_4(s.x * A2) * (h + s.y * v);
            else
                h = exp2_4(s.x * A2) * h + s.y * v;
            total += s.x;
        }
        __syncthreads();
    }
    const int64_t own = (int64_t)w.b * sg.nseg + seg;
    lane.store(sg.state + own * C * N, h);
    if (lane.ok && lane.q == 0)
        sg.total[own * C + lane.c] = total;
}

// exp2(2 x) h, a segment's part in what it passes on of h: the product is finite
// wherever its value is, although exp2(2 x) may not be (a state that grows token by
// token from a small value, or one that is still zero, which the walk keeps zero).
// From 2^127 on the half's factor is held there: its square takes every h but zero past
// the largest number, as the factor itself.
__device__ __forceinline__ floatx4 across(floatx4 x, const floatx4& h)
{
#pragma unroll
    for (int j = 0; j < 4; ++j)
        x[j] = fminf(x[j], 127.f);
    x = exp2_4(x);
    return x * (x * h);
}

// The state that enters segment `seg` (REVERSE: the gradient that enters it from
// behind), from what those before it in order make.
template <int N, bool REVERSE>
__device__ __forceinline__ floatx4 enter(const Segments& sg, const Lane<N>& lane, const floatx4& A2, int b, int seg, int C)
{
    constexpr int W = 16;   // segments read together
    const int order = REVERSE ? sg.nseg - 1 - seg : seg;
    const int64_t at = (int64_t)b * sg.nseg + (REVERSE ? sg.nseg - 1 : 0);   // of the first in order
    const int64_t step = REVERSE ? -1 : 1;
    if (order == 0)
        return lane.load(sg.state + ((int64_t)b * sg.nseg + (REVERSE ? 0 : sg.nseg - 1)) * C * N);
    // (half of A2, not of the sums: a product formed where they are loaded would wait for each)
    const floatx4 half = 0.5f * A2;
    floatx4 h = lane.load(sg.state + at * C * N);
    for (int k = 1; k < order; k += W) {
        floatx4 own[W];
        float d[W];
#pragma unroll
        for (int u = 0; u < W; ++u) {
            const int64_t i = at + min(k + u, order - 1) * step;
            own[u] = lane.load(sg.state + i * C * N);
            d[u] = lane.ok ? sg.total[i * C + lane.c] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < W; ++u)
            if (k + u < order)
                h = across(d[u] * half, h) + own[u];
    }
    return h;
}

// ---- forward -----------------------------------------------------------------
//
// 4 x 4096 x 2048 x 16 states, bf16, ragged: 99 + 130 us (the segments' pass and the
// walk).  Loads of the walk's operands 4 tokens ahead, pinned by scheduling barriers,
// took 50 registers and gained nothing (344 us at two waves a SIMD, 165 for 151 at
// three instead of four).

template <typename T, typename OT, int N>
__global__ __launch_bounds__(NT) void scan_fwd_kernel(In<T> in, const float* h_in, const int* n_new, Act<OT> y, float* h_out,
                                                      float* saved, Segments sg, int T_, int C, int G, int blocks)
{
    typedef Rows<T, N> R;
    constexpr int CW = Geo<N>::CW, L = Geo<N>::L, TILE = Geo<N>::TILE, VN = R::VN, PV = R::PV;
    __shared__ __attribute__((aligned(16))) float2 step[TILE][CW + 2];   // d, d x (rows 4 banks apart, as those below)
    __shared__ __attribute__((aligned(16))) float ysum[TILE][CW + 4];
    __shared__ __attribute__((aligned(16))) float bc[2][TILE][N];
    const Where w = where<N>(n_new, T_, C, G, blocks);
    const R rows(w);
    const Lane<N> lane(w);
    const int at = 2 * R::pair(lane.col / 2) + lane.col % 2;   // where this channel's step lies
    const int seg = blockIdx.y;
    const int begin = seg * sg.seg, end = begin + min(max(w.n - begin, 0), sg.seg);
    floatx4 A2 = lane.load(in.A), h = zero4();
    A2 *= LOG2E;
    h = sg.nseg > 1 ? enter<N, false>(sg, lane, A2, w.b, seg, C) : lane.load(h_in ? h_in + (int64_t)w.b * C * N : nullptr);
    float bias[VN], skip[VN];
    load_floats<VN>(bias, in.dt_bias ? in.dt_bias + rows.c : nullptr, rows.nc);
    load_floats<VN>(skip, in.D ? in.D + rows.c : nullptr, rows.nc);
    u32x4 xv[PV], dv[PV], zv[PV] = {};
    Projections<T, N, 2> proj(in.b, in.c, w, begin, 1);
    Stream<const T, R> xs(in.x, w, rows, begin), ds(in.dt, w, rows, begin), zs(in.z, w, rows, begin);
    Stream<OT, R> ys(y, w, rows, begin);
    auto fetch = [&](int t0) {
        xs.load(xv, rows, end - t0);
        ds.load(dv, rows, end - t0);
        if (in.z.ptr)
            zs.load(zv, rows, end - t0);
        proj.load(end - t0);
        xs.move(TILE);
        ds.move(TILE);
        zs.move(TILE);
    };
    if (begin < end)
        fetch(begin);
    for (int t0 = begin; t0 < end; t0 += TILE) {
        pace(t0 - begin, end - begin);
        u32x4 xc[PV], zc[PV];
#pragma unroll
        for (int i = 0; i < PV; ++i) {
            xc[i] = xv[i];
            zc[i] = zv[i];
            const int r = rows.token(i);
            float d[VN];
            steps<T, VN>(d, dv[i], bias, in.softplus);
            if (R::COUNT >= NT || (int)threadIdx.x < R::COUNT) {
                absent<VN>(d, t0 + TILE > end, t0 + r >= end);   // a token that is not there leaves the state as it is
#pragma unroll
                for (int j = 0; j < VN; j += 2)
                    *reinterpret_cast<floatx4*>(&step[r][2 * (R::pair(rows.col() / 2) ^ j / 2)]) =
                        floatx4{d[j], d[j] * vec_get<T>(xv[i], j), d[j + 1], d[j + 1] * vec_get<T>(xv[i], j + 1)};
            }
        }
        proj.store(bc);
        if (t0 + TILE < end)
            fetch(t0 + TILE);
        __syncthreads();
        float* sp = saved ? saved + ((int64_t)w.b * ((T_ + BLOCK - 1) / BLOCK) + t0 / BLOCK) * C * N : nullptr;
        for (int k = 0; k < TILE; k += BLOCK) {
            if (sp && t0 + k < end)
                lane.store(sp + (int64_t)(k / BLOCK) * C * N, h);
            float o[BLOCK];
#pragma unroll
            for (int t = 0; t < BLOCK; ++t) {
                const float2 s = step[k + t][at];
                const floatx4 bv = *reinterpret_cast<const floatx4*>(&bc[0][k + t][lane.q * NS]);
                h = exp2_4(s.x * A2) * h + s.y * bv;
                o[t] = dot4(*reinterpret_cast<const floatx4*>(&bc[1][k + t][lane.q * NS]), h);
            }
#pragma unroll
            for (int t = 0; t < BLOCK; t += 4) {   // every lane writes a token's sum: no branch in the walk
                float r[ChannelSums<L>::COUNT];
                ChannelSums<L>::sum(r, {o[t], o[t + 1], o[t + 2], o[t + 3]});
#pragma unroll
                for (int i = 0; i < ChannelSums<L>::COUNT; ++i)
                    ysum[k + t + 2 * i + (lane.q & (L == 2 ? 1 : 3))][lane.col] = r[i];
            }
        }
        __syncthreads();
        arrived(xv);
        arrived(dv);
        arrived(zv);
        arrived(proj.v);
#pragma unroll
        for (int i = 0; i < PV; ++i) {
            const int r = rows.token(i);
            if (t0 + r < end && rows.nc > 0) {
                float out[VN];
#pragma unroll
                for (int j = 0; j < VN; ++j)
                    out[j] = __builtin_fmaf(skip[j], vec_get<T>(xc[i], j), ysum[r][rows.col() + j]);
                if (in.z.ptr)
#pragma unroll
                    for (int j = 0; j < VN; ++j) {
                        const float z = vec_get<T>(zc[i], j);
                        out[j] *= z * sigmoid(z);
                    }
                store_vec<OT, VN>(ys.at(i), out, rows.nc);
            }
        }
        ys.move(TILE);
    }
    if (seg == sg.nseg - 1)
        lane.store(h_out + (int64_t)w.b * C * N, h);
}

// ---- backward ----------------------------------------------------------------
//
// Blocks of 8 tokens from behind: the block's states are formed again from the saved
// one that enters it, and kept with their gates in registers (64 of them), then
//   G_t = c_t e_t + g,  g = a_t G_t,  q_t = g h_{t-1}
// gives every gradient.  Saved states cost 8 bytes a token and channel at 16 states
// each way; fewer would take registers that two waves a SIMD do not have, or the
// exponentials a second time.  Sums over states and channels stay in order: lane
// swaps in the wave, LDS over the workgroup, a second kernel over workgroups.
// 8 x 2048 x 4096 bf16: 904 us; the same with sums over channels by single shuffles
// 2250, with the loader's values in the order of the channels in LDS 973, with the
// saved states read when they are needed 1060.
// GATE: there is a z.  Without one nothing takes c . h, and its product and sum are
// left out (4 x 2048 x 2048 x 16 bf16, a training step: 343 us, with them 358).  With
// one the pointer is asked for all the same: the branches keep the compiler from
// mixing the vectors' chains, which takes 12 registers more than there are.

template <typename OT>
struct Grads {
    Act<OT> dx, ddt, db, dc, dz;
    float* dh_in;
    float* params;   // [B * nseg][C N + 2 C]: dA, dD, ddt_bias of a workgroup
    float* proj;     // [G * blocks][B][T][2 N]: db, dc of a workgroup's channels
};

template <typename T, typename OT, int N, bool GATE>
__global__ __launch_bounds__(NT, 2) void scan_bwd_kernel(In<T> in, const float* saved, const int* n_new, Act<const T> dy,
                                                      const float* dh_out, Grads<OT> out, Segments sg, int T_, int C, int G,
                                                      int blocks)
{
    typedef Rows<T, N> R;
    constexpr int CW = Geo<N>::CW, L = Geo<N>::L, TILE = Geo<N>::TILE, VN = R::VN, PV = R::PV;
    // a row: d, d x, e, c . h of the channels (G . b in d x's place after the walk; in the order of R::place),
    // then the sums of q A
    constexpr int PITCH = (5 * CW + 31) / 32 * 32, SUMS = 4 * CW;
    constexpr int MANY = !GATE ? 2 : (L > 2) ? 3 : 4;   // sums over the states of a channel
    __shared__ __attribute__((aligned(128))) float slot[TILE][PITCH];
    __shared__ __attribute__((aligned(16))) float bc[2][TILE][N];
    __shared__ __attribute__((aligned(16))) float part[NT / 64][TILE][2 * N];
    const Where w = where<N>(n_new, T_, C, G, blocks);
    const R rows(w);
    const Lane<N> lane(w);
    const int seg = blockIdx.y;
    const int begin = seg * sg.seg, end = begin + min(max(w.n - begin, 0), sg.seg);
    const floatx4 A2 = lane.load(in.A) * LOG2E;
    floatx4 g = sg.nseg > 1 ? enter<N, true>(sg, lane, A2, w.b, seg, C)
                            : lane.load(dh_out ? dh_out + (int64_t)w.b * C * N : nullptr);
    floatx4 dA = zero4();
    typedef WaveSums<L> Sums;
    // where this lane's sums lie in the rows of its channel and of the tokens
    const float* const mine = &slot[0][4 * R::place(lane.col)];
    float* const own_at = &slot[0][lane.q & 3 ? 4 * R::place(lane.col) + (lane.q & 2 ? 3 : 1) : SUMS + lane.col];
    const int own_o = (int)(mine + 3 - own_at);   // (L == 2 writes c . h apart)
    float* const part_at = &part[threadIdx.x >> 6][Sums::token()][Sums::set() * N + lane.q * NS + Sums::of()];
    float bias[VN], skip[VN], dD[VN], dbias[VN];
    load_floats<VN>(bias, in.dt_bias ? in.dt_bias + rows.c : nullptr, rows.nc);
    load_floats<VN>(skip, in.D ? in.D + rows.c : nullptr, rows.nc);
#pragma unroll
    for (int j = 0; j < VN; ++j)
        dD[j] = dbias[j] = 0.f;
    u32x4 xv[PV], dv[PV], zv[PV] = {}, gv[PV];
    const int last = begin + (end - 1 - begin) / TILE * TILE;
    Projections<T, N, 2> proj(in.b, in.c, w, last, -1);
    Stream<const T, R> xs(in.x, w, rows, last), ts(in.dt, w, rows, last), zs(in.z, w, rows, last), gs(dy, w, rows, last);
    Stream<OT, R> dxs(out.dx, w, rows, last), dts(out.ddt, w, rows, last), dzs(out.dz, w, rows, last);
    auto fetch = [&](int t0) {
        xs.load(xv, rows, end - t0);
        ts.load(dv, rows, end - t0);
        if (GATE && in.z.ptr)
            zs.load(zv, rows, end - t0);
        gs.load(gv, rows, end - t0);
        proj.load(end - t0);
        xs.move(-TILE);
        ts.move(-TILE);
        zs.move(-TILE);
        gs.move(-TILE);
    };
    const float* sp = saved + ((int64_t)w.b * ((T_ + BLOCK - 1) / BLOCK) + (end - 1) / BLOCK) * C * N;
    floatx4 hn = zero4();
    if (begin < end) {
        fetch(last);
        hn = lane.load(sp);
    }
    for (int t0 = last; t0 >= begin && begin < end; t0 -= TILE) {
        pace(last - t0, end - begin);
        u32x4 xc[PV];
        float ds[PV][VN], dg[PV][VN];   // slope of the step, dy times the slope of the gate
#pragma unroll
        for (int i = 0; i < PV; ++i) {
            xc[i] = xv[i];
            const int r = rows.token(i);
            float d[VN], e[VN];
            steps<T, VN>(d, ds[i], dv[i], bias, in.softplus);
#pragma unroll
            for (int j = 0; j < VN; ++j)
                e[j] = dg[i][j] = vec_get<T>(gv[i], j);
            if (GATE && in.z.ptr)
#pragma unroll
                for (int j = 0; j < VN; ++j) {
                    const float z = vec_get<T>(zv[i], j), q = sigmoid(z), y = z * q;
                    dg[i][j] *= __builtin_fmaf(y, 1.f - q, q);
                    e[j] *= y;
                }
            absent<VN>(d, t0 + TILE > end, t0 + r >= end);   // a token that is not there passes the gradient on (its x and dy are zeros)
            if (R::COUNT >= NT || (int)threadIdx.x < R::COUNT)
#pragma unroll
                for (int j = 0; j < VN; ++j)
                    *reinterpret_cast<floatx4*>(&slot[0][0] + ((r * PITCH + 4 * rows.first()) ^ 4 * j)) =
                        floatx4{d[j], d[j] * vec_get<T>(xc[i], j), e[j], 0.f};
        }
        proj.store(bc);
        if (t0 > begin)
            fetch(t0 - TILE);
        __syncthreads();
        for (int k = (min(end - t0, TILE) - 1) / BLOCK; k >= 0; --k) {
            const int tk = k * BLOCK;
            const floatx4 h0 = hn;
            if (t0 + tk > begin) {   // the block before's, a block ahead
                sp -= (int64_t)C * N;
                hn = lane.load(sp);
            }
            floatx4 h = h0, hs[BLOCK], as[BLOCK];
#pragma unroll
            for (int t = 0; t < BLOCK; ++t) {
                const floatx4 s = *reinterpret_cast<const floatx4*>(mine + (tk + t) * PITCH);
                const floatx4 bv = *reinterpret_cast<const floatx4*>(&bc[0][tk + t][lane.q * NS]);
                as[t] = exp2_4(s[0] * A2);
                hs[t] = h = as[t] * h + s[1] * bv;
            }
            float sb[Sums::TOKENS], sc[Sums::TOKENS];
#pragma unroll
            for (int t = BLOCK - 1; t >= 0; --t) {
                const floatx4 s = *reinterpret_cast<const floatx4*>(mine + (tk + t) * PITCH);
                const floatx4 bv = *reinterpret_cast<const floatx4*>(&bc[0][tk + t][lane.q * NS]);
                const floatx4 cv = *reinterpret_cast<const floatx4*>(&bc[1][tk + t][lane.q * NS]);
                const floatx4 Gt = g + s[2] * cv;
                floatx4 pc = s[2] * hs[t], pb = s[1] * Gt;
                g = as[t] * Gt;
                const floatx4 qv = g * (t ? hs[t - 1] : h0);
                dA += s[0] * qv;
                // the channel's lanes write its sums together, and no lane branches
                float own[ChannelSums<L>::COUNT];
                const float o = GATE ? dot4(cv, hs[t]) : 0.f;   // (only dz takes it)
                ChannelSums<L>::template sum<MANY>(own, {dot4(qv, A2), dot4(Gt, bv), o, o});
#pragma unroll
                for (int i = 0; i < (GATE ? ChannelSums<L>::COUNT : 1); ++i)
                    own_at[(tk + t) * PITCH + (i ? own_o : 0)] = own[i];
                sb[t % Sums::TOKENS] = Sums::sum(pb);
                sc[t % Sums::TOKENS] = Sums::sum(pc);
                if (t % Sums::TOKENS == 0) {
                    float r[Sums::COUNT];
                    Sums::pick(r, sb, sc);
#pragma unroll
                    for (int i = 0; i < Sums::COUNT; ++i)
                        part_at[(tk + t) * 2 * N + i * N] = r[i];
                }
            }
        }
        __syncthreads();
        arrived(xv);
        arrived(dv);
        arrived(zv);
        arrived(gv);
        arrived(proj.v);
        asm volatile("" : "+v"(hn));
        // db, dc of this workgroup's channels
        float* pp = out.proj + (((int64_t)blockIdx.x * gridDim.z + w.b) * T_ + t0) * 2 * N;
#pragma unroll
        for (int i = threadIdx.x * 4; i < TILE * 2 * N; i += NT * 4)
            if (t0 + i / (2 * N) < end) {
                floatx4 s = zero4();
#pragma unroll
                for (int k = 0; k < NT / 64; ++k)
                    s += *reinterpret_cast<const floatx4*>(&part[k][i / (2 * N)][i % (2 * N)]);
                *reinterpret_cast<floatx4*>(pp + i) = s;
            }
#pragma unroll
        for (int i = 0; i < PV; ++i) {
            const int r = rows.token(i);
            if (t0 + r < end && rows.nc > 0) {
                float dx[VN], ddt[VN], dz[VN];
#pragma unroll
                for (int j = 0; j < VN; ++j) {
                    const floatx4 s =   // d, G . b, e, c . h
                        *reinterpret_cast<const floatx4*>(&slot[0][0] + ((r * PITCH + 4 * rows.first()) ^ 4 * j));
                    const float x = vec_get<T>(xc[i], j), da = slot[r][SUMS + rows.col() + j];
                    dx[j] = __builtin_fmaf(s[2], skip[j], s[1] * s[0]);
                    ddt[j] = __builtin_fmaf(s[1], x, da * LN2) * ds[i][j];   // (the walk sums q A in base 2)
                    if (GATE)
                        dz[j] = dg[i][j] * __builtin_fmaf(skip[j], x, s[3]);
                    dD[j] = __builtin_fmaf(s[2], x, dD[j]);
                    dbias[j] += ddt[j];
                }
                store_vec<OT, VN>(dxs.at(i), dx, rows.nc);
                store_vec<OT, VN>(dts.at(i), ddt, rows.nc);
                if (GATE && in.z.ptr)
                    store_vec<OT, VN>(dzs.at(i), dz, rows.nc);
            }
        }
        dxs.move(-TILE);
        dts.move(-TILE);
        dzs.move(-TILE);
        __syncthreads();   // before the next tile's values
    }
    if (seg == 0)
        lane.store(out.dh_in + (int64_t)w.b * C * N, g);
    float* pp = out.params + ((int64_t)w.b * sg.nseg + seg) * ((int64_t)C * N + 2 * C);
    lane.store(pp, dA);
    // dD and ddt_bias over the rows of a channel
    constexpr int ROWS = R::COUNT < NT ? TILE : NT / R::VPR;
    float* red = &slot[0][0];   // [2][ROWS][CW]
    static_assert(2 * ROWS <= 4 * TILE, "the sums fit the slots");
    __syncthreads();
    if ((int)threadIdx.x < R::COUNT)
#pragma unroll
        for (int j = 0; j < VN; ++j) {
            red[rows.row * CW + rows.col() + j] = dD[j];
            red[(ROWS + rows.row) * CW + rows.col() + j] = dbias[j];
        }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * CW; i += NT)
        if (w.c0 + i % CW < w.cend) {
            double s = 0.0;
            for (int r = 0; r < ROWS; ++r)
                s += red[((i / CW) * ROWS + r) * CW + i % CW];
            pp[(int64_t)C * N + (i / CW) * C + w.c0 + i % CW] = (float)s;
        }
}

// The sums over workgroups, in order: db and dc over those of a group's channels, 4
// values a thread, then (the last `cols` workgroups) dA, dD and ddt_bias over the
// sequences and segments, 64 columns and 4 slices of the sums a workgroup, in 64 bits:
// there are up to 32767 sums, and the kernel waits for memory either way.  Within a
// segment they are added in 32: the walk has no registers for more.
template <typename OT, int N>
__global__ __launch_bounds__(NT) void scan_finish_kernel(Grads<OT> out, float* dA, float* dD, float* dbias, const int* n_new,
                                                         int B, int T_, int C, int G, int blocks, int parts, int cols)
{
    __shared__ double sums[NT / 64][64];
    const int rows = gridDim.x - cols;
    if ((int)blockIdx.x < rows) {
        const int64_t ld = (int64_t)B * T_ * 2 * N, per = (int64_t)T_ * (2 * N / 4), count = per * B * G;
        for (int64_t i = blockIdx.x * (int64_t)NT + threadIdx.x; i < count; i += (int64_t)rows * NT) {
            const int64_t r = i % per, t = r / (2 * N / 4);
            const int b = (int)(i / per % B), g = (int)(i / per / B), at = (int)(r % (2 * N / 4)) * 4;
            if (t >= tokens_of(n_new, b, T_))
                continue;
            const float* p = out.proj + ((int64_t)g * blocks * B + b) * T_ * 2 * N + r * 4;
            floatx4 s = zero4();
#pragma unroll 8
            for (int k = 0; k < blocks; ++k)
                s += *reinterpret_cast<const floatx4*>(p + k * ld);
            const Act<OT>& o = at < N ? out.db : out.dc;
            const float v[4] = {s[0], s[1], s[2], s[3]};
            store_vec<OT, 4>(o.head(b, g) + t * o.st + at % N, v, 4);
        }
        return;
    }
    const int col = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const int64_t i = (blockIdx.x - rows) * 64ll + col, cn = (int64_t)C * N, ld = cn + 2 * C;
    double s = 0.0;
    if (i < ld)
#pragma unroll 8
        for (int q = slice; q < parts; q += NT / 64)
            s += out.params[q * ld + i];
    sums[slice][col] = s;
    __syncthreads();
    if (slice == 0 && i < ld) {
        for (int q = 1; q < NT / 64; ++q)
            s += sums[q][col];
        if (i < cn)
            dA[i] = (float)s;
        else if (i < cn + C) {
            if (dD)
                dD[i - cn] = (float)s;
        } else if (dbias) {
            dbias[i - cn - C] = (float)s;
        }
    }
}

// ---- token step --------------------------------------------------------------

// Bound by the states' bytes, read once and written once: 128 x 4096 x 16 states 17 us,
// 4.2 TB/s, as a pass among others; one sequence of 2048 3.4 us.  What a token needs
// beside its state is asked for before the slot is known, so that only the state's
// own latency follows the look at the slots.
template <typename T, typename OT, int N>
__global__ __launch_bounds__(NT) void scan_step_kernel(In<T> in, float* S, const int* slots, int nslots, Act<OT> y, int T_,
                                                       int C, int G)
{
    constexpr int CW = Geo<N>::CW, L = Geo<N>::L;
    const Where w{(int)blockIdx.y, 0, (int)blockIdx.x * CW, C, T_};
    const Lane<N> lane(w);
    const int c = min(lane.c, C - 1), g = c / (C / G);   // (a lane without a channel reads the last one's and writes nothing)
    const T* xp = in.x.ptr + w.b * in.x.sb + c;
    const T* dp = in.dt.ptr + w.b * in.dt.sb + c;
    const T* zp = in.z.ptr ? in.z.ptr + w.b * in.z.sb + c : nullptr;
    const T* bp = in.b.head(w.b, g) + lane.q * NS;
    const T* cp = in.c.head(w.b, g) + lane.q * NS;
    float x, d, z = 0.f;
    floatx4 bv, cv;
    auto token = [&](int64_t t) {
        x = (float)xp[t * in.x.st];
        d = (float)dp[t * in.dt.st];
        if (zp)
            z = (float)zp[t * in.z.st];
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            bv[j] = (float)bp[t * in.b.st + j];
            cv[j] = (float)cp[t * in.c.st + j];
        }
    };
    token(0);
    const floatx4 A2 = lane.load(in.A) * LOG2E;
    const float bias = in.dt_bias ? in.dt_bias[c] : 0.f, skip = in.D ? in.D[c] : 0.f;
    OT* yp = y.ptr + w.b * y.sb + lane.c;
    int slot = w.b;
    if (slots) {
        slot = slots[w.b];
        int bad = slot < 0 || slot >= nslots;
        for (int i = threadIdx.x; i < w.b; i += NT)
            bad |= slots[i] == slot;
        if (__syncthreads_or(bad)) {
            if (lane.ok && lane.q == 0)
                for (int t = 0; t < T_; ++t)
                    yp[(int64_t)t * y.st] = (OT)0.f;
            return;
        }
    }
    floatx4* Sp = reinterpret_cast<floatx4*>(S + ((int64_t)slot * C + c) * N + lane.q * NS);
    floatx4 h = *Sp;
    for (int t = 0; t < T_; ++t) {
        if (t > 0)
            token(t);
        d += bias;
        if (in.softplus)
            d = softplus(d);
        h = exp2_4(d * A2) * h + (d * x) * bv;
        float o = __builtin_fmaf(skip, x, channel_sum<L>(dot4(cv, h)));
        if (zp)
            o *= z * sigmoid(z);
        if (lane.ok && lane.q == 0)
            yp[(int64_t)t * y.st] = (OT)o;
    }
    if (lane.ok)
        *Sp = h;
}

// ---- host --------------------------------------------------------------------

int channels_per_block(int N) { return NT / 64 * 64 / (N / NS); }

// How a piece is split: `blocks` workgroups over the channels of a group, nseg
// segments of seg tokens.  Segments cost a pass that forms what they make of zeros
// (0.7 of the forward, 0.25 of the backward), so they are taken where the channels
// alone leave the GPU short of workgroups: at 256 of them (4 x 2048 x 4096, 16 states)
// a training step takes as long either way (877 us in one, 871 in four segments), at
// 512 splitting loses, at 128 (4 x 4096 x 2048) it wins.  Then 1024 workgroups, four a
// CU: 512 leave the forward 17% slower (16384 x 2048: 188 against 161 us).  At least 64
// tokens a segment (3 x 1023 x 1000: 60 + 21 us for the two walks, 64 + 26 with 128
// tokens).  Every segment's workgroup reads what those before it make, so there are at
// most 128 (65536 x 256: 417 us a step; 64 segments 584, 256 454), or 256 where a
// segment is one workgroup (32768 x 64: 158 us, with 128 188).
struct Plan {
    int blocks, nseg, seg;
    Plan(const linrec_scan_desc* d)
    {
        const int cw = channels_per_block(d->N);
        blocks = (d->C / d->G + cw - 1) / cw;
        const int64_t wgs = (int64_t)blocks * d->G * d->B;
        const int64_t want = wgs >= 320 ? 1 : std::min<int64_t>({(1023 + wgs) / wgs, (d->T + 63) / 64, wgs == 1 ? 256 : 128});
        const int64_t len = (d->T + want - 1) / want;
        seg = (int)((len + SEG - 1) / SEG * SEG);
        nseg = (int)((d->T + (int64_t)seg - 1) / seg);
    }
};

linrec_status check_scan_desc(const linrec_scan_desc* d)
{
    if (!d)
        return LINREC_E_NULL;
    if ((d->dtype != LINREC_BF16 && d->dtype != LINREC_F32) ||
        (d->out_dtype != LINREC_BF16 && d->out_dtype != LINREC_F32) ||
        (d->dtype == LINREC_F32 && d->out_dtype != LINREC_F32))
        return LINREC_E_DTYPE;
    if (d->B < 1 || d->B > 32767 || d->C < 1 || d->C > (1 << 20) || d->T < 0 || d->T > LINREC_MAX_T)
        return LINREC_E_SHAPE;
    if (d->N != 8 && d->N != 16 && d->N != 32 && d->N != 64)
        return LINREC_E_SHAPE;
    if (d->G < 1 || d->G > 65535 || d->C % d->G || (d->G > 1 && (d->C / d->G * elem_size(d->dtype)) % 16))
        return LINREC_E_SHAPE;
    if (d->softplus != 0 && d->softplus != 1)
        return LINREC_E_LAYOUT;
    return LINREC_OK;
}

linrec_status check_proj(const linrec_scan_desc* d, const linrec_tensor& t, int dtype, bool out)
{
    return check_view(t, d->B, d->G, d->T, d->N, elem_size(dtype), out);
}

linrec_status check_inputs(const linrec_scan_desc* d, const linrec_scan_inputs* in)
{
    linrec_status st;
    if (!in)
        return LINREC_E_NULL;
    if ((st = check_rows(d, in->x, d->dtype, false)) != LINREC_OK || (st = check_rows(d, in->dt, d->dtype, false)) != LINREC_OK ||
        (st = check_proj(d, in->b, d->dtype, false)) != LINREC_OK || (st = check_proj(d, in->c, d->dtype, false)) != LINREC_OK ||
        (in->z.ptr && (st = check_rows(d, in->z, d->dtype, false)) != LINREC_OK) ||
        (st = check_state_ptr(in->A, true)) != LINREC_OK || (st = check_state_ptr(in->D, false)) != LINREC_OK ||
        (st = check_state_ptr(in->dt_bias, false)) != LINREC_OK)
        return st;
    return LINREC_OK;
}

template <typename T>
Act<const T> chead(const linrec_tensor& a) { return Act<const T>{(const T*)a.ptr, a.sb, a.sh, a.st}; }
template <typename T>
Act<T> mhead(const linrec_tensor& a) { return Act<T>{(T*)a.ptr, a.sb, a.sh, a.st}; }

template <typename T>
In<T> inputs(const linrec_scan_desc* d, const linrec_scan_inputs* in)
{
    return In<T>{cact<T>(in->x), cact<T>(in->dt), chead<T>(in->b), chead<T>(in->c), cact<T>(in->z),
                 in->A, in->D, in->dt_bias, d->softplus};
}

// Calls f with (input type, output type, states) of the description.
template <typename F>
hipError_t dispatch(const linrec_scan_desc* d, F&& f)
{
    auto states = [&](auto t, auto o) {
        switch (d->N) {
        case 8: return f(t, o, std::integral_constant<int, 8>{});
        case 16: return f(t, o, std::integral_constant<int, 16>{});
        case 32: return f(t, o, std::integral_constant<int, 32>{});
        default: return f(t, o, std::integral_constant<int, 64>{});
        }
    };
    if (d->dtype == LINREC_F32)
        return states(float{}, float{});
    return d->out_dtype == LINREC_F32 ? states(bf16{}, float{}) : states(bf16{}, bf16{});
}

int64_t state_floats(const linrec_scan_desc* d) { return (int64_t)d->B * d->C * d->N; }

// The segments' part of a workspace.
int64_t segment_floats(const linrec_scan_desc* d, const Plan& p)
{
    return p.nseg > 1 ? p.nseg * state_floats(d) + round4((int64_t)d->B * p.nseg * d->C) : 0;
}

Segments segments(const linrec_scan_desc* d, const Plan& p, void* workspace)
{
    float* w = (float*)workspace;
    return p.nseg > 1 ? Segments{p.nseg, p.seg, w, w + p.nseg * state_floats(d)} : Segments{1, p.seg, nullptr, nullptr};
}

int64_t params_floats(const linrec_scan_desc* d, const Plan& p)
{
    return round4((int64_t)d->B * p.nseg * ((int64_t)d->C * d->N + 2 * d->C));
}

}  // namespace
}  // namespace linrec

using namespace linrec;

extern "C" {

size_t linrec_scan_saved_bytes(const linrec_scan_desc* d)
{
    if (check_scan_desc(d) != LINREC_OK)
        return 0;
    return (size_t)(((int64_t)d->T + BLOCK - 1) / BLOCK) * (size_t)state_floats(d) * sizeof(float);
}

size_t linrec_scan_fwd_workspace_bytes(const linrec_scan_desc* d)
{
    if (check_scan_desc(d) != LINREC_OK || d->T == 0)
        return 0;
    return (size_t)segment_floats(d, Plan(d)) * sizeof(float);
}

size_t linrec_scan_bwd_workspace_bytes(const linrec_scan_desc* d)
{
    if (check_scan_desc(d) != LINREC_OK || d->T == 0)
        return 0;
    const Plan p(d);
    return (size_t)(segment_floats(d, p) + params_floats(d, p) + (int64_t)d->G * p.blocks * d->B * d->T * 2 * d->N) *
           sizeof(float);
}

linrec_status linrec_scan_fwd(linrec_ctx* ctx, const linrec_scan_desc* d, const linrec_scan_inputs* in, const float* h_in,
                              const int32_t* n_new, linrec_tensor y, float* h_out, void* saved, void* workspace, void* stream)
{
    linrec_status st;
    if ((st = check_scan_desc(d)) != LINREC_OK || (st = check_state_ptr(h_in, false)) != LINREC_OK ||
        (st = check_state_ptr(h_out, true)) != LINREC_OK)
        return st;
    if (d->T > 0) {
        if ((st = check_inputs(d, in)) != LINREC_OK || (st = check_rows(d, y, d->out_dtype, true)) != LINREC_OK)
            return st;
        if (!aligned(n_new, 4))
            return LINREC_E_ALIGN;
        if ((saved && (st = check_buffer(saved)) != LINREC_OK) ||
            (linrec_scan_fwd_workspace_bytes(d) && (st = check_buffer(workspace)) != LINREC_OK))
            return st;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    hipStream_t s = (hipStream_t)stream;
    if (d->T == 0)
        return pass_carry(h_in, h_out, state_floats(d), s);
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_SCAN_FWD, s, [&] {
        return dispatch(d, [&](auto t, auto o, auto n) {
            using T = decltype(t);
            using OT = decltype(o);
            constexpr int N = decltype(n)::value;
            const Plan p(d);
            const Segments sg = segments(d, p, workspace);
            const In<T> a = inputs<T>(d, in);
            const unsigned wgs = (unsigned)p.blocks * d->G;
            if (p.nseg > 1)
                launch_kernel(scan_sum_kernel<T, N, false>, dim3(wgs, p.nseg - 1, d->B), dim3(NT), s, a, h_in, n_new,
                              cact<T>(in->x), sg, d->T, d->C, d->G, p.blocks);
            launch_kernel(scan_fwd_kernel<T, OT, N>, dim3(wgs, p.nseg, d->B), dim3(NT), s, a, h_in, n_new, mact<OT>(y),
                          h_out, (float*)saved, sg, d->T, d->C, d->G, p.blocks);
            return hipGetLastError();
        });
    }));
    return LINREC_OK;
}

linrec_status linrec_scan_bwd(linrec_ctx* ctx, const linrec_scan_desc* d, const linrec_scan_inputs* in, const void* saved,
                              const int32_t* n_new, linrec_tensor dy, const float* dh_out, const linrec_scan_grads* out,
                              void* workspace, void* stream)
{
    linrec_status st;
    if ((st = check_scan_desc(d)) != LINREC_OK || (st = check_state_ptr(dh_out, false)) != LINREC_OK)
        return st;
    if (!out)
        return LINREC_E_NULL;
    if ((st = check_state_ptr(out->dh_in, true)) != LINREC_OK || (st = check_state_ptr(out->dA, true)) != LINREC_OK ||
        (st = check_state_ptr(out->dD, false)) != LINREC_OK || (st = check_state_ptr(out->ddt_bias, false)) != LINREC_OK)
        return st;
    if (d->T > 0) {
        if ((st = check_inputs(d, in)) != LINREC_OK || (st = check_rows(d, dy, d->dtype, false)) != LINREC_OK ||
            (st = check_rows(d, out->dx, d->out_dtype, true)) != LINREC_OK ||
            (st = check_rows(d, out->ddt, d->out_dtype, true)) != LINREC_OK ||
            (st = check_proj(d, out->db, d->out_dtype, true)) != LINREC_OK ||
            (st = check_proj(d, out->dc, d->out_dtype, true)) != LINREC_OK ||
            (in->z.ptr && (st = check_rows(d, out->dz, d->out_dtype, true)) != LINREC_OK))
            return st;
        if (!aligned(n_new, 4))
            return LINREC_E_ALIGN;
        if ((st = check_buffer(saved)) != LINREC_OK || (st = check_buffer(workspace)) != LINREC_OK)
            return st;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    hipStream_t s = (hipStream_t)stream;
    if (d->T == 0) {
        LAUNCH(launch_carry_copy(nullptr, out->dA, (int64_t)d->C * d->N, s));
        if (out->dD)
            LAUNCH(launch_carry_copy(nullptr, out->dD, d->C, s));
        if (out->ddt_bias)
            LAUNCH(launch_carry_copy(nullptr, out->ddt_bias, d->C, s));
        return pass_carry(dh_out, out->dh_in, state_floats(d), s);
    }
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_SCAN_BWD, s, [&] {
        return dispatch(d, [&](auto t, auto o, auto n) {
            using T = decltype(t);
            using OT = decltype(o);
            constexpr int N = decltype(n)::value;
            const Plan p(d);
            const Segments sg = segments(d, p, workspace);
            const In<T> a = inputs<T>(d, in);
            float* params = (float*)workspace + segment_floats(d, p);
            const Grads<OT> gr{mact<OT>(out->dx), mact<OT>(out->ddt), mhead<OT>(out->db), mhead<OT>(out->dc),
                               mact<OT>(out->dz), out->dh_in, params, params + params_floats(d, p)};
            const unsigned wgs = (unsigned)p.blocks * d->G;
            const int64_t cn = (int64_t)d->C * N;
            if (p.nseg > 1)
                launch_kernel(scan_sum_kernel<T, N, true>, dim3(wgs, p.nseg - 1, d->B), dim3(NT), s, a, dh_out, n_new, cact<T>(dy),
                              sg, d->T, d->C, d->G, p.blocks);
            launch_kernel(in->z.ptr ? scan_bwd_kernel<T, OT, N, true> : scan_bwd_kernel<T, OT, N, false>,
                          dim3(wgs, p.nseg, d->B), dim3(NT), s, a, (const float*)saved, n_new, cact<T>(dy), dh_out, gr, sg,
                          d->T, d->C, d->G, p.blocks);
            const int cols = (int)((cn + 2 * d->C + 63) / 64);
            const int64_t rounds = ((int64_t)d->B * d->G * d->T * (2 * N / 4) + NT - 1) / NT;
            launch_kernel(scan_finish_kernel<OT, N>, dim3((unsigned)std::min<int64_t>(rounds, 8192) + cols), dim3(NT), s, gr,
                          out->dA, out->dD, out->ddt_bias, n_new, d->B, d->T, d->C, d->G, p.blocks, d->B * p.nseg, cols);
            return hipGetLastError();
        });
    }));
    return LINREC_OK;
}

linrec_status linrec_scan_step(linrec_ctx* ctx, const linrec_scan_desc* d, const linrec_scan_inputs* in, float* S,
                               const int32_t* slots, int32_t nslots, linrec_tensor y, void* stream)
{
    linrec_status st;
    if ((st = check_scan_desc(d)) != LINREC_OK)
        return st;
    if (d->T > 0) {
        if (!S)
            return LINREC_E_NULL;
        if (nslots < 1 || (!slots && nslots < d->B))
            return LINREC_E_SHAPE;
        if ((st = check_inputs(d, in)) != LINREC_OK || (st = check_rows(d, y, d->out_dtype, true)) != LINREC_OK)
            return st;
        if (!aligned(S, 16) || !aligned(slots, 4))
            return LINREC_E_ALIGN;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    if (d->T == 0)
        return LINREC_OK;
    hipStream_t s = (hipStream_t)stream;
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_SCAN_STEP, s, [&] {
        return dispatch(d, [&](auto t, auto o, auto n) {
            using T = decltype(t);
            using OT = decltype(o);
            constexpr int N = decltype(n)::value;
            launch_kernel(scan_step_kernel<T, OT, N>, dim3((d->C + Geo<N>::CW - 1) / Geo<N>::CW, d->B), dim3(NT), s,
                          inputs<T>(d, in), S, slots, nslots, mact<OT>(y), d->T, d->C, d->G);
            return hipGetLastError();
        });
    }));
    return LINREC_OK;
}

}  // extern "C"
