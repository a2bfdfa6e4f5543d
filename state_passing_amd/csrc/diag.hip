// diag.hip -- the elementwise gated recurrence (linrec_diag_fwd / _bwd):
//   h_t = a_t h_{t-1} + b_t,  a = exp(g),  b = x or (1 - a) x,
// one state per batch and channel.
//
// A token step is the affine map h -> a h + b, so 256 tokens (a segment) of a
// channel are one map (P, B) too.  A workgroup holds a segment of CH channels
// in registers: a lane owns one 16-byte vector of channels and 8 consecutive
// tokens (a run), so a load instruction reads 8 rows of 128 bytes.  Each run is
// folded to its map, the maps of the 32 runs are folded through LDS from the
// state that enters the segment, and the run is replayed from its entry.
//
// Segments of a piece are chained in one pass over the data: a workgroup
// publishes its segment's map, then finds the state that enters it by looking
// back: from the nearest segment whose leaving state is published, through the
// maps published since.  Whichever segment that is, the arithmetic is the same
// sequence s <- P s + B, so results do not depend on timing.
//
// Bound by HBM: 3 elements a token and channel forward, 5 backward.  65536 x 2048
// bf16: 166 us forward (4.9 TB/s), 254 us backward (5.3 TB/s); 2 x 4096 x 1024
// fp32 forward 20 us (4.9 TB/s); a copy reaches 4.85.  A ragged 3 x 4099 x 1000
// in the mix form, about one round of workgroups, takes 28 and 47 us (2.6 TB/s):
// its loads, exponentials and stores follow each other.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ctx.hpp"
#include "device.hpp"

namespace linrec {
namespace {

constexpr int SEG = 256;   // tokens per segment
constexpr int RUN = 8;     // tokens per lane

// Views [B, T, C]: sh unused.
template <typename T>
struct Vec {
    static constexpr int N = 16 / sizeof(T);
};

// The 16-byte vector of channels c .. c+N-1 of a token row; channels past n
// are not read and come as zeros.
template <typename T>
__device__ __forceinline__ u32x4 load_vec(const T* p, int n)
{
    if (n >= Vec<T>::N)
        return *reinterpret_cast<const u32x4*>(p);
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j)
        if (j < n) {
            if constexpr (sizeof(T) == 2)
                v[j / 2] |= (unsigned)reinterpret_cast<const unsigned short*>(p)[j] << (16 * (j & 1));
            else
                v[j] = reinterpret_cast<const unsigned*>(p)[j];
        }
    return v;
}

template <typename T>
__device__ __forceinline__ float vec_get(const u32x4& v, int j)
{
    if constexpr (sizeof(T) == 2)
        return __uint_as_float((j & 1) ? v[j / 2] & 0xffff0000u : v[j / 2] << 16);
    else
        return __uint_as_float(v[j]);
}

// N values of a token row, rounded to OT (nearest even).
template <typename OT, int N>
__device__ __forceinline__ void store_vec(OT* p, const float* y, int n)
{
    if (n >= N) {
        if constexpr (sizeof(OT) == 2) {
            static_assert(N == 8, "16-byte rows of bf16");
            bf16x8 o;
#pragma unroll
            for (int j = 0; j < N; ++j)
                o[j] = (bf16)y[j];
            *reinterpret_cast<bf16x8*>(p) = o;
        } else {
#pragma unroll
            for (int j = 0; j < N; j += 4)
                *reinterpret_cast<floatx4*>(p + j) = floatx4{y[j], y[j + 1], y[j + 2], y[j + 3]};
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < n)
                p[j] = (OT)y[j];
    }
}

// N floats of a carried state, n of which exist; p may be NULL (zeros).
template <int N>
__device__ __forceinline__ void load_floats(float (&y)[N], const float* p, int n)
{
    if (p && n >= N && ((uintptr_t)p & 15) == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 4) {
            const floatx4 v = *reinterpret_cast<const floatx4*>(p + j);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                y[j + i] = v[i];
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            y[j] = p && j < n ? p[j] : 0.f;
    }
}

template <int N>
__device__ __forceinline__ void store_floats(float* p, const float (&y)[N], int n)
{
    if (n >= N && ((uintptr_t)p & 15) == 0) {
#pragma unroll
        for (int j = 0; j < N; j += 4)
            *reinterpret_cast<floatx4*>(p + j) = floatx4{y[j], y[j + 1], y[j + 2], y[j + 3]};
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < n)
                p[j] = y[j];
    }
}

// 1 - exp(g): near 0 the difference would cancel (relative error 2^-24 / |g|),
// so the series takes over there; its first dropped term, g^5 / 720, is 2^-24 of
// the sum at |g| = 1/8.
__device__ __forceinline__ float one_minus_exp(float g, float a)
{
    float s = -g * (1.f + g * (1.f / 2 + g * (1.f / 6 + g * (1.f / 24 + g * (1.f / 120)))));
    asm("" : "+v"(s));   // both sides and a select: a branch for every value costs more
    return fabsf(g) < 0.125f ? s : 1.f - a;
}

template <bool MIX>
__device__ __forceinline__ float added(float g, float a, float x)
{
    return MIX ? one_minus_exp(g, a) * x : x;
}

// Where a lane's run lies.
template <typename T, int NRUN>
struct Place {
    int c0, nc, run, t0, nt;   // first channel, channels that exist, run, first token, tokens that exist
    __device__ __forceinline__ Place(int cg, int seg, int T_, int C, int block)
    {
        const int lanes = block / NRUN;   // channel lanes
        c0 = (cg * lanes + threadIdx.x % lanes) * Vec<T>::N;
        nc = C - c0;
        run = threadIdx.x / lanes;
        t0 = seg * SEG + run * RUN;
        nt = nc > 0 ? min(RUN, T_ - t0) : 0;
    }
};

template <typename T, int R = RUN>
__device__ __forceinline__ void load_run(u32x4 (&v)[R], const T* base, int64_t st, int t0, int nt, int nc)
{
#pragma unroll
    for (int r = 0; r < R; ++r)
        v[r] = r < nt ? load_vec(base + (int64_t)(t0 + r) * st, nc) : u32x4{0u, 0u, 0u, 0u};
}

// A token that does not exist has g = 0 and x = 0 (dh = 0): the identity.

// ---- the chain of segments ---------------------------------------------------
//
// Per segment and channel, in workspace: its map (product, sum) in 64 bits and
// the state leaving it in 32, both all ones until they are published, each by one
// atomic store: a reader that sees a value sees all of it, so no fence orders
// anything.  Counters hand out the segments of the chains (a channel group of a
// batch each) in the order the workgroups start: whoever waits for a map waits
// for a workgroup that runs already, and that publishes its map before it waits
// for anything itself, so every wait ends.  One counter is the bottleneck of a
// launch (about 25 ns a workgroup); one a chain lets chains drift apart, and rows
// are then read 128 bytes here and there.
constexpr unsigned UNSET = 0xffffffffu;

constexpr int COUNTERS = 8;   // at most
constexpr int COUNTER = 16;   // words from one counter to the next (64 bytes)

struct Chain {
    unsigned* counter;
    unsigned long long* map;
    unsigned* value;
};

__device__ __forceinline__ unsigned settled(float x)   // any NaN but the mark
{
    const unsigned u = __float_as_uint(x);
    return u == UNSET ? 0x7fc00000u : u;
}

__device__ __forceinline__ void publish_map(unsigned long long* p, float P, float B)
{
    __hip_atomic_store(p, (unsigned long long)settled(P) | (unsigned long long)__float_as_uint(B) << 32,
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ void publish_value(unsigned* p, float s)
{
    __hip_atomic_store(p, settled(s), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ unsigned long long look(const unsigned long long* p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ unsigned look(const unsigned* p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ float step_map(unsigned long long m, float s)
{
    return __builtin_fmaf(__uint_as_float((unsigned)m), s, __uint_as_float((unsigned)(m >> 32)));
}

// The state entering position i > 0 of a chain (this lane's channel; map and
// value point at position 0, `ld` apart), called by the lanes of one wave
// together.  The state that enters the piece is position 0's alone to read (its
// memory may be the last position's output): it comes with value[0], which
// waits for nobody.
__device__ __forceinline__ float chain_enter(const unsigned long long* map, const unsigned* value, int64_t ld, int i)
{
    constexpr int W = 8;   // positions looked at together
    int k = i - 1;         // nearest position of the window
    float s;
    for (;;) {
        unsigned v[W];
        unsigned long long m[W];
#pragma unroll
        for (int u = 0; u < W; ++u) {
            v[u] = look(value + max(k - u, 0) * ld);
            m[u] = look(map + max(k - u, 0) * ld);
        }
        int at = W;        // window offset of the state to start from
        bool open = true;  // every map before it is there
#pragma unroll
        for (int u = 0; u < W; ++u)
            if (at == W && open) {
                if (k - u < 0) {
                    open = false;
                } else if (__all(v[u] != UNSET)) {
                    at = u;
                    s = __uint_as_float(v[u]);
                } else {
                    open = __all((unsigned)m[u] != UNSET);
                }
            }
        // something is missing, or all is there but the window's last position is 0,
        // whose state is about to be: look again (never past position 0)
        if (!open || (at == W && k < W)) {
            __builtin_amdgcn_s_sleep(1);
            continue;
        }
        if (at < W) {
#pragma unroll
            for (int u = W - 1; u >= 0; --u)
                if (u < at)
                    s = step_map(m[u], s);
            break;
        }
        k -= W;
    }
    for (int j = k + 1; j < i; j += W) {   // the windows passed over: their maps are there
        unsigned long long m[W];
#pragma unroll
        for (int u = 0; u < W; ++u)
            m[u] = look(map + min(j + u, i - 1) * ld);
#pragma unroll
        for (int u = 0; u < W; ++u)
            if (j + u < i)
                s = step_map(m[u], s);
    }
    return s;
}

// This workgroup's place: its channel group, position in the chain and batch.
struct Work {
    int cg, pos, b;
    __device__ __forceinline__ Work(const Chain& ch, int ncg, int B, int nseg)
    {
        const int chains = ncg * B, c = blockIdx.x % chains;
        int chain = c;
        pos = 0;
        if (nseg > 1) {
            // counter k hands out the segments of chains [first, end), a row of them at a time
            const int K = min(COUNTERS, chains), k = (int)((int64_t)c * K / chains);
            const int first = (int)(((int64_t)k * chains + K - 1) / K), end = (int)(((int64_t)(k + 1) * chains + K - 1) / K);
            __shared__ int next;
            if (threadIdx.x == 0)
                next = (int)(atomicAdd(ch.counter + k * COUNTER, 1u) + 1u);   // starts at all ones
            __syncthreads();
            pos = next / (end - first);
            chain = first + next % (end - first);
        }
        cg = chain % ncg;
        b = chain / ncg;
    }
};

// Orders the work: what is computed from the packed inputs behind these does not
// move in front of them, neither to the pass before (which would keep gates of
// every token: twice the inputs' registers) nor to the tokens before.
__device__ __forceinline__ void forget(u32x4 (&v)[RUN])
{
#pragma unroll
    for (int r = 0; r < RUN; ++r)
        asm volatile("" : "+v"(v[r]));
}

template <int N>
__device__ __forceinline__ void after(u32x4& v, u32x4& w, float (&state)[N])
{
#pragma unroll
    for (int j = 0; j < N; j += 4)
        asm volatile("" : "+v"(v), "+v"(w), "+v"(state[j]), "+v"(state[j + 1]), "+v"(state[j + 2]), "+v"(state[j + 3]));
}

__global__ __launch_bounds__(256) void diag_clear_kernel(u32x4* p, int64_t n)
{
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll)
        p[i] = u32x4{UNSET, UNSET, UNSET, UNSET};
}

// Forward over R tokens at most, for generation: one lane a vector of channels,
// no LDS, no barrier, and code that fits the first instruction fetches (the
// segment kernel took 7.5 us for one token of 64 x 2048, this takes 3.2).
template <typename T, typename OT, bool MIX, int R>
__global__ __launch_bounds__(64) void diag_token_kernel(Act<const T> g, Act<const T> x, Act<OT> h, const float* h_in,
                                                        float* states, float* h_out, int T_, int C)
{
    constexpr int N = Vec<T>::N;
    const int c0 = (blockIdx.x * 64 + threadIdx.x) * N, b = blockIdx.y, nc = C - c0;
    if (nc <= 0)
        return;
    u32x4 gv[R], xv[R];
    load_run<T, R>(gv, g.ptr + b * g.sb + c0, g.st, 0, T_, nc);
    load_run<T, R>(xv, x.ptr + b * x.sb + c0, x.st, 0, T_, nc);
    const int64_t at = (int64_t)b * C + c0;
    float hc[N];
    load_floats<N>(hc, h_in ? h_in + at : nullptr, nc);
    store_floats<N>(states + at, hc, nc);
    OT* hp = h.ptr + b * h.sb + c0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float gg = vec_get<T>(gv[r], j), a = __expf(gg);
            hc[j] = a * hc[j] + added<MIX>(gg, a, vec_get<T>(xv[r], j));
        }
        if (r < T_)
            store_vec<OT, N>(hp + (int64_t)r * h.st, hc, nc);
    }
    store_floats<N>(h_out + at, hc, nc);
}

// Forward over a segment.  Four workgroups a CU: gates are formed twice (once for
// the map, once for the replay) rather than kept, which takes 112 registers
// where keeping them took 206 (ragged forward 40 -> 28 us with the selects above).
template <typename T, typename OT, bool MIX>
__global__ __launch_bounds__(256, 4) void diag_fwd_kernel(
    Act<const T> g, Act<const T> x, Act<OT> h, const float* h_in, float* states, float* h_out, Chain ch,
    int B_, int T_, int C, int ncg, int nseg)
{
    constexpr int N = Vec<T>::N, NT = 256, NRUN = SEG / RUN, CH = NT / NRUN * N;
    __shared__ float sP[NRUN][CH], sB[NRUN][CH];
    const Work work(ch, ncg, B_, nseg);
    const int cg = work.cg, seg = work.pos, b = work.b;
    const Place<T, NRUN> p(cg, seg, T_, C, NT);
    u32x4 gv[RUN], xv[RUN];
    load_run(gv, g.ptr + b * g.sb + p.c0, g.st, p.t0, p.nt, p.nc);
    load_run(xv, x.ptr + b * x.sb + p.c0, x.st, p.t0, p.nt, p.nc);
    float hc[N];
    float P[N], B[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        P[j] = 1.f;
        B[j] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
        after<N>(gv[r], xv[r], B);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float gg = vec_get<T>(gv[r], j), a = __expf(gg);
            P[j] *= a;
            B[j] = a * B[j] + added<MIX>(gg, a, vec_get<T>(xv[r], j));
        }
    }
    const int cl = (threadIdx.x % (NT / NRUN)) * N;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        sP[p.run][cl + j] = P[j];
        sB[p.run][cl + j] = B[j];
    }
    __syncthreads();
    const int c = cg * CH + threadIdx.x;
    if (threadIdx.x < CH && c < C) {
        float s = seg == 0 && h_in ? h_in[(int64_t)b * C + c] : 0.f;
        if (nseg > 1) {
            const int64_t chain = (int64_t)b * nseg * C + c, at = chain + (int64_t)seg * C;
            float sp = 1.f, sb = 0.f;
#pragma unroll 8
            for (int i = 0; i < NRUN; ++i) {
                sb = sP[i][threadIdx.x] * sb + sB[i][threadIdx.x];
                sp *= sP[i][threadIdx.x];
            }
            publish_map(ch.map + at, sp, sb);
            if (seg > 0)
                s = chain_enter(ch.map + chain, ch.value + chain, C, seg);
            publish_value(ch.value + at, __builtin_fmaf(sp, s, sb));
        }
        states[((int64_t)b * nseg + seg) * C + c] = s;
#pragma unroll 8
        for (int i = 0; i < NRUN; ++i) {   // sB becomes the state entering run i
            const float bb = sB[i][threadIdx.x];
            sB[i][threadIdx.x] = s;
            s = sP[i][threadIdx.x] * s + bb;
        }
        if (seg == nseg - 1)
            h_out[(int64_t)b * C + c] = s;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j)
        hc[j] = sB[p.run][cl + j];
    OT* hp = h.ptr + b * h.sb + p.c0;
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
        after<N>(gv[r], xv[r], hc);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float gg = vec_get<T>(gv[r], j), a = __expf(gg);
            hc[j] = a * hc[j] + added<MIX>(gg, a, vec_get<T>(xv[r], j));
        }
        if (r < p.nt)
            store_vec<OT, N>(hp + (int64_t)(p.t0 + r) * h.st, hc, p.nc);
    }
}

// Backward of one segment: the states before each token from the state that
// enters the segment, then, from the right, with R the gradient arriving at h_t
// from later tokens:  G = dh + R,  dx = G or (1 - a) G,  dg = a G (h_{t-1} - [mix] x),
// R <- a G.  A run is also the map R -> P R + Q from its right end to its left.
// Channel by channel, so that the gates and states of one channel's run are live
// at a time (160 registers, three workgroups a CU).
template <typename T, typename OT, bool MIX>
__global__ __launch_bounds__(256, sizeof(T) == 2 && sizeof(OT) == 2 ? 3 : 2) void diag_bwd_kernel(
    Act<const T> g, Act<const T> x, Act<const T> dh, Act<OT> dg, Act<OT> dx, const float* states,
    const float* dh_out, float* dh_in, Chain ch, int B_, int T_, int C, int ncg, int nseg)
{
    constexpr int N = Vec<T>::N, NT = 256, NRUN = SEG / RUN, CH = NT / NRUN * N;
    __shared__ float sP[NRUN][CH], sB[NRUN][CH], sQ[NRUN][CH];
    const Work work(ch, ncg, B_, nseg);
    const int cg = work.cg, seg = nseg - 1 - work.pos, b = work.b;   // the chain runs from the right
    const Place<T, NRUN> p(cg, seg, T_, C, NT);
    u32x4 gv[RUN], xv[RUN], dv[RUN];
    load_run(gv, g.ptr + b * g.sb + p.c0, g.st, p.t0, p.nt, p.nc);
    load_run(xv, x.ptr + b * x.sb + p.c0, x.st, p.t0, p.nt, p.nc);
    load_run(dv, dh.ptr + b * dh.sb + p.c0, dh.st, p.t0, p.nt, p.nc);
    const int cl = (threadIdx.x % (NT / NRUN)) * N;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float P = 1.f, B = 0.f, Q = 0.f;
#pragma unroll
        for (int r = 0; r < RUN; ++r) {
            const float gg = vec_get<T>(gv[r], j), a = __expf(gg);
            Q += P * (a * vec_get<T>(dv[r], j));   // P: the gates of the run's earlier tokens
            P *= a;
            B = a * B + added<MIX>(gg, a, vec_get<T>(xv[r], j));
        }
        sP[p.run][cl + j] = P;
        sB[p.run][cl + j] = B;
        sQ[p.run][cl + j] = Q;
        forget(gv);
    }
    __syncthreads();
    // one wave-sized group of threads folds forward, another backward
    const int col = threadIdx.x % CH, c = cg * CH + col;
    if (threadIdx.x < CH && c < C) {
        float s = states[((int64_t)b * nseg + seg) * C + c];
#pragma unroll 8
        for (int i = 0; i < NRUN; ++i) {
            const float bb = sB[i][col];
            sB[i][col] = s;
            s = sP[i][col] * s + bb;
        }
    } else if (threadIdx.x >= 64 && threadIdx.x - 64 < CH && cg * CH + (int)threadIdx.x - 64 < C) {
        const int cc = threadIdx.x - 64;
        const int64_t at = (int64_t)b * C + cg * CH + cc;
        float R = work.pos == 0 && dh_out ? dh_out[at] : 0.f;
        if (nseg > 1) {
            const int64_t chain = (int64_t)b * nseg * C + cg * CH + cc, to = chain + (int64_t)work.pos * C;
            float sp = 1.f, sq = 0.f;
#pragma unroll 8
            for (int i = NRUN - 1; i >= 0; --i) {
                sq = sP[i][cc] * sq + sQ[i][cc];
                sp *= sP[i][cc];
            }
            publish_map(ch.map + to, sp, sq);
            if (work.pos > 0)
                R = chain_enter(ch.map + chain, ch.value + chain, C, work.pos);
            publish_value(ch.value + to, __builtin_fmaf(sp, R, sq));
        }
#pragma unroll 8
        for (int i = NRUN - 1; i >= 0; --i) {
            const float q = sQ[i][cc];
            sQ[i][cc] = R;
            R = sP[i][cc] * R + q;
        }
        if (seg == 0)
            dh_in[at] = R;
    }
    __syncthreads();
    // channel by channel, so that only one run of states is live; results take
    // the place of the inputs' registers
    float outg[RUN][2], outx[RUN][2];
    OT* gp = dg.ptr + b * dg.sb + p.c0;
    OT* xp = dx.ptr + b * dx.sb + p.c0;
    constexpr bool PACK = sizeof(T) == 2 && sizeof(OT) == 2;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (j % 2 == 0) {
            forget(gv);
            forget(xv);
            forget(dv);
        }
        float s = sB[p.run][cl + j], R = sQ[p.run][cl + j];
        float hp[RUN], a[RUN], w[RUN];   // h_{t-1}, the gate, what it lets in
#pragma unroll
        for (int r = 0; r < RUN; ++r) {
            const float gg = vec_get<T>(gv[r], j);
            a[r] = __expf(gg);
            w[r] = MIX ? one_minus_exp(gg, a[r]) : 1.f;
            hp[r] = s;
            s = a[r] * s + w[r] * vec_get<T>(xv[r], j);
        }
#pragma unroll
        for (int r = RUN - 1; r >= 0; --r) {
            const float G = vec_get<T>(dv[r], j) + R;
            R = a[r] * G;
            outg[r][j & 1] = R * (MIX ? hp[r] - vec_get<T>(xv[r], j) : hp[r]);
            outx[r][j & 1] = w[r] * G;
        }
        if constexpr (PACK) {
            if (j & 1) {
#pragma unroll
                for (int r = 0; r < RUN; ++r) {
                    gv[r][j / 2] = __builtin_bit_cast(unsigned, bf16x2{(bf16)outg[r][0], (bf16)outg[r][1]});
                    xv[r][j / 2] = __builtin_bit_cast(unsigned, bf16x2{(bf16)outx[r][0], (bf16)outx[r][1]});
                }
            }
        } else if (j & 1) {
#pragma unroll
            for (int r = 0; r < RUN; ++r)
                if (r < p.nt) {
                    const int64_t at = p.t0 + r;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (j - 1 + i < p.nc) {
                            gp[at * dg.st + j - 1 + i] = (OT)outg[r][i];
                            xp[at * dx.st + j - 1 + i] = (OT)outx[r][i];
                        }
                }
        }
    }
    if constexpr (PACK) {
#pragma unroll
        for (int r = 0; r < RUN; ++r)
            if (r < p.nt) {
                OT* go = gp + (int64_t)(p.t0 + r) * dg.st;
                OT* xo = xp + (int64_t)(p.t0 + r) * dx.st;
                if (p.nc >= N) {
                    *reinterpret_cast<u32x4*>(go) = gv[r];
                    *reinterpret_cast<u32x4*>(xo) = xv[r];
                } else {
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        if (j < p.nc) {
                            go[j] = (OT)vec_get<T>(gv[r], j);
                            xo[j] = (OT)vec_get<T>(xv[r], j);
                        }
                }
            }
    }
}

// ---- host ------------------------------------------------------------------

int64_t nseg_of(int64_t T) { return (T + SEG - 1) / SEG; }

int channels_per_group(int dtype) { return 8 * 16 / elem_size(dtype); }

linrec_status check_diag_desc(const linrec_diag_desc* d)
{
    if (!d)
        return LINREC_E_NULL;
    if ((d->dtype != LINREC_BF16 && d->dtype != LINREC_F32) ||
        (d->out_dtype != LINREC_BF16 && d->out_dtype != LINREC_F32) ||
        (d->dtype == LINREC_F32 && d->out_dtype != LINREC_F32))
        return LINREC_E_DTYPE;
    if (d->B < 1 || d->B > 32767 || d->C < 1 || d->C > (1 << 20) || d->T < 0 || d->T > LINREC_MAX_T)
        return LINREC_E_SHAPE;
    // a launch holds at most 2^32 - 1 threads along x
    const int64_t ncg = (d->C + channels_per_group(d->dtype) - 1) / channels_per_group(d->dtype);
    if (nseg_of(d->T) * ncg * d->B * 256 > 0xffffffffll)
        return LINREC_E_SHAPE;
    if (d->form != LINREC_DIAG_PLAIN && d->form != LINREC_DIAG_MIX)
        return LINREC_E_LAYOUT;
    return LINREC_OK;
}

linrec_status check_diag_rows(const linrec_diag_desc* d, const linrec_tensor& t, int dtype, bool out)
{
    return check_view(linrec_tensor{t.ptr, t.sb, 0, t.st}, d->B, 1, d->T, d->C, elem_size(dtype), out);
}

template <typename T>
Act<const T> cact(const linrec_tensor& a) { return Act<const T>{(const T*)a.ptr, a.sb, 0, a.st}; }
template <typename T>
Act<T> mact(const linrec_tensor& a) { return Act<T>{(T*)a.ptr, a.sb, 0, a.st}; }

// Calls f with (input type, output type, mix) of the description.
template <typename F>
hipError_t dispatch(const linrec_diag_desc* d, F&& f)
{
    auto form = [&](auto t, auto o) {
        return d->form == LINREC_DIAG_MIX ? f(t, o, std::true_type{}) : f(t, o, std::false_type{});
    };
    if (d->dtype == LINREC_F32)
        return form(float{}, float{});
    return d->out_dtype == LINREC_F32 ? form(bf16{}, float{}) : form(bf16{}, bf16{});
}

// Workspace: the chains' counters, then the maps, then the states leaving.
int64_t chain_cells(const linrec_diag_desc* d) { return (int64_t)d->B * nseg_of(d->T) * d->C; }

constexpr int64_t COUNTER_BYTES = COUNTERS * COUNTER * sizeof(unsigned);

Chain chain_of(const linrec_diag_desc* d, void* workspace)
{
    if (d->T <= SEG)
        return Chain{nullptr, nullptr, nullptr};
    unsigned long long* map = (unsigned long long*)((char*)workspace + COUNTER_BYTES);
    return Chain{(unsigned*)workspace, map, (unsigned*)(map + chain_cells(d))};
}

void clear_chain(const linrec_diag_desc* d, void* workspace, hipStream_t s)
{
    const int64_t n = (int64_t)linrec_diag_workspace_bytes(d) / 16;
    if (n > 0)
        launch_kernel(diag_clear_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 2048)), dim3(256), s,
                      (u32x4*)workspace, n);
}

hipError_t launch_diag_fwd(const linrec_diag_desc* d, const linrec_tensor& g, const linrec_tensor& x,
                           const float* h_in, const linrec_tensor& h, float* h_out, float* states,
                           void* workspace, hipStream_t s)
{
    return dispatch(d, [&](auto t, auto o, auto mix) {
        using T = decltype(t);
        using OT = decltype(o);
        constexpr bool MIX = decltype(mix)::value;
        const int cpg = channels_per_group(d->dtype), ncg = (d->C + cpg - 1) / cpg;
        const int nseg = (int)nseg_of(d->T);
        if (d->T <= RUN) {
            const dim3 grid((d->C + 64 * Vec<T>::N - 1) / (64 * Vec<T>::N), d->B);
            if (d->T == 1)
                launch_kernel(diag_token_kernel<T, OT, MIX, 1>, grid, dim3(64), s, cact<T>(g), cact<T>(x), mact<OT>(h),
                              h_in, states, h_out, d->T, d->C);
            else
                launch_kernel(diag_token_kernel<T, OT, MIX, RUN>, grid, dim3(64), s, cact<T>(g), cact<T>(x),
                              mact<OT>(h), h_in, states, h_out, d->T, d->C);
            return hipGetLastError();
        }
        clear_chain(d, workspace, s);
        launch_kernel(diag_fwd_kernel<T, OT, MIX>, dim3(ncg * nseg * d->B), dim3(256), s, cact<T>(g),
                      cact<T>(x), mact<OT>(h), h_in, states, h_out, chain_of(d, workspace), d->B, d->T, d->C,
                      ncg, nseg);
        return hipGetLastError();
    });
}

hipError_t launch_diag_bwd(const linrec_diag_desc* d, const linrec_tensor& g, const linrec_tensor& x,
                           const float* states, const linrec_tensor& dh, const float* dh_out,
                           const linrec_tensor& dg, const linrec_tensor& dx, float* dh_in, void* workspace,
                           hipStream_t s)
{
    return dispatch(d, [&](auto t, auto o, auto mix) {
        using T = decltype(t);
        using OT = decltype(o);
        constexpr bool MIX = decltype(mix)::value;
        const int cpg = channels_per_group(d->dtype), ncg = (d->C + cpg - 1) / cpg;
        const int nseg = (int)nseg_of(d->T);
        clear_chain(d, workspace, s);
        launch_kernel(diag_bwd_kernel<T, OT, MIX>, dim3(ncg * nseg * d->B), dim3(256), s, cact<T>(g), cact<T>(x),
                      cact<T>(dh), mact<OT>(dg), mact<OT>(dx), states, dh_out, dh_in, chain_of(d, workspace),
                      d->B, d->T, d->C, ncg, nseg);
        return hipGetLastError();
    });
}

linrec_status pass(const linrec_diag_desc* d, const float* in, float* out, hipStream_t s)
{
    if (in == out)
        return LINREC_OK;
    LAUNCH(launch_carry_copy(in, out, (int64_t)d->B * d->C, s));
    return LINREC_OK;
}

}  // namespace
}  // namespace linrec

using namespace linrec;

extern "C" {

size_t linrec_diag_states_bytes(const linrec_diag_desc* d)
{
    if (check_diag_desc(d) != LINREC_OK)
        return 0;
    return (size_t)d->B * (size_t)nseg_of(d->T) * (size_t)d->C * sizeof(float);
}

size_t linrec_diag_workspace_bytes(const linrec_diag_desc* d)
{
    if (check_diag_desc(d) != LINREC_OK || d->T <= SEG)
        return 0;
    return ((size_t)COUNTER_BYTES + 12 * (size_t)chain_cells(d) + 15) / 16 * 16;
}

linrec_status linrec_diag_fwd(linrec_ctx* ctx, const linrec_diag_desc* d, linrec_tensor g, linrec_tensor x,
                              const float* h_in, linrec_tensor h, float* h_out, void* states,
                              void* workspace, void* stream)
{
    linrec_status st;
    if ((st = check_diag_desc(d)) != LINREC_OK || (st = check_state_ptr(h_in, false)) != LINREC_OK ||
        (st = check_state_ptr(h_out, true)) != LINREC_OK)
        return st;
    if (d->T > 0) {
        if ((st = check_diag_rows(d, g, d->dtype, false)) != LINREC_OK ||
            (st = check_diag_rows(d, x, d->dtype, false)) != LINREC_OK ||
            (st = check_diag_rows(d, h, d->out_dtype, true)) != LINREC_OK ||
            (st = check_buffer(states)) != LINREC_OK)
            return st;
        if (d->T > SEG && (st = check_buffer(workspace)) != LINREC_OK)
            return st;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    hipStream_t s = (hipStream_t)stream;
    if (d->T == 0)
        return pass(d, h_in, h_out, s);
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_DIAG_FWD, s, [&] {
        return launch_diag_fwd(d, g, x, h_in, h, h_out, (float*)states, workspace, s);
    }));
    return LINREC_OK;
}

linrec_status linrec_diag_bwd(linrec_ctx* ctx, const linrec_diag_desc* d, linrec_tensor g, linrec_tensor x,
                              const void* states, linrec_tensor dh, const float* dh_out, linrec_tensor dg,
                              linrec_tensor dx, float* dh_in, void* workspace, void* stream)
{
    linrec_status st;
    if ((st = check_diag_desc(d)) != LINREC_OK || (st = check_state_ptr(dh_out, false)) != LINREC_OK ||
        (st = check_state_ptr(dh_in, true)) != LINREC_OK)
        return st;
    if (d->T > 0) {
        if ((st = check_diag_rows(d, g, d->dtype, false)) != LINREC_OK ||
            (st = check_diag_rows(d, x, d->dtype, false)) != LINREC_OK ||
            (st = check_diag_rows(d, dh, d->dtype, false)) != LINREC_OK ||
            (st = check_diag_rows(d, dg, d->out_dtype, true)) != LINREC_OK ||
            (st = check_diag_rows(d, dx, d->out_dtype, true)) != LINREC_OK ||
            (st = check_buffer(states)) != LINREC_OK)
            return st;
        if (d->T > SEG && (st = check_buffer(workspace)) != LINREC_OK)
            return st;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    hipStream_t s = (hipStream_t)stream;
    if (d->T == 0)
        return pass(d, dh_out, dh_in, s);
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_DIAG_BWD, s, [&] {
        return launch_diag_bwd(d, g, x, (const float*)states, dh, dh_out, dg, dx, dh_in, workspace, s);
    }));
    return LINREC_OK;
}

}  // extern "C"
