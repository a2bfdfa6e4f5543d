// conv.hip -- the short causal convolution (linrec_conv_fwd / _bwd / _step):
//   p_t = bias + sum_k w_k x_{t-K+1+k},  y = p or silu(p) = p / (1 + e^-p),
// K = 2..4 taps a channel, the K-1 inputs before the piece carried in fp32.
//
// Bound by HBM: 2 elements a token and channel forward, 3 backward.  65536 x 2048
// bf16, 4 taps, silu: 98-101 us forward (5.4 TB/s: a part comes from the last-level
// cache), 188 us backward (4.3 TB/s; its 34 vector instructions a token and channel
// are issued in 70% of the cycles, three waves a SIMD); 3 x 4099 x 1000 fp32, 3 taps,
// 19 and 34 us (5.2 and 4.3 TB/s).
// A lane owns a vector of channels and a run of consecutive tokens, and slides the
// last K-1 inputs through registers, so a run reads K-1 tokens that its neighbour
// reads too and nothing else twice.  The backward slides the K-1 unfinished sums
//   dx_t = sum_k w_k dp_{t+K-1-k},  dp = dy act'(p)
// the same way, with p formed again from x, and adds dp_t x_{t-K+1+k} into the
// taps' gradients, summed over a run in registers (at most 64 tokens), over a workgroup
// through LDS and over workgroups by a second kernel, in a fixed order.  The last two
// add in 64 bits, which costs nothing there (both wait for memory); a run's sums would
// take 40 registers more.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ctx.hpp"
#include "device.hpp"
#include "rows.hpp"

namespace linrec {
namespace {

constexpr int NT = 256;

// N packed values of a token row.
template <typename T, int N>
struct Packed {
    static constexpr int W = N * sizeof(T) / 4;
    typedef unsigned words __attribute__((ext_vector_type(W)));
    words v;
    // channels past n are not read and come as zeros
    __device__ __forceinline__ void load(const T* p, int n)
    {
        if (n >= N) {
            v = *reinterpret_cast<const words*>(p);
            return;
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
            v[i] = 0u;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < n) {
                if constexpr (sizeof(T) == 2)
                    v[j / 2] |= (unsigned)reinterpret_cast<const unsigned short*>(p)[j] << (16 * (j & 1));
                else
                    v[j] = reinterpret_cast<const unsigned*>(p)[j];
            }
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < W; ++i)
            v[i] = 0u;
    }
    __device__ __forceinline__ float operator[](int j) const
    {
        if constexpr (sizeof(T) == 2)
            return __uint_as_float((j & 1) ? v[j / 2] & 0xffff0000u : v[j / 2] << 16);
        else
            return __uint_as_float(v[j]);
    }
};

// Taps and bias of N channels.
template <int N, int K>
__device__ __forceinline__ void load_taps(float (&w)[K][N], float (&bias)[N], const float* wp, const float* bp, int c0, int nc)
{
    load_floats<N>(bias, bp ? bp + c0 : nullptr, nc);
    wp += (int64_t)c0 * K;
    if (nc >= N) {   // K N floats in a row
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < K; ++k)
                w[k][j] = wp[j * K + k];
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int k = 0; k < K; ++k)
                w[k][j] = j < nc ? wp[j * K + k] : 0.f;
    }
}

// Where a lane's run lies: `shift` = log2 of the lanes side by side over the channels.
struct Run {
    int c0, nc, t0, n, b, tg;   // first channel, channels that exist, first token, tokens of the sequence, sequence, group of runs
    __device__ __forceinline__ Run(const int* n_new, int T_, int C, int ncg, int shift, int vec, int run)
    {
        const int lane = threadIdx.x & ((1 << shift) - 1);
        c0 = (((int)(blockIdx.x % ncg) << shift) + lane) * vec;
        nc = C - c0;
        tg = blockIdx.x / ncg;
        // (a run behind the largest T starts there: it has no tokens)
        t0 = (int)min(((int64_t)tg * (NT >> shift) + (threadIdx.x >> shift)) * run, (int64_t)LINREC_MAX_T);
        b = blockIdx.y;
        n = tokens_of(n_new, b, T_);
    }
};

// The K-1 inputs before token t0 of a run: of the piece, or (t0 == 0) of the state.
template <typename T, int N, int K>
__device__ __forceinline__ void load_window(float (&win)[K - 1][N], const T* xp, int64_t st, const float* state, int t0, int C, int nc)
{
#pragma unroll
    for (int m = 0; m < K - 1; ++m) {
        if (t0 == 0) {
            load_floats<N>(win[m], state ? state + (int64_t)m * C : nullptr, nc);
        } else {
            Packed<T, N> v;
            v.load(xp + (int64_t)(t0 - (K - 1) + m) * st, nc);
#pragma unroll
            for (int j = 0; j < N; ++j)
                win[m][j] = v[j];
        }
    }
}

template <typename T, typename OT, int K, bool ACT, int RUN>
__global__ __launch_bounds__(NT) void conv_fwd_kernel(Act<const T> x, const float* w, const float* bias,
                                                      const float* state_in, const int* n_new, Act<OT> y,
                                                      float* state_out, int T_, int C, int ncg, int shift)
{
    constexpr int N = Vec<T>::N, R = 8;
    const Run p(n_new, T_, C, ncg, shift, N, RUN);
    if (p.nc <= 0 || (p.t0 >= p.n && p.t0 > 0))
        return;
    const T* xp = x.ptr + p.b * x.sb + p.c0;
    const int64_t carry = (int64_t)p.b * (K - 1) * C + p.c0;
    float wk[K][N], bk[N], win[K - 1][N];
    load_window<T, N, K>(win, xp, x.st, state_in ? state_in + carry : nullptr, p.t0, C, p.nc);
    load_taps<N, K>(wk, bk, w, bias, p.c0, p.nc);
    if (p.t0 == 0) {
        // the state that leaves, by the lane that has read the one that enters (they may be one memory)
        for (int m = 0; m < K - 1; ++m) {
            const int at = p.n - (K - 1) + m;
            float s[N];
            if (at >= 0) {
                Packed<T, N> v;
                v.load(xp + (int64_t)at * x.st, p.nc);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    s[j] = v[j];
            } else {
#pragma unroll
                for (int i = 0; i < K - 1; ++i)
                    if (i == at + K - 1)
#pragma unroll
                        for (int j = 0; j < N; ++j)
                            s[j] = win[i][j];
            }
            store_floats<N>(state_out + carry + (int64_t)m * C, s, p.nc);
        }
    }
    OT* yp = y.ptr + p.b * y.sb + p.c0;
    const int end = min(p.n, p.t0 + RUN);
    for (int t = p.t0; t < end; t += R) {
        Packed<T, N> v[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (t + r < end)
                v[r].load(xp + (int64_t)(t + r) * x.st, p.nc);
            else
                v[r].clear();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float out[N];
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float in = v[r][j];
                float s = bk[j];
#pragma unroll
                for (int m = 0; m < K - 1; ++m)
                    s = __builtin_fmaf(wk[m][j], win[m][j], s);
                s = __builtin_fmaf(wk[K - 1][j], in, s);
#pragma unroll
                for (int m = 0; m < K - 2; ++m)
                    win[m][j] = win[m + 1][j];
                win[K - 2][j] = in;
                out[j] = ACT ? s * sigmoid(s) : s;
            }
            if (t + r < end)
                store_vec<OT, N>(yp + (int64_t)(t + r) * y.st, out, p.nc);
        }
    }
}

// Backward.  A run sees dp of its own tokens and of the K-1 behind them; the
// gradient of the K-1 inputs before the piece goes to the workspace (the caller's
// dstate_in may be its dstate_out, which other workgroups still read).  Vectors of 4
// channels (8 bytes of bf16): with 8, the taps, their gradients and the sums take
// twice 68 registers.  4 tokens in flight and 4 loaded ahead: 188 us; 8 in flight 263
// (two waves a SIMD), 4 without loading ahead 195.
template <typename T, typename OT, int K, bool ACT, int RUN>
__global__ __launch_bounds__(NT, sizeof(T) == 4 && K == 4 ? 2 : 3) void conv_bwd_kernel(Act<const T> x, const float* w, const float* bias,
                                                      const float* state_in, const int* n_new, Act<const T> dy,
                                                      const float* dstate_out, Act<OT> dx, float* dstate, float* part,
                                                      int T_, int C, int ncg, int shift)
{
    constexpr int N = 4, R = 4;
    __shared__ float sums[NT][(K + 1) * N + 1];
    const Run p(n_new, T_, C, ncg, shift, N, RUN);
    float dw[K][N], db[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        db[j] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            dw[k][j] = 0.f;
    }
    if (p.nc > 0 && (p.t0 < p.n || p.t0 == 0)) {
        const T* xp = x.ptr + p.b * x.sb + p.c0;
        const T* dp = dy.ptr + p.b * dy.sb + p.c0;
        OT* op = dx.ptr + p.b * dx.sb + p.c0;
        const int64_t carry = (int64_t)p.b * (K - 1) * C + p.c0;
        float wk[K][N], bk[N], win[K - 1][N], acc[K][N];
        load_window<T, N, K>(win, xp, x.st, state_in ? state_in + carry : nullptr, p.t0, C, p.nc);
        load_taps<N, K>(wk, bk, w, bias, p.c0, p.nc);
#pragma unroll
        for (int m = 0; m < K; ++m)
#pragma unroll
            for (int j = 0; j < N; ++j)
                acc[m][j] = 0.f;
        // token i's dp into the K sums that it is part of, and (own: i is of this run) the taps' gradients
        auto add = [&](const Packed<T, N>& xv, const Packed<T, N>& dv, bool own, bool live) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float in = xv[j];
                float s = bk[j];
#pragma unroll
                for (int m = 0; m < K - 1; ++m)
                    s = __builtin_fmaf(wk[m][j], win[m][j], s);
                s = __builtin_fmaf(wk[K - 1][j], in, s);
                float d = dv[j];
                if constexpr (ACT) {
                    const float q = sigmoid(s);
                    d *= __builtin_fmaf(s * q, 1.f - q, q);
                }
                d = live ? d : 0.f;   // whatever the inputs behind the last token's are
#pragma unroll
                for (int m = 0; m < K; ++m)
                    acc[m][j] = __builtin_fmaf(wk[m][j], d, acc[m][j]);
                if (own) {
                    db[j] += d;
#pragma unroll
                    for (int m = 0; m < K - 1; ++m)
                        dw[m][j] = __builtin_fmaf(d, win[m][j], dw[m][j]);
                    dw[K - 1][j] = __builtin_fmaf(d, in, dw[K - 1][j]);
                }
#pragma unroll
                for (int m = 0; m < K - 2; ++m)
                    win[m][j] = win[m + 1][j];
                win[K - 2][j] = in;
            }
        };
        auto shift_sums = [&] {
#pragma unroll
            for (int j = 0; j < N; ++j) {
#pragma unroll
                for (int m = 0; m < K - 1; ++m)
                    acc[m][j] = acc[m + 1][j];
                acc[K - 1][j] = 0.f;
            }
        };
        // token i finishes the sum of token i - (K-1), which may be of the run before, of the state, or one of the last
        auto token = [&](int i, const Packed<T, N>& xv, const Packed<T, N>& dv, bool own, bool live) {
            add(xv, dv, own, live);
            const int at = i - (K - 1);
            if (at < p.n && (at >= p.t0 || p.t0 == 0)) {
                if (dstate_out && at >= p.n - (K - 1)) {
                    float e[N];
                    load_floats<N>(e, dstate_out + carry + (int64_t)(at - (p.n - (K - 1))) * C, p.nc);
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        acc[0][j] += e[j];
                }
                if (at >= 0)
                    store_vec<OT, N>(op + (int64_t)at * dx.st, acc[0], p.nc);
                else
                    store_floats<N>(dstate + carry + (int64_t)(at + K - 1) * C, acc[0], p.nc);
            }
            shift_sums();
        };
        const int end = min(p.n, p.t0 + RUN);
        Packed<T, N> xn[R], dn[R];   // R tokens, loaded while those before are added
        auto load = [&](int t) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (t + r < end) {
                    xn[r].load(xp + (int64_t)(t + r) * x.st, p.nc);
                    dn[r].load(dp + (int64_t)(t + r) * dy.st, p.nc);
                } else {
                    xn[r].clear();
                    dn[r].clear();
                }
        };
        load(p.t0);
        for (int t = p.t0; t < end; t += R) {
            Packed<T, N> xv[R], dv[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                xv[r] = xn[r];
                dv[r] = dn[r];
            }
            load(t + R);
            if (t > p.t0 && t + R <= end) {   // inside the run: the sums of tokens t - (K-1) ..
                static_assert(R >= K - 1, "of the run");
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    add(xv[r], dv[r], true, true);
                    store_vec<OT, N>(op + (int64_t)(t + r - (K - 1)) * dx.st, acc[0], p.nc);
                    shift_sums();
                }
            } else {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (t + r < end)
                        token(t + r, xv[r], dv[r], true, true);
            }
        }
#pragma unroll
        for (int r = 0; r < K - 1; ++r) {   // the tokens behind: of the next run, or none
            const int i = end + r;
            Packed<T, N> xv, dv;
            xv.clear();
            dv.clear();
            if (i < p.n) {
                xv.load(xp + (int64_t)i * x.st, p.nc);
                dv.load(dp + (int64_t)i * dy.st, p.nc);
            }
            token(i, xv, dv, false, i < p.n);
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            sums[threadIdx.x][k * N + j] = dw[k][j];
        sums[threadIdx.x][K * N + j] = db[j];
    }
    __syncthreads();
    // part: [sequence, group of runs][K + 1][C]
    const int lanes = 1 << shift;
    float* out = part + ((int64_t)p.b * (gridDim.x / ncg) + p.tg) * (K + 1) * C;
    for (int i = threadIdx.x; i < lanes * (K + 1) * N; i += NT) {
        const int k = i / (lanes * N), col = i % (lanes * N), c = ((int)(blockIdx.x % ncg) << shift) * N + col;
        if (c < C) {
            double s = 0.0;
            for (int r = 0; r < NT >> shift; ++r)
                s += sums[(r << shift) + col / N][k * N + col % N];
            out[(int64_t)k * C + c] = (float)s;
        }
    }
}

// The taps' and the bias's gradients from the workgroups' sums, 64 columns and
// 16 slices of the sums a workgroup; the last workgroups copy dstate_in.
template <int K>
__global__ __launch_bounds__(1024) void conv_finish_kernel(const float* part, int64_t parts, float* dw, float* dbias,
                                                           const float* dstate, float* dstate_in, int64_t nstate, int C,
                                                           int cols)
{
    __shared__ double sums[16][64];
    if ((int)blockIdx.x >= cols) {
        for (int64_t i = (blockIdx.x - cols) * 1024ll + threadIdx.x; i < nstate; i += (gridDim.x - cols) * 1024ll)
            dstate_in[i] = dstate[i];
        return;
    }
    const int col = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const int64_t i = blockIdx.x * 64ll + col, ld = (int64_t)(K + 1) * C;
    double s = 0.0;
    if (i < ld)
#pragma unroll 8
        for (int64_t q = slice; q < parts; q += 16)
            s += part[q * ld + i];
    sums[slice][col] = s;
    __syncthreads();
    if (slice == 0 && i < ld) {
        for (int q = 1; q < 16; ++q)
            s += sums[q][col];
        const int k = (int)(i / C), c = (int)(i % C);
        if (k < K)
            dw[(int64_t)c * K + k] = (float)s;
        else if (dbias)
            dbias[c] = (float)s;
    }
}

// Token by token on the states of a pool, one lane a vector of channels.
template <typename T, typename OT, int K, bool ACT>
__global__ __launch_bounds__(64) void conv_step_kernel(Act<const T> x, const float* w, const float* bias, float* S,
                                                       const int* slots, int nslots, Act<OT> y, int T_, int C)
{
    constexpr int N = 4;
    const int b = blockIdx.y, c0 = (blockIdx.x * 64 + threadIdx.x) * N, nc = C - c0;
    OT* yp = y.ptr + b * y.sb + c0;
    int slot = b;
    if (slots) {
        slot = slots[b];
        int skip = slot < 0 || slot >= nslots;
        for (int i = threadIdx.x; i < b; i += 64)
            skip |= slots[i] == slot;
        if (__any(skip)) {
            if (nc > 0) {
                const float none[N] = {};
                for (int t = 0; t < T_; ++t)
                    store_vec<OT, N>(yp + (int64_t)t * y.st, none, nc);
            }
            return;
        }
    }
    if (nc <= 0)
        return;
    float* Sp = S + (int64_t)slot * (K - 1) * C + c0;
    const T* xp = x.ptr + b * x.sb + c0;
    float wk[K][N], bk[N], win[K - 1][N];
    load_window<T, N, K>(win, xp, x.st, Sp, 0, C, nc);
    load_taps<N, K>(wk, bk, w, bias, c0, nc);
    for (int t = 0; t < T_; ++t) {
        Packed<T, N> v;
        v.load(xp + (int64_t)t * x.st, nc);
        float out[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float s = bk[j];
#pragma unroll
            for (int m = 0; m < K - 1; ++m)
                s = __builtin_fmaf(wk[m][j], win[m][j], s);
            s = __builtin_fmaf(wk[K - 1][j], v[j], s);
#pragma unroll
            for (int m = 0; m < K - 2; ++m)
                win[m][j] = win[m + 1][j];
            win[K - 2][j] = v[j];
            out[j] = ACT ? s * sigmoid(s) : s;
        }
        store_vec<OT, N>(yp + (int64_t)t * y.st, out, nc);
    }
#pragma unroll
    for (int m = 0; m < K - 1; ++m)
        store_floats<N>(Sp + (int64_t)m * C, win[m], nc);
}

// ---- host ------------------------------------------------------------------

// The runs of a launch: `vec` channels a lane.  Long runs read less twice; they are
// taken from two waves a SIMD on (4 x 4096 x 2048 bf16 forward, as many: runs of 32
// tokens 27.5 us, of 8 30.3; 65536 x 2048 backward: of 64 199 us, of 32 215, of 16 251).
struct Plan {
    int shift, run, ncg, ntg;
    Plan(const linrec_conv_desc* d, int vec, int longest)
    {
        const int vecs = (d->C + vec - 1) / vec;
        shift = 0;
        while (shift < 6 && (1 << shift) < vecs)
            ++shift;
        ncg = (vecs + (1 << shift) - 1) >> shift;
        const int64_t lanes = (int64_t)d->B * ncg << shift;
        run = lanes * (((int64_t)d->T + longest - 1) / longest) >= 2048 * 64 ? longest : 8;
        const int span = run * (NT >> shift);
        ntg = (int)((d->T + (int64_t)span - 1) / span);
    }
    int64_t blocks() const { return (int64_t)ncg * ntg; }
    // a launch holds at most 2^32 - 1 threads along x
    bool fits() const { return blocks() * NT <= 0xffffffffll; }
};

constexpr int BWD_VEC = 4, FWD_RUN = 32, BWD_RUN = 64;

linrec_status check_conv_desc(const linrec_conv_desc* d)
{
    if (!d)
        return LINREC_E_NULL;
    if ((d->dtype != LINREC_BF16 && d->dtype != LINREC_F32) ||
        (d->out_dtype != LINREC_BF16 && d->out_dtype != LINREC_F32) ||
        (d->dtype == LINREC_F32 && d->out_dtype != LINREC_F32))
        return LINREC_E_DTYPE;
    if (d->B < 1 || d->B > 32767 || d->C < 1 || d->C > (1 << 20) || d->T < 0 || d->T > LINREC_MAX_T || d->K < 2 || d->K > 4)
        return LINREC_E_SHAPE;
    if (d->T > 0 && !Plan(d, BWD_VEC, BWD_RUN).fits())
        return LINREC_E_SHAPE;
    if (d->act != LINREC_ACT_NONE && d->act != LINREC_ACT_SILU)
        return LINREC_E_LAYOUT;
    return LINREC_OK;
}

// The forward's own launch: of fp32 it has twice the backward's workgroups (runs half as long).
linrec_status check_fwd_desc(const linrec_conv_desc* d)
{
    const linrec_status st = check_conv_desc(d);
    if (st != LINREC_OK || d->T == 0)
        return st;
    return Plan(d, d->dtype == LINREC_F32 ? Vec<float>::N : Vec<bf16>::N, FWD_RUN).fits() ? LINREC_OK : LINREC_E_SHAPE;
}

linrec_status check_taps(const float* w, const float* bias)
{
    if (!w)
        return LINREC_E_NULL;
    return aligned(w, 4) && aligned(bias, 4) ? LINREC_OK : LINREC_E_ALIGN;
}

// Calls f with (input type, output type, taps, activation) of the description.
template <typename F>
hipError_t dispatch(const linrec_conv_desc* d, F&& f)
{
    auto act = [&](auto t, auto o, auto k) {
        return d->act == LINREC_ACT_SILU ? f(t, o, k, std::true_type{}) : f(t, o, k, std::false_type{});
    };
    auto taps = [&](auto t, auto o) {
        if (d->K == 2)
            return act(t, o, std::integral_constant<int, 2>{});
        if (d->K == 3)
            return act(t, o, std::integral_constant<int, 3>{});
        return act(t, o, std::integral_constant<int, 4>{});
    };
    if (d->dtype == LINREC_F32)
        return taps(float{}, float{});
    return d->out_dtype == LINREC_F32 ? taps(bf16{}, float{}) : taps(bf16{}, bf16{});
}

int64_t state_floats(const linrec_conv_desc* d) { return (int64_t)d->B * (d->K - 1) * d->C; }

}  // namespace
}  // namespace linrec

using namespace linrec;

extern "C" {

size_t linrec_conv_bwd_workspace_bytes(const linrec_conv_desc* d)
{
    if (check_conv_desc(d) != LINREC_OK || d->T == 0)
        return 0;
    const Plan p(d, BWD_VEC, BWD_RUN);
    return (size_t)(round4(state_floats(d)) + round4((int64_t)d->B * p.ntg * (d->K + 1) * d->C)) * sizeof(float);
}

linrec_status linrec_conv_fwd(linrec_ctx* ctx, const linrec_conv_desc* d, linrec_tensor x, const float* w,
                              const float* bias, const float* state_in, const int32_t* n_new, linrec_tensor y,
                              float* state_out, void* stream)
{
    linrec_status st;
    if ((st = check_fwd_desc(d)) != LINREC_OK || (st = check_state_ptr(state_in, false)) != LINREC_OK ||
        (st = check_state_ptr(state_out, true)) != LINREC_OK)
        return st;
    if (d->T > 0) {
        if ((st = check_rows(d, x, d->dtype, false)) != LINREC_OK || (st = check_taps(w, bias)) != LINREC_OK ||
            (st = check_rows(d, y, d->out_dtype, true)) != LINREC_OK)
            return st;
        if (!aligned(n_new, 4))
            return LINREC_E_ALIGN;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    hipStream_t s = (hipStream_t)stream;
    if (d->T == 0)
        return pass_carry(state_in, state_out, state_floats(d), s);
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_CONV_FWD, s, [&] {
        return dispatch(d, [&](auto t, auto o, auto k, auto act) {
            using T = decltype(t);
            using OT = decltype(o);
            constexpr int K = decltype(k)::value;
            constexpr bool ACT = decltype(act)::value;
            const Plan p(d, Vec<T>::N, FWD_RUN);
            launch_kernel(p.run == FWD_RUN ? conv_fwd_kernel<T, OT, K, ACT, FWD_RUN> : conv_fwd_kernel<T, OT, K, ACT, 8>,
                          dim3((unsigned)p.blocks(), d->B), dim3(NT), s, cact<T>(x), w, bias, state_in, n_new, mact<OT>(y),
                          state_out, d->T, d->C, p.ncg, p.shift);
            return hipGetLastError();
        });
    }));
    return LINREC_OK;
}

linrec_status linrec_conv_bwd(linrec_ctx* ctx, const linrec_conv_desc* d, linrec_tensor x, const float* w,
                              const float* bias, const float* state_in, const int32_t* n_new, linrec_tensor dy,
                              const float* dstate_out, linrec_tensor dx, float* dw, float* dbias, float* dstate_in,
                              void* workspace, void* stream)
{
    linrec_status st;
    if ((st = check_conv_desc(d)) != LINREC_OK || (st = check_state_ptr(dstate_out, false)) != LINREC_OK ||
        (st = check_state_ptr(dstate_in, true)) != LINREC_OK || (st = check_state_ptr(dw, true)) != LINREC_OK ||
        (st = check_state_ptr(dbias, false)) != LINREC_OK)
        return st;
    if (d->T > 0) {
        if ((st = check_rows(d, x, d->dtype, false)) != LINREC_OK || (st = check_taps(w, bias)) != LINREC_OK ||
            (st = check_state_ptr(state_in, false)) != LINREC_OK ||
            (st = check_rows(d, dy, d->dtype, false)) != LINREC_OK ||
            (st = check_rows(d, dx, d->out_dtype, true)) != LINREC_OK || (st = check_buffer(workspace)) != LINREC_OK)
            return st;
        if (!aligned(n_new, 4))
            return LINREC_E_ALIGN;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    hipStream_t s = (hipStream_t)stream;
    if (d->T == 0) {
        LAUNCH(launch_carry_copy(nullptr, dw, (int64_t)d->C * d->K, s));
        if (dbias)
            LAUNCH(launch_carry_copy(nullptr, dbias, d->C, s));
        return pass_carry(dstate_out, dstate_in, state_floats(d), s);
    }
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_CONV_BWD, s, [&] {
        return dispatch(d, [&](auto t, auto o, auto k, auto act) {
            using T = decltype(t);
            using OT = decltype(o);
            constexpr int K = decltype(k)::value;
            constexpr bool ACT = decltype(act)::value;
            const Plan p(d, BWD_VEC, BWD_RUN);
            float* dstate = (float*)workspace;
            float* part = dstate + round4(state_floats(d));
            launch_kernel(p.run == BWD_RUN ? conv_bwd_kernel<T, OT, K, ACT, BWD_RUN> : conv_bwd_kernel<T, OT, K, ACT, 8>,
                          dim3((unsigned)p.blocks(), d->B), dim3(NT), s, cact<T>(x), w, bias, state_in, n_new, cact<T>(dy),
                          dstate_out, mact<OT>(dx), dstate, part, d->T, d->C, p.ncg, p.shift);
            const int cols = (int)(((int64_t)(K + 1) * d->C + 63) / 64);
            const int copies = (int)std::min<int64_t>((state_floats(d) + 1023) / 1024, 1024);
            launch_kernel(conv_finish_kernel<K>, dim3(cols + copies), dim3(1024), s, part, (int64_t)d->B * p.ntg, dw, dbias, dstate,
                          dstate_in, state_floats(d), d->C, cols);
            return hipGetLastError();
        });
    }));
    return LINREC_OK;
}

linrec_status linrec_conv_step(linrec_ctx* ctx, const linrec_conv_desc* d, linrec_tensor x, const float* w,
                               const float* bias, float* S, const int32_t* slots, int32_t nslots, linrec_tensor y,
                               void* stream)
{
    linrec_status st;
    if ((st = check_conv_desc(d)) != LINREC_OK)
        return st;
    if (d->T > 0) {
        if ((st = check_state_ptr(S, true)) != LINREC_OK)
            return st;
        if (nslots < 1 || (!slots && nslots < d->B))
            return LINREC_E_SHAPE;
        if ((st = check_rows(d, x, d->dtype, false)) != LINREC_OK || (st = check_taps(w, bias)) != LINREC_OK ||
            (st = check_rows(d, y, d->out_dtype, true)) != LINREC_OK)
            return st;
        if (!aligned(slots, 4))
            return LINREC_E_ALIGN;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    if (d->T == 0)
        return LINREC_OK;
    hipStream_t s = (hipStream_t)stream;
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_CONV_STEP, s, [&] {
        return dispatch(d, [&](auto t, auto o, auto k, auto act) {
            using T = decltype(t);
            using OT = decltype(o);
            launch_kernel(conv_step_kernel<T, OT, decltype(k)::value, decltype(act)::value>,
                          dim3((d->C + 255) / 256, d->B), dim3(64), s, cact<T>(x), w, bias, S, slots, nslots, mact<OT>(y),
                          d->T, d->C);
            return hipGetLastError();
        });
    }));
    return LINREC_OK;
}

}  // extern "C"
