// diag.hip -- the elementwise gated recurrence (linrec_diag_fwd / _bwd):
//   h_t = a_t h_{t-1} + b_t,  a = exp(g),  b = x or (1 - a) x,
// one state per batch and channel.
//
// A token step is the affine map h -> a h + b, so 256 tokens (a segment) of a
// channel are one map (P, B) too.  A workgroup holds a segment of CH channels
// in registers: a lane owns one 16-byte vector of channels and R consecutive
// tokens (a run), so a load instruction reads 8 rows of 128 bytes.  Each run is
// folded to its map, the maps of the 32 runs are folded through LDS from the
// state that enters the segment, and the run is replayed from its entry.
// Longer pieces first reduce every segment to its map (diag_sum_kernel), fold
// the maps along the piece (diag_fold_kernel), then run the segments.
#include <hip/hip_runtime.h>

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

// 1 - exp(g): near 0 the difference would cancel (relative error 2^-24 / |g|),
// so the series takes over there; its first dropped term, g^7 / 8!, is below
// 2^-28 of the sum at |g| = 1/4.
__device__ __forceinline__ float one_minus_exp(float g, float a)
{
    const float s = 1.f + g * (1.f / 2 + g * (1.f / 6 + g * (1.f / 24 + g * (1.f / 120 + g * (1.f / 720 + g * (1.f / 5040))))));
    return fabsf(g) < 0.25f ? -g * s : 1.f - a;
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

template <typename T>
__device__ __forceinline__ void load_run(u32x4 (&v)[RUN], const T* base, int64_t st, int t0, int nt, int nc)
{
#pragma unroll
    for (int r = 0; r < RUN; ++r)
        v[r] = r < nt ? load_vec(base + (int64_t)(t0 + r) * st, nc) : u32x4{0u, 0u, 0u, 0u};
}

// A token that does not exist has g = 0 and x = 0 (dh = 0): the identity.

// Forward.  NRUN = 32: 256 threads, a segment.  NRUN = 1: 64 threads, up to 8
// tokens of 64 vectors of channels (generation: no LDS, no barrier).
template <typename T, typename OT, bool MIX, int NRUN>
__global__ __launch_bounds__(NRUN == 1 ? 64 : 256) void diag_fwd_kernel(
    Act<const T> g, Act<const T> x, Act<OT> h, const float* h_in, float* states, float* h_out, int T_,
    int C, int ncg, int nseg)
{
    constexpr int N = Vec<T>::N, NT = NRUN == 1 ? 64 : 256, CH = NT / NRUN * N;
    const int cg = blockIdx.x % ncg, seg = blockIdx.x / ncg, b = blockIdx.y;
    const Place<T, NRUN> p(cg, seg, T_, C, NT);
    u32x4 gv[RUN], xv[RUN];
    load_run(gv, g.ptr + b * g.sb + p.c0, g.st, p.t0, p.nt, p.nc);
    load_run(xv, x.ptr + b * x.sb + p.c0, x.st, p.t0, p.nt, p.nc);
    float hc[N];
    if constexpr (NRUN == 1) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            hc[j] = h_in && j < p.nc ? h_in[(int64_t)b * C + p.c0 + j] : 0.f;
            if (j < p.nc)
                states[(int64_t)b * C + p.c0 + j] = hc[j];
        }
    } else {
        __shared__ float sP[NRUN][CH], sB[NRUN][CH];
        float P[N], B[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            P[j] = 1.f;
            B[j] = 0.f;
        }
#pragma unroll
        for (int r = 0; r < RUN; ++r)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float gg = vec_get<T>(gv[r], j), a = __expf(gg);
                P[j] *= a;
                B[j] = a * B[j] + added<MIX>(gg, a, vec_get<T>(xv[r], j));
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
            float s;
            if (nseg == 1) {
                s = h_in ? h_in[(int64_t)b * C + c] : 0.f;
                states[(int64_t)b * C + c] = s;
            } else {
                s = states[((int64_t)b * nseg + seg) * C + c];
            }
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
    }
    OT* hp = h.ptr + b * h.sb + p.c0;
#pragma unroll
    for (int r = 0; r < RUN; ++r) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float gg = vec_get<T>(gv[r], j), a = __expf(gg);
            hc[j] = a * hc[j] + added<MIX>(gg, a, vec_get<T>(xv[r], j));
        }
        if (r < p.nt)
            store_vec<OT, N>(hp + (int64_t)(p.t0 + r) * h.st, hc, p.nc);
    }
    if constexpr (NRUN == 1) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j < p.nc)
                h_out[(int64_t)b * C + p.c0 + j] = hc[j];
    }
}

// Backward of one segment: the states before each token from the state that
// enters the segment, then, from the right, with R the gradient arriving at h_t
// from later tokens:  G = dh + R,  dx = G or (1 - a) G,  dg = a G (h_{t-1} - [mix] x),
// R <- a G.  A run is also the map R -> P R + Q from its right end to its left.
template <typename T, typename OT, bool MIX>
__global__ __launch_bounds__(256) void diag_bwd_kernel(
    Act<const T> g, Act<const T> x, Act<const T> dh, Act<OT> dg, Act<OT> dx, const float* states,
    const float* right, const float* dh_out, float* dh_in, int T_, int C, int ncg, int nseg)
{
    constexpr int N = Vec<T>::N, NT = 256, NRUN = SEG / RUN, CH = NT / NRUN * N;
    __shared__ float sP[NRUN][CH], sB[NRUN][CH], sQ[NRUN][CH];
    const int cg = blockIdx.x % ncg, seg = blockIdx.x / ncg, b = blockIdx.y;
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
        float R = nseg == 1 ? (dh_out ? dh_out[at] : 0.f)
                            : right[((int64_t)b * nseg + seg) * C + cg * CH + cc];
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
        float s = sB[p.run][cl + j], R = sQ[p.run][cl + j];
        float hp[RUN];
#pragma unroll
        for (int r = 0; r < RUN; ++r) {
            const float gg = vec_get<T>(gv[r], j), a = __expf(gg);
            hp[r] = s;
            s = a * s + added<MIX>(gg, a, vec_get<T>(xv[r], j));
        }
#pragma unroll
        for (int r = RUN - 1; r >= 0; --r) {
            const float gg = vec_get<T>(gv[r], j), a = __expf(gg), xx = vec_get<T>(xv[r], j);
            const float G = vec_get<T>(dv[r], j) + R;
            R = a * G;
            outg[r][j & 1] = R * (MIX ? hp[r] - xx : hp[r]);
            outx[r][j & 1] = MIX ? one_minus_exp(gg, a) * G : G;
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

// A segment's map.  REV: y = dh, the map R -> P R + Q (see diag_bwd_kernel);
// else y = x, the map h -> P h + B.
template <typename T, bool MIX, bool REV>
__global__ __launch_bounds__(256) void diag_sum_kernel(Act<const T> g, Act<const T> y, float* prod,
                                                       float* sum, int T_, int C, int ncg, int nseg)
{
    constexpr int N = Vec<T>::N, NT = 256, NRUN = SEG / RUN, CH = NT / NRUN * N;
    __shared__ float sP[NRUN][CH], sB[NRUN][CH];
    const int cg = blockIdx.x % ncg, seg = blockIdx.x / ncg, b = blockIdx.y;
    const Place<T, NRUN> p(cg, seg, T_, C, NT);
    u32x4 gv[RUN], yv[RUN];
    load_run(gv, g.ptr + b * g.sb + p.c0, g.st, p.t0, p.nt, p.nc);
    load_run(yv, y.ptr + b * y.sb + p.c0, y.st, p.t0, p.nt, p.nc);
    const int cl = (threadIdx.x % (NT / NRUN)) * N;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        float P = 1.f, B = 0.f;
#pragma unroll
        for (int r = 0; r < RUN; ++r) {
            const float gg = vec_get<T>(gv[r], j), a = __expf(gg), yy = vec_get<T>(yv[r], j);
            if constexpr (REV) {
                B += P * (a * yy);
                P *= a;
            } else {
                P *= a;
                B = a * B + added<MIX>(gg, a, yy);
            }
        }
        sP[p.run][cl + j] = P;
        sB[p.run][cl + j] = B;
    }
    __syncthreads();
    const int c = cg * CH + threadIdx.x;
    if (threadIdx.x < CH && c < C) {
        float P = 1.f, B = 0.f;
#pragma unroll 8
        for (int i = 0; i < NRUN; ++i) {
            const int k = REV ? NRUN - 1 - i : i;
            B = sP[k][threadIdx.x] * B + sB[k][threadIdx.x];
            P *= sP[k][threadIdx.x];
        }
        const int64_t at = ((int64_t)b * nseg + seg) * C + c;
        prod[at] = P;
        sum[at] = B;
    }
}

// Fold of the segments' maps along the piece, from `in` (NULL: zeros); each
// segment's sum is replaced by the value that enters it (REV: from the right).
template <bool REV>
__global__ __launch_bounds__(64) void diag_fold_kernel(const float* prod, float* sum, const float* in,
                                                       int C, int nseg)
{
    const int c = blockIdx.x * 64 + threadIdx.x, b = blockIdx.y;
    if (c >= C)
        return;
    float s = in ? in[(int64_t)b * C + c] : 0.f;
    const int64_t base = (int64_t)b * nseg * C + c;
    constexpr int U = 16;
    for (int i0 = 0; i0 < nseg; i0 += U) {
        float P[U], B[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = min(i0 + u, nseg - 1), k = REV ? nseg - 1 - i : i;
            P[u] = prod[base + (int64_t)k * C];
            B[u] = sum[base + (int64_t)k * C];
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + u < nseg) {
                const int k = REV ? nseg - 1 - (i0 + u) : i0 + u;
                sum[base + (int64_t)k * C] = s;
                s = P[u] * s + B[u];
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
    if (nseg_of(d->T) * ncg * 256 > 0xffffffffll)
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

hipError_t launch_diag_fwd(const linrec_diag_desc* d, const linrec_tensor& g, const linrec_tensor& x,
                           const float* h_in, const linrec_tensor& h, float* h_out, float* states,
                           float* prod, hipStream_t s)
{
    return dispatch(d, [&](auto t, auto o, auto mix) {
        using T = decltype(t);
        using OT = decltype(o);
        constexpr bool MIX = decltype(mix)::value;
        const int cpg = channels_per_group(d->dtype), ncg = (d->C + cpg - 1) / cpg;
        const int nseg = (int)nseg_of(d->T);
        if (d->T <= RUN) {
            const int n = (d->C + 64 * Vec<T>::N - 1) / (64 * Vec<T>::N);
            launch_kernel(diag_fwd_kernel<T, OT, MIX, 1>, dim3(n, d->B), dim3(64), s, cact<T>(g),
                          cact<T>(x), mact<OT>(h), h_in, states, h_out, d->T, d->C, n, 1);
            return hipGetLastError();
        }
        if (nseg > 1) {
            launch_kernel(diag_sum_kernel<T, MIX, false>, dim3(ncg * nseg, d->B), dim3(256), s, cact<T>(g),
                          cact<T>(x), prod, states, d->T, d->C, ncg, nseg);
            launch_kernel(diag_fold_kernel<false>, dim3((d->C + 63) / 64, d->B), dim3(64), s,
                          (const float*)prod, states, h_in, d->C, nseg);
        }
        launch_kernel(diag_fwd_kernel<T, OT, MIX, SEG / RUN>, dim3(ncg * nseg, d->B), dim3(256), s,
                      cact<T>(g), cact<T>(x), mact<OT>(h), h_in, states, h_out, d->T, d->C, ncg, nseg);
        return hipGetLastError();
    });
}

hipError_t launch_diag_bwd(const linrec_diag_desc* d, const linrec_tensor& g, const linrec_tensor& x,
                           const float* states, const linrec_tensor& dh, const float* dh_out,
                           const linrec_tensor& dg, const linrec_tensor& dx, float* dh_in, float* prod,
                           float* sum, hipStream_t s)
{
    return dispatch(d, [&](auto t, auto o, auto mix) {
        using T = decltype(t);
        using OT = decltype(o);
        constexpr bool MIX = decltype(mix)::value;
        const int cpg = channels_per_group(d->dtype), ncg = (d->C + cpg - 1) / cpg;
        const int nseg = (int)nseg_of(d->T);
        if (nseg > 1) {
            launch_kernel(diag_sum_kernel<T, MIX, true>, dim3(ncg * nseg, d->B), dim3(256), s, cact<T>(g),
                          cact<T>(dh), prod, sum, d->T, d->C, ncg, nseg);
            launch_kernel(diag_fold_kernel<true>, dim3((d->C + 63) / 64, d->B), dim3(64), s,
                          (const float*)prod, sum, dh_out, d->C, nseg);
        }
        launch_kernel(diag_bwd_kernel<T, OT, MIX>, dim3(ncg * nseg, d->B), dim3(256), s, cact<T>(g),
                      cact<T>(x), cact<T>(dh), mact<OT>(dg), mact<OT>(dx), states, (const float*)sum,
                      dh_out, dh_in, d->T, d->C, ncg, nseg);
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
    return d && d->T <= SEG ? 0 : 2 * linrec_diag_states_bytes(d);
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
        return launch_diag_fwd(d, g, x, h_in, h, h_out, (float*)states, (float*)workspace, s);
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
    float* prod = (float*)workspace;
    float* sum = workspace ? prod + (size_t)d->B * nseg_of(d->T) * d->C : nullptr;
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_DIAG_BWD, s, [&] {
        return launch_diag_bwd(d, g, x, (const float*)states, dh, dh_out, dg, dx, dh_in, prod, sum, s);
    }));
    return LINREC_OK;
}

}  // extern "C"
