// kv_append.hip -- appending keys and values to the paged 8-bit cache, with the
// rotation by position applied on the way (linrec_kv_append).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "kv.hpp"

namespace linrec {
namespace {

struct AppendArgs {
    KvCache c;
    Act<const bf16> k, v, q;
    Act<bf16> q_out;
    const int* past;
    const int* n_new;
    const double* freq;
    const unsigned long long* owner;   // by page: the first touched block that has it; NULL: each block looks itself
    int B, T, Hq, half, nblk;   // half: rotated pairs; nblk: pages a sequence may touch
    int qshift;                 // queries: 1 << qshift tokens a workgroup
    bool inter;
};

// cos and sin of position * freq.  The product and its reduction to a fraction
// of a turn are fp64: at position 2^20 an fp32 angle would be off by 2^-5 rad.
__device__ __forceinline__ void turn(int64_t pos, double freq, float& c, float& s)
{
    const double t = (double)pos * freq * 0.15915494309189535;   // 1 / (2 pi)
    sincospif((float)(2.0 * (t - rint(t))), &s, &c);
}

// A row of D features is handled in units of 16: two 8-vectors that the rotation
// keeps among themselves.  Half-split pairs (i, i + half): the first half / 8
// units are vectors (u, u + half / 8); every other unit is (2 u, 2 u + 1).
__device__ __forceinline__ void unit_vectors(int u, int half, bool inter, int& v0, int& v1)
{
    const bool split = !inter && u < half / 8;
    v0 = split ? u : 2 * u;
    v1 = split ? u + half / 8 : 2 * u + 1;
}

// The 8 pairs of a rotated unit, cosines and sines given per pair.
template <typename CosSin>
__device__ __forceinline__ void rotate_unit(float (&y)[16], int u, int half, bool inter, CosSin cs)
{
    if (u >= half / 8)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // split: (8 u + i, that + half) is pair 8 u + i; interleaved: (16 u + 2 i, + 1) is pair 8 u + i
        const int a = inter ? 2 * i : i, b = inter ? 2 * i + 1 : 8 + i;
        float c, s;
        cs(8 * u + i, c, s);
        const float p = y[a], q = y[b];
        y[a] = p * c - q * s;
        y[b] = q * c + p * s;
    }
}

struct Unit {
    bf16x8 a, b;
};

__device__ __forceinline__ Unit load_unit(const bf16* row, int v0, int v1)
{
    return Unit{*reinterpret_cast<const bf16x8*>(row + 8 * v0), *reinterpret_cast<const bf16x8*>(row + 8 * v1)};
}

__device__ __forceinline__ void widen(float (&y)[16], const Unit& u)
{
    const bf16x8 a = u.a, b = u.b;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        y[i] = (float)a[i];
        y[8 + i] = (float)b[i];
    }
}

// The least power of two s with amax <= 448 s (448 = 1.75 * 2^8 is the largest
// e4m3 value), not below 2^-100, from the bits of amax.
__device__ __forceinline__ float scale_of(float amax)
{
    const unsigned u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((unsigned)max(e, 27) << 23);
}

// Saturating, NaN kept (the conversion itself would make an overflow NaN).
__device__ __forceinline__ float saturated(float x)
{
    return x != x ? x : fminf(fmaxf(x, -448.f), 448.f);
}

// Four values as e4m3 codes in a word, round to nearest even.
__device__ __forceinline__ unsigned codes4(float a, float b, float c, float d)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(saturated(a), saturated(b), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(saturated(c), saturated(d), w, true);
    return (unsigned)w;
}

// |x| for the scale: values that are not finite do not count.
__device__ __forceinline__ float finite_abs(float x)
{
    const float y = fabsf(x);
    return y <= 3.402823466e38f ? y : 0.f;
}

__device__ __forceinline__ float decode(unsigned char c)
{
    return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
}

// The codes of a page's earlier tokens under a scale that grew (rare).
template <int D>
__device__ __forceinline__ void rescale_old(uint8_t* kc, uint8_t* vc, int lo, int P, float kshrink, float vshrink)
{
    for (int i = threadIdx.x; i < lo * D; i += 256) {
        if (kshrink != 1.f)
            kc[i] = (uint8_t)codes4(decode(kc[i]) * kshrink, 0.f, 0.f, 0.f);
        if (vshrink != 1.f) {
            uint8_t* at = vc + (i / lo) * P + i % lo;
            *at = (uint8_t)codes4(decode(*at) * vshrink, 0.f, 0.f, 0.f);
        }
    }
}

// The page of the call's touched block e = b * nblk + j, -1 if there is none.
__device__ __forceinline__ int touched_page(const AppendArgs& a, int64_t e)
{
    const int b = (int)(e / a.nblk), j = (int)(e % a.nblk);
    const Span sp(a.past, a.n_new, b, a.T);
    const int first = sp.past >> a.c.shift;
    if (sp.n <= 0 || j > ((sp.past + sp.n - 1) >> a.c.shift) - first)
        return -1;
    return page_of(a.c, b, first + j);
}

// A page belongs to the first of the call's touched blocks that names it.  Every
// page and head may look through the blocks before its own, which takes no memory
// and no launch but time in the square of their number; or two small kernels
// write each page's owner down first: MARK = false empties the entries that the
// call uses, MARK = true takes the minimum.
template <bool MARK>
__global__ __launch_bounds__(256) void kv_owner_kernel(AppendArgs a, unsigned long long* owner)
{
    for (int64_t e = blockIdx.x * 256ll + threadIdx.x; e < (int64_t)a.B * a.nblk; e += gridDim.x * 256ll) {
        const int page = touched_page(a, e);
        if (page < 0)
            continue;
        if constexpr (MARK)
            atomicMin(owner + page, (unsigned long long)e);
        else
            owner[page] = ~0ull;
    }
}

// Keys and values of one page and head.  Bound by the bytes (6 D a token: two
// rows of bf16 read, two of codes written); rotated keys stay in registers
// between the maximum and the conversion, values are read as 4 tokens x 8
// features a thread so that four neighbouring codes of V's row make a word, and
// turned through LDS.  With the queries in the same launch, 2 x 4096 tokens of
// 32 + 8 heads take 50 us (185 MB, 3.7 TB/s; element by element through an LDS
// tile, in two launches: 283 us); one token of 64 sequences 8.9 us, the time of
// four dependent loads (length, table, scale, row) and a launch.
template <int D, int P>
__device__ __forceinline__ void append_page(const AppendArgs& a, int j, int h, int b)
{
    constexpr int U = D / 16, KR = 256 / U, KI = (P + KR - 1) / KR;           // units a row, rows a pass, passes
    constexpr int VV = D / 8, VU = P / 4 * VV, VI = (VU + 255) / 256;         // V: vectors a row, units, passes
    __shared__ __align__(16) uint8_t turned[D][P + 16];
    __shared__ float red[2][4];
    const int tid = threadIdx.x;
    const Span sp(a.past, a.n_new, b, a.T);
    const int64_t blk = (sp.past >> a.c.shift) + (int64_t)j, base = blk << a.c.shift;
    // new tokens of the page: [lo, hi)
    const int lo = (int)max((int64_t)0, sp.past - base);
    const int hi = (int)min((int64_t)P, (int64_t)sp.past + sp.n - base);
    if (lo >= hi)
        return;
    const int page = page_of(a.c, b, (int)blk);
    if (page < 0)
        return;
    const int64_t ph = (int64_t)page * a.c.H + h;
    const float kwas = a.c.ks[ph], vwas = a.c.vs[ph];
    const int64_t t0 = base - sp.past;            // the call's token of the page's first place
    const int u = tid % U, kr = tid / U, vv = tid % VV, vq = tid / VV;
    int v0, v1;
    unit_vectors(u, a.half, a.inter, v0, v1);
    float ky[KI][16], kmax = 0.f, vmax = 0.f;
    u32x4 vr[VI][4];
#pragma unroll
    for (int i = 0; i < VI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 4 * (vq + 256 / VV * i) + r;
            vr[i][r] = u32x4{0u, 0u, 0u, 0u};
            if (t >= lo && t < hi)
                vr[i][r] = *reinterpret_cast<const u32x4*>(a.v.head(b, h) + (t0 + t) * a.v.st + 8 * vv);
        }
    Unit kraw[KI];
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int t = kr + KR * i;
        if (t >= lo && t < hi)
            kraw[i] = load_unit(a.k.head(b, h) + (t0 + t) * a.k.st, v0, v1);
    }
    // (while those loads are in flight)
    // an earlier touched block with the same page owns it
    int dup = 0;
    const int64_t before = (int64_t)b * a.nblk + j;
    if (a.owner)
        dup = a.owner[page] != (unsigned long long)before;
    else
        for (int64_t e = tid; e < before; e += 256)
            dup |= touched_page(a, e) == page;
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int t = kr + KR * i;
        if (t >= lo && t < hi) {
            widen(ky[i], kraw[i]);
            rotate_unit(ky[i], u, a.half, a.inter,
                        [&](int pair, float& c, float& s) { turn(base + t, a.freq[pair], c, s); });
#pragma unroll
            for (int e = 0; e < 16; ++e)
                kmax = fmaxf(kmax, finite_abs(ky[i][e]));
        }
    }
#pragma unroll
    for (int i = 0; i < VI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                vmax = fmaxf(vmax, finite_abs((float)__builtin_bit_cast(bf16x8, vr[i][r])[e]));
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        kmax = fmaxf(kmax, __shfl_xor(kmax, off, 64));
        vmax = fmaxf(vmax, __shfl_xor(vmax, off, 64));
    }
    if ((tid & 63) == 0) {
        red[0][tid >> 6] = kmax;
        red[1][tid >> 6] = vmax;
    }
    if (__syncthreads_or(dup))
        return;
    float ks = scale_of(fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3])));
    float vs = scale_of(fmaxf(fmaxf(red[1][0], red[1][1]), fmaxf(red[1][2], red[1][3])));
    uint8_t* kc = a.c.k + ph * P * D;
    uint8_t* vc = a.c.v + ph * P * D;
    if (lo > 0) {
        ks = fmaxf(ks, kwas);
        vs = fmaxf(vs, vwas);
        if (ks != kwas || vs != vwas)
            rescale_old<D>(kc, vc, lo, P, kwas / ks, vwas / vs);
    }
    const float kinv = 1.f / ks, vinv = 1.f / vs;
#pragma unroll
    for (int i = 0; i < KI; ++i) {
        const int t = kr + KR * i;
        if (t >= lo && t < hi) {
            unsigned w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = codes4(ky[i][4 * e] * kinv, ky[i][4 * e + 1] * kinv, ky[i][4 * e + 2] * kinv,
                              ky[i][4 * e + 3] * kinv);
            *reinterpret_cast<u32x2*>(kc + t * D + 8 * v0) = u32x2{w[0], w[1]};
            *reinterpret_cast<u32x2*>(kc + t * D + 8 * v1) = u32x2{w[2], w[3]};
        }
    }
#pragma unroll
    for (int i = 0; i < VI; ++i) {
        const int t = 4 * (vq + 256 / VV * i);
        if (t < hi && t + 3 >= lo) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float y[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    y[r] = (float)__builtin_bit_cast(bf16x8, vr[i][r])[e] * vinv;
                *reinterpret_cast<unsigned*>(&turned[8 * vv + e][t]) = codes4(y[0], y[1], y[2], y[3]);
            }
        }
    }
    __syncthreads();
    // rows of V: 16 tokens a thread, whole where all of them are new
    for (int e = tid; e < D * P / 16; e += 256) {
        const int f = e / (P / 16), t = e % (P / 16) * 16;
        if (t >= lo && t + 16 <= hi)
            *reinterpret_cast<u32x4*>(vc + f * P + t) = *reinterpret_cast<const u32x4*>(&turned[f][t]);
        else
            for (int i = max(t, lo); i < min(t + 16, hi); ++i)
                vc[f * P + i] = turned[f][i];
    }
    if (tid == 0) {
        a.c.ks[ph] = ks;
        a.c.vs[ph] = vs;
    }
}

// Queries of 1 << qshift tokens, all heads: the angles are shared by the heads,
// so their cosines and sines are formed once, in LDS.  A unit is read before it
// is written and by the thread that writes it, so q_out may be q.
template <int D>
__device__ __forceinline__ void rotate_queries(const AppendArgs& a, int tile, int b)
{
    constexpr int U = D / 16;
    __shared__ float2 cs[16 * D / 2];
    const Span sp(a.past, a.n_new, b, a.T);
    const int rows = 1 << a.qshift, t0 = tile << a.qshift, n = min(rows, sp.n - t0);
    if (n <= 0)
        return;
    for (int i = threadIdx.x; i < n * a.half; i += 256)
        turn((int64_t)sp.past + t0 + i / a.half, a.freq[i % a.half], cs[i].x, cs[i].y);
    __syncthreads();
    for (int e = threadIdx.x; e < a.Hq * rows * U; e += 256) {
        const int u = e % U, r = (e / U) & (rows - 1), h = e / U >> a.qshift;
        if (r >= n)
            continue;
        int v0, v1;
        unit_vectors(u, a.half, a.inter, v0, v1);
        float y[16];
        widen(y, load_unit(a.q.head(b, h) + (int64_t)(t0 + r) * a.q.st, v0, v1));
        rotate_unit(y, u, a.half, a.inter, [&](int pair, float& c, float& s) {
            c = cs[r * a.half + pair].x;
            s = cs[r * a.half + pair].y;
        });
        bf16x8 o0, o1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o0[i] = (bf16)y[i];
            o1[i] = (bf16)y[8 + i];
        }
        bf16* out = a.q_out.head(b, h) + (int64_t)(t0 + r) * a.q_out.st;
        *reinterpret_cast<bf16x8*>(out + 8 * v0) = o0;
        *reinterpret_cast<bf16x8*>(out + 8 * v1) = o1;
    }
}

// One launch: the pages of every head, then the queries.
template <int D, int P>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a)
{
    const int b = blockIdx.y, pages = a.nblk * a.c.H;
    if ((int)blockIdx.x < pages)
        append_page<D, P>(a, blockIdx.x / a.c.H, blockIdx.x % a.c.H, b);
    else
        rotate_queries<D>(a, blockIdx.x - pages, b);
}

template <int D>
hipError_t launch_append(const AppendArgs& a, hipStream_t s)
{
    const int tiles = a.q.ptr ? (a.T + (1 << a.qshift) - 1) >> a.qshift : 0;
    const dim3 grid(a.nblk * a.c.H + tiles, a.B), block(256);
    switch (a.c.shift) {
    case 4: launch_kernel(kv_append_kernel<D, 16>, grid, block, s, a); break;
    case 5: launch_kernel(kv_append_kernel<D, 32>, grid, block, s, a); break;
    case 6: launch_kernel(kv_append_kernel<D, 64>, grid, block, s, a); break;
    default: launch_kernel(kv_append_kernel<D, 128>, grid, block, s, a);
    }
    return hipGetLastError();
}

int blocks_of(const linrec_kv_cache* c, int32_t T) { return (int)(((int64_t)T + c->page - 2) / c->page + 1); }

// From this many touched blocks on their owners are written down.  Looking against
// writing down, 8 heads of 128: 19.6 / 22.0 us at 512 sequences of one token, 38.1 /
// 35.5 at 1024, 216 / 113 at 4096; 92.8 / 68.3 at 32768 tokens in pages of 16 (2049
// blocks), 7450 / 1200 at 64 x 8192, 1270 / 677 in pages of 64.
constexpr int64_t OWNERS_FROM = 1024;

Act<const bf16> cact(const linrec_tensor& t) { return Act<const bf16>{(const bf16*)t.ptr, t.sb, t.sh, t.st}; }

}  // namespace
}  // namespace linrec

using namespace linrec;

extern "C" size_t linrec_kv_append_workspace_bytes(const linrec_kv_cache* cache, int32_t B, int32_t T)
{
    if (check_kv(cache, B, T) != LINREC_OK || T == 0 || (int64_t)B * blocks_of(cache, T) < OWNERS_FROM)
        return 0;
    return (size_t)cache->pages * sizeof(unsigned long long);
}

extern "C" linrec_status linrec_kv_append(linrec_ctx* ctx, const linrec_kv_cache* cache, int32_t B, int32_t T,
                                          linrec_tensor k, linrec_tensor v, const int32_t* past,
                                          const int32_t* n_new, const double* inv_freq, int32_t rot,
                                          int32_t interleaved, int32_t Hq, linrec_tensor q,
                                          linrec_tensor q_out, void* workspace, void* stream)
{
    linrec_status st;
    if ((st = check_kv(cache, B, T)) != LINREC_OK)
        return st;
    if (rot < 0 || rot > cache->D || rot % 16 || (q.ptr && (Hq < 1 || Hq > 65535)))
        return LINREC_E_SHAPE;
    // a launch holds at most 2^32 - 1 threads along x
    if (((int64_t)T / cache->page + 2) * cache->H + T > 0xffffff)
        return LINREC_E_SHAPE;
    if (T > 0) {
        if ((st = check_kv_ptrs(cache, B, past, n_new)) != LINREC_OK ||
            (st = check_view(k, B, cache->H, T, cache->D, 2, false)) != LINREC_OK ||
            (st = check_view(v, B, cache->H, T, cache->D, 2, false)) != LINREC_OK)
            return st;
        if (q.ptr && ((st = check_view(q, B, Hq, T, cache->D, 2, false)) != LINREC_OK ||
                      (st = check_view(q_out, B, Hq, T, cache->D, 2, true)) != LINREC_OK))
            return st;
        if (rot && !inv_freq)
            return LINREC_E_NULL;
        if (!aligned(inv_freq, 8))
            return LINREC_E_ALIGN;
        if (linrec_kv_append_workspace_bytes(cache, B, T) && (st = check_buffer(workspace)) != LINREC_OK)
            return st;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    if (T == 0)
        return LINREC_OK;
    AppendArgs a{};
    a.c = kv_arg(cache);
    a.k = cact(k);
    a.v = cact(v);
    a.q = cact(q);
    a.q_out = Act<bf16>{(bf16*)q_out.ptr, q_out.sb, q_out.sh, q_out.st};
    a.past = past;
    a.n_new = n_new;
    a.freq = inv_freq;
    a.B = B;
    a.T = T;
    a.Hq = Hq;
    a.half = rot / 2;
    a.nblk = blocks_of(cache, T);
    a.inter = interleaved != 0;
    while (a.qshift < 4 && 1 << a.qshift < T)
        ++a.qshift;
    hipStream_t s = (hipStream_t)stream;
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_KV_APPEND, s, [&] {
        if (linrec_kv_append_workspace_bytes(cache, B, T)) {
            unsigned long long* owner = (unsigned long long*)workspace;
            const dim3 grid((unsigned)std::min<int64_t>(((int64_t)B * a.nblk + 255) / 256, 2048));
            launch_kernel(kv_owner_kernel<false>, grid, dim3(256), s, a, owner);
            launch_kernel(kv_owner_kernel<true>, grid, dim3(256), s, a, owner);
            a.owner = owner;
        }
        return cache->D == 128 ? launch_append<128>(a, s) : launch_append<64>(a, s);
    }));
    return LINREC_OK;
}
