// kv_append.hip -- appending keys and values to the paged 8-bit cache, with the
// rotation by position applied on the way (linrec_kv_append).
#include <hip/hip_runtime.h>

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
    int B, T, Hq, half, nblk;   // half: rotated pairs; nblk: pages a sequence may touch
    bool inter;
};

// cos and sin of position * freq.  The product and its reduction to a fraction
// of a turn are fp64: at position 2^20 an fp32 angle would be off by 2^-5 rad.
__device__ __forceinline__ void turn(int64_t pos, double freq, float& c, float& s)
{
    const double t = (double)pos * freq * 0.15915494309189535;   // 1 / (2 pi)
    sincospif((float)(2.0 * (t - rint(t))), &s, &c);
}

// Element i of a head's row after the rotation by `pos` (i: the feature).
__device__ __forceinline__ float rotated(const AppendArgs& a, const bf16* row, int64_t pos, int i)
{
    const float x = (float)row[i];
    if (i >= 2 * a.half)
        return x;
    float c, s;
    if (a.inter) {
        turn(pos, a.freq[i >> 1], c, s);
        return (i & 1) ? x * c + (float)row[i - 1] * s : x * c - (float)row[i + 1] * s;
    }
    const int p = i < a.half ? i : i - a.half;
    turn(pos, a.freq[p], c, s);
    return i < a.half ? x * c - (float)row[i + a.half] * s : x * c + (float)row[i - a.half] * s;
}

// The least power of two s with amax <= 448 s (448 = 1.75 * 2^8 is the largest
// e4m3 value), not below 2^-100, from the bits of amax.
__device__ __forceinline__ float scale_of(float amax)
{
    const unsigned u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((unsigned)max(e, 27) << 23);
}

// Two values as e4m3 codes in the low half-word: saturating, NaN kept.
__device__ __forceinline__ unsigned codes2(float x, float y)
{
    const float cx = x != x ? x : fminf(fmaxf(x, -448.f), 448.f);
    const float cy = y != y ? y : fminf(fmaxf(y, -448.f), 448.f);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(cx, cy, 0, false) & 0xffffu;
}

__device__ __forceinline__ float decode(unsigned char c)
{
    return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
}

// One workgroup per (touched page, head, sequence): keys, then values, of the
// page's new tokens through an LDS tile [token][feature].
template <int D>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a)
{
    __shared__ float tile[128][D + 1];
    __shared__ float red[4];
    const int P = 1 << a.c.shift, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const Span sp(a.past, a.n_new, b, a.T);
    const int64_t blk = (sp.past >> a.c.shift) + (int64_t)blockIdx.x, base = blk << a.c.shift;
    // new tokens of the page: [lo, hi)
    const int lo = (int)max((int64_t)0, sp.past - base);
    const int hi = (int)min((int64_t)P, (int64_t)sp.past + sp.n - base);
    if (lo >= hi)
        return;
    const int page = page_of(a.c, b, (int)blk);
    if (page < 0)
        return;
    // an earlier touched block with the same page owns it
    int dup = 0;
    for (int64_t e = tid; e < (int64_t)b * a.nblk + blockIdx.x; e += 256) {
        const int eb = (int)(e / a.nblk), ej = (int)(e % a.nblk);
        const Span es(a.past, a.n_new, eb, a.T);
        const int first = es.past >> a.c.shift;
        if (es.n > 0 && ej <= ((es.past + es.n - 1) >> a.c.shift) - first)
            dup |= page_of(a.c, eb, first + ej) == page;
    }
    if (__syncthreads_or(dup))
        return;
    const int64_t ph = (int64_t)page * a.c.H + h;
    for (int which = 0; which < 2; ++which) {
        const bool keys = which == 0;
        const Act<const bf16>& x = keys ? a.k : a.v;
        float amax = 0.f;
        for (int i = tid; i < (hi - lo) * D; i += 256) {
            const int t = lo + i / D, f = i % D;
            const bf16* row = x.head(b, h) + (base + t - sp.past) * x.st;
            const float y = keys ? rotated(a, row, base + t, f) : (float)row[f];
            tile[t][f] = y;
            if (fabsf(y) <= 3.402823466e38f)
                amax = fmaxf(amax, fabsf(y));
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
            amax = fmaxf(amax, __shfl_xor(amax, off, 64));
        if ((tid & 63) == 0)
            red[tid >> 6] = amax;
        __syncthreads();
        amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        float* sptr = keys ? a.c.ks : a.c.vs;
        const float was = sptr[ph];
        float s = scale_of(amax), shrink = 1.f;
        if (lo > 0) {
            s = fmaxf(s, was);
            shrink = was / s;
        }
        uint8_t* codes = (keys ? a.c.k : a.c.v) + ph * P * D;
        if (shrink != 1.f)
            for (int i = tid; i < lo * D; i += 256) {
                uint8_t* at = codes + (keys ? (i / D) * D + i % D : (i / lo) * P + i % lo);
                *at = (uint8_t)codes2(decode(*at) * shrink, 0.f);
            }
        const float inv = 1.f / s;
        for (int i = tid; i < (hi - lo) * D; i += 256) {
            const int t = keys ? lo + i / D : lo + i % (hi - lo), f = keys ? i % D : i / (hi - lo);
            codes[keys ? t * D + f : f * P + t] = (uint8_t)codes2(tile[t][f] * inv, 0.f);
        }
        __syncthreads();   // everyone has read `was`; the tile is free
        if (tid == 0)
            sptr[ph] = s;
    }
}

// Queries: one workgroup per (16 tokens, head, sequence).  A row is staged
// before it is written, so q_out may be q.
template <int D>
__global__ __launch_bounds__(256) void kv_rotate_q_kernel(AppendArgs a)
{
    const int h = blockIdx.y, b = blockIdx.z;
    const Span sp(a.past, a.n_new, b, a.T);
    const int t0 = blockIdx.x * 16;
    float y[16 * D / 256];
#pragma unroll
    for (int i = 0; i < 16 * D / 256; ++i) {
        const int e = threadIdx.x + 256 * i, t = t0 + e / D;
        if (t < sp.n)
            y[i] = rotated(a, a.q.head(b, h) + (int64_t)t * a.q.st, sp.past + t, e % D);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16 * D / 256; ++i) {
        const int e = threadIdx.x + 256 * i, t = t0 + e / D;
        if (t < sp.n)
            a.q_out.head(b, h)[(int64_t)t * a.q_out.st + e % D] = (bf16)y[i];
    }
}

template <int D>
hipError_t launch_append(const AppendArgs& a, hipStream_t s)
{
    launch_kernel(kv_append_kernel<D>, dim3(a.nblk, a.c.H, a.B), dim3(256), s, a);
    if (a.q.ptr)
        launch_kernel(kv_rotate_q_kernel<D>, dim3((a.T + 15) / 16, a.Hq, a.B), dim3(256), s, a);
    return hipGetLastError();
}

Act<const bf16> cact(const linrec_tensor& t) { return Act<const bf16>{(const bf16*)t.ptr, t.sb, t.sh, t.st}; }

}  // namespace
}  // namespace linrec

using namespace linrec;

extern "C" linrec_status linrec_kv_append(linrec_ctx* ctx, const linrec_kv_cache* cache, int32_t B, int32_t T,
                                          linrec_tensor k, linrec_tensor v, const int32_t* past,
                                          const int32_t* n_new, const double* inv_freq, int32_t rot,
                                          int32_t interleaved, int32_t Hq, linrec_tensor q,
                                          linrec_tensor q_out, void* stream)
{
    linrec_status st;
    if ((st = check_kv(cache, B, T)) != LINREC_OK)
        return st;
    if (rot < 0 || rot > cache->D || rot % 16 || (q.ptr && (Hq < 1 || Hq > 65535)))
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
    a.nblk = (int)(((int64_t)T + cache->page - 2) / cache->page + 1);
    a.inter = interleaved != 0;
    hipStream_t s = (hipStream_t)stream;
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_KV_APPEND, s, [&] {
        return cache->D == 128 ? launch_append<128>(a, s) : launch_append<64>(a, s);
    }));
    return LINREC_OK;
}
