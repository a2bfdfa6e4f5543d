// kv_attn.hip -- attention over the paged 8-bit cache (linrec_kv_attn).
#include <hip/hip_runtime.h>

#include <math.h>

#include "kv.hpp"

namespace linrec {
namespace {

struct AttnArgs {
    KvCache c;
    Act<const bf16> q;
    Act<bf16> o;
    float* lse;
    const int* past;
    const int* n_new;
    int B, T, Hq, group, window;
    float scale;
};

__device__ __forceinline__ float decode(unsigned char c)
{
    return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
}

// One workgroup per query row: 256 keys at a time, one per thread, with the
// running maximum and sum of the softmax; then the threads take (feature, part
// of the keys) for the weighted sum.
template <int D>
__global__ __launch_bounds__(256) void kv_attn_row_kernel(AttnArgs a)
{
    constexpr int PARTS = 256 / D;
    __shared__ float qs[D], ps[256], red[4], acc[PARTS][D];
    __shared__ int pg[256];
    const int t = blockIdx.x, hq = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const Span sp(a.past, a.n_new, b, a.T);
    if (t >= sp.n)
        return;
    const int h = hq / a.group, P = 1 << a.c.shift;
    const int64_t pos = sp.past + t, lo = a.window > 0 ? max((int64_t)0, pos - a.window + 1) : 0;
    const int64_t end = min(pos + 1, (int64_t)a.c.max_pages << a.c.shift);
    if (tid < D)
        qs[tid] = (float)a.q.head(b, hq)[t * a.q.st + tid];
    float m = -INFINITY, l = 0.f, o = 0.f;
    const int f = tid % D, part = tid / D;
    for (int64_t k0 = lo; k0 < end; k0 += 256) {
        __syncthreads();
        const int64_t key = k0 + tid;
        const int page = key < end ? page_of(a.c, b, key >> a.c.shift) : -1;
        float s = -INFINITY;
        if (page >= 0) {
            const int64_t ph = (int64_t)page * a.c.H + h;
            const uint8_t* kp = a.c.k + (ph * P + (key & (P - 1))) * D;
            float x = 0.f;
            for (int i = 0; i < D; ++i)
                x += qs[i] * decode(kp[i]);
            s = x * a.c.ks[ph] * a.scale;
        }
        pg[tid] = page;
        float mx = s;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
            mx = fmaxf(mx, __shfl_xor(mx, off, 64));
        if ((tid & 63) == 0)
            red[tid >> 6] = mx;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        // a score of NaN spreads through p; the maximum passes it over
        const float ref = mn == -INFINITY ? 0.f : mn, keep = __expf(m - ref);
        const float p = page >= 0 ? __expf(s - ref) : 0.f;
        ps[tid] = p;
        l = l * keep + p;
        o *= keep;
        m = mn;
        __syncthreads();
        for (int j = part; j < 256; j += PARTS)
            if (pg[j] >= 0) {
                const int64_t ph = (int64_t)pg[j] * a.c.H + h;
                o += ps[j] * a.c.vs[ph] * decode(a.c.v[(ph * D + f) * P + ((k0 + j) & (P - 1))]);
            }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        l += __shfl_xor(l, off, 64);
    __syncthreads();
    if ((tid & 63) == 0)
        red[tid >> 6] = l;
    acc[part][f] = o;
    __syncthreads();
    l = red[0] + red[1] + red[2] + red[3];
    if (tid < D) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
            y += acc[i][tid];
        a.o.head(b, hq)[t * a.o.st + tid] = (bf16)(l == 0.f ? 0.f : y / l);
    }
    if (a.lse && tid == 0)
        a.lse[((int64_t)b * a.Hq + hq) * a.T + t] = l == 0.f ? -INFINITY : m + logf(l);
}

template <int D>
hipError_t launch_attn(const AttnArgs& a, hipStream_t s)
{
    launch_kernel(kv_attn_row_kernel<D>, dim3(a.T, a.Hq, a.B), dim3(256), s, a);
    return hipGetLastError();
}

linrec_status check_attn(const linrec_kv_cache* cache, int32_t B, int32_t T, int32_t Hq)
{
    const linrec_status st = check_kv(cache, B, T);
    if (st != LINREC_OK)
        return st;
    return Hq < 1 || Hq > 65535 || Hq % cache->H ? LINREC_E_SHAPE : LINREC_OK;
}

}  // namespace
}  // namespace linrec

using namespace linrec;

extern "C" {

size_t linrec_kv_attn_workspace_bytes(const linrec_kv_cache* cache, int32_t B, int32_t T, int32_t Hq)
{
    return 0;
}

linrec_status linrec_kv_attn(linrec_ctx* ctx, const linrec_kv_cache* cache, int32_t B, int32_t T, int32_t Hq,
                             linrec_tensor q, const int32_t* past, const int32_t* n_new, float scale,
                             int32_t window, linrec_tensor o, float* lse, void* workspace, void* stream)
{
    linrec_status st;
    if ((st = check_attn(cache, B, T, Hq)) != LINREC_OK)
        return st;
    if (!isfinite(scale))
        return LINREC_E_SHAPE;
    if (T > 0) {
        if ((st = check_kv_ptrs(cache, B, past, n_new)) != LINREC_OK ||
            (st = check_view(q, B, Hq, T, cache->D, 2, false)) != LINREC_OK ||
            (st = check_view(o, B, Hq, T, cache->D, 2, true)) != LINREC_OK)
            return st;
        if (!aligned(lse, 4))
            return LINREC_E_ALIGN;
        if (linrec_kv_attn_workspace_bytes(cache, B, T, Hq) && (st = check_buffer(workspace)) != LINREC_OK)
            return st;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    if (T == 0)
        return LINREC_OK;
    AttnArgs a{};
    a.c = kv_arg(cache);
    a.q = Act<const bf16>{(const bf16*)q.ptr, q.sb, q.sh, q.st};
    a.o = Act<bf16>{(bf16*)o.ptr, o.sb, o.sh, o.st};
    a.lse = lse;
    a.past = past;
    a.n_new = n_new;
    a.B = B;
    a.T = T;
    a.Hq = Hq;
    a.group = Hq / cache->H;
    a.window = window;
    a.scale = scale;
    hipStream_t s = (hipStream_t)stream;
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_KV_ATTN, s, [&] {
        return cache->D == 128 ? launch_attn<128>(a, s) : launch_attn<64>(a, s);
    }));
    return LINREC_OK;
}

}  // extern "C"
