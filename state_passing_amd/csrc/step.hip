// step.hip -- the layer's recurrence and the delta rule token by token
// (linrec_step), for generation.
//
// Bound by the state's bytes: 8 d_k d_v per head, read once and written once
// (96 x 32 heads of 128 x 128: 80 us, 5.0 TB/s, where a copy reaches 4.85).
// Columns of the state are independent, so a workgroup takes 64 of them with
// all d_k rows in registers (a thread: 4 neighbouring columns of every 16th
// row): 32 columns cost the large calls 2-15%, 128 the small ones (64 heads:
// 5.1 against 4.5 us).  With w = q S and m = k S over the old state, the new one gives
//   u = beta (v - a m)  (linear layer: u = v),  S <- a S + k^T u,
//   o = q S_new = a w + (q . k) u,
// so one pass over the registers and one reduction over the rows serve both
// products, and the output does not wait for the update.
#include <hip/hip_runtime.h>

#include "ctx.hpp"
#include "device.hpp"

namespace linrec {
namespace {

template <typename T, typename OT, int DK, int DV, bool DELTA>
__global__ __launch_bounds__(256) void step_kernel(Act<const T> q, Act<const T> k, Act<const T> v,
                                                   Act<const float> beta, DecayArg dec, float* S,
                                                   const int* slots, int nslots, Act<OT> o, int H, int T_)
{
    constexpr int DVT = 64, VL = DVT / 4, RG = 256 / VL, RPT = DK / RG;   // columns, column lanes, row groups, rows a thread
    // one record per wave and column lane: w, m (4 each) and q . k
    __shared__ float part[2][4][VL][9];
    const int vl = threadIdx.x % VL, rg = threadIdx.x / VL, wave = threadIdx.x >> 6;
    const int h = blockIdx.y, b = blockIdx.z, c0 = blockIdx.x * DVT + 4 * vl;
    int slot = b;
    if (slots) {
        slot = slots[b];
        int skip = slot < 0 || slot >= nslots;
        for (int i = threadIdx.x; i < b; i += 256)
            skip |= slots[i] == slot;
        if (__syncthreads_or(skip)) {
            for (int64_t i = threadIdx.x; i < (int64_t)T_ * DVT; i += 256)
                o.head(b, h)[i / DVT * o.st + blockIdx.x * DVT + i % DVT] = (OT)0.f;
            return;
        }
    }
    float* Sp = S + ((int64_t)slot * H + h) * DK * DV + c0;
    floatx4 s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        s[i] = *reinterpret_cast<const floatx4*>(Sp + (rg + RG * i) * DV);
    const T* qp = q.head(b, h);
    const T* kp = k.head(b, h);
    const T* vp = v.head(b, h) + c0;
    for (int t = 0; t < T_; ++t) {
        const float a = dec.kind == 0   ? 1.f
                        : dec.kind == 1 ? dec.ptr[h * dec.sh]
                                        : dec.ptr[b * dec.sb + h * dec.sh + t * dec.st];
        float kk[RPT];
        floatx4 w = zero4(), m = zero4();
        float qk = 0.f;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float qq = (float)qp[t * q.st + rg + RG * i];
            kk[i] = (float)kp[t * k.st + rg + RG * i];
            w += qq * s[i];
            if constexpr (DELTA)
                m += kk[i] * s[i];
            qk += qq * kk[i];
        }
        floatx4 vv;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            vv[j] = (float)vp[t * v.st + j];
#pragma unroll
        for (int off = VL; off < 64; off <<= 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] += __shfl_xor(w[j], off, 64);
                if constexpr (DELTA)
                    m[j] += __shfl_xor(m[j], off, 64);
            }
            qk += __shfl_xor(qk, off, 64);
        }
        float(*pt)[VL][9] = part[t & 1];
        if ((threadIdx.x & 63) < VL) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                pt[wave][vl][j] = w[j];
                pt[wave][vl][4 + j] = m[j];
            }
            pt[wave][vl][8] = qk;
        }
        __syncthreads();   // the other half of `part` serves the next token
        w = zero4();
        m = zero4();
        qk = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[j] += pt[i][vl][j];
                m[j] += pt[i][vl][4 + j];
            }
            qk += pt[i][vl][8];
        }
        floatx4 u = vv;
        if constexpr (DELTA) {
            const float bt = beta.head(b, h)[t * beta.st];
            u = bt * (vv - a * m);
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            s[i] = a * s[i] + kk[i] * u;
        if (rg == 0) {
            OT* op = o.head(b, h) + t * o.st + c0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                op[j] = (OT)(a * w[j] + qk * u[j]);
        }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i)
        *reinterpret_cast<floatx4*>(Sp + (rg + RG * i) * DV) = s[i];
}

struct StepArgs {
    const linrec_desc* d;
    linrec_tensor q, k, v, beta, decay, o;
    float* S;
    const int* slots;
    int nslots;
};

template <typename T, typename OT, int DK, int DV>
hipError_t step_impl(const StepArgs& s, hipStream_t stream)
{
    const linrec_desc* d = s.d;
    auto c = [](const linrec_tensor& t) { return Act<const T>{(const T*)t.ptr, t.sb, t.sh, t.st}; };
    const Act<OT> o{(OT*)s.o.ptr, s.o.sb, s.o.sh, s.o.st};
    const Act<const float> beta{(const float*)s.beta.ptr, s.beta.sb, s.beta.sh, s.beta.st};
    const DecayArg dec{(const float*)s.decay.ptr, s.decay.sb, s.decay.sh, s.decay.st, d->decay};
    const dim3 grid(DV / 64, d->H, d->B);
    if (s.beta.ptr)
        launch_kernel(step_kernel<T, OT, DK, DV, true>, grid, dim3(256), stream, c(s.q), c(s.k), c(s.v),
                      beta, dec, s.S, s.slots, s.nslots, o, d->H, d->T);
    else
        launch_kernel(step_kernel<T, OT, DK, DV, false>, grid, dim3(256), stream, c(s.q), c(s.k), c(s.v),
                      beta, dec, s.S, s.slots, s.nslots, o, d->H, d->T);
    return hipGetLastError();
}

template <typename T, typename OT>
hipError_t step_dims(const StepArgs& s, hipStream_t stream)
{
    const linrec_desc* d = s.d;
    if (d->dk == 128 && d->dv == 128)
        return step_impl<T, OT, 128, 128>(s, stream);
    if (d->dk == 64 && d->dv == 64)
        return step_impl<T, OT, 64, 64>(s, stream);
    if (d->dk == 64)
        return step_impl<T, OT, 64, 128>(s, stream);
    return step_impl<T, OT, 128, 64>(s, stream);
}

hipError_t launch_step(const StepArgs& s, hipStream_t stream)
{
    if (s.d->dtype == LINREC_F32)
        return step_impl<float, float, 64, 64>(s, stream);
    return s.d->out_dtype == LINREC_F32 ? step_dims<bf16, float>(s, stream) : step_dims<bf16, bf16>(s, stream);
}

}  // namespace
}  // namespace linrec

using namespace linrec;

extern "C" linrec_status linrec_step(linrec_ctx* ctx, const linrec_desc* d, linrec_tensor q, linrec_tensor k,
                                     linrec_tensor v, linrec_tensor beta, linrec_tensor decay, float* S,
                                     const int32_t* slots, int32_t nslots, linrec_tensor o, void* stream)
{
    linrec_status st;
    if ((st = check_desc(d)) != LINREC_OK)
        return st;
    if (d->T > 0) {
        const int esz = elem_size(d->dtype), osz = elem_size(d->out_dtype);
        if (!S)
            return LINREC_E_NULL;
        if (nslots < 1 || (!slots && nslots < d->B))
            return LINREC_E_SHAPE;
        if ((st = check_view(q, d->B, d->H, d->T, d->dk, esz, false)) != LINREC_OK ||
            (st = check_view(k, d->B, d->H, d->T, d->dk, esz, false)) != LINREC_OK ||
            (st = check_view(v, d->B, d->H, d->T, d->dv, esz, false)) != LINREC_OK ||
            (st = check_view(o, d->B, d->H, d->T, d->dv, osz, true)) != LINREC_OK ||
            (st = check_decay(d, decay)) != LINREC_OK)
            return st;
        if (beta.ptr && (beta.sb < 0 || beta.sh < 0 || beta.st < 0))
            return LINREC_E_LAYOUT;
        if (!aligned(S, 16) || !aligned(beta.ptr, 4) || !aligned(slots, 4))
            return LINREC_E_ALIGN;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    if (d->T == 0)
        return LINREC_OK;
    hipStream_t s = (hipStream_t)stream;
    const StepArgs args{d, q, k, v, beta, decay, o, S, slots, nslots};
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_STEP, s, [&] { return launch_step(args, s); }));
    return LINREC_OK;
}
