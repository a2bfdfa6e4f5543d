// ctx.hpp -- the context behind the C ABI and what every source that declares
// entry points of include/linrec.h shares: status helpers, the device check
// and the launch wrapper that carries the opt-in kernel timing.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>
#include <vector>

#include "launch.hpp"
#include "linrec.h"

struct TimedLaunch {
    int kind;
    hipEvent_t begin, end;
};

struct linrec_ctx {
    int device;
    void* scratch;          // this device's address of the no-allocation scratch
    hipError_t scratch_err; // result of looking that address up
    hipStream_t aux;        // state transitions
    hipEvent_t ev_start;    // inputs ready on the caller's stream
    hipEvent_t ev_scan;     // a piece's scan finished (aux)
    hipEvent_t ev_slot[2];  // a workspace slot's last reader finished (aux)
    // opt-in per-kernel timing (linrec_ctx_set_timing)
    int timing;
    std::vector<TimedLaunch> pending;
    std::vector<hipEvent_t> pool;
    double ms[LINREC_KERNEL_KINDS];
    int64_t count[LINREC_KERNEL_KINDS];
};

namespace linrec {

extern thread_local int g_last_hip_error;

inline linrec_status hip_fail(hipError_t e, linrec_status code)
{
    g_last_hip_error = (int)e;
    return code;
}

inline int elem_size(int dtype) { return dtype == LINREC_BF16 ? 2 : 4; }

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int kChunk = 64;

inline linrec_status check_desc(const linrec_desc* d)
{
    if (!d)
        return LINREC_E_NULL;
    if (d->dtype != LINREC_BF16 && d->dtype != LINREC_F32)
        return LINREC_E_DTYPE;
    // B: the sequence backward's launches carry another piece's segment sums
    // as a second set of grid rows z, so 2 B must fit the grid's 65535
    if (d->chunk != kChunk || d->B < 1 || d->H < 1 || d->B > 32767 || d->H > 65535 || d->T < 0 ||
        d->T > LINREC_MAX_T)
        return LINREC_E_SHAPE;
    if ((d->dk != 64 && d->dk != 128) || (d->dv != 64 && d->dv != 128))
        return LINREC_E_SHAPE;
    if (d->out_dtype != LINREC_BF16 && d->out_dtype != LINREC_F32)
        return LINREC_E_DTYPE;
    if (d->dtype == LINREC_F32 && (d->dk != 64 || d->dv != 64 || d->out_dtype != LINREC_F32))
        return LINREC_E_DTYPE;
    if (d->decay != LINREC_DECAY_NONE && d->decay != LINREC_DECAY_HEAD &&
        d->decay != LINREC_DECAY_TOKEN)
        return LINREC_E_LAYOUT;
    return LINREC_OK;
}

// An activation view: 16-byte aligned rows, non-negative strides, rows at
// least `width` elements apart.
inline linrec_status check_act(const linrec_tensor& t, int width, int esz)
{
    if (!t.ptr)
        return LINREC_E_NULL;
    if (t.sb < 0 || t.sh < 0 || t.st < width)
        return LINREC_E_LAYOUT;
    if (!aligned(t.ptr, 16) || (t.st * esz) % 16 || (t.sh * esz) % 16 || (t.sb * esz) % 16)
        return LINREC_E_ALIGN;
    return LINREC_OK;
}

inline linrec_status check_decay(const linrec_desc* d, const linrec_tensor& a)
{
    if (d->decay == LINREC_DECAY_NONE)
        return LINREC_OK;
    if (!a.ptr)
        return LINREC_E_NULL;
    if (!aligned(a.ptr, 4))
        return LINREC_E_ALIGN;
    if (a.sh < 0 || (d->decay == LINREC_DECAY_TOKEN && (a.sb < 0 || a.st < 0)))
        return LINREC_E_LAYOUT;
    return LINREC_OK;
}

inline linrec_status check_state_ptr(const void* p, bool required)
{
    if (!p)
        return required ? LINREC_E_NULL : LINREC_OK;
    return aligned(p, 4) ? LINREC_OK : LINREC_E_ALIGN;
}

inline linrec_status check_buffer(const void* p)
{
    if (!p)
        return LINREC_E_WORKSPACE;
    return aligned(p, 16) ? LINREC_OK : LINREC_E_WORKSPACE;
}

// A [B,H,T,width] view whose strides are looked at only where the dimension
// has more than one entry; `out`: its rows must not overlap (strides that nest:
// each at least the extent of the dimensions inside it).
inline linrec_status check_view(const linrec_tensor& t, int64_t B, int64_t H, int64_t T, int64_t width,
                                int esz, bool out)
{
    if (!t.ptr)
        return LINREC_E_NULL;
    int64_t n[3] = {B, H, T}, s[3] = {t.sb, t.sh, t.st};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && s[i] < 0)
            return LINREC_E_LAYOUT;
    if (T > 1 && t.st < width)
        return LINREC_E_LAYOUT;
    if (out) {
        for (int i = 0; i < 3; ++i)          // by stride, ascending
            for (int j = i + 1; j < 3; ++j)
                if (s[j] < s[i]) {
                    std::swap(s[i], s[j]);
                    std::swap(n[i], n[j]);
                }
        __int128 extent = width;             // no overflow, whatever the strides
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1) {
                if (s[i] < extent)
                    return LINREC_E_LAYOUT;
                extent += (__int128)s[i] * (n[i] - 1);
            }
    }
    if (!aligned(t.ptr, 16))
        return LINREC_E_ALIGN;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (s[i] * esz) % 16)
            return LINREC_E_ALIGN;
    return LINREC_OK;
}

inline linrec_status check_ctx(linrec_ctx* ctx)
{
    if (!ctx)
        return LINREC_E_NULL;
    int cur = -1;
    hipError_t e = hipGetDevice(&cur);
    if (e != hipSuccess)
        return hip_fail(e, LINREC_E_DEVICE);
    if (cur != ctx->device)
        return hip_fail(hipErrorInvalidDevice, LINREC_E_DEVICE);
    return LINREC_OK;
}

inline hipError_t pool_event(linrec_ctx* ctx, hipEvent_t* ev)
{
    if (!ctx->pool.empty()) {
        *ev = ctx->pool.back();
        ctx->pool.pop_back();
        return hipSuccess;
    }
    // no system-scope release at the event: it would write back L2 after
    // the bracketed kernel and bill that to the kernel's duration
    return hipEventCreateWithFlags(ev, hipEventDisableSystemFence);
}

// Launch `fn` on `stream`; with timing on, the kernels it launches carry a pair
// of events as their own start and end stamps (launch_kernel).
template <typename F>
hipError_t timed_launch(linrec_ctx* ctx, int kind, hipStream_t stream, F fn)
{
    if (!ctx->timing)
        return fn();
    TimedLaunch t{kind, nullptr, nullptr};
    hipError_t e = pool_event(ctx, &t.begin);
    if (e == hipSuccess)
        e = pool_event(ctx, &t.end);
    if (e == hipSuccess) {
        // the events become the launched kernels' own start and end stamps
        linrec::launch_stamps() = linrec::LaunchStamps{t.begin, t.end};
        e = fn();
        linrec::launch_stamps() = linrec::LaunchStamps{};
    }
    if (e != hipSuccess) {
        if (t.begin)
            ctx->pool.push_back(t.begin);
        if (t.end)
            ctx->pool.push_back(t.end);
        return e;
    }
    ctx->pending.push_back(t);
    return hipSuccess;
}

}  // namespace linrec

#define LAUNCH(call)                                              \
    do {                                                          \
        hipError_t e_ = (call);                                   \
        if (e_ != hipSuccess)                                     \
            return linrec::hip_fail(e_, LINREC_E_LAUNCH);         \
    } while (0)
