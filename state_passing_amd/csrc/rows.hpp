// rows.hpp -- token rows [B, T, C] with the channel index contiguous, read and
// written 16 bytes at a time, and carried fp32 states beside them; what the calls on
// such rows check and share.
#pragma once

#include "ctx.hpp"
#include "device.hpp"

namespace linrec {

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
            typedef bf16 row __attribute__((ext_vector_type(N)));
            row o;
#pragma unroll
            for (int j = 0; j < N; ++j)
                o[j] = (bf16)y[j];
            *reinterpret_cast<row*>(p) = o;
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

__device__ __forceinline__ float sigmoid(float p) { return __builtin_amdgcn_rcpf(1.f + __expf(-p)); }

// Tokens of sequence b that are there.
__device__ __forceinline__ int tokens_of(const int* n_new, int b, int T_)
{
    return n_new ? min(max(n_new[b], 0), T_) : T_;
}

template <typename D>
inline linrec_status check_rows(const D* d, const linrec_tensor& t, int dtype, bool out)
{
    return check_view(linrec_tensor{t.ptr, t.sb, 0, t.st}, d->B, 1, d->T, d->C, elem_size(dtype), out);
}

inline int64_t round4(int64_t n) { return (n + 3) / 4 * 4; }

// What an empty piece does: n floats of carry from `in` (NULL: zeros) to `out`.
inline linrec_status pass_carry(const float* in, float* out, int64_t n, hipStream_t s)
{
    if (in == out)
        return LINREC_OK;
    LAUNCH(launch_carry_copy(in, out, n, s));
    return LINREC_OK;
}

template <typename T>
inline Act<const T> cact(const linrec_tensor& a) { return Act<const T>{(const T*)a.ptr, a.sb, 0, a.st}; }
template <typename T>
inline Act<T> mact(const linrec_tensor& a) { return Act<T>{(T*)a.ptr, a.sb, 0, a.st}; }

}  // namespace linrec
