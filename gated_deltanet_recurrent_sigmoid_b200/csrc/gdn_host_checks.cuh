// gdn_host_checks.cuh -- host helpers shared by the C entry points: descriptor
// checks, byte ranges for the aliasing rules, one-time set-up per device and
// the launch wrapper.  Host code only.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "gdn_decode.h"
#include "gdn_spec.h"

namespace gdn {
namespace host {

inline int64_t elem_size(int32_t dtype)
{
    switch (dtype) {
    case GDN_DTYPE_BF16: return 2;
    case GDN_DTYPE_F32: return 4;
    case GDN_DTYPE_I32: return 4;
    case GDN_DTYPE_I64: return 8;
    default: return 0;
    }
}

inline bool aligned(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) % bytes) == 0; }

// Byte range a descriptor can reach: [lo, hi).  Empty when any dim is 0.
struct Span {
    uintptr_t lo = 0, hi = 0;
    bool empty() const { return hi <= lo; }
};

inline Span span_of(const gdn_tensor *t)
{
    Span s;
    if (!t || !t->data)
        return s;
    int64_t last = 0;
    for (int d = 0; d < t->ndim; ++d) {
        if (t->shape[d] == 0)
            return s;
        last += (t->shape[d] - 1) * t->stride[d];
    }
    s.lo = reinterpret_cast<uintptr_t>(t->data);
    s.hi = s.lo + static_cast<uintptr_t>((last + 1) * elem_size(t->dtype));
    return s;
}

inline bool overlap(const Span &x, const Span &y)
{
    if (x.empty() || y.empty())
        return false;
    return x.lo < y.hi && y.lo < x.hi;
}

// Basic descriptor sanity: rank, non-negative shape and strides, and a data
// pointer unless the tensor has no elements.  `dtype2` is a second accepted
// element type (0: none).
inline int check_desc(const gdn_tensor *t, int32_t dtype, int32_t dtype2 = 0)
{
    if (!t)
        return GDN_ERR_NULL_ARG;
    if (t->dtype != dtype && (dtype2 == 0 || t->dtype != dtype2))
        return GDN_ERR_DTYPE;
    if (t->ndim < 1 || t->ndim > 4)
        return GDN_ERR_SHAPE;
    bool empty = false;
    for (int d = 0; d < t->ndim; ++d) {
        if (t->shape[d] < 0 || t->stride[d] < 0)
            return GDN_ERR_SHAPE;
        empty = empty || t->shape[d] == 0;
    }
    if (!t->data && !empty)
        return GDN_ERR_NULL_ARG;
    return GDN_OK;
}

// Token layout of an activation whose trailing `trail` dims are per token.
// Varlen: leading dims [T_tot] or [1, T_tot].  Fixed length: [N, T], which
// must flatten to one token dimension.
struct TokenLayout {
    int64_t T_tot = 0;   // tokens
    int64_t T = 0;       // tokens per sequence (fixed-length mode)
    int64_t tok = 0;     // stride between consecutive tokens, in elements
};

inline int token_layout(const gdn_tensor *t, int trail, bool varlen, int64_t N, TokenLayout *L)
{
    const int lead = t->ndim - trail;
    if (varlen) {
        if (lead == 1) {
            L->T_tot = t->shape[0];
            L->tok = t->stride[0];
        } else if (lead == 2 && t->shape[0] == 1) {
            L->T_tot = t->shape[1];
            L->tok = t->stride[1];
        } else {
            return GDN_ERR_SHAPE;
        }
        L->T = -1;
        return GDN_OK;
    }
    if (lead != 2 || t->shape[0] != N)
        return GDN_ERR_SHAPE;
    const int64_t T = t->shape[1];
    L->T = T;
    L->T_tot = N * T;
    if (T == 0 || N == 0)
        L->tok = 0;  // no tokens: the stride is never used
    else if (T == 1)
        L->tok = t->stride[0];
    else if (N == 1)
        L->tok = t->stride[1];
    else if (t->stride[0] != T * t->stride[1])
        return GDN_ERR_SHAPE;
    else
        L->tok = t->stride[1];
    return GDN_OK;
}

// The stride of a dim matters only when the dim has more than one entry.
inline bool stride_ok(int64_t extent, int64_t stride, int64_t multiple)
{
    return extent <= 1 || stride % multiple == 0;
}

#define GDN_TRY(expr)              \
    do {                           \
        const int rc_ = (expr);    \
        if (rc_ != GDN_OK)         \
            return rc_;            \
    } while (0)

// One-time set-up per device (shared-memory opt-ins, SM counts), safe when
// several host threads make their first call on a device at once: the first
// caller runs `init` under the lock; the flag is published with release
// order after everything `init` wrote, so a thread that sees it set also
// sees those writes.  A failed `init` leaves the flag clear (the next call
// tries again).
struct PerDevice {
    static constexpr int kMaxDevices = 64;
    std::mutex lock;
    std::atomic<bool> ready[kMaxDevices] = {};
};

template <typename Init>
cudaError_t once_per_device(PerDevice &pd, int dev, Init &&init)
{
    if (dev < 0 || dev >= PerDevice::kMaxDevices)
        return cudaErrorInvalidDevice;
    if (pd.ready[dev].load(std::memory_order_acquire))
        return cudaSuccess;
    std::lock_guard<std::mutex> guard(pd.lock);
    if (pd.ready[dev].load(std::memory_order_relaxed))
        return cudaSuccess;
    const cudaError_t err = init();
    if (err == cudaSuccess)
        pd.ready[dev].store(true, std::memory_order_release);
    return err;
}

// Streaming multiprocessors of the current device (read once per device).
inline cudaError_t current_sm_count(int *sms)
{
    static PerDevice once;
    static int count[PerDevice::kMaxDevices];      // written once per device, inside `once`
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err == cudaSuccess)
        err = once_per_device(once, dev, [&]() {
            return cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev);
        });
    if (err == cudaSuccess)
        *sms = count[dev];
    return err;
}

// Launch with or without the programmatic-stream-serialization attribute.
template <typename Kernel, typename... Args>
cudaError_t launch_ex(Kernel kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool pdl,
                      const Args &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace host
}  // namespace gdn
