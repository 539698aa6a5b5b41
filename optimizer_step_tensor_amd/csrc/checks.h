// The argument checks of the calls over rows of logits (losses_api.hip, scores_api.hip,
// routing_api.hip), and the kernels' views of their structs.
#pragma once

#include <cmath>

#include "losses.h"

namespace mpk {
namespace {

constexpr int64_t kMaxVocab = int64_t(1) << 30;
constexpr int64_t kMaxRows = (int64_t(1) << 22) - 1;     // 1024 lanes a row: a launch below 2^32 lanes
constexpr int64_t kMaxStride = int64_t(1) << 32;

int elem_bytes(int32_t dtype)
{
    return dtype == MP_FP32 ? 4 : 2;
}

bool aligned(const void* p, uintptr_t to)
{
    return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}

bool known_dtype(int32_t d)
{
    return d == MP_BF16 || d == MP_FP16 || d == MP_FP32;
}

// Bytes from the first to the last element of rows x vocab at a stride.
uintptr_t extent(int64_t rows, int64_t vocab, int64_t stride, int es)
{
    return static_cast<uintptr_t>(((rows - 1) * stride + vocab) * es);
}

mp_status check_logits(const mp_logits* x)
{
    if (x == nullptr) return set_error(MP_ERR_INVALID, "logits is NULL");
    if (!known_dtype(x->dtype)) return set_error(MP_ERR_INVALID, "logits: unknown dtype");
    if (x->rows < 0 || x->rows > kMaxRows)
        return set_error(MP_ERR_INVALID, "logits: rows must be 0 to 2^22 - 1");
    if (x->vocab < 1 || x->vocab > kMaxVocab)
        return set_error(MP_ERR_INVALID, "logits: vocab must be 1 to 2^30");
    if (x->rows > 1 && (x->stride < x->vocab || x->stride > kMaxStride))
        return set_error(MP_ERR_INVALID, "logits: stride must be vocab to 2^32 elements");
    if (!(x->temperature >= 0x1p-20f && x->temperature <= 0x1p20f))
        return set_error(MP_ERR_INVALID, "logits: temperature must be 2^-20 to 2^20");
    if (x->rows > 0 && x->data == nullptr) return set_error(MP_ERR_INVALID, "logits: NULL buffer");
    if (!aligned(x->data, elem_bytes(x->dtype)))
        return set_error(MP_ERR_ALIGN, "logits must be aligned to their element type");
    if (!aligned(x->workspace, 16))
        return set_error(MP_ERR_ALIGN, "the workspace must be 16-byte aligned");
    return MP_OK;
}

mp_status check_grad(const mp_logits* x, const mp_logits_grad* g)
{
    if (g == nullptr) return MP_OK;
    if (x->rows > 0 && g->data == nullptr) return set_error(MP_ERR_INVALID, "gradient: NULL buffer");
    if (x->rows > 1 && (g->stride < x->vocab || g->stride > kMaxStride))
        return set_error(MP_ERR_INVALID, "gradient: stride must be vocab to 2^32 elements");
    if (!std::isfinite(g->scale)) return set_error(MP_ERR_INVALID, "gradient: scale must be finite");
    const int es = elem_bytes(x->dtype);
    if (!aligned(g->data, es))
        return set_error(MP_ERR_ALIGN, "the gradient must be aligned to its element type");
    if (!aligned(g->dev_scale, 4) || !aligned(g->dev_count, 8))
        return set_error(MP_ERR_ALIGN, "dev_scale must be 4-byte, dev_count 8-byte aligned");
    if (x->rows > 0 && !(g->data == x->data && (x->rows == 1 || g->stride == x->stride))) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(x->data);
        const uintptr_t b = reinterpret_cast<uintptr_t>(g->data);
        const uintptr_t na = extent(x->rows, x->vocab, x->rows > 1 ? x->stride : x->vocab, es);
        const uintptr_t nb = extent(x->rows, x->vocab, x->rows > 1 ? g->stride : x->vocab, es);
        if (a < b + nb && b < a + na)
            return set_error(MP_ERR_INVALID, "the gradient overlaps the logits without being them "
                                             "(same address and stride)");
    }
    return MP_OK;
}

// The arrays of a call besides the logits and their gradient: each is checked as it is added, and
// `disjoint` refuses what the kernels would read and write at once -- the parts of a split row read
// the row's inputs while the first writes its outputs, and inputs are taken as constant.
class Arrays {
public:
    mp_status in(const void* p, uintptr_t elem, int64_t n, bool required, const char* name)
    {
        return add(p, elem, n, required, false, name);
    }
    mp_status out(const void* p, uintptr_t elem, int64_t n, bool required, const char* name)
    {
        return add(p, elem, n, required, true, name);
    }
    // a caller's optional scratch memory, which no call without rows touches
    mp_status scratch(const void* p, uintptr_t bytes, int64_t rows)
    {
        if (!aligned(p, 16)) return set_error(MP_ERR_ALIGN, "the workspace must be 16-byte aligned");
        if (rows > 0) put(p, bytes, true, "workspace");
        return MP_OK;
    }
    mp_status disjoint(const mp_logits* x, const mp_logits_grad* g)
    {
        if (x->rows > 0) put(x->workspace, MP_LOSS_WORKSPACE_BYTES, true, "workspace");
        if (g != nullptr) {
            put(g->dev_scale, 4, false, "dev_scale");
            put(g->dev_count, 8, false, "dev_count");
        }
        for (int i = 0; i < count_; ++i) {
            const One& a = one_[i];
            for (int j = 0; j < i; ++j) {
                const One& b = one_[j];
                if ((a.written || b.written) && a.at < b.at + b.bytes && b.at < a.at + a.bytes)
                    return set_error(MP_ERR_INVALID, "%s overlaps %s", b.name, a.name);
            }
            if (a.written && in_rows(a, x->data, x->stride, x))
                return set_error(MP_ERR_INVALID, "%s overlaps the logits", a.name);
            if (g != nullptr && in_rows(a, g->data, g->stride, x))
                return set_error(MP_ERR_INVALID, "%s overlaps the gradient", a.name);
        }
        return MP_OK;
    }

private:
    struct One {
        uintptr_t at, bytes;
        const char* name;
        bool written;
    };
    One one_[16];           // a policy loss has 11: 5 read, 3 written, the workspace, two scalars
    int count_ = 0;

    void put(const void* p, uintptr_t bytes, bool written, const char* name)
    {
        if (p != nullptr && bytes > 0)
            one_[count_++] = One{reinterpret_cast<uintptr_t>(p), bytes, name, written};
    }
    mp_status add(const void* p, uintptr_t elem, int64_t n, bool required, bool written, const char* name)
    {
        if (required && n > 0 && p == nullptr) return set_error(MP_ERR_INVALID, "%s is NULL", name);
        if (!aligned(p, elem))
            return set_error(MP_ERR_ALIGN, "%s must be %d-byte aligned", name, static_cast<int>(elem));
        put(p, static_cast<uintptr_t>(n) * elem, written, name);
        return MP_OK;
    }
    // Does `a` meet one of the rows?  (What lies between them is not the call's.)
    static bool in_rows(const One& a, const void* data, int64_t stride, const mp_logits* x)
    {
        if (x->rows == 0) return false;
        const int es = elem_bytes(x->dtype);
        const uintptr_t base = reinterpret_cast<uintptr_t>(data);
        const uintptr_t row = static_cast<uintptr_t>(x->vocab) * es;
        if (a.at >= base + extent(x->rows, x->vocab, x->rows > 1 ? stride : x->vocab, es) ||
            a.at + a.bytes <= base)
            return false;
        if (a.at < base || x->rows == 1) return true;
        const uintptr_t step = static_cast<uintptr_t>(stride) * es;
        const uintptr_t within = (a.at - base) % step;
        return within < row || within + a.bytes > step;
    }
};

// The work is launched on the current device: `data` (the logits) has to live
// there, and the stream, too.
mp_status check_place(const void* data, const char* what, mp_stream stream)
{
    int cur = -1, dev = -1;
    hipError_t e = hipGetDevice(&cur);
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "hipGetDevice: %s", hipGetErrorString(e));
    hipPointerAttribute_t at{};
    e = hipPointerGetAttributes(&at, data);
    if (e != hipSuccess) (void)hipGetLastError();        // an address that HIP does not know
    if (e != hipSuccess || (at.type != hipMemoryTypeDevice && at.type != hipMemoryTypeManaged))
        return set_error(MP_ERR_INVALID, "%s: not device memory", what);
    if (at.device != cur)
        return set_error(MP_ERR_INVALID, "%s: on device %d but device %d is current", what, at.device,
                         cur);
    if (stream != nullptr) {
        e = hipStreamGetDevice(static_cast<hipStream_t>(stream), &dev);
        if (e != hipSuccess) return set_error(MP_ERR_HIP, "hipStreamGetDevice: %s", hipGetErrorString(e));
        if (dev != cur)
            return set_error(MP_ERR_INVALID, "the stream is of device %d but device %d is current", dev,
                             cur);
    }
    return MP_OK;
}

LogitsView view_of(const mp_logits* x)
{
    LogitsView v{};
    v.x = x->data;
    v.stride = x->rows > 1 ? x->stride : x->vocab;
    v.rows = static_cast<int32_t>(x->rows);
    v.vocab = static_cast<int32_t>(x->vocab);
    v.inv_t = 1.0 / static_cast<double>(x->temperature);
    const double k = 1.4426950408889634 * v.inv_t;
    v.k_hi = static_cast<float>(k);
    if (static_cast<double>(v.k_hi) >= k) v.k_hi = std::nextafter(v.k_hi, 0.0f);
    v.k_lo = static_cast<float>(k - static_cast<double>(v.k_hi));
    return v;
}

GradView view_of(const mp_logits* x, const mp_logits_grad* g)
{
    GradView v{};
    if (g == nullptr) return v;
    v.dx = g->data;
    v.stride = x->rows > 1 ? g->stride : x->vocab;
    v.dev_scale = g->dev_scale;
    v.dev_count = g->dev_count;
    v.scale = static_cast<double>(g->scale) / static_cast<double>(x->temperature);
    return v;
}

}  // namespace
}  // namespace mpk
