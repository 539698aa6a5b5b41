// C-ABI layer of the losses over vocabulary logits: argument checks and kernel
// launches.  Every entry point is declared and documented in include/mpstep.h.
#include <cmath>

#include "losses.h"

using mpk::GradView;
using mpk::LogitsView;
using mpk::LossArgs;
using mpk::set_error;
using mpk::set_ok;

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

mp_status run_rows(const mp_logits* x, const mp_logits_grad* g, LossArgs& a, mp_stream stream)
{
    if (x->rows == 0) return set_ok();
    mp_status st = check_place(x->data, "logits", stream);
    if (st != MP_OK) return st;
    a.x = view_of(x);
    a.g = view_of(x, g);
    a.workspace = x->workspace;
    hipError_t e = mpk::launch_rows(a, x->dtype, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "loss launch: %s", hipGetErrorString(e));
    return set_ok();
}

}  // namespace

extern "C" {

mp_status mp_target_count(int64_t n, const int64_t* targets, int64_t* count, mp_stream stream)
{
    if (n < 0) return set_error(MP_ERR_INVALID, "n must be >= 0");
    Arrays arrays;
    mp_status st = arrays.in(targets, 8, n, true, "targets");
    if (st == MP_OK) st = arrays.out(count, 8, 1, true, "count");
    if (st == MP_OK) st = check_place(count, "count", stream);
    if (st != MP_OK) return st;
    hipError_t e = mpk::launch_target_count(n, targets, count, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "target count launch: %s", hipGetErrorString(e));
    return set_ok();
}

mp_status mp_token_logprob(const mp_logits* x, const int64_t* targets, float* logp, float* lse,
                           mp_stream stream)
{
    mp_status st = check_logits(x);
    Arrays arrays;
    if (st == MP_OK) st = arrays.in(targets, 8, x->rows, true, "targets");
    if (st == MP_OK) st = arrays.out(logp, 4, x->rows, true, "logp");
    if (st == MP_OK) st = arrays.out(lse, 4, x->rows, false, "lse");
    if (st == MP_OK) st = arrays.disjoint(x, nullptr);
    if (st != MP_OK) return st;
    LossArgs a{};
    a.kind = mpk::kLogprob;
    a.targets = targets;
    a.logp = logp;
    a.lse = lse;
    return run_rows(x, nullptr, a, stream);
}

mp_status mp_token_logprob_grad(const mp_logits* x, const int64_t* targets, const float* lse,
                                const float* dlogp, const mp_logits_grad* grad, mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st == MP_OK && grad == nullptr) st = set_error(MP_ERR_INVALID, "grad is NULL");
    if (st == MP_OK) st = check_grad(x, grad);
    Arrays arrays;
    if (st == MP_OK) st = arrays.in(targets, 8, x->rows, true, "targets");
    if (st == MP_OK) st = arrays.in(lse, 4, x->rows, true, "lse");
    if (st == MP_OK) st = arrays.in(dlogp, 4, x->rows, true, "dlogp");
    if (st == MP_OK) st = arrays.disjoint(x, grad);
    if (st != MP_OK) return st;
    if (x->rows == 0) return set_ok();
    st = check_place(x->data, "logits", stream);
    if (st != MP_OK) return st;
    hipError_t e = mpk::launch_logprob_grad(view_of(x), targets, lse, dlogp, view_of(x, grad), x->dtype,
                                            static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "gradient launch: %s", hipGetErrorString(e));
    return set_ok();
}

mp_status mp_cross_entropy(const mp_logits* x, const int64_t* targets, const float* weights,
                           float* loss, const mp_logits_grad* grad, mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st == MP_OK) st = check_grad(x, grad);
    Arrays arrays;
    if (st == MP_OK) st = arrays.in(targets, 8, x->rows, true, "targets");
    if (st == MP_OK) st = arrays.in(weights, 4, x->rows, false, "weights");
    if (st == MP_OK) st = arrays.out(loss, 4, x->rows, true, "loss");
    if (st == MP_OK) st = arrays.disjoint(x, grad);
    if (st != MP_OK) return st;
    LossArgs a{};
    a.kind = mpk::kXent;
    a.targets = targets;
    a.weights = weights;
    a.loss = loss;
    return run_rows(x, grad, a, stream);
}

mp_status mp_policy_loss(const mp_logits* x, const int64_t* targets, const float* old_logp,
                         const float* ref_logp, const float* advantage, const float* weights,
                         const mp_policy_cfg* cfg, float* loss, float* logp, float* kl,
                         const mp_logits_grad* grad, mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st == MP_OK) st = check_grad(x, grad);
    if (st != MP_OK) return st;
    if (cfg == nullptr) return set_error(MP_ERR_INVALID, "cfg is NULL");
    if (!(cfg->clip_low >= 0.0f && cfg->clip_low <= 1.0f))
        return set_error(MP_ERR_INVALID, "clip_low must be in [0, 1]");
    if (!(cfg->clip_high >= 0.0f) || !std::isfinite(cfg->clip_high))
        return set_error(MP_ERR_INVALID, "clip_high must be finite and >= 0");
    if (!(cfg->kl_coef >= 0.0f) || !std::isfinite(cfg->kl_coef))
        return set_error(MP_ERR_INVALID, "kl_coef must be finite and >= 0");
    if (x->rows > 0 && ref_logp == nullptr && (cfg->kl_coef != 0.0f || kl != nullptr))
        return set_error(MP_ERR_INVALID, "a KL term needs ref_logp");
    Arrays arrays;
    st = arrays.in(targets, 8, x->rows, true, "targets");
    if (st == MP_OK) st = arrays.in(old_logp, 4, x->rows, true, "old_logp");
    if (st == MP_OK) st = arrays.in(ref_logp, 4, x->rows, false, "ref_logp");
    if (st == MP_OK) st = arrays.in(advantage, 4, x->rows, true, "advantage");
    if (st == MP_OK) st = arrays.in(weights, 4, x->rows, false, "weights");
    if (st == MP_OK) st = arrays.out(loss, 4, x->rows, true, "loss");
    if (st == MP_OK) st = arrays.out(logp, 4, x->rows, false, "logp");
    if (st == MP_OK) st = arrays.out(kl, 4, x->rows, false, "kl");
    if (st == MP_OK) st = arrays.disjoint(x, grad);
    if (st != MP_OK) return st;
    LossArgs a{};
    a.kind = mpk::kPolicy;
    a.targets = targets;
    a.weights = weights;
    a.loss = loss;
    a.logp = logp;
    a.kl = kl;
    a.old_logp = old_logp;
    a.ref_logp = ref_logp;
    a.advantage = advantage;
    a.clip_low = cfg->clip_low;
    a.clip_high = cfg->clip_high;
    a.kl_coef = cfg->kl_coef;
    return run_rows(x, grad, a, stream);
}

mp_status mp_preference_loss(const mp_logits* x, const int64_t* targets, int64_t n_pairs,
                             const int64_t* seq_start, const float* ref_logp,
                             const mp_preference_cfg* cfg, float* loss, float* seq_logp,
                             float* logp, float* lse, float* dlogp, const mp_logits_grad* grad,
                             mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st == MP_OK) st = check_grad(x, grad);
    if (st != MP_OK) return st;
    if (cfg == nullptr) return set_error(MP_ERR_INVALID, "cfg is NULL");
    if (cfg->kind != MP_PREF_SIGMOID && cfg->kind != MP_PREF_SQUARED)
        return set_error(MP_ERR_INVALID, "kind must be MP_PREF_SIGMOID or MP_PREF_SQUARED");
    if (!(cfg->beta > 0.0f) || !std::isfinite(cfg->beta))
        return set_error(MP_ERR_INVALID, "beta must be finite and > 0");
    if (!(cfg->label_smoothing >= 0.0f && cfg->label_smoothing <= 0.5f))
        return set_error(MP_ERR_INVALID, "label_smoothing must be in [0, 0.5]");
    if (!std::isfinite(cfg->margin)) return set_error(MP_ERR_INVALID, "margin must be finite");
    if (n_pairs < 1 || n_pairs > kMaxRows)
        return set_error(MP_ERR_INVALID, "n_pairs must be 1 to 2^22 - 1");
    Arrays arrays;
    st = arrays.in(targets, 8, x->rows, true, "targets");
    if (st == MP_OK) st = arrays.in(seq_start, 8, 2 * n_pairs + 1, true, "seq_start");
    if (st == MP_OK) st = arrays.in(ref_logp, 4, 2 * n_pairs, false, "ref_logp");
    if (st == MP_OK) st = arrays.out(loss, 4, n_pairs, true, "loss");
    if (st == MP_OK) st = arrays.out(seq_logp, 4, 2 * n_pairs, true, "seq_logp");
    if (st == MP_OK) st = arrays.out(logp, 4, x->rows, true, "logp");
    if (st == MP_OK) st = arrays.out(lse, 4, x->rows, true, "lse");
    if (st == MP_OK) st = arrays.out(dlogp, 4, x->rows, true, "dlogp");
    if (st == MP_OK) st = arrays.disjoint(x, grad);
    if (st == MP_OK) st = check_place(x->rows > 0 ? x->data : seq_start,
                                      x->rows > 0 ? "logits" : "seq_start", stream);
    if (st != MP_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    LossArgs a{};
    a.kind = mpk::kLogprob;
    a.x = view_of(x);
    a.workspace = x->workspace;
    a.targets = targets;
    a.logp = logp;
    a.lse = lse;
    mpk::PairArgs p{};
    p.targets = targets;
    p.seq_start = seq_start;
    p.ref_logp = ref_logp;
    p.logp = logp;
    p.loss = loss;
    p.seq_logp = seq_logp;
    p.dlogp = dlogp;
    p.n_pairs = n_pairs;
    p.rows = static_cast<int32_t>(x->rows);
    p.kind = cfg->kind;
    p.length_mean = cfg->length_mean != 0;
    p.beta = static_cast<double>(cfg->beta);
    p.label_smoothing = static_cast<double>(cfg->label_smoothing);
    p.margin = static_cast<double>(cfg->margin);
    hipError_t e = x->rows > 0 ? mpk::launch_rows(a, x->dtype, s) : hipSuccess;
    if (e == hipSuccess) e = mpk::launch_pairs(p, s);
    if (e == hipSuccess && grad != nullptr && x->rows > 0)
        e = mpk::launch_logprob_grad(a.x, targets, lse, dlogp, view_of(x, grad), x->dtype, s);
    if (e != hipSuccess) return set_error(MP_ERR_HIP, "preference launch: %s", hipGetErrorString(e));
    return set_ok();
}

mp_status mp_distill_loss(const mp_logits* x, const mp_teacher* teacher, const float* weights,
                          float* loss, const mp_logits_grad* grad, mp_stream stream)
{
    mp_status st = check_logits(x);
    if (st == MP_OK) st = check_grad(x, grad);
    if (st != MP_OK) return st;
    if (teacher == nullptr) return set_error(MP_ERR_INVALID, "teacher is NULL");
    if (teacher->k < 1 || teacher->k > MP_DISTILL_MAX_K)
        return set_error(MP_ERR_INVALID, "teacher: k must be 1 to %d", MP_DISTILL_MAX_K);
    if (!known_dtype(teacher->dtype)) return set_error(MP_ERR_INVALID, "teacher: unknown dtype");
    Arrays arrays;
    const int64_t entries = x->rows * teacher->k;
    st = arrays.in(teacher->values, elem_bytes(teacher->dtype), entries, true, "teacher values");
    if (st == MP_OK) st = arrays.in(teacher->ids, 8, entries, true, "teacher ids");
    if (st == MP_OK) st = arrays.in(teacher->lse, 4, x->rows, false, "teacher lse");
    if (st == MP_OK) st = arrays.in(weights, 4, x->rows, false, "weights");
    if (st == MP_OK) st = arrays.out(loss, 4, x->rows, true, "loss");
    if (st == MP_OK) st = arrays.disjoint(x, grad);
    if (st != MP_OK) return st;
    LossArgs a{};
    a.kind = mpk::kDistill;
    a.weights = weights;
    a.loss = loss;
    a.k = teacher->k;
    a.teacher_dtype = teacher->dtype;
    a.teacher_values = teacher->values;
    a.teacher_ids = teacher->ids;
    a.teacher_lse = teacher->lse;
    return run_rows(x, grad, a, stream);
}

}  // extern "C"
