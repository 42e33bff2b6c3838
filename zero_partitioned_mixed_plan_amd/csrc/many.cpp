// Entry points of the many-tensor AdamW step (zero_many_*): argument checks,
// the handle's tables, and launches on the caller's stream.
#include <cmath>
#include <cstring>
#include <memory>
#include <new>

#include "many.h"

using namespace zmi;

namespace {

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Sections of the device allocation.
struct Layout {
    size_t block, part, flags, tensors, chunks, end;
    explicit Layout(const zero_many* w) {
        block = 0;
        part = up256(sizeof(ManyBlock));
        flags = part + up256(kNormParts * sizeof(double));
        tensors = flags + up256(kNormParts * sizeof(int32_t));
        chunks = tensors + up256(w->numels.size() * sizeof(ManyTensor));
        end = chunks + up256(static_cast<size_t>(w->n_chunks) * sizeof(uint32_t));
    }
    // the pinned mirror holds one block and the tensors
    static size_t host_tensors() { return up256(sizeof(ManyBlock)); }
};

int check_device(const zero_many* w) {
    int dev = -1;
    const hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    if (w->ready && dev != w->device) {
        return fail(ZERO_ESTATE, "the handle is bound to another device than the current one");
    }
    return ZERO_OK;
}

// Device and pinned memory, and the chunk table, on the first device call.
int ensure(zero_many* w, hipStream_t s) {
    int rc = check_device(w);
    if (rc != ZERO_OK || w->ready) return rc;
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
    const Layout at(w);
    std::vector<uint32_t> chunks;
    chunks.reserve(static_cast<size_t>(w->n_chunks));
    for (size_t i = 0; i < w->numels.size(); ++i) {
        const int64_t n = many_chunks(w->numels[i], w->bits);
        chunks.insert(chunks.end(), static_cast<size_t>(n), static_cast<uint32_t>(i));
    }
    void *d = nullptr, *h = nullptr;
    e = hipMalloc(&d, at.end);
    if (e != hipSuccess) return hip_fail(e, "hipMalloc(tensor table)");
    const size_t host = Layout::host_tensors() + w->numels.size() * sizeof(ManyTensor);
    e = hipHostMalloc(&h, host, hipHostMallocDefault);
    if (e == hipSuccess && !chunks.empty()) {
        e = hipMemcpyAsync(static_cast<char*>(d) + at.chunks, chunks.data(),
                           chunks.size() * sizeof(uint32_t), hipMemcpyHostToDevice, s);
        if (e == hipSuccess) e = hipStreamSynchronize(s);
    }
    if (e != hipSuccess) {
        if (h != nullptr) (void)hipHostFree(h);
        (void)hipFree(d);
        return hip_fail(e, "tensor table");
    }
    std::memset(h, 0, host);
    w->d_mem = static_cast<char*>(d);
    w->h_mem = static_cast<char*>(h);
    w->view.block = reinterpret_cast<ManyBlock*>(w->d_mem + at.block);
    w->view.part = reinterpret_cast<double*>(w->d_mem + at.part);
    w->view.part_flag = reinterpret_cast<int32_t*>(w->d_mem + at.flags);
    w->view.tensors = reinterpret_cast<const ManyTensor*>(w->d_mem + at.tensors);
    w->view.chunk_tensor = reinterpret_cast<const uint32_t*>(w->d_mem + at.chunks);
    w->view.n_chunks = w->n_chunks;
    w->view.chunk = many_chunk(w->bits);
    w->device = dev;
    w->ready = true;
    return ZERO_OK;
}

uint64_t address(const void* p) { return static_cast<uint64_t>(reinterpret_cast<uintptr_t>(p)); }

// Table entry of tensor i, after checking its pointers.
int fill_tensor(const zero_many* w, const zero_many_buffers_t* b, size_t i, int64_t chunk0,
                ManyTensor* t) {
    const bool any = w->numels[i] > 0;
    const bool full = b->master != nullptr;
    *t = ManyTensor{};
    t->numel = w->numels[i];
    t->chunk0 = chunk0;
    t->chunks = many_chunks(t->numel, w->bits);
    t->elem0 = w->offsets[i];
    t->group = w->groups[i];
    if (!any) return ZERO_OK;
    t->grad = address(b->grad[i]);
    const uint64_t gsize = b->grad_dtype == ZERO_F32 ? 4 : 2;
    bool off = t->grad % gsize != 0;
    if (full) {
        t->master = address(b->master[i]);
        t->m = address(b->exp_avg[i]);
        t->v = address(b->exp_avg_sq[i]);
        if (t->master == 0 || t->m == 0 || t->v == 0) {
            return fail(ZERO_ENULL, "tensor " + std::to_string(i) +
                                        ": master, exp_avg and exp_avg_sq must be non-NULL");
        }
        off |= t->master % 4 != 0;
        if (w->bits == 8) {
            t->m_scale = address(b->exp_avg_scale[i]);
            t->v_scale = address(b->exp_avg_sq_scale[i]);
            if (t->m_scale == 0 || t->v_scale == 0) {
                return fail(ZERO_ENULL, "tensor " + std::to_string(i) +
                                            ": 8-bit moments need their scales");
            }
        } else {
            off |= t->m % 4 != 0 || t->v % 4 != 0;
        }
        if (b->param != nullptr) {
            t->param = address(b->param[i]);
            if (t->param == 0) {
                return fail(ZERO_ENULL, "tensor " + std::to_string(i) + ": param is NULL");
            }
            off |= t->param % 2 != 0;
        }
    }
    if (off) {
        return fail(ZERO_EALIGN, "tensor " + std::to_string(i) +
                                     ": a pointer is not aligned to its element");
    }
    return ZERO_OK;
}

int require_state(const zero_many* w) {
    if (!w->ready || !w->state_ready) {
        return fail(ZERO_ESTATE, "no device state: call zero_many_state_upload first");
    }
    return check_device(w);
}

int require_bound(const zero_many* w, bool full) {
    if (!w->bound || (full && !w->full)) {
        return fail(ZERO_ESTATE, full ? "no tensors: call zero_many_bind with master weights and "
                                        "moments first"
                                      : "no tensors: call zero_many_bind first");
    }
    return check_device(w);
}

}  // namespace

extern "C" {

int zero_many_create(const int64_t* numels, const int32_t* groups, int32_t n_tensors,
                     int32_t n_groups, int32_t state_bits, zero_many_t** out) {
    if (out == nullptr) return fail(ZERO_ENULL, "out is NULL");
    *out = nullptr;
    if (n_tensors < 0) return fail(ZERO_EINVAL, "n_tensors must be >= 0");
    if (n_tensors > 0 && numels == nullptr) return fail(ZERO_ENULL, "numels is NULL");
    if (n_groups < 1 || n_groups > ZERO_MANY_MAX_GROUPS) {
        return fail(ZERO_EINVAL, "n_groups must be in [1, ZERO_MANY_MAX_GROUPS]");
    }
    if (state_bits != 8 && state_bits != 32) return fail(ZERO_EINVAL, "state_bits must be 8 or 32");
    try {
        auto w = std::unique_ptr<zero_many>(new zero_many);
        w->n_groups = n_groups;
        w->bits = state_bits;
        for (int32_t i = 0; i < n_tensors; ++i) {
            const int64_t n = numels[i];
            const int32_t g = groups != nullptr ? groups[i] : 0;
            // every element has a place below 2^48 in the padded order
            if (n < 0 || n > (int64_t(1) << 48) - w->padded - kManyBlock) {
                return fail(ZERO_EINVAL, "numels[" + std::to_string(i) + "] is out of range");
            }
            if (g < 0 || g >= n_groups) {
                return fail(ZERO_EINVAL, "groups[" + std::to_string(i) + "] is out of range");
            }
            w->numels.push_back(n);
            w->groups.push_back(g);
            w->offsets.push_back(w->padded);
            w->total += n;
            w->padded += (n + kManyBlock - 1) / kManyBlock * kManyBlock;
            w->n_chunks += many_chunks(n, w->bits);
        }
        *out = w.release();
    } catch (const std::bad_alloc&) {
        return fail(ZERO_ENOMEM, "out of host memory");
    }
    return ZERO_OK;
}

int zero_many_info(const zero_many_t* w, zero_many_info_t* out) {
    if (w == nullptr || out == nullptr) return fail(ZERO_ENULL, "many or out is NULL");
    *out = zero_many_info_t{};
    out->total_numel = w->total;
    out->padded_numel = w->padded;
    out->state_bytes = w->bits == 8 ? 2 * (w->total + w->padded / kManyBlock) : 8 * w->total;
    out->n_tensors = static_cast<int32_t>(w->numels.size());
    out->n_groups = w->n_groups;
    out->state_bits = w->bits;
    return ZERO_OK;
}

int64_t zero_many_offsets(const zero_many_t* w, int64_t* out, int64_t cap) {
    if (w == nullptr) return fail(ZERO_ENULL, "many is NULL");
    if (cap < 0) return fail(ZERO_EINVAL, "cap must be >= 0");
    if (cap > 0 && out == nullptr) return fail(ZERO_ENULL, "out is NULL");
    const int64_t n = static_cast<int64_t>(w->offsets.size());
    for (int64_t i = 0; i < n && i < cap; ++i) out[i] = w->offsets[static_cast<size_t>(i)];
    return n;
}

void zero_many_destroy(zero_many_t* w) {
    if (w == nullptr) return;
    if (w->h_mem != nullptr) (void)hipHostFree(w->h_mem);
    if (w->d_mem != nullptr) (void)hipFree(w->d_mem);
    delete w;
}

int zero_many_bind(zero_many_t* w, const zero_many_buffers_t* b, void* stream) {
    if (w == nullptr || b == nullptr) return fail(ZERO_ENULL, "many or buffers is NULL");
    const bool any = !w->numels.empty();
    if (any && b->grad == nullptr) return fail(ZERO_ENULL, "grad is NULL");
    if (!valid_grad_dtype(b->grad_dtype)) return bad_grad_dtype();
    const bool full = b->master != nullptr;
    if (full != (b->exp_avg != nullptr) || full != (b->exp_avg_sq != nullptr) ||
        (!full && b->param != nullptr)) {
        return fail(ZERO_ENULL, "master, exp_avg and exp_avg_sq go together, and param needs them");
    }
    const bool scales = b->exp_avg_scale != nullptr;
    if (scales != (b->exp_avg_sq_scale != nullptr) || scales != (full && w->bits == 8)) {
        return fail(ZERO_EINVAL, "scales belong to moments in 8 bits, both or neither");
    }
    if (b->param != nullptr && !valid_dtype(b->param_dtype)) {
        return fail(ZERO_EINVAL, "param_dtype must be ZERO_F16 or ZERO_BF16");
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    int32_t grad_dtype = b->grad_dtype;
    const int32_t param_dtype = b->param != nullptr ? b->param_dtype : 0;
    try {
        // every pointer is checked before anything of the handle changes
        std::vector<ManyTensor> table(w->numels.size());
        int64_t chunk = 0;
        bool grads = false;
        for (size_t i = 0; i < table.size(); ++i) {
            const int rc = fill_tensor(w, b, i, chunk, &table[i]);
            if (rc != ZERO_OK) return rc;
            chunk += many_chunks(w->numels[i], w->bits);
            grads |= table[i].grad != 0;
        }
        if (capturing(s)) return fail(ZERO_ESTATE, "zero_many_bind cannot be captured");
        // A captured kernel reads this table through the types it was
        // captured with: other ones would take it out of the tensors.
        if (w->captured && !grads) grad_dtype = w->grad_dtype;
        if ((w->captured && grad_dtype != w->grad_dtype) ||
            (w->captured_full && (!full || param_dtype != w->param_dtype))) {
            return fail(ZERO_ESTATE, "a graph captured from this handle holds other types");
        }
        const int rc = ensure(w, s);
        if (rc != ZERO_OK) return rc;
        hipError_t e = hipStreamSynchronize(s);  // the mirror and the table are free again
        if (e != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
        if (!table.empty()) {
            char* h = w->h_mem + Layout::host_tensors();
            std::memcpy(h, table.data(), table.size() * sizeof(ManyTensor));
            e = hipMemcpyAsync(w->d_mem + Layout(w).tensors, h, table.size() * sizeof(ManyTensor),
                               hipMemcpyHostToDevice, s);
            if (e == hipSuccess) e = hipStreamSynchronize(s);
            if (e != hipSuccess) return hip_fail(e, "tensor table upload");
        }
    } catch (const std::bad_alloc&) {
        return fail(ZERO_ENOMEM, "out of host memory");
    }
    w->grad_dtype = grad_dtype;
    w->param_dtype = param_dtype;
    w->bound = true;
    w->full = full;
    return ZERO_OK;
}

int zero_many_state_upload(zero_many_t* w, int64_t applied_steps, const zero_scaler_t* scaler,
                           uint64_t seed, void* stream) {
    if (w == nullptr || scaler == nullptr) return fail(ZERO_ENULL, "many or scaler is NULL");
    if (applied_steps < 0) return fail(ZERO_EINVAL, "applied_steps must be >= 0");
    int rc = check_scaler(scaler);
    if (rc != ZERO_OK) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (capturing(s)) return fail(ZERO_ESTATE, "zero_many_state_upload cannot be captured");
    try {
        if ((rc = ensure(w, s)) != ZERO_OK) return rc;
    } catch (const std::bad_alloc&) {
        return fail(ZERO_ENOMEM, "out of host memory");
    }
    hipError_t e = hipStreamSynchronize(s);
    if (e != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
    auto* h = reinterpret_cast<ManyBlock*>(w->h_mem);
    *h = ManyBlock{};
    h->st.t = applied_steps;
    h->st.scale = scaler->scale;
    h->st.min_scale = scaler->min_scale;
    h->st.backoff = scaler->backoff;
    h->st.growth = scaler->growth;
    h->st.window = scaler->window;
    h->st.good_steps = scaler->good_steps;
    h->st.dynamic = scaler->dynamic != 0;
    h->seed = seed;
    e = hipMemcpyAsync(w->view.block, h, sizeof(ManyBlock), hipMemcpyHostToDevice, s);
    if (e == hipSuccess) e = hipStreamSynchronize(s);
    if (e != hipSuccess) return hip_fail(e, "state upload");
    w->state_ready = true;
    return ZERO_OK;
}

int zero_many_state_download(zero_many_t* w, int64_t* applied_steps, zero_scaler_t* scaler,
                             int32_t* last_flag, int64_t* skipped_steps, void* stream) {
    if (w == nullptr) return fail(ZERO_ENULL, "many is NULL");
    int rc = require_state(w);
    if (rc != ZERO_OK) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (capturing(s)) return fail(ZERO_ESTATE, "zero_many_state_download cannot be captured");
    auto* h = reinterpret_cast<ManyBlock*>(w->h_mem);
    hipError_t e = hipMemcpyAsync(&h->st, &w->view.block->st, sizeof(DeviceStep),
                                  hipMemcpyDeviceToHost, s);
    if (e == hipSuccess) e = hipStreamSynchronize(s);
    if (e != hipSuccess) return hip_fail(e, "state download");
    const DeviceStep& d = h->st;
    if (applied_steps) *applied_steps = d.t;
    if (skipped_steps) *skipped_steps = d.skipped;
    if (last_flag) *last_flag = d.last_flag;
    if (scaler) {
        scaler->scale = d.scale;
        scaler->min_scale = d.min_scale;
        scaler->backoff = d.backoff;
        scaler->growth = d.growth;
        scaler->window = d.window;
        scaler->good_steps = d.good_steps;
        scaler->dynamic = d.dynamic;
    }
    return ZERO_OK;
}

int zero_many_device_scale(zero_many_t* w, const double** out) {
    if (w == nullptr || out == nullptr) return fail(ZERO_ENULL, "many or out is NULL");
    const int rc = require_state(w);
    if (rc != ZERO_OK) return rc;
    *out = &w->view.block->st.scale;
    return ZERO_OK;
}

int zero_many_grad_norm(zero_many_t* w, double* sumsq, int32_t* flag, void* stream) {
    if (w == nullptr || sumsq == nullptr || flag == nullptr) {
        return fail(ZERO_ENULL, "many, sumsq or flag is NULL");
    }
    if ((reinterpret_cast<uintptr_t>(sumsq) & 7u) != 0 || !aligned4(flag)) {
        return fail(ZERO_EALIGN, "sumsq must be 8-byte and flag 4-byte aligned");
    }
    const int rc = require_bound(w, false);
    if (rc != ZERO_OK) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!w->captured && capturing(s)) w->captured = true;
    const hipError_t e = launch_many_norm(w->view, w->grad_dtype, sumsq, flag, s);
    return e == hipSuccess ? ZERO_OK : hip_fail(e, "gradient norm launch");
}

int zero_many_adam_step(zero_many_t* w, const zero_adam_hparams_t* hp, int32_t n_groups,
                        const int32_t* flag, const double* sumsq, double max_norm,
                        float* norm_out, void* stream) {
    if (w == nullptr || hp == nullptr) return fail(ZERO_ENULL, "many or hp is NULL");
    if (n_groups != w->n_groups) {
        return fail(ZERO_EINVAL, "n_groups must be the handle's number of groups");
    }
    ManyHparams all{};
    for (int32_t g = 0; g < n_groups; ++g) {
        const int rc = check_hparams(hp + g);
        if (rc != ZERO_OK) return rc;
        all.g[g] = hp[g];
    }
    if (!(max_norm >= 0)) return fail(ZERO_EINVAL, "max_norm must be >= 0 (0: no clipping)");
    if (max_norm > 0 && sumsq == nullptr) return fail(ZERO_ENULL, "max_norm needs sumsq");
    if (norm_out != nullptr && sumsq == nullptr) return fail(ZERO_ENULL, "norm_out needs sumsq");
    if ((reinterpret_cast<uintptr_t>(sumsq) & 7u) != 0 || !aligned4(flag) || !aligned4(norm_out)) {
        return fail(ZERO_EALIGN, "sumsq must be 8-byte, flag and norm_out 4-byte aligned");
    }
    int rc = require_bound(w, true);
    if (rc != ZERO_OK) return rc;
    if ((rc = require_state(w)) != ZERO_OK) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!w->captured_full && capturing(s)) w->captured = w->captured_full = true;
    hipError_t e = launch_many_prologue(w->view, all, n_groups, flag, sumsq, max_norm, norm_out, s);
    if (e != hipSuccess) return hip_fail(e, "step prologue launch");
    e = launch_many_adam(w->view, w->grad_dtype, w->param_dtype, w->bits, s);
    return e == hipSuccess ? ZERO_OK : hip_fail(e, "adam launch");
}

int zero_many_state_values(zero_many_t* w, float* exp_avg, float* exp_avg_sq, void* stream) {
    if (w == nullptr) return fail(ZERO_ENULL, "many is NULL");
    if (!aligned16(exp_avg) || !aligned16(exp_avg_sq)) {
        return fail(ZERO_EALIGN, "exp_avg and exp_avg_sq must be 16-byte aligned");
    }
    const int rc = require_bound(w, true);
    if (rc != ZERO_OK) return rc;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (!w->captured_full && capturing(s)) w->captured_full = true;
    const hipError_t e = launch_many_values(w->view, w->bits, exp_avg, exp_avg_sq, s);
    return e == hipSuccess ? ZERO_OK : hip_fail(e, "state values launch");
}

}  // extern "C"
