// Fine-tuning losses: log-probabilities of the labels, their gradient to the
// logits, the preference loss of pairs and the clipped policy loss, with
// their entry points.
#include <cmath>

#include "device.h"

namespace zmi {
namespace {

constexpr int kRowThreads = 256;  // of the per-pair and summing kernels
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A vector of 16 bytes at any element's address: rows start wherever their
// stride puts them.
template <int DT>
struct Elem {
    typedef uint16_t T;
    static constexpr int kPer = 8;
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
    static constexpr uint32_t kNegInf = DT == ZERO_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
};
template <>
struct Elem<ZERO_F32> {
    typedef uint32_t T;
    static constexpr int kPer = 4;
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(4)));
    static constexpr uint32_t kNegInf = 0xFF800000u;
};

template <int DT>
__device__ __forceinline__ typename Elem<DT>::T from_f32(float x) {
    if constexpr (DT == ZERO_F32) return __float_as_uint(x);
    else return f32_to_half<DT>(x);
}

// Element e of a vector.
template <int DT>
__device__ __forceinline__ float get(const u32x4& q, int e) {
    if constexpr (DT == ZERO_F32) return __uint_as_float(q[e]);
    if constexpr (DT == ZERO_BF16) {
        return __uint_as_float((e & 1) ? (q[e >> 1] & 0xFFFF0000u) : (q[e >> 1] << 16));
    }
    return grad_to_f32<DT>((e & 1) ? (q[e >> 1] >> 16) : (q[e >> 1] & 0xFFFFu));
}

template <int DT>
__device__ __forceinline__ u32x4 put(const float* d) {
    u32x4 q;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if constexpr (DT == ZERO_F32) q[w] = __float_as_uint(d[w]);
        else q[w] = uint32_t(f32_to_half<DT>(d[2 * w])) | (uint32_t(f32_to_half<DT>(d[2 * w + 1])) << 16);
    }
    return q;
}

// Vector k of a row; what lies behind the row's end is -inf.
template <int DT>
__device__ __forceinline__ u32x4 load_vec(const typename Elem<DT>::T* row, int vocab, int k) {
    constexpr int per = Elem<DT>::kPer;
    if (k * per + per <= vocab) {
        return __builtin_nontemporal_load(reinterpret_cast<const typename Elem<DT>::V*>(row + k * per));
    }
    u32x4 q = {Elem<DT>::kNegInf, Elem<DT>::kNegInf, Elem<DT>::kNegInf, Elem<DT>::kNegInf};
    for (int e = 0; k * per + e < vocab; ++e) {
        const uint32_t x = row[k * per + e];
        if constexpr (DT == ZERO_F32) q[e] = x;
        else q[e >> 1] = (e & 1) ? ((q[e >> 1] & 0xFFFFu) | (x << 16)) : ((q[e >> 1] & 0xFFFF0000u) | x);
    }
    return q;
}

template <int DT>
__device__ __forceinline__ void store_vec(typename Elem<DT>::T* row, int vocab, int k,
                                          const u32x4& q) {
    constexpr int per = Elem<DT>::kPer;
    if (k * per + per <= vocab) {
        __builtin_nontemporal_store(q, reinterpret_cast<typename Elem<DT>::V*>(row + k * per));
        return;
    }
    for (int e = 0; k * per + e < vocab; ++e) {
        if constexpr (DT == ZERO_F32) row[k * per + e] = q[e];
        else row[k * per + e] = static_cast<uint16_t>((e & 1) ? (q[e >> 1] >> 16) : q[e >> 1]);
    }
}

// Reductions over the T threads of a row (T = 64: one wave, no LDS; larger:
// the whole workgroup).
template <int T>
__device__ __forceinline__ float row_max(float x, float* lds) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor(x, d));
    if (T == 64) return x;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = lds[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) x = fmaxf(x, lds[w]);
    return x;
}

template <int T>
__device__ __forceinline__ double row_sum(double x, double* lds) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
    if (T == 64) return x;
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = lds[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) x += lds[w];
    return x;
}

template <int W>
__device__ __forceinline__ double block_sum(double x, double* lds) { return row_sum<64 * W>(x, lds); }

// The largest finite value below: a base that an exponential's argument can
// be taken from even where a row holds -inf alone (its sum is then 0).
constexpr float kLowest = -3.402823466e38f;

// Largest raw logit and the sum of exp((raw - largest) * inv_t) of one row,
// read once: each thread keeps a running maximum and sum and rescales when
// a group of vectors brings a larger value.
template <int DT, int T>
__device__ __forceinline__ void row_stats(const typename Elem<DT>::T* row, int vocab, float c,
                                          int lane, float* lmax, double* lsum, float* top,
                                          double* sum) {
    constexpr int per = Elem<DT>::kPer, kGroup = 4;
    const int nv = (vocab + per - 1) / per;
    float m = kLowest, s = 0.f;
    for (int k0 = lane; k0 < nv; k0 += T * kGroup) {
        u32x4 q[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            const int k = k0 + i * T;
            if (k < nv) q[i] = load_vec<DT>(row, vocab, k);
            else q[i] = u32x4{Elem<DT>::kNegInf, Elem<DT>::kNegInf, Elem<DT>::kNegInf, Elem<DT>::kNegInf};
        }
        float g = m;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
#pragma unroll
            for (int e = 0; e < per; ++e) g = fmaxf(g, get<DT>(q[i], e));
        }
        s *= exp2_fast((m - g) * c);
        m = g;
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
#pragma unroll
            for (int e = 0; e < per; ++e) s += exp2_fast((get<DT>(q[i], e) - m) * c);
        }
    }
    *top = row_max<T>(m, lmax);
    *sum = row_sum<T>(static_cast<double>(s * exp2_fast((m - *top) * c)), lsum);
}

// log-probability of the label, in fp64: -inf when the row holds nothing,
// NaN for a label outside the vocabulary.
template <int DT>
__device__ __forceinline__ double label_logp(const typename Elem<DT>::T* row, int64_t label,
                                             int vocab, float inv_t, double lse) {
    if (label >= vocab) return NAN;
    if (lse == -INFINITY) return -INFINITY;
    return static_cast<double>(grad_to_f32<DT>(row[label])) * static_cast<double>(inv_t) - lse;
}

// Rows a workgroup of the row kernels takes, and its threads.
template <int T>
constexpr int rows_per_group() { return T == 64 ? 4 : 1; }

template <int DT, int T>
__global__ void __launch_bounds__(T * rows_per_group<T>())
logp_kernel(const typename Elem<DT>::T* __restrict__ logits, int64_t rows, int vocab,
            int64_t stride, const int64_t* __restrict__ labels, float inv_t,
            float* __restrict__ logp, float* __restrict__ lse) {
    __shared__ float lmax[T / 64];
    __shared__ double lsum[T / 64];
    const int lane = static_cast<int>(threadIdx.x) % T;
    const int64_t r = block_id() * rows_per_group<T>() + threadIdx.x / T;
    if (r >= rows) return;
    const int64_t label = labels[r];
    if (label < 0) {
        if (lane == 0) {
            logp[r] = 0.f;
            if (lse != nullptr) lse[r] = 0.f;
        }
        return;
    }
    const auto* row = logits + r * stride;
    float top;
    double sum;
    row_stats<DT, T>(row, vocab, inv_t * kLog2e, lane, lmax, lsum, &top, &sum);
    if (lane == 0) {
        const double l = static_cast<double>(top) * static_cast<double>(inv_t) + log(sum);
        logp[r] = static_cast<float>(label_logp<DT>(row, label, vocab, inv_t, l));
        if (lse != nullptr) lse[r] = static_cast<float>(l);
    }
}

// Zeros over one row.
template <int DT, int T>
__device__ __forceinline__ void zero_row(typename Elem<DT>::T* out, int vocab, int lane) {
    constexpr int per = Elem<DT>::kPer;
    const int nv = (vocab + per - 1) / per;
    for (int k = lane; k < nv; k += T) store_vec<DT>(out, vocab, k, u32x4{0, 0, 0, 0});
}

// One vector of gradient: -g exp2((raw - base) c - shift).
template <int DT>
__device__ __forceinline__ u32x4 grad_vec(const u32x4& q, float base, float c, float shift,
                                          float g) {
    float d[Elem<DT>::kPer];
#pragma unroll
    for (int e = 0; e < Elem<DT>::kPer; ++e) {
        d[e] = -g * exp2_fast((get<DT>(q, e) - base) * c - shift);
    }
    return put<DT>(d);
}

template <int DT, int T>
__global__ void __launch_bounds__(T * rows_per_group<T>())
logp_grad_kernel(const typename Elem<DT>::T* logits, int64_t rows, int vocab, int64_t stride,
                 const int64_t* __restrict__ labels, float inv_t, const float* __restrict__ lse,
                 const float* __restrict__ dlogp, typename Elem<DT>::T* dlogits,
                 int64_t out_stride) {
    constexpr int per = Elem<DT>::kPer, kGroup = 4;
    const int lane = static_cast<int>(threadIdx.x) % T;
    const int64_t r = block_id() * rows_per_group<T>() + threadIdx.x / T;
    if (r >= rows) return;
    const int64_t label = labels[r];
    const float g = label < 0 ? 0.f : dlogp[r] * inv_t;
    const float l = g == 0.f ? 0.f : lse[r];
    const auto* row = logits + r * stride;
    auto* out = dlogits + r * out_stride;
    if (g == 0.f || l == -INFINITY) return zero_row<DT, T>(out, vocab, lane);
    const float c = inv_t * kLog2e, shift = l * kLog2e;
    const int nv = (vocab + per - 1) / per;
    const int mine = label < vocab ? static_cast<int>(label) / per : -1;
    for (int k0 = lane; k0 < nv; k0 += T * kGroup) {
        u32x4 q[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            const int k = k0 + i * T;
            if (k < nv) q[i] = load_vec<DT>(row, vocab, k);
        }
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
            const int k = k0 + i * T;
            if (k < nv) store_vec<DT>(out, vocab, k, grad_vec<DT>(q[i], 0.f, c, shift, g));
            if (k == mine) {
                const int e = static_cast<int>(label) % per;
                float x = 0.f;
#pragma unroll
                for (int j = 0; j < per; ++j) x = j == e ? get<DT>(q[i], j) : x;
                out[label] = from_f32<DT>(g * (1.f - exp2_fast(x * c - shift)));
            }
        }
    }
}

// ------------------------------------------------------------ preference
__device__ __forceinline__ double softplus(double y) {
    return fmax(y, 0.0) + log1p(exp(-fabs(y)));
}

__global__ void __launch_bounds__(kRowThreads)
preference_kernel(const float* __restrict__ logp, const float* __restrict__ ref,
                  const int64_t* __restrict__ labels, int64_t rows,
                  const int64_t* __restrict__ seq, int64_t pairs, const zero_preference_t cfg,
                  double scale_host, const double* __restrict__ scale_dev,
                  float* __restrict__ pair_loss, float* __restrict__ rewards,
                  float* __restrict__ dlogp) {
    __shared__ double lds[4][kRowThreads / 64];
    __shared__ float slope[2];
    const int64_t i = block_id();
    if (i >= pairs) return;
    int64_t a[2], b[2];
    double d[2], n[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        // offsets outside [0, rows] would reach past the buffers
        a[s] = min(max(seq[2 * i + s], int64_t(0)), rows);
        b[s] = min(max(seq[2 * i + s + 1], int64_t(0)), rows);
        double sum = 0, cnt = 0;
        for (int64_t t = a[s] + threadIdx.x; t < b[s]; t += kRowThreads) {
            if (labels != nullptr && labels[t] < 0) continue;
            sum += static_cast<double>(logp[t]) - (ref != nullptr ? static_cast<double>(ref[t]) : 0.0);
            cnt += 1;
        }
        d[s] = block_sum<kRowThreads / 64>(sum, lds[2 * s]);
        n[s] = block_sum<kRowThreads / 64>(cnt, lds[2 * s + 1]);
        if (!cfg.average || n[s] < 1) n[s] = 1;
        d[s] /= n[s];
    }
    if (threadIdx.x == 0) {
        const double beta = cfg.beta, e = cfg.label_smoothing, delta = d[0] - d[1];
        double loss, dd;
        if (cfg.kind == ZERO_PREF_SQUARED) {
            const double u = delta - 1.0 / (2.0 * beta);
            loss = u * u;
            dd = 2.0 * u;
        } else {
            const double h = beta * delta;
            loss = (1.0 - e) * softplus(-h) + e * softplus(h);
            dd = beta * (e / (1.0 + exp(-h)) - (1.0 - e) / (1.0 + exp(h)));
        }
        pair_loss[i] = static_cast<float>(loss);
        rewards[2 * i] = static_cast<float>(beta * d[0]);
        rewards[2 * i + 1] = static_cast<float>(beta * d[1]);
        const double k = (scale_dev != nullptr ? *scale_dev : scale_host) * cfg.norm * dd;
        slope[0] = static_cast<float>(k / n[0]);
        slope[1] = static_cast<float>(-k / n[1]);
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        for (int64_t t = a[s] + threadIdx.x; t < b[s]; t += kRowThreads) {
            dlogp[t] = labels != nullptr && labels[t] < 0 ? 0.f : slope[s];
        }
    }
}

// One workgroup: loss[0] = norm * the sum of n values.
__global__ void __launch_bounds__(kRowThreads)
sum_kernel(const float* __restrict__ x, int64_t n, double norm, float* __restrict__ loss) {
    __shared__ double lds[kRowThreads / 64];
    double s = 0;
    for (int64_t i = threadIdx.x; i < n; i += kRowThreads) s += static_cast<double>(x[i]);
    s = block_sum<kRowThreads / 64>(s, lds);
    if (threadIdx.x == 0) *loss = static_cast<float>(norm * s);
}

// ------------------------------------------------------------ policy
struct PolicyTerms {
    float pg, kl, clipped, weight;
};

// The terms of one token and the gradient of its log-probability.
__device__ __forceinline__ double policy_token(double logp, float old, const float* ref, float adv,
                                               float weight, const zero_policy_t& cfg,
                                               PolicyTerms* out) {
    const double a = adv, r = exp(logp - static_cast<double>(old));
    const double lo = 1.0 - static_cast<double>(cfg.clip_low);
    const double hi = 1.0 + static_cast<double>(cfg.clip_high);
    const double kept = r * a, cut = fmin(fmax(r, lo), hi) * a;
    const bool clipped = kept > cut;
    double kl = 0, dkl = 0;
    if (ref != nullptr) {
        const double q = static_cast<double>(*ref) - logp;
        const double em = expm1(q);
        kl = em - q;
        dkl = -em;
    }
    out->pg = static_cast<float>(-(clipped ? cut : kept));
    out->kl = static_cast<float>(kl);
    out->clipped = clipped ? 1.f : 0.f;
    out->weight = weight;
    return (clipped ? 0.0 : -kept) + static_cast<double>(cfg.kl_coef) * dkl;
}

// What every thread of a row needs for its gradient.
struct RowGrad {
    float base, c, shift, g, at_label;
};

// The terms of row r from its statistics; the row's gradient is
// -g exp2((raw - base) c - shift), and at_label at the label.
template <int DT>
__device__ __forceinline__ RowGrad policy_row(const typename Elem<DT>::T* row, int64_t r,
                                              int64_t label, int vocab, float top, double sum,
                                              const float* old, const float* ref, const float* adv,
                                              const float* weight, const zero_policy_t& cfg,
                                              double scale, float* logp, PolicyTerms* terms) {
    const double lsum = log(sum);
    const double lse = static_cast<double>(top) * static_cast<double>(cfg.inv_temperature) + lsum;
    const double lp = label_logp<DT>(row, label, vocab, cfg.inv_temperature, lse);
    const float w = weight != nullptr ? weight[r] : 1.f;
    PolicyTerms t{0.f, 0.f, 0.f, 0.f};
    float g = 0.f;
    if (w != 0.f) {
        g = static_cast<float>(
            policy_token(lp, old[r], ref != nullptr ? ref + r : nullptr, adv[r], w, cfg, &t) *
            (scale * cfg.norm * static_cast<double>(w)));
    }
    logp[r] = static_cast<float>(lp);
    terms[r] = t;
    RowGrad o;
    o.base = top;
    o.c = cfg.inv_temperature * kLog2e;
    o.shift = static_cast<float>(lsum * 1.4426950408889634074);
    o.g = lse == -INFINITY ? 0.f : g * cfg.inv_temperature;
    o.at_label = o.g * static_cast<float>(-expm1(lp));
    return o;
}

// Writes a row of gradient from a source of its vectors.
template <int DT, int T>
__device__ __forceinline__ void patch_label(typename Elem<DT>::T* out, int64_t label, int vocab,
                                            int k, float at_label) {
    if (label < vocab && k == static_cast<int>(label) / Elem<DT>::kPer) {
        out[label] = from_f32<DT>(at_label);
    }
}

// VPT > 0: the row stays in registers, VPT vectors a thread, between its
// statistics and its gradient.  VPT = 0: it is read twice.
template <int DT, int T, int VPT>
__global__ void __launch_bounds__(T * rows_per_group<T>())
policy_kernel(const typename Elem<DT>::T* logits, int64_t rows, int vocab, int64_t stride,
              const int64_t* __restrict__ labels, const float* __restrict__ old,
              const float* __restrict__ ref, const float* __restrict__ adv,
              const float* __restrict__ weight, const zero_policy_t cfg, double scale_host,
              const double* __restrict__ scale_dev, float* __restrict__ logp,
              PolicyTerms* __restrict__ terms, typename Elem<DT>::T* dlogits, int64_t out_stride) {
    __shared__ float lmax[T / 64];
    __shared__ double lsum[T / 64];
    __shared__ RowGrad share[rows_per_group<T>()];
    constexpr int per = Elem<DT>::kPer;
    const int lane = static_cast<int>(threadIdx.x) % T;
    const int64_t r = block_id() * rows_per_group<T>() + threadIdx.x / T;
    if (r >= rows) return;
    const int64_t label = labels[r];
    const auto* row = logits + r * stride;
    auto* out = dlogits + r * out_stride;
    if (label < 0) {
        if (lane == 0) {
            logp[r] = 0.f;
            terms[r] = PolicyTerms{0.f, 0.f, 0.f, 0.f};
        }
        return zero_row<DT, T>(out, vocab, lane);
    }
    const int nv = (vocab + per - 1) / per;
    const float c = cfg.inv_temperature * kLog2e;
    float top;
    double sum;
    u32x4 q[VPT > 0 ? VPT : 1];
    if (VPT > 0) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int k = lane + i * T;
            if (k < nv) q[i] = load_vec<DT>(row, vocab, k);
            else q[i] = u32x4{Elem<DT>::kNegInf, Elem<DT>::kNegInf, Elem<DT>::kNegInf, Elem<DT>::kNegInf};
        }
        float m = kLowest, s = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int e = 0; e < per; ++e) m = fmaxf(m, get<DT>(q[i], e));
        }
        top = row_max<T>(m, lmax);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
#pragma unroll
            for (int e = 0; e < per; ++e) s += exp2_fast((get<DT>(q[i], e) - top) * c);
        }
        sum = row_sum<T>(static_cast<double>(s), lsum);
    } else {
        row_stats<DT, T>(row, vocab, c, lane, lmax, lsum, &top, &sum);
    }
    const int slot = T == 64 ? static_cast<int>(threadIdx.x / T) : 0;
    if (lane == 0) {
        share[slot] = policy_row<DT>(row, r, label, vocab, top, sum, old, ref, adv, weight, cfg,
                                     scale_dev != nullptr ? *scale_dev : scale_host, logp, terms);
    }
    // T = 64: the row's own wave wrote its slot
    if (T > 64) __syncthreads();
    else __builtin_amdgcn_wave_barrier();
    const RowGrad o = share[slot];
    if (o.g == 0.f) return zero_row<DT, T>(out, vocab, lane);
    if (VPT > 0) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int k = lane + i * T;
            if (k >= nv) break;
            store_vec<DT>(out, vocab, k, grad_vec<DT>(q[i], o.base, o.c, o.shift, o.g));
            patch_label<DT, T>(out, label, vocab, k, o.at_label);
        }
    } else {
        for (int k = lane; k < nv; k += T) {
            const u32x4 x = load_vec<DT>(row, vocab, k);
            store_vec<DT>(out, vocab, k, grad_vec<DT>(x, o.base, o.c, o.shift, o.g));
            patch_label<DT, T>(out, label, vocab, k, o.at_label);
        }
    }
}

// One workgroup: the four sums of the batch.
__global__ void __launch_bounds__(kRowThreads)
policy_sum_kernel(const PolicyTerms* __restrict__ terms, int64_t rows, double norm, double kl_coef,
                  float* __restrict__ loss) {
    __shared__ double lds[3][kRowThreads / 64];
    double s[3] = {0, 0, 0};
    for (int64_t i = threadIdx.x; i < rows; i += kRowThreads) {
        const PolicyTerms t = terms[i];
        const double w = t.weight;
        if (w == 0) continue;
        s[0] += w * static_cast<double>(t.pg);
        s[1] += w * static_cast<double>(t.kl);
        s[2] += w * static_cast<double>(t.clipped);
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) s[k] = norm * block_sum<kRowThreads / 64>(s[k], lds[k]);
    if (threadIdx.x == 0) {
        loss[0] = static_cast<float>(s[0] + kl_coef * s[1]);
        loss[1] = static_cast<float>(s[0]);
        loss[2] = static_cast<float>(s[1]);
        loss[3] = static_cast<float>(s[2]);
    }
}

// ------------------------------------------------------------ checks
int elem_bytes(int32_t dtype) { return dtype == ZERO_F32 ? 4 : 2; }

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_matrix(const void* logits, int32_t dtype, int64_t rows, int64_t vocab, int64_t stride,
                 const int64_t* labels, float inv_temperature) {
    if (!valid_grad_dtype(dtype)) {
        return fail(ZERO_EINVAL, "dtype must be ZERO_F16, ZERO_BF16 or ZERO_F32");
    }
    if (rows < 0) return fail(ZERO_EINVAL, "rows must be >= 0");
    if (vocab < 1 || vocab > (int64_t(1) << 30)) {
        return fail(ZERO_EINVAL, "vocab must be in [1, 2^30]");
    }
    if (stride < vocab) return fail(ZERO_EINVAL, "row_stride must be >= vocab");
    if (rows > 0 && stride > (int64_t(1) << 60) / rows) {
        return fail(ZERO_EINVAL, "rows * row_stride is out of range");
    }
    if (!(std::isfinite(inv_temperature) && inv_temperature > 0)) {
        return fail(ZERO_EINVAL, "inv_temperature must be finite and > 0");
    }
    if (rows > 0 && (logits == nullptr || labels == nullptr)) {
        return fail(ZERO_ENULL, "logits and labels must be non-NULL");
    }
    if (!aligned_to(logits, elem_bytes(dtype)) || !aligned_to(labels, 8)) {
        return fail(ZERO_EALIGN, "logits must be aligned to their element, labels to 8 bytes");
    }
    return ZERO_OK;
}

int check_out_matrix(const void* logits, int64_t stride, const void* dlogits, int32_t dtype,
                     int64_t rows, int64_t vocab, int64_t out_stride) {
    if (out_stride < vocab) return fail(ZERO_EINVAL, "dlogits_stride must be >= vocab");
    if (rows > 0 && out_stride > (int64_t(1) << 60) / rows) {
        return fail(ZERO_EINVAL, "rows * dlogits_stride is out of range");
    }
    if (rows > 0 && dlogits == nullptr) return fail(ZERO_ENULL, "dlogits is NULL");
    if (!aligned_to(dlogits, elem_bytes(dtype))) {
        return fail(ZERO_EALIGN, "dlogits must be aligned to its element");
    }
    if (rows > 0 && dlogits == logits && out_stride != stride) {
        return fail(ZERO_EINVAL, "an in-place gradient needs the logits' row stride");
    }
    return ZERO_OK;
}

int check_floats(std::initializer_list<const float*> ps, bool required) {
    for (const float* p : ps) {
        if (required && p == nullptr) return fail(ZERO_ENULL, "a required array is NULL");
        if (!aligned4(p)) return fail(ZERO_EALIGN, "float arrays must be 4-byte aligned");
    }
    return ZERO_OK;
}

int check_loss_scale(double loss_scale, const double* dev, double norm) {
    if (dev == nullptr && !(std::isfinite(loss_scale) && loss_scale > 0)) {
        return fail(ZERO_EINVAL, "loss_scale must be finite and > 0");
    }
    if (!aligned_to(dev, 8)) return fail(ZERO_EALIGN, "loss_scale_dev must be 8-byte aligned");
    if (!std::isfinite(norm)) return fail(ZERO_EINVAL, "norm must be finite");
    return ZERO_OK;
}

int launched(const char* what) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? ZERO_OK : hip_fail(e, what);
}

template <int N>
using Const = std::integral_constant<int, N>;

// Calls f with the dtype as a compile-time constant.
template <typename F>
void with_dtype(int32_t dtype, F f) {
    if (dtype == ZERO_F16) f(Const<ZERO_F16>());
    else if (dtype == ZERO_BF16) f(Const<ZERO_BF16>());
    else f(Const<ZERO_F32>());
}

// Calls f with the threads that take a row of nv vectors.
template <typename F>
void with_threads(int64_t nv, int64_t rows, F f) {
    if (nv <= 64 * 8 && rows >= 2048) f(Const<64>());
    else if (nv <= 256 * 16) f(Const<256>());
    else if (nv <= 512 * 16) f(Const<512>());
    else f(Const<1024>());
}

// The same for a kernel that keeps the row in registers: threads and
// vectors per thread (0: the row does not fit).
template <typename F>
void with_row_shape(int64_t nv, int64_t rows, F f) {
    if (nv <= 64 * 8 && rows >= 2048) f(Const<64>(), Const<8>());
    else if (nv <= 256 * 4) f(Const<256>(), Const<4>());
    else if (nv <= 256 * 8) f(Const<256>(), Const<8>());
    else if (nv <= 256 * 16) f(Const<256>(), Const<16>());
    else if (nv <= 512 * 16) f(Const<512>(), Const<16>());
    else if (nv <= 1024 * 16) f(Const<1024>(), Const<16>());
    else f(Const<1024>(), Const<0>());
}

int64_t vectors(int32_t dtype, int64_t vocab) {
    const int64_t per = dtype == ZERO_F32 ? 4 : 8;
    return (vocab + per - 1) / per;
}

template <int T>
dim3 row_grid(int64_t rows) {
    return grid_2d((rows + rows_per_group<T>() - 1) / rows_per_group<T>());
}
template <int T>
dim3 row_block() { return dim3(T * rows_per_group<T>()); }

}  // namespace
}  // namespace zmi

using namespace zmi;

extern "C" {

int zero_token_logp(const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                    int64_t row_stride, const int64_t* labels, float inv_temperature,
                    float* logp, float* lse, void* stream) {
    int rc = check_matrix(logits, dtype, rows, vocab, row_stride, labels, inv_temperature);
    if (rc != ZERO_OK) return rc;
    if ((rc = check_floats({logp}, rows > 0)) != ZERO_OK) return rc;
    if ((rc = check_floats({lse}, false)) != ZERO_OK) return rc;
    if (rows == 0) return ZERO_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        with_threads(vectors(dtype, vocab), rows, [&](auto threads) {
            constexpr int T = decltype(threads)::value;
            hipLaunchKernelGGL((logp_kernel<DT, T>), row_grid<T>(rows), row_block<T>(), 0, s,
                               static_cast<const typename Elem<DT>::T*>(logits), rows,
                               static_cast<int>(vocab), row_stride, labels, inv_temperature, logp,
                               lse);
        });
    });
    return launched("log-probability launch");
}

int zero_token_logp_grad(const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                         int64_t row_stride, const int64_t* labels, float inv_temperature,
                         const float* lse, const float* dlogp, void* dlogits,
                         int64_t dlogits_stride, void* stream) {
    int rc = check_matrix(logits, dtype, rows, vocab, row_stride, labels, inv_temperature);
    if (rc != ZERO_OK) return rc;
    rc = check_out_matrix(logits, row_stride, dlogits, dtype, rows, vocab, dlogits_stride);
    if (rc != ZERO_OK) return rc;
    if ((rc = check_floats({lse, dlogp}, rows > 0)) != ZERO_OK) return rc;
    if (rows == 0) return ZERO_OK;
    hipStream_t s = static_cast<hipStream_t>(stream);
    with_dtype(dtype, [&](auto dt) {
        constexpr int DT = decltype(dt)::value;
        with_threads(vectors(dtype, vocab), rows, [&](auto threads) {
            constexpr int T = decltype(threads)::value;
            hipLaunchKernelGGL((logp_grad_kernel<DT, T>), row_grid<T>(rows), row_block<T>(), 0, s,
                               static_cast<const typename Elem<DT>::T*>(logits), rows,
                               static_cast<int>(vocab), row_stride, labels, inv_temperature, lse,
                               dlogp, static_cast<typename Elem<DT>::T*>(dlogits), dlogits_stride);
        });
    });
    return launched("log-probability gradient launch");
}

int zero_preference_loss(const float* logp, const float* ref_logp, const int64_t* labels,
                         int64_t rows, const int64_t* seq_offsets, int64_t pairs,
                         const zero_preference_t* cfg, double loss_scale,
                         const double* loss_scale_dev, float* loss, float* pair_loss,
                         float* rewards, float* dlogp, void* stream) {
    if (cfg == nullptr || loss == nullptr) return fail(ZERO_ENULL, "cfg or loss is NULL");
    if (rows < 0 || pairs < 0 || pairs > (int64_t(1) << 32)) {
        return fail(ZERO_EINVAL, "rows must be >= 0 and pairs in [0, 2^32]");
    }
    if (!(std::isfinite(cfg->beta) && cfg->beta > 0) ||
        !(cfg->label_smoothing >= 0 && cfg->label_smoothing < 1) ||
        (cfg->kind != ZERO_PREF_SIGMOID && cfg->kind != ZERO_PREF_SQUARED)) {
        return fail(ZERO_EINVAL, "beta must be > 0, label_smoothing in [0, 1) and kind one of "
                                 "enum zero_preference_kind");
    }
    if (cfg->kind == ZERO_PREF_SQUARED && cfg->label_smoothing != 0) {
        return fail(ZERO_EINVAL, "label_smoothing belongs to the sigmoid kind");
    }
    int rc = check_loss_scale(loss_scale, loss_scale_dev, cfg->norm);
    if (rc != ZERO_OK) return rc;
    if ((rc = check_floats({logp, dlogp}, rows > 0 && pairs > 0)) != ZERO_OK) return rc;
    if ((rc = check_floats({pair_loss, rewards}, pairs > 0)) != ZERO_OK) return rc;
    if ((rc = check_floats({ref_logp, loss}, false)) != ZERO_OK) return rc;
    if (pairs > 0 && seq_offsets == nullptr) return fail(ZERO_ENULL, "seq_offsets is NULL");
    if (!aligned_to(labels, 8) || !aligned_to(seq_offsets, 8)) {
        return fail(ZERO_EALIGN, "labels and seq_offsets must be 8-byte aligned");
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (pairs > 0) {
        hipLaunchKernelGGL(preference_kernel, grid_2d(pairs), dim3(kRowThreads), 0, s, logp,
                           ref_logp, labels, rows, seq_offsets, pairs, *cfg, loss_scale,
                           loss_scale_dev, pair_loss, rewards, dlogp);
    }
    hipLaunchKernelGGL(sum_kernel, dim3(1), dim3(kRowThreads), 0, s, pair_loss, pairs, cfg->norm,
                       loss);
    return launched("preference loss launch");
}

int zero_policy_loss(const void* logits, int32_t dtype, int64_t rows, int64_t vocab,
                     int64_t row_stride, const int64_t* labels, const float* old_logp,
                     const float* ref_logp, const float* advantage, const float* weight,
                     const zero_policy_t* cfg, double loss_scale, const double* loss_scale_dev,
                     float* logp, float* terms, float* loss, void* dlogits,
                     int64_t dlogits_stride, void* stream) {
    if (cfg == nullptr || loss == nullptr) return fail(ZERO_ENULL, "cfg or loss is NULL");
    int rc = check_matrix(logits, dtype, rows, vocab, row_stride, labels, cfg->inv_temperature);
    if (rc != ZERO_OK) return rc;
    rc = check_out_matrix(logits, row_stride, dlogits, dtype, rows, vocab, dlogits_stride);
    if (rc != ZERO_OK) return rc;
    if (!(cfg->clip_low >= 0 && cfg->clip_low < 1) ||
        !(std::isfinite(cfg->clip_high) && cfg->clip_high >= 0) ||
        !(std::isfinite(cfg->kl_coef) && cfg->kl_coef >= 0)) {
        return fail(ZERO_EINVAL, "clip_low must be in [0, 1), clip_high and kl_coef >= 0");
    }
    if (ref_logp == nullptr && cfg->kl_coef != 0) {
        return fail(ZERO_EINVAL, "kl_coef needs ref_logp");
    }
    if ((rc = check_loss_scale(loss_scale, loss_scale_dev, cfg->norm)) != ZERO_OK) return rc;
    if ((rc = check_floats({old_logp, advantage, logp, terms}, rows > 0)) != ZERO_OK) return rc;
    if ((rc = check_floats({ref_logp, weight, loss}, false)) != ZERO_OK) return rc;
    if (!aligned16(terms)) return fail(ZERO_EALIGN, "terms must be 16-byte aligned");
    hipStream_t s = static_cast<hipStream_t>(stream);
    auto* t = reinterpret_cast<PolicyTerms*>(terms);
    if (rows > 0) {
        with_dtype(dtype, [&](auto dt) {
            constexpr int DT = decltype(dt)::value;
            with_row_shape(vectors(dtype, vocab), rows, [&](auto threads, auto vecs) {
                constexpr int T = decltype(threads)::value, V = decltype(vecs)::value;
                hipLaunchKernelGGL((policy_kernel<DT, T, V>), row_grid<T>(rows), row_block<T>(), 0,
                                   s, static_cast<const typename Elem<DT>::T*>(logits), rows,
                                   static_cast<int>(vocab), row_stride, labels, old_logp, ref_logp,
                                   advantage, weight, *cfg, loss_scale, loss_scale_dev, logp, t,
                                   static_cast<typename Elem<DT>::T*>(dlogits), dlogits_stride);
            });
        });
    }
    hipLaunchKernelGGL(policy_sum_kernel, dim3(1), dim3(kRowThreads), 0, s, t, rows, cfg->norm,
                       static_cast<double>(cfg->kl_coef), loss);
    return launched("policy loss launch");
}

}  // extern "C"
