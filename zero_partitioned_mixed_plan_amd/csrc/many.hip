// Kernels of the many-tensor AdamW step: gradient norm, prologue, update with
// moments in fp32 or 8 bits, and the moments read back.
#include "device.h"
#include "many.h"

namespace zmi {
namespace {

constexpr int kWaves = kManyWaves;
constexpr int kThreads = kWaves * 64;

template <typename T>
__device__ __forceinline__ __attribute__((address_space(1))) T* gptr(uint64_t addr) {
    return reinterpret_cast<__attribute__((address_space(1))) T*>(addr);
}

// ------------------------------------------------------------ norm
// A workgroup sweeps tiles of kNormTile chunks, kNormVecs vectors of 16
// bytes under way in each thread; within a tile it walks the runs of chunks
// that one tensor holds.
constexpr int kNormTile = 2;
constexpr int kNormVecs = 4;

// Sum of squares and nonfinite test of one 16-byte vector.
template <int DT>
__device__ __forceinline__ void norm_vec(const u32x4& q, double& sum, bool& bad) {
    constexpr int per = DT == ZERO_F32 ? 4 : 8;
#pragma unroll
    for (int e = 0; e < per; ++e) {
        const uint32_t x = DT == ZERO_F32 ? q[e] : (q[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
        bad |= elem_nonfinite<DT>(x);
        const double g = static_cast<double>(grad_to_f32<DT>(x));
        sum = __builtin_fma(g, g, sum);  // the square is exact in fp64
    }
}

template <int DT>
__device__ __forceinline__ void norm_run(uint64_t base, int64_t e0, int64_t e1, double& sum,
                                         bool& bad) {
    constexpr int size = DT == ZERO_F32 ? 4 : 2, per = 16 / size;
    const uint64_t first = base + static_cast<uint64_t>(e0) * size;
    const int n = static_cast<int>(e1 - e0);
    // elements before the first aligned vector, and behind the last
    const int head = min(static_cast<int>((per - first % 16 / size) % per), n);
    const int nv = (n - head) / per;
    const int lane = static_cast<int>(threadIdx.x);
    const int tail = head + nv * per + lane;
    const int edge = lane < per ? (tail < n ? tail : -1) : (lane - per < head ? lane - per : -1);
    if (edge >= 0) {
        u32x4 q = {0, 0, 0, 0};
        q[0] = DT == ZERO_F32 ? *gptr<const uint32_t>(first + 4u * edge)
                              : *gptr<const uint16_t>(first + 2u * edge);
        norm_vec<DT>(q, sum, bad);
    }
    const uint64_t at = first + static_cast<uint64_t>(head) * size;
    for (int k0 = lane; k0 < nv; k0 += kThreads * kNormVecs) {
        u32x4 q[kNormVecs];
#pragma unroll
        for (int i = 0; i < kNormVecs; ++i) {
            const int k = k0 + i * kThreads;
            q[i] = u32x4{0, 0, 0, 0};
            if (k < nv) q[i] = __builtin_nontemporal_load(gptr<const u32x4>(at + 16u * k));
        }
#pragma unroll
        for (int i = 0; i < kNormVecs; ++i) norm_vec<DT>(q[i], sum, bad);
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
norm_kernel(const ManyView w) {
    __shared__ double lsum[kWaves];
    __shared__ int lbad[kWaves];
    double sum = 0;
    bool bad = false;
    for (int64_t c0 = int64_t(blockIdx.x) * kNormTile; c0 < w.n_chunks;
         c0 += int64_t(gridDim.x) * kNormTile) {
        const int64_t c1 = min(c0 + kNormTile, w.n_chunks);
        for (int64_t c = c0; c < c1;) {
            const ManyTensor& t = w.tensors[w.chunk_tensor[c]];
            const int64_t e0 = (c - t.chunk0) * kManyChunk;
            const int64_t e1 = min(e0 + (c1 - c) * kManyChunk, t.numel);
            if (t.grad != 0) norm_run<DT>(t.grad, e0, e1, sum, bad);
            c += (e1 - e0 + kManyChunk - 1) / kManyChunk;
        }
    }
    sum = wave_sum(sum);
    const bool any = __ballot(bad) != 0ull;
    if ((threadIdx.x & 63) == 0) {
        lsum[threadIdx.x >> 6] = sum;
        lbad[threadIdx.x >> 6] = any;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int f = 0;
        sum = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            sum += lsum[i];
            f |= lbad[i];
        }
        w.part[blockIdx.x] = sum;
        w.part_flag[blockIdx.x] = f;
    }
}

// One workgroup: the parts in a fixed order.
__global__ void __launch_bounds__(kThreads)
norm_join_kernel(const double* __restrict__ part, const int32_t* __restrict__ part_flag, int n,
                 double* __restrict__ sumsq, int32_t* __restrict__ flag) {
    __shared__ double lsum[kWaves];
    __shared__ int lbad[kWaves];
    double sum = 0;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kNormParts / kThreads; ++j) {
        const int i = j * kThreads + static_cast<int>(threadIdx.x);
        if (i < n) {
            sum += part[i];
            bad |= part_flag[i] != 0;
        }
    }
    sum = wave_sum(sum);
    const bool any = __ballot(bad) != 0ull;
    if ((threadIdx.x & 63) == 0) {
        lsum[threadIdx.x >> 6] = sum;
        lbad[threadIdx.x >> 6] = any;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int f = 0;
        sum = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            sum += lsum[i];
            f |= lbad[i];
        }
        *sumsq = sum;
        *flag = f;
    }
}

// ------------------------------------------------------------ prologue
__device__ __forceinline__ uint64_t mix64(uint64_t z) {
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}

// One wave, a thread per group: whether the step is skipped, the clip, the
// scalars of step t + 1 and its random key; then the loss-scale policy.
__global__ void __launch_bounds__(64)
many_prologue_kernel(ManyBlock* __restrict__ b, const ManyHparams hp, int n_groups,
                     const int32_t* __restrict__ flag, const double* __restrict__ sumsq,
                     double max_norm, float* __restrict__ norm_out) {
    DeviceStep d = b->st;
    const uint64_t seed = b->seed;
    __syncthreads();  // every thread has the old state before thread 0 writes the new one
    double norm = 0, coef = 1;
    if (sumsq != nullptr) {
        norm = sqrt(*sumsq) / d.scale;
        if (max_norm > 0) coef = fmin(1.0, max_norm / (norm + 1e-6));
    }
    const bool skip = (flag != nullptr && *flag != 0) || !(norm <= 1.7976931348623157e308);
    const int g = static_cast<int>(threadIdx.x);
    if (g < n_groups && !skip) {
        const zero_adam_hparams_t& h = hp.g[g];
        ManyScalars o;
        o.a = make_scalars(h.lr, h.beta1, h.beta2, h.eps, h.weight_decay, h.adamw,
                           static_cast<double>(d.t + 1), d.scale);
        o.a.inv_scale = static_cast<float>(coef / d.scale);
        o.adamw = h.adamw != 0;
        o._pad = 0;
        b->sc[g] = o;
    }
    if (g == 0) {
        if (norm_out != nullptr) {
            norm_out[0] = static_cast<float>(norm);
            norm_out[1] = static_cast<float>(coef);
        }
        b->skip = skip;
        b->key = static_cast<uint32_t>(
            mix64(seed + static_cast<uint64_t>(d.t + 1) * 0x9E3779B97F4A7C15ull));
        apply_scale_policy(d, skip);
        b->st = d;
    }
}

// ------------------------------------------------------------ update
// Four consecutive elements of a lane, wide where the tensor allows it.
__device__ __forceinline__ void load4(uint64_t base, int64_t e, int n, bool wide, float (&x)[4]) {
    if (wide) {
        const f32x4 q = __builtin_nontemporal_load(gptr<const f32x4>(base + 4 * e));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = q[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = i < n ? *gptr<const float>(base + 4 * (e + i)) : 0.f;
    }
}

__device__ __forceinline__ void store4(uint64_t base, int64_t e, int n, bool wide,
                                       const float (&x)[4]) {
    if (wide) {
        __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, gptr<f32x4>(base + 4 * e));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < n) *gptr<float>(base + 4 * (e + i)) = x[i];
        }
    }
}

template <int DT>
__device__ __forceinline__ void load_grad4(uint64_t base, int64_t e, int n, bool wide,
                                           float (&x)[4]) {
    if (DT == ZERO_F32) return load4(base, e, n, wide, x);
    if (wide) {
        const u32x2 q = __builtin_nontemporal_load(gptr<const u32x2>(base + 2 * e));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = grad_to_f32<DT>((q[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = i < n ? grad_to_f32<DT>(*gptr<const uint16_t>(base + 2 * (e + i))) : 0.f;
        }
    }
}

template <int DT>
__device__ __forceinline__ void store_half4(uint64_t base, int64_t e, int n, bool wide,
                                            const float (&x)[4]) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = f32_to_half<DT>(x[i]);
    if (wide) {
        __builtin_nontemporal_store(u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)}, gptr<u32x2>(base + 2 * e));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < n) *gptr<uint16_t>(base + 2 * (e + i)) = static_cast<uint16_t>(h[i]);
        }
    }
}

// Four codes as one word, element 0 in the low byte.
__device__ __forceinline__ uint32_t load_codes(uint64_t base, int64_t e, int n, bool wide) {
    if (wide) return __builtin_nontemporal_load(gptr<const uint32_t>(base + e));
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i < n) w |= static_cast<uint32_t>(*gptr<const uint8_t>(base + e + i)) << (8 * i);
    }
    return w;
}

__device__ __forceinline__ void store_codes(uint64_t base, int64_t e, int n, bool wide,
                                            uint32_t w) {
    if (wide) {
        __builtin_nontemporal_store(w, gptr<uint32_t>(base + e));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i < n) *gptr<uint8_t>(base + e + i) = static_cast<uint8_t>(w >> (8 * i));
        }
    }
}

__device__ __forceinline__ void unpack_m(uint32_t w, int scale, float (&m)[4]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    const float x[4] = {a[0], a[1], b[0], b[1]};
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = __builtin_ldexpf(x[i], scale - 134);
}

__device__ __forceinline__ void unpack_v(uint32_t w, int scale, float (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = __builtin_ldexpf(__uint_as_float(((w >> (8 * i)) & 0xFFu) << 20), scale - 31);
    }
}

// Exponent field of the largest |x| of the wave's block (NaNs aside).
__device__ __forceinline__ int block_exponent(const float (&x)[4]) {
    const float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    return static_cast<int>(__float_as_uint(wave_max(fmaxf(m, 0.f), 0.f)) >> 23);
}

__device__ __forceinline__ uint32_t pack_m(const float (&m)[4], int scale) {
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[i] = __builtin_ldexpf(m[i], 134 - scale);
        // what is not finite becomes NaN
        if (!(fabsf(x[i]) <= 256.f)) x[i] = NAN;
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
    return static_cast<uint32_t>(w);
}

// Random bits of the element pair `pair` of the padded order: 16 for its
// even element (low half), 16 for its odd one.
__device__ __forceinline__ uint32_t random_pair(uint64_t pair, uint32_t key) {
    const uint32_t hi = static_cast<uint32_t>(pair >> 32) * 0x6A09E667u;
    uint32_t x = static_cast<uint32_t>(pair) * 0x9E3779B1u + (key ^ hi);
    x ^= x >> 16;
    x *= 0xBB67AE85u;
    return x ^ (x >> 15);
}

__device__ __forceinline__ uint32_t pack_v(const float (&v)[4], int scale, uint64_t elem,
                                           uint32_t key) {
    const uint32_t r[2] = {random_pair(elem >> 1, key), random_pair((elem >> 1) + 1, key)};
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t bits = __float_as_uint(__builtin_ldexpf(v[i], 31 - scale)) & 0x7FFFFFFFu;
        const uint32_t rnd = (r[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
        uint32_t c = min((bits + (rnd << 4)) >> 20, 255u);
        if ((__float_as_uint(v[i]) & 0x7FFFFFFFu) != 0) c = max(c, 1u);
        else c = 0;
        w |= c << (8 * i);
    }
    return w;
}

// What a wave holds of one block: four consecutive elements a lane.
template <int GDT, int BITS>
struct Block {
    float g[4], p[4], m[4], v[4];
    uint32_t mc, vc;  // 8-bit codes
    int ms, vs;

    __device__ __forceinline__ void load(const ManyTensor& t, int64_t blk, int64_t e, int n,
                                         bool wide) {
        load_grad4<GDT>(t.grad, e, n, wide, g);
        load4(t.master, e, n, wide, p);
        if (BITS == 8) {
            ms = *gptr<const uint8_t>(t.m_scale + blk);
            vs = *gptr<const uint8_t>(t.v_scale + blk);
            mc = load_codes(t.m, e, n, wide);
            vc = load_codes(t.v, e, n, wide);
        } else {
            load4(t.m, e, n, wide, m);
            load4(t.v, e, n, wide, v);
        }
    }

    template <int PDT>
    __device__ __forceinline__ void step(const ManyTensor& t, const ManyScalars& sc, uint32_t key,
                                         int64_t blk, int64_t e, int n, bool wide) {
        if (BITS == 8) {
            unpack_m(mc, ms, m);
            unpack_v(vc, vs, v);
        }
        if (sc.adamw) {
#pragma unroll
            for (int i = 0; i < 4; ++i) adam_elem<true>(g[i], p[i], m[i], v[i], sc.a);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) adam_elem<false>(g[i], p[i], m[i], v[i], sc.a);
        }
        store4(t.master, e, n, wide, p);
        if (PDT != 0) store_half4<PDT>(t.param, e, n, wide, p);
        if (BITS == 8) {
            ms = block_exponent(m);
            vs = block_exponent(v);
            store_codes(t.m, e, n, wide, pack_m(m, ms));
            store_codes(t.v, e, n, wide, pack_v(v, vs, static_cast<uint64_t>(t.elem0 + e), key));
            if ((threadIdx.x & 63) == 0) {
                *gptr<uint8_t>(t.m_scale + blk) = static_cast<uint8_t>(ms);
                *gptr<uint8_t>(t.v_scale + blk) = static_cast<uint8_t>(vs);
            }
        } else {
            store4(t.m, e, n, wide, m);
            store4(t.v, e, n, wide, v);
        }
    }
};

// Wave w of a chunk takes its blocks w, w + 4, w + 8 and w + 12, so that a
// short tensor's blocks still spread over the waves.  Where all four are
// whole and aligned, everything they read is under way before any of it is
// used.
template <int GDT, int PDT, int BITS>
__global__ void __launch_bounds__(kThreads)
many_adam_kernel(const ManyView w) {
    const int64_t c = block_id();
    if (c >= w.n_chunks || w.block->skip != 0) return;
    const ManyTensor t = w.tensors[w.chunk_tensor[c]];
    if (t.grad == 0) return;
    const ManyScalars sc = w.block->sc[t.group];
    const uint32_t key = w.block->key;
    const int lane = static_cast<int>(threadIdx.x & 63);
    const int64_t chunk0 = (c - t.chunk0) * (kWaves * kManyBlocks);
    const int64_t blk0 = chunk0 + (threadIdx.x >> 6);
    if (t.wide && (chunk0 + kWaves * kManyBlocks) * kManyBlock <= t.numel) {
        Block<GDT, BITS> b[kManyBlocks];
#pragma unroll
        for (int i = 0; i < kManyBlocks; ++i) {
            const int64_t blk = blk0 + i * kWaves;
            b[i].load(t, blk, blk * kManyBlock + lane * 4, 4, true);
        }
#pragma unroll
        for (int i = 0; i < kManyBlocks; ++i) {
            const int64_t blk = blk0 + i * kWaves;
            b[i].template step<PDT>(t, sc, key, blk, blk * kManyBlock + lane * 4, 4, true);
            __builtin_amdgcn_sched_barrier(0);
        }
        return;
    }
#pragma unroll 1
    for (int i = 0; i < kManyBlocks; ++i) {
        const int64_t blk = blk0 + i * kWaves;
        if (blk * kManyBlock >= t.numel) return;
        const int64_t e = blk * kManyBlock + lane * 4;
        const int n = static_cast<int>(min(max(t.numel - e, int64_t(0)), int64_t(4)));
        const bool wide = t.wide && n == 4;
        Block<GDT, BITS> b;
        b.load(t, blk, e, n, wide);
        b.template step<PDT>(t, sc, key, blk, e, n, wide);
    }
}

// One block of one moment as fp32.
template <int BITS, bool SECOND>
__device__ __forceinline__ void moment4(const ManyTensor& t, int64_t blk, int64_t e, int n,
                                        bool wide, float (&x)[4]) {
    const uint64_t base = SECOND ? t.v : t.m;
    if (BITS == 32) return load4(base, e, n, wide, x);
    const uint32_t codes = load_codes(base, e, n, wide);
    const int scale = *gptr<const uint8_t>((SECOND ? t.v_scale : t.m_scale) + blk);
    if (SECOND) unpack_v(codes, scale, x);
    else unpack_m(codes, scale, x);
}

template <int BITS, bool SECOND>
__device__ __forceinline__ void write_values(const ManyTensor& t, int64_t chunk0, int64_t blk0,
                                             int lane, float* out) {
    const bool whole = t.wide && (chunk0 + kWaves * kManyBlocks) * kManyBlock <= t.numel;
    float x[kManyBlocks][4];
    if (whole) {
#pragma unroll
        for (int i = 0; i < kManyBlocks; ++i) {
            const int64_t blk = blk0 + i * kWaves;
            moment4<BITS, SECOND>(t, blk, blk * kManyBlock + lane * 4, 4, true, x[i]);
        }
    } else {
        for (int i = 0; i < kManyBlocks; ++i) {
            const int64_t blk = blk0 + i * kWaves, e = blk * kManyBlock + lane * 4;
            const int n = static_cast<int>(min(max(t.numel - e, int64_t(0)), int64_t(4)));
            if (blk * kManyBlock < t.numel) {
                moment4<BITS, SECOND>(t, blk, e, n, t.wide && n == 4, x[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kManyBlocks; ++i) {
        const int64_t blk = blk0 + i * kWaves;
        if (whole || blk * kManyBlock < t.numel) {
            __builtin_nontemporal_store(
                f32x4{x[i][0], x[i][1], x[i][2], x[i][3]},
                reinterpret_cast<f32x4*>(out + t.elem0 + blk * kManyBlock + lane * 4));
        }
    }
}

template <int BITS>
__global__ void __launch_bounds__(kThreads)
many_values_kernel(const ManyView w, float* __restrict__ mo, float* __restrict__ vo) {
    const int64_t c = block_id();
    if (c >= w.n_chunks) return;
    const ManyTensor t = w.tensors[w.chunk_tensor[c]];
    const int64_t chunk0 = (c - t.chunk0) * (kWaves * kManyBlocks);
    const int64_t blk0 = chunk0 + (threadIdx.x >> 6);
    const int lane = static_cast<int>(threadIdx.x & 63);
    if (mo != nullptr) write_values<BITS, false>(t, chunk0, blk0, lane, mo);
    if (vo != nullptr) write_values<BITS, true>(t, chunk0, blk0, lane, vo);
}

template <int GDT, int PDT>
void adam_bits(const ManyView& w, int bits, hipStream_t s) {
    const dim3 grid = grid_2d(w.n_chunks);
    if (bits == 8) {
        hipLaunchKernelGGL((many_adam_kernel<GDT, PDT, 8>), grid, dim3(kThreads), 0, s, w);
    } else {
        hipLaunchKernelGGL((many_adam_kernel<GDT, PDT, 32>), grid, dim3(kThreads), 0, s, w);
    }
}

template <int GDT>
void adam_param(const ManyView& w, int pdt, int bits, hipStream_t s) {
    if (pdt == 0) adam_bits<GDT, 0>(w, bits, s);
    else if (pdt == ZERO_F16) adam_bits<GDT, ZERO_F16>(w, bits, s);
    else adam_bits<GDT, ZERO_BF16>(w, bits, s);
}

}  // namespace

hipError_t launch_many_norm(const ManyView& w, int grad_dtype, double* sumsq, int32_t* flag,
                            hipStream_t s) {
    const int64_t tiles = (w.n_chunks + kNormTile - 1) / kNormTile;
    const int parts = static_cast<int>(tiles < kNormParts ? tiles : kNormParts);
    if (parts > 0) {
        const dim3 grid(static_cast<unsigned>(parts));
        if (grad_dtype == ZERO_F16) {
            hipLaunchKernelGGL(norm_kernel<ZERO_F16>, grid, dim3(kThreads), 0, s, w);
        } else if (grad_dtype == ZERO_BF16) {
            hipLaunchKernelGGL(norm_kernel<ZERO_BF16>, grid, dim3(kThreads), 0, s, w);
        } else {
            hipLaunchKernelGGL(norm_kernel<ZERO_F32>, grid, dim3(kThreads), 0, s, w);
        }
    }
    hipLaunchKernelGGL(norm_join_kernel, dim3(1), dim3(kThreads), 0, s, w.part, w.part_flag, parts,
                       sumsq, flag);
    return hipGetLastError();
}

hipError_t launch_many_prologue(const ManyView& w, const ManyHparams& hp, int n_groups,
                                const int32_t* flag, const double* sumsq, double max_norm,
                                float* norm_out, hipStream_t s) {
    hipLaunchKernelGGL(many_prologue_kernel, dim3(1), dim3(64), 0, s, w.block, hp, n_groups, flag,
                       sumsq, max_norm, norm_out);
    return hipGetLastError();
}

hipError_t launch_many_adam(const ManyView& w, int grad_dtype, int param_dtype, int state_bits,
                            hipStream_t s) {
    if (w.n_chunks <= 0) return hipSuccess;
    if (grad_dtype == ZERO_F16) adam_param<ZERO_F16>(w, param_dtype, state_bits, s);
    else if (grad_dtype == ZERO_BF16) adam_param<ZERO_BF16>(w, param_dtype, state_bits, s);
    else adam_param<ZERO_F32>(w, param_dtype, state_bits, s);
    return hipGetLastError();
}

hipError_t launch_many_values(const ManyView& w, int state_bits, float* m, float* v,
                              hipStream_t s) {
    if (w.n_chunks <= 0 || (m == nullptr && v == nullptr)) return hipSuccess;
    const dim3 grid = grid_2d(w.n_chunks);
    if (state_bits == 8) {
        hipLaunchKernelGGL(many_values_kernel<8>, grid, dim3(kThreads), 0, s, w, m, v);
    } else {
        hipLaunchKernelGGL(many_values_kernel<32>, grid, dim3(kThreads), 0, s, w, m, v);
    }
    return hipGetLastError();
}

}  // namespace zmi
