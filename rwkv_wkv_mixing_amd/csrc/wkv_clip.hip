// The norm of all gradients together, and the gradients scaled so that it is at most max_norm:
//     norm = sqrt(sum over the tensors of the sums of their squares),  g' = g min(1, max_norm / (norm + eps))
// Two passes over memory, which is what bounds them (1.4 GB in bf16 and float32: sums 232 us, 6.1 TB/s, scaling 510 us,
// 5.5 TB/s read and written); the second one mostly reads from the last level cache where the gradients fit it.  A
// launch takes many tensors: their addresses and sizes come as kernel arguments, their elements are dealt out in
// chunks, and every workgroup takes every so many-th chunk of a fixed grid, so sums have a fixed order.
//
// Squares and sums are float64, so nothing that float32 holds over- or underflows and the norm is the float32 next to the
// root (but for roots within n 2^-53 of the middle of two).  That takes as many conversions as products: 232 us for 1.4 GB,
// with squares and sums of eights in float32 224.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wkv_lanes.h"
#include "wkv_launch.h"

namespace wkv {
namespace {

constexpr int kThreads = 256;

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// The tensor that a chunk belongs to: the last one whose first chunk is not behind it.
__device__ __forceinline__ int tensor_of(const ClipTable& t, int64_t chunk) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.chunk0[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ double squares(const float (&f)[8]) {
    double d = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) d = fma(static_cast<double>(f[i]), static_cast<double>(f[i]), d);
    return d;
}

// Eight elements at e of a tensor whose address is on the 16-byte grid (kVec) or not; zeros behind its end.
template <typename T, bool Vec>
__device__ __forceinline__ void load8(const T* p, int64_t e, int64_t n, float (&f)[8]) {
    if (Vec && e + 8 <= n) {
        if constexpr (sizeof(T) == 4) {
            const f4 a = *reinterpret_cast<const f4*>(p + e), b = *reinterpret_cast<const f4*>(p + e + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
        } else {
            const u4 a = *reinterpret_cast<const u4*>(p + e);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(a[i] << 16), f[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = e + i < n ? widen(p[e + i]) : 0.f;
}

template <bool PastCache, typename V>
__device__ __forceinline__ void store_vec(V* p, V v) {
    if constexpr (PastCache) __builtin_nontemporal_store(v, p);
    else *p = v;
}

template <typename T, bool Vec, bool PastCache>
__device__ __forceinline__ void store8(T* p, int64_t e, int64_t n, const float (&f)[8]) {
    if (Vec && e + 8 <= n) {
        if constexpr (sizeof(T) == 4) {
            store_vec<PastCache>(reinterpret_cast<f4*>(p + e), f4{f[0], f[1], f[2], f[3]});
            store_vec<PastCache>(reinterpret_cast<f4*>(p + e + 4), f4{f[4], f[5], f[6], f[7]});
        } else {
            store_vec<PastCache>(reinterpret_cast<u4*>(p + e), u4{pk2(f[0], f[1]), pk2(f[2], f[3]), pk2(f[4], f[5]), pk2(f[6], f[7])});
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (e + i < n) {
            if constexpr (sizeof(T) == 4) p[e + i] = f[i];
            else p[e + i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(f[i]));
        }
    }
}

// Eight elements as they lie in memory.
template <typename T>
struct Raw8 {
    u4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const u4*>(p)[i];
    }
    __device__ __forceinline__ void widen(float (&f)[8]) const {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[i / 4][i % 4]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(v[0][i] << 16), f[2 * i + 1] = __uint_as_float(v[0][i] & 0xffff0000u);
        }
    }
};

// The elements of a chunk: eight a thread, and the next eights a workgroup's width on.  A whole chunk of a tensor on the
// 16-byte grid has kBatch eights of a thread on their way at once.
constexpr int kStep = kThreads * 8, kBatch = 4;
static_assert(kClipChunk % (kStep * kBatch) == 0, "whole batches a chunk");

template <typename T, bool Vec>
__device__ __forceinline__ double sum_chunk(const T* p, int64_t first, int64_t n) {
    double sum = 0.0;
    float f[8];
    if (Vec && first + kClipChunk <= n) {
        const T* at = p + first + threadIdx.x * 8;
        for (int k = 0; k < kClipChunk / kStep; k += kBatch) {
            Raw8<T> raw[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) raw[q].load(at + (k + q) * kStep);
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                raw[q].widen(f);
                sum += squares(f);
            }
        }
        return sum;
    }
    const int64_t end = first + kClipChunk < n ? first + kClipChunk : n;
    for (int64_t e = first + threadIdx.x * 8; e < end; e += kStep) {
        load8<T, Vec>(p, e, n, f);
        sum += squares(f);
    }
    return sum;
}

// A factor as two numbers to multiply by in turn, since one below float32's normal numbers (gradients above 1e38 to a norm
// below 1) has lost digits where products with it are ordinary numbers.  The second one is 1, or 2^-126 and the first one then
// up to 1, so nothing overflows on the way, and what the first product loses ends as zero.
struct Factor {
    float by;
    bool tiny;  // the same for all lanes, in a scalar register: a branch that is free otherwise (a second product always: 735 -> 743 us)
    __device__ __forceinline__ void finish(float (&f)[8]) const {
        if (!tiny) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= 0x1p-126f;
    }
};

template <typename T, bool Vec, bool PastCache>
__device__ __forceinline__ void scale_chunk(const T* p, T* to, int64_t first, int64_t n, Factor by) {
    float f[8];
    if (Vec && first + kClipChunk <= n) {
        const int64_t at = first + threadIdx.x * 8;
        for (int k = 0; k < kClipChunk / kStep; k += kBatch) {
            Raw8<T> raw[kBatch];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) raw[q].load(p + at + (k + q) * kStep);
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                raw[q].widen(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] *= by.by;
                by.finish(f);
                store8<T, true, PastCache>(to, at + (k + q) * kStep, n, f);
            }
        }
        return;
    }
    const int64_t end = first + kClipChunk < n ? first + kClipChunk : n;
    for (int64_t e = first + threadIdx.x * 8; e < end; e += kStep) {
        load8<T, Vec>(p, e, n, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= by.by;
        by.finish(f);
        store8<T, Vec, PastCache>(to, e, n, f);
    }
}

__device__ __forceinline__ bool on_grid(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The sum of a workgroup's numbers, to all its threads.
__device__ __forceinline__ double sum_block(double v) {
    __shared__ double all[kThreads];
    all[threadIdx.x] = v;
    __syncthreads();
#pragma unroll
    for (int k = kThreads / 2; k > 0; k >>= 1) {
        if (threadIdx.x < k) all[threadIdx.x] += all[threadIdx.x + k];
        __syncthreads();
    }
    return all[0];
}

__global__ __launch_bounds__(kThreads) void clip_sums_kernel(ClipTable t, double* part) {
    double sum = 0.0;
    for (int64_t chunk = blockIdx.x; chunk < t.chunks; chunk += gridDim.x) {
        const int k = tensor_of(t, chunk);
        const int64_t first = (chunk - t.chunk0[k]) * kClipChunk, n = t.n[k];
        const bool vec = on_grid(t.in[k]);
        if (t.bf16[k] != 0) {
            const uint16_t* p = static_cast<const uint16_t*>(t.in[k]);
            sum += vec ? sum_chunk<uint16_t, true>(p, first, n) : sum_chunk<uint16_t, false>(p, first, n);
        } else {
            const float* p = static_cast<const float*>(t.in[k]);
            sum += vec ? sum_chunk<float, true>(p, first, n) : sum_chunk<float, false>(p, first, n);
        }
    }
    sum = sum_block(sum);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ double sum_parts(const double* part, int64_t n) {
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) sum += part[i];
    return sum_block(sum);
}

__global__ __launch_bounds__(kThreads) void clip_norm_kernel(const double* part, int64_t n, float* norm, double* total) {
    const double sum = sum_parts(part, n);
    if (threadIdx.x != 0) return;
    if (norm != nullptr) *norm = static_cast<float>(sqrt(sum));
    if (total != nullptr) *total = sum;
}

// Every workgroup adds up the partial sums for itself, so the factor needs no launch of its own.  PastCache: outputs leave
// past the caches, where the gradients do not fit them anyway and the stores would drive out what is read next (282 MB
// of gradients: 185 -> 169 us, 1.4 GB: 788 -> 746; 86 MB take 57 us either way, and are still there for the optimizer).
template <bool PastCache>
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(ClipTable t, const double* part, int64_t nparts, float max_norm,
                                                              float eps, float* norm) {
    const double all = sqrt(sum_parts(part, nparts)), with = all + static_cast<double>(eps);
    // 1 up to max_norm; a norm that is not a number is handed on to every gradient
    const double factor = with <= static_cast<double>(max_norm) ? 1.0 : static_cast<double>(max_norm) / with;
    const bool tiny = __builtin_amdgcn_readfirstlane(factor < 0x1p-126 ? 1 : 0) != 0;
    const Factor by{static_cast<float>(tiny ? factor * 0x1p126 : factor), tiny};
    if (blockIdx.x == 0 && threadIdx.x == 0 && norm != nullptr) *norm = static_cast<float>(all);
    // from the last chunk to the first, as the launches go: what the sums read last is still in the last level cache
    for (int64_t chunk = t.chunks - 1 - blockIdx.x; chunk >= 0; chunk -= gridDim.x) {
        const int k = tensor_of(t, chunk);
        const int64_t first = (chunk - t.chunk0[k]) * kClipChunk, n = t.n[k];
        if (by.by == 1.f && !by.tiny && t.in[k] == t.out[k]) continue;
        const bool vec = on_grid(t.in[k]) && on_grid(t.out[k]);
        if (t.bf16[k] != 0) {
            const uint16_t* p = static_cast<const uint16_t*>(t.in[k]);
            uint16_t* to = static_cast<uint16_t*>(t.out[k]);
            if (vec) scale_chunk<uint16_t, true, PastCache>(p, to, first, n, by);
            else scale_chunk<uint16_t, false, PastCache>(p, to, first, n, by);
        } else {
            const float* p = static_cast<const float*>(t.in[k]);
            float* to = static_cast<float*>(t.out[k]);
            if (vec) scale_chunk<float, true, PastCache>(p, to, first, n, by);
            else scale_chunk<float, false, PastCache>(p, to, first, n, by);
        }
    }
}

}  // namespace

int64_t clip_blocks(const ClipTable& t) { return t.chunks < kClipBlocks ? t.chunks : kClipBlocks; }

hipError_t launch_clip_sums(const ClipTable& t, double* part, hipStream_t stream) {
    hipLaunchKernelGGL(clip_sums_kernel, dim3(static_cast<unsigned>(clip_blocks(t))), dim3(kThreads), 0, stream, t, part);
    return hipGetLastError();
}

hipError_t launch_clip_norm(const double* part, int64_t nparts, float* norm, double* total, hipStream_t stream) {
    hipLaunchKernelGGL(clip_norm_kernel, dim3(1), dim3(kThreads), 0, stream, part, nparts, norm, total);
    return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipTable& t, const double* part, int64_t nparts, float max_norm, float eps, float* norm,
                             bool past_cache, hipStream_t stream) {
    const int64_t blocks = clip_blocks(t);
    const dim3 grid(static_cast<unsigned>(blocks)), block(kThreads);
    if (past_cache) hipLaunchKernelGGL(clip_scale_kernel<true>, grid, block, 0, stream, t, part, nparts, max_norm, eps, norm);
    else hipLaunchKernelGGL(clip_scale_kernel<false>, grid, block, 0, stream, t, part, nparts, max_norm, eps, norm);
    return hipGetLastError();
}

}  // namespace wkv
