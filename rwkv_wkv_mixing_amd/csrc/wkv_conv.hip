// Short causal convolution over time, a filter of K taps a channel, with its activation: what stands before the
// selective scan as the token shift stands before the other mixes.  With X the K - 1 carried inputs followed by the
// row's tokens (so that X[t + K - 1] is token t):
//     pre_t = bias + sum_j weight[j] X[t + j],   out_t = act(pre_t)
// Streaming work: a thread owns V channels over a run of tokens, so x is read once (and K - 1 tokens a run twice) and
// the window stays in registers; what bounds it is memory (8 x 1024 x 4096 bf16, K = 4: 23 us, 5.7 TB/s).
//
// Backward, with g_t = gout_t act'(pre_t) of the row's tokens (zero elsewhere):
//     dX[e] = sum_j weight[j] g_{e - j} (+ the carried-out inputs' gradient),   dweight[j] = sum g_t X[t + j],   dbias = sum g
// A thread walks its run and K - 1 tokens more, computing pre again from x.  The weights' sums are kept a thread, added
// over a workgroup's runs in LDS and over workgroups by a second kernel (in float64), each in a fixed order.  Some 40 vector
// instructions an element next to 6 bytes: at the same size 52 us, 3.9 TB/s, with the vector units busy two thirds of them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wkv_lanes.h"
#include "wkv_launch.h"

namespace wkv {
namespace {
constexpr int kThreads = 256, kCols = 64, kRuns = kThreads / kCols;  // a workgroup: 64 vectors of channels, 4 runs

typedef uint32_t u2 __attribute__((ext_vector_type(2)));

// V elements as they lie in memory, widened and narrowed.
template <typename T, int V>
struct Vec;
template <>
struct Vec<float, 4> {
    typedef f4 Raw;
    static __device__ __forceinline__ void widen(Raw r, float (&f)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = r[i];
    }
    static __device__ __forceinline__ Raw narrow(const float (&f)[4]) { return Raw{f[0], f[1], f[2], f[3]}; }
};
template <>
struct Vec<float, 1> {
    typedef float Raw;
    static __device__ __forceinline__ void widen(Raw r, float (&f)[1]) { f[0] = r; }
    static __device__ __forceinline__ Raw narrow(const float (&f)[1]) { return f[0]; }
};
template <>
struct Vec<float, 2> {
    typedef f2 Raw;
    static __device__ __forceinline__ void widen(Raw r, float (&f)[2]) { f[0] = r.x, f[1] = r.y; }
    static __device__ __forceinline__ Raw narrow(const float (&f)[2]) { return Raw{f[0], f[1]}; }
};
template <>
struct Vec<uint16_t, 2> {
    typedef uint32_t Raw;
    static __device__ __forceinline__ void widen(Raw r, float (&f)[2]) {
        f[0] = __uint_as_float(r << 16), f[1] = __uint_as_float(r & 0xffff0000u);
    }
    static __device__ __forceinline__ Raw narrow(const float (&f)[2]) { return pk2(f[0], f[1]); }
};
template <>
struct Vec<uint16_t, 4> {
    typedef u2 Raw;
    static __device__ __forceinline__ void widen(Raw r, float (&f)[4]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) f[2 * i] = __uint_as_float(r[i] << 16), f[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
    static __device__ __forceinline__ Raw narrow(const float (&f)[4]) { return Raw{pk2(f[0], f[1]), pk2(f[2], f[3])}; }
};
template <>
struct Vec<uint16_t, 1> {
    typedef uint16_t Raw;
    static __device__ __forceinline__ void widen(Raw r, float (&f)[1]) { f[0] = wkv::widen(r); }
    static __device__ __forceinline__ Raw narrow(const float (&f)[1]) {
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f[0]));
    }
};

// act(v), and g act'(v): the activation is looked up once for all of them.  Wide with float32 tensors; with bf16 ones results
// are rounded to 2^-9, or are sums of gradients that were.
template <bool Wide, int V>
__device__ __forceinline__ void act_of(int act, float (&v)[V]) {
    if (act == kActSilu) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] *= sigmoid<Wide>(v[i]);
    } else if (act == kActSigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = sigmoid<Wide>(v[i]);
    }
}
template <bool Wide, int V>
__device__ __forceinline__ void act_grad(int act, const float (&v)[V], float (&g)[V]) {
    if (act == kActSilu) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float p = sigmoid<Wide>(v[i]);
            g[i] *= p * fmaf(v[i], 1.f - p, 1.f);
        }
    } else if (act == kActSigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float p = sigmoid<Wide>(v[i]);
            g[i] *= p * (1.f - p);
        }
    }
}

// A row's tokens.
__device__ __forceinline__ int row_length(const ConvArgs& P, int64_t b) {
    const int all = static_cast<int>(P.T), len = P.lengths != nullptr ? __builtin_amdgcn_readfirstlane(P.lengths[b]) : all;
    return len < 0 ? 0 : len > all ? all : len;
}

// V elements of channel c at row e of X (zeros where there is none: before the carried inputs when none are given,
// and behind the row's length).
template <typename T, int V>
__device__ __forceinline__ typename Vec<T, V>::Raw load_ext(const ConvArgs& P, int64_t b, int len, int e, int64_t c, int K) {
    typedef typename Vec<T, V>::Raw Raw;
    const int t = e - (K - 1);
    if (t >= len) return Raw{};
    if (t >= 0) return *reinterpret_cast<const Raw*>(static_cast<const T*>(P.x) + (b * P.T + t) * P.C + c);
    if (P.s_in == nullptr) return Raw{};
    return *reinterpret_cast<const Raw*>(static_cast<const T*>(P.s_in) + (b * (K - 1) + e) * P.C + c);
}

template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(ConvArgs P, int run, int64_t ncb) {
    typedef Vec<T, V> Ops;
    typedef typename Ops::Raw Raw;
    // Tokens whose loads are on their way at once (4 of them: 32.5 us for 31.1 of 8): a multiple of K, so that the window, a
    // ring of K rows, is back where it was.
    constexpr int kAhead = K == 3 ? 6 : 8;
    const int64_t blk = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t cb = blk % ncb, rest = blk / ncb, ntb = (P.T + kRuns * run - 1) / (kRuns * run);
    const int64_t b = rest / ntb, c = (cb * kCols + threadIdx.x % kCols) * V;
    const int64_t first = (rest % ntb) * kRuns * run + __builtin_amdgcn_readfirstlane(threadIdx.x / kCols) * run;
    if (b >= P.B || c >= P.C || first >= P.T) return;
    const int all = static_cast<int>(P.T), t0 = static_cast<int>(first), t1 = all - t0 < run ? all : t0 + run, len = row_length(P, b),
              te = len < t1 ? len : t1;
    float w[K][V], bias[V], win[K][V];
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) w[j][i] = P.weight[j * P.C + c + i];
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = P.bias != nullptr ? P.bias[c + i] : 0.f;
    Raw last[K - 1];  // the carried inputs of the next call: rows len .. len + K - 2 of X
    const bool carry = t0 == 0 && P.s_out != nullptr;
    if (carry) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) last[j] = load_ext<T, V>(P, b, len, len + j, c, K);
    }
    if (t0 < len) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) Ops::widen(load_ext<T, V>(P, b, len, t0 + j, c, K), win[j]);
    }
    const T* x = static_cast<const T*>(P.x) + (b * P.T) * P.C + c;
    T* out = static_cast<T*>(P.out) + (b * P.T) * P.C + c;
    for (int t = t0; t < te; t += kAhead) {
        Raw raw[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)  // (behind the last token: that one again)
            raw[k] = *reinterpret_cast<const Raw*>(x + static_cast<int64_t>(t + k < te ? t + k : te - 1) * P.C);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (t + k < te) {
                Ops::widen(raw[k], win[(k + K - 1) % K]);
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    o[i] = bias[i];
#pragma unroll
                    for (int j = 0; j < K; ++j) o[i] = fmaf(w[j][i], win[(k + j) % K][i], o[i]);
                }
                act_of<sizeof(T) == 4>(P.act, o);
                *reinterpret_cast<Raw*>(out + static_cast<int64_t>(t + k) * P.C) = Ops::narrow(o);
            }
        }
    }
    for (int t = te > t0 ? te : t0; t < t1; ++t) *reinterpret_cast<Raw*>(out + static_cast<int64_t>(t) * P.C) = Raw{};
    if (carry) {  // (s_out may be s_in: this thread alone reads and writes these rows of it)
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            *reinterpret_cast<Raw*>(static_cast<T*>(P.s_out) + (b * (K - 1) + j) * P.C + c) = last[j];
    }
}

// One token a row: everything it needs is asked for at once, where the walk waits for the carried inputs, then for the token
// (bf16, K = 4, layers in turn: 256 rows of 4096 channels 9.3 -> 5.8 us, of 4095 29 -> 8.9, 2048 rows 53 -> 29.7, 4.6 TB/s).
template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(ConvArgs P, int64_t ncb) {
    typedef Vec<T, V> Ops;
    typedef typename Ops::Raw Raw;
    const int64_t blk = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t b = blk / ncb * kRuns + __builtin_amdgcn_readfirstlane(threadIdx.x / kCols), c = (blk % ncb * kCols + threadIdx.x % kCols) * V;
    if (b >= P.B || c >= P.C) return;
    const bool live = P.lengths == nullptr || P.lengths[b] > 0;
    const T* s_in = static_cast<const T*>(P.s_in) + b * (K - 1) * P.C + c;
    T* s_out = static_cast<T*>(P.s_out) + b * (K - 1) * P.C + c;
    Raw raw[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) raw[j] = P.s_in != nullptr ? *reinterpret_cast<const Raw*>(s_in + j * P.C) : Raw{};
    // (a row without its token is not read: the weights are, in its place, and dropped.  A load under a condition has the others
    // wait: 256 rows of 4096 float32 channels 9.2 -> 10.4 us)
    raw[K - 1] = *reinterpret_cast<const Raw*>((live ? static_cast<const T*>(P.x) + b * P.C : reinterpret_cast<const T*>(P.weight)) + c);
    float w[K][V], o[V];
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) w[j][i] = P.weight[j * P.C + c + i];
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = P.bias != nullptr ? P.bias[c + i] : 0.f;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        float f[V];
        Ops::widen(raw[j], f);
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = fmaf(w[j][i], f[i], o[i]);
    }
    act_of<sizeof(T) == 4>(P.act, o);
    *reinterpret_cast<Raw*>(static_cast<T*>(P.out) + b * P.C + c) = live ? Ops::narrow(o) : Raw{};
    if (P.s_out == nullptr) return;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) *reinterpret_cast<Raw*>(s_out + j * P.C) = live ? raw[j + 1] : raw[j];
}

template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvArgs P, int run, int64_t ncb) {
    typedef Vec<T, V> Ops;
    typedef typename Ops::Raw Raw;
    constexpr int kAhead = K == 3 ? 3 : 4;  // a multiple of K: the windows are rings (2: 60 us, 4: 52, 8: 58)
    __shared__ float sums[kRuns][K + 1][V][kCols];
    const int64_t blk = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t cb = blk % ncb, slot = blk / ncb;
    if (slot >= P.slots) return;  // (the whole workgroup)
    const int col = threadIdx.x % kCols, r = __builtin_amdgcn_readfirstlane(threadIdx.x / kCols);
    const int64_t c = (cb * kCols + col) * V;
    const bool valid = c < P.C;
    const int64_t ntb = (P.T + kRuns * run - 1) / (kRuns * run);
    float w[K][V], bias[V], dw[K][V], db[V];
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) w[j][i] = valid ? P.weight[j * P.C + c + i] : 0.f, dw[j][i] = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = valid && P.bias != nullptr ? P.bias[c + i] : 0.f, db[i] = 0.f;
    // tiles of kRuns runs, every slots-th one
    for (int64_t tile = slot; tile < P.B * ntb; tile += P.slots) {
        const int64_t b = tile / ntb, first = (tile % ntb) * kRuns * run + r * run;
        if (!valid || first >= P.T) continue;
        const int all = static_cast<int>(P.T), t0 = static_cast<int>(first), t1 = all - t0 < run ? all : t0 + run, len = row_length(P, b);
        const T* x = static_cast<const T*>(P.x) + (b * P.T) * P.C + c;
        const T* go = static_cast<const T*>(P.gout) + (b * P.T) * P.C + c;
        T* dx = static_cast<T*>(P.dx) + (b * P.T) * P.C + c;
        float win[K][V], g[K][V];  // of X, and of g: the window's last row is the token at hand
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) win[j][i] = g[j][i] = 0.f;
        if (t0 < len) {
#pragma unroll
            for (int j = 0; j < K - 1; ++j) Ops::widen(load_ext<T, V>(P, b, len, t0 + j, c, K), win[j]);
        }
        // row e = t of X (token t - (K - 1)) has all its g once token t is done; the run answers for the tokens
        // t0 .. t1 - 1, and the first one for the carried inputs too
        const int end = t1 + K - 1, live = len < end ? len : end;
        // one token: its g, and (own) its part of the weights' sums.  The windows start at row `at` of their rings.
        const auto take = [&](auto at, Raw rx, Raw rg, bool own) {
            constexpr int a0 = decltype(at)::value;
            float (&gt)[V] = g[(a0 + K - 1) % K];
            float pre[V];
            Ops::widen(rx, win[(a0 + K - 1) % K]);
            Ops::widen(rg, gt);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                pre[i] = bias[i];
#pragma unroll
                for (int j = 0; j < K; ++j) pre[i] = fmaf(w[j][i], win[(a0 + j) % K][i], pre[i]);
            }
            act_grad<sizeof(T) == 4>(P.act, pre, gt);
            if (own) {
#pragma unroll
                for (int i = 0; i < V; ++i) {
#pragma unroll
                    for (int j = 0; j < K; ++j) dw[j][i] = fmaf(gt[i], win[(a0 + j) % K][i], dw[j][i]);
                    db[i] += gt[i];
                }
            }
        };
        // dX at the window's first row: sum_j weight[j] g_{t - j}
        const auto give = [&](auto at, float (&o)[V]) {
            constexpr int a0 = decltype(at)::value;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                o[i] = w[0][i] * g[(a0 + K - 1) % K][i];
#pragma unroll
                for (int j = 1; j < K; ++j) o[i] = fmaf(w[j][i], g[(a0 + K - 1 - j) % K][i], o[i]);
            }
        };
        const auto shift = [&] {
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) win[j][i] = win[j + 1][i], g[j][i] = g[j + 1][i];
        };
        Raw rx[kAhead], rg[kAhead];
        const auto fetch = [&](int tt) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                rx[k] = rg[k] = Raw{};
                if (tt + k < len && tt < end) {
                    rx[k] = *reinterpret_cast<const Raw*>(x + static_cast<int64_t>(tt + k) * P.C);
                    rg[k] = *reinterpret_cast<const Raw*>(go + static_cast<int64_t>(tt + k) * P.C);
                }
            }
        };
        fetch(t0);
        for (int tt = t0; tt < end; tt += kAhead) {
            Raw cx[kAhead], cg[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) cx[k] = rx[k], cg[k] = rg[k];
            fetch(tt + kAhead);
            if (tt + kAhead <= len && !(tt == 0 && P.ds_in != nullptr)) {  // all of them tokens, no carried input's gradient
                each<kAhead>([&](auto k) {
                    const int to = tt + k - (K - 1);
                    take(k, cx[k], cg[k], tt + k < t1);
                    float o[V];
                    give(k, o);
                    if (to >= t0 && to < t1) *reinterpret_cast<Raw*>(dx + static_cast<int64_t>(to) * P.C) = Ops::narrow(o);
                });
                continue;
            }
#pragma unroll 1
            for (int k = 0; k < kAhead; ++k) {
                const int t = tt + k;
                if (t >= end) break;
                Raw vx = cx[0], vg = cg[0];
#pragma unroll
                for (int q = 1; q < kAhead; ++q)
                    if (k == q) vx = cx[q], vg = cg[q];
                if (t < live) {
                    take(std::integral_constant<int, 0>{}, vx, vg, t < t1);
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) g[K - 1][i] = 0.f;
                }
                const int to = t - (K - 1);
                if (to >= t0 || (t0 == 0 && P.ds_in != nullptr)) {
                    float o[V];
                    give(std::integral_constant<int, 0>{}, o);
                    if (P.ds_out != nullptr && t >= len && t < len + K - 1) {
                        float e[V];
                        Ops::widen(*reinterpret_cast<const Raw*>(static_cast<const T*>(P.ds_out) + (b * (K - 1) + t - len) * P.C + c), e);
#pragma unroll
                        for (int i = 0; i < V; ++i) o[i] += e[i];
                    }
                    Raw ro = Ops::narrow(o);
                    if (to < 0) {
                        *reinterpret_cast<Raw*>(static_cast<T*>(P.ds_in) + (b * (K - 1) + t) * P.C + c) = ro;
                    } else {
                        if (to >= len) ro = Raw{};
                        *reinterpret_cast<Raw*>(dx + static_cast<int64_t>(to) * P.C) = ro;
                    }
                }
                shift();
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < K; ++j) sums[r][j][i][col] = dw[j][i];
        sums[r][K][i][col] = db[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < (K + 1) * V * kCols; e += kThreads) {
        const int q = e % kCols, i = e / kCols % V, j = e / (kCols * V);
        const int64_t ch = (cb * kCols + q) * V + i;
        if (ch >= P.C) continue;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kRuns; ++k) sum += sums[k][j][i][q];
        P.part[(slot * (K + 1) + j) * P.C + ch] = sum;
    }
}

// dweight and dbias from the slots' sums, in order and in float64: a lane takes an output, each of the workgroup's 16 waves a sixteenth
// of the slots.
constexpr int kParts = 16;
__global__ __launch_bounds__(64 * kParts) void conv_reduce_kernel(ConvArgs P) {
    __shared__ double sums[kParts][64];
    const int64_t n = (P.K + 1) * P.C, i = static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63);
    const int q = threadIdx.x >> 6;
    const int64_t each = (P.slots + kParts - 1) / kParts, first = q * each, last = first + each < P.slots ? first + each : P.slots;
    double sum = 0.0;
    if (i < n) {
#pragma unroll 4
        for (int64_t s = first; s < last; ++s) sum += P.part[s * n + i];
    }
    sums[q][threadIdx.x & 63] = sum;
    __syncthreads();
    if (q != 0 || i >= n) return;
    sum = 0.0;
#pragma unroll
    for (int k = 0; k < kParts; ++k) sum += sums[k][threadIdx.x];
    const float all = static_cast<float>(sum);
    if (i < P.K * P.C) P.dweight[i] = all;
    else if (P.dbias != nullptr) P.dbias[i - P.K * P.C] = all;
}

// Carried inputs of a call without tokens: they pass on (or zeros do).
template <typename T>
__global__ __launch_bounds__(256) void conv_copy_kernel(const T* from, T* to, int64_t n) {
    const int64_t i = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    if (i < n) to[i] = from != nullptr ? from[i] : T{0};
}

// Tokens a run: long ones read less twice, but the card wants some 2048 workgroups (4096 of them: 32 x 1024 x 768 forward
// 30.6 us for 22.9).
int run_of(int64_t B, int64_t T, int64_t ncb, int longest) {
    int run = longest;
    while (run > 4 && B * ((T + kRuns * run - 1) / (kRuns * run)) * ncb < 2048) run /= 2;
    return run;
}

dim3 grid_of(int64_t blocks) {
    constexpr int64_t kMost = int64_t{1} << 20;
    if (blocks <= kMost) return dim3(static_cast<unsigned>(blocks));
    return dim3(static_cast<unsigned>(kMost), static_cast<unsigned>((blocks + kMost - 1) / kMost));
}

template <typename T, int V, int K>
hipError_t fwd_launch(const ConvArgs& a, hipStream_t stream) {
    const int64_t ncb = (a.C + kCols * V - 1) / (kCols * V);
    if (a.T == 1) {
        hipLaunchKernelGGL((conv_step_kernel<T, V, K>), grid_of((a.B + kRuns - 1) / kRuns * ncb), dim3(kThreads), 0, stream, a, ncb);
        return hipGetLastError();
    }
    // (8 x 1024 x 4096: runs of 8 and 16 bf16 28.9 and 31.1 us, float32 49.8 and 54.5, 4095 channels 61.2 and 50.0)
    const int run = run_of(a.B, a.T, ncb, V > 1 ? 8 : 16);
    const int64_t ntb = (a.T + kRuns * static_cast<int64_t>(run) - 1) / (kRuns * static_cast<int64_t>(run));
    hipLaunchKernelGGL((conv_fwd_kernel<T, V, K>), grid_of(a.B * ntb * ncb), dim3(kThreads), 0, stream, a, run, ncb);
    return hipGetLastError();
}

template <typename T, int V, int K>
hipError_t bwd_launch(const ConvArgs& a, hipStream_t stream) {
    const int64_t ncb = (a.C + kCols * V - 1) / (kCols * V);
    // (8 x 1024 x 4096: runs of 16, 32 and 64 bf16 63.0, 60.8 and 61 us, 4095 channels 88, 83 and 94; float32 93, 104 and 106)
    const int run = run_of(a.B, a.T, ncb, V > 1 && sizeof(T) == 4 ? 16 : 32);
    hipLaunchKernelGGL((conv_bwd_kernel<T, V, K>), grid_of(a.slots * ncb), dim3(kThreads), 0, stream, a, run, ncb);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t n = (K + 1) * a.C;
    hipLaunchKernelGGL(conv_reduce_kernel, dim3(static_cast<unsigned>((n + 63) / 64)), dim3(64 * kParts), 0, stream, a);
    return hipGetLastError();
}

template <typename T, int V>
hipError_t fwd_k(const ConvArgs& a, hipStream_t stream) {
    switch (a.K) {
        case 2: return fwd_launch<T, V, 2>(a, stream);
        case 3: return fwd_launch<T, V, 3>(a, stream);
        default: return fwd_launch<T, V, 4>(a, stream);
    }
}

template <typename T, int V>
hipError_t bwd_k(const ConvArgs& a, hipStream_t stream) {
    switch (a.K) {
        case 2: return bwd_launch<T, V, 2>(a, stream);
        case 3: return bwd_launch<T, V, 3>(a, stream);
        default: return bwd_launch<T, V, 4>(a, stream);
    }
}

}  // namespace

// Rows of partial sums of the backward: as many workgroups as fill the card (4096 of one channel a thread: 4095 channels
// 83 us; 2048: 92) and no more than there are tiles of the shortest runs.  But one for every 512 tokens, so that a thread adds up
// 128 in float32: one sum over thousands of terms that are alike loses up to 2^-25 of itself with each.
int64_t conv_slots(int64_t B, int64_t T, int64_t C) {
    const int64_t ncb = (C + kCols - 1) / kCols, tiles = B * ((T + kRuns * 4 - 1) / (kRuns * 4));
    const int64_t longest = B * ((T + kRuns * 32 - 1) / (kRuns * 32)), fewest = (longest + 3) / 4;
    int64_t most = 4096 / (ncb > 0 ? ncb : 1);
    most = most < 16 ? 16 : most;
    most = most < fewest ? fewest : most;
    return tiles < most ? tiles : most;
}

hipError_t launch_conv_copy(const void* from, void* to, int64_t n, bool bf16, hipStream_t stream) {
    if (to == nullptr || to == from || n <= 0) return hipSuccess;
    const dim3 grid = grid_of((n + 255) / 256);
    if (bf16) hipLaunchKernelGGL(conv_copy_kernel<uint16_t>, grid, dim3(256), 0, stream, static_cast<const uint16_t*>(from), static_cast<uint16_t*>(to), n);
    else hipLaunchKernelGGL(conv_copy_kernel<float>, grid, dim3(256), 0, stream, static_cast<const float*>(from), static_cast<float*>(to), n);
    return hipGetLastError();
}

// Four channels a thread forward, two backward, where four leave room for fewer waves (bf16 52 us, 64 of four).
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t stream) {
    if (a.vec) return a.bf16 ? fwd_k<uint16_t, 4>(a, stream) : fwd_k<float, 4>(a, stream);
    return a.bf16 ? fwd_k<uint16_t, 1>(a, stream) : fwd_k<float, 1>(a, stream);
}
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t stream) {
    if (a.vec) return a.bf16 ? bwd_k<uint16_t, 2>(a, stream) : bwd_k<float, 2>(a, stream);
    return a.bf16 ? bwd_k<uint16_t, 1>(a, stream) : bwd_k<float, 1>(a, stream);
}

}  // namespace wkv
