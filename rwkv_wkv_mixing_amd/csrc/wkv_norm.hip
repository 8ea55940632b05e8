// The norms around the mixing.
//
// Head norm (behind the matrix-state mixing, and on keys before it): per row and head of G channels
//     out = act(gate) * (norm(y) * weight + bias)
// Block norm (between two blocks): per row of C channels
//     z = act(gate) * (norm(y) * post_w + post_b),   x_out = x + scale * z,   h = norm(x_out) * pre_w + pre_b
// with norm(y) = (y - m) / sqrt(mean((y - m)^2) + eps), m the mean, or 0 (root mean square).
//
// Streaming work: every element is read once and stays in registers between the statistics and the
// outputs.  The mean is taken first and the squares of what is left of it second, so a mean far above
// the deviation costs no digits.  A head is held by 1 .. 64 lanes of a wave (8 elements each, 16 with
// more than 512 channels) and its sums meet by shuffles; a row of a block norm by 64 .. 1024 threads.
//
// Backward, with g the gradient of norm(y) (that of z times act(gate) weight):
//     dy = (g - yhat mean(g yhat) - [mean(g)]) / sqrt(mean((y - m)^2) + eps)
// from statistics computed again.  The gradients of weights are sums over the rows: every workgroup
// keeps its channels' sums in registers over the rows it takes, writes them as one row of partial
// sums, and norm_reduce_kernel adds those in order (bitwise reproducible).
//
// Measured, whole calls: head norm of 8192 x 64 heads of 64, float32 to bf16 with a gate, 46 us (5.8 TB/s);
// its gradients at 8192 x 32 heads of 128, bf16, 70 us (4.8 TB/s); block norm of 8192 x 4096, bf16, 77 us
// (4.4 TB/s, four sums over a row with a barrier each), its gradients 125 us (4.3 TB/s and 42 MB of partial sums).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wkv_lanes.h"
#include "wkv_launch.h"

namespace wkv {
namespace {

typedef uint32_t u4 __attribute__((ext_vector_type(4)));

// V consecutive elements as float32: 8 in 16-byte accesses, or 1.
template <int V>
__device__ __forceinline__ void load(const uint16_t* p, float (&f)[V]) {
    if constexpr (V == 8) {
        const u4 x = *reinterpret_cast<const u4*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(x[i] << 16);
            f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        }
    } else {
        f[0] = widen(*p);
    }
}
template <int V>
__device__ __forceinline__ void load(const float* p, float (&f)[V]) {
    if constexpr (V == 8) {
        const f4 a = *reinterpret_cast<const f4*>(p), b = *reinterpret_cast<const f4*>(p + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    } else {
        f[0] = *p;
    }
}
template <int V>
__device__ __forceinline__ void store(uint16_t* p, const float (&f)[V]) {
    if constexpr (V == 8) {
        *reinterpret_cast<u4*>(p) = u4{pk2(f[0], f[1]), pk2(f[2], f[3]), pk2(f[4], f[5]), pk2(f[6], f[7])};
    } else {
        *p = static_cast<uint16_t>(pk2(f[0], f[0]) & 0xffffu);
    }
}
template <int V>
__device__ __forceinline__ void store(float* p, const float (&f)[V]) {
    if constexpr (V == 8) {
        *reinterpret_cast<f4*>(p) = f4{f[0], f[1], f[2], f[3]};
        *reinterpret_cast<f4*>(p + 4) = f4{f[4], f[5], f[6], f[7]};
    } else {
        *p = f[0];
    }
}

// V consecutive elements as they are in memory: loads issued long before their use.
template <typename T, int V>
struct Raw {
    static constexpr int kWords = V == 8 ? V * static_cast<int>(sizeof(T)) / 16 : 1;
    u4 w[V == 8 ? kWords : 1];
    T one;
    __device__ __forceinline__ void fetch(const T* p) {
        if constexpr (V == 8) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const u4*>(p)[i];
        } else {
            one = *p;
        }
    }
    __device__ __forceinline__ void get(float (&f)[V]) const {
        if constexpr (V == 1) {
            f[0] = widen(one);
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[0][i] << 16);
                f[2 * i + 1] = __uint_as_float(w[0][i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i / 4][i % 4]);
        }
    }
};

// act(g) and (kGrad) its derivative of a thread's V elements; without a gate 1 and 0.  exp overflows to
// inf for g below -88, where both sigmoids are 0.  The choice is made once for the V elements: made for
// each it took as many instructions as the arithmetic.
template <int V, bool kGrad>
__device__ __forceinline__ void activate(int act, bool gated, const float (&g)[V], float (&a)[V], float (&da)[V]) {
    if (!gated || act == kActNone) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            a[j] = gated ? g[j] : 1.f;
            da[j] = gated ? 1.f : 0.f;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) a[j] = __builtin_amdgcn_rcpf(1.f + __expf(-g[j]));  // within 1 ulp of the quotient
    if (act == kActSigmoid) {
        if constexpr (kGrad) {
#pragma unroll
            for (int j = 0; j < V; ++j) da[j] = a[j] * (1.f - a[j]);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const float s = a[j];
        a[j] = g[j] * s;
        if constexpr (kGrad) da[j] = s * fmaf(g[j], 1.f - s, 1.f);
    }
}

// V elements of an optional [C] parameter
template <int V>
__device__ __forceinline__ void load_or(const float* p, int64_t c, float otherwise, float (&f)[V]) {
    if (p != nullptr) {
        load<V>(p + c, f);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = otherwise;
    }
}

// 1 / sqrt, within 1 ulp
__device__ __forceinline__ float rsqrt1(float x) { return __builtin_amdgcn_rsqf(x); }

constexpr int kBlock = 256;

// Workgroups counted over two dimensions of the grid: one holds fewer than 2^32 threads.
dim3 grid_of(int64_t blocks) {
    constexpr int64_t kMost = int64_t{1} << 20;
    if (blocks <= kMost) return dim3(static_cast<unsigned>(blocks));
    return dim3(static_cast<unsigned>(kMost), static_cast<unsigned>((blocks + kMost - 1) / kMost));
}
__device__ __forceinline__ int64_t block_id() { return static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x; }

constexpr int kPairs = 1024;      // channels from which a thread of the block norm holds two vectors
constexpr int kScalarVecs = 16;  // elements a lane of the element-by-element path: G up to 1024

// What a lane holds of its head: NV vectors of V channels, vector i at channel (i lanes + lane) V.
template <typename TY, typename TG, int V, int NV>
__global__ void __launch_bounds__(kBlock) head_norm_kernel(HeadNormArgs P) {
    const int lanes = P.lanes, lane = threadIdx.x & (lanes - 1);
    const int64_t id = block_id() * (kBlock / lanes) + threadIdx.x / lanes;
    const bool live = id < P.rows * P.H;
    const int64_t h = id % P.H, base = id * P.G, wb = h * P.G;
    const int G = static_cast<int>(P.G);
    const float inv_g = 1.f / static_cast<float>(G);
    float y[NV][V];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * lanes + lane) * V;
        if (live && c < G) {
            load<V>(static_cast<const TY*>(P.y) + base + c, y[i]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) y[i][j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) sum += y[i][j];
    }
    const float mean = P.center ? sum_lanes(sum, lanes) * inv_g : 0.f;
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if ((i * lanes + lane) * V < G) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                y[i][j] -= mean;
                sq = fmaf(y[i][j], y[i][j], sq);
            }
        }
    }
    const float inv = rsqrt1(sum_lanes(sq, lanes) * inv_g + P.eps);
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * lanes + lane) * V;
        if (c >= G) continue;
        float w[V], b[V], g[V], a[V], da[V];
        load<V>(P.weight + wb + c, w);
        load_or<V>(P.bias, wb + c, 0.f, b);
        if (P.gate != nullptr) load<V>(static_cast<const TG*>(P.gate) + base + c, g);
        activate<V, false>(P.act, P.gate != nullptr, g, a, da);
#pragma unroll
        for (int j = 0; j < V; ++j) y[i][j] = fmaf(y[i][j] * inv, w[j], b[j]) * a[j];
        store<V>(static_cast<TG*>(P.out) + base + c, y[i]);
    }
}

// A workgroup takes hpb consecutive heads of rows r0, r0 + step, .., `rpb` rows at a time, and adds its
// rows' sums in LDS at the end.
template <typename TY, typename TG, int V, int NV>
__global__ void __launch_bounds__(kBlock) head_norm_bwd_kernel(HeadNormArgs P) {
    extern __shared__ float part[];  // [rpb][hpb G]
    const int lanes = P.lanes, lane = threadIdx.x & (lanes - 1), slot = threadIdx.x / lanes;
    const int hpb = P.hpb, rpb = kBlock / lanes / hpb;
    const int64_t hblocks = (P.H + hpb - 1) / hpb;
    const int64_t hb = block_id() % hblocks, chunk = block_id() / hblocks;
    if (chunk >= P.chunks) return;  // (a whole workgroup, behind the last one of a grid of two dimensions)
    const int hs = slot % hpb, rs = slot / hpb;
    const int64_t h = hb * hpb + hs;
    const int G = static_cast<int>(P.G);
    const int64_t C = P.H * P.G, wb = h * P.G;
    const float inv_g = 1.f / static_cast<float>(G);
    float w[NV][V], b[NV][V], dw[NV][V], db[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * lanes + lane) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) w[i][j] = b[i][j] = dw[i][j] = db[i][j] = 0.f;
        if (h < P.H && c < G) {
            load<V>(P.weight + wb + c, w[i]);
            if (P.bias != nullptr) load<V>(P.bias + wb + c, b[i]);
        }
    }
    for (int64_t r0 = chunk * rpb; r0 < P.rows; r0 += P.chunks * rpb) {
        const int64_t row = r0 + rs;
        const bool live = h < P.H && row < P.rows;
        const int64_t base = row * C + h * P.G;
        float y[NV][V], go[NV][V], g[NV][V];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * lanes + lane) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) y[i][j] = go[i][j] = g[i][j] = 0.f;
            if (live && c < G) {
                load<V>(static_cast<const TY*>(P.y) + base + c, y[i]);
                load<V>(static_cast<const TG*>(P.gout) + base + c, go[i]);
                if (P.gate != nullptr) load<V>(static_cast<const TG*>(P.gate) + base + c, g[i]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) sum += y[i][j];
        }
        const float mean = P.center ? sum_lanes(sum, lanes) * inv_g : 0.f;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((i * lanes + lane) * V < G) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    y[i][j] -= mean;
                    sq = fmaf(y[i][j], y[i][j], sq);
                }
            }
        }
        const float scaled = sum_lanes(sq, lanes) * inv_g + P.eps;
        const float inv = live ? rsqrt1(scaled) : 0.f;  // (a slot without a row adds 0 to the sums, with eps 0 too)
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float a[V], da[V];
            activate<V, true>(P.act, P.gate != nullptr, g[i], a, da);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float yh = y[i][j] * inv, dz = go[i][j] * a[j];
                g[i][j] = go[i][j] * fmaf(yh, w[i][j], b[i][j]) * da[j];
                dw[i][j] = fmaf(dz, yh, dw[i][j]);
                db[i][j] += dz;
                const float d = dz * w[i][j];
                s1 += d;
                s2 = fmaf(d, yh, s2);
                y[i][j] = yh;
                go[i][j] = d;
            }
        }
        s1 = P.center ? sum_lanes(s1, lanes) * inv_g : 0.f;
        s2 = sum_lanes(s2, lanes) * inv_g;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * lanes + lane) * V;
            if (c >= G) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) y[i][j] = inv * fmaf(-y[i][j], s2, go[i][j] - s1);
            store<V>(static_cast<TY*>(P.dy) + base + c, y[i]);
            if (P.gate != nullptr) store<V>(static_cast<TG*>(P.dgate) + base + c, g[i]);
        }
    }
    // the workgroup's rows in order, first dweight, then dbias
    for (int what = 0; what < (P.bias != nullptr ? 2 : 1); ++what) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * lanes + lane) * V;
            if (c >= G) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) part[(rs * hpb + hs) * G + c + j] = what ? db[i][j] : dw[i][j];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < hpb * G; i += kBlock) {
            if (hb * hpb * G + i >= C) continue;
            float s = 0.f;
            for (int q = 0; q < rpb; ++q) s += part[q * hpb * G + i];
            P.ws[(what * P.chunks + chunk) * C + hb * hpb * G + i] = s;
        }
    }
}

// Partial sums [rows][cols] at part[k] to out[k][cols], k = blockIdx.y: 16 columns and 64 runs of rows a
// workgroup, each run and then the runs in order.
struct ReduceArgs {
    int64_t rows, cols;
    int count = 0;
    const float* part[5];
    float* out[5];
    void add(const float* from, float* to) {
        part[count] = from;
        out[count++] = to;
    }
};

__global__ void __launch_bounds__(1024) norm_reduce_kernel(ReduceArgs P) {
    __shared__ float s[64][17];
    const int c = threadIdx.x & 15, run = threadIdx.x >> 4;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 16 + c;
    const float* part = P.part[blockIdx.y];
    float a = 0.f;
    if (col < P.cols) {
#pragma unroll 8  // eight reads on their way: with few columns a run is nothing but latency (2048 x 128 12 us -> 5)
        for (int64_t r = run; r < P.rows; r += 64) a += part[r * P.cols + col];
    }
    s[run][c] = a;
    __syncthreads();
    if (run == 0 && col < P.cols) {
        float t = 0.f;
        for (int i = 0; i < 64; ++i) t += s[i][c];
        P.out[blockIdx.y][col] = t;
    }
}

hipError_t launch_reduce(const ReduceArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(norm_reduce_kernel, dim3(static_cast<unsigned>((a.cols + 15) / 16), a.count), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

// ---- block norm -----------------------------------------------------------------------------------

// Sums of K values over the `threads` threads that hold a row (64: one wave; else the whole workgroup),
// to all of them.  Every call of a row uses another half of the table, so one barrier a call is enough.
template <int K>
__device__ __forceinline__ void row_sums(float (&x)[K], int threads, float (*tab)[16][K], int& turn) {
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = sum_lanes(x[k], 64);
    if (threads == 64) return;
    const int waves = threads / 64, wv = threadIdx.x / 64;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) tab[turn][wv][k] = x[k];
    }
    __syncthreads();
    const int i = threadIdx.x & (waves - 1);  // a power of two
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = sum_lanes(tab[turn][i][k], waves);
}

// `threads` threads hold a row, vector i of a thread at channel (i threads + thread) V.  With 64 the
// workgroup's other waves hold other rows.
template <typename TX, typename TY, int V, int NV>
__global__ void __launch_bounds__(1024) block_norm_kernel(BlockNormArgs P) {
    __shared__ float tab[2][16][1];
    int turn = 0;
    const int n = P.threads, th = threadIdx.x % n;
    const int64_t row = block_id() * (blockDim.x / n) + threadIdx.x / n;
    if (row >= P.rows) return;  // a whole wave of a 64-thread row; a whole workgroup otherwise
    const int C = static_cast<int>(P.C);
    const float inv_c = 1.f / static_cast<float>(C);
    const int64_t base = row * P.C;
    // every input is on its way before the first sum waits for its own
    Raw<TY, V> ry[NV], rg[NV];
    Raw<TX, V> rx[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * n + th) * V;
        if (c >= C) continue;
        ry[i].fetch(static_cast<const TY*>(P.y) + base + c);
        rx[i].fetch(static_cast<const TX*>(P.x) + base + c);
        if (P.gate != nullptr) rg[i].fetch(static_cast<const TY*>(P.gate) + base + c);
    }
    float z[NV][V];
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int j = 0; j < V; ++j) z[i][j] = 0.f;
        if ((i * n + th) * V < C) ry[i].get(z[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) s[0] += z[i][j];
    }
    if (P.post_w != nullptr) {
        float mean = 0.f;
        if (P.center) {
            row_sums<1>(s, n, tab, turn);
            mean = s[0] * inv_c;
        }
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((i * n + th) * V >= C) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                z[i][j] -= mean;
                s[0] = fmaf(z[i][j], z[i][j], s[0]);
            }
        }
        row_sums<1>(s, n, tab, turn);
        const float inv = rsqrt1(s[0] * inv_c + P.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * n + th) * V;
            if (c >= C) continue;
            float w[V], b[V];
            load<V>(P.post_w + c, w);
            load_or<V>(P.post_b, c, 0.f, b);
#pragma unroll
            for (int j = 0; j < V; ++j) z[i][j] = fmaf(z[i][j] * inv, w[j], b[j]);
        }
    }
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * n + th) * V;
        if (c >= C) continue;
        float x[V], g[V], sc[V], a[V], da[V];
        rx[i].get(x);
        if (P.gate != nullptr) rg[i].get(g);
        load_or<V>(P.scale, c, 1.f, sc);
        activate<V, false>(P.act, P.gate != nullptr, g, a, da);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            z[i][j] = fmaf(z[i][j], a[j] * sc[j], x[j]);
            s[0] += z[i][j];
        }
        store<V>(static_cast<TX*>(P.x_out) + base + c, z[i]);
    }
    float mean = 0.f;
    if (P.center) {
        row_sums<1>(s, n, tab, turn);
        mean = s[0] * inv_c;
    }
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if ((i * n + th) * V >= C) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            z[i][j] -= mean;
            s[0] = fmaf(z[i][j], z[i][j], s[0]);
        }
    }
    row_sums<1>(s, n, tab, turn);
    const float inv = rsqrt1(s[0] * inv_c + P.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * n + th) * V;
        if (c >= C) continue;
        float w[V], b[V];
        load<V>(P.pre_w + c, w);
        load_or<V>(P.pre_b, c, 0.f, b);
#pragma unroll
        for (int j = 0; j < V; ++j) z[i][j] = fmaf(z[i][j] * inv, w[j], b[j]);
        store<V>(static_cast<TY*>(P.h) + base + c, z[i]);
    }
}

// The rows of slot q (of `slots`): q, q + slots, ..  Partial sums [5][slots][C]: dpre_w, dpre_b, dpost_w,
// dpost_b, dscale.
//
// A row's inputs are fetched while the row before it is worked on (NV == 1), and the channels' four weights
// are kept in registers beside the five sums; with NV > 1 there is room for neither.
template <typename TX, typename TY, int V, int NV, int Threads>
__global__ void __launch_bounds__(Threads) block_norm_bwd_kernel(BlockNormArgs P) {
    __shared__ float tab[2][16][2];
    constexpr bool kAhead = NV == 1;
    int turn = 0;
    const int n = P.threads, th = threadIdx.x % n;
    const int64_t slot = static_cast<int64_t>(blockIdx.x) * (blockDim.x / n) + threadIdx.x / n;
    // A spare wave of the last workgroup (with 64 threads a row only, where nothing waits at a barrier).  Its rows
    // are other slots' rows, whose gx may already hold their dx.
    if (slot >= P.slots) return;
    const int C = static_cast<int>(P.C);
    const float inv_c = 1.f / static_cast<float>(C);
    const bool post = P.post_w != nullptr, gated = P.gate != nullptr;
    float acc[5][NV][V];
#pragma unroll
    for (int k = 0; k < 5; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) acc[k][i][j] = 0.f;
    struct Weights {
        float pre[V], post[V], bias[V], scale[V];
    };
    const auto weights = [&](int c, Weights& w) {
        load<V>(P.pre_w + c, w.pre);
        load_or<V>(P.post_w, c, 1.f, w.post);
        load_or<V>(P.post_b, c, 0.f, w.bias);
        load_or<V>(P.scale, c, 1.f, w.scale);
    };
    Raw<TX, V> rx[NV], rt[kAhead ? NV : 1];
    Raw<TY, V> ry[NV], rd[NV], rg[kAhead ? NV : 1];
    const auto fetch_late = [&](int64_t at, int i) {  // needed after the statistics only
        if (gated) rg[i].fetch(static_cast<const TY*>(P.gate) + at);
        if (P.gx != nullptr) rt[i].fetch(static_cast<const TX*>(P.gx) + at);
    };
    const auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * n + th) * V;
            if (c >= C) continue;
            const int64_t at = row * P.C + c;
            rx[i].fetch(static_cast<const TX*>(P.x) + at);
            ry[i].fetch(static_cast<const TY*>(P.y) + at);
            rd[i].fetch(static_cast<const TY*>(P.gh) + at);
            if constexpr (kAhead) fetch_late(at, i);
        }
    };
    Weights kept;
    if (kAhead && th * V < C) weights(th * V, kept);
    if (kAhead && slot < P.rows) fetch(slot);
    for (int64_t row = slot; row < P.rows; row += P.slots) {  // the same trip count for a row's threads
        const int64_t base = row * P.C;
        if constexpr (!kAhead) fetch(row);
        float x[NV][V], y[NV][V], d[NV][V], g[V], t[V];
        const auto late = [&](int i) {
#pragma unroll
            for (int j = 0; j < V; ++j) g[j] = t[j] = 0.f;
            if (gated) rg[i].get(g);
            if (P.gx != nullptr) rt[i].get(t);
        };
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int j = 0; j < V; ++j) x[i][j] = y[i][j] = d[i][j] = 0.f;
            if ((i * n + th) * V < C) {
                rx[i].get(x[i]);
                ry[i].get(y[i]);
                rd[i].get(d[i]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                s[0] += x[i][j];
                s[1] += y[i][j];
            }
        }
        if constexpr (kAhead) {
            late(0);
            if (row + P.slots < P.rows) fetch(row + P.slots);
        }
        float mx = 0.f, my = 0.f;
        if (P.center) {
            row_sums<2>(s, n, tab, turn);
            mx = s[0] * inv_c;
            my = post ? s[1] * inv_c : 0.f;
        }
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((i * n + th) * V >= C) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                x[i][j] -= mx;
                s[0] = fmaf(x[i][j], x[i][j], s[0]);
                y[i][j] -= my;
                s[1] = fmaf(y[i][j], y[i][j], s[1]);
            }
        }
        row_sums<2>(s, n, tab, turn);
        const float ix = rsqrt1(s[0] * inv_c + P.eps);
        const float iy = post ? rsqrt1(s[1] * inv_c + P.eps) : 1.f;
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * n + th) * V;
            if (c >= C) continue;
            float w[V];
            if constexpr (!kAhead) load<V>(P.pre_w + c, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                x[i][j] *= ix;
                y[i][j] *= iy;
                acc[0][i][j] = fmaf(d[i][j], x[i][j], acc[0][i][j]);
                acc[1][i][j] += d[i][j];
                d[i][j] *= kAhead ? kept.pre[j] : w[j];
                s[0] += d[i][j];
                s[1] = fmaf(d[i][j], x[i][j], s[1]);
            }
        }
        row_sums<2>(s, n, tab, turn);
        const float m1 = P.center ? s[0] * inv_c : 0.f, m2 = s[1] * inv_c;
        s[0] = s[1] = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * n + th) * V;
            if (c >= C) continue;
            Weights here;
            if constexpr (!kAhead) weights(c, here);
            if constexpr (!kAhead) {
                fetch_late(base + c, 0);
                late(0);
            }
            const Weights& w = kAhead ? kept : here;
            float a[V], da[V];
            activate<V, true>(P.act, gated, g, a, da);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float dx = fmaf(ix, fmaf(-x[i][j], m2, d[i][j] - m1), t[j]);
                x[i][j] = dx;
                const float z = fmaf(y[i][j], w.post[j], w.bias[j]);
                acc[4][i][j] = fmaf(dx, z * a[j], acc[4][i][j]);
                const float ds = dx * w.scale[j];
                g[j] = ds * z * da[j];
                const float dz = ds * a[j];
                acc[2][i][j] = fmaf(dz, y[i][j], acc[2][i][j]);
                acc[3][i][j] += dz;
                d[i][j] = dz * w.post[j];
                s[0] += d[i][j];
                s[1] = fmaf(d[i][j], y[i][j], s[1]);
            }
            store<V>(static_cast<TX*>(P.dx) + base + c, x[i]);
            if (gated) store<V>(static_cast<TY*>(P.dgate) + base + c, g);
        }
        float p1 = 0.f, p2 = 0.f;
        if (post) {
            row_sums<2>(s, n, tab, turn);
            p1 = P.center ? s[0] * inv_c : 0.f;
            p2 = s[1] * inv_c;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * n + th) * V;
            if (c >= C) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) d[i][j] = iy * fmaf(-y[i][j], p2, d[i][j] - p1);
            store<V>(static_cast<TY*>(P.dy) + base + c, d[i]);
        }
    }
    const bool want[5] = {true, P.pre_b != nullptr, post, P.post_b != nullptr, P.scale != nullptr};
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        if (!want[k]) continue;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * n + th) * V;
            if (c < C) store<V>(P.ws + (k * P.slots + slot) * P.C + c, acc[k][i]);
        }
    }
}

__global__ void zero_kernel(float* p, int64_t n) {
    const int64_t i = block_id() * kBlock + threadIdx.x;
    if (i < n) p[i] = 0.f;
}

int64_t pow2_at_least(int64_t x) {
    int64_t p = 1;
    while (p < x) p *= 2;
    return p;
}

template <typename TY, typename TG, int V, int NV>
hipError_t launch_head(const HeadNormArgs& a, bool bwd, hipStream_t stream) {
    if (!bwd) {
        const int64_t per = kBlock / a.lanes;
        hipLaunchKernelGGL((head_norm_kernel<TY, TG, V, NV>), grid_of((a.rows * a.H + per - 1) / per), dim3(kBlock), 0, stream, a);
        return hipGetLastError();
    }
    const int64_t C = a.H * a.G;
    const size_t lds = static_cast<size_t>(kBlock / a.lanes) * a.G * sizeof(float);
    hipLaunchKernelGGL((head_norm_bwd_kernel<TY, TG, V, NV>), grid_of((a.H + a.hpb - 1) / a.hpb * a.chunks), dim3(kBlock), lds,
                       stream, a);
    hipError_t e = hipGetLastError();
    ReduceArgs r{a.chunks, C};
    r.add(a.ws, a.dweight);
    if (a.bias != nullptr) r.add(a.ws + a.chunks * C, a.dbias);
    return e == hipSuccess ? launch_reduce(r, stream) : e;
}

template <typename TY, typename TG>
hipError_t launch_head_v(const HeadNormArgs& a, bool bwd, hipStream_t stream) {
    if (!a.vec) {  // as many elements a lane as the head needs (16 always: gradients of 64 heads of 100 took nine
                   // times as long as those of as many elements in heads of 128, float32; now 1.2 times)
        if (a.G <= 128) return launch_head<TY, TG, 1, 2>(a, bwd, stream);
        if (a.G <= 256) return launch_head<TY, TG, 1, 4>(a, bwd, stream);
        return launch_head<TY, TG, 1, kScalarVecs>(a, bwd, stream);
    }
    return a.G <= 512 ? launch_head<TY, TG, 8, 1>(a, bwd, stream) : launch_head<TY, TG, 8, 2>(a, bwd, stream);
}

hipError_t launch_head_t(HeadNormArgs a, bool bwd, hipStream_t stream) {
    if (a.shared) {  // one weight for all heads: rows H rows of one head
        a.rows *= a.H;
        a.H = 1;
    }
    a.lanes = a.vec ? static_cast<int>(pow2_at_least(a.G / 8 < 64 ? a.G / 8 : 64)) : 64;
    const int slots = kBlock / a.lanes;
    // heads side by side for at least 512 bytes a row of bf16, the workgroup's other slots over rows
    a.hpb = 1;
    while (a.hpb < slots && a.hpb < a.H && a.hpb * a.G < 256) a.hpb *= 2;
    a.chunks = head_norm_chunks(a.rows, a.H * a.G);
    if (a.y_bf16) return launch_head_v<uint16_t, uint16_t>(a, bwd, stream);
    return a.bf16 ? launch_head_v<float, uint16_t>(a, bwd, stream) : launch_head_v<float, float>(a, bwd, stream);
}

template <typename TX, typename TY, int V, int NV>
hipError_t launch_block_fwd(const BlockNormArgs& a, hipStream_t stream) {
    const int64_t block = a.threads == 64 ? 256 : a.threads, per = block / a.threads;
    hipLaunchKernelGGL((block_norm_kernel<TX, TY, V, NV>), grid_of((a.rows + per - 1) / per), dim3(static_cast<unsigned>(block)),
                       0, stream, a);
    return hipGetLastError();
}

template <typename TX, typename TY, int V, int NV, int Threads>
hipError_t launch_block_bwd(const BlockNormArgs& a, hipStream_t stream) {
    const int64_t block = a.threads == 64 ? 256 : a.threads, per = block / a.threads;
    hipLaunchKernelGGL((block_norm_bwd_kernel<TX, TY, V, NV, Threads>), dim3(static_cast<unsigned>((a.slots + per - 1) / per)),
                       dim3(static_cast<unsigned>(block)), 0, stream, a);
    hipError_t e = hipGetLastError();
    float* const out[5] = {a.dpre_w, a.pre_b ? a.dpre_b : nullptr, a.post_w ? a.dpost_w : nullptr,
                           a.post_b ? a.dpost_b : nullptr, a.scale ? a.dscale : nullptr};
    ReduceArgs r{a.slots, a.C};
    for (int k = 0; k < 5; ++k)
        if (out[k] != nullptr) r.add(a.ws + k * a.slots * a.C, out[k]);
    return e == hipSuccess ? launch_reduce(r, stream) : e;
}

// Threads that hold a row: a wave up to 512 channels, else 8 channels each from the smallest count that does (the
// forward 16 from kPairs channels, half the threads to sum over: 8192 rows of 4096 with everything given 75 us
// against 80; the backward 16 above 4096, for which 1024 threads have not the registers: 4096 rows of 8192 259 us
// against 656).  Off the 16-byte grid, single elements: 512 threads in the forward up to 4096 (4096 rows of 1001
// 24 us; 1024 threads 37), else 1024 (of 8191 140 us; 512 threads 214), and 1024 in the backward (of 4001 241 us;
// 512 threads, which spill, 319).  All of these in bf16.
template <typename TX, typename TY>
hipError_t launch_block_v(BlockNormArgs a, bool bwd, hipStream_t stream) {
    a.slots = block_norm_slots(a.rows, a.C);
    const int wide = static_cast<int>(pow2_at_least((a.C + 7) / 8));
    if (!bwd) {
        a.threads = a.C <= 512 ? 64 : !a.vec ? (a.C <= 4096 ? 512 : 1024) : a.C < kPairs ? wide : wide / 2;
        if (!a.vec) return launch_block_fwd<TX, TY, 1, 8>(a, stream);
        return a.C < kPairs ? launch_block_fwd<TX, TY, 8, 1>(a, stream) : launch_block_fwd<TX, TY, 8, 2>(a, stream);
    }
    a.threads = a.C <= 512 ? 64 : !a.vec ? 1024 : a.C <= 4096 ? wide : 512;
    if (a.vec) return a.C <= 4096 ? launch_block_bwd<TX, TY, 8, 1, 512>(a, stream) : launch_block_bwd<TX, TY, 8, 2, 512>(a, stream);
    if (a.C <= 512) return launch_block_bwd<TX, TY, 1, 8, 512>(a, stream);
    return a.C <= 4096 ? launch_block_bwd<TX, TY, 1, 4, 1024>(a, stream) : launch_block_bwd<TX, TY, 1, 8, 1024>(a, stream);
}

hipError_t launch_block_t(const BlockNormArgs& a, bool bwd, hipStream_t stream) {
    if (a.x_bf16) return launch_block_v<uint16_t, uint16_t>(a, bwd, stream);
    return a.bf16 ? launch_block_v<float, uint16_t>(a, bwd, stream) : launch_block_v<float, float>(a, bwd, stream);
}

}  // namespace

// Rows of partial sums of a head norm's backward: enough workgroups to fill the card (256 channels each),
// and no fewer than 32 rows behind each.
int64_t head_norm_chunks(int64_t rows, int64_t C) {
    const int64_t most = (int64_t{1} << 19) / C, n = (rows + 31) / 32;
    const int64_t cap = most < 32 ? 32 : most > 2048 ? 2048 : most;
    return n < cap ? n : cap;
}

// Rows of partial sums of a block norm's backward: 8 waves a compute unit, 4 rows or more behind each.
int64_t block_norm_slots(int64_t rows, int64_t C) {
    const int64_t threads = C <= 512 ? 64 : C > 4096 ? 512 : pow2_at_least((C + 7) / 8);
    const int64_t most = 256 * 512 / threads, n = (rows + 3) / 4;
    return n < most ? n : most;
}

hipError_t launch_zero(float* p, int64_t n, hipStream_t stream) {
    if (p == nullptr || n <= 0) return hipSuccess;
    hipLaunchKernelGGL(zero_kernel, grid_of((n + kBlock - 1) / kBlock), dim3(kBlock), 0, stream, p, n);
    return hipGetLastError();
}

hipError_t launch_head_norm(const HeadNormArgs& a, hipStream_t stream) { return launch_head_t(a, false, stream); }
hipError_t launch_head_norm_bwd(const HeadNormArgs& a, hipStream_t stream) { return launch_head_t(a, true, stream); }
hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream) { return launch_block_t(a, false, stream); }
hipError_t launch_block_norm_bwd(const BlockNormArgs& a, hipStream_t stream) { return launch_block_t(a, true, stream); }

}  // namespace wkv
