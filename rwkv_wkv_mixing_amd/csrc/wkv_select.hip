// Selective state space scan: per channel a diagonal state of N numbers whose decay and whose writes depend on the
// token.  With a_t = e^{-delta_t w}, delta_t = softplus(dt_t + dt_bias):
//     h_t[n] = a_t[n] h_{t-1}[n] + delta_t x_t b_t[n],   y_t = sum_n c_t[n] h_t[n] + d x_t,   out_t = y_t silu(z_t)
// b and c are shared by the channels of a group.  Every (channel, n) decays at a rate of its own, so nothing here is a
// matrix product: the work is one exponential, two multiplications and two multiply-adds a (token, channel, n) on the
// vector units, which is what bounds it (a channel-token of N = 16 moves 8 bytes in bf16 and takes some 130 lane
// instructions: 4.9 us a million of them, 1.3 for the bytes).
//
// A workgroup takes 64 channels, a lane each, and its W waves share out the N states, four or two a wave: a
// wave's b_t and c_t are then the same for all its lanes and reach its multiplications as lane broadcasts, and only
// delta, the written value and the waves' parts of y pass through LDS.  Tiles of 16 tokens: the threads first work out
// delta and what is written for (token, channel) pairs, one each; then every wave walks the tile; then the threads add
// the waves' parts, gate and store.
//
// Measured at B = 8, T = 1024, C = 4096, bf16 (the data alone would take 43 us forward and 75 us back):
//     N = 8: 140 us forward, 280 us for the gradients;  N = 16: 162 and 396 us.
// At N = 16 two waves a vector unit keep it busy 75 % of the time forward and 80 % in the gradients.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "wkv_lanes.h"
#include "wkv_launch.h"

namespace wkv {
namespace {

constexpr int kTile = kSelectTile;  // tokens a tile
constexpr float kLog2e = 1.44269504088896340736f;

template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ uint16_t narrow<uint16_t>(float x) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(x)); }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// e^{-|x|} by the hardware's exp2 (within 2^-23).  Wide: the rounding of x log2 e, up to |x| 2^-24 of the result, is put back.
template <bool Wide>
__device__ __forceinline__ float exp_neg_abs(float x) {
    const float a = -__builtin_fabsf(x), t = a * kLog2e;
    const float e = exp2_fast(t);
    if constexpr (!Wide) return e;
    const float lost = fmaf(a, kLog2e, -t) + a * 1.92596299e-8f;  // log2 e = kLog2e + 1.92596299e-8
    return a < -100.f ? e : fmaf(e, 0.693147180559945f * lost, e);
}

// log(1 + e) for e in [0, 1]: e times a polynomial through the Chebyshev points of [0, 1] of log(1 + e) / e (within
// 1.3e-7 of it), so a small e keeps its digits.
__device__ __forceinline__ float log1p_unit(float e) {
    float p = -0.0031760570127516985f;
    p = fmaf(p, e, 0.019542526453733444f);
    p = fmaf(p, e, -0.056373611092567444f);
    p = fmaf(p, e, 0.10543623566627502f);
    p = fmaf(p, e, -0.1526966691017151f);
    p = fmaf(p, e, 0.1966327428817749f);
    p = fmaf(p, e, -0.24951615929603577f);
    p = fmaf(p, e, 0.33329710364341736f);
    p = fmaf(p, e, -0.49999892711639404f);
    p = fmaf(p, e, 1.0f);
    return p * e;
}

// The gate's sigmoid, without what its exponent's rounding costs a negative z (|z| 2^-24 of the value): y comes from a state
// that tokens by the hundred have rounded.  (Put back, the float32 forward of 8 x 1024 x 4096 takes 188 us for 181.)
__device__ __forceinline__ float gate_of(float z) { return sigmoid<false>(z); }

// A decay e^{-delta w} from delta and w2 = -w log2 e.  The product's rule is that 0 times anything is 0, so a step of zero keeps
// the state whatever the rate, and a rate of infinity (w2 -inf) forgets it in any other step, however small.
__device__ __forceinline__ float decay(float delta, float w2) {
    return exp2_fast(mul_zero(delta, w2));
}

// delta of some tokens from dt + dt_bias, and its derivative by dt.  Wide with float32 tensors; a bf16 dt is itself rounded by
// 2^-9, next to which the |dt| 2^-24 of a step that is left in is nothing (put back, the bf16 forward of 8 x 1024 x 4096 takes
// 165 us for 162, the gradients 399 for 395).
template <bool Wide, bool Grad, int E>
__device__ __forceinline__ void steps_of(float (&raw)[E], bool softplus, float (&grad)[E]) {
    if (!softplus) {
        if constexpr (Grad) {
#pragma unroll
            for (int k = 0; k < E; ++k) grad[k] = 1.f;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < E; ++k) {
        const float e = exp_neg_abs<Wide>(raw[k]);
        if constexpr (Grad) grad[k] = (raw[k] >= 0.f ? 1.f : e) * __builtin_amdgcn_rcpf(1.f + e);
        raw[k] = __builtin_amdgcn_fmed3f(raw[k], 0.f, __builtin_inff()) + log1p_unit(e);  // (of NaN: 0 + NaN)
    }
}

// The element `bytes` behind place `at` (in bytes, the whole wave's) of a tensor.  Places are counted in bytes all the way:
// a 64-bit place shifted by the size of an element is worked out lane by lane.
template <typename T>
__device__ __forceinline__ T load_at(const T* p, int64_t at, uint32_t bytes) {
    asm("" : "+s"(at));
    return *reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) + at + bytes);
}
template <typename T>
__device__ __forceinline__ void store_at(T* p, int64_t at, uint32_t bytes, T v) {
    *reinterpret_cast<T*>(reinterpret_cast<char*>(p) + at + bytes) = v;
}
// Keeps an offset one of 32 bits in a loop, next to a wave's address, and not part of a sum of 64 bits.
__device__ __forceinline__ void keep32(uint32_t& v) { asm volatile("" : "+v"(v)); }

// The values of lane K of every row of 16 lanes, to the row: folded into the multiplication that takes them.
template <int K>
__device__ __forceinline__ float row_lane(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x150 + K, 0xf, 0xf, true));  // row_newbcast
}

// The sum over the wave's states of (lane K + s of its row of c) h[s].  A lane of another register cannot be read within two
// instructions of a write to that register, which the compiler does not look for inside here: hence the wait, which
// costs this wave a moment and the others of its SIMD nothing.
template <int K>
__device__ __forceinline__ float dot_row(float c, const float (&h)[4]) {
    float y;
    asm("s_nop 1\n\t"
        "v_mul_f32_dpp %0, %1, %2 row_newbcast:%6 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %3 row_newbcast:%7 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %4 row_newbcast:%8 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
        : "=&v"(y) : "v"(c), "v"(h[0]), "v"(h[1]), "v"(h[2]), "v"(h[3]), "n"(K), "n"(K + 1), "n"(K + 2), "n"(K + 3));
    return y;
}
template <int K>
__device__ __forceinline__ float dot_row(float c, const float (&h)[2]) {
    float y;
    asm("s_nop 1\n\t"
        "v_mul_f32_dpp %0, %1, %2 row_newbcast:%4 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %3 row_newbcast:%5 row_mask:0xf bank_mask:0xf"
        : "=&v"(y) : "v"(c), "v"(h[0]), "v"(h[1]), "n"(K), "n"(K + 1));
    return y;
}
// g[s] += (lane K + s of its row of c) v.
template <int K>
__device__ __forceinline__ void add_row(float (&g)[4], float c, float v) {
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %4, %5 row_newbcast:%6 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %4, %5 row_newbcast:%7 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %2, %4, %5 row_newbcast:%8 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %3, %4, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
        : "+v"(g[0]), "+v"(g[1]), "+v"(g[2]), "+v"(g[3])
        : "v"(c), "v"(v), "n"(K), "n"(K + 1), "n"(K + 2), "n"(K + 3));
}
template <int K>
__device__ __forceinline__ void add_row(float (&g)[2], float c, float v) {
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %2, %3 row_newbcast:%4 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %1, %2, %3 row_newbcast:%5 row_mask:0xf bank_mask:0xf"
        : "+v"(g[0]), "+v"(g[1]) : "v"(c), "v"(v), "n"(K), "n"(K + 1));
}

// A token's numbers (b and c of the wave's states) summed over pairs of lanes 8 apart, then over mirrored lanes of an eight (i
// and 7 - i): state 0 + (bit 2 of the lane) of b (bit 3: of c) in q0, of four states state 2 + (bit 2) in q1.  The four lanes
// that agree in bits 2 to 5 hold a sum's parts between them, whichever lane a mirror gave which, until they are added up
// behind the tile.  An addition with a lane exchange writes the quarters
// of its rows that the number belongs to, so two of them add up two numbers into one register.  The first wait is
// for what the products before have written, the last one for the exchange that reads the results; in between nothing is
// read through an exchange sooner than three instructions after it is written.
__device__ __forceinline__ void fold_rows(const float (&b)[4], const float (&c)[4], float& q0, float& q1) {
    float r0, r1, r2, r3;
    asm("s_nop 1\n\t"
        "v_add_f32_dpp %2, %6, %6 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %2, %10, %10 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %3, %7, %7 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %3, %11, %11 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %4, %8, %8 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %4, %12, %12 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %5, %9, %9 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %5, %13, %13 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %0, %2, %2 row_half_mirror row_mask:0xf bank_mask:0x5\n\t"
        "v_add_f32_dpp %0, %3, %3 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
        "v_add_f32_dpp %1, %4, %4 row_half_mirror row_mask:0xf bank_mask:0x5\n\t"
        "v_add_f32_dpp %1, %5, %5 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
        "s_nop 1"
        : "=&v"(q0), "=&v"(q1), "=&v"(r0), "=&v"(r1), "=&v"(r2), "=&v"(r3)
        : "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "v"(c[0]), "v"(c[1]), "v"(c[2]), "v"(c[3]));
}

__device__ __forceinline__ void fold_rows(const float (&b)[2], const float (&c)[2], float& q0) {
    float r0, r1;
    asm("s_nop 1\n\t"
        "v_add_f32_dpp %1, %3, %3 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %1, %5, %5 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "v_add_f32_dpp %2, %4, %4 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
        "v_add_f32_dpp %2, %6, %6 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
        "s_nop 1\n\t"
        "v_add_f32_dpp %0, %1, %1 row_half_mirror row_mask:0xf bank_mask:0x5\n\t"
        "v_add_f32_dpp %0, %2, %2 row_half_mirror row_mask:0xf bank_mask:0xa\n\t"
        "s_nop 1"
        : "=&v"(q0), "=&v"(r0), "=&v"(r1) : "v"(b[0]), "v"(b[1]), "v"(c[0]), "v"(c[1]));
}

// A wave's NS values a token of b or c for a tile: every row of 16 lanes holds the 16 NS numbers of the tile's tokens in
// NS registers, token by token, so that each of them is one lane of one register.
template <typename T, int NS>
struct Row {
    static constexpr int kPer = 16 / NS, kRegs = kTile / kPer;  // tokens a register, registers
    T raw[kRegs];
    float f[kRegs];
    // where a lane reads: its state, its token of the first register's, the bytes from token to token
    struct Where {
        uint32_t stride, s, first;
        int j;
    };
    static __device__ __forceinline__ Where where(int64_t GN, int lane) {
        Where w;
        w.stride = static_cast<uint32_t>(GN) * sizeof(T);
        w.s = (lane % NS) * sizeof(T);
        w.j = (lane & 15) / NS;
        w.first = w.j * w.stride + w.s;
        return w;
    }
    // the tile's tokens from p on, `left` of them there (at least one): the others are zeros
    __device__ __forceinline__ void fetch(const T* p, int64_t at, Where& w, int left) {
        keep32(w.first);
        if (left >= kTile) {
#pragma unroll
            for (int r = 0; r < kRegs; ++r) raw[r] = load_at(p, at + static_cast<int64_t>(r * kPer) * w.stride, w.first);
        } else {
#pragma unroll
            for (int r = 0; r < kRegs; ++r) {
                const int j = r * kPer + w.j;
                const T v = load_at(p, at, (j < left ? j : left - 1) * w.stride + w.s);
                raw[r] = j < left ? v : T{0};
            }
        }
    }
    __device__ __forceinline__ void ready() {
#pragma unroll
        for (int r = 0; r < kRegs; ++r) {
            f[r] = widen(raw[r]);
            asm volatile("" : "+v"(f[r]));  // (here and now, not where it is used)
        }
    }
    // The compiler is to broadcast again rather than keep what it broadcast before.
    __device__ __forceinline__ void forget() {
#pragma unroll
        for (int r = 0; r < kRegs; ++r) asm volatile("" : "+v"(f[r]));
    }
    // the lane and the register of token J's first state
    template <int J>
    static constexpr int lane_of() { return J * NS % 16; }
    template <int J>
    __device__ __forceinline__ float reg() const { return f[J * NS / 16]; }
    template <int J, int S>
    __device__ __forceinline__ float get() const { return row_lane<lane_of<J>() + S>(reg<J>()); }
};

// Past: past the caches.
template <bool Past = false, int NS>
__device__ __forceinline__ void load_states(const float* p, bool valid, float (&h)[NS]) {
    typedef float Some __attribute__((ext_vector_type(NS)));
    Some v = {};
    if constexpr (Past) {
        if (valid) v = __builtin_nontemporal_load(reinterpret_cast<const Some*>(p));
    } else {
        if (valid) v = *reinterpret_cast<const Some*>(p);
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) h[i] = v[i];
}
template <bool Past = false, int NS>
__device__ __forceinline__ void store_states(float* p, const float (&h)[NS]) {
    typedef float Some __attribute__((ext_vector_type(NS)));
    Some v;
#pragma unroll
    for (int i = 0; i < NS; ++i) v[i] = h[i];
    if constexpr (Past) __builtin_nontemporal_store(v, reinterpret_cast<Some*>(p));
    else *reinterpret_cast<Some*>(p) = v;
}

// Where a workgroup works: tile of channels, batch row, segment; its lane's channel and its tokens.
struct Place {
    int64_t b;           // batch row
    uint32_t ch;         // the lane's channel (a spare lane's: the last one of its group)
    int ct, g, seg;
    int t0, t1, te;      // rows t0 .. t1 - 1 of which those before te are tokens
    bool valid;          // not a spare lane
};

// The batch row of the slot-th workgroups: of up to 64 ragged rows the longest first, so that the last workgroups to begin are
// short ones.  Each workgroup ranks the rows for itself, a row a lane (4096 channels, N = 16, bf16, random lengths, in the
// order given and so: 32 rows of up to 2048 tokens forward 740 -> 652 us, gradients 2300 -> 1900; 6 of up to 1501 189 ->
// 179 and 469 -> 438; 3 of up to 200 tokens of 2048 channels 24.3 -> 24.7).
__device__ __forceinline__ uint32_t row_of(const SelectArgs& P, uint32_t slot, int lane) {
    const int B = static_cast<int>(P.B);
    if (P.lengths == nullptr || B > 64) return slot;
    const int len = lane < B ? P.lengths[lane] : 0;
    int before = 0;
    for (int k = 0; k < B; ++k) {
        const int other = __builtin_amdgcn_readlane(len, k);
        before += other > len || (other == len && k < lane) ? 1 : 0;
    }
    return static_cast<uint32_t>(__builtin_ctzll(__ballot(lane < B && before == static_cast<int>(slot))));
}

__device__ __forceinline__ Place place_of(const SelectArgs& P, int lane, int first_seg = 0) {
    Place p;
    const uint32_t nct = static_cast<uint32_t>(P.ctiles);
    // (quotients are worked out in vector registers: readfirstlane says that they are the wave's)
    const uint32_t blk = blockIdx.x, rest = __builtin_amdgcn_readfirstlane(blk / nct);
    p.ct = __builtin_amdgcn_readfirstlane(blk - rest * nct);
    const int seg = __builtin_amdgcn_readfirstlane(rest / static_cast<uint32_t>(P.B));
    p.b = row_of(P, rest - static_cast<uint32_t>(seg) * static_cast<uint32_t>(P.B), lane);
    p.seg = first_seg + seg;
    const int per_group = __builtin_amdgcn_readfirstlane(P.ctiles / static_cast<int>(P.G));
    p.g = __builtin_amdgcn_readfirstlane(p.ct / per_group);
    const int width = __builtin_amdgcn_readfirstlane(static_cast<int>(P.C) / static_cast<int>(P.G)), c = (p.ct - p.g * per_group) * 64 + lane;
    p.valid = c < width;
    p.ch = static_cast<uint32_t>(p.g * width + (p.valid ? c : width - 1));
    const int T = static_cast<int>(P.T), seg_len = static_cast<int>(P.seg_len);
    int len = P.lengths != nullptr ? __builtin_amdgcn_readfirstlane(P.lengths[p.b]) : T;
    len = len < 0 ? 0 : len > T ? T : len;
    p.t0 = p.seg * seg_len;
    p.t1 = T - p.t0 < seg_len ? T : p.t0 + seg_len;
    p.te = len < p.t0 ? p.t0 : len < p.t1 ? len : p.t1;
    return p;
}

// Where a wave's states of its lane before the tile at t are kept: [B, tiles, N / 4, C, 4].
template <int NS>
__device__ __forceinline__ int64_t saved_at(const SelectArgs& P, const Place& p, int t, int wave, int N) {
    return (((p.b * P.tiles + t / kTile) * (N / 4) + wave * NS / 4) * P.C + p.ch) * 4 + wave * NS % 4;
}

// Two workgroups on a compute unit do not share it evenly: the waves that came first go first, so one workgroup is done
// early and the other one walks its rest alone, which leaves the vector units waiting (132 and 182 us at B = 8, T = 1024,
// C = 4096, N = 16).  A wave's priority falls with every quarter of its tiles, so that who is behind goes first: the
// forward 188 -> 180 us, the gradients 465 -> 447.
__device__ __forceinline__ void yield_to_later(int done, int all) {
    const int quarter = (all + 3) / 4;
    if (done == 0) __builtin_amdgcn_s_setprio(3);
    else if (done == quarter) __builtin_amdgcn_s_setprio(2);
    else if (done == 2 * quarter) __builtin_amdgcn_s_setprio(1);
    else if (done == 3 * quarter) __builtin_amdgcn_s_setprio(0);
}

// What a walk does: the outputs; what each segment does to a state of zero; the same for the states' gradients, from
// the last token to the first: g <- a (g + c gy).
enum { kWalkOut = 0, kWalkLocal = 1, kWalkAdjoint = 2, kGrad = 3 };  // kGrad: select_grad_kernel

template <typename T, int NS, int W, int Mode>
__global__ __launch_bounds__(64 * W) void select_walk_kernel(SelectArgs P) {
    constexpr int N = NS * W, kEach = kTile / W;  // (token, channel) pairs a thread works out
    constexpr bool kWide = sizeof(T) == 4, kOut = Mode == kWalkOut, kAdj = Mode == kWalkAdjoint;
    __shared__ float2 put[2][kTile][64];                         // delta and the written value
    __shared__ float parts[kOut ? 2 : 1][kOut ? W : 1][kTile][64];  // the waves' parts of y
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place p = place_of(P, lane, kAdj ? 1 : 0);  // (what the last, or backwards the first, segment does is not asked for)
    const T* __restrict__ x = static_cast<const T*>(P.x);
    const T* __restrict__ dt = static_cast<const T*>(P.dt);
    const T* __restrict__ z = static_cast<const T*>(P.z);
    const T* __restrict__ go = static_cast<const T*>(P.go);
    T* __restrict__ out = static_cast<T*>(P.out);
    const int64_t row0 = p.b * P.T, GN = P.G * N;
    const T* bt = static_cast<const T*>(kAdj ? P.c : P.b) + (row0 * GN + p.g * N + wave * NS);
    const T* ct = static_cast<const T*>(P.c) + (row0 * GN + p.g * N + wave * NS);
    const float bias = P.dt_bias != nullptr ? P.dt_bias[p.ch] : 0.f;
    const float skip = P.d != nullptr ? P.d[p.ch] : 0.f;
    const int ntiles = (p.te - p.t0 + kTile - 1) / kTile;

    float w2[NS], h[NS];
    load_states(P.w + static_cast<int64_t>(p.ch) * N + wave * NS, true, w2);
#pragma unroll
    for (int i = 0; i < NS; ++i) w2[i] = -w2[i] * kLog2e, h[i] = 0.f;
    const int64_t state = (p.b * P.C + p.ch) * N + wave * NS;
    if constexpr (kOut) {
        if (P.nseg > 1) load_states(P.local + (static_cast<int64_t>(p.seg) * P.B * P.C) * N + state, p.valid, h);
        else if (P.s_in != nullptr) load_states(P.s_in + state, p.valid, h);
    }

    // Inputs come in two tiles ahead, in the raw, and are worked out one tile ahead; a tile's outputs leave while the
    // next one is walked.  ex, ez: what the outputs need of x and z, of the tiles i + 1, i and i - 1.
    const bool has_z = z != nullptr, spare = !__all(p.valid);
    const T* const first_in = kAdj ? go : x;
    const T* const gate_in = has_z ? z : dt;
    uint32_t chb = p.ch * static_cast<uint32_t>(sizeof(T));
    const int64_t CB = P.C * static_cast<int64_t>(sizeof(T)), GNB = GN * static_cast<int64_t>(sizeof(T));  // bytes a token
    T rx[kEach], rd[kEach], rz[kEach];
    float ex[3][kEach], ez[3][kEach];
    Row<T, NS> b, c;
    const auto tile_at = [&](int i) { return p.t0 + (kAdj ? ntiles - 1 - i : i) * kTile; };
    const auto fetch = [&](int i) {
        keep32(chb);
        const int t = tile_at(i < ntiles ? i : ntiles - 1) + wave;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int at = t + W * k < p.te ? t + W * k : p.te - 1;  // (behind the last token: that one again)
            const int64_t row = (row0 + at) * CB;
            rd[k] = load_at(dt, row, chb);
            rx[k] = load_at(first_in, row, chb);
            if constexpr (kOut || kAdj) rz[k] = load_at(gate_in, row, chb);
        }
    };
    typename Row<T, NS>::Where where = Row<T, NS>::where(GN, lane);
    const auto fetch_bc = [&](int i) {
        const int t = tile_at(i < ntiles ? i : ntiles - 1);
        b.fetch(bt, t * GNB, where, p.te - t);
        if constexpr (kOut) c.fetch(ct, t * GNB, where, p.te - t);
    };
    float total = 0.f;  // of delta
    const auto stage = [&](int i) {
        float delta[kEach], v[kEach], unused[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) delta[k] = widen(rd[k]) + bias, v[k] = widen(rx[k]);
        steps_of<kWide, false>(delta, P.softplus, unused);
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            if constexpr (kOut || kAdj) {
                const float zz = widen(rz[k]), gate = has_z ? zz * gate_of(zz) : 1.f;
                if constexpr (kAdj) v[k] *= gate;
                else ex[0][k] = skip * v[k], ez[0][k] = gate;
            }
            if constexpr (!kAdj) v[k] *= delta[k];
        }
        const int left = i < ntiles ? p.te - tile_at(i) - wave : 0;
        if (spare || left < kTile) {
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const bool live = W * k < left && p.valid;
                delta[k] = live ? delta[k] : 0.f;
                v[k] = live ? v[k] : 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            put[i & 1][wave + W * k][lane] = make_float2(delta[k], v[k]);
            if constexpr (!kOut) total += delta[k];
        }
    };
    const auto pass = [&] {  // on to the next tile
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
#pragma unroll
            for (int q = 2; q > 0; --q) ex[q][k] = ex[q - 1][k], ez[q][k] = ez[q - 1][k];
        }
    };
    // the outputs of tile i, from the waves' parts
    T o[kEach];
    const auto add_up = [&](int i) {
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            float y = ex[2][k];
#pragma unroll
            for (int q = 0; q < W; ++q) y += parts[i & 1][q][wave + W * k][lane];
            o[k] = narrow<T>(y * ez[2][k]);
        }
    };
    const auto write = [&](int i) {
        const int t = tile_at(i) + wave, left = p.te - t;
        const int64_t row = (row0 + t) * CB;
        keep32(chb);
        if (out == nullptr || i < 0) return;
        if (spare || left < kTile) {
#pragma unroll
            for (int k = 0; k < kEach; ++k)
                if (W * k < left && p.valid) store_at(out, row + W * k * CB, chb, o[k]);
        } else {
#pragma unroll
            for (int k = 0; k < kEach; ++k) store_at(out, row + W * k * CB, chb, o[k]);
        }
    };

    if (ntiles > 0) {
        fetch(0);
        fetch_bc(0);
        if constexpr (kOut) {
#pragma unroll
            for (int k = 0; k < kEach; ++k) ex[1][k] = ez[1][k] = 0.f;
        }
        stage(0);
        b.ready();
        if constexpr (kOut) {
            c.ready();
            pass();
        }
        fetch(1);
        __syncthreads();
    }
    for (int i = 0; i < ntiles; ++i) {
        yield_to_later(i, ntiles);
        if constexpr (kOut) {
            if (P.ckpt != nullptr && p.valid)
                store_states(P.ckpt + saved_at<NS>(P, p, tile_at(i), wave, N), h);
            if (i > 0) add_up(i - 1);
        }
        fetch_bc(i + 1);
        const float2(&now)[kTile][64] = put[i & 1];
        each<kTile>([&](auto jj) {
            constexpr int j = kAdj ? kTile - 1 - decltype(jj)::value : decltype(jj)::value;
            const float2 dv = now[j][lane];
            each<NS>([&](auto ss) {
                constexpr int s = decltype(ss)::value;
                const float a = decay(dv.x, w2[s]);
                if constexpr (kAdj) h[s] = a * fmaf(b.template get<j, s>(), dv.y, h[s]);
                else h[s] = fmaf(a, h[s], b.template get<j, s>() * dv.y);
            });
            if constexpr (kOut) {
                parts[i & 1][wave][j][lane] = dot_row<c.template lane_of<j>()>(c.template reg<j>(), h);
            }
        });
        stage(i + 1);
        b.ready();
        if constexpr (kOut) {
            c.ready();
            // (worked out here, before the stores: a load waited for behind them would wait for them too)
#pragma unroll
            for (int k = 0; k < kEach; ++k) asm volatile("" : "+v"(ex[0][k]), "+v"(ez[0][k]));
            write(i - 1);
            pass();
        }
        __syncthreads();
        fetch(i + 2);
    }
    if constexpr (kOut) {
        if (ntiles > 0) {
            add_up(ntiles - 1);
            write(ntiles - 1);
        }
    }
    if constexpr (kOut) {
        if (p.valid) {
            for (int t = p.te + wave; t < p.t1 && out != nullptr; t += W) out[(row0 + t) * P.C + p.ch] = T{0};
            if (P.s_out != nullptr && p.seg == P.nseg - 1) store_states(P.s_out + state, h);
        }
    } else {
        const int64_t at = static_cast<int64_t>(p.seg) * P.B * P.C;
        if (p.valid) store_states(P.local + at * N + state, h);
        __syncthreads();
        put[0][wave][lane].x = total;
        __syncthreads();
        if (wave == 0 && p.valid) {
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < W; ++q) sum += put[0][q][lane].x;
            P.steps[at + p.b * P.C + p.ch] = sum;
        }
    }
}

// The states before the segments (or their gradients behind them, from the last one), in place of what the segments do
// to a state of zero: a state passes a segment by e^{-w (sum of its steps)}.
__global__ __launch_bounds__(256) void select_chain_kernel(SelectArgs P, bool reverse) {
    const int64_t n = P.B * P.C * P.N;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t bc = i / P.N;
    const float w2 = -P.w[bc % P.C * P.N + i % P.N] * kLog2e;
    const float* first = reverse ? P.ds_out : P.s_in;
    float h = first != nullptr ? first[i] : 0.f;
    for (int64_t k = 0; k < P.nseg; ++k) {
        const int64_t s = reverse ? P.nseg - 1 - k : k;
        float* at = P.local + s * n + i;
        const float own = k + 1 < P.nseg ? *at : 0.f, step = k + 1 < P.nseg ? P.steps[s * P.B * P.C + bc] : 0.f;
        *at = h;
        h = fmaf(decay(step, w2), h, own);
    }
}

// Gradients, tile by tile from the last: the tile's states are walked again from the one that the forward kept, then its
// tokens are taken back to front,
//     g += c_t gy_t,   dc_t = sum gy_t h_t,   db_t = sum g u_t  (over channels),   du_t = sum_n g b_t,
//     g *= a_t,   q = g h_{t-1},   ddelta_t = du_t x_t - sum_n w q,   dw -= delta_t q
// An infinite rate is left out of the sum over w q (q is zero but in a step of zero, which is the end of the steps' range),
// and where the softplus has no slope so is all of it: a large rate times q may be infinite there.  The tile's 16 states and decays stay in registers.  db and dc of a token are sums over the lanes: 8 numbers a token,
// of which every exchange between lanes halves the registers, so 16 tokens end as two registers of one number a lane.
template <typename T, int NS, int W>
__global__ __launch_bounds__(64 * W, 2) void select_grad_kernel(SelectArgs P) {
    constexpr int N = NS * W, kEach = kTile / W;
    constexpr bool kWide = sizeof(T) == 4;
    __shared__ float4 put[kTile][64];           // delta, the written value, the gradient of y, x
    __shared__ float parts[3][W][kTile][64];    // the waves' parts of y, du and -ddelta
    // The sums over tokens (dw, then dd and the bias's): of kRun tiles in float32 registers, of these runs in float64 here, where
    // there is room for them.  (One float32 sum over a row would lose up to 2^-25 of itself with every token.  With each tile a
    // run the forward and gradients of 8 x 1024 x 4096 take 576 us, with these 557.)
    constexpr int kRun = 8;
    __shared__ double sums[NS + 2][64 * W];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Place p = place_of(P, lane);
    const T* __restrict__ x = static_cast<const T*>(P.x);
    const T* __restrict__ dt = static_cast<const T*>(P.dt);
    const T* __restrict__ z = static_cast<const T*>(P.z);
    const T* __restrict__ go = static_cast<const T*>(P.go);
    T* __restrict__ dx = static_cast<T*>(P.dx);
    T* __restrict__ ddt = static_cast<T*>(P.ddt);
    T* __restrict__ dz = static_cast<T*>(P.dz);
    const int64_t row0 = p.b * P.T, GN = P.G * N;
    const T* bt = static_cast<const T*>(P.b) + (row0 * GN + p.g * N + wave * NS);
    const T* ct = static_cast<const T*>(P.c) + (row0 * GN + p.g * N + wave * NS);
    const float bias = P.dt_bias != nullptr ? P.dt_bias[p.ch] : 0.f;
    const float skip = P.d != nullptr ? P.d[p.ch] : 0.f;
    const int ntiles = (p.te - p.t0 + kTile - 1) / kTile;

    float w1[NS], w2[NS], g[NS], dw[NS], first[NS];
    load_states(P.w + static_cast<int64_t>(p.ch) * N + wave * NS, true, w1);
    const int64_t state = (p.b * P.C + p.ch) * N + wave * NS;
    const float* from = P.nseg > 1 ? P.local + (static_cast<int64_t>(p.seg) * P.B * P.C) * N : P.ds_out;
#pragma unroll
    for (int i = 0; i < NS; ++i) w2[i] = -w1[i] * kLog2e, w1[i] = w2[i] == -__builtin_inff() ? 0.f : w1[i], dw[i] = g[i] = 0.f;
#pragma unroll
    for (int i = 0; i < NS + 2; ++i) sums[i][threadIdx.x] = 0.0;
    if (from != nullptr) load_states(from + state, p.valid, g);

    const bool has_z = z != nullptr, spare = !__all(p.valid);
    const T* const gate_in = has_z ? z : dt;
    uint32_t chb = p.ch * static_cast<uint32_t>(sizeof(T));
    const int64_t CB = P.C * static_cast<int64_t>(sizeof(T)), GNB = GN * static_cast<int64_t>(sizeof(T));  // bytes a token
    T rx[kEach], rd[kEach], rz[kEach], rg[kEach];
    Row<T, NS> b, c;
    typename Row<T, NS>::Where where = Row<T, NS>::where(GN, lane);
    const auto tile_at = [&](int i) { return p.t0 + i * kTile; };
    const auto fetch = [&](int i) {  // (behind the last token: that one again; before the first tile: nothing new)
        keep32(chb);
        const int tile = tile_at(i > 0 ? i : 0), t = tile + wave, left = p.te - tile;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int at = t + W * k < p.te ? t + W * k : p.te - 1;
            const int64_t row = (row0 + at) * CB;
            rd[k] = load_at(dt, row, chb);
            rx[k] = load_at(x, row, chb);
            rg[k] = load_at(go, row, chb);
            rz[k] = load_at(gate_in, row, chb);
        }
        load_states(P.saved + saved_at<NS>(P, p, tile, wave, N), p.valid, first);
        b.fetch(bt, tile * GNB, where, left);
        c.fetch(ct, tile * GNB, where, left);
    };
    float dd = 0.f, dbias = 0.f;
    const auto end_run = [&] {
#pragma unroll
        for (int s = 0; s < NS; ++s) sums[s][threadIdx.x] += dw[s], dw[s] = 0.f;
        sums[NS][threadIdx.x] += dd, sums[NS + 1][threadIdx.x] += dbias;
        dd = dbias = 0.f;
    };
    if (ntiles > 0) fetch(ntiles - 1);
    for (int i = ntiles - 1; i >= 0; --i) {
        yield_to_later(ntiles - 1 - i, ntiles);
        const int t = tile_at(i), n = p.te - t;
        float egs[kEach], eslope[kEach], delta[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) delta[k] = widen(rd[k]) + bias;
        steps_of<kWide, true>(delta, P.softplus, eslope);
        const bool edge = spare || n < kTile;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const float zz = widen(rz[k]), gg = widen(rg[k]), sg = gate_of(zz), xx = widen(rx[k]);
            const float gate = has_z ? zz * sg : 1.f;
            egs[k] = gg * fmaf(gate, 1.f - sg, sg);  // times the gate's derivative, sg (1 + z (1 - sg))
            put[wave + W * k][lane] = make_float4(delta[k], delta[k] * xx, gg * gate, xx);
        }
        if (edge) {
#pragma unroll
            for (int k = 0; k < kEach; ++k)
                if (!(wave + W * k < n && p.valid)) put[wave + W * k][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float h[kTile + 1][NS], a[kTile][NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) h[0][s] = first[s];
        b.ready();
        c.ready();
        __syncthreads();
        fetch(i - 1);
        each<kTile>([&](auto jj) {
            constexpr int j = decltype(jj)::value;
            const float4 v = put[j][lane];
            each<NS>([&](auto ss) {
                constexpr int s = decltype(ss)::value;
                a[j][s] = decay(v.x, w2[s]);
                h[j + 1][s] = fmaf(a[j][s], h[j][s], b.template get<j, s>() * v.y);
            });
            parts[0][wave][j][lane] = dot_row<c.template lane_of<j>()>(c.template reg<j>(), h[j + 1]);
        });
        b.forget();
        c.forget();
        float tokens[8];
        each<kTile>([&](auto jj) {
            constexpr int j = kTile - 1 - decltype(jj)::value;
            const float4 v = put[j][lane];
            float down = 0.f, pb[NS], pc[NS];
            add_row<c.template lane_of<j>()>(g, c.template reg<j>(), v.z);
            parts[1][wave][j][lane] = dot_row<b.template lane_of<j>()>(b.template reg<j>(), g);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                pb[s] = g[s] * v.y, pc[s] = v.z * h[j + 1][s];
                g[s] *= a[j][s];
                const float m = g[s] * h[j][s];
                down = fmaf(m, w1[s], down);
                dw[s] = fmaf(-m, v.x, dw[s]);
            }
            parts[2][wave][j][lane] = down;
            // of four states 0 and 1 to the even rows of 16 lanes, 2 and 3 to the odd ones; then token j to one half of the
            // lanes that are left to tell apart (two states: to the even rows), j + 8 to the other
            float one;
            if constexpr (NS == 4) {
                float q0, q1;
                fold_rows(pb, pc, q0, q1);
                const auto x1 = __builtin_amdgcn_permlane16_swap(__float_as_uint(q0), __float_as_uint(q1), false, false);
                one = __uint_as_float(x1[0]) + __uint_as_float(x1[1]);
            } else {
                fold_rows(pb, pc, one);
            }
            if constexpr (j >= 8) {
                tokens[j - 8] = one;
            } else {
                const uint32_t lo = __float_as_uint(one), hi = __float_as_uint(tokens[j]);
                if constexpr (NS == 4) {
                    const auto x2 = __builtin_amdgcn_permlane32_swap(lo, hi, false, false);
                    tokens[j] = __uint_as_float(x2[0]) + __uint_as_float(x2[1]);
                } else {
                    const auto x2 = __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
                    tokens[j] = __uint_as_float(x2[0]) + __uint_as_float(x2[1]);
                }
            }
        });
        constexpr int kFour = NS == 4 ? 8 : 4;  // registers before the lanes of a four are told apart
        if constexpr (NS == 2) {  // token k to the lower half of the lanes, k + 4 to the upper
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const auto x2 = __builtin_amdgcn_permlane32_swap(__float_as_uint(tokens[k]), __float_as_uint(tokens[k + 4]), false, false);
                tokens[k] = __uint_as_float(x2[0]) + __uint_as_float(x2[1]);
            }
        }
#pragma unroll
        for (int k = 0; k < kFour / 2; ++k) {
            const float lo = tokens[k] + dpp<0x4E>(tokens[k]), hi = tokens[k + kFour / 2] + dpp<0x4E>(tokens[k + kFour / 2]);  // lane ^ 2
            tokens[k] = (lane & 2) != 0 ? hi : lo;
        }
#pragma unroll
        for (int k = 0; k < kFour / 4; ++k) {
            const float lo = tokens[k] + dpp<0xB1>(tokens[k]), hi = tokens[k + kFour / 4] + dpp<0xB1>(tokens[k + kFour / 4]);  // lane ^ 1
            const int bit0 = lane & 1, bit1 = (lane >> 1) & 1, bit4 = (lane >> 4) & 1, bit5 = lane >> 5;
            const int tok = NS == 4 ? k + bit1 * 4 + bit0 * 2 + bit5 * 8 : bit1 * 2 + bit0 + bit5 * 4 + bit4 * 8;
            const int state = wave * NS + (NS == 4 ? bit4 * 2 : 0) + ((lane >> 2) & 1);
            if (tok < n) {
                const int64_t row = (static_cast<int64_t>(p.ct) * P.B * P.T + row0 + t + tok) * (2 * N);
                P.part[row + ((lane >> 3) & 1) * N + state] = bit0 != 0 ? hi : lo;
            }
        }
        __syncthreads();
        T oz[kEach], ox[kEach], od[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int j = wave + W * k;
            const float4 v = put[j][lane];
            float y = skip * v.w, du = 0.f, down = 0.f;
#pragma unroll
            for (int q = 0; q < W; ++q) y += parts[0][q][j][lane], du += parts[1][q][j][lane], down += parts[2][q][j][lane];
            float gd = fmaf(du, v.w, eslope[k] != 0.f ? -down : 0.f) * eslope[k];
            if (edge) gd = j < n && p.valid ? gd : 0.f;
            oz[k] = narrow<T>(egs[k] * y);
            ox[k] = narrow<T>(fmaf(du, v.x, skip * v.z));
            od[k] = narrow<T>(gd);
            dd = fmaf(v.z, v.w, dd);
            dbias += gd;
        }
        if (i % kRun == 0) end_run();
        const int64_t row = (row0 + t + wave) * CB;
        keep32(chb);
        if (!edge) {
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                store_at(dx, row + W * k * CB, chb, ox[k]);
                store_at(ddt, row + W * k * CB, chb, od[k]);
                if (has_z) store_at(dz, row + W * k * CB, chb, oz[k]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                if (!(wave + W * k < n && p.valid)) continue;
                store_at(dx, row + W * k * CB, chb, ox[k]);
                store_at(ddt, row + W * k * CB, chb, od[k]);
                if (has_z) store_at(dz, row + W * k * CB, chb, oz[k]);
            }
        }
    }
    if (p.valid) {
        for (int t = p.te + wave; t < p.t1; t += W) {
            const int64_t at = (row0 + t) * P.C + p.ch;
            dx[at] = ddt[at] = T{0};
            if (z != nullptr) dz[at] = T{0};
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) dw[s] = static_cast<float>(sums[s][threadIdx.x]);
        store_states(P.dw_part + (static_cast<int64_t>(p.seg) * P.B * P.C) * N + state, dw);
        if (P.ds_in != nullptr && p.seg == 0) store_states(P.ds_in + state, g);
    }
    __syncthreads();
    if (wave == 0 && p.valid) {
        double sum_dd = 0.0, sum_dbias = 0.0;
#pragma unroll
        for (int q = 0; q < W; ++q) sum_dd += sums[NS][q * 64 + lane], sum_dbias += sums[NS + 1][q * 64 + lane];
        const int64_t at = (static_cast<int64_t>(p.seg) * P.B + p.b) * P.C + p.ch;
        P.vec_part[2 * at] = static_cast<float>(sum_dd);
        P.vec_part[2 * at + 1] = static_cast<float>(sum_dbias);
    }
}

// db and dc from the channel tiles' sums; dw, dd and the bias's gradient from the rows' (and segments'), added up in
// float64: there may be tens of thousands.  All in a fixed order.  The first bc_blocks workgroups take b and c.
template <typename T>
__global__ __launch_bounds__(256) void select_reduce_kernel(SelectArgs P, int64_t bc_blocks) {
    if (blockIdx.x < bc_blocks) {
        // four numbers a lane, a quarter of the channel tiles a wave
        __shared__ f4 quarters[4][64];
        const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
        const int64_t i = (static_cast<int64_t>(blockIdx.x) * 64 + lane) * 4;  // (row, group, b or c, n)
        const int64_t n2 = 2 * P.N, rows = P.B * P.T;
        const bool here = i < rows * P.G * n2;
        const int64_t e = i % n2, g = i / n2 % P.G, row = i / (n2 * P.G);
        const int per_group = P.ctiles / static_cast<int>(P.G), each = (per_group + 3) / 4;
        const int first = q * each, last = first + each < per_group ? first + each : per_group;
        const bool live = here && (P.lengths == nullptr || row % P.T < P.lengths[row / P.T]);
        f4 sum = {0.f, 0.f, 0.f, 0.f};
        if (live) {
            const float* at = P.part + (g * per_group * rows + row) * n2 + e;
#pragma unroll 8
            for (int k = first; k < last; ++k) sum += *reinterpret_cast<const f4*>(at + k * rows * n2);
        }
        quarters[q][lane] = sum;
        __syncthreads();
        if (q != 0 || !here) return;
        sum = (quarters[0][lane] + quarters[1][lane]) + (quarters[2][lane] + quarters[3][lane]);
        T* to = static_cast<T*>(e < P.N ? P.db : P.dc) + (row * P.G + g) * P.N + e % P.N;
        if constexpr (sizeof(T) == 4) *reinterpret_cast<f4*>(to) = sum;
        else *reinterpret_cast<uint2*>(to) = make_uint2(pk2(sum[0], sum[1]), pk2(sum[2], sum[3]));
        return;
    }
    // an output a lane, a quarter of the rows a wave
    __shared__ double sums[4][64];
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int64_t i = (static_cast<int64_t>(blockIdx.x) - bc_blocks) * 64 + lane;
    const int64_t nw = P.C * P.N, n = nw + 2 * P.C, rows = P.B * P.nseg, each = (rows + 3) / 4;
    const int64_t first = q * each, last = first + each < rows ? first + each : rows;
    const float* from = i < nw ? P.dw_part + i : P.vec_part + (i - nw);  // (vec_part: dd and the bias's in turn)
    const int64_t stride = i < nw ? nw : 2 * P.C;
    double sum = 0.0;
    if (i < n) {
#pragma unroll 8
        for (int64_t r = first; r < last; ++r) sum += from[r * stride];
    }
    sums[q][lane] = sum;
    __syncthreads();
    if (q != 0 || i >= n) return;
    const float all = static_cast<float>((sums[0][lane] + sums[1][lane]) + (sums[2][lane] + sums[3][lane]));
    if (i < nw) {
        P.dw[i] = all;
    } else {
        float* to = ((i - nw) & 1) == 0 ? P.dd : P.ddt_bias;
        if (to != nullptr) to[(i - nw) >> 1] = all;
    }
}

// A few tokens: four states a lane, token by token in registers, the state one trip through memory, which is what bounds
// it (256 rows of 4096 channels, N = 16, bf16, 8 layers in turn: 143 MB in 31 us, 4.7 TB/s; one layer over and over, part
// of it in the last level cache, without Past 26 us).  A workgroup takes 256 / Lanes channels of a batch row (and of every
// gridDim.y-th row after it).
template <typename T, int Lanes, bool Past>
__global__ __launch_bounds__(256) void select_step_kernel(SelectArgs P) {
    constexpr bool kWide = sizeof(T) == 4;
    constexpr int NS = 4, N = NS * Lanes;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * (256 / Lanes) + threadIdx.x / Lanes;
    const bool valid = at < P.C;
    const int ch = static_cast<int>(valid ? at : P.C - 1), q = threadIdx.x % Lanes;  // spare lanes take part in the sums
    const int g = P.G > 1 ? ch / (static_cast<int>(P.C) / static_cast<int>(P.G)) : 0;
    const int64_t GN = P.G * N;
    float w2[NS];
    load_states(P.w + static_cast<int64_t>(ch) * N + 4 * q, true, w2);
#pragma unroll
    for (int s = 0; s < NS; ++s) w2[s] = -w2[s] * kLog2e;
    const float bias = P.dt_bias != nullptr ? P.dt_bias[ch] : 0.f, skip = P.d != nullptr ? P.d[ch] : 0.f;
    const int tokens = static_cast<int>(P.T);
    for (int64_t b = blockIdx.y; b < P.B; b += gridDim.y) {
        const int64_t state = (b * P.C + ch) * N + 4 * q;
        float h[NS] = {0.f, 0.f, 0.f, 0.f};
        if (P.s_in != nullptr) load_states<Past>(P.s_in + state, true, h);
        int len = P.lengths != nullptr ? P.lengths[b] : tokens;
        len = len < 0 ? 0 : len > tokens ? tokens : len;
        for (int t = 0; t < tokens; ++t) {
            const int64_t row = b * P.T + t, to = row * P.C + ch;
            if (t >= len) {
                if (valid && q == 0) static_cast<T*>(P.out)[to] = T{0};
                continue;
            }
            const int64_t from = row * GN + g * N + 4 * q;
            T bb[NS], cc[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s) bb[s] = static_cast<const T*>(P.b)[from + s], cc[s] = static_cast<const T*>(P.c)[from + s];
            const float vx = widen(static_cast<const T*>(P.x)[to]);
            float gate = 1.f, y = 0.f, d1[1] = {widen(static_cast<const T*>(P.dt)[to]) + bias}, unused[1];
            if (P.z != nullptr) {
                const float zz = widen(static_cast<const T*>(P.z)[to]);
                gate = zz * gate_of(zz);
            }
            steps_of<kWide, false>(d1, P.softplus, unused);
            const float u = d1[0] * vx;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                h[s] = fmaf(decay(d1[0], w2[s]), h[s], widen(bb[s]) * u);
                y = fmaf(widen(cc[s]), h[s], y);
            }
            y = sum_lanes(y, Lanes);
            if (valid && q == 0) static_cast<T*>(P.out)[to] = narrow<T>(fmaf(skip, vx, y) * gate);
        }
        if (valid && P.s_out != nullptr) store_states<Past>(P.s_out + state, h);
    }
}

template <typename T, int NS, int W>
hipError_t walk_t(const SelectArgs& a, int mode, hipStream_t stream) {
    const bool all = mode == kWalkOut || mode == kGrad;
    const dim3 grid(static_cast<unsigned>(a.ctiles * a.B * (all ? a.nseg : a.nseg - 1))), block(64 * W);
    switch (mode) {
        case kWalkOut: hipLaunchKernelGGL((select_walk_kernel<T, NS, W, kWalkOut>), grid, block, 0, stream, a); break;
        case kWalkLocal: hipLaunchKernelGGL((select_walk_kernel<T, NS, W, kWalkLocal>), grid, block, 0, stream, a); break;
        case kWalkAdjoint: hipLaunchKernelGGL((select_walk_kernel<T, NS, W, kWalkAdjoint>), grid, block, 0, stream, a); break;
        default: hipLaunchKernelGGL((select_grad_kernel<T, NS, W>), grid, block, 0, stream, a); break;
    }
    return hipGetLastError();
}

template <typename T>
hipError_t walk_n(const SelectArgs& a, int mode, hipStream_t stream) {
    switch (a.N) {
        // Two states a wave of N = 8, since with two waves of four the card is half empty (B = 8, T = 1024, C = 4096, bf16:
        // forward and gradients together 833 us, of two states 422).  And of N = 16 where no compute unit has two
        // workgroups, so that its eight waves keep each vector unit with two (4 rows of these: 125 + 303 us of four
        // states, 110 + 256 of two; 6 rows 160 + 382 and 157 + 396, 8 rows 167 + 397 and 178 + 397).
        case 8: return walk_t<T, 2, 4>(a, mode, stream);
        case 16: return a.B * a.ctiles * a.nseg <= 256 ? walk_t<T, 2, 8>(a, mode, stream) : walk_t<T, 4, 4>(a, mode, stream);
        default: return walk_t<T, 4, 8>(a, mode, stream);
    }
}

hipError_t walk(const SelectArgs& a, int mode, hipStream_t stream) {
    return a.bf16 ? walk_n<uint16_t>(a, mode, stream) : walk_n<float>(a, mode, stream);
}

hipError_t chain(const SelectArgs& a, bool reverse, hipStream_t stream) {
    const int64_t n = a.B * a.C * a.N;
    hipLaunchKernelGGL(select_chain_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, stream, a, reverse);
    return hipGetLastError();
}

}  // namespace

// A time split walks everything twice (once for what the segments do to a state of zero, then from their start states), and
// pays where the channel tiles alone leave most of the card idle or there are tokens without end.  The model, in us: a
// tile of 16 tokens takes a workgroup on a compute unit of its own about `alone`, and the unit's workgroups together at
// least `shared` each; the backward 2.6 times that; the second walk 0.8 of the first; its launches 8.  Forward and backward
// split, and whole, in us:
//     2 rows of 333 tokens, 1002 channels, N = 8, float32   22 + 33 and 37 + 81          (7 segments)
//     the same, N = 16                                      24 + 36 and 41 + 88          (7)
//     1 row of 300 tokens, 768 channels, N = 16, bf16       19 + 27 and 35 + 78          (10)
//     1 row of 2000 tokens, 4096 channels, N = 16, bf16     83 + 147 and 208 + 483       (8; N = 8: 68 + 112 and 186 + 430)
//     2 rows of 1024 tokens, 4096 channels, N = 16, bf16    86 + 149 and 108 + 252       (4)
//     3 rows of 929 tokens, 4008 channels, N = 16, bf16     not forward; 210 and 241     (4)
//     1 row of 32768 tokens, 4096 channels, N = 16, bf16    1040 + 2030 and 3340 + 7780  (16)
int64_t select_segments(int64_t B, int64_t T, int64_t ctiles, int64_t N, bool bwd, int64_t* per) {
    const int64_t tiles = (T + kTile - 1) / kTile, groups = B * ctiles;
    *per = tiles * kTile;
    if (groups <= 0 || groups >= 512 || tiles < 4) return 1;
    const double alone = N == 8 ? 1.2 : 1.7, shared = N == 8 ? 0.9 : 0.35 * static_cast<double>(N / 4), scale = bwd ? 2.6 : 1.0;
    const auto tile_us = [&](int64_t workgroups) {
        const double busy = shared * static_cast<double>((workgroups + 255) / 256);
        return scale * (busy > alone ? busy : alone);
    };
    double best = static_cast<double>(tiles) * tile_us(groups);
    int64_t n = 1;
    for (int64_t each = 2; each < tiles; each = each < 16 ? each + 1 : each + each / 8) {
        const int64_t k = (tiles + each - 1) / each;
        if (groups * k > (int64_t{1} << 20)) continue;
        const double second = bwd ? 1.0 + 0.8 / 2.6 : 1.8;
        const double us = second * static_cast<double>(each) * tile_us(groups * k) + 8.0 + 0.1 * static_cast<double>(k);
        if (us < best) best = us, n = k, *per = each * kTile;
    }
    return n;
}

namespace {

template <typename T, bool Past>
hipError_t step_past(const SelectArgs& a, hipStream_t stream) {
    const int64_t per = 1024 / a.N;  // channels a workgroup
    const dim3 grid(static_cast<unsigned>((a.C + per - 1) / per), static_cast<unsigned>(a.B < 65535 ? a.B : 65535));
    if (a.N == 8) hipLaunchKernelGGL((select_step_kernel<T, 2, Past>), grid, dim3(256), 0, stream, a);
    else if (a.N == 16) hipLaunchKernelGGL((select_step_kernel<T, 4, Past>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((select_step_kernel<T, 8, Past>), grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

// States of 16 MB and more pass the caches, which those of sixteen layers do not fit (bf16, N = 16, as many layers in turn as
// take 0.5 GB: 256 rows of 4096 channels 34.7 -> 30.7 us, 128 rows 19.4 -> 16.9, 64 rows 11.2 -> 9.5; four layers of 128
// rows, which fit them, 15.2 -> 16.3; below, calls of 5 to 7 us, no difference).
template <typename T>
hipError_t step_t(const SelectArgs& a, hipStream_t stream) {
    return a.B * a.C * a.N >= (int64_t{1} << 22) ? step_past<T, true>(a, stream) : step_past<T, false>(a, stream);
}

}  // namespace

hipError_t launch_select_step(const SelectArgs& a, hipStream_t stream) {
    return a.bf16 ? step_t<uint16_t>(a, stream) : step_t<float>(a, stream);
}

hipError_t launch_select_fwd(const SelectArgs& a, hipStream_t stream) {
    if (a.nseg > 1) {
        hipError_t e = walk(a, kWalkLocal, stream);
        if (e == hipSuccess) e = chain(a, false, stream);
        if (e != hipSuccess) return e;
    }
    return walk(a, kWalkOut, stream);
}

hipError_t launch_select_bwd(const SelectArgs& a, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.nseg > 1) {
        e = walk(a, kWalkAdjoint, stream);
        if (e == hipSuccess) e = chain(a, true, stream);
        if (e != hipSuccess) return e;
    }
    e = walk(a, kGrad, stream);
    if (e != hipSuccess) return e;
    const int64_t bc = (a.B * a.T * a.G * 2 * a.N / 4 + 63) / 64, rest = (a.C * a.N + 2 * a.C + 63) / 64;
    const dim3 grid(static_cast<unsigned>(bc + rest));
    if (a.bf16) hipLaunchKernelGGL(select_reduce_kernel<uint16_t>, grid, dim3(256), 0, stream, a, bc);
    else hipLaunchKernelGGL(select_reduce_kernel<float>, grid, dim3(256), 0, stream, a, bc);
    return hipGetLastError();
}

}  // namespace wkv
