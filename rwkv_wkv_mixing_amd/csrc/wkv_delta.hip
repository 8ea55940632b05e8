// The gated delta rule: a matrix state per head that is decayed, corrected and read.
//
// Per (batch row, value head), with a state S [N, N] (key x value), N = 64 or 128:
//     D_t = e^{-w_t} S_{t-1}                    (decay, one rate per token and head)
//     e_t = v_t - k_t D_t                       (what the state gets wrong about this key)
//     S_t = D_t + beta_t k_t^T e_t,   o_t = r_t S_t
// H value heads share HK key heads (H a multiple of HK): head h reads r, k of key head h / (H / HK).
//
// Over a block of tokens i = 0.. from the state S0, with the decay products
//     since_i = prod_{l <= i} e^{-w_l},  ratio_ij = prod_{j < l <= i} e^{-w_l},  until_j = prod_{l > j} e^{-w_l}
// the recurrence unrolls to a triangular system for the errors and two products:
//     (I + M diag(beta)) e = V - diag(since) K S0,     M_ij = ratio_ij k_i . k_j   (j < i)
//     o   = diag(since) R S0 + A e,                    A_ij = ratio_ij r_i . k_j beta_j   (j <= i)
//     S1  = since_last S0 + K^T diag(until beta) e
// The block here is 16 tokens: the system's inverse X = (I + M diag(beta))^{-1} is a 16 x 16 unit
// lower triangle found by forward substitution (no cancellation, whatever the keys), and the state
// stays in the accumulators of its products.  Every ratio is exp of a sum of the rates between its
// two tokens, never a quotient or a difference of running sums, so a rate of any size (+inf included:
// the state is cleared) gives factors in [0, 1].
//
// Lane layout.  A wave owns 16 value columns of the state: N / 16 accumulators of the 16 x 16 products,
// where lane (l16, g) holds four rows of column l16 of each (which four: state_row).  As the right
// operand of the next product the same registers are already in place when the contracted index runs in
// that order; the left operand is then read from its rows in the same order.  So neither the state nor
// e, nor anything between the products, ever crosses lanes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "wkv_lanes.h"
#include "wkv_launch.h"

namespace wkv {
namespace {

typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

constexpr int kTile = 64;   // tokens staged at a time, and between saved states
constexpr int kSub = 16;    // tokens of one triangular system
constexpr int kWaves = 4;   // 16-token blocks of a tile; waves of the step and the float32 gradient kernel
constexpr int kPadM = kSub + 4;  // floats a row of the float32 gradient kernel's 16 x 16 tables
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }

// four consecutive elements as float32
__device__ __forceinline__ f4 load4(const uint16_t* p) {
    const u16x4 x = *reinterpret_cast<const u16x4*>(p);
    return f4{widen(x[0]), widen(x[1]), widen(x[2]), widen(x[3])};
}
__device__ __forceinline__ f4 load4(const float* p) { return *reinterpret_cast<const f4*>(p); }

__device__ __forceinline__ uint16_t narrow(float x) { return static_cast<uint16_t>(pk2(x, x) & 0xffffu); }

__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = narrow(x); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store4(uint16_t* p, f4 x) {
    *reinterpret_cast<u32x2*>(p) = u32x2{pk2(x[0], x[1]), pk2(x[2], x[3])};
}
__device__ __forceinline__ void store4(float* p, f4 x) { *reinterpret_cast<f4*>(p) = x; }

// float32 product: lane (l16, g) gives row l16 of A and column l16 of B at contracted index g
__device__ __forceinline__ f4 mfma4(float a, float b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// acc += A B over 16 contracted indices 4 g + r
__device__ __forceinline__ f4 mma16(f4 a, f4 b, f4 c) {
#pragma unroll
    for (int r = 0; r < 4; ++r) c = mfma4(a[r], b[r], c);
    return c;
}

// Elements a row of a staged [kTile, N] array, and where element c of row t lies.  Float32 rows are padded by
// 16 bytes, so that 16 lanes reading 16 consecutive rows start in different banks.  bf16 rows are not (two
// workgroups a compute unit, or all of a tile's terms, would not fit): the 16-byte piece q of row t lies at
// q ^ swizzle(t), the same for a row of every 16, so that 16 rows' pieces q meet 16 different bank groups.
template <typename T, int N>
constexpr int kRow = sizeof(T) == 2 ? N : N + 4;

template <int N>
__device__ __forceinline__ int swizzled(int t, int c) {
    const int s = N == 64 ? (t >> 1) & 7 : t & 15;
    return (((c >> 3) ^ s) << 3) | (c & 7);
}
template <typename T, int N>
__device__ __forceinline__ int place(int t, int c) {
    return t * kRow<T, N> + (sizeof(T) == 2 ? swizzled<N>(t, c) : c);
}

// ---- products with bf16 inputs -------------------------------------------------------------------
// A bf16 input is exact as an operand of the bf16 products, which run 16 times as fast as the float32
// ones.  A float32 factor x is given as three bf16 terms, x = hi + mid + lo, each what the ones before leave,
// rounded: 8 bits and a sign a term, so the split is exact and the products summed in float32 are those of
// float32 operands.  Where a result is rounded to bf16 and goes nowhere else, hi + mid (off by at most 2^-18)
// are used: rounding moves the result by up to 2^-8, so what is left out shows where its terms cancel by 2^9 or
// more.  That is o's reading of the state (times<true>) and of the pair's first block (times_table<2>, which leaves
// out mid mid too: 3 2^-18), and dr's and dk's dA and dM.  With all three terms in o, ragged prompts of 32 / 16
// heads of 128 took 174 us instead of 160, one document of 32768 tokens 1104 instead of 1068, 8 x 1024 tokens of 64
// heads of 64 99.5 instead of 97; dA's and dM's third would not leave LDS for two workgroups at N = 64.
struct Terms {
    u32x2 hi, mid, lo;
};

// What two rounded values leave of x: one dot product with (-1, 0) or (0, -1) each, exact, instead of a
// widening and a subtraction (14 instructions for a split of four instead of 22).  The factors are kept from
// the compiler, which turns (-1, 0) into an inline constant that multiplies the upper value.
__device__ __forceinline__ f2 left_of(uint32_t rounded, f2 x) {
    uint32_t first = 0x0000bf80u, second = 0xbf800000u;
    asm("" : "+s"(first), "+s"(second));
    const bf2 h = __builtin_bit_cast(bf2, rounded);
    return f2{__builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf2, first), x[0], false),
              __builtin_amdgcn_fdot2_f32_bf16(h, __builtin_bit_cast(bf2, second), x[1], false)};
}

__device__ __forceinline__ Terms split(f4 x) {
    Terms t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f2 a = {x[2 * i], x[2 * i + 1]};
        t.hi[i] = pk2(a[0], a[1]);
        const f2 b = left_of(t.hi[i], a);
        t.mid[i] = pk2(b[0], b[1]);
        const f2 c = left_of(t.mid[i], b);
        t.lo[i] = pk2(c[0], c[1]);
    }
    return t;
}

__device__ __forceinline__ bf8 pair(u32x2 a, u32x2 b) { return __builtin_bit_cast(bf8, u32x4{a[0], a[1], b[0], b[1]}); }
__device__ __forceinline__ bf8 raw8(const uint16_t* p) { return __builtin_bit_cast(bf8, *reinterpret_cast<const u32x4*>(p)); }

// 32 contracted indices, eight a lane; which of them a lane holds is the same for A and B.  Sums of 16
// indices take it too, one half filled twice or with zeros: a 16-index product that adds to what a
// 32-index one has just written (or the other way round) has been measured to lose part of it.
__device__ __forceinline__ f4 mfma32(bf8 a, bf8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
// Row of the state that register r of group g holds in accumulator c: a lane's registers of the
// accumulators 2 m and 2 m + 1 are eight consecutive rows, so that one 16-byte read of a token's k gives
// the matching left operand.
__device__ __forceinline__ constexpr int state_row(int c, int g, int r) { return 32 * (c >> 1) + 8 * g + 4 * (c & 1) + r; }

// A block's rows are given by the address of the first of its 16.

// acc[i][j] = sum over the N channels of a row i of A and a row j of B (rows l16 of each), both staged
template <int N>
__device__ __forceinline__ f4 rows_product(const uint16_t* a, const uint16_t* b, int l16, int g) {
    f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < N / 32; ++m) {
        const int at = place<uint16_t, N>(l16, 32 * m + 8 * g);
        acc = mfma32(raw8(a + at), raw8(b + at), acc);
    }
    return acc;
}
template <int N>
__device__ __forceinline__ f4 rows_product(const float* a, const float* b, int l16, int g) {
    f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < N / 16; ++c) {
        const int at = place<float, N>(l16, 16 * c + 4 * g);
        acc = mma16(load4(a + at), load4(b + at), acc);
    }
    return acc;
}

// A block's rows as a left operand (row l16 a lane): bf16 rows are held in registers, so that they are read
// while the state is still being split; float32 rows are read as they are used.
template <typename T, int N>
struct LeftRows;

template <int N>
struct LeftRows<float, N> {
    const float* row;
    __device__ __forceinline__ LeftRows(const float* x, int l16, int) : row(x + place<float, N>(l16, 0)) {}
};
template <int N>
struct LeftRows<uint16_t, N> {
    bf8 a[N / 32];
    __device__ __forceinline__ LeftRows(const uint16_t* x, int l16, int g) {
#pragma unroll
        for (int m = 0; m < N / 32; ++m) a[m] = raw8(x + place<uint16_t, N>(l16, 32 * m + 8 * g));
    }
};

// The state's 16 columns as a right operand.
template <typename T, int N>
struct StateOperand;

template <int N>
struct StateOperand<float, N> {
    f4 s[N / 16];
    __device__ __forceinline__ explicit StateOperand(const f4 (&S)[N / 16]) {
#pragma unroll
        for (int c = 0; c < N / 16; ++c) s[c] = S[c];
    }
    template <bool kRounded>
    __device__ __forceinline__ f4 times(const LeftRows<float, N>& x, int g) const {
        f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < N / 16; ++c) acc = mma16(load4(x.row + state_row(c, g, 0)), s[c], acc);
        return acc;
    }
};

template <int N>
struct StateOperand<uint16_t, N> {
    bf8 hi[N / 32], mid[N / 32], lo[N / 32];
    __device__ __forceinline__ explicit StateOperand(const f4 (&S)[N / 16]) {
#pragma unroll
        for (int m = 0; m < N / 32; ++m) {
            const Terms a = split(S[2 * m]), b = split(S[2 * m + 1]);
            hi[m] = pair(a.hi, b.hi);
            mid[m] = pair(a.mid, b.mid);
            lo[m] = pair(a.lo, b.lo);
        }
    }
    // kRounded: the result is rounded to bf16 and used for nothing else
    template <bool kRounded>
    __device__ __forceinline__ f4 times(const LeftRows<uint16_t, N>& x, int) const {
        f4 acc = {0.f, 0.f, 0.f, 0.f}, acc2 = {0.f, 0.f, 0.f, 0.f};  // two chains of dependent products
#pragma unroll
        for (int m = 0; m < N / 32; ++m) {
            acc2 = mfma32(x.a[m], mid[m], acc2);
            acc = mfma32(x.a[m], hi[m], acc);
            if constexpr (!kRounded) {
                if (m & 1) acc = mfma32(x.a[m], lo[m], acc);
                else acc2 = mfma32(x.a[m], lo[m], acc2);
            }
        }
        return acc + acc2;
    }
};

// The rows of kG blocks as the left operand of S += X^T u: four tokens of one channel a lane, in the state's
// row order.  bf16: one transposing LDS read gives a lane its four tokens of one channel (in each group of 16
// lanes, lane 4 e + p reads four channels of token e, and lane j receives element j % 4 of lane 4 e + j / 4's
// read for e = 0 .. 3).
__device__ __forceinline__ u32x2 read_tr(const uint16_t* at) {
    const s4 raw = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4*)at);
    return __builtin_bit_cast(u32x2, raw);
}

template <typename T, int N>
struct LeftCols;

template <int N>
struct LeftCols<float, N> {
    const float* x;
    int l16, g;
    __device__ __forceinline__ LeftCols(const float* X, int l16_, int g_) : x(X), l16(l16_), g(g_) {}
    __device__ __forceinline__ void add_outer(f4 (&S)[N / 16], const f4 (&u)[1]) const {
#pragma unroll
        for (int c = 0; c < N / 16; ++c) {
            f4 a;
#pragma unroll
            for (int q = 0; q < 4; ++q) a[q] = x[place<float, N>(4 * g + q, state_row(c, l16 >> 2, l16 & 3))];
            S[c] = mma16(a, u[0], S[c]);
        }
    }
};
template <int N>
struct LeftCols<uint16_t, N> {
    u32x2 a[2][N / 16];
    __device__ __forceinline__ LeftCols(const uint16_t* X, int l16, int g) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int c = 0; c < N / 16; ++c)
                a[j][c] = read_tr(X + j * kSub * kRow<uint16_t, N> +
                                  place<uint16_t, N>(4 * g + (l16 >> 2), state_row(c, l16 & 3, 0)));
    }
    // the two blocks' tokens are the 32 contracted indices
    __device__ __forceinline__ void add_outer(f4 (&S)[N / 16], const f4 (&u)[2]) const {
        const Terms t = split(u[0]), t2 = split(u[1]);
        const bf8 b[3] = {pair(t.lo, t2.lo), pair(t.mid, t2.mid), pair(t.hi, t2.hi)};
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
            for (int c = 0; c < N / 16; ++c) S[c] = mfma32(pair(a[0][c], a[1][c]), b[i], S[c]);
    }
};

// Four tokens 4 g .. of a block, column c0 + l16, of a staged array of value columns.
template <int N>
__device__ __forceinline__ f4 value_column(const float* X, int c0, int l16, int g) {
    f4 x;
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = X[place<float, N>(4 * g + q, c0 + l16)];
    return x;
}
template <int N>
__device__ __forceinline__ f4 value_column(const uint16_t* X, int c0, int l16, int g) {
    const u32x2 x = read_tr(X + place<uint16_t, N>(4 * g + (l16 >> 2), c0 + 4 * (l16 & 3)));
    return f4{__uint_as_float(x[0] << 16), __uint_as_float(x[0] & 0xffff0000u), __uint_as_float(x[1] << 16),
              __uint_as_float(x[1] & 0xffff0000u)};
}

// Rows t0 .. t0 + 63 of a [rows, stride] array, W columns from its base, on their way to LDS: held in
// registers between fetch and put, so that the next tile's loads overlap this tile's arithmetic.
// Rows at or past `end` are zeros and are not read.
template <typename T, int W>
struct Staged {
    static constexpr int kPer = 16 / static_cast<int>(sizeof(T));  // elements a 16-byte vector
    static constexpr int kRowVecs = W / kPer;
    static constexpr int kVecs = kTile * kRowVecs / (64 * kWaves);
    u32x4 x[kVecs];

    __device__ __forceinline__ void fetch(const T* base, int64_t stride, int64_t t0, int64_t end) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int q = static_cast<int>(threadIdx.x) + i * 64 * kWaves;
            const int64_t t = t0 + q / kRowVecs;
            x[i] = t < end ? *reinterpret_cast<const u32x4*>(base + t * stride + q % kRowVecs * kPer) : u32x4{0, 0, 0, 0};
        }
    }
    template <int ROW>
    __device__ __forceinline__ void put(T (*dst)[ROW]) const {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int q = static_cast<int>(threadIdx.x) + i * 64 * kWaves;
            *reinterpret_cast<u32x4*>(&dst[q / kRowVecs][q % kRowVecs * kPer]) = x[i];
        }
    }
};

__device__ __forceinline__ int64_t row_length(const int32_t* lengths, int64_t b, int64_t T) {
    if (lengths == nullptr) return T;
    const int64_t n = lengths[b];
    return n < 0 ? 0 : n < T ? n : T;
}

// ---- the walk -----------------------------------------------------------------------------------
// Forward and adjoint walk a sequence tile by tile (64 tokens; 32 where LDS has no room for two tiles of
// float32 rows) with the state in registers.  A workgroup has two kinds of waves:
//   N / 16 state waves, 16 value columns each, take the tile's blocks one after the other;
//   one preparing wave per block of a tile, which meanwhile writes out its 16 rows of the last tile's
//   results, stages its 16 rows of the next tile, and finds that block's decays, X and A from them (no
//   other wave's rows are needed), its loads for the tile after that already on their way.
// All buffers are double, and one barrier a tile is all that is left of waiting for each other: 3.1 us a tile
// at N = 64 for a workgroup alone on its compute unit and 5.9 for two side by side, 6.3 at N = 128.  (Four waves
// that did both in turn, with three barriers a tile, took 5.2 at N = 64.)  What bounds it: the state waves wait
// for nobody, and their chain of products with the splits between takes the time; a full SIMD issues vector
// instructions on about 55 % of its cycles and has products under way on 32 %, and the float32 ones (measured)
// keep it from vector instructions.  Fewer vector instructions or LDS accesses alone no longer moved it.
//
// Adjoint, for L = <go, o> + <ds_out, S_T>, over a block with G the gradient of the state after it:
//     y      = A^T go + diag(beta until) K G
//     lambda = X^T y                               (the gradient of v, and of V - diag(since) K S0)
//     G0     = since_last G + R^T diag(since) go - K^T diag(since) lambda
// which needs neither the states nor the errors of the forward: it writes lambda and the gradient of the
// state after every 64 tokens and leaves the rest, which is independent from tile to tile, to the
// gradient kernels below.
template <typename T, int N>
constexpr int kWalkTile = sizeof(T) * N > 256 ? 32 : 64;

struct WalkArgs {
    int64_t B, T, H, HK, nseg, per;
    const int32_t* lengths;
    const float* w;
    const float* beta;
    const void* r;
    const void* k;
    const void* x;        // v; adjoint: go
    void* y;              // o; adjoint: dv
    const float* first;   // the state before the walk, or NULL (zero)
    const float* starts;  // the same for every segment, or NULL
    float* last;          // the state after it, or NULL
    float* local;         // [B H, nseg, 2, N, N]: a pass for what the segments do
    float* rows;          // the errors, or NULL; adjoint: lambda
    float* states;        // the states before every 64 tokens, or NULL; adjoint: their gradients after
};

// Blocks that the state is split for at once (bf16; see the pairs below).
template <typename T>
constexpr int kPair = sizeof(T) == 2 ? 2 : 1;

template <typename T, int N>
struct WalkShared {
    static constexpr int kTok = kWalkTile<T, N>, kPairs = kTok / (kSub * kPair<T>);
    T k[2][kTok * kRow<T, N>], r[2][kTok * kRow<T, N>];
    T v[2][kTok * kRow<T, N>];                    // x and, block by block, y in its place
    float since[2][kTok];                         // decay from the block's start through the token
    float put[2][kTok];                           // beta until: the write strength, decayed to the block's end
    float inv[2][kTok / kSub][kSub * kSub];       // X or its transpose; before that M diag(beta)
    float att[2][kTok / kSub][kSub * kSub];       // A or its transpose
    uint16_t off[kPair<T> == 2 ? 2 * kPairs : 1][6][64][4];  // terms of what a pair's blocks do to each other, per lane
};

// The piece of four elements 4 q .. of row i of a 16 x 16 table: 16 rows' pieces q lie in different banks.
__device__ __forceinline__ int piece(int i, int q) { return 16 * i + 4 * (q ^ ((i >> 1) & 3)); }

// A wave's 16 rows of N elements between memory (from `base`, the same for the wave) and LDS.  Rows from
// `left` on are zeros and not read, or not written.  Offsets from the base are 32 bits (the host's checks
// keep 64 rows below 2^31 bytes): one register serves every row.
template <typename T, int N>
struct BlockRows {
    static constexpr int kPer = 16 / static_cast<int>(sizeof(T));
    static constexpr int kRowVecs = N / kPer, kRows = 64 / kRowVecs;  // vectors a row, rows an access
    static constexpr int kVecs = kSub / kRows;
    u32x4 x[kVecs];

    __device__ __forceinline__ void fetch(const T* base, int stride, int left, int lane) {
        const int row = lane / kRowVecs;
        const uint32_t at = static_cast<uint32_t>(row * stride + lane % kRowVecs * kPer);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const T* p = base + static_cast<int64_t>(i * kRows) * stride;
            x[i] = u32x4{0, 0, 0, 0};
            if (row + i * kRows < left) x[i] = *reinterpret_cast<const u32x4*>(p + at);
        }
    }
    __device__ __forceinline__ void put(T* dst, int lane) const {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
            *reinterpret_cast<u32x4*>(dst + place<T, N>(lane / kRowVecs + i * kRows, lane % kRowVecs * kPer)) = x[i];
    }
    // rows below `live`, and zeros from there to `left`
    static __device__ __forceinline__ void flush(const T* src, T* base, int stride, int live, int left, int lane) {
        const int row = lane / kRowVecs;
        const uint32_t at = static_cast<uint32_t>(row * stride + lane % kRowVecs * kPer);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            T* p = base + static_cast<int64_t>(i * kRows) * stride;
            if (row + i * kRows < live)
                *reinterpret_cast<u32x4*>(p + at) =
                    *reinterpret_cast<const u32x4*>(src + place<T, N>(row + i * kRows, lane % kRowVecs * kPer));
        }
        if (live >= left || live >= kSub) return;
#pragma unroll 1
        for (int t = live + row; t < left && t < kSub; t += kRows)
            *reinterpret_cast<u32x4*>(base + static_cast<int64_t>(t) * stride + lane % kRowVecs * kPer) = u32x4{0, 0, 0, 0};
    }
};

// rows from `at` up to `end` as an int, 0 when there are none, at most a tile
__device__ __forceinline__ int rows_left(int64_t at, int64_t end) {
    const int64_t n = end - at;
    return n < 0 ? 0 : n < kTile ? static_cast<int>(n) : kTile;
}

// The state's registers (state_row) to and from columns `col` of a row-major [N, N] array.
template <int N>
__device__ __forceinline__ void store_state(float* to, const f4 (&S)[N / 16], int col, int g) {
    const uint32_t at = static_cast<uint32_t>(state_row(0, g, 0) * N + col);
#pragma unroll
    for (int c = 0; c < N / 16; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) (to + state_row(c, 0, q) * N)[at] = S[c][q];
}
template <int N>
__device__ __forceinline__ void load_state(const float* from, f4 (&S)[N / 16], int col, int g) {
    const uint32_t at = static_cast<uint32_t>(state_row(0, g, 0) * N + col);
#pragma unroll
    for (int c = 0; c < N / 16; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) S[c][q] = (from + state_row(c, 0, q) * N)[at];
}

// Pairs (bf16).  Splitting the state for each block of 16 tokens took as long as the products, so two blocks
// 0, 1 share one split: K_j S and R_j S are taken from the state before both, and what block 0 does to block 1
// goes through two more 16 x 16 tables, their decays taken apart at the border of the blocks:
//     e_1 = X_1 (v_1 - total_0 since_1 K_1 S - since_1 (K_1 K_0^T) put_0 e_0),   o_1 += since_1 (R_1 K_0^T) put_0 e_0
// Adjoint: block 1 acts on block 0,
//     y_0 += put_0 ((K_0 R_1^T) since_1 go_1 - (K_0 K_1^T) since_1 lambda_1)
// The tables are split into terms here, once; the wave that prepares the block they lead to reads the other
// one's rows itself, in the order of the products, so it waits for no other wave.  The state's update sums
// over both blocks' tokens at once.
template <typename T, int N, bool kAdj>
struct Partner {};

template <int N, bool kAdj>
struct Partner<uint16_t, N, kAdj> {
    bf8 k[N / 32], r[kAdj ? N / 32 : 1];

    // rows of the other block from `k0` and `r0`, zeros from `left` on
    __device__ __forceinline__ void fetch(const uint16_t* k0, const uint16_t* r0, int stride, int left, int l16, int g) {
        const uint32_t at = static_cast<uint32_t>(l16 * stride + 8 * g);
        const bf8 none = __builtin_bit_cast(bf8, u32x4{0, 0, 0, 0});
#pragma unroll
        for (int m = 0; m < N / 32; ++m) {
            k[m] = none;
            if constexpr (kAdj) r[m] = none;
        }
        if (l16 < left) {
#pragma unroll
            for (int m = 0; m < N / 32; ++m) {
                k[m] = raw8(k0 + 32 * m + at);
                if constexpr (kAdj) r[m] = raw8(r0 + 32 * m + at);
            }
        }
    }
    // x, a row l16 of a table at columns 4 g .., as its terms
    template <int kCount>
    static __device__ __forceinline__ void put(f4 x, uint16_t (*to)[64][4], int lane) {
        const Terms t = split(x);
        *reinterpret_cast<u32x2*>(to[0][lane]) = t.hi;
        *reinterpret_cast<u32x2*>(to[1][lane]) = t.mid;
        if constexpr (kCount == 3) *reinterpret_cast<u32x2*>(to[2][lane]) = t.lo;
    }
    // scale: of row l16
    template <bool kAtt>
    __device__ __forceinline__ void connect(const uint16_t* K, const uint16_t* R, float scale, uint16_t (*off)[64][4], int l16,
                                            int g) const {
        f4 kk = {0.f, 0.f, 0.f, 0.f}, rk = kk;
#pragma unroll
        for (int m = 0; m < N / 32; ++m) {
            const int at = place<uint16_t, N>(l16, 32 * m + 8 * g);
            kk = mfma32(k[m], raw8(K + at), kk);
            if constexpr (kAdj) rk = mfma32(r[m], raw8(K + at), rk);
            else if constexpr (kAtt) rk = mfma32(k[m], raw8(R + at), rk);
        }
        put<3>((kAdj ? -scale : scale) * kk, off, l16 + 16 * g);
        if constexpr (kAdj) put<3>(scale * rk, off + 3, l16 + 16 * g);
        else if constexpr (kAtt) put<2>(-scale * rk, off + 3, l16 + 16 * g);
    }
};

// A table's product with t: all three terms, or (kTerms 2) for a result that is rounded to bf16.
template <int kTerms>
__device__ __forceinline__ f4 times_table(const uint16_t (*off)[64][4], const Terms& t, int lane) {
    const u32x2 hi = *reinterpret_cast<const u32x2*>(off[0][lane]), mid = *reinterpret_cast<const u32x2*>(off[1][lane]);
    f4 acc = {0.f, 0.f, 0.f, 0.f};
    if constexpr (kTerms == 3) {
        const u32x2 lo = *reinterpret_cast<const u32x2*>(off[2][lane]);
        acc = mfma32(pair(hi, lo), pair(t.lo, t.hi), acc);
        acc = mfma32(pair(mid, mid), pair(t.hi, t.mid), acc);
    } else {
        acc = mfma32(pair(mid, mid), pair(t.hi, u32x2{0, 0}), acc);
    }
    return mfma32(pair(hi, hi), pair(t.hi, t.mid), acc);
}

// One wave prepares a block whose rows K, R it has staged: decays, X and (kAtt) A, or (kAdj) their
// transposes.  wt, bt: rate (log2 units) and write strength of token l16.  Register r of group g holds
// element (i = 4 g + r, j = l16) of the 16 x 16 products.  off (bf16, or NULL): this block is the one of its
// pair that the other, whose rows are given, is connected to.
template <typename T, int N, bool kAtt, bool kAdj>
__device__ __forceinline__ void prepare_block(int l16, int g, const T* K, const T* R, float wt, float bt, float* since, float* put,
                                              float* inv, float* att, const Partner<T, N, kAdj>& partner, uint16_t (*off)[64][4]) {
    asm volatile("" : "+v"(l16), "+v"(g));  // else the comparisons below are kept in registers from tile to tile
    const f4 kk = rows_product<N>(K, K, l16, g);
    f4 rk = {0.f, 0.f, 0.f, 0.f};
    if constexpr (kAtt) rk = rows_product<N>(R, K, l16, g);
    // sums through the token and after it, by shifts along the rows of 16 lanes
    float pre = wt, suf = dpp<0x101>(wt);
    pre += dpp<0x111>(pre);
    suf += dpp<0x101>(suf);
    pre += dpp<0x112>(pre);
    suf += dpp<0x102>(suf);
    pre += dpp<0x114>(pre);
    suf += dpp<0x104>(suf);
    pre += dpp<0x118>(pre);
    suf += dpp<0x108>(suf);
    const float from_start = ex2(-pre), to_end = ex2(-suf) * bt;
    if (g == 0) {
        since[l16] = from_start;
        put[l16] = to_end;
    }
    if constexpr (kPair<T> == 2) {
        if (off != nullptr) partner.template connect<kAtt>(K, R, kAdj ? to_end : -from_start, off, l16, g);
        __builtin_amdgcn_sched_barrier(0);  // the other block's rows are done with
    }
    // sum of w over j < l <= i, by quads of tokens: after j in its quad, whole quads between, through i in its
    // own; or what lies between the two when they share one
    const int jq = l16 >> 2, jr = l16 & 3;
    const float w1 = dpp<0x55>(wt), w2 = dpp<0xAA>(wt), w3 = dpp<0xFF>(wt);  // the quad's; by every lane
    const float after = (jr < 1 ? w1 : 0.f) + (jr < 2 ? w2 : 0.f) + (jr < 3 ? w3 : 0.f);
    float quad = wt + dpp<0xB1>(wt);
    quad += dpp<0x4E>(quad);
    const float quad1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(quad), 4));
    const float quad2 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(quad), 8));
    float run = jq == g ? 0.f : after;
    run += jq == 0 && g >= 2 ? quad1 : 0.f;
    run += jq <= 1 && g == 3 ? quad2 : 0.f;
    float gap[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float wi = __shfl(wt, 4 * g + r, 64);
        run += jq == g && r <= jr ? 0.f : wi;
        gap[r] = run;
    }
    f4 m, a;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = 4 * g + r;
        const float f = ex2(-gap[r]) * bt;
        m[r] = l16 < i ? f * kk[r] : 0.f;
        a[r] = l16 <= i ? f * rk[r] : 0.f;
    }
    // X = (I + M)^{-1} four rows at a time (M here with its beta): x is what remains of I's rows of a block of
    // four, less M's other blocks times the rows above, solved against the block's own six numbers.  Each pass
    // takes all four blocks at once from the rows of the pass before, so after three all are what substitution
    // from the first block down gives, with the products on the matrix cores (12 of them, against 120
    // multiplications and 36 LDS reads a lane when each solved a row on its own, whose registers were what the
    // walks spilled).
#pragma unroll
    for (int r = 0; r < 4; ++r) inv[piece(4 * g + r, l16 >> 2) + (l16 & 3)] = m[r];
    if constexpr (kAdj) {
        *reinterpret_cast<f4*>(&att[piece(l16, g)]) = a;
    } else if constexpr (kAtt) {
#pragma unroll
        for (int r = 0; r < 4; ++r) att[piece(4 * g + r, l16 >> 2) + (l16 & 3)] = a[r];
    }
    __builtin_amdgcn_wave_barrier();  // the table is read back by the wave that wrote it
    f4 others = load4(&inv[piece(l16, g)]), unit;
    const f4 m1 = load4(&inv[piece(4 * g + 1, g)]), m2 = load4(&inv[piece(4 * g + 2, g)]), m3 = load4(&inv[piece(4 * g + 3, g)]);
    __builtin_amdgcn_wave_barrier();  // and has been read
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        others[r] = jq > g ? -others[r] : 0.f;
        unit[r] = l16 == 4 * g + r ? 1.f : 0.f;
    }
    const auto own_block = [&](f4 x) {
        x[1] = fmaf(-m1[0], x[0], x[1]);
        x[2] = fmaf(-m2[1], x[1], fmaf(-m2[0], x[0], x[2]));
        x[3] = fmaf(-m3[2], x[2], fmaf(-m3[1], x[1], fmaf(-m3[0], x[0], x[3])));
        return x;
    };
    f4 x = own_block(unit);
#pragma unroll
    for (int n = 0; n < 3; ++n) x = own_block(mma16(others, x, unit));
    // as the state waves read it: X, or its transpose
    if constexpr (kAdj) {
        *reinterpret_cast<f4*>(&inv[piece(l16, g)]) = x;
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) inv[piece(4 * g + r, l16 >> 2) + (l16 & 3)] = x[r];
    }
}

// Four rows 4 g + q of a wave's columns to a float32 array of value rows, those below `rows`.
__device__ __forceinline__ void store_rows(float* base, int stride, int at, f4 x, int g, int rows) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
        if (4 * g + q < rows) (base + q * stride)[static_cast<uint32_t>(4 * g * stride + at)] = x[q];
}

template <typename T, int N>
constexpr int kWalkThreads = 64 * (N / 16 + kWalkTile<T, N> / kSub);
// waves a SIMD: two workgroups a compute unit where LDS has room for them (bf16 at N = 64), else one
template <typename T, int N>
constexpr int kWalkWaves = ((sizeof(T) * N <= 128 ? 2 : 1) * kWalkThreads<T, N> / 64 + 3) / 4;

// kOut false: a pass without o (adjoint: dv, lambda and the states' gradients): for the saved errors and
// states, for the final state, or (local) for what the segments of a time split do.
template <typename T, int N, bool kAdj, bool kOut>
__global__ void __launch_bounds__((kWalkThreads<T, N>), (kWalkWaves<T, N>)) delta_walk_kernel(WalkArgs P) {
    using Shared = WalkShared<T, N>;
    __shared__ Shared sm;
    constexpr int kTok = Shared::kTok, kBlocks = kTok / kSub, kStateWaves = N / 16, kG = kPair<T>, kLen = kRow<T, N>;
    constexpr bool kNeedR = kAdj || kOut;
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int l16 = lane & 15, g = lane >> 4;
    // (batch row, head) fastest, so that what shares rows of r and k runs together; then value columns or
    // (local) the identity's; then the segment.  A pass over segments leaves out the one nothing follows.
    const bool pass = !kOut && P.local != nullptr;
    const int64_t BH = P.B * P.H, bh = blockIdx.x % BH, rest = blockIdx.x / BH;
    const bool unit = pass && (rest & 1) != 0;
    const int64_t seg = (pass ? rest >> 1 : rest) + (kAdj && pass ? 1 : 0);
    const bool given = seg == (kAdj ? P.nseg - 1 : 0);  // starts from the call's own state
    if (unit && given) return;
    const int64_t begin = seg * P.per * kTile, stop = seg == P.nseg - 1 ? P.T : (seg + 1) * P.per * kTile;
    const int64_t b = bh / P.H, h = bh % P.H, hk = h / (P.H / P.HK);
    const int64_t len = row_length(P.lengths, b, P.T);
    const int64_t end = len < stop ? len : stop;
    const int64_t count = end > begin ? (end - begin + kTok - 1) / kTok : 0;  // tiles with a token of this row
    const int64_t vs = P.H * N, vo = b * P.T * vs + h * N;
    const auto start_of = [&](int64_t n) { return begin + (kAdj ? count - 1 - n : n) * kTok; };

    if (wv < kStateWaves) {
        const int c0 = 16 * wv, col = c0 + l16;  // this wave's columns, and this lane's
        const float* first = P.starts != nullptr ? P.starts + (bh * P.nseg + seg) * N * N
                             : P.first != nullptr && given ? P.first + bh * N * N : nullptr;
        f4 S[N / 16];
#pragma unroll
        for (int c = 0; c < N / 16; ++c)
#pragma unroll
            for (int q = 0; q < 4; ++q) S[c][q] = unit && state_row(c, g, q) == col ? 1.f : 0.f;
        if (!unit && first != nullptr) load_state<N>(first, S, col, g);
        __syncthreads();  // the first tile is prepared
#pragma unroll 1
        for (int64_t n = 0; n < count; ++n) {
            asm volatile("" : "+v"(l16), "+v"(g));  // as in prepare_block
            const int64_t t0 = start_of(n);
            const int f = static_cast<int>(n & 1);
            if (P.states != nullptr && !pass && (kTok == kTile || n == 0 || t0 % kTile == (kAdj ? kTile - kTok : 0))) {
                store_state<N>(P.states + (bh * ((P.T + kTile - 1) / kTile) + t0 / kTile) * N * N, S, col, g);
            }
#pragma unroll 1
            for (int i = 0; i < kBlocks / kG; ++i) {
                const int p = kAdj ? kBlocks / kG - 1 - i : i, tb = kSub * kG * p;
                const T *K = sm.k[f] + tb * kLen, *R = sm.r[f] + tb * kLen;
                T* V = sm.v[f] + tb * kLen;
                f4 since[kG], put[kG], inv[kG], att[kG];
                f4 x[kG], kS[kG], out[kG], result[kG];  // result: e; adjoint: lambda
                float total[kG], all = 1.f;
#pragma unroll
                for (int j = 0; j < kG; ++j) {
                    since[j] = load4(&sm.since[f][tb + kSub * j + 4 * g]);
                    total[j] = sm.since[f][tb + kSub * j + kSub - 1];
                    all *= total[j];
                }
                const uint16_t(*off)[64][4] = sm.off[kG == 2 ? f * Shared::kPairs + p : 0];
                const f4 none = {0.f, 0.f, 0.f, 0.f};
                {
                    const StateOperand<T, N> op(S);
#pragma unroll
                    for (int j = 0; j < kG; ++j) kS[j] = op.template times<false>(LeftRows<T, N>(K + j * kSub * kLen, l16, g), g);
                    if constexpr (kOut && !kAdj) {
#pragma unroll
                        for (int j = 0; j < kG; ++j) {
                            const f4 rS = op.template times<true>(LeftRows<T, N>(R + j * kSub * kLen, l16, g), g);
                            out[j] = (j == 0 ? since[j] : total[0] * since[j]) * rS;
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < kG; ++j) {
                    x[j] = value_column<N>(V + j * kSub * kLen, c0, l16, g);
                    put[j] = load4(&sm.put[f][tb + kSub * j + 4 * g]);
                    inv[j] = load4(&sm.inv[f][kG * p + j][piece(l16, g)]);
                    if constexpr (kNeedR) att[j] = load4(&sm.att[f][kG * p + j][piece(l16, g)]);
                }
                f4 u[kG], u2[kG];
#pragma unroll
                for (int c = 0; c < N / 16; ++c) S[c] *= all;
                if constexpr (kAdj) {
                    constexpr int L = kG - 1;
                    result[L] = mma16(inv[L], mma16(att[L], x[L], put[L] * kS[L]), none);
                    u[L] = since[L] * x[L];
                    u2[L] = -since[L] * result[L];
                    if constexpr (kG == 2) {
                        const f4 past = times_table<3>(off + 3, split(u[1]), lane) - times_table<3>(off, split(u2[1]), lane);
                        result[0] = mma16(inv[0], mma16(att[0], x[0], total[1] * put[0] * kS[0] + past), none);
                        u[1] *= total[0];
                        u2[1] *= total[0];
                        u[0] = since[0] * x[0];
                        u2[0] = -since[0] * result[0];
                    }
                } else {
                    result[0] = mma16(inv[0], x[0] - since[0] * kS[0], none);
                    u[0] = put[0] * result[0];
                    if constexpr (kG == 2) {
                        const Terms t = split(u[0]);
                        const f4 rest = x[1] - total[0] * since[1] * kS[1];
                        result[1] = mma16(inv[1], rest + times_table<3>(off, t, lane), none);
                        if constexpr (kOut) out[1] += times_table<2>(off + 3, t, lane);
                        u[0] *= total[1];
                        u[1] = put[1] * result[1];
                    }
                }
                if constexpr (kAdj) LeftCols<T, N>(R, l16, g).add_outer(S, u);
                LeftCols<T, N>(K, l16, g).add_outer(S, kAdj ? u2 : u);
#pragma unroll
                for (int j = 0; j < kG; ++j) {
                    if constexpr (kOut) {
                        const f4 y = kAdj ? result[j] : mma16(att[j], result[j], out[j]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) store1(V + place<T, N>(kSub * j + 4 * g + q, col), y[q]);
                    }
                    const int64_t left = P.T - t0 - tb - kSub * j;
                    if (P.rows != nullptr && !pass && left > 0)
                        store_rows(P.rows + vo + (t0 + tb + kSub * j) * vs + c0, static_cast<int>(vs), l16, result[j], g,
                                   left < kSub ? static_cast<int>(left) : kSub);
                }
            }
            __syncthreads();  // the next tile is prepared, this one's results are in place
        }
        float* last = pass ? P.local + ((bh * P.nseg + seg) * 2 + unit) * N * N
                      : P.last != nullptr && seg == (kAdj ? 0 : P.nseg - 1) ? P.last + bh * N * N : nullptr;
        if (last != nullptr) store_state<N>(last, S, col, g);
    } else {
        const int s = wv - kStateWaves;  // this wave's block of every tile
        const int64_t ks = P.HK * N;
        const T* r = static_cast<const T*>(P.r) + b * P.T * ks + hk * N;
        const T* k = static_cast<const T*>(P.k) + b * P.T * ks + hk * N;
        const T* x = static_cast<const T*>(P.x) + vo;
        T* y = static_cast<T*>(P.y) + vo;
        const float* w = P.w + b * P.T * P.H + h;
        const float* beta = P.beta + b * P.T * P.H + h;
        BlockRows<T, N> fk, fr, fx;
        float wt = 0.f, bt = 0.f;
        const bool connected = kG == 2 && (s & 1) == (kAdj ? 0 : 1);
        const auto fetch = [&](int64_t n) {
            const int64_t t0 = start_of(n) + kSub * s;
            const int left = rows_left(t0, len);
            fk.fetch(k + t0 * ks, static_cast<int>(ks), left, lane);
            if constexpr (kNeedR) fr.fetch(r + t0 * ks, static_cast<int>(ks), left, lane);
            fx.fetch(x + t0 * vs, static_cast<int>(vs), unit ? 0 : left, lane);
            wt = bt = 0.f;
            if (l16 < left) {
                const uint32_t at = static_cast<uint32_t>(l16 * static_cast<int>(P.H));
                wt = (w + t0 * P.H)[at];
                bt = (beta + t0 * P.H)[at];
            }
        };
        const auto prepare = [&](int64_t n) {  // what has been fetched, as tile n; then tile n + 1 is fetched
            const int f = static_cast<int>(n & 1), tb = kSub * s;
            fk.put(sm.k[f] + tb * kLen, lane);
            if constexpr (kNeedR) fr.put(sm.r[f] + tb * kLen, lane);
            fx.put(sm.v[f] + tb * kLen, lane);
            const float wn = wt * kLog2e, bn = bt;
            Partner<T, N, kAdj> other;
            if constexpr (kG == 2) {
                const int64_t tp = start_of(n) + kSub * (kAdj ? s + 1 : s - 1);  // the pair's other block
                if (connected) other.fetch(k + tp * ks, r + tp * ks, static_cast<int>(ks), rows_left(tp, len), l16, g);
            }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_wave_barrier();  // the rows are read back by the wave that wrote them
            prepare_block<T, N, kNeedR, kAdj>(l16, g, sm.k[f] + tb * kLen, sm.r[f] + tb * kLen, wn, bn, &sm.since[f][tb],
                                              &sm.put[f][tb], sm.inv[f][s], sm.att[f][s], other,
                                              connected ? sm.off[kG == 2 ? f * Shared::kPairs + s / kG : 0] : nullptr);
            __builtin_amdgcn_sched_barrier(0);
            if (n + 1 < count) fetch(n + 1);
        };
        const auto flush = [&](int64_t n) {
            const int64_t t0 = start_of(n) + kSub * s;
            // (behind the row's length zero keys met the state, which may not be finite)
            BlockRows<T, N>::flush(sm.v[n & 1] + kSub * s * kLen, y + t0 * vs, static_cast<int>(vs), rows_left(t0, len),
                                   rows_left(t0, P.T), lane);
        };
        if (count > 0) {
            fetch(0);
            prepare(0);
        }
        __syncthreads();
#pragma unroll 1
        for (int64_t n = 0; n < count; ++n) {
            if (kOut && n > 0) flush(n - 1);
            if (n + 1 < count) prepare(n + 1);
            __syncthreads();
        }
        if constexpr (kOut) {
            if (count > 0) flush(count - 1);
            // whole tiles behind the row's length: zeros
            constexpr int kPer = 64 * kBlocks * 4 / N;  // rows at a time
            const int at = static_cast<int>(threadIdx.x) - 64 * kStateWaves;
            for (int64_t t = begin + count * kTok + at / (N / 4); t < stop; t += kPer)
                store4(&y[t * vs + at % (N / 4) * 4], f4{0.f, 0.f, 0.f, 0.f});
        }
    }
}

// A few tokens (decoding): the state makes one trip through memory, updated token by token in
// registers.  One wave per (batch row, head, 64 value columns): lane (q, g) owns columns 4 q .. 4 q + 3
// of rows g N/4 .. (g + 1) N/4 - 1.  k S and r S are both taken from the state before the token, so one
// round of shuffles serves both:  o = e^{-w} r S + (r . k) beta e.  Bound by that trip: 256 streams of 64 heads
// of 64 take 95.5 us, 545 MB at 5.7 TB/s.
template <typename T, int N>
__global__ void __launch_bounds__(256) delta_step_kernel(DeltaArgs P) {
    constexpr int M = N / 4;  // rows a lane
    __shared__ __attribute__((aligned(16))) float tab[kWaves][2][N];
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = static_cast<int64_t>(blockIdx.x) * kWaves + wv;
    if (id >= P.B * P.H * (N / 64)) return;  // a whole wave; the kernel has no barrier
    const int64_t bh = id / (N / 64), cb = id % (N / 64);
    const int64_t b = bh / P.H, h = bh % P.H, hk = h / (P.H / P.HK);
    const int64_t len = row_length(P.lengths, b, P.T);
    const int q = lane & 15, g = lane >> 4;
    const int64_t c0 = cb * 64 + 4 * q;
    const int64_t e0 = (bh * N + g * M) * N + c0;
    f4 x[M];
#pragma unroll
    for (int m = 0; m < M; ++m)
        x[m] = P.s_in != nullptr ? __builtin_nontemporal_load(reinterpret_cast<const f4*>(P.s_in + e0 + m * N))
                                 : f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int64_t t = 0; t < len; ++t) {
        const int64_t row = b * P.T + t;
        float rk = 0.f;
#pragma unroll
        for (int c = 0; c < N; c += 64) {
            const float rl = widen(static_cast<const T*>(P.r)[(row * P.HK + hk) * N + c + lane]);
            const float kl = widen(static_cast<const T*>(P.k)[(row * P.HK + hk) * N + c + lane]);
            tab[wv][0][c + lane] = rl;
            tab[wv][1][c + lane] = kl;
            rk = fmaf(rl, kl, rk);
        }
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) rk += __shfl_xor(rk, m, 64);
        const f4 v = load4(static_cast<const T*>(P.v) + (row * P.H + h) * N + c0);
        const float a = ex2(-P.w[row * P.H + h] * kLog2e), beta = P.beta[row * P.H + h];
        __builtin_amdgcn_wave_barrier();
        f4 kS = {0.f, 0.f, 0.f, 0.f}, rS = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < M; m += 4) {
            const f4 r4 = load4(&tab[wv][0][g * M + m]), k4 = load4(&tab[wv][1][g * M + m]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                rS += r4[i] * x[m + i];
                kS += k4[i] * x[m + i];
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            kS[c] += __shfl_xor(kS[c], 16, 64);
            rS[c] += __shfl_xor(rS[c], 16, 64);
            kS[c] += __shfl_xor(kS[c], 32, 64);
            rS[c] += __shfl_xor(rS[c], 32, 64);
        }
        const f4 u = beta * (v - a * kS);
#pragma unroll
        for (int m = 0; m < M; m += 4) {
            const f4 k4 = load4(&tab[wv][1][g * M + m]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[m + i] = a * x[m + i] + k4[i] * u;
        }
        if (g == 0) store4(static_cast<T*>(P.o) + (row * P.H + h) * N + c0, a * rS + rk * u);
        __builtin_amdgcn_wave_barrier();  // tab is read before the next token overwrites it
    }
    for (int64_t t = len; t < P.T; ++t)
        if (g == 0) store4(static_cast<T*>(P.o) + ((b * P.T + t) * P.H + h) * N + c0, f4{0.f, 0.f, 0.f, 0.f});
    if (P.s_out != nullptr) {
#pragma unroll
        for (int m = 0; m < M; ++m) __builtin_nontemporal_store(x[m], reinterpret_cast<f4*>(P.s_out + e0 + m * N));
    }
}

// ---- gradients ----------------------------------------------------------------------------------
// The gradients that are sums over the value columns, tile by tile.  Over a tile of 64 tokens from the
// state S0 with G the gradient of the state after it, all decays now counted inside the tile:
//     dA_ij = ratio_ij beta_j go_i . e_j  (j <= i),   dM_ij = -ratio_ij beta_j lambda_i . e_j  (j < i)
//     dr_i = since_i S0 go_i + sum_j dA_ij k_j
//     dk_i = -since_i S0 lambda_i + until_i beta_i G e_i
//            + sum_{j < i} dM_ij k_j + sum_{l >= i} dA_li r_l + sum_{l > i} dM_li k_l
//     dbeta_j = until_j k_j . G e_j + sum_i P_ij,   P_ij = ratio_ij (r_i . k_j go_i - k_i . k_j lambda_i) . e_j
// and the rate of token t takes every term whose path crosses from before t to t or later:
//     -dw_t = sum_{j < t <= i} beta_j P_ij + sum_{i >= t} since_i (r_i . S0 go_i - k_i . S0 lambda_i)
//             + sum_{j < t} until_j beta_j k_j . G e_j + since_last <G, S0>
// sums of the terms themselves, so no running sum is subtracted from another.
//
// One workgroup per (tile, batch row, key head); it takes the value heads of its key head one after the
// other and keeps dr, dk in registers (a fixed order of summation).  Wave x owns tokens 16 x .. 16 x + 15:
// as i it meets the blocks J <= x, as j the blocks I >= x (5 blocks for every wave).  Both times the
// 16 x 16 block is formed with the wave's own tokens as its columns, so it is already the right operand
// of the products that follow; dr and dk come out transposed, four consecutive channels a lane.  Bound by the
// latency of 670 float32 products a wave and head, two heads of a tile 43 us (rows of 333 tokens, 48 workgroups).
template <int N>
struct GradShared {
    static constexpr bool kGoInLds = N == 64;  // N = 128 reads go from memory: 160 KB of LDS
    float k[kTile][kRow<float, N>];
    float r[kTile][kRow<float, N>];
    float go[kGoInLds ? kTile : 1][kRow<float, N>];
    float e[kTile][N + 4];
    float lam[kTile][N + 4];
    float w[kTile], beta[kTile];
    float pre[kTile], suf[kTile];        // sums of w in the token's block: through it, and after it
    float total[kWaves];                 // of w in each block
    float diag[kWaves][kSub][kPadM];     // beta_j P_ij of the blocks I == J
    float cross[kWaves][kWaves];         // [I][J]: sum of beta_j P_ij
    float rows[kWaves], cols[kWaves];    // block sums of the terms that pair with S0, and with G
    float rowv[kWaves][kSub], colv[kWaves][kSub];
};

// The gradients of a tile from its row `from` on, which lies behind the row's length: zeros.  (What the products
// would give there is 0 times the states, which need not be finite.)
template <typename T, int N>
__device__ void zero_tile(const DeltaBwdArgs& P, T* dr, T* dk, int64_t b, int64_t hk, int64_t t0, int from) {
    const int64_t rows = P.T - t0 < kTile ? P.T - t0 : kTile, per = P.H / P.HK, ks = P.HK * N;
    for (int64_t t = from + threadIdx.x / 16; t < rows; t += blockDim.x / 16) {
        for (int c = threadIdx.x % 16 * 4; c < N; c += 64) {
            store4(&dr[(t0 + t) * ks + c], f4{0.f, 0.f, 0.f, 0.f});
            store4(&dk[(t0 + t) * ks + c], f4{0.f, 0.f, 0.f, 0.f});
        }
    }
    for (int64_t i = from * per + threadIdx.x; i < rows * per; i += blockDim.x) {
        const int64_t at = (b * P.T + t0 + i / per) * P.H + hk * per + i % per;
        P.dw[at] = 0.f;
        P.dbeta[at] = 0.f;
    }
}

__device__ __forceinline__ float sum16(float x) { return sum_lanes(x, 16); }

template <int N>
__global__ void __launch_bounds__(64 * kWaves, 1) delta_grad_kernel(DeltaBwdArgs P) {
    using T = float;
    __shared__ GradShared<N> sm;
    constexpr int NC = N / 16;
    const int lane = threadIdx.x & 63;
    const int x = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int l16 = lane & 15, g = lane >> 4;
    const int64_t ntile = (P.T + kTile - 1) / kTile;
    const int64_t bhk = blockIdx.x % (P.B * P.HK), tile = blockIdx.x / (P.B * P.HK);
    const int64_t b = bhk / P.HK, hk = bhk % P.HK, per = P.H / P.HK;
    const int64_t len = row_length(P.lengths, b, P.T);
    const int64_t ks = P.HK * N, vs = P.H * N, t0 = tile * kTile;
    const int64_t ko = b * P.T * ks + hk * N;
    T* dr = static_cast<T*>(P.dr) + ko;
    T* dk = static_cast<T*>(P.dk) + ko;
    const int left = rows_left(t0, len);
    if (left < kTile) zero_tile<T, N>(P, dr, dk, b, hk, t0, left);
    if (left == 0) return;  // nothing of this row here
    {
        Staged<T, N> s;
        s.fetch(static_cast<const T*>(P.k) + ko, ks, t0, len);
        s.put(sm.k);
        s.fetch(static_cast<const T*>(P.r) + ko, ks, t0, len);
        s.put(sm.r);
    }
    f4 drT[NC], dkT[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) drT[c] = dkT[c] = f4{0.f, 0.f, 0.f, 0.f};
    const int mine = kSub * x + l16;  // this lane's token of the tile

#pragma unroll 1
    for (int64_t h = hk * per; h < (hk + 1) * per; ++h) {
        const int64_t bh = b * P.H + h, vo = b * P.T * vs + h * N;
        const T* go = static_cast<const T*>(P.go) + vo;
        __syncthreads();  // the last head's readers are done
        if constexpr (GradShared<N>::kGoInLds) {
            Staged<T, N> s;
            s.fetch(go, vs, t0, len);
            s.put(sm.go);
        }
        {
            Staged<float, N> s;
            s.fetch(P.errs + vo, vs, t0, len);
            s.put(sm.e);
            s.fetch(P.lambda + vo, vs, t0, len);
            s.put(sm.lam);
        }
        if (threadIdx.x < kTile) {
            const int64_t t = t0 + threadIdx.x;
            sm.w[threadIdx.x] = t < len ? P.w[(b * P.T + t) * P.H + h] * kLog2e : 0.f;
            sm.beta[threadIdx.x] = t < len ? P.beta[(b * P.T + t) * P.H + h] : 0.f;
        }
        __syncthreads();
        asm volatile("" : "+v"(l16), "+v"(g));
        float pre = 0.f, suf = 0.f;  // of this lane's token
#pragma unroll
        for (int l = 0; l < kSub; ++l) {
            const float wl = sm.w[kSub * x + l];
            pre += l <= l16 ? wl : 0.f;
            suf += l > l16 ? wl : 0.f;
        }
        if (g == 0) {
            sm.pre[mine] = pre;
            sm.suf[mine] = suf;
            if (l16 == 15) sm.total[x] = pre;
        }
        __syncthreads();
        float before = 0.f, after = 0.f;  // rates of the blocks before and after this wave's
        for (int i = 0; i < kWaves; ++i) {
            before += i < x ? sm.total[i] : 0.f;
            after += i > x ? sm.total[i] : 0.f;
        }
        const float since = ex2(-(before + pre)), until = ex2(-(suf + after)), beta = sm.beta[mine];
        const float all = ex2(-(before + sm.total[x] + after));

        // rows of this wave's tokens: go, lambda, e as right operands
        const auto go4 = [&](int row, int c) -> f4 {
            if constexpr (GradShared<N>::kGoInLds) {
                return load4(&sm.go[row][16 * c + 4 * g]);
            } else {
                return t0 + row < len ? load4(&go[(t0 + row) * vs + 16 * c + 4 * g]) : f4{0.f, 0.f, 0.f, 0.f};
            }
        };
        f4 goX[NC], laX[NC], eX[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            goX[c] = go4(mine, c);
            laX[c] = load4(&sm.lam[mine][16 * c + 4 * g]);
            eX[c] = load4(&sm.e[mine][16 * c + 4 * g]);
        }
        // products with the states before and after the tile
        const float* S0 = P.states + (bh * ntile + tile) * N * N;
        const float* G1 = P.gstates + (bh * ntile + tile) * N * N;
        float withS = 0.f, withG = 0.f, inner = 0.f;
#pragma unroll 1
        for (int c = 0; c < NC; ++c) {
            f4 sg = {0.f, 0.f, 0.f, 0.f}, sl = {0.f, 0.f, 0.f, 0.f}, ge = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int d = 0; d < NC; ++d) {
                const f4 s4 = load4(&S0[(16 * c + l16) * N + 16 * d + 4 * g]);
                const f4 g4 = load4(&G1[(16 * c + l16) * N + 16 * d + 4 * g]);
                sg = mma16(s4, goX[d], sg);
                sl = mma16(s4, laX[d], sl);
                ge = mma16(g4, eX[d], ge);
#pragma unroll
                for (int q = 0; q < 4; ++q) inner = fmaf(s4[q], g4[q], inner);
            }
            const f4 rr = load4(&sm.r[mine][16 * c + 4 * g]), kk = load4(&sm.k[mine][16 * c + 4 * g]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                withS += rr[q] * sg[q] - kk[q] * sl[q];
                withG += kk[q] * ge[q];
            }
            const f4 a = since * sg, d = until * beta * ge - since * sl;
#pragma unroll
            for (int j = 0; j < NC; ++j) {  // (drT[c] with c known only at run time would spill)
                if (j == c) {
                    drT[j] += a;
                    dkT[j] += d;
                }
            }
        }
        withS = since * sum_rows(withS);
        withG = until * sum_rows(withG);
        inner = sum16(sum_rows(inner));
        float rowv = withS, colv = beta * withG, dbeta = withG;

        // blocks J <= x with this wave's tokens as i: rows j = 4 g + q, columns i
#pragma unroll 1
        for (int J = 0; J <= x; ++J) {
            asm volatile("" : "+v"(l16), "+v"(g));  // else comparisons are worked out ahead and kept (spilled)
            f4 ae = {0.f, 0.f, 0.f, 0.f}, le = {0.f, 0.f, 0.f, 0.f}, kk = {0.f, 0.f, 0.f, 0.f}, rk = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const f4 e4 = load4(&sm.e[kSub * J + l16][16 * c + 4 * g]);
                ae = mma16(e4, goX[c], ae);
                le = mma16(e4, laX[c], le);
                const f4 k4 = load4(&sm.k[kSub * J + l16][16 * c + 4 * g]);
                kk = mma16(k4, load4(&sm.k[mine][16 * c + 4 * g]), kk);
                rk = mma16(k4, load4(&sm.r[mine][16 * c + 4 * g]), rk);
            }
            float mid = pre;
            for (int i = 0; i < kWaves; ++i) mid += i > J && i < x ? sm.total[i] : 0.f;
            float gap[4];
            if (J == x) {
                float run = 0.f;
#pragma unroll
                for (int l = kSub - 1; l >= 0; --l) {  // rates after token l, through l16
                    if (l / 4 == g) gap[l % 4] = run;
                    run += l <= l16 ? sm.w[kSub * x + l] : 0.f;
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) gap[q] = mid + sm.suf[kSub * J + 4 * g + q];
            }
            f4 da, dm;
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int j = 4 * g + q;
                const bool ia = J < x || j <= l16, im = J < x || j < l16;
                const float f = ex2(-gap[q]) * sm.beta[kSub * J + j];
                da[q] = ia ? f * ae[q] : 0.f;
                dm[q] = im ? -f * le[q] : 0.f;
                sum += da[q] * rk[q] + dm[q] * kk[q];
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                f4 a;
#pragma unroll
                for (int q = 0; q < 4; ++q) a[q] = widen(sm.k[kSub * J + 4 * g + q][16 * c + l16]);
                drT[c] = mma16(a, da, drT[c]);
                dkT[c] = mma16(a, dm, dkT[c]);
            }
            if (J < x) {
                sum = sum_rows(sum);
                rowv += sum;
                sum = sum16(sum);
                if (lane == 0) sm.cross[x][J] = sum;
            }
        }
        // blocks I >= x with this wave's tokens as j: rows i = 4 g + q, columns j
#pragma unroll 1
        for (int I = x; I < kWaves; ++I) {
            asm volatile("" : "+v"(l16), "+v"(g));
            f4 ae = {0.f, 0.f, 0.f, 0.f}, le = {0.f, 0.f, 0.f, 0.f}, kk = {0.f, 0.f, 0.f, 0.f}, rk = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                ae = mma16(go4(kSub * I + l16, c), eX[c], ae);
                le = mma16(load4(&sm.lam[kSub * I + l16][16 * c + 4 * g]), eX[c], le);
                const f4 k4 = load4(&sm.k[mine][16 * c + 4 * g]);
                kk = mma16(load4(&sm.k[kSub * I + l16][16 * c + 4 * g]), k4, kk);
                rk = mma16(load4(&sm.r[kSub * I + l16][16 * c + 4 * g]), k4, rk);
            }
            float mid = suf;
            for (int i = 0; i < kWaves; ++i) mid += i > x && i < I ? sm.total[i] : 0.f;
            float gap[4];
            if (I == x) {
                float run = 0.f;
#pragma unroll
                for (int l = 0; l < kSub; ++l) {  // rates after l16, through token l
                    run += l > l16 ? sm.w[kSub * x + l] : 0.f;
                    if (l / 4 == g) gap[l % 4] = run;
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) gap[q] = mid + sm.pre[kSub * I + 4 * g + q];
            }
            f4 da, dm;
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = 4 * g + q;
                const bool ia = I > x || l16 <= i, im = I > x || l16 < i;
                const float f = ex2(-gap[q]);
                da[q] = ia ? f * ae[q] : 0.f;
                dm[q] = im ? -f * le[q] : 0.f;
                const float p = da[q] * rk[q] + dm[q] * kk[q];
                if (I == x) sm.diag[x][i][l16] = beta * p;
                sum += p;
            }
            sum = sum_rows(sum);
            dbeta += sum;
            if (I > x) colv += beta * sum;
            da *= beta;
            dm *= beta;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                f4 a, a2;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    a[q] = widen(sm.r[kSub * I + 4 * g + q][16 * c + l16]);
                    a2[q] = widen(sm.k[kSub * I + 4 * g + q][16 * c + l16]);
                }
                dkT[c] = mma16(a2, dm, mma16(a, da, dkT[c]));
            }
        }
        // the rates
        const float rowsum = sum16(withS), colsum = sum16(beta * withG);
        if (lane == 0) {
            sm.rows[x] = rowsum;
            sm.cols[x] = colsum;
        }
        if (g == 0) {
            sm.rowv[x][l16] = rowv;
            sm.colv[x][l16] = colv;
        }
        __syncthreads();
        asm volatile("" : "+v"(l16), "+v"(g));
        float c = 0.f;  // this group's four rows of the token's block
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int i = 4 * g + q;
            c += i >= l16 ? sm.rowv[x][i] : sm.colv[x][i];
#pragma unroll
            for (int j = 0; j < kSub; ++j) c += j < l16 && i >= l16 ? sm.diag[x][i][j] : 0.f;
        }
        c = sum_rows(c);
        if (g == 0 && t0 + mine < len) {
            c = fmaf(all, inner, c);
            for (int I = x + 1; I < kWaves; ++I) {
                c += sm.rows[I];
                for (int J = 0; J < x; ++J) c += sm.cross[I][J];
            }
            for (int J = 0; J < x; ++J) c += sm.cols[J];
            const int64_t at = (b * P.T + t0 + mine) * P.H + h;
            P.dw[at] = -c;
            P.dbeta[at] = dbeta;
        }
    }
    if (t0 + mine < len) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            store4(&dr[(t0 + mine) * ks + 16 * c + 4 * g], drT[c]);
            store4(&dk[(t0 + mine) * ks + 16 * c + 4 * g], dkT[c]);
        }
    }
}

// The same from bf16 inputs.  Here a wave owns 16 channels of r and k instead of 16 tokens: it reads its
// rows of S0 and G once, splits them in registers, and takes the tile's tokens of go, lambda and e, split
// when they are staged, past them (eight waves; at N = 64 two of them share a slice, 32 tokens each).
// Phases between barriers:
//   1. stage k, r, go, and the three terms of e and lambda
//   2. the products with S0 and G; the 16 x 16 blocks (I, J), J <= I, of dA, dM and P: ten blocks dealt
//      to the waves
//   3. dA, dM and their transposes, as hi + mid (dr and dk are rounded to bf16), to LDS over e and
//      lambda, each lane's eight values where the lane that needs them reads them
//   4. every wave: its channels of the products of k and r with all ten blocks; and the rates
// Everything the tile needs of a head is on its way before the first of it is put into LDS, and chains of
// dependent products are taken in turn.  At N = 64 two workgroups share a compute unit (128 registers, some
// spilled), each one's loads behind the other's work; one with twice the registers that fetched its next tile
// ahead took as long (8 x 1024 tokens of 64 heads, forward and backward, 601 us against 607).  The 870 MB of
// that case take 325 to 347 us (2.5 to 2.7 TB/s): the phases' products and LDS traffic, which meet at four barriers
// a tile.
constexpr int kGradWaves = 8;
template <int N>
constexpr int kGradShare = N == 64 ? 2 : 1;  // workgroups a compute unit
constexpr int kGradThreads = 64 * kGradWaves;

template <int N>
struct GradShared16 {
    uint16_t k[kTile][N], r[kTile][N], go[kTile][N];
    union {
        struct {
            uint16_t e[3][kTile][N], lam[3][kTile][N];
        };
        uint16_t da[10][4][64][8];  // [block][dA, dM, dA^T, dM^T][lane][hi 4, mid 4]
    };
    float w[kTile], beta[kTile];
    float pre[kTile], suf[kTile], since[kTile], until[kTile];
    float total[kWaves];
    float rowsum[10][kSub], colsum[10][kSub];  // of beta_j P_ij over j, of P_ij over i
    float withS[N / 16][kTile], withG[N / 16][kTile], inner[N / 16];
    float diag[kTile];                         // the crossing pairs inside the token's own block
};

template <int N>
__device__ __forceinline__ bf8 row8(const uint16_t (*X)[N], int t, int c) { return raw8(&X[t][swizzled<N>(t, c)]); }

// tokens tb + 4 g .. + 3 of channel c0 + l16, twice
template <int N>
__device__ __forceinline__ bf8 col_twice(const uint16_t (*X)[N], int tb, int c0, int l16, int g) {
    const int t = tb + 4 * g + (l16 >> 2);
    const s4 raw = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s4*)&X[t][swizzled<N>(t, c0 + 4 * (l16 & 3))]);
    const u32x2 a = __builtin_bit_cast(u32x2, raw);
    return pair(a, a);
}

__device__ __forceinline__ void split8(f4 a, f4 b, bf8 (&out)[3]) {
    const Terms x = split(a), y = split(b);
    out[0] = pair(x.hi, y.hi);
    out[1] = pair(x.mid, y.mid);
    out[2] = pair(x.lo, y.lo);
}

// A workgroup's rows t0 .. t0 + 63 of a [rows, N] array at `base` (the first row), between memory and LDS:
// all of a tile's loads are issued before the first is waited for.
template <int N>
struct GradRows {
    static constexpr int kRowVecs = N / 8, kRows = kGradThreads / kRowVecs, kVecs = kTile / kRows;
    u32x4 x[kVecs];
    __device__ __forceinline__ void fetch(const uint16_t* base, int stride, int left) {
        const int row = static_cast<int>(threadIdx.x) / kRowVecs;
        const uint32_t at = static_cast<uint32_t>(row * stride + static_cast<int>(threadIdx.x) % kRowVecs * 8);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            x[i] = u32x4{0, 0, 0, 0};
            if (row + i * kRows < left)
                x[i] = *reinterpret_cast<const u32x4*>(base + static_cast<int64_t>(i * kRows) * stride + at);
        }
    }
    __device__ __forceinline__ void put(uint16_t (*dst)[N]) const {
        const int row = static_cast<int>(threadIdx.x) / kRowVecs, c = static_cast<int>(threadIdx.x) % kRowVecs * 8;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) *reinterpret_cast<u32x4*>(&dst[row + i * kRows][swizzled<N>(row + i * kRows, c)]) = x[i];
    }
};

// the same from float32, split into its terms
template <int N>
struct GradTerms {
    static constexpr int kRowVecs = N / 8, kRows = kGradThreads / kRowVecs, kVecs = kTile / kRows;
    f4 a[kVecs], b[kVecs];
    __device__ __forceinline__ void fetch(const float* base, int stride, int left) {
        const int row = static_cast<int>(threadIdx.x) / kRowVecs;
        const uint32_t at = static_cast<uint32_t>(row * stride + static_cast<int>(threadIdx.x) % kRowVecs * 8);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            a[i] = b[i] = f4{0.f, 0.f, 0.f, 0.f};
            if (row + i * kRows < left) {
                const float* p = base + static_cast<int64_t>(i * kRows) * stride + at;
                a[i] = load4(p);
                b[i] = load4(p + 4);
            }
        }
    }
    __device__ __forceinline__ void put(uint16_t (*dst)[kTile][N]) const {
        const int row = static_cast<int>(threadIdx.x) / kRowVecs, c = static_cast<int>(threadIdx.x) % kRowVecs * 8;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            bf8 x[3];
            split8(a[i], b[i], x);
#pragma unroll
            for (int p = 0; p < 3; ++p) *reinterpret_cast<bf8*>(&dst[p][row + i * kRows][swizzled<N>(row + i * kRows, c)]) = x[p];
        }
    }
};

// Step i of a b for two factors in three terms each: all but the products below 2^-24 of the whole, the
// smallest first.
__device__ __forceinline__ f4 mma_step(int i, const bf8 (&a)[3], const bf8 (&b)[3], f4 c) {
    constexpr int kA[6] = {2, 0, 1, 1, 0, 0}, kB[6] = {0, 2, 1, 0, 1, 0};
    return mfma32(a[kA[i]], b[kB[i]], c);
}

template <int N>
__global__ void __launch_bounds__(kGradThreads, 2 * kGradShare<N>) delta_grad16_kernel(DeltaBwdArgs P) {
    __shared__ GradShared16<N> sm;
    constexpr int NS = N / 16;               // slices of 16 channels
    constexpr int NX = 4 * NS / kGradWaves;  // token blocks a wave takes of its slice
    constexpr int NM = N / 32;
    int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int l16 = lane & 15, g = lane >> 4;
    // counted in 32 bits (the host's checks keep the tiles of all pairs below 2^31), stepped without a division
    const uint32_t ntile = static_cast<uint32_t>((P.T + kTile - 1) / kTile), HK = static_cast<uint32_t>(P.HK);
    const uint32_t pairs = static_cast<uint32_t>(P.B) * HK, per = static_cast<uint32_t>(P.H) / HK;
    const uint32_t tiles_on = gridDim.x / pairs, pairs_on = gridDim.x % pairs;
    const int64_t ks = P.HK * N, vs = P.H * N;
    const int slice = wv % NS, c0 = 16 * slice, X0 = wv / NS * NX;

    // A (tile, batch row, key head), batch row and head fastest, and one of its value heads.
    struct Place {
        uint32_t pair, tile, b, hk, h;
        int left;
    };
    Place at, next;
    const auto advance = [&](Place& p) {
        p.tile += tiles_on;
        p.pair += pairs_on;
        if (p.pair >= pairs) {
            p.pair -= pairs;
            ++p.tile;
        }
    };
    // from a place on, the workgroup's first that holds tokens; what lies behind the rows' lengths gets zeros
    const auto settle = [&](Place& p) {
        for (; p.tile < ntile; advance(p)) {
            p.b = p.pair / HK;
            p.hk = p.pair % HK;
            p.h = p.hk * per;
            const int64_t t0 = static_cast<int64_t>(p.tile) * kTile;
            p.left = rows_left(t0, row_length(P.lengths, p.b, P.T));
            if (p.left < kTile) {
                const int64_t ko = p.b * P.T * ks + p.hk * N;
                zero_tile<uint16_t, N>(P, static_cast<uint16_t*>(P.dr) + ko, static_cast<uint16_t*>(P.dk) + ko, p.b, p.hk, t0,
                                       p.left);
                if (p.left == 0) continue;
            }
            return;
        }
    };
    GradRows<N> fk, fr, fg;
    GradTerms<N> fe, fl;
    float wt, bt;
    const auto fetch = [&](const Place& p) {
        const int64_t row = p.b * P.T + static_cast<int64_t>(p.tile) * kTile;
        const int64_t ko = row * ks + p.hk * N, vo = row * vs + p.h * N;
        fk.fetch(static_cast<const uint16_t*>(P.k) + ko, static_cast<int>(ks), p.left);
        fr.fetch(static_cast<const uint16_t*>(P.r) + ko, static_cast<int>(ks), p.left);
        fg.fetch(static_cast<const uint16_t*>(P.go) + vo, static_cast<int>(vs), p.left);
        fe.fetch(P.errs + vo, static_cast<int>(vs), p.left);
        fl.fetch(P.lambda + vo, static_cast<int>(vs), p.left);
        wt = bt = 0.f;
        if (static_cast<int>(threadIdx.x) < p.left) {
            wt = P.w[(row + lane) * P.H + p.h] * kLog2e;
            bt = P.beta[(row + lane) * P.H + p.h];
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    f4 drT[NX], dkT[NX];  // of token block X0 + x: channels c0 + 4 g .. + 3 of token l16
#pragma unroll
    for (int x = 0; x < NX; ++x) drT[x] = dkT[x] = f4{0.f, 0.f, 0.f, 0.f};

    at.pair = blockIdx.x % pairs;
    at.tile = blockIdx.x / pairs;
    settle(at);
    if (at.tile >= ntile) return;
    bool first = true;
#pragma unroll 1
    while (at.tile < ntile) {
        // else every address and comparison below is worked out before the loop and kept in registers
        asm volatile("" : "+v"(lane), "+v"(l16), "+v"(g));
        const int64_t b = at.b, h = at.h, t0 = static_cast<int64_t>(at.tile) * kTile;
        const int64_t len = t0 + at.left;
        fetch(at);
        if (!first) __syncthreads();  // the last tile's readers are done
        first = false;
        fk.put(sm.k);
        fr.put(sm.r);
        fg.put(sm.go);
        fe.put(sm.e);
        fl.put(sm.lam);
        if (threadIdx.x < kTile) {  // one wave: the decays of its 64 tokens
            // sums in the token's block, through it and after it, by shifts along the rows of 16 lanes
            float pre = wt, suf = dpp<0x101>(wt);
            pre += dpp<0x111>(pre);
            suf += dpp<0x101>(suf);
            pre += dpp<0x112>(pre);
            suf += dpp<0x102>(suf);
            pre += dpp<0x114>(pre);
            suf += dpp<0x104>(suf);
            pre += dpp<0x118>(pre);
            suf += dpp<0x108>(suf);
            float before = 0.f, after = 0.f;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                const float total = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(pre), kSub * i + kSub - 1));
                before += i < g ? total : 0.f;
                after += i > g ? total : 0.f;
            }
            sm.w[lane] = wt;
            sm.beta[lane] = bt;
            sm.pre[lane] = pre;
            sm.suf[lane] = suf;
            sm.since[lane] = ex2(-(before + pre));
            sm.until[lane] = ex2(-(suf + after));
            if (l16 == kSub - 1) sm.total[g] = pre;
        }
        __syncthreads();

        next = at;
        if (++next.h == (at.hk + 1) * per) {
            advance(next);
            settle(next);
        }

        // ---- products with the states before and after the tile, for this wave's channels and tokens
        {
            float inner = 0.f;
            f4 sg[NX], sl[NX], ge[NX];
#pragma unroll
            for (int x = 0; x < NX; ++x) sg[x] = sl[x] = ge[x] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const int v = 32 * m + 8 * g;
                const int64_t from = ((b * P.H + h) * ntile + at.tile) * N * N + 32 * m;
                const uint32_t mine = static_cast<uint32_t>((c0 + l16) * N + 8 * g);
                const f4 sa = load4(P.states + from + mine), sb = load4(P.states + from + 4 + mine);
                const f4 ga = load4(P.gstates + from + mine), gb = load4(P.gstates + from + 4 + mine);
#pragma unroll
                for (int q = 0; q < 4; ++q) inner = fmaf(sa[q], ga[q], fmaf(sb[q], gb[q], inner));
                bf8 s3[3];
                split8(sa, sb, s3);
#pragma unroll
                for (int x = 0; x < NX; ++x) {
                    const int t = kSub * (X0 + x) + l16;
                    const bf8 la[3] = {row8<N>(sm.lam[0], t, v), row8<N>(sm.lam[1], t, v), row8<N>(sm.lam[2], t, v)};
                    const bf8 go = row8<N>(sm.go, t, v);
#pragma unroll
                    for (int i = 0; i < 6; ++i) {
                        sl[x] = mma_step(i, s3, la, sl[x]);
                        if (i % 2) sg[x] = mfma32(s3[2 - i / 2], go, sg[x]);
                    }
                    __builtin_amdgcn_sched_barrier(0);  // more of the reads at once would spill
                }
                bf8 g3[3];
                split8(ga, gb, g3);
#pragma unroll
                for (int x = 0; x < NX; x += 2) {
                    const int t = kSub * (X0 + x) + l16;
                    const bf8 e[3] = {row8<N>(sm.e[0], t, v), row8<N>(sm.e[1], t, v), row8<N>(sm.e[2], t, v)};
                    const bf8 e2[3] = {row8<N>(sm.e[0], t + kSub, v), row8<N>(sm.e[1], t + kSub, v),
                                       row8<N>(sm.e[2], t + kSub, v)};
#pragma unroll
                    for (int i = 0; i < 6; ++i) {
                        ge[x] = mma_step(i, g3, e, ge[x]);
                        ge[x + 1] = mma_step(i, g3, e2, ge[x + 1]);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                const int t = kSub * (X0 + x) + l16, at = swizzled<N>(t, c0 + 4 * g);
                const f4 rr = load4(&sm.r[t][at]), kk = load4(&sm.k[t][at]);
                const float since = sm.since[t], until = sm.until[t], put = until * sm.beta[t];
                float withS = 0.f, withG = 0.f;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    withS += rr[q] * sg[x][q] - kk[q] * sl[x][q];
                    withG += kk[q] * ge[x][q];
                }
                drT[x] += since * sg[x];
                dkT[x] += put * ge[x] - since * sl[x];
                withS = sum_rows(since * withS);
                withG = sum_rows(until * withG);
                if (g == 0) {
                    sm.withS[slice][t] = withS;
                    sm.withG[slice][t] = withG;
                }
            }
            inner = sum_lanes(inner, 64);
            if (lane == 0) sm.inner[slice] = inner;
        }
        asm volatile("" : "+v"(lane), "+v"(l16), "+v"(g));
        __builtin_amdgcn_sched_barrier(0);
        // ---- the 16 x 16 blocks: rows i = 4 g + q of block I, column j = l16 of block J
        f4 da[2], dm[2];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int id = wv + (kGradWaves - 6) * n;  // waves 6 and 7 take two; wave 0 has the rates
            if (n > 0 && wv < 6) continue;
            __builtin_amdgcn_sched_barrier(0);
            const int I = id >= 6 ? 3 : id >= 3 ? 2 : id >= 1 ? 1 : 0, J = id - I * (I + 1) / 2;
            const int ti = kSub * I + l16, tj = kSub * J + l16;
            f4 ae = {0.f, 0.f, 0.f, 0.f}, le = ae, kk = ae, rk = ae;
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const int c = 32 * m + 8 * g;
                const bf8 e[3] = {row8<N>(sm.e[0], tj, c), row8<N>(sm.e[1], tj, c), row8<N>(sm.e[2], tj, c)};
                const bf8 la[3] = {row8<N>(sm.lam[0], ti, c), row8<N>(sm.lam[1], ti, c), row8<N>(sm.lam[2], ti, c)};
                const bf8 go = row8<N>(sm.go, ti, c), kj = row8<N>(sm.k, tj, c);
                const bf8 ri = row8<N>(sm.r, ti, c), ki = row8<N>(sm.k, ti, c);
                le = mma_step(0, la, e, le);
                ae = mfma32(go, e[2], ae);
                le = mma_step(1, la, e, le);
                ae = mfma32(go, e[1], ae);
                le = mma_step(2, la, e, le);
                ae = mfma32(go, e[0], ae);
                le = mma_step(3, la, e, le);
                rk = mfma32(ri, kj, rk);
                le = mma_step(4, la, e, le);
                kk = mfma32(ki, kj, kk);
                le = mma_step(5, la, e, le);
                __builtin_amdgcn_sched_barrier(0);
            }
            float mid = sm.suf[tj];
            for (int i = J + 1; i < I; ++i) mid += sm.total[i];
            float gap[4];
            if (I == J) {
                float run = 0.f;
                int lj = l16;
                asm volatile("" : "+v"(lj));  // else the comparisons are kept in registers for the whole kernel
#pragma unroll
                for (int l = 0; l < kSub; ++l) {
                    run += l > lj ? sm.w[kSub * I + l] : 0.f;
                    if (l / 4 == g) gap[l % 4] = run;
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) gap[q] = mid + sm.pre[kSub * I + 4 * g + q];
            }
            const float beta = sm.beta[tj];
            f4 p;
            float col = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int i = 4 * g + q;
                const float f = ex2(-gap[q]);
                da[n][q] = I > J || l16 <= i ? f * ae[q] : 0.f;
                dm[n][q] = I > J || l16 < i ? -f * le[q] : 0.f;
                p[q] = da[n][q] * rk[q] + dm[n][q] * kk[q];
                col += p[q];
            }
            const float all = sum_rows(col);
            if (g == 0) sm.colsum[id][l16] = all;
            da[n] *= beta;
            dm[n] *= beta;
            p *= beta;
            if (I > J) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float s = sum16(p[q]);
                    if (l16 == 0) sm.rowsum[id][4 * g + q] = s;
                }
            } else {  // pairs j < t <= i: sums over i >= t down the columns, then over j < t along the row
                const float down = beta * col;  // of this lane's four rows
                float below = 0.f;
#pragma unroll
                for (int o = 1; o < 4; ++o) {
                    const float x = __shfl(down, (lane + 16 * o) & 63, 64);
                    below += g + o < 4 ? x : 0.f;
                }
#pragma unroll
                for (int q = 3; q >= 0; --q) {
                    below += p[q];
                    const float s = sum16(l16 < 4 * g + q ? below : 0.f);
                    if (l16 == 0) sm.diag[kSub * I + 4 * g + q] = s;
                }
            }
        }

        __syncthreads();  // e and lambda are read; the sums are in place

        asm volatile("" : "+v"(lane), "+v"(l16), "+v"(g));
        __builtin_amdgcn_sched_barrier(0);
        // ---- dA, dM and their transposes as right operands
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int id = wv + (kGradWaves - 6) * n;
            if (n > 0 && wv < 6) continue;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const Terms x = split(w ? dm[n] : da[n]);
                *reinterpret_cast<bf8*>(sm.da[id][w][lane]) = pair(x.hi, x.mid);
                // the lane of row i, columns 4 (l16 / 4) ..: this lane's value is its number l16 % 4
                uint16_t* to = &sm.da[id][2 + w][16 * (l16 >> 2) + 4 * g][l16 & 3];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    to[8 * q] = static_cast<uint16_t>(x.hi[q / 2] >> (16 * (q & 1)));
                    to[8 * q + 4] = static_cast<uint16_t>(x.mid[q / 2] >> (16 * (q & 1)));
                }
            }
        }
        if (wv == 0) {  // dbeta and dw: token `lane`, of block g
            float sS = 0.f, sG = 0.f, total = 0.f, dbeta = 0.f, later = 0.f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                sS += sm.withS[i][lane];
                sG += sm.withG[i][lane];
                total += sm.inner[i];
            }
            const float beta = sm.beta[lane];
            // sums over the blocks (I, J): down the token's column, along its row, and of the whole blocks that
            // cross its own
            float rowv = sS, whole = 0.f;
#pragma unroll
            for (int I = 0; I < kWaves; ++I) {
#pragma unroll
                for (int J = 0; J <= I; ++J) {
                    const int id = I * (I + 1) / 2 + J;
                    const float c = sm.colsum[id][l16];
                    dbeta += J == g ? c : 0.f;
                    if (I == J) continue;
                    later += J == g ? c : 0.f;
                    const float r = sm.rowsum[id][l16];
                    rowv += I == g ? r : 0.f;
                    const float all = sum16(r);
                    whole += I > g && J < g ? all : 0.f;
                }
            }
            float colv = beta * (later + sG);
            const float rowS = sum16(sS), colG = sum16(beta * sG);
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                const float x = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(rowS), kSub * i));
                const float y = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(colG), kSub * i));
                whole += (i > g ? x : 0.f) + (i < g ? y : 0.f);
            }
            // rows of the block from the token on, columns before it, by shifts along the rows of 16 lanes
            rowv += dpp<0x101>(rowv);
            colv = dpp<0x111>(colv);
            rowv += dpp<0x102>(rowv);
            colv += dpp<0x111>(colv);
            rowv += dpp<0x104>(rowv);
            colv += dpp<0x112>(colv);
            rowv += dpp<0x108>(rowv);
            colv += dpp<0x114>(colv);
            colv += dpp<0x118>(colv);
            const float dw = fmaf(total, sm.since[kTile - 1], whole) + rowv + colv + sm.diag[lane];
            if (t0 + lane < len) {
                const int64_t to = (b * P.T + t0 + lane) * P.H + h;
                P.dbeta[to] = sG + dbeta;
                P.dw[to] = -dw;
            }
        }
        __syncthreads();
        asm volatile("" : "+v"(lane), "+v"(l16), "+v"(g));
        __builtin_amdgcn_sched_barrier(0);
        // ---- k and r times the blocks, for this wave's channels and tokens
#pragma unroll
        for (int X = 0; X < 4; ++X) {
            const bf8 kT = col_twice<N>(sm.k, kSub * X, c0, l16, g), rT = col_twice<N>(sm.r, kSub * X, c0, l16, g);
            const auto at = [&](int I, int J, int w) { return raw8(sm.da[I * (I + 1) / 2 + J][w][lane]); };
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                const int Y = X0 + x;
                if (X <= Y) {  // as j, for the rows of block Y
                    drT[x] = mfma32(kT, at(Y, X, 2), drT[x]);
                    dkT[x] = mfma32(kT, at(Y, X, 3), dkT[x]);
                }
                if (X >= Y) {  // as i, for the columns of block Y
                    dkT[x] = mfma32(rT, at(X, Y, 0), dkT[x]);
                    dkT[x] = mfma32(kT, at(X, Y, 1), dkT[x]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (next.pair != at.pair || next.tile != at.tile) {
            const int64_t ko = b * P.T * ks + at.hk * N;
#pragma unroll
            for (int x = 0; x < NX; ++x) {
                const int64_t t = t0 + kSub * (X0 + x) + l16;
                if (t < len) {
                    store4(static_cast<uint16_t*>(P.dr) + ko + t * ks + c0 + 4 * g, drT[x]);
                    store4(static_cast<uint16_t*>(P.dk) + ko + t * ks + c0 + 4 * g, dkT[x]);
                }
                drT[x] = dkT[x] = f4{0.f, 0.f, 0.f, 0.f};
            }
        }
        at = next;
    }
}

// ---- time split ---------------------------------------------------------------------------------
// A segment maps the state before it linearly: S -> M S + L.  Both are found by walking the segment
// without outputs, L from a zero state and M from the identity without values (its columns are 2 N
// independent ones, N / 8 waves).  Then the segments' start states follow one from the other, and all
// segments are walked at once.  The adjoint walk does the same from the other end.
//
// One workgroup per (pair, 16 columns); wave w owns rows 16 w .. of the product and the columns meet
// in LDS.  M_p and L_p are read before the state they act on is known: 2.2 us a segment at N = 128, latency.
template <int N>
__global__ void __launch_bounds__(4 * N) delta_chain_kernel(DeltaChainArgs P) {
    __shared__ float x[N][kSub + 1];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
    const int64_t bh = blockIdx.x % P.BH, col = blockIdx.x / P.BH * 16 + l16;
    const int row = 16 * wv + 4 * g;  // this lane's four rows
    f4 s;
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = P.first != nullptr ? P.first[(bh * N + row + q) * N + col] : 0.f;
    for (int64_t n = 0; n < P.nseg; ++n) {
        const int64_t seg = P.reverse ? P.nseg - 1 - n : n;
        float* to = P.starts + (bh * P.nseg + seg) * N * N;
#pragma unroll
        for (int q = 0; q < 4; ++q) to[(row + q) * N + col] = s[q];
        if (n == P.nseg - 1) break;
        const float* L = P.local + (bh * P.nseg + seg) * 2 * N * N;
        f4 next;
#pragma unroll
        for (int q = 0; q < 4; ++q) next[q] = L[(row + q) * N + col];
        if (n > 0) {  // the first segment's local end is its end
            const float* M = L + N * N + (16 * wv + l16) * N + 4 * g;
            f4 m[N / 16];
#pragma unroll
            for (int c = 0; c < N / 16; ++c) m[c] = load4(M + 16 * c);
            __syncthreads();
#pragma unroll
            for (int q = 0; q < 4; ++q) x[row + q][l16] = s[q];
            __syncthreads();
#pragma unroll
            for (int c = 0; c < N / 16; ++c) {
                f4 b;
#pragma unroll
                for (int q = 0; q < 4; ++q) b[q] = x[16 * c + 4 * g + q][l16];
                next = mma16(m[c], b, next);
            }
        }
        s = next;
    }
}

template <typename T, int N, bool kAdj, bool kOut>
hipError_t launch_walk(const WalkArgs& a, hipStream_t stream) {
    const int64_t groups = a.B * a.H * (a.local != nullptr ? 2 * (a.nseg - 1) : a.nseg);
    hipLaunchKernelGGL((delta_walk_kernel<T, N, kAdj, kOut>), dim3(static_cast<unsigned>(groups)), dim3(kWalkThreads<T, N>), 0,
                       stream, a);
    return hipGetLastError();
}

template <typename T, int N>
hipError_t launch_fwd(const DeltaArgs& a, hipStream_t stream) {
    if (a.states == nullptr && a.o != nullptr && a.T <= kDeltaStepMaxT) {
        const int64_t waves = a.B * a.H * (N / 64);
        hipLaunchKernelGGL((delta_step_kernel<T, N>), dim3(static_cast<unsigned>((waves + kWaves - 1) / kWaves)),
                           dim3(64 * kWaves), 0, stream, a);
        return hipGetLastError();
    }
    const WalkArgs w{a.B, a.T, a.H, a.HK, a.nseg, a.per, a.lengths, a.w, a.beta, a.r, a.k, a.v, a.o, a.s_in, a.starts, a.s_out,
                     a.local, a.errs, a.states};
    return a.o != nullptr ? launch_walk<T, N, false, true>(w, stream) : launch_walk<T, N, false, false>(w, stream);
}

template <typename T, int N>
hipError_t launch_bwd(const DeltaBwdArgs& a, hipStream_t stream) {
    const WalkArgs w{a.B, a.T, a.H, a.HK, a.nseg, a.per, a.lengths, a.w, a.beta, a.r, a.k, a.go, a.dv, a.ds_out, a.starts,
                     a.ds_in, a.local, a.lambda, a.gstates};
    if (a.local != nullptr) return launch_walk<T, N, true, false>(w, stream);  // what the segments do, for the chain
    hipError_t e = launch_walk<T, N, true, true>(w, stream);
    if (e != hipSuccess) return e;
    const int64_t ntile = (a.T + kTile - 1) / kTile;
    const dim3 grid(static_cast<unsigned>(a.B * a.HK * ntile));
    if constexpr (std::is_same_v<T, uint16_t>) {
        // as many workgroups as the card holds at once walk the tiles
        const unsigned most = 256 * kGradShare<N>;
        const dim3 some(grid.x < most ? grid.x : most);
        hipLaunchKernelGGL((delta_grad16_kernel<N>), some, dim3(kGradThreads), 0, stream, a);
    } else {
        hipLaunchKernelGGL((delta_grad_kernel<N>), grid, dim3(64 * kWaves), 0, stream, a);
    }
    return hipGetLastError();
}

}  // namespace

// Segments of a time split, by what the walks would take, in units of one tile of a workgroup alone on its
// compute unit (3.1 us at N = 64, 6.3 at N = 128; two at N = 64 share one in 1.9, at N = 128 only one fits).
// A split walks the segments twice, once without outputs (0.65 of a tile) for the state and for the identity,
// chains them (0.3 each) and launches two kernels more (2.5; 1.3 of float32's tiles, which take twice as long).
// Measured whole and split, bf16:
//   8192 tokens, N = 64:  8 pairs 387 and 71 us, 64 pairs 391 and 245, 128 pairs 403 and 367
//   8192 tokens, N = 128: 64 pairs 805 and 522, 128 pairs 808 and 746
//   1024 tokens, N = 64:  64 pairs 54 and 48, 128 pairs 56 and 59 (not split);  training 213 and 218 (not split)
//   1024 tokens, N = 128, training: 128 pairs 462 and 497 (not split)
//   512 tokens, N = 64:   4 pairs 30 and 25
// float32: 512 tokens, N = 64, 4 pairs 48 and 32, 64 pairs 50 and 47;  N = 128, 16 pairs 150 and 80;  333 tokens,
// N = 64, 16 pairs, training 111 and 100
int64_t delta_segments(int64_t BH, int64_t T, int64_t N, bool bf16, int64_t* per) {
    const int64_t tiles = (T + kTile - 1) / kTile;
    const auto walk = [&](int64_t groups) {
        if (N != 64) return static_cast<double>((groups + 255) / 256);
        const int64_t rest = groups % 512;
        return 1.9 * static_cast<double>(groups / 512) + (rest == 0 ? 0.0 : rest <= 256 ? 1.0 : 1.9);
    };
    *per = tiles;
    int64_t nseg = 1;
    if (BH < 1 || BH > 512) return nseg;
    const double more = bf16 ? 2.5 : 1.3;
    double best = walk(BH) * static_cast<double>(tiles);
    for (int64_t n = 2; n <= 64 && 2 * n <= tiles; ++n) {
        const int64_t p = (tiles + n - 1) / n;
        if ((tiles + p - 1) / p != n) continue;
        const double t = static_cast<double>(p) * (0.65 * walk(2 * BH * (n - 1)) + walk(BH * n)) + 0.3 * static_cast<double>(n) + more;
        if (t < best) {
            best = t;
            nseg = n;
            *per = p;
        }
    }
    return nseg;
}

hipError_t launch_delta_chain(const DeltaChainArgs& a, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(a.BH * (a.N / 16)));
    if (a.N == 64) {
        hipLaunchKernelGGL(delta_chain_kernel<64>, grid, dim3(256), 0, stream, a);
    } else {
        hipLaunchKernelGGL(delta_chain_kernel<128>, grid, dim3(512), 0, stream, a);
    }
    return hipGetLastError();
}

hipError_t launch_delta_fwd(const DeltaArgs& a, hipStream_t stream) {
    if (a.bf16) return a.N == 64 ? launch_fwd<uint16_t, 64>(a, stream) : launch_fwd<uint16_t, 128>(a, stream);
    return a.N == 64 ? launch_fwd<float, 64>(a, stream) : launch_fwd<float, 128>(a, stream);
}

hipError_t launch_delta_bwd(const DeltaBwdArgs& a, hipStream_t stream) {
    if (a.bf16) return a.N == 64 ? launch_bwd<uint16_t, 64>(a, stream) : launch_bwd<uint16_t, 128>(a, stream);
    return a.N == 64 ? launch_bwd<float, 64>(a, stream) : launch_bwd<float, 128>(a, stream);
}

}  // namespace wkv
