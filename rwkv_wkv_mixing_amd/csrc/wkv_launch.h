// Host-side launch interface between the C ABI (wkv_api.hip) and the kernel
// translation units.  Internal to the library; not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace wkv {

constexpr int64_t kCkptLen = 16;  // = WKV_CKPT_LEN in include/wkv.h

// Polls a wait for a carry between workgroups makes before it gives up and
// flags the workspace's error word (wkv_debug_spin_limit sets it; default 2^22).
uint32_t spin_limit();

// Header at the start of a wkv_forward / wkv_backward workspace (the device
// code's CallHdr in wkv_scan.h has this layout).
struct CallHdrLayout {
    uint32_t unused0, error, streams_done, gen;
};

struct FwdArgs {
    int64_t B, T, C;
    bool bf16;
    const float* w;
    const float* u;
    const void* k;
    const void* v;
    float* y;
    void* ckpt;     // nullable
    int64_t nblk;   // ceil(T / kCkptLen)
    void* ws;
    size_t ws_bytes;
    // optional receptance [B, T, C] (in dtype): y becomes sigmoid(r) y
    const void* r = nullptr;
    // optional state before token 1 and after token T, each [B, C] (a, b, p as
    // wkv_step): all three pointers NULL or all set
    const float* a_in = nullptr;
    const float* b_in = nullptr;
    const float* p_in = nullptr;
    float* a_out = nullptr;
    float* b_out = nullptr;
    float* p_out = nullptr;
};

struct BwdArgs {
    int64_t B, T, C;
    bool bf16;
    const float* w;
    const float* u;
    const void* k;
    const void* v;
    const void* gy;
    float* dk;
    float* dv;
    float* dw;
    float* du;
    const void* ckpt;  // nullable
    int64_t nblk;
    void* ws;
    size_t ws_bytes;
    // optional receptance [B, T, C] (in dtype): gy is then the gradient of
    // sigmoid(r) y, and dr [B, T, C] float32 receives the gradient of r
    const void* r = nullptr;
    float* dr = nullptr;
    // optional, through carried state ([B, C] each; each triple all NULL or all set): the state before
    // token 1 (as FwdArgs), the gradient (ga, gb) of the state after token T at the p the forward
    // wrote, and the gradients (ga, gb, gp) of the state before token 1 (needs a_in)
    const float* a_in = nullptr;
    const float* b_in = nullptr;
    const float* p_in = nullptr;
    const float* ga_out = nullptr;
    const float* gb_out = nullptr;
    const float* p_out = nullptr;
    float* ga_in = nullptr;
    float* gb_in = nullptr;
    float* gp_in = nullptr;
};

struct StepArgs {
    int64_t L, B, C;
    bool bf16;
    bool vec4;
    const float* w;
    const float* u;
    const void* k;
    const void* v;
    float* y;
    float* a;
    float* b;
    float* p;
};

struct ShiftArgs {
    int64_t B, T, C, M;
    bool bf16;
    bool vec;              // 16-byte vectors: C a multiple of 16 / element size, pointers 16-byte aligned
    const float* mu;       // [M, C]
    const void* x;         // [B, T, C]
    const void* x_prev;    // [B, C] or NULL (zeros)
    void* out;             // forward: [M, B, T, C], dtype of x
    const void* g;         // backward: [M, B, T, C], dtype of x
    float* dx;             // backward: [B, T, C]
    float* dmu;            // backward: [M, C]
    float* dx_prev;        // backward: [B, C] or NULL
    float* ws;             // backward: shift_partial_rows(B, T) * M * C floats
};

struct Wkv5Args {
    int64_t B, T, H;     // head size 64; C = 64 H
    const float* w;      // [H, 64] decay rates
    const float* u;      // [H, 64] bonus
    const uint16_t* r;   // [B, T, C] bf16, 16-byte aligned
    const uint16_t* k;
    const uint16_t* v;
    float* o;            // [B, T, C]
    const float* s_in;   // [B, H, 64, 64] or NULL (zero state)
    float* s_out;        // [B, H, 64, 64] or NULL
    uint16_t* ckpt = nullptr;  // [B, H, nchunks, 64, 64] bf16 [key][value]: the state before each chunk, or NULL
    // time split: nseg > 1 runs segment s of (batch row, head) bh as workgroup bh * nseg + s over
    // chunks [s cps, (s + 1) cps), with s_in / s_out then [B * H, nseg, 64, 64] (the segments' own
    // start and end states); the saved states keep their global chunk index
    int64_t nseg = 1, cps = 0;
    float* seg_rates = nullptr;  // RWKV-6 only: [B * H, nseg, 64] each segment's summed capped rates (log2 e units)
};

// The segments' start states from their local end states (time split), and the final state.
struct SegChainArgs {
    int64_t BH, H, T, nseg, cps;
    const float* w5;         // RWKV-5: [H, 64] rates, or NULL
    const float* rates6;     // RWKV-6: [BH, nseg, 64] summed capped rates (log2 e units), or NULL
    const float* s_in;       // [BH, 64, 64] or NULL (zero)
    const float* loc;        // [BH, nseg, 64, 64] each segment's end state from the zero state
    float* start;            // [BH, nseg, 64, 64] each segment's start state
    float* s_out;            // [BH, 64, 64] or NULL
    int reverse = 0;         // 1: the backwards' adjoint chain, last segment first (start = the adjoint after it)
};

hipError_t launch_seg_chain(const SegChainArgs& a, hipStream_t stream);

// time split of the matrix-state backwards: every segment's adjoint before it from a zero adjoint
// after it (and, per token rates, the segment's summed capped rates in log2 e units)
struct AdjLocalArgs {
    int64_t B, T, H, nseg, cps;
    const float* w;          // RWKV-5: [H, 64]; RWKV-6: [B, T, C] per-token rates
    bool per_token;          // RWKV-6
    const uint16_t* r;
    const uint16_t* go;
    float* loc;              // [BH, nseg, 64, 64]
    float* rates;            // [BH, nseg, 64] (per_token only)
};

hipError_t launch_adj_local(const AdjLocalArgs& a, hipStream_t stream);
// segments for a time split of B * H (batch row, head) pairs over T tokens (1: no split); the
// forwards split below 256 pairs, the backwards up to 256
int64_t wkv56_segments(int64_t BH, int64_t T, int64_t* cps, int64_t max_bh = 255);

struct Wkv5BwdArgs {
    int64_t B, T, H;
    const float* w;
    const float* u;
    const uint16_t* r;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* go;     // [B, T, C] bf16 gradient of o
    const uint16_t* ckpt;   // as Wkv5Args::ckpt
    const float* ds_out;    // [B, H, 64, 64] gradient of the final state, or NULL (zero)
    float* dr;              // [B, T, C]
    float* dk;
    float* dv;
    float* part;            // [nseg, B, H, 2, 64]: dw, du of each (segment, batch row, head)
    float* dw;              // [H, 64], summed over batch rows
    float* du;
    float* ds_in;           // [B, H, 64, 64] gradient of the initial state, or NULL
    int64_t nseg = 1, cps = 0;      // time split: segments per sequence, chunks per segment
    const float* gstart = nullptr;  // nseg > 1: [B H, nseg, 64, 64] the adjoint after each segment
};

// chunked forward (wkv_fwd.hip)
hipError_t launch_fwd_chunk(const FwdArgs& a, hipStream_t stream);
// T == 0 with a state: the output state is the input state (or the empty one)
hipError_t launch_state_passthrough(const FwdArgs& a, hipStream_t stream);
size_t fwd_chunk_workspace_bytes(int64_t B, int64_t T, int64_t C);

// chunked backward (wkv_bwd.hip)
hipError_t launch_bwd_chunk(const BwdArgs& a, hipStream_t stream);
size_t bwd_chunk_workspace_bytes(int64_t B, int64_t T, int64_t C);

// token-shift mix (wkv_shift.hip)
hipError_t launch_shift_fwd(const ShiftArgs& a, hipStream_t stream);
hipError_t launch_shift_bwd(const ShiftArgs& a, hipStream_t stream);
hipError_t launch_shift_zero(float* p, int64_t n, hipStream_t stream);
int64_t shift_partial_rows(int64_t B, int64_t T);
int shift_vector_width(bool bf16, bool bwd);

// RWKV-5 matrix-state forward (wkv5.hip)
hipError_t launch_wkv5_fwd(const Wkv5Args& a, hipStream_t stream);

struct Wkv6Args {
    int64_t B, T, H;     // head size 64; C = 64 H
    const float* w;      // [B, T, C] per-token decay rates (>= 0)
    const float* u;      // [H, 64] bonus
    const uint16_t* r;   // [B, T, C] bf16, 16-byte aligned
    const uint16_t* k;
    const uint16_t* v;
    float* o;            // [B, T, C]
    const float* s_in;   // [B, H, 64, 64] or NULL (zero state)
    float* s_out;        // [B, H, 64, 64] or NULL
    uint16_t* ckpt = nullptr;  // as Wkv5Args::ckpt
    int64_t nseg = 1, cps = 0;   // as Wkv5Args
    float* seg_rates = nullptr;
};

hipError_t launch_wkv6_fwd(const Wkv6Args& a, hipStream_t stream);

struct Wkv6BwdArgs {
    int64_t B, T, H;
    const float* w;         // [B, T, C] per-token rates
    const float* u;
    const uint16_t* r;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* go;     // [B, T, C] bf16 gradient of o
    const uint16_t* ckpt;   // as Wkv6Args::ckpt
    const float* ds_out;    // [B, H, 64, 64] gradient of the final state, or NULL (zero)
    float* dr;              // [B, T, C]
    float* dk;
    float* dv;
    float* dw;              // [B, T, C], per token
    float* part;            // [nseg, B, H, 64]: du of each (segment, batch row, head)
    float* du;              // [H, 64]
    float* ds_in;           // [B, H, 64, 64] or NULL
    int64_t nseg = 1, cps = 0;      // as Wkv5BwdArgs
    const float* gstart = nullptr;
};

hipError_t launch_wkv6_bwd(const Wkv6BwdArgs& a, hipStream_t stream);
hipError_t launch_wkv5_state_copy(const float* s_in, float* s_out, int64_t n, hipStream_t stream);
hipError_t launch_wkv5_bwd(const Wkv5BwdArgs& a, hipStream_t stream);

// Up to this many tokens without saved states the delta rule runs token by token (delta_step_kernel).
constexpr int64_t kDeltaStepMaxT = 16;

struct DeltaArgs {
    int64_t B, T, H, HK, N;   // H value heads of N channels share HK key heads
    bool bf16;
    const int32_t* lengths;   // [B] tokens of each row, or NULL (T)
    const float* w;           // [B, T, H] decay rates
    const float* beta;        // [B, T, H] write strengths
    const void* r;            // [B, T, HK N]
    const void* k;
    const void* v;            // [B, T, H N]
    void* o;                  // [B, T, H N] or NULL (a pass for the saved states only)
    const float* s_in;        // [B, H, N, N] or NULL (zero state)
    float* s_out;             // [B, H, N, N] or NULL
    float* errs;              // [B, T, H, N] the errors e_t, or NULL
    float* states;            // [B, H, ceil(T / 64), N, N] the state before every 64 tokens, or NULL
    // time split: nseg > 1 segments of `per` 64-token tiles a sequence, each by workgroups of its own
    int64_t nseg = 1, per = 0;
    const float* starts = nullptr;  // [B H, nseg, N, N] the segments' start states, in place of s_in
    float* local = nullptr;         // [B H, nseg, 2, N, N]: a pass for what each segment but the last does to a state:
                                    // its end state from zero (the first segment: from s_in), and the end states
                                    // from the columns of the identity without its values
};

struct DeltaBwdArgs {
    int64_t B, T, H, HK, N;
    bool bf16;
    const int32_t* lengths;
    const float* w;
    const float* beta;
    const void* r;
    const void* k;
    const void* go;           // [B, T, H N] gradient of o
    const float* errs;        // as DeltaArgs
    const float* states;
    const float* ds_out;      // [B, H, N, N] or NULL (zero)
    float* lambda;            // scratch [B, T, H, N]
    float* gstates;           // scratch [B, H, ceil(T / 64), N, N]
    void* dr;                 // [B, T, HK N]
    void* dk;
    void* dv;                 // [B, T, H N]
    float* dw;                // [B, T, H]
    float* dbeta;
    float* ds_in;             // [B, H, N, N] or NULL
    // time split, as DeltaArgs, from the last segment: starts holds the gradients of the states after the
    // segments, local those before each segment but the first
    int64_t nseg = 1, per = 0;
    const float* starts = nullptr;
    float* local = nullptr;
};

// The states at the segments' starts from what the segments do (DeltaArgs::local): x_0 = first,
// x_1 = its local end, x_{p+1} = M_p x_p + L_p; reverse: the same from the last segment.
struct DeltaChainArgs {
    int64_t BH, N, nseg;
    bool reverse;
    const float* first;  // [B H, N, N] or NULL (zero)
    const float* local;
    float* starts;
};

hipError_t launch_delta_chain(const DeltaChainArgs& a, hipStream_t stream);
// segments for a time split of BH pairs over T tokens (1: no split), *per 64-token tiles each
int64_t delta_segments(int64_t BH, int64_t T, int64_t N, bool bf16, int64_t* per);

// gated delta rule (wkv_delta.hip)
hipError_t launch_delta_fwd(const DeltaArgs& a, hipStream_t stream);
hipError_t launch_delta_bwd(const DeltaBwdArgs& a, hipStream_t stream);

enum { kActNone = 0, kActSigmoid = 1, kActSilu = 2 };  // = WKV_ACT_* in include/wkv.h

struct HeadNormArgs {
    int64_t rows, H, G;
    bool y_bf16, bf16;        // dtype of y, dy; of gate, gout, out, dgate
    bool center, shared;      // mean taken off; weight and bias [G] for all heads
    bool vec;                 // 16-byte vectors: G a multiple of 8, pointers 16-byte aligned
    int act;
    float eps;
    const void* y;            // [rows, H G]
    const float* weight;      // [H G] or [G]
    const float* bias;        // or NULL
    const void* gate;         // [rows, H G] or NULL
    void* out = nullptr;
    // backward
    const void* gout = nullptr;
    void* dy = nullptr;
    void* dgate = nullptr;
    float* dweight = nullptr;
    float* dbias = nullptr;
    float* ws = nullptr;      // 2 head_norm_chunks(rows, H G) H G floats (rows H and G when shared)
    int lanes = 0, hpb = 0;   // lanes a head, heads a workgroup (set by the launch)
    int64_t chunks = 0;
};

struct BlockNormArgs {
    int64_t rows, C;
    bool x_bf16, bf16;        // dtype of x, x_out, gx, dx; of y, gate, h and their gradients
    bool center, vec;
    int act;
    float eps;
    const void* x;            // [rows, C]; backward: the forward's x_out
    const void* y;
    const void* gate;         // or NULL
    const float* post_w;      // [C] or NULL (y as it is)
    const float* post_b;      // or NULL
    const float* scale;       // or NULL (1)
    const float* pre_w;
    const float* pre_b;       // or NULL
    void* x_out = nullptr;
    void* h = nullptr;
    // backward
    const void* gx = nullptr; // or NULL (zero)
    const void* gh = nullptr;
    void* dx = nullptr;
    void* dy = nullptr;
    void* dgate = nullptr;
    float* dpre_w = nullptr;
    float* dpre_b = nullptr;
    float* dpost_w = nullptr;
    float* dpost_b = nullptr;
    float* dscale = nullptr;
    float* ws = nullptr;      // 5 block_norm_slots(rows, C) C floats
    int threads = 0;          // that hold a row (set by the launch)
    int64_t slots = 0;
};

// norms (wkv_norm.hip)
hipError_t launch_head_norm(const HeadNormArgs& a, hipStream_t stream);
hipError_t launch_head_norm_bwd(const HeadNormArgs& a, hipStream_t stream);
hipError_t launch_block_norm(const BlockNormArgs& a, hipStream_t stream);
hipError_t launch_block_norm_bwd(const BlockNormArgs& a, hipStream_t stream);
hipError_t launch_zero(float* p, int64_t n, hipStream_t stream);  // p may be NULL
int64_t head_norm_chunks(int64_t rows, int64_t C);
int64_t block_norm_slots(int64_t rows, int64_t C);

struct ConvArgs {
    int64_t B, T, C, K;       // K taps, 2 to 4
    bool bf16, vec;           // vec: vectors of 4 elements (C a multiple of 4, pointers aligned to them)
    int act;
    const int32_t* lengths;   // [B] tokens of each row, or NULL (T)
    const void* x;            // [B, T, C]
    const float* weight;      // [K, C]
    const float* bias;        // [C] or NULL
    const void* s_in;         // [B, K - 1, C] the inputs before token 1, or NULL (zeros)
    void* out = nullptr;      // [B, T, C]
    void* s_out = nullptr;    // [B, K - 1, C] or NULL; may be s_in
    // backward
    const void* gout = nullptr;    // [B, T, C]
    const void* ds_out = nullptr;  // [B, K - 1, C] or NULL
    void* dx = nullptr;            // [B, T, C]
    float* dweight = nullptr;      // [K, C]
    float* dbias = nullptr;        // [C], with bias
    void* ds_in = nullptr;         // [B, K - 1, C] or NULL
    float* part = nullptr;         // [slots, K + 1, C]
    int64_t slots = 0;             // = conv_slots(B, T, C)
};

// short causal convolution (wkv_conv.hip)
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t stream);
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t stream);
hipError_t launch_conv_copy(const void* from, void* to, int64_t n, bool bf16, hipStream_t stream);  // from NULL: zeros
int64_t conv_slots(int64_t B, int64_t T, int64_t C);

// Gradient norm and clipping (wkv_clip.hip): a launch takes up to kClipTensors tensors, by value.
constexpr int kClipTensors = 96;
struct ClipTable {
    const void* in[kClipTensors];
    void* out[kClipTensors];          // unused for the norm alone
    int64_t n[kClipTensors];          // elements
    int64_t chunk0[kClipTensors];     // number of the tensor's first chunk in this launch
    uint8_t bf16[kClipTensors];
    int count;
    int64_t chunks;                   // of all the tensors
};
// workgroups of a launch at most, and partial sums it writes (1.4 GB of gradients: 512 848 us, 1024 747, 2048 795)
constexpr int64_t kClipBlocks = 1024;
constexpr int64_t kClipChunk = 16384;  // elements (8192 as fast, 32768 781 us)
constexpr int64_t kClipCached = int64_t{200} << 20;  // bytes that stay in the last level cache (256 MB) with something to spare
// partial sums of squares: one a workgroup, from part on; their number
int64_t clip_blocks(const ClipTable& t);
hipError_t launch_clip_sums(const ClipTable& t, double* part, hipStream_t stream);
// nparts partial sums to one, behind them, when there are too many for every workgroup to add up
hipError_t launch_clip_norm(const double* part, int64_t nparts, float* norm, double* total, hipStream_t stream);
hipError_t launch_clip_scale(const ClipTable& t, const double* part, int64_t nparts, float max_norm, float eps, float* norm,
                             bool past_cache, hipStream_t stream);  // past_cache: the outputs are written past the caches

constexpr int kSelectTile = 16;  // tokens between saved states of the selective scan
// Up to this many tokens without saved states it runs token by token (select_step_kernel; against the walk, N = 16 bf16,
// 64 rows of 4096 channels: 4 tokens 13.6 us for 33.3, 8 21.2 for 31.6, 12 29 for 32.5, 16 36.5 for 30.8; 4 rows of 768:
// 4 tokens 4.6 us for 5.6, 8 5.9 for 5.5, 16 8.8 for 5.5).
constexpr int64_t kSelectStepMaxT = 8;

struct SelectArgs {
    int64_t B, T, C, G, N;    // channels in G groups that share b and c; N states a channel
    bool bf16, softplus;
    const int32_t* lengths;   // [B] tokens of each row, or NULL (T)
    const void* x;            // [B, T, C]
    const void* dt;           // [B, T, C]
    const float* w;           // [C, N] decay rates
    const void* b;            // [B, T, G N]
    const void* c;
    const float* d;           // [C] or NULL
    const void* z;            // [B, T, C] or NULL (no gate)
    const float* dt_bias;     // [C] or NULL
    const float* s_in;        // [B, C, N] or NULL (zero state)
    int64_t tiles = 0;        // ceil(T / kSelectTile)
    int ctiles = 0;           // tiles of 64 channels: G ceil(C / G / 64)
    int64_t nseg = 1, seg_len = 0;  // time split: segments of seg_len tokens (a multiple of kSelectTile)
    float* local = nullptr;   // [nseg, B, C, N] what the segments do to a state of zero, then their start states
    float* steps = nullptr;   // [nseg, B, C] the segments' sums of delta
    // forward
    void* out = nullptr;      // [B, T, C]
    float* s_out = nullptr;   // [B, C, N] or NULL
    float* ckpt = nullptr;    // [B, tiles, N / 4, C, 4] the state before every kSelectTile tokens, or NULL
    // backward
    const float* saved = nullptr;  // the forward's ckpt
    const void* go = nullptr;      // [B, T, C]
    const float* ds_out = nullptr; // [B, C, N] or NULL
    void* dx = nullptr;
    void* ddt = nullptr;
    float* dw = nullptr;           // [C, N]
    void* db = nullptr;
    void* dc = nullptr;
    float* dd = nullptr;           // [C], with d
    void* dz = nullptr;            // with z
    float* ddt_bias = nullptr;     // [C], with dt_bias
    float* ds_in = nullptr;        // [B, C, N] or NULL
    float* part = nullptr;         // [ctiles, B, T, 2 N] sums over a tile's channels for db and dc
    float* dw_part = nullptr;      // [nseg, B, C, N]
    float* vec_part = nullptr;     // [nseg, B, C, 2] for dd and ddt_bias
};

// selective scan (wkv_select.hip)
hipError_t launch_select_step(const SelectArgs& a, hipStream_t stream);
hipError_t launch_select_fwd(const SelectArgs& a, hipStream_t stream);
hipError_t launch_select_bwd(const SelectArgs& a, hipStream_t stream);
// segments for a time split (1: no split), *per tokens each
int64_t select_segments(int64_t B, int64_t T, int64_t ctiles, int64_t N, bool bwd, int64_t* per);

// decode step (wkv_step.hip)
hipError_t launch_step(const StepArgs& s, hipStream_t stream);

}  // namespace wkv
