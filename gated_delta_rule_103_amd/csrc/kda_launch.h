// kda_launch.h -- host-side launchers implemented in the .hip files and
// called by the argument-checking layer in kda_abi.cpp. Every launcher
// assumes its arguments were already validated and returns a hipError_t.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

enum class Dt : int { F32 = 0, BF16 = 1 };

struct PrefillArgs {
    const void *q, *k, *v;
    const float *g;
    const void *beta;
    const float *S0;
    void *out;
    float *S_out;
    const int32_t *cu_seqlens;  // device, or nullptr (dense)
    int N, B, T, H, Dk, Dv, C;
    Dt io, beta_dt, out_dt;
    void *ws;
    size_t ws_bytes;
    hipStream_t stream;
    // optional state snapshots: [N][H][max_snaps][Dv][Dk] fp32, one every
    // snap_every chunks of each sequence (nullptr: none)
    float *snaps = nullptr;
    int snap_every = 0, max_snaps = 0;
    // gate layout: false: g [T_total][H][Dk], one log-decay per key channel (KDA);
    // true: g [T_total][H], one per head broadcast over the channels (Gated
    // DeltaNet), and g == nullptr means no decay (DeltaNet)
    bool g_head = false;
    // L2-normalise q and k over Dk inside the kernels: x / sqrt(sum x^2 + norm_eps)
    bool qk_norm = false;
    float norm_eps = 0.f;
    // run everything on `stream` (no side stream or events created), as for
    // callers that must not create runtime objects (the no-allocation entry)
    bool in_order = false;
};

struct DecodeArgs {
    const void *q, *k, *v;
    const float *g;
    const void *beta;
    float *S;
    void *out;
    int N, H, Dk, Dv;
    Dt io, beta_dt, out_dt;
    hipStream_t stream;
    bool g_head = false;        // as in PrefillArgs: g [N][H] or nullptr
    bool qk_norm = false;       // as in PrefillArgs
    float norm_eps = 0.f;
};

struct OutputGateArgs {
    const void *o, *gate;
    const float *weight;        // [Dv] or nullptr (ones)
    void *out;
    int rows, H, Dv;
    float eps;
    Dt o_dt, gate_dt, out_dt;
    hipStream_t stream;
};

struct RecurrentArgs {
    const void *q, *k, *v;
    const float *g;
    const void *beta;
    float *S;                   // [slots][H][Dv][Dk]
    void *out;
    const int32_t *cu;          // [N + 1], device
    const int32_t *slot_in;     // [N], device, or nullptr (zero states)
    const int32_t *slot_out;    // [T], device, or nullptr (no state is kept)
    int N, T, H, Dk, Dv, slots;
    Dt io, beta_dt, out_dt;
    hipStream_t stream;
    bool g_head = false;        // as in PrefillArgs
    bool qk_norm = false;
    float norm_eps = 0.f;
    bool zero_rows = false;     // out rows of no sequence become zero
};

struct PrefillBackwardArgs {
    const void *q, *k, *v;
    const float *g;
    const void *beta;
    const void *dout;
    const float *S0, *dS_out;   // or nullptr (zero)
    void *dq, *dk, *dv;
    float *dg;                  // or nullptr (no gate)
    void *dbeta;
    float *dS0;                 // or nullptr (not wanted)
    const int32_t *cu_seqlens;  // device, or nullptr (dense)
    int N, B, T, H, Dk, Dv;
    Dt io, beta_dt, dout_dt;
    void *ws;
    hipStream_t stream;
    bool g_head = false;        // as in PrefillArgs
    bool qk_norm = false;
    float norm_eps = 0.f;
    int zero_rows = 0;          // KDA_ZERO_*: gradients whose rows of no sequence become zero
};

struct OutputGateBackwardArgs {
    const void *o, *gate, *dout;
    const float *weight;        // [Dv] or nullptr (ones)
    void *do_, *dgate;
    float *dweight;             // [Dv] or nullptr (not wanted)
    int rows, H, Dv;
    float eps;
    Dt o_dt, gate_dt, dout_dt;
    float *ws;
    hipStream_t stream;
};

struct LayerNormArgs {
    const void *x;
    const float *weight, *bias; // [W] or nullptr
    void *out;
    float *mean, *rstd;         // [rows] or nullptr (not wanted)
    int rows, W;
    float eps;
    bool rms;                   // no mean is taken
    Dt x_dt, out_dt;
    hipStream_t stream;
};

struct LayerNormBackwardArgs {
    const void *x, *dy;
    const float *mean, *rstd, *weight;
    void *dx;
    float *dweight, *dbias;     // [W] or nullptr (not wanted)
    int rows, W;
    bool rms;
    Dt x_dt, dy_dt;
    float *ws;
    hipStream_t stream;
};

struct LinPrefillArgs {
    const void *q, *k, *v;      // q, k of Hk heads, v of H
    const float *g;             // [T_total][H], fixed: [H]; nullptr: no decay
    const float *S0;            // or nullptr (zero)
    void *out;
    float *S_out;               // or nullptr (not wanted)
    const int32_t *cu_seqlens;  // device, or nullptr (dense)
    int N, B, T, H, Hk, Dk, Dv;
    Dt io, out_dt;
    bool fixed, zero_rows;
    void *ws;
    hipStream_t stream;
};

struct LinBackwardArgs {
    const void *q, *k, *v;
    const float *g;
    const void *dout;
    const float *S0, *dS_out;   // or nullptr (zero)
    void *dq, *dk, *dv;
    float *dg, *dS0;            // dg nullptr when g is; dS0 or nullptr (not wanted)
    const int32_t *cu_seqlens;
    int N, B, T, H, Hk, Dk, Dv;
    Dt io;
    bool fixed;
    int zero_rows;              // KDA_ZERO_*
    void *ws;
    hipStream_t stream;
};

struct LinRecurrentArgs {
    const void *q, *k, *v;
    const float *g;
    float *S;                   // [slots][H][Dv][Dk]
    void *out;
    const int32_t *cu;          // [N + 1], device; nullptr: one token per sequence, sequence n in slot n
    const int32_t *slot_in;     // [N], device, or nullptr (zero states)
    const int32_t *slot_out;    // [T], device, or nullptr (no state is kept)
    int N, T, H, Hk, Dk, Dv, slots;
    Dt io, out_dt;
    bool fixed, zero_rows;
    hipStream_t stream;
};

struct TreeArgs {
    const void *q, *k, *v;      // [N][T][Hk or H][D]
    const float *g;
    const void *beta;           // or nullptr: no delta rule
    float *S;                   // [slots][H][Dv][Dk]
    void *out;                  // [N][T][H][Dv]
    const int32_t *slot_in;     // [N] or nullptr (zero states)
    const int32_t *slot_out;    // [N], accept only
    const int32_t *parent;      // [N][T]
    const int32_t *node;        // [N], accept only
    int N, T, H, Hk, Dk, Dv, slots;
    Dt io, beta_dt, out_dt;
    int gate;                   // kda_gate
    bool qk_norm;
    float norm_eps;
    bool zero_rows;
    hipStream_t stream;
};

struct SlotsCopyArgs {
    const char *from;
    char *to;
    const int32_t *src, *dst;
    int n, layers, from_slots, to_slots;
    size_t slot_bytes;
    hipStream_t stream;
};

struct SlotsCompactArgs {
    char *pool;
    int32_t *uses, *count;
    int32_t *table;             // entries naming slots, or nullptr
    int slots, layers, table_n;
    size_t slot_bytes;
    int32_t *moved;             // workspace: [slots] new place of each slot, then the moves
    hipStream_t stream;
};

// Upper bound on the number of chunks of all sequences (each sequence adds at
// most one partial chunk).
inline long long max_chunks(int N, long long T_total, int C) {
    return (T_total + C - 1) / C + N;
}

// Device-side chunk table of packed sequences: chunk_off[n] for n <= N.
hipError_t launch_chunk_plan(const int32_t *cu, int N, int C, int32_t *chunk_off, hipStream_t stream);

// fp32-arithmetic chunked prefill (plan + prep + scan kernels).
size_t prefill_f32_workspace(int N, long long T_total, int H, int Dk, int Dv, int C);
hipError_t launch_prefill_f32(const PrefillArgs &a);

// MFMA chunked prefill for bf16 inputs (fp16 and fp32 MFMA, fp32 accumulation).
size_t prefill_mfma_workspace(int N, long long T_total, int H, int Dk, int Dv, int C);
hipError_t launch_prefill_mfma(const PrefillArgs &a);

// kda_prefill_noalloc: the size of its fixed device workspace, and the address
// of that workspace on the current device (looked up once per device).
constexpr size_t kNoAllocScratchBytes = size_t(128) << 20;
hipError_t noalloc_scratch(void **ptr);

// single-token decode.
hipError_t launch_decode(const DecodeArgs &a);

// per-head RMS norm and sigmoid output gate of o.
hipError_t launch_output_gate(const OutputGateArgs &a);

// several tokens per sequence through the recurrence, states in a slot pool.
bool recurrent_fits(int N, int H, int Dk);   // a launch has fewer than 2^32 threads
hipError_t launch_recurrent(const RecurrentArgs &a);

// the chunked form's gradient (fp32 arithmetic). fits: whether the launches
// stay within the runtime's limits.
size_t prefill_backward_workspace(int N, long long T_total, int H, int Dk);
bool prefill_backward_fits(int N, long long T_total, int H, int Dk);
hipError_t launch_prefill_backward(const PrefillBackwardArgs &a);

// the output gate's gradient.
size_t output_gate_backward_workspace(long long rowheads, int Dv);
hipError_t launch_output_gate_backward(const OutputGateBackwardArgs &a);

// linear attention with a decay per head: chunked, its gradient, and the recurrent form.
size_t lin_prefill_workspace(int N, long long T_total, int H, int Dk, int Dv);
size_t lin_backward_workspace(int N, long long T_total, int H, int Hk, int Dk, int Dv);
bool lin_chunk_fits(int N, long long T_total, int H);
hipError_t launch_lin_prefill(const LinPrefillArgs &a);
hipError_t launch_lin_backward(const LinBackwardArgs &a);
bool lin_recurrent_fits(int N, int H, int Dk, int Dv);
hipError_t launch_lin_recurrent(const LinRecurrentArgs &a);

// trees of drafted tokens over a state each, and the state behind an accepted node.
constexpr int kMaxTreeNodes = 64;
bool tree_fits(int N, int H);
hipError_t launch_tree(const TreeArgs &a);
hipError_t launch_tree_accept(const TreeArgs &a);

// the slots of a state pool. fits: the launch stays within the runtime's limits.
bool slots_copy_fits(long long n, int layers, size_t slot_bytes);
bool slots_compact_fits(int slots, size_t slot_bytes);
hipError_t launch_slots_copy(const SlotsCopyArgs &a);
hipError_t launch_slots_count(int32_t *uses, const int32_t *which, int n, int slots, int add, hipStream_t stream);
hipError_t launch_slots_acquire(int32_t *uses, int slots, int32_t *taken, int n, hipStream_t stream);
hipError_t launch_slots_compact(const SlotsCompactArgs &a);

// layer norm and RMS norm of rows of at most kMaxNormWidth channels, and the gradient.
constexpr int kMaxNormWidth = 16384;
hipError_t launch_layer_norm(const LayerNormArgs &a);
size_t layer_norm_backward_workspace(int rows, int W);
hipError_t launch_layer_norm_backward(const LayerNormBackwardArgs &a);

}  // namespace kda
