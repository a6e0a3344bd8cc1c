// Internal interface of the matrix-state scan, its single-token step and the
// query/key norm with rotation, between the C ABI and their kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <hip/hip_runtime.h>

namespace gscan {

// Element strides of a [batch][token][head][width] operand (packed: batch 0);
// the width is contiguous.  Tokens and heads are less than 2^31 apart.
struct Strides {
    int64_t b = 0;
    uint32_t t = 0, h = 0;
};

// What the scan's kernels take by value.
struct StateArgs {
    const void *q = nullptr, *k = nullptr, *v = nullptr, *gate = nullptr, *dout = nullptr;
    Strides qs, ks, vs, gs, ds;
    const int32_t *off = nullptr;  // packed: first token of each sequence (B + 1 values)
    const float *s0 = nullptr;     // initial state [B][H][Dk][Dv] (null: zero)
    const float *dsT = nullptr;    // gradient of the final state (null: zero)
    void *out = nullptr;           // [tokens][H][Dv]
    float *sT = nullptr;           // final state (null: not written)
    void *dq = nullptr, *dk = nullptr, *dv = nullptr, *dgate = nullptr;
    float *ds0 = nullptr;          // gradient of the initial state (null: not written)
    void *ws = nullptr;
    int64_t B = 0, T = 0;          // packed: T is the number of tokens of all sequences
    int64_t chunks = 0;            // chunk slots there are (StatePlan)
    int H = 0, Hk = 0, Dk = 0, Dv = 0;
    int dtype = 0, gate_dtype = 0, gate_form = 0;
    float gate_shift = 0.f, scale = 1.f;
};

// Decomposition of a call (pure host arithmetic).
struct StatePlan {
    int chunk = 64;           // tokens per chunk: 64 (bf16) or 32 (fp32)
    int nk = 2, nv = 2;       // 32-wide units of the padded widths: 2 or 4
    int64_t per = 0;          // tokens per unit (a sequence, or a part of one)
    int64_t units = 0;        // units over all sequences (an upper bound when packed)
    bool split = false;       // some sequence may have several units
    size_t st_part = 0, st_dec = 0;  // workspace: what the units add to the state, their decays
    size_t st_part_r = 0, st_dec_r = 0;  // backward: the same of the state's gradient
    int64_t chunks = 0;       // chunk slots over all sequences (an upper bound when packed)
    size_t st_s = 0, st_ds = 0;  // workspace: the backward's chunk states and their gradients
    size_t down = 0;          // bf16: the powers of two of their column tiles
    size_t bytes = 0;
};

StatePlan make_state_plan(const StateArgs &a, bool backward);
hipError_t launch_state_forward(const StatePlan &p, const StateArgs &a, hipStream_t stream);
hipError_t launch_state_backward(const StatePlan &p, const StateArgs &a, hipStream_t stream);

// One token per request over a pool of states.
struct StepArgs {
    const void *q = nullptr, *k = nullptr, *v = nullptr, *gate = nullptr;
    int64_t qn = 0, qh = 0, kn = 0, kh = 0, vn = 0, vh = 0, gn = 0, gh = 0;  // request, head strides
    float *state = nullptr;        // [pool][H][Dk][Dv]
    const int32_t *slots = nullptr;
    void *out = nullptr;           // [N][H][Dv]
    int64_t N = 0, pool = 0;
    int H = 0, Hk = 0, Dk = 0, Dv = 0;
    int dtype = 0, gate_dtype = 0, gate_form = 0;
    float gate_shift = 0.f, scale = 1.f;
};
hipError_t launch_state_step(const StepArgs &a, hipStream_t stream);

// Per-head RMS norm of queries and keys with the position rotation.
struct NormArgs {
    const void *x[2] = {nullptr, nullptr};       // q, k
    const void *dy[2] = {nullptr, nullptr};      // backward: upstream gradients
    int64_t xn[2] = {0, 0}, xh[2] = {0, 0};      // token, head strides of x
    int64_t dn[2] = {0, 0}, dh[2] = {0, 0};      // token, head strides of dy
    const float *w[2] = {nullptr, nullptr};      // [D], null: ones
    void *y[2] = {nullptr, nullptr};             // forward: y, backward: dx; dense
    float *dw[2] = {nullptr, nullptr};
    const void *pos = nullptr;                   // [tokens], int32 or int64
    int pos64 = 0;
    const float *freq = nullptr;                 // [rot / 2]
    int64_t tokens = 0;
    int heads[2] = {0, 0};
    int D = 0, rot = 0, layout = 0, dtype = 0;
    float eps = 0.f, magnitude = 1.f;
    void *ws = nullptr;
};
size_t norm_workspace_bytes(int64_t tokens, int heads, int D);
hipError_t launch_norm_forward(const NormArgs &a, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs &a, hipStream_t stream);

}  // namespace gscan
