// Internal interface of the token embedding, the gated projection and the
// vocabulary's cross entropy, between the C ABI and their kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <hip/hip_runtime.h>

namespace gscan {

// Rows of a table by token, and the table's gradient.
struct EmbedArgs {
    const void *table = nullptr;   // forward: [V][D], rows ld apart
    const void *tokens = nullptr;  // [N], int32 or int64; outside 0 .. V - 1: padding
    void *out = nullptr;           // forward: [N][D]
    const void *dout = nullptr;    // backward: [N][D], rows ld apart
    void *dtable = nullptr;        // backward: [V][D]
    int64_t N = 0, V = 0, ld = 0;
    int D = 0;
    int tok64 = 0, table_dtype = 0, dtype = 0;  // dtype: of out and dout
    float scale = 1.f;
    void *ws = nullptr;
};
size_t embed_workspace_bytes(int64_t N, int64_t V, int D);
hipError_t launch_embed_forward(const EmbedArgs &a, hipStream_t stream);
hipError_t launch_embed_backward(const EmbedArgs &a, hipStream_t stream);

// act(x Wg^T) * (x Wu^T) and its gradients.
struct GateArgs {
    const void *x = nullptr;       // [N][D], rows ldx apart
    const void *wg = nullptr, *wu = nullptr;  // [F][D], rows ldg, ldu apart
    const void *dout = nullptr;    // backward: [N][F], rows ldd apart
    void *out = nullptr;           // forward: [N][F]
    void *dx = nullptr;            // backward: [N][D] (null: not wanted)
    void *dwg = nullptr, *dwu = nullptr;  // backward: [F][D] (both null: not wanted)
    int64_t N = 0, ldx = 0, ldg = 0, ldu = 0, ldd = 0;
    int D = 0, F = 0;
    int dtype = 0, act = 0;
    void *ws = nullptr;            // parts of tiles; backward: gradients of both products, [N][2 F]
};
size_t gate_workspace_bytes(const GateArgs &a, bool backward);
hipError_t launch_gate_forward(const GateArgs &a, hipStream_t stream);
hipError_t launch_gate_backward(const GateArgs &a, hipStream_t stream);

// Cross entropy of softmax(scale * h W^T).
struct XentArgs {
    const void *h = nullptr;       // [N][D], rows ldh apart
    const void *w = nullptr;       // [V][D], rows ldw apart
    const void *target = nullptr;  // [N], int32 or int64; outside 0 .. V - 1: not counted
    float *loss = nullptr;         // forward: [N], or [1]
    float *lse = nullptr;          // [N] (forward: written, backward: read)
    const float *dloss = nullptr;  // backward: [N] or [1]
    void *dh = nullptr, *dw = nullptr;  // backward (null: not wanted); dense
    int64_t N = 0, V = 0, ldh = 0, ldw = 0;
    int D = 0;
    int dtype = 0, target64 = 0, reduction = 0;  // 0 none, 1 sum, 2 mean
    float scale = 1.f;
    void *ws = nullptr;
};
size_t xent_forward_workspace_bytes(int64_t N, int64_t V, int D, int dtype);
size_t xent_backward_workspace_bytes(int64_t N, int64_t V, int D, int dtype);
hipError_t launch_xent_forward(const XentArgs &a, hipStream_t stream);
hipError_t launch_xent_backward(const XentArgs &a, hipStream_t stream);

}  // namespace gscan
