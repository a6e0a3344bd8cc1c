// C ABI of the gated temporal scan (declared in include/gscan.h).
//
// Every call validates all arguments before enqueueing anything (the
// validate-then-launch order of the Kimi-K3 KDA decode launcher page, whose
// entry point checks every length before its first allocation or launch),
// returns a status code instead of aborting, and records a detail string in
// thread-local storage.
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "gscan.h"
#include "gscan_internal.h"
#include "gscan_state.h"
#include "gscan_lm.h"

namespace {

thread_local char g_last_error[512] = "";

int fail(int status, const char *fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return status;
}

bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// hipGetLastError() returns and resets the calling thread's most recent HIP
// error, whichever call raised it.  Each entry point clears it once its
// arguments have passed validation and before it enqueues anything, so the
// checks after its own launches report only its own failures.
void clear_stale_error()
{
    (void)hipGetLastError();
}

int check_common(const void *hh, const void *hs2, const float *WA, const float *WB,
                 const float *WC, int64_t B, int64_t K, int64_t SH2, int64_t D, int dtype,
                 gscan::Plan *plan)
{
    if (!hh || !hs2 || !WA || !WB || !WC)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null input pointer");
    if (B <= 0 || K <= 0 || SH2 <= 0 || D <= 0)
        return fail(GSCAN_ERR_INVALID_ARGUMENT,
                    "sizes must be positive (B=%lld K=%lld SH2=%lld D=%lld)", (long long)B,
                    (long long)K, (long long)SH2, (long long)D);
    if (dtype != GSCAN_F32 && dtype != GSCAN_BF16)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "unknown input dtype %d", dtype);
    if (!gscan::make_plan(B, K, SH2, D, dtype, plan))
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE,
                    "unsupported shape B=%lld K=%lld SH2=%lld D=%lld (need 16<=SH2<=1024, "
                    "SH2%%16==0, 16<=D<=256, D%%16==0)",
                    (long long)B, (long long)K, (long long)SH2, (long long)D);
    if (!aligned16(hh) || !aligned16(hs2) || !aligned16(WA) || !aligned16(WB) || !aligned16(WC))
        return fail(GSCAN_ERR_MISALIGNED, "input pointers must be 16-byte aligned");
    return GSCAN_OK;
}

int check_backward(const void *h_history, const void *h_s2, const float *W_A, const float *W_B,
                   const float *W_C, int64_t B, int64_t K, int64_t SH2, int64_t D,
                   const float *d_context, int dtype, gscan::Plan *plan)
{
    int st = check_common(h_history, h_s2, W_A, W_B, W_C, B, K, SH2, D, dtype, plan);
    if (st != GSCAN_OK) return st;
    if (!d_context) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null d_context");
    if (!aligned16(d_context))
        return fail(GSCAN_ERR_MISALIGNED, "d_context must be 16-byte aligned");
    return GSCAN_OK;
}

int check_outputs(const float *dW_A, const float *dW_B, const float *dW_C)
{
    if (!dW_A || !dW_B || !dW_C) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null dW pointer");
    if (!aligned16(dW_A) || !aligned16(dW_B) || !aligned16(dW_C))
        return fail(GSCAN_ERR_MISALIGNED, "dW pointers must be 16-byte aligned");
    return GSCAN_OK;
}

// Workspace of the backward with input gradients: the partials, then
// dL/dA | dL/dB per row and dL/dC per sample (each 256-byte aligned).
struct FullLayout {
    size_t dab = 0, dc = 0, bytes = 0;
};

FullLayout full_layout(const gscan::Plan &p)
{
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    FullLayout f;
    if (p.fused_dinput()) {  // phase 1 writes the input gradients: partials only
        f.dab = f.dc = 0;
        f.bytes = p.ws_bytes;
        return f;
    }
    if (p.bwd_split || p.generic) {  // the workspace already holds both
        f.dab = p.split_dab;
        f.dc = p.split_dc;
        f.bytes = p.ws_bytes;
        return f;
    }
    f.dab = up(p.ws_bytes);
    f.dc = up(f.dab + (size_t)(p.B * p.K) * (size_t)(2 * p.D) * sizeof(float));
    f.bytes = f.dc + (size_t)p.B * (size_t)p.D * sizeof(float);
    return f;
}

int check_workspace(const void *workspace, size_t workspace_bytes, const gscan::Plan &plan)
{
    if (!workspace) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null workspace");
    if (workspace_bytes < plan.ws_bytes)
        return fail(GSCAN_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < required %zu",
                    workspace_bytes, plan.ws_bytes);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(GSCAN_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    return GSCAN_OK;
}

// ------------------------------------------- static scratch (no allocation)
// The weight-gradient partials of gscan_backward_noalloc live in this
// file-scope device array instead of caller or runtime memory.  Its host-side
// name is only a stand-in: host code uses the device address that
// hipGetSymbolAddress returns, looked up once per device (with that device
// current) and kept.  Each device holds its own copy for the life of the
// process.
static __device__ __align__(256) unsigned char scratch[GSCAN_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices] = {};

// The current device's copy of `scratch`.
int current_scratch(void **out)
{
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess)
        return fail(GSCAN_ERR_HIP, "hipGetDevice failed: %s", hipGetErrorString(e));
    if (dev < 0 || dev >= kMaxDevices)
        return fail(GSCAN_ERR_HIP, "device index %d outside 0..%d", dev, kMaxDevices - 1);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void *p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess || !p)
            return fail(GSCAN_ERR_HIP, "hipGetSymbolAddress(scratch) failed on device %d: %s",
                        dev, hipGetErrorString(e));
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return GSCAN_OK;
}

// A caller's forward workspace, checked only where the plan uses one.
int check_forward_workspace(const void *workspace, size_t workspace_bytes,
                            const gscan::Plan &plan)
{
    if (!plan.fwd_scratch || !workspace) return GSCAN_OK;
    if (workspace_bytes < plan.fwd_scratch)
        return fail(GSCAN_ERR_WORKSPACE_TOO_SMALL, "forward workspace %zu bytes < required %zu",
                    workspace_bytes, plan.fwd_scratch);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return fail(GSCAN_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    return GSCAN_OK;
}

// The forward with the scratch its plan asks for (the materialised
// projections of the shapes outside the fused kernels): the caller's
// workspace, or memory from the stream-ordered allocator released on the
// same stream.
int run_forward(const gscan::Plan &plan, const void *hh, const void *hs2, const float *WA,
                const float *WB, const float *WC, float a_shift, const gscan::CtxOut &out,
                void *workspace, hipStream_t stream)
{
    if (plan.fwd_scratch && workspace) {
        hipError_t e = gscan::launch_forward(plan, hh, hs2, WA, WB, WC, a_shift, out, workspace,
                                             stream);
        if (e != hipSuccess)
            return fail(GSCAN_ERR_HIP, "forward launch failed: %s", hipGetErrorString(e));
        return GSCAN_OK;
    }
    void *sc = nullptr;
    if (plan.fwd_scratch) {
        hipError_t e = hipMallocAsync(&sc, plan.fwd_scratch, stream);
        if (e != hipSuccess)
            return fail(GSCAN_ERR_HIP, "forward scratch allocation (%zu bytes) failed: %s",
                        plan.fwd_scratch, hipGetErrorString(e));
    }
    hipError_t e = gscan::launch_forward(plan, hh, hs2, WA, WB, WC, a_shift, out, sc, stream);
    if (sc) {
        hipError_t f = hipFreeAsync(sc, stream);
        if (e == hipSuccess) e = f;
    }
    if (e != hipSuccess)
        return fail(GSCAN_ERR_HIP, "forward launch failed: %s", hipGetErrorString(e));
    return GSCAN_OK;
}


// ------------------------------------------- matrix-state scan, norm, rotation

int esize(int dtype) { return dtype == GSCAN_BF16 ? 2 : 4; }

bool known(int dtype) { return dtype == GSCAN_F32 || dtype == GSCAN_BF16; }

bool strides16(const int64_t *s, int n, int dtype)
{
    for (int i = 0; i < n; ++i)
        if (s[i] * esize(dtype) % 16 != 0) return false;
    return true;
}

constexpr int64_t kMaxTokens = 2147483647 - 128;
constexpr int64_t kMaxGrid = 2147483647;
constexpr int64_t kMaxHeads = 16384;        // a chunk's outputs stay below 2 GiB
constexpr int64_t kMaxNormHeads = 1 << 20;
constexpr int64_t kMaxStride = 1 << 23;     // and so do a chunk's rows of an operand

// Sizes, types and strides of a scan (and of a step, which is a scan of one
// token each).
int check_state_desc(const gscan_state_scan_t *d, bool backward, gscan::StateArgs *a)
{
    if (!d) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null descriptor");
    if (!known(d->dtype) || !known(d->gate_dtype))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "unknown dtype %d / %d", (int)d->dtype,
                    (int)d->gate_dtype);
    if (d->gate_form != GSCAN_GATE_SIGMOID && d->gate_form != GSCAN_GATE_LOG)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "unknown gate form %d", (int)d->gate_form);
    if (d->B < 1 || d->T < 0 || d->H < 1 || d->Hk < 1 || d->Dk < 1 || d->Dv < 1)
        return fail(GSCAN_ERR_INVALID_ARGUMENT,
                    "need B, H, Hk, Dk, Dv >= 1 and T >= 0 (B=%lld T=%lld H=%lld Hk=%lld Dk=%lld "
                    "Dv=%lld)", (long long)d->B, (long long)d->T, (long long)d->H,
                    (long long)d->Hk, (long long)d->Dk, (long long)d->Dv);
    if (d->Dk % 8 || d->Dv % 8 || d->Dk > 128 || d->Dv > 128 || d->H % d->Hk || d->H > kMaxHeads ||
        d->B > kMaxTokens || d->T > kMaxTokens)
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE,
                    "unsupported shape B=%lld T=%lld H=%lld Hk=%lld Dk=%lld Dv=%lld (need Dk and "
                    "Dv multiples of 8 up to 128, Hk dividing H <= 16384, B and T below 2^31 - 128)",
                    (long long)d->B, (long long)d->T, (long long)d->H, (long long)d->Hk,
                    (long long)d->Dk, (long long)d->Dv);
    if (!strides16(d->q_stride, 3, d->dtype) || !strides16(d->k_stride, 3, d->dtype) ||
        !strides16(d->v_stride, 3, d->dtype) ||
        (backward && !strides16(d->d_out_stride, 3, d->dtype)))
        return fail(GSCAN_ERR_MISALIGNED, "strides of q, k, v, d_out must be multiples of 16 bytes");
    auto far = [](const int64_t *s) {
        return s[0] < 0 || s[1] < 0 || s[1] >= kMaxStride || s[2] < 0 || s[2] > 2147483647;
    };
    if (far(d->q_stride) || far(d->k_stride) || far(d->v_stride) || far(d->gate_stride) ||
        (backward && far(d->d_out_stride)))
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE,
                    "strides must not be negative, token strides below 2^23, head strides below 2^31");
    auto st = [&](const int64_t *s) {
        return gscan::Strides{d->seq_offsets ? 0 : s[0], (uint32_t)s[1], (uint32_t)s[2]};
    };
    a->qs = st(d->q_stride);
    a->ks = st(d->k_stride);
    a->vs = st(d->v_stride);
    a->gs = st(d->gate_stride);
    if (backward) a->ds = st(d->d_out_stride);
    a->off = d->seq_offsets;
    a->B = d->B;
    a->T = d->T;
    a->H = (int)d->H;
    a->Hk = (int)d->Hk;
    a->Dk = (int)d->Dk;
    a->Dv = (int)d->Dv;
    a->dtype = d->dtype;
    a->gate_dtype = d->gate_dtype;
    a->gate_form = d->gate_form;
    a->gate_shift = d->gate_shift;
    a->scale = d->scale;
    return GSCAN_OK;
}

// The decomposition, refused where a launch or an index would not fit.
int state_plan(const gscan::StateArgs &a, bool backward, gscan::StatePlan *p)
{
    const int64_t nc = a.T / 32 + 1;  // at least the chunks of a sequence
    const int64_t slots = a.off ? nc + a.B : nc > kMaxGrid / a.B ? kMaxGrid : nc * a.B;
    // eight workgroups at most per chunk and head in any launch
    if (slots > kMaxGrid / 8 / a.H)
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE, "too many chunks times heads (B=%lld T=%lld H=%d)",
                    (long long)a.B, (long long)a.T, a.H);
    *p = gscan::make_state_plan(a, backward);
    return GSCAN_OK;
}

bool mis(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

int check_state_inputs(const gscan::StateArgs &a)
{
    // without tokens there is nothing to read
    if (a.T > 0 && (!a.q || !a.k || !a.v || !a.gate))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null q, k, v or gate");
    if (mis(a.q, 16) || mis(a.k, 16) || mis(a.v, 16) || mis(a.s0, 16) ||
        mis(a.gate, (uintptr_t)esize(a.gate_dtype)) || mis(a.off, 4))
        return fail(GSCAN_ERR_MISALIGNED, "q, k, v and states must be 16-byte aligned, the gate "
                    "and seq_offsets aligned to their elements");
    return GSCAN_OK;
}

// Runs `go(workspace)` with the caller's workspace or stream-ordered memory.
template <class F>
int with_workspace(const char *what, void *ws, size_t ws_bytes, size_t need, hipStream_t stream, F go)
{
    if (need && ws) {
        if (ws_bytes < need)
            return fail(GSCAN_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < required %zu", ws_bytes,
                        need);
        if (mis(ws, 256)) return fail(GSCAN_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    }
    clear_stale_error();
    void *own = nullptr;
    if (need && !ws) {
        hipError_t e = hipMallocAsync(&own, need, stream);
        if (e != hipSuccess)
            return fail(GSCAN_ERR_HIP, "%s workspace allocation (%zu bytes) failed: %s", what, need,
                        hipGetErrorString(e));
    }
    hipError_t e = go(own ? own : ws);
    if (own) {
        hipError_t f = hipFreeAsync(own, stream);
        if (e == hipSuccess) e = f;
    }
    if (e != hipSuccess) return fail(GSCAN_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
    g_last_error[0] = '\0';
    return GSCAN_OK;
}

constexpr int64_t kMaxWidth = 65536;        // of the embedding and what follows
constexpr int64_t kMaxRowStride = 1 << 21;  // 256 of its rows stay below 2 GiB

int check_embed(const gscan_embed_t *d, const void *tokens, gscan::EmbedArgs *a, bool pointers = true)
{
    if (!d) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null descriptor");
    if (!known(d->table_dtype) || !known(d->dtype))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "unknown dtype %d / %d", (int)d->table_dtype, (int)d->dtype);
    if (d->tokens < 0 || d->vocabulary < 1 || d->width < 1 || d->stride < 0)
        return fail(GSCAN_ERR_INVALID_ARGUMENT,
                    "need tokens, stride >= 0 and vocabulary, width >= 1 (tokens=%lld vocabulary=%lld "
                    "width=%lld stride=%lld)", (long long)d->tokens, (long long)d->vocabulary,
                    (long long)d->width, (long long)d->stride);
    if (d->width % 8 || d->width > kMaxWidth || d->tokens > kMaxTokens || d->vocabulary > kMaxTokens ||
        d->stride > (int64_t(1) << 31) || d->vocabulary > (int64_t(1) << 40) / d->width)
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE,
                    "unsupported shape tokens=%lld vocabulary=%lld width=%lld (need a width that is a "
                    "multiple of 8 up to 65536, tokens and vocabulary below 2^31 - 128, a table of at most "
                    "2^40 elements)", (long long)d->tokens, (long long)d->vocabulary, (long long)d->width);
    if (pointers && d->tokens > 0 && !tokens) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null tokens");
    if (mis(tokens, d->token_int64 ? 8 : 4)) return fail(GSCAN_ERR_MISALIGNED, "misaligned tokens");
    a->tokens = tokens;
    a->N = d->tokens;
    a->V = d->vocabulary;
    a->D = (int)d->width;
    a->ld = d->stride;
    a->tok64 = d->token_int64 != 0;
    a->table_dtype = (int)d->table_dtype;
    a->dtype = (int)d->dtype;
    a->scale = d->scale;
    return GSCAN_OK;
}

constexpr int64_t kMaxProducts = int64_t(1) << 43;  // rows times columns of an output: 2^30 tiles

int check_gate(const gscan_gated_projection_t *d, const void *x, const void *wg, const void *wu,
               gscan::GateArgs *a, bool pointers = true)
{
    if (!d) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null descriptor");
    if (!known(d->dtype)) return fail(GSCAN_ERR_INVALID_ARGUMENT, "unknown dtype %d", (int)d->dtype);
    if (d->activation != GSCAN_ACT_SILU && d->activation != GSCAN_ACT_GELU &&
        d->activation != GSCAN_ACT_GELU_TANH)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "unknown activation %d", (int)d->activation);
    if (d->tokens < 0 || d->width < 1 || d->inner < 1)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "need tokens >= 0 and width, inner >= 1 (tokens=%lld width=%lld "
                    "inner=%lld)", (long long)d->tokens, (long long)d->width, (long long)d->inner);
    if (d->width % 8 || d->inner % 8 || d->width > kMaxWidth || d->inner > kMaxWidth || d->tokens > kMaxTokens ||
        d->tokens > kMaxProducts / (2 * (d->width > d->inner ? d->width : d->inner)))
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE,
                    "unsupported shape tokens=%lld width=%lld inner=%lld (need widths that are multiples of 8 "
                    "up to 65536, tokens below 2^31 - 128, tokens times the larger width at most 2^42)",
                    (long long)d->tokens, (long long)d->width, (long long)d->inner);
    for (int64_t s : {d->x_stride, d->gate_stride, d->up_stride}) {
        if (s < 0 || s > kMaxRowStride)
            return fail(GSCAN_ERR_UNSUPPORTED_SHAPE, "row strides must be 0 .. 2^21 elements");
        if (!strides16(&s, 1, d->dtype))
            return fail(GSCAN_ERR_MISALIGNED, "row strides must be multiples of 16 bytes");
    }
    if (pointers && (!wg || !wu || (d->tokens > 0 && !x)))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null x or weight");
    if (mis(x, 16) || mis(wg, 16) || mis(wu, 16))
        return fail(GSCAN_ERR_MISALIGNED, "x and the weights must be 16-byte aligned");
    a->x = x;
    a->wg = wg;
    a->wu = wu;
    a->N = d->tokens;
    a->D = (int)d->width;
    a->F = (int)d->inner;
    a->ldx = d->x_stride;
    a->ldg = d->gate_stride;
    a->ldu = d->up_stride;
    a->dtype = (int)d->dtype;
    a->act = (int)d->activation;
    return GSCAN_OK;
}

int check_xent(const gscan_linear_cross_entropy_t *d, const void *h, const void *w, const void *target,
               gscan::XentArgs *a, bool pointers = true)
{
    if (!d) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null descriptor");
    if (!known(d->dtype)) return fail(GSCAN_ERR_INVALID_ARGUMENT, "unknown dtype %d", (int)d->dtype);
    if (d->reduction != GSCAN_LOSS_EACH && d->reduction != GSCAN_LOSS_SUM && d->reduction != GSCAN_LOSS_MEAN)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "unknown reduction %d", (int)d->reduction);
    if (d->tokens < 0 || d->width < 1 || d->vocabulary < 1)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "need tokens >= 0 and width, vocabulary >= 1 (tokens=%lld "
                    "width=%lld vocabulary=%lld)", (long long)d->tokens, (long long)d->width,
                    (long long)d->vocabulary);
    if (d->width % 8 || d->width > kMaxWidth || d->tokens > kMaxTokens || d->vocabulary > kMaxTokens ||
        d->vocabulary > (int64_t(1) << 40) / d->width ||
        d->tokens > kMaxProducts / (d->width > d->vocabulary ? d->width : d->vocabulary))
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE,
                    "unsupported shape tokens=%lld width=%lld vocabulary=%lld (need a width that is a multiple of "
                    "8 up to 65536, tokens and vocabulary below 2^31 - 128, vocabulary * width at most 2^40, "
                    "tokens times the larger of both at most 2^43)", (long long)d->tokens, (long long)d->width,
                    (long long)d->vocabulary);
    for (int64_t s : {d->h_stride, d->weight_stride}) {
        if (s < 0 || s > kMaxRowStride)
            return fail(GSCAN_ERR_UNSUPPORTED_SHAPE, "row strides must be 0 .. 2^21 elements");
        if (!strides16(&s, 1, d->dtype))
            return fail(GSCAN_ERR_MISALIGNED, "row strides must be multiples of 16 bytes");
    }
    if (pointers && (!w || (d->tokens > 0 && (!h || !target))))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null h, weight or target");
    if (mis(h, 16) || mis(w, 16) || mis(target, d->target_int64 ? 8 : 4))
        return fail(GSCAN_ERR_MISALIGNED, "h and weight must be 16-byte aligned, targets to their elements");
    a->h = h;
    a->w = w;
    a->target = target;
    a->N = d->tokens;
    a->V = d->vocabulary;
    a->D = (int)d->width;
    a->ldh = d->h_stride;
    a->ldw = d->weight_stride;
    a->dtype = (int)d->dtype;
    a->target64 = d->target_int64 != 0;
    a->reduction = (int)d->reduction;
    a->scale = d->scale;
    return GSCAN_OK;
}

int check_norm(const gscan_qk_norm_t *d, const void *q, const void *k, const float *wq,
               const float *wk, const void *pos, const float *freq, gscan::NormArgs *a)
{
    if (!d) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null descriptor");
    if (!known(d->dtype)) return fail(GSCAN_ERR_INVALID_ARGUMENT, "unknown dtype %d", (int)d->dtype);
    if (d->layout != GSCAN_ROTATE_HALF && d->layout != GSCAN_ROTATE_INTERLEAVED)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "unknown rotation layout %d", (int)d->layout);
    if (d->tokens < 0 || d->Hq < 1 || d->Hk < 0 || d->D < 1 || d->rot < 0 || !(d->eps > 0.f))
        return fail(GSCAN_ERR_INVALID_ARGUMENT,
                    "need tokens, Hk, rot >= 0, Hq, D >= 1, eps > 0 (tokens=%lld Hq=%lld Hk=%lld "
                    "D=%lld rot=%lld eps=%g)", (long long)d->tokens, (long long)d->Hq,
                    (long long)d->Hk, (long long)d->D, (long long)d->rot, (double)d->eps);
    if (d->D % 8 || d->D > 256 || d->rot % 8 || d->rot > d->D || d->Hq > kMaxNormHeads ||
        d->Hk > kMaxNormHeads || d->tokens > kMaxTokens)
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE,
                    "unsupported shape tokens=%lld Hq=%lld Hk=%lld D=%lld rot=%lld (need D a "
                    "multiple of 8 up to 256, rot a multiple of 8 up to D, at most 2^20 heads)",
                    (long long)d->tokens, (long long)d->Hq, (long long)d->Hk, (long long)d->D,
                    (long long)d->rot);
    if (d->tokens > 0 && (!q || (d->Hk > 0 && !k)))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null q or k");
    if (d->tokens > 0 && d->rot > 0 && (!pos || !freq))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null positions or freq");
    if (mis(q, 16) || mis(k, 16) || mis(wq, 16) || mis(wk, 16) || mis(pos, d->pos_int64 ? 8 : 4) ||
        mis(freq, 4) || !strides16(d->q_stride, 2, d->dtype) ||
        (d->Hk > 0 && !strides16(d->k_stride, 2, d->dtype)))
        return fail(GSCAN_ERR_MISALIGNED, "q, k, weights and the strides of q, k must be multiples of "
                    "16 bytes, positions and freq aligned to their elements");
    a->x[0] = q;
    a->x[1] = k;
    a->w[0] = wq;
    a->w[1] = wk;
    a->xn[0] = d->q_stride[0];
    a->xh[0] = d->q_stride[1];
    a->xn[1] = d->k_stride[0];
    a->xh[1] = d->k_stride[1];
    a->pos = pos;
    a->pos64 = d->pos_int64;
    a->freq = freq;
    a->tokens = d->tokens;
    a->heads[0] = (int)d->Hq;
    a->heads[1] = (int)d->Hk;
    a->D = (int)d->D;
    a->rot = (int)d->rot;
    a->layout = d->layout;
    a->dtype = d->dtype;
    a->eps = d->eps;
    a->magnitude = d->magnitude;
    return GSCAN_OK;
}

}  // namespace

extern "C" {

int gscan_forward_ex(const void *h_history, const void *h_s2, const float *W_A, const float *W_B,
                     const float *W_C, int64_t B, int64_t K, int64_t SH2, int64_t D,
                     float *context_out, gscan_dtype_t in_dtype, float a_shift,
                     void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    gscan::Plan plan;
    int st = check_common(h_history, h_s2, W_A, W_B, W_C, B, K, SH2, D, (int)in_dtype, &plan);
    if (st != GSCAN_OK) return st;
    if (!context_out) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null context_out");
    if (!aligned16(context_out))
        return fail(GSCAN_ERR_MISALIGNED, "context_out must be 16-byte aligned");
    if ((st = check_forward_workspace(workspace, workspace_bytes, plan)) != GSCAN_OK) return st;
    clear_stale_error();
    gscan::CtxOut out;
    out.ctx = context_out;
    st = run_forward(plan, h_history, h_s2, W_A, W_B, W_C, a_shift, out, workspace, stream);
    if (st != GSCAN_OK) return st;
    g_last_error[0] = '\0';
    return GSCAN_OK;
}

int gscan_forward_enrich(const void *h_history, const void *h_s2, const float *W_A,
                         const float *W_B, const float *W_C, int64_t B, int64_t K, int64_t SH2,
                         int64_t D, float *context_out, float *h_enriched, int64_t ld_enriched,
                         int64_t col_offset, gscan_dtype_t in_dtype, float a_shift,
                         void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    gscan::Plan plan;
    int st = check_common(h_history, h_s2, W_A, W_B, W_C, B, K, SH2, D, (int)in_dtype, &plan);
    if (st != GSCAN_OK) return st;
    if (!h_enriched) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null h_enriched");
    if (ld_enriched < D || col_offset < 0 || col_offset > ld_enriched - D)
        return fail(GSCAN_ERR_INVALID_ARGUMENT,
                    "need ld_enriched >= D and 0 <= col_offset <= ld_enriched - D (ld=%lld "
                    "offset=%lld D=%lld)",
                    (long long)ld_enriched, (long long)col_offset, (long long)D);
    if (ld_enriched > (int64_t(1) << 40) / B)
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE, "B x ld_enriched above 2^40");
    if ((reinterpret_cast<uintptr_t>(h_enriched) & 3u) != 0)
        return fail(GSCAN_ERR_MISALIGNED, "h_enriched must be 4-byte aligned");
    if (context_out) {
        if (!aligned16(context_out))
            return fail(GSCAN_ERR_MISALIGNED, "context_out must be 16-byte aligned");
        // the two outputs must not overlap (each element has one writer)
        const uintptr_t c0 = reinterpret_cast<uintptr_t>(context_out);
        const uintptr_t c1 = c0 + (uintptr_t)(B * D) * sizeof(float);
        const uintptr_t e0 = reinterpret_cast<uintptr_t>(h_enriched);
        const uintptr_t e1 = e0 + (uintptr_t)((B - 1) * ld_enriched + col_offset + D) * sizeof(float);
        if (c0 < e1 && e0 < c1)
            return fail(GSCAN_ERR_INVALID_ARGUMENT, "context_out overlaps h_enriched");
    }
    if ((st = check_forward_workspace(workspace, workspace_bytes, plan)) != GSCAN_OK) return st;
    clear_stale_error();
    gscan::CtxOut out;
    out.ctx = context_out;
    out.enr = h_enriched + col_offset;
    out.ld = ld_enriched;
    st = run_forward(plan, h_history, h_s2, W_A, W_B, W_C, a_shift, out, workspace, stream);
    if (st != GSCAN_OK) return st;
    g_last_error[0] = '\0';
    return GSCAN_OK;
}

int gscan_forward(const void *h_history, const void *h_s2, const float *W_A, const float *W_B,
                  const float *W_C, int64_t B, int64_t K, int64_t SH2, int64_t D,
                  float *context_out, hipStream_t stream)
{
    return gscan_forward_ex(h_history, h_s2, W_A, W_B, W_C, B, K, SH2, D, context_out, GSCAN_F32,
                            0.0f, nullptr, 0, stream);
}

size_t gscan_forward_workspace_bytes(int64_t B, int64_t K, int64_t SH2, int64_t D,
                                     gscan_dtype_t in_dtype)
{
    if (B <= 0 || K <= 0 || SH2 <= 0 || D <= 0) return 0;
    gscan::Plan plan;
    if (!gscan::make_plan(B, K, SH2, D, (int)in_dtype, &plan)) return 0;
    return plan.fwd_scratch;
}

size_t gscan_backward_workspace_bytes(int64_t B, int64_t K, int64_t SH2, int64_t D,
                                      gscan_dtype_t in_dtype)
{
    gscan::Plan plan;
    if (!gscan::make_plan(B, K, SH2, D, (int)in_dtype, &plan)) return 0;
    return plan.ws_bytes;
}

int gscan_backward_ex(const void *h_history, const void *h_s2, const float *W_A,
                      const float *W_B, const float *W_C, int64_t B, int64_t K, int64_t SH2,
                      int64_t D, const float *d_context, float *dW_A, float *dW_B, float *dW_C,
                      gscan_dtype_t in_dtype, float a_shift, void *workspace,
                      size_t workspace_bytes, hipStream_t stream)
{
    gscan::Plan plan;
    int st = check_backward(h_history, h_s2, W_A, W_B, W_C, B, K, SH2, D, d_context,
                            (int)in_dtype, &plan);
    if (st != GSCAN_OK) return st;
    if ((st = check_outputs(dW_A, dW_B, dW_C)) != GSCAN_OK) return st;
    if (workspace && (st = check_workspace(workspace, workspace_bytes, plan)) != GSCAN_OK)
        return st;
    clear_stale_error();
    void *ws = workspace;
    if (!ws) {
        hipError_t e = hipMallocAsync(&ws, plan.ws_bytes, stream);
        if (e != hipSuccess)
            return fail(GSCAN_ERR_HIP, "workspace allocation of %zu bytes failed: %s",
                        plan.ws_bytes, hipGetErrorString(e));
    }
    float *part = static_cast<float *>(ws);
    hipError_t e = gscan::launch_backward_partials(plan, h_history, h_s2, W_A, W_B, W_C, a_shift,
                                                   d_context, part, nullptr, nullptr, nullptr,
                                                   nullptr, stream);
    if (e == hipSuccess) e = gscan::launch_backward_reduce(plan, part, dW_A, dW_B, dW_C, stream);
    if (!workspace) {
        hipError_t f = hipFreeAsync(ws, stream);
        if (e == hipSuccess) e = f;
    }
    if (e != hipSuccess)
        return fail(GSCAN_ERR_HIP, "backward launch failed: %s", hipGetErrorString(e));
    g_last_error[0] = '\0';
    return GSCAN_OK;
}

size_t gscan_backward_full_workspace_bytes(int64_t B, int64_t K, int64_t SH2, int64_t D,
                                           gscan_dtype_t in_dtype)
{
    if (B <= 0 || K <= 0 || SH2 <= 0 || D <= 0) return 0;
    gscan::Plan plan;
    if (!gscan::make_plan(B, K, SH2, D, (int)in_dtype, &plan)) return 0;
    return full_layout(plan).bytes;
}

int gscan_backward_full_ex(const void *h_history, const void *h_s2, const float *W_A,
                           const float *W_B, const float *W_C, int64_t B, int64_t K, int64_t SH2,
                           int64_t D, const float *d_context, float *dW_A, float *dW_B,
                           float *dW_C, float *d_h_history, float *d_h_s2,
                           gscan_dtype_t in_dtype, float a_shift, void *workspace,
                           size_t workspace_bytes, hipStream_t stream)
{
    gscan::Plan plan;
    int st = check_backward(h_history, h_s2, W_A, W_B, W_C, B, K, SH2, D, d_context,
                            (int)in_dtype, &plan);
    if (st != GSCAN_OK) return st;
    if ((st = check_outputs(dW_A, dW_B, dW_C)) != GSCAN_OK) return st;
    if (!d_h_history || !d_h_s2)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null input-gradient pointer");
    if (!aligned16(d_h_history) || !aligned16(d_h_s2))
        return fail(GSCAN_ERR_MISALIGNED, "input-gradient pointers must be 16-byte aligned");
    const FullLayout lay = full_layout(plan);
    if (workspace) {
        if (workspace_bytes < lay.bytes)
            return fail(GSCAN_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < required %zu",
                        workspace_bytes, lay.bytes);
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
            return fail(GSCAN_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    }
    clear_stale_error();
    void *ws = workspace;
    if (!ws) {
        hipError_t e = hipMallocAsync(&ws, lay.bytes, stream);
        if (e != hipSuccess)
            return fail(GSCAN_ERR_HIP, "workspace allocation of %zu bytes failed: %s", lay.bytes,
                        hipGetErrorString(e));
    }
    char *base = static_cast<char *>(ws);
    float *part = reinterpret_cast<float *>(base);
    hipError_t e;
    if (plan.fused_dinput()) {
        // phase 1 writes d_h_history and d_h_s2 itself
        e = gscan::launch_backward_partials(plan, h_history, h_s2, W_A, W_B, W_C, a_shift,
                                            d_context, part, nullptr, nullptr, d_h_history,
                                            d_h_s2, stream);
        if (e == hipSuccess) e = gscan::launch_backward_reduce(plan, part, dW_A, dW_B, dW_C, stream);
    } else {
        float *dab = reinterpret_cast<float *>(base + lay.dab);
        float *dc = reinterpret_cast<float *>(base + lay.dc);
        e = gscan::launch_backward_partials(plan, h_history, h_s2, W_A, W_B, W_C, a_shift,
                                            d_context, part, dab, dc, nullptr, nullptr, stream);
        if (e == hipSuccess) e = gscan::launch_backward_reduce(plan, part, dW_A, dW_B, dW_C, stream);
        if (e == hipSuccess && !plan.adjoints_final())
            e = gscan::launch_adjoint(plan, dab, dc, d_context, a_shift, stream);
        if (e == hipSuccess)
            e = gscan::launch_dinput(dab, W_A, W_B, D, 2 * D, SH2, B * K, d_h_history, stream);
        if (e == hipSuccess) e = gscan::launch_dinput(dc, W_C, nullptr, D, D, SH2, B, d_h_s2, stream);
    }
    if (!workspace) {
        hipError_t f = hipFreeAsync(ws, stream);
        if (e == hipSuccess) e = f;
    }
    if (e != hipSuccess)
        return fail(GSCAN_ERR_HIP, "backward launch failed: %s", hipGetErrorString(e));
    g_last_error[0] = '\0';
    return GSCAN_OK;
}

size_t gscan_bias_grad_reduce_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 1 || rows > (int64_t(1) << 40) / cols) return 0;
    return gscan::colsum_workspace_bytes(rows, cols);
}

int gscan_bias_grad_reduce(const float *grad, int64_t rows, int64_t cols, float *out,
                           void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!out || (rows > 0 && !grad))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null pointer");
    if (rows < 0 || cols < 1)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "need rows >= 0 and cols >= 1 (rows=%lld cols=%lld)",
                    (long long)rows, (long long)cols);
    if (rows > (int64_t(1) << 40) / cols)
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE, "rows x cols above 2^40");
    if ((reinterpret_cast<uintptr_t>(grad) & 3u) != 0 || (reinterpret_cast<uintptr_t>(out) & 3u) != 0)
        return fail(GSCAN_ERR_MISALIGNED, "grad and out must be 4-byte aligned");
    const size_t need = gscan::colsum_workspace_bytes(rows, cols);
    if (workspace) {
        if (workspace_bytes < need)
            return fail(GSCAN_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < required %zu",
                        workspace_bytes, need);
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
            return fail(GSCAN_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    }
    clear_stale_error();
    void *ws = workspace;
    if (!ws) {
        hipError_t e = hipMallocAsync(&ws, need, stream);
        if (e != hipSuccess)
            return fail(GSCAN_ERR_HIP, "workspace allocation of %zu bytes failed: %s", need,
                        hipGetErrorString(e));
    }
    hipError_t e = gscan::launch_colsum(grad, rows, cols, out, ws, stream);
    if (!workspace) {
        hipError_t f = hipFreeAsync(ws, stream);
        if (e == hipSuccess) e = f;
    }
    if (e != hipSuccess)
        return fail(GSCAN_ERR_HIP, "bias-gradient reduction launch failed: %s", hipGetErrorString(e));
    g_last_error[0] = '\0';
    return GSCAN_OK;
}

int gscan_backward_partials(const void *h_history, const void *h_s2, const float *W_A,
                            const float *W_B, const float *W_C, int64_t B, int64_t K,
                            int64_t SH2, int64_t D, const float *d_context,
                            gscan_dtype_t in_dtype, float a_shift, void *workspace,
                            size_t workspace_bytes, hipStream_t stream)
{
    gscan::Plan plan;
    int st = check_backward(h_history, h_s2, W_A, W_B, W_C, B, K, SH2, D, d_context,
                            (int)in_dtype, &plan);
    if (st != GSCAN_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, plan)) != GSCAN_OK) return st;
    clear_stale_error();
    hipError_t e = gscan::launch_backward_partials(plan, h_history, h_s2, W_A, W_B, W_C, a_shift,
                                                   d_context, static_cast<float *>(workspace),
                                                   nullptr, nullptr, nullptr, nullptr, stream);
    if (e != hipSuccess)
        return fail(GSCAN_ERR_HIP, "backward phase 1 launch failed: %s", hipGetErrorString(e));
    g_last_error[0] = '\0';
    return GSCAN_OK;
}

int gscan_backward_reduce(const void *workspace, size_t workspace_bytes, int64_t B, int64_t K,
                          int64_t SH2, int64_t D, gscan_dtype_t in_dtype, float *dW_A,
                          float *dW_B, float *dW_C, hipStream_t stream)
{
    gscan::Plan plan;
    if (B <= 0 || K <= 0 || SH2 <= 0 || D <= 0)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "sizes must be positive");
    if (in_dtype != GSCAN_F32 && in_dtype != GSCAN_BF16)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "unknown input dtype %d", (int)in_dtype);
    if (!gscan::make_plan(B, K, SH2, D, (int)in_dtype, &plan))
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE, "unsupported shape");
    int st;
    if ((st = check_workspace(workspace, workspace_bytes, plan)) != GSCAN_OK) return st;
    if ((st = check_outputs(dW_A, dW_B, dW_C)) != GSCAN_OK) return st;
    clear_stale_error();
    hipError_t e = gscan::launch_backward_reduce(plan, static_cast<const float *>(workspace), dW_A,
                                                 dW_B, dW_C, stream);
    if (e != hipSuccess)
        return fail(GSCAN_ERR_HIP, "backward phase 2 launch failed: %s", hipGetErrorString(e));
    g_last_error[0] = '\0';
    return GSCAN_OK;
}

int gscan_backward_noalloc(const void *h_history, const void *h_s2, const float *W_A,
                           const float *W_B, const float *W_C, int64_t B, int64_t K, int64_t SH2,
                           int64_t D, const float *d_context, float *dW_A, float *dW_B,
                           float *dW_C, gscan_dtype_t in_dtype, float a_shift,
                           hipStream_t stream)
{
    gscan::Plan plan;
    int st = check_backward(h_history, h_s2, W_A, W_B, W_C, B, K, SH2, D, d_context,
                            (int)in_dtype, &plan);
    if (st != GSCAN_OK) return st;
    if ((st = check_outputs(dW_A, dW_B, dW_C)) != GSCAN_OK) return st;
    if (plan.ws_bytes > (size_t)GSCAN_NOALLOC_SCRATCH_BYTES)
        return fail(GSCAN_ERR_WORKSPACE_TOO_SMALL,
                    "shape B=%lld K=%lld SH2=%lld D=%lld needs %zu bytes of partials, more than "
                    "the %zu-byte static scratch of gscan_backward_noalloc (use "
                    "gscan_backward_ex with a workspace)",
                    (long long)B, (long long)K, (long long)SH2, (long long)D, plan.ws_bytes,
                    (size_t)GSCAN_NOALLOC_SCRATCH_BYTES);
    void *ws = nullptr;
    if ((st = current_scratch(&ws)) != GSCAN_OK) return st;
    clear_stale_error();
    // phase 1 overwrites every partial it leaves for phase 2: nothing in the
    // scratch needs to start at zero
    float *part = static_cast<float *>(ws);
    hipError_t e = gscan::launch_backward_partials(plan, h_history, h_s2, W_A, W_B, W_C, a_shift,
                                                   d_context, part, nullptr, nullptr, nullptr,
                                                   nullptr, stream);
    if (e == hipSuccess) e = gscan::launch_backward_reduce(plan, part, dW_A, dW_B, dW_C, stream);
    if (e != hipSuccess)
        return fail(GSCAN_ERR_HIP, "backward launch failed: %s", hipGetErrorString(e));
    g_last_error[0] = '\0';
    return GSCAN_OK;
}

int gscan_backward(const void *h_history, const void *h_s2, const float *W_A, const float *W_B,
                   const float *W_C, int64_t B, int64_t K, int64_t SH2, int64_t D,
                   const float *d_context, float *dW_A, float *dW_B, float *dW_C,
                   hipStream_t stream)
{
    return gscan_backward_ex(h_history, h_s2, W_A, W_B, W_C, B, K, SH2, D, d_context, dW_A, dW_B,
                             dW_C, GSCAN_F32, 0.0f, nullptr, 0, stream);
}

int gscan_batched_cifg_update(float *C_batch, const float *H, const float *X, const float *W_f,
                              const float *b_f, int64_t B, int64_t d_model, int64_t d_input,
                              hipStream_t stream)
{
    if (!C_batch || !H || !W_f || !b_f || (d_input > 0 && !X))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null pointer");
    if (B < 1 || d_model < 1 || d_input < 0)
        return fail(GSCAN_ERR_INVALID_ARGUMENT,
                    "need B >= 1, d_model >= 1, d_input >= 0 (B=%lld d_model=%lld d_input=%lld)",
                    (long long)B, (long long)d_model, (long long)d_input);
    if (d_model % 4 != 0 || d_input % 4 != 0 || d_model > 16384 || d_input > (int64_t(1) << 24) ||
        B > (int64_t(1) << 40) / (d_model * d_model))
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE,
                    "unsupported shape B=%lld d_model=%lld d_input=%lld (need d_model and d_input "
                    "multiples of 4, d_model <= 16384, B*d_model^2 <= 2^40)",
                    (long long)B, (long long)d_model, (long long)d_input);
    if (!aligned16(C_batch) || !aligned16(H) || (d_input > 0 && !aligned16(X)) ||
        !aligned16(W_f) || (reinterpret_cast<uintptr_t>(b_f) & 3u) != 0)
        return fail(GSCAN_ERR_MISALIGNED,
                    "C_batch, H, X, W_f must be 16-byte aligned and b_f 4-byte aligned");
    // C_batch is updated in place and must not overlap any input
    const uintptr_t c0 = reinterpret_cast<uintptr_t>(C_batch);
    const uintptr_t c1 = c0 + (uintptr_t)(B * d_model * d_model) * sizeof(float);
    auto overlaps = [&](const void *p, int64_t n) {
        const uintptr_t a0 = reinterpret_cast<uintptr_t>(p);
        return p && n > 0 && a0 < c1 && c0 < a0 + (uintptr_t)n * sizeof(float);
    };
    if (overlaps(H, B * d_model) || overlaps(X, B * d_input) ||
        overlaps(W_f, d_model * (d_model + d_input)) || overlaps(b_f, d_model))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "C_batch overlaps an input");
    clear_stale_error();
    hipError_t e = gscan::launch_cifg(C_batch, H, d_input > 0 ? X : H, W_f, b_f, B, d_model,
                                      d_input, stream);
    if (e != hipSuccess)
        return fail(GSCAN_ERR_HIP, "CIFG update launch failed: %s", hipGetErrorString(e));
    g_last_error[0] = '\0';
    return GSCAN_OK;
}

int gscan_state_scan_forward(const gscan_state_scan_t *desc, const void *q, const void *k,
                             const void *v, const void *gate, const float *initial_state,
                             void *out, float *final_state, void *workspace,
                             size_t workspace_bytes, hipStream_t stream)
{
    gscan::StateArgs a;
    gscan::StatePlan p;
    int st = check_state_desc(desc, false, &a);
    if (st != GSCAN_OK) return st;
    a.q = q;
    a.k = k;
    a.v = v;
    a.gate = gate;
    a.s0 = initial_state;
    a.out = out;
    a.sT = final_state;
    if ((st = check_state_inputs(a)) != GSCAN_OK) return st;
    if (a.T > 0 && !out) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null out");
    if (mis(out, 16) || mis(final_state, 16))
        return fail(GSCAN_ERR_MISALIGNED, "out and final_state must be 16-byte aligned");
    if ((st = state_plan(a, false, &p)) != GSCAN_OK) return st;
    if (a.T == 0 && !final_state) return GSCAN_OK;
    return with_workspace("state scan forward", workspace, workspace_bytes, p.bytes, stream,
                          [&](void *ws) {
                              a.ws = ws;
                              return gscan::launch_state_forward(p, a, stream);
                          });
}

int gscan_state_scan_backward(const gscan_state_scan_t *desc, const void *q, const void *k,
                              const void *v, const void *gate, const float *initial_state,
                              const void *d_out, const float *d_final_state, void *dq, void *dk,
                              void *dv, void *dgate, float *d_initial_state, void *workspace,
                              size_t workspace_bytes, hipStream_t stream)
{
    gscan::StateArgs a;
    gscan::StatePlan p;
    int st = check_state_desc(desc, true, &a);
    if (st != GSCAN_OK) return st;
    a.q = q;
    a.k = k;
    a.v = v;
    a.gate = gate;
    a.s0 = initial_state;
    a.dout = d_out;
    a.dsT = d_final_state;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dgate = dgate;
    a.ds0 = d_initial_state;
    if ((st = check_state_inputs(a)) != GSCAN_OK) return st;
    if (a.T > 0 && (!d_out || !dq || !dk || !dv || !dgate))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null d_out or gradient pointer");
    if (mis(d_out, 16) || mis(d_final_state, 16) || mis(dq, 16) || mis(dk, 16) || mis(dv, 16) ||
        mis(dgate, (uintptr_t)esize(a.gate_dtype)) || mis(d_initial_state, 16))
        return fail(GSCAN_ERR_MISALIGNED, "gradients must be 16-byte aligned, dgate to its elements");
    if ((st = state_plan(a, true, &p)) != GSCAN_OK) return st;
    if (a.T == 0 && !d_initial_state) return GSCAN_OK;
    return with_workspace("state scan backward", workspace, workspace_bytes, p.bytes, stream,
                          [&](void *ws) {
                              a.ws = ws;
                              return gscan::launch_state_backward(p, a, stream);
                          });
}

size_t gscan_state_scan_forward_workspace_bytes(const gscan_state_scan_t *desc)
{
    gscan::StateArgs a;
    gscan::StatePlan p;
    if (check_state_desc(desc, false, &a) != GSCAN_OK || state_plan(a, false, &p) != GSCAN_OK) return 0;
    return p.bytes;
}

size_t gscan_state_scan_backward_workspace_bytes(const gscan_state_scan_t *desc)
{
    gscan::StateArgs a;
    gscan::StatePlan p;
    if (check_state_desc(desc, false, &a) != GSCAN_OK || state_plan(a, true, &p) != GSCAN_OK) return 0;
    return p.bytes;
}

int gscan_state_scan_step(const gscan_state_scan_t *desc, const void *q, const void *k,
                          const void *v, const void *gate, float *state, int64_t pool,
                          const int32_t *slots, void *out, hipStream_t stream)
{
    gscan::StateArgs a;
    int st = check_state_desc(desc, false, &a);
    if (st != GSCAN_OK) return st;
    if (a.T != 1 || a.off)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "a step takes T = 1 and no seq_offsets (T=%lld)",
                    (long long)a.T);
    a.q = q;
    a.k = k;
    a.v = v;
    a.gate = gate;
    a.s0 = state;
    if ((st = check_state_inputs(a)) != GSCAN_OK) return st;
    if (!state || !out) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null state or out");
    if (mis(out, 16) || mis(slots, 4))
        return fail(GSCAN_ERR_MISALIGNED, "out must be 16-byte aligned, slots to its elements");
    if (pool < 1 || (!slots && a.B > pool))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "pool of %lld states for %lld requests",
                    (long long)pool, (long long)a.B);
    if (a.B > kMaxGrid / 8 / a.H)
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE, "too many requests times heads (%lld x %d)",
                    (long long)a.B, a.H);
    gscan::StepArgs s;
    s.q = q;
    s.k = k;
    s.v = v;
    s.gate = gate;
    s.qn = a.qs.b;
    s.qh = a.qs.h;
    s.kn = a.ks.b;
    s.kh = a.ks.h;
    s.vn = a.vs.b;
    s.vh = a.vs.h;
    s.gn = a.gs.b;
    s.gh = a.gs.h;
    s.state = state;
    s.slots = slots;
    s.out = out;
    s.N = a.B;
    s.pool = pool;
    s.H = a.H;
    s.Hk = a.Hk;
    s.Dk = a.Dk;
    s.Dv = a.Dv;
    s.dtype = a.dtype;
    s.gate_dtype = a.gate_dtype;
    s.gate_form = a.gate_form;
    s.gate_shift = a.gate_shift;
    s.scale = a.scale;
    return with_workspace("state scan step", nullptr, 0, 0, stream,
                          [&](void *) { return gscan::launch_state_step(s, stream); });
}

int gscan_qk_norm_rope_forward(const gscan_qk_norm_t *desc, const void *q, const void *k,
                               const float *weight_q, const float *weight_k,
                               const void *positions, const float *freq, void *q_out, void *k_out,
                               hipStream_t stream)
{
    gscan::NormArgs a;
    int st = check_norm(desc, q, k, weight_q, weight_k, positions, freq, &a);
    if (st != GSCAN_OK) return st;
    if (a.tokens > 0 && (!q_out || (a.heads[1] > 0 && !k_out)))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null output");
    if (mis(q_out, 16) || mis(k_out, 16))
        return fail(GSCAN_ERR_MISALIGNED, "outputs must be 16-byte aligned");
    a.y[0] = q_out;
    a.y[1] = k_out;
    return with_workspace("query/key norm", nullptr, 0, 0, stream,
                          [&](void *) { return gscan::launch_norm_forward(a, stream); });
}

int gscan_qk_norm_rope_backward(const gscan_qk_norm_t *desc, const void *q, const void *k,
                                const float *weight_q, const float *weight_k,
                                const void *positions, const float *freq, const void *dy_q,
                                const void *dy_k, void *dq, void *dk, float *d_weight_q,
                                float *d_weight_k, void *workspace, size_t workspace_bytes,
                                hipStream_t stream)
{
    gscan::NormArgs a;
    int st = check_norm(desc, q, k, weight_q, weight_k, positions, freq, &a);
    if (st != GSCAN_OK) return st;
    const bool keys = a.heads[1] > 0;
    if (a.tokens > 0 && (!dy_q || !dq || (keys && (!dy_k || !dk))))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null gradient pointer");
    if (mis(dy_q, 16) || mis(dy_k, 16) || mis(dq, 16) || mis(dk, 16) || mis(d_weight_q, 4) ||
        mis(d_weight_k, 4) || !strides16(desc->dy_q_stride, 2, a.dtype) ||
        (keys && !strides16(desc->dy_k_stride, 2, a.dtype)))
        return fail(GSCAN_ERR_MISALIGNED, "gradients and their strides must be multiples of 16 bytes");
    a.dy[0] = dy_q;
    a.dy[1] = dy_k;
    a.dn[0] = desc->dy_q_stride[0];
    a.dh[0] = desc->dy_q_stride[1];
    a.dn[1] = desc->dy_k_stride[0];
    a.dh[1] = desc->dy_k_stride[1];
    a.y[0] = dq;
    a.y[1] = dk;
    a.dw[0] = d_weight_q;
    a.dw[1] = d_weight_k;
    const bool weights = d_weight_q || d_weight_k;
    const size_t need = weights ? gscan::norm_workspace_bytes(a.tokens, a.heads[0] + a.heads[1], a.D) : 0;
    return with_workspace("query/key norm backward", weights ? workspace : nullptr, workspace_bytes,
                          need, stream, [&](void *ws) {
                              a.ws = ws;
                              return gscan::launch_norm_backward(a, stream);
                          });
}

size_t gscan_qk_norm_rope_workspace_bytes(const gscan_qk_norm_t *desc)
{
    if (!desc || desc->tokens < 0 || desc->D < 1 || desc->D > 256 || desc->Hq < 1 || desc->Hk < 0 ||
        desc->Hq > kMaxNormHeads || desc->Hk > kMaxNormHeads)
        return 0;
    return gscan::norm_workspace_bytes(desc->tokens, (int)(desc->Hq + desc->Hk), (int)desc->D);
}

int gscan_embed_forward(const gscan_embed_t *desc, const void *table, const void *tokens, void *out,
                        hipStream_t stream)
{
    gscan::EmbedArgs a;
    int st = check_embed(desc, tokens, &a);
    if (st != GSCAN_OK) return st;
    if (a.N > 0 && (!table || !out)) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null table or out");
    if (mis(table, 16) || mis(out, 16) || !strides16(&desc->stride, 1, a.table_dtype))
        return fail(GSCAN_ERR_MISALIGNED, "table, its row stride and out must be multiples of 16 bytes");
    a.table = table;
    a.out = out;
    return with_workspace("embedding", nullptr, 0, 0, stream,
                          [&](void *) { return gscan::launch_embed_forward(a, stream); });
}

int gscan_embed_backward(const gscan_embed_t *desc, const void *d_out, const void *tokens, void *d_table,
                         void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    gscan::EmbedArgs a;
    int st = check_embed(desc, tokens, &a);
    if (st != GSCAN_OK) return st;
    if (!d_table || (a.N > 0 && !d_out)) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null d_out or d_table");
    if (mis(d_out, 16) || mis(d_table, 16) || !strides16(&desc->stride, 1, a.dtype))
        return fail(GSCAN_ERR_MISALIGNED, "d_out, its row stride and d_table must be multiples of 16 bytes");
    a.dout = d_out;
    a.dtable = d_table;
    return with_workspace("embedding backward", workspace, workspace_bytes,
                          gscan::embed_workspace_bytes(a.N, a.V, a.D), stream, [&](void *ws) {
                              a.ws = ws;
                              return gscan::launch_embed_backward(a, stream);
                          });
}

size_t gscan_embed_workspace_bytes(const gscan_embed_t *desc)
{
    gscan::EmbedArgs a;
    if (check_embed(desc, nullptr, &a, false) != GSCAN_OK) return 0;
    return gscan::embed_workspace_bytes(a.N, a.V, a.D);
}

int gscan_gated_projection_forward(const gscan_gated_projection_t *desc, const void *x, const void *w_gate,
                                   const void *w_up, void *out, void *workspace, size_t workspace_bytes,
                                   hipStream_t stream)
{
    gscan::GateArgs a;
    int st = check_gate(desc, x, w_gate, w_up, &a);
    if (st != GSCAN_OK) return st;
    if (a.N > 0 && !out) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null out");
    if (mis(out, 16)) return fail(GSCAN_ERR_MISALIGNED, "out must be 16-byte aligned");
    a.out = out;
    return with_workspace("gated projection", workspace, workspace_bytes, gscan::gate_workspace_bytes(a, false),
                          stream, [&](void *ws) {
                              a.ws = ws;
                              return gscan::launch_gate_forward(a, stream);
                          });
}

int gscan_gated_projection_backward(const gscan_gated_projection_t *desc, const void *x, const void *w_gate,
                                    const void *w_up, const void *d_out, void *dx, void *d_w_gate,
                                    void *d_w_up, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    gscan::GateArgs a;
    int st = check_gate(desc, x, w_gate, w_up, &a);
    if (st != GSCAN_OK) return st;
    if (a.N > 0 && !d_out) return fail(GSCAN_ERR_INVALID_ARGUMENT, "null d_out");
    if (!d_w_gate != !d_w_up)
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "d_w_gate and d_w_up go together");
    if (mis(d_out, 16) || mis(dx, 16) || mis(d_w_gate, 16) || mis(d_w_up, 16) ||
        !strides16(&desc->d_out_stride, 1, a.dtype))
        return fail(GSCAN_ERR_MISALIGNED, "gradients and d_out's row stride must be multiples of 16 bytes");
    if (desc->d_out_stride < 0 || desc->d_out_stride > kMaxRowStride)
        return fail(GSCAN_ERR_UNSUPPORTED_SHAPE, "row strides must be 0 .. 2^21 elements");
    a.dout = d_out;
    a.ldd = desc->d_out_stride;
    a.dx = dx;
    a.dwg = d_w_gate;
    a.dwu = d_w_up;
    return with_workspace("gated projection backward", workspace, workspace_bytes,
                          gscan::gate_workspace_bytes(a, true), stream, [&](void *ws) {
                              a.ws = ws;
                              return gscan::launch_gate_backward(a, stream);
                          });
}

size_t gscan_gated_projection_forward_workspace_bytes(const gscan_gated_projection_t *desc)
{
    gscan::GateArgs a;
    if (check_gate(desc, nullptr, nullptr, nullptr, &a, false) != GSCAN_OK) return 0;
    return gscan::gate_workspace_bytes(a, false);
}

size_t gscan_gated_projection_backward_workspace_bytes(const gscan_gated_projection_t *desc)
{
    gscan::GateArgs a;
    if (check_gate(desc, nullptr, nullptr, nullptr, &a, false) != GSCAN_OK) return 0;
    return gscan::gate_workspace_bytes(a, true);
}

int gscan_linear_cross_entropy_forward(const gscan_linear_cross_entropy_t *desc, const void *h, const void *weight,
                                       const void *target, float *loss, float *lse, void *workspace,
                                       size_t workspace_bytes, hipStream_t stream)
{
    gscan::XentArgs a;
    int st = check_xent(desc, h, weight, target, &a);
    if (st != GSCAN_OK) return st;
    if ((!loss && (a.N > 0 || a.reduction)) || (a.N > 0 && !lse))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null loss or lse");
    if (mis(loss, 4) || mis(lse, 4)) return fail(GSCAN_ERR_MISALIGNED, "misaligned loss or lse");
    if (!a.N && !a.reduction) return GSCAN_OK;
    a.loss = loss;
    a.lse = lse;
    return with_workspace("cross entropy", workspace, workspace_bytes,
                          gscan::xent_forward_workspace_bytes(a.N, a.V, a.D, a.dtype), stream, [&](void *ws) {
                              a.ws = ws;
                              return gscan::launch_xent_forward(a, stream);
                          });
}

int gscan_linear_cross_entropy_backward(const gscan_linear_cross_entropy_t *desc, const void *h, const void *weight,
                                        const void *target, const float *lse, const float *d_loss, void *dh,
                                        void *d_weight, void *workspace, size_t workspace_bytes,
                                        hipStream_t stream)
{
    gscan::XentArgs a;
    int st = check_xent(desc, h, weight, target, &a);
    if (st != GSCAN_OK) return st;
    if ((!d_loss && (a.N > 0 || a.reduction)) || (a.N > 0 && !lse))
        return fail(GSCAN_ERR_INVALID_ARGUMENT, "null lse or d_loss");
    if (mis(lse, 4) || mis(d_loss, 4) || mis(dh, 16) || mis(d_weight, 16))
        return fail(GSCAN_ERR_MISALIGNED, "dh and d_weight must be 16-byte aligned, lse and d_loss to their elements");
    a.lse = const_cast<float *>(lse);
    a.dloss = d_loss;
    a.dh = dh;
    a.dw = d_weight;
    return with_workspace("cross entropy backward", workspace, workspace_bytes,
                          gscan::xent_backward_workspace_bytes(a.N, a.V, a.D, a.dtype), stream, [&](void *ws) {
                              a.ws = ws;
                              return gscan::launch_xent_backward(a, stream);
                          });
}

size_t gscan_linear_cross_entropy_forward_workspace_bytes(const gscan_linear_cross_entropy_t *desc)
{
    gscan::XentArgs a;
    if (check_xent(desc, nullptr, nullptr, nullptr, &a, false) != GSCAN_OK) return 0;
    return gscan::xent_forward_workspace_bytes(a.N, a.V, a.D, a.dtype);
}

size_t gscan_linear_cross_entropy_backward_workspace_bytes(const gscan_linear_cross_entropy_t *desc)
{
    gscan::XentArgs a;
    if (check_xent(desc, nullptr, nullptr, nullptr, &a, false) != GSCAN_OK) return 0;
    return gscan::xent_backward_workspace_bytes(a.N, a.V, a.D, a.dtype);
}

const char *gscan_status_string(int status)
{
    switch (status) {
    case GSCAN_OK: return "ok";
    case GSCAN_ERR_INVALID_ARGUMENT: return "invalid argument";
    case GSCAN_ERR_UNSUPPORTED_SHAPE: return "unsupported shape";
    case GSCAN_ERR_MISALIGNED: return "misaligned pointer";
    case GSCAN_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case GSCAN_ERR_HIP: return "HIP runtime error";
    default: return "unknown status";
    }
}

const char *gscan_last_error(void)
{
    return g_last_error;
}

int gscan_version(void)
{
    return 100;  // 0.1.0
}

}  // extern "C"
