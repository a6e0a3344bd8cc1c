// The matrix-state scan for single tokens (serving), for gfx950 (MI355X).
//
// Per request n and head h, with the state S = pool[slot_n][h] (fp32):
//   S <- g S + k v^T,   o = scale S^T q,   g = sigmoid(a + shift) or exp(a).
// The state is read once and written once and nothing else is of size, so
// the kernel is a stream: one workgroup per request and head, sixteen bytes
// per thread and row of S, up to eight rows of a thread in flight.  The sum
// over Dk of o is kept per thread and joined in LDS in a fixed order.
// Measured: 250 requests, 32 heads of 128 x 64: 524 MB in 112 us a call with cold
// caches, 4.7 TB/s (a large copy: 4.8), 85 us on the same states again; one
// request, 16 heads of 64 x 64: 5 us, launch and latency.
// Arithmetic is fp32; only o is rounded to the type of v.
#include "gscan_state_dev.h"

namespace gscan {
namespace {

constexpr int kStepThreads = 256;
constexpr int kStepRows = 8;  // rows of a thread in flight

__global__ void __launch_bounds__(kStepThreads) gscan_state_step_kernel(StepArgs a)
{
    __shared__ f4 red[kStepThreads];
    __shared__ float qs[128], ks[128];
    const int tid = threadIdx.x;
    const int64_t n = blockIdx.x / a.H;
    const int h = blockIdx.x % a.H, hk = h / (a.H / a.Hk);
    const int cpr = a.Dv / 4, rpp = kStepThreads / cpr;  // pieces per row, rows per pass
    const int r0 = tid / cpr, c = tid % cpr;
    const int64_t slot = a.slots ? a.slots[n] : n;
    char *out = reinterpret_cast<char *>(a.out) + (n * a.H + h) * a.Dv * (a.dtype ? 2 : 4);
    if (slot < 0 || slot >= a.pool) {  // no state: the request is padding
        if (tid < a.Dv) {
            if (a.dtype) reinterpret_cast<uint16_t *>(out)[tid] = 0;
            else reinterpret_cast<float *>(out)[tid] = 0.f;
        }
        return;
    }
    f4 *st = reinterpret_cast<f4 *>(a.state + (slot * a.H + h) * a.Dk * a.Dv);
    const bool live = r0 < rpp;
    f4 x[kStepRows];
#pragma unroll
    for (int i = 0; i < kStepRows; ++i)
        if (live && r0 + i * rpp < a.Dk) x[i] = st[(r0 + i * rpp) * cpr + c];
    if (tid < a.Dk) qs[tid] = load_scalar(a.q, n * a.qn + hk * a.qh + tid, a.dtype);
    else if (tid >= 128 && tid - 128 < a.Dk)
        ks[tid - 128] = load_scalar(a.k, n * a.kn + hk * a.kh + tid - 128, a.dtype);
    f4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = load_scalar(a.v, n * a.vn + h * a.vh + 4 * c + j, a.dtype);
    const float g = expf(log_gate(load_scalar(a.gate, n * a.gn + h * a.gh, a.gate_dtype) + a.gate_shift,
                                  a.gate_form));
    __syncthreads();
    f4 o = {0.f, 0.f, 0.f, 0.f};
    for (int b = 0; b < a.Dk; b += kStepRows * rpp) {
        if (b) {
#pragma unroll
            for (int i = 0; i < kStepRows; ++i)
                if (live && b + r0 + i * rpp < a.Dk) x[i] = st[(b + r0 + i * rpp) * cpr + c];
        }
#pragma unroll
        for (int i = 0; i < kStepRows; ++i) {
            const int r = b + r0 + i * rpp;
            if (live && r < a.Dk) {
                const float k = ks[r], q = qs[r];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] = fmaf(g, x[i][j], k * v[j]);
                    o[j] = fmaf(q, x[i][j], o[j]);
                }
                st[r * cpr + c] = x[i];
            }
        }
    }
    red[tid] = o;
    __syncthreads();
    if (tid < a.Dv) {
        const float *p = reinterpret_cast<const float *>(red) + tid;
        float s = 0.f;
        for (int r = 0; r < rpp && r < a.Dk; ++r) s += p[r * a.Dv];
        s *= a.scale;
        if (a.dtype) reinterpret_cast<uint16_t *>(out)[tid] = to_bf16(s);
        else reinterpret_cast<float *>(out)[tid] = s;
    }
}

}  // namespace

hipError_t launch_state_step(const StepArgs &a, hipStream_t st)
{
    hipLaunchKernelGGL(gscan_state_step_kernel, dim3((unsigned)(a.N * a.H)), dim3(kStepThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace gscan
