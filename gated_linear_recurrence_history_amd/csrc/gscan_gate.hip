// Gated projection, forward and backward, for gfx950 (MI355X):
//
//   a = x Wg^T,  b = x Wu^T,  out = act(a) * b
//   da = dout * b * act'(a),  db = dout * act(a)
//   dx = da Wg + db Wu,  dWg = da^T x,  dWu = db^T x
//
// Forward: one kernel.  A tile holds the same columns of both products, so that
// a lane has a and b of the same elements and neither reaches memory.
// Backward: the same kernel again, whose epilogue leaves da | db (in the type of
// the operands: the one rounding between the products; unrounded they would need fp32
// products, at a seventh of the rate), then a product for dx over the columns of da and db
// in turn, and one for both weights' gradients.
// 8192 tokens, 2048 x 2 x 5504: forward 325 us (1136 TFLOP/s); 4109 tokens, backward: 561 us
// (991 TFLOP/s).
#include "gscan_few.h"

namespace gscan {

namespace {

struct Layout {
    size_t partial = 0, bytes = 0;
};
size_t round_up(size_t x) { return (x + 255) & ~(size_t)255; }

Layout lay_out(const GateArgs &g, bool backward)
{
    const int64_t F2 = 2 * (int64_t)g.F;
    Layout l;
    size_t parts = mm_bytes(g.F, g.N, g.D, 0, true, false, g.dtype);
    if (backward) {
        l.partial = round_up((size_t)g.N * F2 * (g.dtype ? 2 : 4));  // behind da | db
        const size_t dx = mm_bytes(g.D, g.N, F2, g.F, false, false, g.dtype);
        const size_t dw = mm_bytes(g.D, F2, g.N, 0, false, false, g.dtype);
        if (dx > parts) parts = dx;
        if (dw > parts) parts = dw;
    }
    l.bytes = l.partial + parts;
    return l;
}

// Both products.
MmArgs products(const GateArgs &g)
{
    MmArgs a;
    a.a = g.wg;
    a.a2 = g.wu;
    a.lda = g.ldg;
    a.lda2 = g.ldu;
    a.b = g.x;
    a.ldb = g.ldx;
    a.M = g.F;
    a.N = g.N;
    a.K = g.D;
    a.act = g.act;
    return a;
}

}  // namespace

size_t gate_workspace_bytes(const GateArgs &g, bool backward)
{
    return g.N && (backward || g.N > kFew) ? lay_out(g, backward).bytes : 0;
}

hipError_t launch_gate_forward(const GateArgs &g, hipStream_t st)
{
    MmArgs a = products(g);
    a.out = g.out;
    a.ldo = g.F;
    if (!g.N) return hipSuccess;
    if (g.N <= kFew) return launch_few<EPI_GATE>(a, g.dtype, st);
    return launch_mm<EPI_GATE, false, false, LIMIT_NONE>(a, g.dtype, g.ws, st);
}

hipError_t launch_gate_backward(const GateArgs &g, hipStream_t st)
{
    const int64_t F2 = 2 * (int64_t)g.F;
    void *partial = reinterpret_cast<char *>(g.ws) + lay_out(g, true).partial;
    hipError_t e;
    MmArgs r = products(g);
    r.out = g.ws;
    r.ldo = F2;
    r.dout = g.dout;
    r.ldd = g.ldd;
    if ((e = launch_mm<EPI_DGATE, false, false, LIMIT_NONE>(r, g.dtype, partial, st)) != hipSuccess) return e;
    if (g.dx) {
        MmArgs a = products(g);
        a.K1 = g.F;
        a.b = g.ws;
        a.ldb = F2;
        a.M = g.D;
        a.K = F2;
        a.out = g.dx;
        a.ldo = g.D;
        a.N1 = g.N;
        if ((e = launch_mm<EPI_STORE, true, false, LIMIT_NONE>(a, g.dtype, partial, st)) != hipSuccess) return e;
    }
    if (!g.dwg) return hipSuccess;
    MmArgs a;
    a.a = g.x;
    a.lda = g.ldx;
    a.b = g.ws;
    a.ldb = F2;
    a.M = g.D;
    a.N = F2;
    a.K = g.N;
    a.out = g.dwg;
    a.out2 = g.dwu;
    a.ldo = g.D;
    a.N1 = g.F;
    return launch_mm<EPI_STORE, true, true, LIMIT_NONE>(a, g.dtype, partial, st);
}

}  // namespace gscan
