// Gated projection, forward and backward, for gfx950 (MI355X):
//
//   a = x Wg^T,  b = x Wu^T,  out = act(a) * b
//   da = dout * b * act'(a),  db = dout * act(a)
//   dx = da Wg + db Wu,  dWg = da^T x,  dWu = db^T x
//
// Forward: one kernel.  A tile holds the same columns of both products, so that
// a lane has a and b of the same elements and neither reaches memory.
// Backward: the same kernel again, whose epilogue leaves da | db (in the type of
// the operands: the one rounding between the products), then a product for dx
// over the columns of da and db in turn, and one for both weights' gradients.
#include "gscan_mm.h"

namespace gscan {

size_t gate_workspace_bytes(int64_t N, int F, int dtype)
{
    return (size_t)N * 2 * (size_t)F * (dtype ? 2 : 4);
}

hipError_t launch_gate_forward(const GateArgs &g, hipStream_t st)
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
    a.out = g.out;
    a.ldo = g.F;
    a.act = g.act;
    return launch_mm<EPI_GATE, false, false, LIMIT_NONE>(a, g.dtype, st);
}

hipError_t launch_gate_backward(const GateArgs &g, hipStream_t st)
{
    const int64_t F2 = 2 * (int64_t)g.F;
    hipError_t e;
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
        a.out = g.ws;
        a.ldo = F2;
        a.dout = g.dout;
        a.ldd = g.ldd;
        a.act = g.act;
        if ((e = launch_mm<EPI_DGATE, false, false, LIMIT_NONE>(a, g.dtype, st)) != hipSuccess) return e;
    }
    if (g.dx) {
        MmArgs a;
        a.a = g.wg;
        a.a2 = g.wu;
        a.lda = g.ldg;
        a.lda2 = g.ldu;
        a.K1 = g.F;
        a.b = g.ws;
        a.ldb = F2;
        a.M = g.D;
        a.N = g.N;
        a.K = F2;
        a.out = g.dx;
        a.ldo = g.D;
        a.N1 = g.N;
        if ((e = launch_mm<EPI_STORE, true, false, LIMIT_NONE>(a, g.dtype, st)) != hipSuccess) return e;
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
    return launch_mm<EPI_STORE, true, true, LIMIT_NONE>(a, g.dtype, st);
}

}  // namespace gscan
