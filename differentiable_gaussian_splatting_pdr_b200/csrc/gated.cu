// gated: h = act(x Wg^T) * (x Wu^T), and its gradients (include/pdr.h).
//
// Forward: one launch.  A tile's accumulator holds 128 gate columns and the
// same 128 up columns side by side (rows of Wg and of Wu in the two halves of
// the B tile), so that the epilogue has g and u of an element in one thread
// and writes h alone: neither g nor u ever leaves the chip.
//
// Backward: g and u are formed again from x and the weights (nothing is saved
// by the forward), and their product's epilogue turns them, with dh, into
//   dg = dh u act'(g),   du = dh act(g),
// rounded to x's type as operands of the three products that follow:
//   dx = dg Wg + du Wu          one product, k running over both sources;
//   dWg = dg^T x, dWu = du^T x  in the same launch, k split over the machine, fp32
//                               partial results added in order.
// In fp16 dg and du are taken times a power of two that fits their bound, as dz in
// linear.cu: |dg| and |du| are at most 1.13 max |dh| D max |x| max |w| (k_largest over the
// four).  The bound is loose by some 2^7, and 2^-28 of it still a normal number.
// (16384 x 256 to 1024 with a cold L2: 85 us, without the factor 76.)
// 65536 x 256 to 1024 in bf16: 61 to 64 us (71 to 74 under the power cap that a long run meets;
// 1100 and 950 TFLOP/s); the backward of 16384 rows 69 us.
#include "gemm.cuh"

namespace pdr {
namespace {

// The workspace: padded copies of what TMA or 32-byte loads cannot address,
// padded results that are copied out at the end, dg and du, and partial sums.
struct GatedLayout {
    size_t x, wg, wu, in, out, dg, du, part, bound, total;
    long long ldk, ldi, ldo, ldf, ldp;
    bool pack_x, pack_in, pack_out, scaled;
    int splits;
    size_t take(size_t bytes) {
        const size_t at = total;
        total += align256(bytes);
        return at;
    }
};

bool sizes_ok(int M, int D, int F) { return M >= 0 && D >= 1 && F >= 1; }
bool in_limits(int M, int D, int F) {
    return M <= PDR_MAX_ROWS && D <= PDR_MAX_FEATURES && F <= PDR_MAX_FEATURES;
}
GatedLayout x_layout(int M, int D, int F, int dtype) {
    GatedLayout L = {};
    const int e = dtype_bytes(dtype);
    L.ldk = padded(D, e, 16);
    L.pack_x = L.ldk != D;
    if (L.pack_x) {
        L.x = L.take((size_t)M * L.ldk * e);
        L.wg = L.take((size_t)F * L.ldk * e);
        L.wu = L.take((size_t)F * L.ldk * e);
    }
    return L;
}

GatedLayout fwd_layout(int M, int D, int F, int dtype, int h_dtype) {
    GatedLayout L = x_layout(M, D, F, dtype);
    const int o = dtype_bytes(h_dtype);
    L.ldo = padded(F, o, 16);
    L.pack_out = L.ldo != F;
    if (L.pack_out) L.out = L.take((size_t)M * L.ldo * o);
    return L;
}

GatedLayout bwd_layout(int M, int D, int F, int dtype) {
    GatedLayout L = x_layout(M, D, F, dtype);
    L.ldi = L.ldf = padded(F, 2, 32);
    L.pack_in = L.ldi != F;
    if (L.pack_in) L.in = L.take((size_t)M * L.ldi * 2);
    L.dg = L.take((size_t)M * L.ldf * 2);
    L.du = L.take((size_t)M * L.ldf * 2);
    L.scaled = dtype == PDR_F16;
    if (L.scaled) L.bound = L.take(3 * kBoundParts * 4);
    L.ldo = padded(D, 2, 16);
    L.pack_out = L.ldo != D;
    if (L.pack_out) L.out = L.take((size_t)M * L.ldo * 2);
    // dW through fp32 partial results, also where only its rows ask for it
    L.splits = gemm_splits(F, D, 2, M);
    L.ldp = padded(D, 4, 16);
    if (L.splits > 1 || D % 8) L.part = L.take((size_t)L.splits * 2 * F * L.ldp * 4);
    return L;
}

// Padded copies of x and the weights, and (backward) of dh.
cudaError_t pack_rows(const GatedLayout &L, const void *&x, const void *&wg, const void *&wu,
                      const void **dh, int M, int D, int F, int e, char *ws, cudaStream_t s) {
    PackJob jobs[4];
    int n = 0;
    if (L.pack_x) {
        jobs[n++] = {x, ws + L.x, M, D, L.ldk, e};
        jobs[n++] = {wg, ws + L.wg, F, D, L.ldk, e};
        jobs[n++] = {wu, ws + L.wu, F, D, L.ldk, e};
        x = ws + L.x;
        wg = ws + L.wg;
        wu = ws + L.wu;
    }
    if (dh && L.pack_in) {
        jobs[n++] = {*dh, ws + L.in, M, F, L.ldi, 2};
        *dh = ws + L.in;
    }
    return launch_pack(jobs, n, s);
}

}  // namespace
}  // namespace pdr

using namespace pdr;

extern "C" {

size_t pdr_gated_workspace_bytes(int M, int D, int F, int dtype, int h_dtype) {
    if (!sizes_ok(M, D, F) || !in_limits(M, D, F) || !(half_type(dtype) || dtype == PDR_E4M3) ||
        !float_type(h_dtype))
        return 0;
    return fwd_layout(M, D, F, dtype, h_dtype).total;
}

pdr_status pdr_gated_fwd(const void *x, const void *w_gate, const void *w_up, int dtype,
                         const float *x_scale, const float *gate_scale, const float *up_scale,
                         int activation, int M, int D, int F, void *h, int h_dtype, void *workspace,
                         size_t workspace_bytes, void *stream) {
    const bool fp8 = dtype == PDR_E4M3;
    if (!sizes_ok(M, D, F) || !(half_type(dtype) || fp8) || !float_type(h_dtype) ||
        !act_ok(activation))
        return PDR_ERR_INVALID_ARG;
    if (!in_limits(M, D, F)) return PDR_ERR_TOO_LARGE;
    if ((M > 0 && (!x || !h)) || !w_gate || !w_up || fp8 != (gate_scale != nullptr) ||
        fp8 != (up_scale != nullptr) || (fp8 ? (M > 0 && !x_scale) : x_scale != nullptr))
        return PDR_ERR_INVALID_ARG;
    if (!aligned_to(x, 16) || !aligned_to(w_gate, 16) || !aligned_to(w_up, 16) ||
        !aligned_to(x_scale, 4) || !aligned_to(gate_scale, 4) || !aligned_to(up_scale, 4) ||
        !aligned_to(h, 16))
        return PDR_ERR_INVALID_ARG;
    const GatedLayout L = fwd_layout(M, D, F, dtype, h_dtype);
    if (L.total && (!workspace || !aligned_to(workspace, 256))) return PDR_ERR_INVALID_ARG;
    if (workspace_bytes < L.total) return PDR_ERR_WORKSPACE_TOO_SMALL;
    if (wait_error_pending()) return PDR_ERR_DEVICE_TIMEOUT;
    if (M == 0) return PDR_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (pack_rows(L, x, w_gate, w_up, nullptr, M, D, F, dtype_bytes(dtype), static_cast<char *>(workspace),
                  s) != cudaSuccess)
        return PDR_ERR_CUDA;
    GemmArgs g;
    g.mode = kDualB;
    g.epi = kEpiGated;
    g.dtype = dtype;
    g.M = M;
    g.N = F;
    g.K[0] = D;
    g.a[0] = {x, M, D, L.ldk};
    g.b[0] = {w_gate, F, D, L.ldk};
    g.b[1] = {w_up, F, D, L.ldk};
    g.act = activation;
    g.scale_m = x_scale;
    g.scale_n = gate_scale;
    g.scale_n2 = up_scale;
    char *out = static_cast<char *>(workspace) + L.out;
    g.out = L.pack_out ? out : h;
    g.out_dtype = h_dtype;
    g.ldo = L.ldo;
    cudaError_t e = launch_gemm(g, s);
    if (e == cudaSuccess && L.pack_out)
        e = launch_unpack(out, M, F, L.ldo, dtype_bytes(h_dtype), h, s);
    return done(e);
}

size_t pdr_gated_bwd_workspace_bytes(int M, int D, int F, int dtype) {
    if (!sizes_ok(M, D, F) || !in_limits(M, D, F) || !half_type(dtype)) return 0;
    return bwd_layout(M, D, F, dtype).total;
}

pdr_status pdr_gated_bwd(const void *grad, const void *x, const void *w_gate, const void *w_up,
                         int dtype, int activation, int M, int D, int F, void *grad_x,
                         void *grad_gate, void *grad_up, void *workspace, size_t workspace_bytes,
                         void *stream) {
    if (!sizes_ok(M, D, F) || !half_type(dtype) || !act_ok(activation)) return PDR_ERR_INVALID_ARG;
    if (!in_limits(M, D, F)) return PDR_ERR_TOO_LARGE;
    if ((M > 0 && (!grad || !x)) || !w_gate || !w_up || !grad_gate != !grad_up)
        return PDR_ERR_INVALID_ARG;
    if (!aligned_to(grad, 32) || !aligned_to(x, 16) || !aligned_to(w_gate, 16) ||
        !aligned_to(w_up, 16) || !aligned_to(grad_x, 16) || !aligned_to(grad_gate, 16) ||
        !aligned_to(grad_up, 16))
        return PDR_ERR_INVALID_ARG;
    const GatedLayout L = bwd_layout(M, D, F, dtype);
    if (L.total && (!workspace || !aligned_to(workspace, 256))) return PDR_ERR_INVALID_ARG;
    if (workspace_bytes < L.total) return PDR_ERR_WORKSPACE_TOO_SMALL;
    if (wait_error_pending()) return PDR_ERR_DEVICE_TIMEOUT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (M == 0) {
        if (grad_gate) e = cudaMemsetAsync(grad_gate, 0, (size_t)F * D * 2, s);
        if (e == cudaSuccess && grad_up) e = cudaMemsetAsync(grad_up, 0, (size_t)F * D * 2, s);
        return done(e);
    }
    if (!grad_x && !grad_gate) return PDR_OK;
    char *ws = static_cast<char *>(workspace);
    Bound bound;
    if (L.scaled) {
        const BoundJob jobs[3] = {{grad, nullptr, (long long)M * F, dtype},
                                  {x, nullptr, (long long)M * D, dtype},
                                  {w_gate, w_up, (long long)F * D, dtype}};
        float *parts = reinterpret_cast<float *>(ws + L.bound);
        if (launch_largest(jobs, 3, parts, s) != cudaSuccess) return PDR_ERR_CUDA;
        bound = {parts, 3, (float)D};
    }
    if (pack_rows(L, x, w_gate, w_up, &grad, M, D, F, 2, ws, s) != cudaSuccess) return PDR_ERR_CUDA;
    const Operand ox = {x, M, D, L.ldk}, og = {w_gate, F, D, L.ldk}, ou = {w_up, F, D, L.ldk};
    const Operand odg = {ws + L.dg, M, F, L.ldf}, odu = {ws + L.du, M, F, L.ldf};
    {
        GemmArgs g;
        g.mode = kDualB;
        g.epi = kEpiGatedBwd;
        g.dtype = dtype;
        g.M = M;
        g.N = F;
        g.K[0] = D;
        g.a[0] = ox;
        g.b[0] = og;
        g.b[1] = ou;
        g.act = activation;
        g.in = grad;
        g.in_dtype = dtype;
        g.ldi = L.ldi;
        g.out = ws + L.dg;
        g.out2 = ws + L.du;
        g.out_dtype = dtype;
        g.ldo = L.ldf;
        g.bound = bound;
        e = launch_gemm(g, s);
    }
    GemmArgs gx, gw;  // dx = dg Wg + du Wu; dWg = dg^T x and dWu = du^T x
    gx.mode = kTwoSources;
    gw.mode = kBatchA;
    gx.dtype = gw.dtype = dtype;
    gx.bound = gw.bound = bound;
    gx.a[0] = gw.a[0] = odg;
    gx.a[1] = gw.a[1] = odu;
    gx.b[0] = og;
    gx.b[1] = ou;
    gw.b[0] = ox;
    gx.b_mn = gw.a_mn = gw.b_mn = true;
    gx.M = M;
    gw.M = F;
    gx.N = gw.N = D;
    gx.K[0] = gx.K[1] = F;
    gw.K[0] = M;
    gx.out = L.pack_out ? ws + L.out : grad_x;
    gx.out_dtype = dtype;
    gx.ldo = L.ldo;
    const bool partial = L.splits > 1 || D % 8;
    const long long n = F * L.ldp;
    float *part = reinterpret_cast<float *>(ws + L.part);
    gw.splits = L.splits;
    if (partial) {
        gw.out = part;
        gw.out_dtype = PDR_F32;
        gw.ldo = L.ldp;
        gw.out_z = n;
        gw.out_split = 2 * n;
    } else {
        gw.out = grad_gate;
        gw.out2 = grad_up;
        gw.out_dtype = dtype;
        gw.ldo = D;
    }
    if (e == cudaSuccess && grad_x && grad_gate)
        e = launch_gemm2(gx, gw, s);
    else if (e == cudaSuccess)
        e = launch_gemm(grad_x ? gx : gw, s);
    if (e == cudaSuccess && grad_x && L.pack_out) e = launch_unpack(ws + L.out, M, D, L.ldo, 2, grad_x, s);
    if (e == cudaSuccess && grad_gate && partial)
        e = launch_join(part, L.splits, F, D, L.ldp, n, grad_gate, grad_up, dtype, {}, s);
    return done(e);
}

}  // extern "C"
