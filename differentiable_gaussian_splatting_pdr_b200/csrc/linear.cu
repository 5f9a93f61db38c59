// linear: y = act(x W^T + b) + r, and its gradients (include/pdr.h).
//
// Forward: one tensor-core product over rows of x and rows of W, both
// contiguous along k; scales, bias, activation and residual are applied to the
// fp32 sums in the epilogue, and y is rounded once.
//
// Backward, with dz = dy act'(z):
//   dz  without an activation dz is dy: read in place where its type and row
//       length allow, else cast once; with one, z = x W^T + b is formed again
//       and dz leaves that product's epilogue (nothing is saved by the
//       forward: at widths up to about 1000 forming z again costs less time
//       than writing and reading it, and no memory);
//   db  sums of dy act'(z) in fp32 before any rounding: per 32-row group in
//       the epilogue (or per block that reads dy), then over the groups in order;
//   dx  = dz W     (W read with its k as rows: an MN-major operand);
//   dW  = dz^T x   (both operands MN-major), k split over the machine, fp32
//       partial results added in order: bitwise reproducible.  In one launch with dx.
// dz is rounded to x's type: it is an operand of 16-bit products, whose
// results are rounded to that type too.  Gradients of a loss that is a mean are far below
// fp16's range (1e-6 for the parameters of a 512 x 512 frame), others may lie above it, and
// dW's sums inside it all the same: an fp16 dz of another type's dy, or of a slope, is
// taken times a power of two that brings the largest |dy| to 2^14 (one more pass over dy:
// k_largest), and dx and dW are formed without it from the fp32 sums.  (16384 x 256 to 1024
// with silu and a cold L2 76 us, without the factor 68.)
// Of an fp32 dy with up to 32 columns (the head's, from the renderer) what the rounding leaves
// is kept in 16 bits too, beside dz: dx's block of 64 k (over W twice) and dW's tile of 256
// rows have room for both, so that dx and dW are rounded once (65536 x 512 to 6:
// 45 us with and without, with the rest as a second block of k 49).
#include "gemm.cuh"

namespace pdr {
namespace {

// The workspace: padded copies of what TMA or 32-byte loads cannot address (rows
// that are no multiple of 16 bytes; of the residual or of dy, of 32), padded
// results that are copied out at the end, dz, and partial sums.
struct LinearLayout {
    size_t x, w, w2, in, out, dz, colsum, part, bound, total;
    long long ldk, ldi, ldo, ldz, ldp, sum_rows;
    bool pack_x, pack_in, pack_out, narrow, cast, scaled;
    int splits, low;  // low: where in a row of dz the rounding's rest is (0: nowhere)
    size_t take(size_t bytes) {
        const size_t at = total;
        total += align256(bytes);
        return at;
    }
};

bool linear_sizes(int M, int N, int K) { return M >= 0 && N >= 1 && K >= 1; }
bool linear_in_limits(int M, int N, int K) {
    return M <= PDR_MAX_ROWS && N <= PDR_MAX_FEATURES && K <= PDR_MAX_FEATURES;
}

LinearLayout fwd_layout(int M, int N, int K, int dtype, int y_dtype, bool residual) {
    LinearLayout L = {};
    const int e = dtype_bytes(dtype), o = dtype_bytes(y_dtype);
    L.ldk = padded(K, e, 16);
    L.pack_x = L.ldk != K;
    if (L.pack_x) {
        L.x = L.take((size_t)M * L.ldk * e);
        L.w = L.take((size_t)N * L.ldk * e);
    }
    L.ldi = L.ldo = N;
    L.narrow = gemm_narrow(N, y_dtype, residual);
    if (L.narrow) return L;
    L.ldi = padded(N, o, 32);
    L.ldo = padded(N, o, 16);
    L.pack_in = residual && L.ldi != N;
    L.pack_out = L.ldo != N;
    if (L.pack_in) L.in = L.take((size_t)M * L.ldi * o);
    if (L.pack_out) L.out = L.take((size_t)M * L.ldo * o);
    return L;
}

LinearLayout bwd_layout(int M, int N, int K, int dtype, int grad_dtype, int act) {
    LinearLayout L = {};
    L.ldk = padded(K, 2, 16);
    L.pack_x = L.ldk != K;
    if (L.pack_x) {
        L.x = L.take((size_t)M * L.ldk * 2);
        L.w = L.take((size_t)N * L.ldk * 2);
    }
    const int ge = dtype_bytes(grad_dtype);
    L.ldi = padded(N, ge, 32);
    L.pack_in = act != PDR_ACT_NONE && L.ldi != N;
    if (L.pack_in) L.in = L.take((size_t)M * L.ldi * ge);
    L.cast = act != PDR_ACT_NONE || grad_dtype != dtype || N % 8 != 0;
    L.ldz = L.cast ? padded(N, 2, 32) : N;
    if (act == PDR_ACT_NONE && grad_dtype == PDR_F32 && N <= 32) {
        L.low = (int)padded(N, 2, 16);
        L.ldz = 2 * L.low;
        L.w2 = L.take((size_t)L.ldz * L.ldk * 2);
    }
    if (L.cast) L.dz = L.take((size_t)M * L.ldz * 2);
    L.scaled = dtype == PDR_F16 && (act != PDR_ACT_NONE || grad_dtype != dtype);
    if (L.scaled) L.bound = L.take(kBoundParts * 4);
    L.narrow = gemm_narrow(K, dtype, false);  // dx
    L.ldo = L.narrow ? K : padded(K, 2, 16);
    L.pack_out = L.ldo != K;
    if (L.pack_out) L.out = L.take((size_t)M * L.ldo * 2);
    L.sum_rows = act != PDR_ACT_NONE ? 4 * (((long long)M + 127) / 128) : column_groups(M, N, grad_dtype, L.low);
    L.colsum = L.take((size_t)L.sum_rows * N * 4);
    // dW through fp32 partial results, also where only its rows ask for it
    L.splits = gemm_splits(N, K, 1, M);
    L.ldp = padded(K, 4, 16);
    if (L.splits > 1 || K % 8 || L.low) L.part = L.take((size_t)L.splits * (L.low ? 2 * L.low : N) * L.ldp * 4);
    return L;
}

}  // namespace
}  // namespace pdr

using namespace pdr;

extern "C" {

size_t pdr_linear_workspace_bytes(int M, int N, int K, int dtype, int y_dtype, int has_residual) {
    if (!linear_sizes(M, N, K) || !linear_in_limits(M, N, K) ||
        !(half_type(dtype) || dtype == PDR_E4M3) || !float_type(y_dtype))
        return 0;
    return fwd_layout(M, N, K, dtype, y_dtype, has_residual != 0).total;
}

pdr_status pdr_linear_fwd(const void *x, const void *weight, int dtype, const float *x_scale,
                          const float *weight_scale, const void *bias, int bias_dtype,
                          const void *residual, int activation, int M, int N, int K, void *y,
                          int y_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    const bool fp8 = dtype == PDR_E4M3;
    if (!linear_sizes(M, N, K) || !(half_type(dtype) || fp8) || !float_type(y_dtype) ||
        !act_ok(activation))
        return PDR_ERR_INVALID_ARG;
    if (!linear_in_limits(M, N, K)) return PDR_ERR_TOO_LARGE;
    if ((M > 0 && (!x || !y)) || !weight || fp8 != (weight_scale != nullptr) ||
        (fp8 ? (M > 0 && !x_scale) : x_scale != nullptr))
        return PDR_ERR_INVALID_ARG;
    if (bias && !float_type(bias_dtype)) return PDR_ERR_INVALID_ARG;
    if (!aligned_to(x, 16) || !aligned_to(weight, 16) || !aligned_to(x_scale, 4) ||
        !aligned_to(weight_scale, 4) || !aligned_to(y, 16) || !aligned_to(residual, 32) ||
        !aligned_to(bias, bias ? dtype_bytes(bias_dtype) : 1))
        return PDR_ERR_INVALID_ARG;
    const LinearLayout L = fwd_layout(M, N, K, dtype, y_dtype, residual != nullptr);
    if (L.total && (!workspace || !aligned_to(workspace, 256))) return PDR_ERR_INVALID_ARG;
    if (workspace_bytes < L.total) return PDR_ERR_WORKSPACE_TOO_SMALL;
    if (wait_error_pending()) return PDR_ERR_DEVICE_TIMEOUT;
    if (M == 0) return PDR_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    GemmArgs g;
    g.dtype = dtype;
    g.M = M;
    g.N = N;
    g.K[0] = K;
    g.a[0] = {x, M, K, L.ldk};
    g.b[0] = {weight, N, K, L.ldk};
    char *ws = static_cast<char *>(workspace);
    const int e = dtype_bytes(dtype), o = dtype_bytes(y_dtype);
    PackJob jobs[3];
    int n = 0;
    if (L.pack_x) {
        jobs[n++] = {x, ws + L.x, M, K, L.ldk, e};
        jobs[n++] = {weight, ws + L.w, N, K, L.ldk, e};
        g.a[0].p = ws + L.x;
        g.b[0].p = ws + L.w;
    }
    if (L.pack_in) {
        jobs[n++] = {residual, ws + L.in, M, N, L.ldi, o};
        residual = ws + L.in;
    }
    cudaError_t err = launch_pack(jobs, n, s);
    g.narrow = L.narrow;
    g.act = activation;
    g.out = L.pack_out ? ws + L.out : y;
    g.out_dtype = y_dtype;
    g.ldo = L.ldo;
    g.bias = bias;
    g.bias_dtype = bias_dtype;
    g.scale_m = x_scale;
    g.scale_n = weight_scale;
    g.in = residual;
    g.in_dtype = y_dtype;
    g.ldi = L.ldi;
    if (err == cudaSuccess) err = launch_gemm(g, s);
    if (err == cudaSuccess && L.pack_out) err = launch_unpack(ws + L.out, M, N, L.ldo, o, y, s);
    return done(err);
}

size_t pdr_linear_bwd_workspace_bytes(int M, int N, int K, int dtype, int grad_dtype,
                                      int activation) {
    if (!linear_sizes(M, N, K) || !linear_in_limits(M, N, K) || !half_type(dtype) ||
        !float_type(grad_dtype) || !act_ok(activation))
        return 0;
    return bwd_layout(M, N, K, dtype, grad_dtype, activation).total;
}

pdr_status pdr_linear_bwd(const void *grad, int grad_dtype, const void *x, const void *weight,
                          int dtype, const void *bias, int bias_dtype, int activation, int M, int N,
                          int K, void *grad_x, void *grad_weight, void *grad_bias, void *workspace,
                          size_t workspace_bytes, void *stream) {
    if (!linear_sizes(M, N, K) || !half_type(dtype) || !float_type(grad_dtype) || !act_ok(activation))
        return PDR_ERR_INVALID_ARG;
    if (!linear_in_limits(M, N, K)) return PDR_ERR_TOO_LARGE;
    if ((M > 0 && (!grad || !x)) || !weight) return PDR_ERR_INVALID_ARG;
    if ((bias || grad_bias) && !float_type(bias_dtype)) return PDR_ERR_INVALID_ARG;
    const int be = bias || grad_bias ? dtype_bytes(bias_dtype) : 1;
    if (!aligned_to(grad, 32) || !aligned_to(x, 16) || !aligned_to(weight, 16) ||
        !aligned_to(bias, be) || !aligned_to(grad_bias, be) || !aligned_to(grad_x, 16) ||
        !aligned_to(grad_weight, 16))
        return PDR_ERR_INVALID_ARG;
    const LinearLayout L = bwd_layout(M, N, K, dtype, grad_dtype, activation);
    if (L.total && (!workspace || !aligned_to(workspace, 256))) return PDR_ERR_INVALID_ARG;
    if (workspace_bytes < L.total) return PDR_ERR_WORKSPACE_TOO_SMALL;
    if (wait_error_pending()) return PDR_ERR_DEVICE_TIMEOUT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (M == 0) {  // no rows: nothing to add up
        if (grad_weight) e = cudaMemsetAsync(grad_weight, 0, (size_t)N * K * 2, s);
        if (e == cudaSuccess && grad_bias) e = cudaMemsetAsync(grad_bias, 0, (size_t)N * be, s);
        return done(e);
    }
    char *ws = static_cast<char *>(workspace);
    const bool act = activation != PDR_ACT_NONE, products = grad_x || grad_weight;
    if (!products && !grad_bias) return PDR_OK;
    PackJob jobs[3];
    int n = 0;
    if (L.pack_x && (act || grad_weight)) {
        jobs[n++] = {x, ws + L.x, M, K, L.ldk, 2};
        x = ws + L.x;
    }
    if (L.pack_x && (act || grad_x) && !L.low) {
        jobs[n++] = {weight, ws + L.w, N, K, L.ldk, 2};
        weight = ws + L.w;
    }
    if (L.pack_in) jobs[n++] = {grad, ws + L.in, M, N, L.ldi, dtype_bytes(grad_dtype)};
    if (launch_pack(jobs, n, s) != cudaSuccess) return PDR_ERR_CUDA;
    float *colsum = grad_bias ? reinterpret_cast<float *>(ws + L.colsum) : nullptr;
    Bound bound;
    if (L.scaled && (act || products)) {
        const BoundJob job = {grad, nullptr, (long long)M * N, grad_dtype};
        float *parts = reinterpret_cast<float *>(ws + L.bound);
        if (launch_largest(&job, 1, parts, s) != cudaSuccess) return PDR_ERR_CUDA;
        bound = {parts, 1, 1.0f};
    }
    const Operand ox = {x, M, K, L.ldk}, ow = {weight, N, K, L.ldk};
    Operand oz = {L.cast ? ws + L.dz : grad, M, N, L.ldz};
    if (act) {
        GemmArgs g;
        g.epi = kEpiSlope;
        g.dtype = dtype;
        g.a[0] = ox;
        g.b[0] = ow;
        g.M = M;
        g.N = N;
        g.K[0] = K;
        g.act = activation;
        g.bias = bias;
        g.bias_dtype = bias_dtype;
        g.in = L.pack_in ? ws + L.in : grad;
        g.in_dtype = grad_dtype;
        g.ldi = L.ldi;
        g.out = ws + L.dz;
        g.out_dtype = dtype;
        g.ldo = L.ldz;
        g.colsum = colsum;
        g.bound = bound;
        e = launch_gemm(g, s);
    } else if ((L.cast && products) || colsum) {
        TwiceJob two;
        if (L.low && grad_x) two = {weight, ws + L.w2, K, L.ldk};
        e = launch_cast_columns(grad, grad_dtype, M, N, L.cast && products ? ws + L.dz : nullptr,
                                dtype, L.ldz, L.low, two, colsum, bound, s);
    }
    GemmArgs gx, gw;  // dx = dz W, dW = dz^T x
    gx.dtype = gw.dtype = dtype;
    gx.bound = gw.bound = bound;
    gx.a[0] = gw.a[0] = oz;
    gx.b[0] = ow;
    gw.b[0] = ox;
    gx.b_mn = gw.a_mn = gw.b_mn = true;
    gx.M = M;
    gw.M = N;
    gx.N = gw.N = K;
    gx.K[0] = N;
    gw.K[0] = M;
    if (L.low) {  // dx: k over dz and the rest; dW: the rest's rows behind dz's
        gx.a[0].cols = gw.a[0].cols = gx.K[0] = gw.M = 2 * L.low;
        gx.b[0] = {ws + L.w2, 2 * L.low, K, L.ldk};
    }
    gx.narrow = L.narrow;
    gx.out = L.pack_out ? ws + L.out : grad_x;
    gx.out_dtype = dtype;
    gx.ldo = L.ldo;
    const bool partial = L.splits > 1 || K % 8 || L.low;
    gw.splits = L.splits;
    gw.out = partial ? ws + L.part : grad_weight;
    gw.out_dtype = partial ? (int)PDR_F32 : dtype;
    gw.ldo = partial ? L.ldp : K;
    gw.out_split = L.splits > 1 ? gw.M * L.ldp : 0;
    if (e == cudaSuccess && grad_x && grad_weight)
        e = launch_gemm2(gx, gw, s);
    else if (e == cudaSuccess && products)
        e = launch_gemm(grad_x ? gx : gw, s);
    if (e == cudaSuccess && grad_x && L.pack_out) e = launch_unpack(ws + L.out, M, K, L.ldo, 2, grad_x, s);
    ColumnJob db;
    if (colsum) db = {colsum, L.sum_rows, N, grad_bias, bias_dtype};
    if (e == cudaSuccess && grad_weight && partial)
        e = launch_join(reinterpret_cast<float *>(ws + L.part), L.low ? 2 * L.splits : L.splits, N, K, L.ldp,
                        (L.low ? L.low : N) * L.ldp, grad_weight, nullptr, dtype, db, s);
    else if (e == cudaSuccess && colsum)
        e = launch_join_columns(db, s);
    return done(e);
}

pdr_status pdr_set_wait_limit(int tries) {
    set_wait_tries(tries);
    return PDR_OK;
}

pdr_status pdr_check_wait_error(void *stream) {
    int bits = 0;
    if (read_wait_error(&bits, static_cast<cudaStream_t>(stream)) != cudaSuccess) return PDR_ERR_CUDA;
    return bits ? PDR_ERR_DEVICE_TIMEOUT : PDR_OK;
}

}  // extern "C"
