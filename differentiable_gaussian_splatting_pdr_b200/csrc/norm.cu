// rms_norm: s = x + r, y = s / sqrt(mean s^2 + eps) * w, y optionally in 8 bits
// with a scale per row; its gradients; and the same 8-bit rows without the
// norm (include/pdr.h).
//
// One pass over the data: a row's elements stay in the registers of the T
// threads that share it (16 per thread; T a power of two, so that a shuffle
// tree, across warps through shared memory, forms its sums).  The forward
// normalises the unrounded fp32 sum x + r.  The backward, with
//   n = s rstd,  p = dy w:   dx = rstd (p - n mean(p n)) + ds,  dw = sum dy n,
// forms rstd again from the row it reads anyway (nothing is saved), and keeps
// dw of its columns in registers over all rows of a block: one partial row
// per block, added in block order (bitwise reproducible).  Everything is
// bound by memory traffic.
#include <cuda_fp8.h>

#include "gemm.cuh"

namespace pdr {
namespace {

constexpr int kPer = 16;              // row elements per thread
constexpr float kE4M3Max = 448.0f;    // largest finite e4m3 value
constexpr float kMinScale = 1.17549435082228751e-38f;  // 2^-126

struct NormArgs {
    const void *x, *r;      // rows and what is added to them (or null)
    const void *w;          // null: no norm (quantize_rows)
    void *s, *y;            // x + r (or null), result
    float *scale;           // e4m3 result: scale of each row
    int dtype, w_dtype, y_dtype;
    float eps;
    long long M;
    int D, T;
};

struct NormBwdArgs {
    const void *dy, *s, *w, *ds;
    void *dx;
    float *dw;              // [blocks][D] partial sums
    int dtype, w_dtype;
    float eps;
    long long M;
    int D, T;
};

// The elements that thread t of a row's T threads holds: vectors of E
// neighbours, T vectors apart (E = 1: single elements, any alignment).
template <int E>
__device__ __forceinline__ int element(int j, int t, int T) {
    return ((j / E) * T + t) * E + j % E;
}

template <int E>
__device__ __forceinline__ void load_row(const void *p, size_t at, int D, int t, int T, int dtype,
                                         float (&v)[kPer]) {
#pragma unroll
    for (int j = 0; j < kPer; j += E) {
        const int c = element<E>(j, t, T);
        if (c < D) {
            if constexpr (E == 1) {
                v[j] = img_load(p, at + c, dtype);
            } else if constexpr (E == 4) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at + c));
                v[j] = f.x; v[j + 1] = f.y; v[j + 2] = f.z; v[j + 3] = f.w;
            } else {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const unsigned short *>(p) + at + c));
                const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = unpack2(w[i], dtype);
                    v[j + 2 * i] = f.x;
                    v[j + 2 * i + 1] = f.y;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) v[j + i] = 0.0f;
        }
    }
}

__device__ __forceinline__ unsigned short e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

template <int E>
__device__ __forceinline__ void store_row(void *p, size_t at, int D, int t, int T, int dtype,
                                          const float (&v)[kPer]) {
#pragma unroll
    for (int j = 0; j < kPer; j += E) {
        const int c = element<E>(j, t, T);
        if (c >= D) continue;
        if constexpr (E == 1) {
            if (dtype == PDR_E4M3)
                static_cast<unsigned char *>(p)[at + c] = (unsigned char)e4m3x2(v[j], 0.0f);
            else
                img_store(p, at + c, dtype, v[j]);
        } else if (dtype == PDR_E4M3) {
            unsigned w[2] = {};
#pragma unroll
            for (int i = 0; i < E / 2; ++i)
                w[i / 2] |= (unsigned)e4m3x2(v[j + 2 * i], v[j + 2 * i + 1]) << (16 * (i & 1));
            unsigned char *q = static_cast<unsigned char *>(p) + at + c;
            if constexpr (E == 8)
                *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<unsigned *>(q) = w[0];
        } else if (dtype == PDR_F32) {
#pragma unroll
            for (int i = 0; i < E; i += 4)
                *reinterpret_cast<float4 *>(static_cast<float *>(p) + at + c + i) =
                    make_float4(v[j + i], v[j + i + 1], v[j + i + 2], v[j + i + 3]);
        } else {
            unsigned w[E / 2];
#pragma unroll
            for (int i = 0; i < E / 2; ++i) w[i] = pack2(v[j + 2 * i], v[j + 2 * i + 1], dtype);
            unsigned short *q = static_cast<unsigned short *>(p) + at + c;
            if constexpr (E == 8)
                *reinterpret_cast<uint4 *>(q) = make_uint4(w[0], w[1], w[2], w[3]);
            else
                *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
        }
    }
}

// Sum (or maximum) over the T threads of a row, for all of them; the whole
// block calls it.  `red`: one float per warp.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, int T, float *red) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        if (d < T) {
            const float o = __shfl_xor_sync(0xffffffffu, v, d);
            v = MAX ? max_nan(v, o) : v + o;
        }
    if (T > 32) {
        const int warp = threadIdx.x >> 5, first = (threadIdx.x & ~(T - 1)) >> 5;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        __syncthreads();
        v = red[first];
        for (int i = 1; i < T >> 5; ++i) v = MAX ? max_nan(v, red[first + i]) : v + red[first + i];
    }
    return v;
}

template <int E>
__global__ void __launch_bounds__(1024) k_rms_norm(const NormArgs a) {
    __shared__ float red[32];
    grid_dep_wait();
    const int T = a.T, t = threadIdx.x & (T - 1), per_block = blockDim.x / T;
    const int D = a.D;
    float w[kPer];
    if (a.w) {
        if (a.w_dtype == a.dtype)
            load_row<E>(a.w, 0, D, t, T, a.dtype, w);
        else  // fp32 weights of 16-bit rows
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int c = element<E>(j, t, T);
                w[j] = c < D ? img_load(a.w, c, a.w_dtype) : 0.0f;
            }
    }
    for (long long base = (long long)blockIdx.x * per_block; base < a.M;
         base += (long long)gridDim.x * per_block) {
        const long long row = base + threadIdx.x / T;
        const int d = row < a.M ? D : 0;  // nothing of rows behind the last
        const size_t at = (size_t)row * D;
        float v[kPer];
        load_row<E>(a.x, at, d, t, T, a.dtype, v);
        if (a.r) {
            float r[kPer];
            load_row<E>(a.r, at, d, t, T, a.dtype, r);
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] += r[j];
            if (a.s) store_row<E>(a.s, at, d, t, T, a.dtype, v);
        }
        if (a.w) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) ss = fmaf(v[j], v[j], ss);
            ss = row_reduce<false>(ss, T, red);
            const float rstd = rsqrtf(ss / (float)D + a.eps);
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] *= rstd * w[j];
        }
        if (a.scale) {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) m = max_nan(m, fabsf(v[j]));
            m = row_reduce<true>(m, T, red);
            const float scale = max_nan(m / kE4M3Max, kMinScale), inv = 1.0f / scale;
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] *= inv;
            if (t == 0 && d) a.scale[row] = scale;
        }
        store_row<E>(a.y, at, d, t, T, a.y_dtype, v);
    }
}

template <int E>
__global__ void __launch_bounds__(1024) k_rms_norm_bwd(const NormBwdArgs a) {
    extern __shared__ float part[];  // [rows of a block][T * kPer] when there are several
    __shared__ float red[32];
    grid_dep_wait();
    const int T = a.T, t = threadIdx.x & (T - 1), per_block = blockDim.x / T;
    const int D = a.D;
    float w[kPer], dw[kPer];
    if (a.w_dtype == a.dtype)
        load_row<E>(a.w, 0, D, t, T, a.dtype, w);
    else
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int c = element<E>(j, t, T);
            w[j] = c < D ? img_load(a.w, c, a.w_dtype) : 0.0f;
        }
#pragma unroll
    for (int j = 0; j < kPer; ++j) dw[j] = 0.0f;
    for (long long base = (long long)blockIdx.x * per_block; base < a.M;
         base += (long long)gridDim.x * per_block) {
        const long long row = base + threadIdx.x / T;
        const int d = row < a.M ? D : 0;
        const size_t at = (size_t)row * D;
        float v[kPer], g[kPer];
        load_row<E>(a.s, at, d, t, T, a.dtype, v);
        load_row<E>(a.dy, at, d, t, T, a.dtype, g);
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) ss = fmaf(v[j], v[j], ss);
        ss = row_reduce<false>(ss, T, red);
        const float rstd = rsqrtf(ss / (float)D + a.eps);
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            v[j] *= rstd;
            dw[j] = fmaf(g[j], v[j], dw[j]);
            g[j] *= w[j];
            dot = fmaf(g[j], v[j], dot);
        }
        dot = row_reduce<false>(dot, T, red) / (float)D;
#pragma unroll
        for (int j = 0; j < kPer; ++j) g[j] = rstd * fmaf(-v[j], dot, g[j]);
        if (a.ds) {
            load_row<E>(a.ds, at, d, t, T, a.dtype, v);
#pragma unroll
            for (int j = 0; j < kPer; ++j) g[j] += v[j];
        }
        if (a.dx) store_row<E>(a.dx, at, d, t, T, a.dtype, g);
    }
    if (!a.dw) return;
    // The block's rows, in order; then one partial row per block.
    const int width = T * kPer, sub = threadIdx.x / T;
    if (per_block > 1) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) part[sub * width + element<E>(j, t, T)] = dw[j];
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += blockDim.x) {
            float s = 0.0f;
            for (int i = 0; i < per_block; ++i) s += part[i * width + c];
            a.dw[(size_t)blockIdx.x * D + c] = s;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int c = element<E>(j, t, T);
            if (c < D) a.dw[(size_t)blockIdx.x * D + c] = dw[j];
        }
    }
}

bool half_type(int t) { return t == PDR_F16 || t == PDR_BF16; }
bool float_type(int t) { return t == PDR_F32 || half_type(t); }

// Threads per row, block size and blocks for M rows of D elements.
struct NormShape {
    int T, threads, blocks;
};
NormShape norm_shape(long long M, int D, int per_sm) {
    NormShape n;
    n.T = 1;
    while (n.T * kPer < D) n.T *= 2;
    n.threads = n.T > 256 ? n.T : 256;
    const long long per_block = n.threads / n.T, need = (M + per_block - 1) / per_block;
    long long most = (long long)kSMs * per_sm * 256 / n.threads;
    if (most < kSMs) most = kSMs;
    n.blocks = (int)(need < most ? need : most);
    return n;
}
constexpr int kFwdPerSm = 8, kBwdPerSm = 4;  // blocks of 256 threads per SM

// Every row of each of the tensors starts at a multiple of 16 bytes.
bool rows_aligned(std::initializer_list<const void *> ps, int D, int dtype) {
    for (const void *p : ps)
        if (!aligned_to(p, 16)) return false;
    return (long long)D * dtype_bytes(dtype) % 16 == 0;
}

pdr_status run_fwd(NormArgs a, cudaStream_t s) {
    const NormShape n = norm_shape(a.M, a.D, kFwdPerSm);
    a.T = n.T;
    const bool vec = rows_aligned({a.x, a.r, a.s, a.y, a.w_dtype == a.dtype ? a.w : nullptr}, a.D, a.dtype);
    const dim3 grid((unsigned)n.blocks), block((unsigned)n.threads);
    cudaError_t e;
    if (!vec)
        e = launch_dependent(k_rms_norm<1>, grid, block, 0, s, a);
    else if (a.dtype == PDR_F32)
        e = launch_dependent(k_rms_norm<4>, grid, block, 0, s, a);
    else
        e = launch_dependent(k_rms_norm<8>, grid, block, 0, s, a);
    return e == cudaSuccess ? PDR_OK : PDR_ERR_CUDA;
}

bool norm_sizes(int M, int D) { return M >= 0 && D >= 1; }
bool norm_in_limits(int M, int D) { return M <= PDR_MAX_ROWS && D <= PDR_MAX_NORM_FEATURES; }

}  // namespace
}  // namespace pdr

using namespace pdr;

extern "C" {

pdr_status pdr_rms_norm_fwd(const void *x, const void *residual, int dtype, const void *weight,
                            int weight_dtype, float eps, int M, int D, void *sum, void *y,
                            int y_dtype, float *y_scale, void *stream) {
    if (!norm_sizes(M, D) || !float_type(dtype) || !(weight_dtype == dtype || weight_dtype == PDR_F32) ||
        !(y_dtype == dtype || y_dtype == PDR_E4M3) || !(eps >= 0.0f))
        return PDR_ERR_INVALID_ARG;
    if (!norm_in_limits(M, D)) return PDR_ERR_TOO_LARGE;
    if (!weight || (M > 0 && (!x || !y)) || (M > 0 && (y_dtype == PDR_E4M3) != (y_scale != nullptr)) ||
        (!residual && sum))
        return PDR_ERR_INVALID_ARG;
    const int e = dtype_bytes(dtype);
    if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(sum, e) ||
        !aligned_to(weight, dtype_bytes(weight_dtype)) || !aligned_to(y, dtype_bytes(y_dtype)) ||
        !aligned_to(y_scale, 4))
        return PDR_ERR_INVALID_ARG;
    if (M == 0) return PDR_OK;
    return run_fwd({x, residual, weight, sum, y, y_scale, dtype, weight_dtype, y_dtype, eps, M, D, 0},
                   static_cast<cudaStream_t>(stream));
}

pdr_status pdr_quantize_rows(const void *x, int dtype, int M, int D, void *y, float *y_scale,
                             void *stream) {
    if (!norm_sizes(M, D) || !float_type(dtype)) return PDR_ERR_INVALID_ARG;
    if (!norm_in_limits(M, D)) return PDR_ERR_TOO_LARGE;
    if (M > 0 && (!x || !y || !y_scale)) return PDR_ERR_INVALID_ARG;
    if (!aligned_to(x, dtype_bytes(dtype)) || !aligned_to(y_scale, 4)) return PDR_ERR_INVALID_ARG;
    if (M == 0) return PDR_OK;
    return run_fwd({x, nullptr, nullptr, nullptr, y, y_scale, dtype, dtype, PDR_E4M3, 0.0f, M, D, 0},
                   static_cast<cudaStream_t>(stream));
}

size_t pdr_rms_norm_bwd_workspace_bytes(int M, int D) {
    if (!norm_sizes(M, D) || !norm_in_limits(M, D)) return 0;
    return align256((size_t)norm_shape(M, D, kBwdPerSm).blocks * D * 4);
}

pdr_status pdr_rms_norm_bwd(const void *grad, const void *sum, int dtype, const void *weight,
                            int weight_dtype, const void *grad_sum, float eps, int M, int D,
                            void *grad_x, void *grad_weight, void *workspace,
                            size_t workspace_bytes, void *stream) {
    if (!norm_sizes(M, D) || !float_type(dtype) || !(weight_dtype == dtype || weight_dtype == PDR_F32) ||
        !(eps >= 0.0f))
        return PDR_ERR_INVALID_ARG;
    if (!norm_in_limits(M, D)) return PDR_ERR_TOO_LARGE;
    if (!weight || (M > 0 && (!grad || !sum))) return PDR_ERR_INVALID_ARG;
    const int e = dtype_bytes(dtype), we = dtype_bytes(weight_dtype);
    if (!aligned_to(grad, e) || !aligned_to(sum, e) || !aligned_to(grad_sum, e) ||
        !aligned_to(grad_x, e) || !aligned_to(weight, we) || !aligned_to(grad_weight, we))
        return PDR_ERR_INVALID_ARG;
    const size_t need = pdr_rms_norm_bwd_workspace_bytes(M, D);
    if (need && grad_weight && (!workspace || !aligned_to(workspace, 256))) return PDR_ERR_INVALID_ARG;
    if (grad_weight && workspace_bytes < need) return PDR_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (M == 0) {
        if (grad_weight) err = cudaMemsetAsync(grad_weight, 0, (size_t)D * we, s);
        return err == cudaSuccess ? PDR_OK : PDR_ERR_CUDA;
    }
    if (!grad_x && !grad_weight) return PDR_OK;
    const NormShape n = norm_shape(M, D, kBwdPerSm);
    const NormBwdArgs a = {grad, sum, weight, grad_sum, grad_x,
                           grad_weight ? static_cast<float *>(workspace) : nullptr,
                           dtype, weight_dtype, eps, M, D, n.T};
    const bool vec = rows_aligned({grad, sum, grad_sum, grad_x, weight_dtype == dtype ? weight : nullptr}, D, dtype);
    const dim3 grid((unsigned)n.blocks), block((unsigned)n.threads);
    const size_t smem = n.threads > n.T ? (size_t)n.threads * kPer * 4 : 0;  // 16 KB
    if (!vec)
        err = launch_dependent(k_rms_norm_bwd<1>, grid, block, smem, s, a);
    else if (dtype == PDR_F32)
        err = launch_dependent(k_rms_norm_bwd<4>, grid, block, smem, s, a);
    else
        err = launch_dependent(k_rms_norm_bwd<8>, grid, block, smem, s, a);
    if (err == cudaSuccess && grad_weight)
        err = launch_join_columns(static_cast<const float *>(workspace), n.blocks, D, grad_weight,
                                  weight_dtype, s);
    return err == cudaSuccess ? PDR_OK : PDR_ERR_CUDA;
}

}  // extern "C"
