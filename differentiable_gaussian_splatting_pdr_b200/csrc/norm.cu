// rms_norm: s = x + r, y = s / sqrt(mean s^2 + eps) * w, y optionally in 8 bits
// with a scale per row; its gradients; and the same 8-bit rows without the
// norm (include/pdr.h).
//
// One pass over the data: a row's elements stay in the registers of the T
// threads that share it (16 per thread; T a power of two or whole warps, so that a
// shuffle tree, across warps through shared memory, forms its sums).  The forward
// normalises the unrounded fp32 sum x + r.  The backward, with
//   n = s rstd,  p = dy w:   dx = rstd (p - n mean(p n)) + ds,  dw = sum dy n,
// forms rstd again from the row it reads anyway (nothing is saved), and keeps
// dw of its columns in registers over all rows of a block: one partial row
// per block, added in block order (bitwise reproducible).  Everything is
// bound by memory traffic: the next row's loads are under way while a row is
// computed.  65536 x 512 bf16 plus a residual to 8 bits: 41 us, 5.8 TB/s; backward of
// 81920 x 512 with the sum's gradient 61 us, 5.5 TB/s.
#include <cuda_fp8.h>
#include <stdint.h>

#include "gemm.cuh"

namespace pdr {
namespace {

constexpr int kPer = 16;              // row elements per thread
// Threads per SM (a thread's share of an fp32 row takes twice the registers): 16384 x 333 in
// fp32 took 15.0 us with 512 against 18.7 with 768, 65536 x 512 in bf16 to 8 bits 41.0
// with 768 against 44.9 with 1024.
constexpr int kFwdThreads = 768, kFwdThreads32 = 512, kBwdThreads = 512;
constexpr float kE4M3Max = 448.0f;    // largest finite e4m3 value
constexpr float kMinScale = 1.17549435082228751e-38f;  // 2^-126

struct NormArgs {
    const void *x, *r;      // rows and what is added to them (or null)
    const void *w;          // null: no norm (quantize_rows)
    void *s, *y;            // x + r (or null), result
    float *scale;           // e4m3 result: scale of each row
    int dtype, w_dtype, y_dtype;
    float eps, inv_d;       // inv_d: 1 / D
    long long M;
    int D, T;
};

struct NormBwdArgs {
    const void *dy, *s, *w, *ds;
    void *dx;
    float *dw;              // [blocks][D] partial sums
    int dtype, w_dtype;
    float eps, inv_d;       // inv_d: 1 / D
    long long M;
    int D, T;
};

// A row as its T threads share it: vectors of E neighbours (16 bytes), T vectors
// apart.  Rows whose length is no multiple of 16 bytes (SHIFT) start `shift`
// elements into a vector; the vectors at their ends belong to the neighbouring
// rows too.  A thread's rows are a multiple of 8 apart, so that its shift, and
// hence its columns, stay the same.
template <int E, bool SHIFT>
struct Row {
    int D, t, T, shift;
    long long total;  // elements of the tensor
    __device__ __forceinline__ int column(int j) const {  // of the thread's element j
        const int c = ((j / E) * T + t) * E + j % E;
        return SHIFT ? c - shift : c;
    }
    __device__ __forceinline__ bool inside(int c) const {
        return (!SHIFT || c >= 0) && c < D;
    }
};

// A thread's share of a row as it lies in memory.
template <int E>
struct Raw {
    unsigned w[E == 8 ? kPer / 2 : kPer];
};

// 16 bytes where `on`, else zeros.  (volatile: the compiler leaves it where it is,
// ahead of the row's arithmetic; predicated: without a branch around each load.)
__device__ __forceinline__ uint4 load16(bool on, const void *p) {
    uint4 u = make_uint4(0, 0, 0, 0);
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n"
        " @p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
        : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w)
        : "l"(p), "r"((unsigned)on));
    return u;
}

template <int E, bool SHIFT>
__device__ __forceinline__ void fetch(Raw<E> &raw, const void *p, long long row, bool on,
                                      const Row<E, SHIFT> &q) {
    const long long at = row * q.D;
#pragma unroll
    for (int j = 0; j < kPer; j += E) {
        const int c = q.column(j);
        const bool some = on && c < q.D && (!SHIFT || c > -E);  // some of it is of the row
        const bool whole = !SHIFT || at + c + E <= q.total;
        uint4 u = load16(some && whole, static_cast<const char *>(p) + (at + c) * (E == 8 ? 2 : 4));
        if (SHIFT && some && !whole) {  // the tensor's last elements
            unsigned w[4] = {};
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (q.inside(c + i)) {
                    if constexpr (E == 8)
                        w[i / 2] |= (unsigned)static_cast<const unsigned short *>(p)[at + c + i] << (16 * (i & 1));
                    else
                        w[i] = static_cast<const unsigned *>(p)[at + c + i];
                }
            u = make_uint4(w[0], w[1], w[2], w[3]);
        }
        raw.w[4 * (j / E)] = u.x;
        raw.w[4 * (j / E) + 1] = u.y;
        raw.w[4 * (j / E) + 2] = u.z;
        raw.w[4 * (j / E) + 3] = u.w;
    }
}

template <int E>
__device__ __forceinline__ void unpack(const Raw<E> &raw, int dtype, float (&v)[kPer]) {
    if constexpr (E == 4) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = __uint_as_float(raw.w[j]);
    } else if (dtype == PDR_F16) {
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j) {
            const float2 f = unpack2(raw.w[j], PDR_F16);
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j) {
            const float2 f = unpack2(raw.w[j], PDR_BF16);
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
    }
}

// Zeroes what is of the neighbouring rows.  16-bit vectors inside the row are passed over
// (17708 x 4170 fp16 to 8 bits 89 us, element by element 109); most warps of fp32 rows
// meet an end (16384 x 333: 12.4 us, passed over 15.7).
template <int E, bool SHIFT>
__device__ __forceinline__ void keep_row(float (&v)[kPer], const Row<E, SHIFT> &q) {
    if constexpr (SHIFT) {
#pragma unroll
        for (int j = 0; j < kPer; j += E) {
            const int c = q.column(j);
            if (E == 8 && c >= 0 && c + E <= q.D) continue;
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (!q.inside(c + i)) v[j + i] = 0.0f;
        }
    }
}

template <int E, bool SHIFT>
__device__ __forceinline__ void load_weight(const void *w, int w_dtype, const Row<E, SHIFT> &q,
                                            float (&v)[kPer]) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int c = q.column(j);
        v[j] = q.inside(c) ? img_load(w, c, w_dtype) : 0.0f;
    }
}

__device__ __forceinline__ unsigned short e4m3x2(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

template <int BYTES>
__device__ __forceinline__ void store_if(bool on, void *p, unsigned w) {
    if constexpr (BYTES == 4)
        asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p st.global.u32 [%0], %1;\n}" ::"l"(p),
                     "r"(w), "r"((unsigned)on)
                     : "memory");
    else if constexpr (BYTES == 2)
        asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p st.global.u16 [%0], %1;\n}" ::"l"(p),
                     "h"((unsigned short)w), "r"((unsigned)on)
                     : "memory");
    else
        asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p st.global.u8 [%0], %1;\n}" ::"l"(p),
                     "r"(w), "r"((unsigned)on)
                     : "memory");
}

// (8-bit rows are shifted like wider ones: a vector of E of their elements starts
// at a multiple of E bytes.)
template <int E, bool SHIFT>
__device__ __forceinline__ void store_row(void *p, long long row, bool on, const Row<E, SHIFT> &q,
                                          int dtype, const float (&v)[kPer]) {
    const long long at = row * q.D;
#pragma unroll
    for (int j = 0; j < kPer; j += E) {
        const int c = q.column(j);
        const bool whole = on && (SHIFT ? c >= 0 && c + E <= q.D : c < q.D);
        const bool edge = SHIFT && on && !whole && c < q.D && c > -E;
        if (dtype == PDR_E4M3) {
            unsigned w[2] = {};
#pragma unroll
            for (int i = 0; i < E / 2; ++i)
                w[i / 2] |= (unsigned)e4m3x2(v[j + 2 * i], v[j + 2 * i + 1]) << (16 * (i & 1));
            unsigned char *o = static_cast<unsigned char *>(p) + at + c;
            if (whole) {
                if constexpr (E == 8)
                    *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
                else
                    *reinterpret_cast<unsigned *>(o) = w[0];
            }
            if (edge)
#pragma unroll
                for (int i = 0; i < E; ++i)
                    store_if<1>(q.inside(c + i), o + i, w[i / 4] >> (8 * (i & 3)) & 255);
        } else {
            unsigned w[4];
            if constexpr (E == 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[j + i]);
            } else if (dtype == PDR_F16) {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = pack2(v[j + 2 * i], v[j + 2 * i + 1], PDR_F16);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = pack2(v[j + 2 * i], v[j + 2 * i + 1], PDR_BF16);
            }
            char *o = static_cast<char *>(p) + (at + c) * (16 / E);
            if (whole) *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
            if (edge)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if constexpr (E == 4)
                        store_if<4>(q.inside(c + i), o + 4 * i, w[i]);
                    else
                        store_if<2>(q.inside(c + i), o + 2 * i, w[i / 2] >> (16 * (i & 1)));
                }
        }
    }
}

// Two sums, or a sum and a maximum, over the T threads of a row, for all of them;
// the whole block calls it.  `red`: one pair per warp, of two such places in turn (a place is
// written again behind the next call's barrier).
template <bool MAX>
__device__ __forceinline__ float2 row_reduce(float a, float b, int T, float2 *&red,
                                             int &red_step) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        if (d < T) {
            const float oa = __shfl_xor_sync(0xffffffffu, a, d), ob = __shfl_xor_sync(0xffffffffu, b, d);
            a += oa;
            b = MAX ? max_nan(b, ob) : b + ob;
        }
    if (T > 32) {
        const int warp = threadIdx.x >> 5, first = T == 64 ? warp & ~1 : 0;  // (wider rows: one a block)
        if ((threadIdx.x & 31) == 0) red[warp] = make_float2(a, b);
        __syncthreads();
        a = red[first].x;
        b = red[first].y;
        for (int i = 1; i < T >> 5; ++i) {
            a += red[first + i].x;
            b = MAX ? max_nan(b, red[first + i].y) : b + red[first + i].y;
        }
        red += red_step;
        red_step = -red_step;
    }
    return make_float2(a, b);
}

template <int E, bool SHIFT>
__device__ __forceinline__ Row<E, SHIFT> make_row(long long row, long long M, int D, int T) {
    Row<E, SHIFT> q;
    q.D = D;
    q.T = T;
    q.t = threadIdx.x % T;
    q.shift = SHIFT ? (int)(row * D & (E - 1)) : 0;
    q.total = M * D;
    return q;
}

// The rows of a block, AHEAD of them under way: a row's registers are fetched anew as
// soon as its elements are unpacked (a copy from register to register would wait for
// the loads).  AHEAD = 0: fetched when they are needed.
template <int E, bool SHIFT, bool ADD, int AHEAD>
__device__ __forceinline__ void norm_rows(const NormArgs &a, const Row<E, SHIFT> &q, long long row,
                                          const float (&w)[kPer], float2 *red) {
    constexpr int S = AHEAD > 0 ? AHEAD : 1;
    const int T = a.T, per_block = blockDim.x / T;
    const long long step = (long long)gridDim.x * per_block;
    int red_step = 32;
    Raw<E> x[S], r[ADD ? S : 1];
    auto fetch_row = [&](int k, long long at) {
        fetch(x[k], a.x, at, at < a.M, q);
        if constexpr (ADD) fetch(r[k], a.r, at, at < a.M, q);
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) fetch_row(k, row + k * step);
    for (long long base = (long long)blockIdx.x * per_block; base < a.M;) {
#pragma unroll
        for (int k = 0; k < S; ++k, base += step, row += step) {
            if (k && base >= a.M) break;
            const bool on = row < a.M;
            if constexpr (AHEAD == 0) fetch_row(k, row);
            float v[kPer];
            unpack<E>(x[k], a.dtype, v);
            if constexpr (ADD) {
                float f[kPer];
                unpack<E>(r[k], a.dtype, f);
#pragma unroll
                for (int j = 0; j < kPer; ++j) v[j] += f[j];
            }
            if constexpr (AHEAD > 0) fetch_row(k, row + AHEAD * step);
            if (ADD && a.s) store_row(a.s, row, on, q, a.dtype, v);
            keep_row(v, q);
            // y = v w rstd: the sum of v^2 and the largest |v w| in one reduction.
            float ss = 0.0f, m = 0.0f;
            if (a.w) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    ss = fmaf(v[j], v[j], ss);
                    v[j] *= w[j];
                }
            }
            if (a.scale) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) m = max_nan(m, fabsf(v[j]));
            }
            const float2 both = row_reduce<true>(ss, m, T, red, red_step);
            float k1 = a.w ? rsqrtf(fmaf(both.x, a.inv_d, a.eps)) : 1.0f;
            if (a.scale) {
                const float scale = max_nan(both.y * k1 * (1.0f / kE4M3Max), kMinScale);
                if (q.t == 0 && on) a.scale[row] = scale;
                // rstd / scale of a row of zeros (1000 x 2^126) is beyond fp32, and 0 times that no
                // zero: one factor after the other there, since |v rstd| <= 448 scale.  (For every
                // row 73416 x 1152 to 8 bits took 81 us against 80.)
                const float rstd = k1, inverse = rcp(scale);
                k1 *= inverse;
                if (__builtin_expect(!(k1 <= 3.402823466e38f), 0)) {
                    asm volatile("");  // (a branch, not 16 conditional products)
#pragma unroll
                    for (int j = 0; j < kPer; ++j) v[j] *= rstd;
                    k1 = inverse;
                }
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) v[j] *= k1;
            store_row(a.y, row, on, q, a.y_dtype, v);
        }
    }
}

template <int E, bool SHIFT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) k_rms_norm(const NormArgs a) {
    __shared__ float2 red[2 * 32];
    grid_dep_wait();
    const long long row = (long long)blockIdx.x * (blockDim.x / a.T) + threadIdx.x / a.T;
    const Row<E, SHIFT> q = make_row<E, SHIFT>(row, a.M, a.D, a.T);
    float w[kPer];
    if (a.w) load_weight(a.w, a.w_dtype, q, w);
    // Two 16-bit rows, or one fp32 row (16384 x 333: 12.4 us, two 13.7) or one and what is
    // added (65536 x 512 to 8 bits: 40.9 us, two of both 44.1 with spilled registers).  Blocks of 1024 threads have none
    // to spare.
    constexpr int some = THREADS < 1024;
    if (a.r)
        norm_rows<E, SHIFT, true, some>(a, q, row, w, red);
    else
        norm_rows<E, SHIFT, false, some * (E == 8 ? 2 : 1)>(a, q, row, w, red);
}

template <int E, bool SHIFT, int THREADS>
__global__ void __launch_bounds__(THREADS, 1)
    k_rms_norm_bwd(const NormBwdArgs a) {
    extern __shared__ float part[];  // [rows of a block][D] when there are several
    __shared__ float2 reds[2][32];
    float2 *red = reds[0];
    int red_step = 32;
    grid_dep_wait();
    const int T = a.T, per_block = blockDim.x / T;
    const long long step = (long long)gridDim.x * per_block;
    long long row = (long long)blockIdx.x * per_block + threadIdx.x / T;
    const Row<E, SHIFT> q = make_row<E, SHIFT>(row, a.M, a.D, T);
    float w[kPer], dw[kPer];
    load_weight(a.w, a.w_dtype, q, w);
#pragma unroll
    for (int j = 0; j < kPer; ++j) dw[j] = 0.0f;
    // The next row is fetched ahead: to other registers (`ahead`), or fp32 rows, which have
    // none to spare, to the same ones when they are unpacked (25620 x 776 62 us, in time for
    // their use 69).  Blocks of 1024 threads have registers for neither.
    constexpr bool ahead = THREADS < 1024 && E == 8, again = THREADS < 1024 && E == 4;
    Raw<E> s, dy, ds, next_s, next_dy;
    if constexpr (ahead || again) {
        fetch(s, a.s, row, row < a.M, q);
        fetch(dy, a.dy, row, row < a.M, q);
    }
    for (long long base = (long long)blockIdx.x * per_block; base < a.M; base += step, row += step) {
        const bool on = row < a.M;
        if constexpr (ahead) {
            if (a.ds) fetch(ds, a.ds, row, on, q);  // needed last
            fetch(next_s, a.s, row + step, row + step < a.M, q);
            fetch(next_dy, a.dy, row + step, row + step < a.M, q);
        } else if constexpr (!again) {
            fetch(s, a.s, row, on, q);
            fetch(dy, a.dy, row, on, q);
        }
        float v[kPer], g[kPer];
        unpack<E>(s, a.dtype, v);
        unpack<E>(dy, a.dtype, g);
        if constexpr (again) {
            fetch(s, a.s, row + step, row + step < a.M, q);
            fetch(dy, a.dy, row + step, row + step < a.M, q);
        }
        keep_row(v, q);
        keep_row(g, q);
        // With p = dy w: sum v^2 and sum p v in one reduction; n = v rstd.
        float ss = 0.0f, pv = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            ss = fmaf(v[j], v[j], ss);
            pv = fmaf(g[j] * w[j], v[j], pv);
        }
        const float2 sums = row_reduce<false>(ss, pv, T, red, red_step);
        // (Behind the last row the norm is eps alone; with eps = 0 infinity times 0 would reach dw.)
        const float rstd = on ? rsqrtf(fmaf(sums.x, a.inv_d, a.eps)) : 0.0f;
        const float dot = rstd * rstd * sums.y * a.inv_d;  // mean(p n) / |v|_rms
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            dw[j] = fmaf(g[j] * rstd, v[j], dw[j]);
            g[j] = rstd * fmaf(-v[j], dot, g[j] * w[j]);
        }
        if (a.ds) {
            if constexpr (!ahead) fetch(ds, a.ds, row, on, q);
            unpack<E>(ds, a.dtype, v);
#pragma unroll
            for (int j = 0; j < kPer; ++j) g[j] += v[j];
        }
        if (a.dx) store_row(a.dx, row, on, q, a.dtype, g);
        if constexpr (ahead) {
            s = next_s;
            dy = next_dy;
        }
    }
    if (!a.dw) return;
    // The block's rows, in order; then one partial row per block.
    const int D = a.D, sub = threadIdx.x / T;
    float *to = per_block > 1 ? part + sub * D : a.dw + (size_t)blockIdx.x * D;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int c = q.column(j);
        if (q.inside(c)) to[c] = dw[j];
    }
    if (per_block > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += blockDim.x) {
            float s = 0.0f;
            for (int i = 0; i < per_block; ++i) s += part[i * D + c];
            a.dw[(size_t)blockIdx.x * D + c] = s;
        }
    }
}

// Threads per row, block size and blocks for M rows of D elements.  Rows of more than
// 1024 elements have a block each, as many blocks as `per_sm` threads an SM make
// (with powers of two for T and blocks of 256, 512 or 1024 threads 73416 x 1152 bf16 to 8 bits
// took 109 us against 80 with a cold L2, 17708 x 4170 195 against 94, the backward of 30114 x 2304 132 against
// 95; that of 60000 x 777, with 64 threads a row either way, 108 against 112).
struct NormShape {
    bool shift;
    int T, threads, blocks;
};
NormShape norm_shape(long long M, int D, int bytes, int per_sm) {
    NormShape n;
    const int E = 16 / bytes;
    n.shift = D % E != 0;
    n.T = 1;
    const int share = (D + (n.shift ? E - 1 : 0) + kPer - 1) / kPer;
    while (n.T < share && n.T < 64) n.T *= 2;
    if (share > 64) n.T = (share + 31) / 32 * 32;
    n.threads = n.T > 64 ? n.T : 256;
    const long long per_block = n.threads / n.T, need = (M + per_block - 1) / per_block;
    long long most = kSMs * (per_sm > n.threads ? per_sm / n.threads : 1);
    if (n.shift && need > most && per_block < 8)  // a thread's rows 8 apart
        most = most * per_block / 8 * 8 / per_block;
    n.blocks = (int)(need < most ? need : most);
    return n;
}

template <bool BWD, int E, bool SHIFT, int THREADS>
auto norm_kernel() {
    if constexpr (BWD)
        return k_rms_norm_bwd<E, SHIFT, THREADS>;
    else
        return k_rms_norm<E, SHIFT, THREADS>;
}
template <bool BWD, typename Args>
cudaError_t launch_norm(const NormShape &n, const Args &a, size_t smem, cudaStream_t s) {
    using Kernel = void (*)(Args);
    constexpr int most = BWD ? kBwdThreads : kFwdThreads, most32 = BWD ? kBwdThreads : kFwdThreads32;
    static const Kernel kernels[2][2][2] = {
        {{norm_kernel<BWD, 8, false, most>(), norm_kernel<BWD, 8, false, 1024>()},
         {norm_kernel<BWD, 8, true, most>(), norm_kernel<BWD, 8, true, 1024>()}},
        {{norm_kernel<BWD, 4, false, most32>(), norm_kernel<BWD, 4, false, 1024>()},
         {norm_kernel<BWD, 4, true, most32>(), norm_kernel<BWD, 4, true, 1024>()}}};
    const bool f32 = a.dtype == PDR_F32;
    return launch_dependent(kernels[f32][n.shift][n.threads > (f32 ? most32 : most)], dim3((unsigned)n.blocks),
                            dim3((unsigned)n.threads), smem, s, a);
}

pdr_status run_fwd(NormArgs a, cudaStream_t s) {
    const NormShape n = norm_shape(a.M, a.D, dtype_bytes(a.dtype), a.dtype == PDR_F32 ? kFwdThreads32 : kFwdThreads);
    a.T = n.T;
    return done(launch_norm<false>(n, a, 0, s));
}

bool norm_sizes(int M, int D) { return M >= 0 && D >= 1; }
// (The vectors of a shifted row take up to E - 1 elements more, and 1024 threads 16 each.)
bool norm_in_limits(int M, int D, int bytes) {
    const int E = 16 / bytes;
    return M <= PDR_MAX_ROWS && D <= PDR_MAX_NORM_FEATURES - (D % E ? E - 1 : 0);
}

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
    if (!norm_in_limits(M, D, dtype_bytes(dtype))) return PDR_ERR_TOO_LARGE;
    if (!weight || (M > 0 && (!x || !y)) || (M > 0 && (y_dtype == PDR_E4M3) != (y_scale != nullptr)) ||
        (!residual && sum))
        return PDR_ERR_INVALID_ARG;
    if (!aligned_to(x, 16) || !aligned_to(residual, 16) || !aligned_to(sum, 16) || !aligned_to(y, 16) ||
        !aligned_to(weight, dtype_bytes(weight_dtype)) || !aligned_to(y_scale, 4))
        return PDR_ERR_INVALID_ARG;
    if (M == 0) return PDR_OK;
    return run_fwd({x, residual, weight, sum, y, y_scale, dtype, weight_dtype, y_dtype, eps, 1.0f / D, M, D, 0},
                   static_cast<cudaStream_t>(stream));
}

pdr_status pdr_quantize_rows(const void *x, int dtype, int M, int D, void *y, float *y_scale,
                             void *stream) {
    if (!norm_sizes(M, D) || !float_type(dtype)) return PDR_ERR_INVALID_ARG;
    if (!norm_in_limits(M, D, dtype_bytes(dtype))) return PDR_ERR_TOO_LARGE;
    if (M > 0 && (!x || !y || !y_scale)) return PDR_ERR_INVALID_ARG;
    if (!aligned_to(x, 16) || !aligned_to(y, 16) || !aligned_to(y_scale, 4)) return PDR_ERR_INVALID_ARG;
    if (M == 0) return PDR_OK;
    return run_fwd({x, nullptr, nullptr, nullptr, y, y_scale, dtype, dtype, PDR_E4M3, 0.0f, 1.0f / D, M, D, 0},
                   static_cast<cudaStream_t>(stream));
}

size_t pdr_rms_norm_bwd_workspace_bytes(int M, int D) {
    if (!norm_sizes(M, D) || !norm_in_limits(M, D, 4)) return 0;
    // (for the type that takes more blocks)
    const int a = norm_shape(M, D, 2, kBwdThreads).blocks, b = norm_shape(M, D, 4, kBwdThreads).blocks;
    return align256((size_t)(a > b ? a : b) * D * 4);
}

pdr_status pdr_rms_norm_bwd(const void *grad, const void *sum, int dtype, const void *weight,
                            int weight_dtype, const void *grad_sum, float eps, int M, int D,
                            void *grad_x, void *grad_weight, void *workspace,
                            size_t workspace_bytes, void *stream) {
    if (!norm_sizes(M, D) || !float_type(dtype) || !(weight_dtype == dtype || weight_dtype == PDR_F32) ||
        !(eps >= 0.0f))
        return PDR_ERR_INVALID_ARG;
    if (!norm_in_limits(M, D, dtype_bytes(dtype))) return PDR_ERR_TOO_LARGE;
    if (!weight || (M > 0 && (!grad || !sum))) return PDR_ERR_INVALID_ARG;
    const int we = dtype_bytes(weight_dtype);
    if (!aligned_to(grad, 16) || !aligned_to(sum, 16) || !aligned_to(grad_sum, 16) ||
        !aligned_to(grad_x, 16) || !aligned_to(weight, we) || !aligned_to(grad_weight, we))
        return PDR_ERR_INVALID_ARG;
    const size_t need = pdr_rms_norm_bwd_workspace_bytes(M, D);
    if (need && grad_weight && (!workspace || !aligned_to(workspace, 256))) return PDR_ERR_INVALID_ARG;
    if (grad_weight && workspace_bytes < need) return PDR_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (M == 0) {
        if (grad_weight) err = cudaMemsetAsync(grad_weight, 0, (size_t)D * we, s);
        return done(err);
    }
    if (!grad_x && !grad_weight) return PDR_OK;
    const NormShape n = norm_shape(M, D, dtype_bytes(dtype), kBwdThreads);
    const NormBwdArgs a = {grad, sum, weight, grad_sum, grad_x,
                           grad_weight ? static_cast<float *>(workspace) : nullptr,
                           dtype, weight_dtype, eps, 1.0f / D, M, D, n.T};
    // One row of dw for each row of a block: at most 256 x 16 floats.
    err = launch_norm<true>(n, a, n.threads > n.T ? (size_t)(n.threads / n.T) * D * 4 : 0, s);
    if (err == cudaSuccess && grad_weight)
        err = launch_join_columns({static_cast<const float *>(workspace), n.blocks, D, grad_weight, weight_dtype}, s);
    return done(err);
}

}  // extern "C"
