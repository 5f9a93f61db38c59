// Tiled matrix products on the fifth-generation tensor cores, with the
// operators' arithmetic in their epilogues: host plan (GemmArgs), launch, and
// the device helpers that linear.cu, gated.cu and norm.cu share.
//
// Every product here is  acc[m][n] = sum_k A(m, k) B(n, k)  with fp32
// accumulators.  An operand lies in memory either "K-major" (its k are
// contiguous: a row of x or of W) or "MN-major" (its m or n are contiguous: x
// and dz read as the transposed factors of dW = dz^T x).
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "pdr.h"

namespace pdr {

constexpr int kSMs = 148;

// ---- activations -----------------------------------------------------------

constexpr float kLog2e = 1.4426950408889634f;

// max that keeps NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + e^-v).  e^-v may overflow to infinity: 0.  Two operations of the
// special-function unit an element, 2048 clocks for a 128 x 128 gated tile.  Two
// elements that share a reciprocal (1 / a = b / (a b)) take 1.5 and three more
// instructions: 61.4 against 60.9 us for 65536 rows of 256 to 1024.  Pairs of
// elements in one f32x2 instruction took 65.4.
__device__ __forceinline__ float logistic(float v) { return rcp(1.0f + ex2(-kLog2e * v)); }

// Phi(z) = erfc(-z / sqrt 2) / 2, and e^{-z^2/2}.  For x >= 0 the form of Abramowitz and
// Stegun, Handbook of Mathematical Functions, 7.1.26, erfc(x) = (c1 t + ... + c8 t^8)
// e^{-x^2}, t = 1 / (1 + p x), with p = 0.43 and eight terms (half of them below) whose largest
// relative error for 0 <= x <= 9.5 is least: 8.4e-8, 4e-7 as evaluated.  Relative, so
// that the negative tail, where 1 + erf would cancel, keeps its bits in fp32 results too: an
// activation there is good to 2^-21 + z^2 2^-23 (the exponent's rounding), down to 2^-126.
// (The handbook's five terms bound the absolute error by 1.5e-7: 1.5e-2 of the value at
// z = -6.  65536 rows of 256 to 1024, gated by gelu: 83 us, with five 79.)
__device__ __forceinline__ float normal_cdf(float z, float &gauss) {
    gauss = ex2(-0.5f * kLog2e * z * z);
    const float t = rcp(fmaf(0.304055929f, fabsf(z), 1.0f));  // 0.43 / sqrt 2
    float p = fmaf(0.0368627422f, t, -0.155225113f);
    p = fmaf(p, t, 0.191922709f);
    p = fmaf(p, t, -0.0429310761f);
    p = fmaf(p, t, 0.123460680f);
    p = fmaf(p, t, 0.102463067f);
    p = fmaf(p, t, 0.122189872f);
    p = fmaf(p, t, 0.121257156f);
    const float half = p * t * gauss;  // erfc(|z| / sqrt 2) / 2
    return z < 0.0f ? half : 1.0f - half;
}

// Value (returned) and derivative of an activation (an unused slope costs nothing).
template <int ACT>
__device__ __forceinline__ float act_both(float z, float &slope) {
    if constexpr (ACT == PDR_ACT_RELU) {
        slope = z > 0.0f ? 1.0f : 0.0f;
        return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    } else if constexpr (ACT == PDR_ACT_SILU) {
        const float t = logistic(z), y = z * t;
        slope = fmaf(y, 1.0f - t, t);
        return y;
    } else if constexpr (ACT == PDR_ACT_GELU) {
        float e;
        const float p = normal_cdf(z, e);
        slope = fmaf(0.39894228040143268f * z, e, p);
        return z * p;
    } else if constexpr (ACT == PDR_ACT_GELU_TANH) {  // (1 + tanh v) / 2 = 1 / (1 + e^{-2 v})
        const float t = logistic(1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.0f)), y = z * t;
        const float c = fminf(fabsf(z), 10.0f);  // beyond, y (1 - t) is 0
        slope = fmaf(y * (1.0f - t), 1.5957691216057308f * fmaf(0.134145f * c, c, 1.0f), t);
        return y;
    } else {
        slope = 1.0f;
        return z;
    }
}

// ---- element types ---------------------------------------------------------

// Bytes of an element of a pdr_dtype.
__host__ __device__ inline int dtype_bytes(int dtype) {
    return dtype == PDR_F32 ? 4 : dtype == PDR_E4M3 ? 1 : 2;
}

// Two fp32 values rounded to nearest even to fp16 / bf16, as one 32-bit word.
__device__ __forceinline__ unsigned pack2(float a, float b, int dtype) {
    if (dtype == PDR_F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const unsigned *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned *>(&h);
}
__device__ __forceinline__ float2 unpack2(unsigned w, int dtype) {
    if (dtype == PDR_F16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// 32-byte loads and stores (one full sector each; 32-byte aligned) of the
// threads whose `on` is set.
__device__ __forceinline__ void load8(bool on, const void *p, unsigned *w) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %9, 0;\n"
        " @p ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n}"
        : "+r"(w[0]), "+r"(w[1]), "+r"(w[2]), "+r"(w[3]), "+r"(w[4]), "+r"(w[5]), "+r"(w[6]),
          "+r"(w[7])
        : "l"(p), "r"((unsigned)on));
}
__device__ __forceinline__ void store8(bool on, void *p, const unsigned *w) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %9, 0;\n"
        " @p st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n}" ::"l"(p),
        "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]),
        "r"((unsigned)on)
        : "memory");
}

// ---- fp16's range --------------------------------------------------------------

// The largest values of up to three arrays, as kBoundParts partial maxima each
// (launch_largest), and what their product is taken times: a bound of what a product's
// fp16 factor can hold.  part null: none.
constexpr int kBoundParts = 256;  // two vectors a lane
struct Bound {
    const float *part = nullptr;
    int groups = 0;
    float times = 1.0f;
};

// 2^k with bound 2^k in [2^14, 2^15): a factor of at most 1.13 bounds (a slope's) stays
// below fp16's largest number then, and 2^-28 of the bound is still a normal one.
// `inverse`: 2^-k.  (Both are normal fp32 numbers: k in [-113, 126].)  The whole warp calls it.
__device__ __forceinline__ float bound_factor(const Bound &r, bool inverse) {
    float b = r.times;
    for (int g = 0; g < r.groups; ++g) {
        const float4 *p = reinterpret_cast<const float4 *>(r.part + g * kBoundParts) + (threadIdx.x & 31);
        const float4 v = __ldg(p), u = __ldg(p + 32);
        float m = fmaxf(fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)), fmaxf(fmaxf(u.x, u.y), fmaxf(u.z, u.w)));
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        b *= m;
    }
    int e = (int)(__float_as_uint(b) >> 23);  // its exponent + 127
    e = b == 0.0f ? 141 : e < 15 ? 15 : e > 254 ? 254 : e;  // (nothing to fit: 1)
    return __uint_as_float((unsigned)(inverse ? e - 14 : 268 - e) << 23);
}

// ---- host plan -------------------------------------------------------------

// One operand of a product as it lies in memory: `rows` x `cols`, rows of `ld`
// elements apart (ld and the address multiples of 16 bytes).
struct Operand {
    const void *p = nullptr;
    long long rows = 0, cols = 0, ld = 0;
};

enum GemmMode {
    kPlain = 0,      // A = a[0], B = b[0]
    kDualB = 1,      // tile columns: first half from b[0], second half from b[1] (gated)
    kTwoSources = 2, // k runs over a[0] b[0], then over a[1] b[1]
    kBatchA = 3      // two products: A = a[z], B = b[0]
};
enum GemmEpi {
    kEpiLinear = 0,   // out = act(acc * scales + bias) + residual
    kEpiGated = 1,    // out = act(g) * u from the two halves of a tile's columns
    kEpiSlope = 2,    // out = dy * act'(acc + bias), and its column sums
    kEpiGatedBwd = 3  // out = dy * u * act'(g), out2 = dy * act(g)
};

struct GemmArgs {
    int mode = kPlain, epi = kEpiLinear;
    int dtype = PDR_BF16;           // of A and B (PDR_F16, PDR_BF16 or PDR_E4M3)
    bool a_mn = false, b_mn = false;  // MN-major operands
    Operand a[2], b[2];
    int M = 0, N = 0;               // extent of the result (of h, in the gated modes)
    long long K[2] = {0, 0};        // extent of k (of each source)
    int splits = 1;                 // k split over this many tiles, fp32 results `out_split` apart
    // epilogue
    int act = PDR_ACT_NONE;
    void *out = nullptr, *out2 = nullptr;  // out2: the second product's (kBatchA), or du
    int out_dtype = PDR_F32;
    long long ldo = 0, out_z = 0, out_split = 0;  // elements
    const void *bias = nullptr;
    int bias_dtype = PDR_F32;
    const float *scale_m = nullptr, *scale_n = nullptr, *scale_n2 = nullptr;
    const void *in = nullptr;       // residual, dy or dh: rows of ldi elements
    // Rows of the results start at multiples of 16 bytes and of the input at
    // multiples of 32 (padded rows); narrow (kEpiLinear, N <= 16): dense rows of any
    // alignment, the input's too.
    bool narrow = false;
    int in_dtype = PDR_F32;
    long long ldi = 0;
    float *colsum = nullptr;        // kEpiSlope: [4 * ceil(M / 128)][N] partial column sums
    // Takes the bound's factor into the results (kEpiSlope, whose column sums stay without
    // it, and kEpiGatedBwd), or out of them (kEpiLinear).
    Bound bound;
};

// Whether a linear result of N columns (with an input of its type) is so narrow that
// rows which TMA could not store, or the input's sectors, are taken as they are.
bool gemm_narrow(int N, int out_dtype, bool has_in);
// Tiles along k that fill the machine for a weight gradient, at most `most`.
int gemm_splits(int M, int N, int nz, long long K);
cudaError_t launch_gemm(const GemmArgs &g, cudaStream_t s);
// Two products without an activation (kEpiLinear) whose B are laid out alike and have
// the same N, in one launch where their tiles go together.
cudaError_t launch_gemm2(const GemmArgs &g0, const GemmArgs &g1, cudaStream_t s);
// Tries of a wait in the launches to come (about 4 us each); negative: the default.
void set_wait_tries(int tries);
// Whether a wait on the current device gave up since read_wait_error last reported one.
bool wait_error_pending();
// Reads (and clears) the word that a bounded wait sets when it gives up.
cudaError_t read_wait_error(int *bits, cudaStream_t s);

// ---- small kernels around the products ---------------------------------------

// Dense rows of `cols` elements (of 1, 2 or 4 bytes; 16-byte aligned) to rows of
// `ld` elements, a multiple of 16 bytes (zeros behind), up to four matrices in one
// launch; and (2 or 4 bytes) back.
struct PackJob {
    const void *from;
    void *to;
    long long rows, cols, ld;
    int bytes;
};
cudaError_t launch_pack(const PackJob *jobs, int n, cudaStream_t s);
cudaError_t launch_unpack(const void *from, long long rows, long long cols, long long ld, int bytes,
                          void *to, cudaStream_t s);
// Elements of a row padded to `unit` bytes.
inline long long padded(long long cols, int bytes, int unit) {
    return (cols * bytes + unit - 1) / unit * unit / bytes;
}
// Column sums of part[rows][cols] to `to`, rounded once to `dtype`; no columns: none.
struct ColumnJob {
    const float *part = nullptr;
    long long rows = 0, cols = 0;
    void *to = nullptr;
    int dtype = PDR_F32;
};
cudaError_t launch_join_columns(const ColumnJob &columns, cudaStream_t s);
// to[r][c] = sum over the splits of part[split][r][c], rounded once to `dtype`;
// partial rows are ld floats apart (a multiple of 4), splits `slice` floats, results
// dense.  With a second result the splits are part[split][2][slice].  And column sums beside it.
cudaError_t launch_join(const float *part, int splits, int rows, int cols, long long ld, long long slice, void *to,
                        void *to2, int dtype, const ColumnJob &columns, cudaStream_t s);
// dz = dy in `dz_dtype` times the bound's factor (rows of ldz; null: not wanted), and partial
// column sums of dy, in column_groups(M, N, dy_dtype, low) rows of `colsum` (null: not wanted).
// With `low` (a multiple of 8, N at least) rows of dz are low elements of an fp32 dy, zeros
// behind the N-th, then low of what that rounding leaves; and `two` takes the 16-bit weight
// [N][cols] twice, one below the other, in rows of ld (zeros likewise; to null: not wanted).
struct TwiceJob {
    const void *from = nullptr;
    void *to = nullptr;
    int cols = 0;
    long long ld = 0;
};
long long column_groups(long long M, int N, int dy_dtype, int low);
cudaError_t launch_cast_columns(const void *dy, int dy_dtype, long long M, int N, void *dz,
                                int dz_dtype, long long ldz, int low, const TwiceJob &two,
                                float *colsum, const Bound &bound, cudaStream_t s);
// kBoundParts partial maxima of |v| over the finite values of each job's arrays (16-byte
// aligned; the second may be null).
struct BoundJob {
    const void *p, *p2;
    long long n;
    int dtype;
};
cudaError_t launch_largest(const BoundJob *jobs, int n, float *part, cudaStream_t s);

// What the entry points check and return.
inline bool half_type(int t) { return t == PDR_F16 || t == PDR_BF16; }
inline bool float_type(int t) { return t == PDR_F32 || half_type(t); }
inline bool act_ok(int act) { return act >= PDR_ACT_NONE && act <= PDR_ACT_GELU_TANH; }
inline pdr_status done(cudaError_t e) { return e == cudaSuccess ? PDR_OK : PDR_ERR_CUDA; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool aligned_to(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace pdr
