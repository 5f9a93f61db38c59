// The tensor-core product kernel behind linear.cu and gated.cu.
//
// One persistent block per SM walks over 128 x BN tiles of the result.  A
// block's warps have fixed parts:
//   warp 0   copies A and B tiles to shared memory with TMA (128-byte
//            swizzle, 64 16-bit or 128 8-bit k per stage, as many stages as
//            fit);
//   warp 1   issues tcgen05.mma (128 x BN x 32 bytes) into one of the
//            accumulators in tensor memory (2 of 256 columns, 4 of fewer);
//   warp 2   owns the tensor memory;
//   warps 4..11 take finished accumulators to registers and run the
//            epilogue, while the next tile's products run.
// What the four epilogues compute is in gemm.cuh (GemmEpi).
#include <stdint.h>

#include <cuda.h>

#include "gemm.cuh"

namespace pdr {
namespace {

constexpr int kBM = 128;              // tile rows
constexpr int kRowBytes = 128;        // k of a stage, in bytes (the swizzle's width)
constexpr int kABytes = kBM * kRowBytes;
constexpr int kMaxStages = 12;
constexpr int kThreads = 384;
constexpr int kEpiWarp = 4;           // first epilogue warp
constexpr int kMaxAcc = 4;            // accumulators in tensor memory
constexpr int kChunk = 32;            // columns an epilogue warp handles at once
constexpr int kStagePitch = 17;       // floats per row of the transposing buffer (16 columns)
constexpr int kTransBytes = 32 * kStagePitch * 4;  // per epilogue warp
// Tries of a bounded wait: each try sleeps in hardware for up to some
// microseconds, so a wait gives up after seconds, far beyond any product.
constexpr int kWaitTries = 1 << 22;

__device__ int g_wait_error;  // set when a bounded wait gave up

struct __align__(64) GemmParams {
    CUtensorMap a[2], b[2];
    int mode, a_mn, b_mn, act;
    int M, N, nm, nn, nz, splits, tiles;
    int kb0, kb;                      // k blocks of the first source, of all
    int bn, bcols, stages, nacc, split_cols;  // bcols: result columns of a tile
    int b_bytes, kelems;              // B bytes of a stage, k of a stage
    unsigned idesc;
    unsigned long long adesc, bdesc;  // smem descriptors without the address
    int a_step, b_step;               // descriptor advance (16-byte units) of one mma
    int fp8;
    void *out, *out2;
    int out_dtype, out_vec;
    long long ldo, out_z, out_split;
    const void *bias;
    int bias_dtype;
    const float *scale_m, *scale_n, *scale_n2;
    const void *in;
    int in_dtype, in_vec;
    long long ldi;
    float *colsum;
};

struct Barriers {
    unsigned long long full[kMaxStages], empty[kMaxStages], acc_full[kMaxAcc], acc_empty[kMaxAcc];
    unsigned long long drain;
    unsigned tmem;
    int abort;
};

__device__ __forceinline__ unsigned smem_u32(const void *p) {
    return static_cast<unsigned>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void bar_init(unsigned long long *b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned long long *b) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(unsigned long long *b, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(b)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool bar_try(unsigned long long *b, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(b)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits for a phase of a barrier, at most kWaitTries tries; false (and the
// block's abort flag and the library's error word set) if it gave up.
__device__ __forceinline__ bool bar_wait(unsigned long long *b, unsigned parity, int *abort) {
    for (int i = 0; i < kWaitTries; ++i) {
        if (bar_try(b, parity)) return true;
        if ((i & 63) == 63 && *(volatile int *)abort) return false;
    }
    *(volatile int *)abort = 1;
    atomicExch(&g_wait_error, 1);
    return false;
}

__device__ __forceinline__ void tma_load(void *dst, const CUtensorMap *map, int x, int y,
                                         unsigned long long *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void mma(unsigned d, unsigned long long a, unsigned long long b,
                                    unsigned idesc, bool acc, bool fp8) {
    if (fp8)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((unsigned)acc)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((unsigned)acc)
            : "memory");
}
__device__ __forceinline__ void mma_commit(unsigned long long *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tmem_load32(unsigned addr, float (&v)[kChunk]) {
    unsigned *r = reinterpret_cast<unsigned *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
// Waits for the warp's tensor-memory loads; `settled` then keeps the compiler
// from using their registers any earlier.
__device__ __forceinline__ void tmem_load_wait() {
    __syncwarp();
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void settled(float (&v)[kChunk]) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) asm volatile("" : "+f"(v[i]));
}

// ---- a row's 32 columns between registers and global memory ----------------
//
// Lane l of a warp holds row l of a 32 x 32 block.  Aligned rows (vec) move as
// full 32-byte sectors; other rows go through the warp's transposing buffer,
// 16 columns at a time, so that a warp access covers runs of 16 neighbouring
// elements.  `rows` x `cols`: what of the block is inside the result.

__device__ __forceinline__ void read_block(const void *p, long long ld, int dtype, bool vec,
                                           long long row0, int rows, int col0, int cols,
                                           float *trans, float (&v)[kChunk]) {
    const int lane = threadIdx.x & 31;
    if (vec && cols >= kChunk) {
        if (lane < rows) {
            const long long at = (row0 + lane) * ld + col0;
            if (dtype == PDR_F32) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    unsigned w[8];
                    load8(static_cast<const float *>(p) + at + 8 * i, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[8 * i + j] = __uint_as_float(w[j]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    unsigned w[8];
                    load8(static_cast<const unsigned short *>(p) + at + 16 * i, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 f = unpack2(w[j], dtype);
                        v[16 * i + 2 * j] = f.x;
                        v[16 * i + 2 * j + 1] = f.y;
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v[i] = 0.0f;
        }
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int r = 2 * i + (lane >> 4), c = 16 * h + (lane & 15);
            float x = 0.0f;
            if (r < rows && c < cols) x = img_load(p, (size_t)((row0 + r) * ld + col0 + c), dtype);
            trans[r * kStagePitch + (lane & 15)] = x;
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) v[16 * h + j] = trans[lane * kStagePitch + j];
    }
    __syncwarp();
}

__device__ __forceinline__ void write_block(void *p, long long ld, int dtype, bool vec,
                                            long long row0, int rows, int col0, int cols,
                                            float *trans, const float (&v)[kChunk]) {
    const int lane = threadIdx.x & 31;
    if (vec && cols >= kChunk) {
        if (lane < rows) {
            const long long at = (row0 + lane) * ld + col0;
            if (dtype == PDR_F32) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    unsigned w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * i + j]);
                    store8(static_cast<float *>(p) + at + 8 * i, w);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    unsigned w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j] = pack2(v[16 * i + 2 * j], v[16 * i + 2 * j + 1], dtype);
                    store8(static_cast<unsigned short *>(p) + at + 16 * i, w);
                }
            }
        }
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 16; ++j) trans[lane * kStagePitch + j] = v[16 * h + j];
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int r = 2 * i + (lane >> 4), c = 16 * h + (lane & 15);
            if (r < rows && c < cols)
                img_store(p, (size_t)((row0 + r) * ld + col0 + c), dtype,
                          trans[r * kStagePitch + (lane & 15)]);
        }
    }
    __syncwarp();
}

// Sums of the 32 columns over the warp's 32 rows: lane l returns column l's.
__device__ __forceinline__ float column_sums(float (&v)[kChunk]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float mine = up ? v[i + w] : v[i], other = up ? v[i] : v[i + w];
            v[i] = mine + __shfl_xor_sync(0xffffffffu, other, w);
        }
    }
    return v[0];
}

template <int ACT>
__device__ __forceinline__ void apply_act(float (&v)[kChunk]) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = act_value<ACT>(v[i]);
}
template <int ACT>
__device__ __forceinline__ void apply_gated(float (&g)[kChunk], const float (&u)[kChunk]) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) g[i] = act_value<ACT>(g[i]) * u[i];
}
template <int ACT>
__device__ __forceinline__ void apply_slope(float (&z)[kChunk], const float (&dy)[kChunk]) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        float s;
        act_both<ACT>(z[i], s);
        z[i] = dy[i] * s;
    }
}
// (g, u) become (dg, du).
template <int ACT>
__device__ __forceinline__ void apply_gated_bwd(float (&g)[kChunk], float (&u)[kChunk],
                                                const float (&dh)[kChunk]) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        float s;
        const float a = act_both<ACT>(g[i], s);
        g[i] = dh[i] * u[i] * s;
        u[i] = dh[i] * a;
    }
}

// f<ACT>(...) for the run's activation, switched once per 32 columns.
#define PDR_BY_ACT(act, f, ...)                                   \
    switch (act) {                                                \
        case PDR_ACT_RELU: f<PDR_ACT_RELU>(__VA_ARGS__); break;   \
        case PDR_ACT_SILU: f<PDR_ACT_SILU>(__VA_ARGS__); break;   \
        case PDR_ACT_GELU: f<PDR_ACT_GELU>(__VA_ARGS__); break;   \
        case PDR_ACT_GELU_TANH: f<PDR_ACT_GELU_TANH>(__VA_ARGS__); break; \
        default: f<PDR_ACT_NONE>(__VA_ARGS__); break;             \
    }

struct Tile {
    int m, n, z, split, k0, k1;
};
__device__ __forceinline__ Tile tile_of(const GemmParams &p, int t) {
    Tile r;
    r.n = t % p.nn;
    t /= p.nn;
    r.m = t % p.nm;
    t /= p.nm;
    r.z = t % p.nz;
    r.split = t / p.nz;
    r.k0 = (int)((long long)p.kb * r.split / p.splits);
    r.k1 = (int)((long long)p.kb * (r.split + 1) / p.splits);
    return r;
}

__device__ __forceinline__ void load_stage(const GemmParams &p, const Tile &t, int kb, char *stage,
                                           unsigned long long *bar) {
    const bool second = p.mode == kTwoSources && kb >= p.kb0;
    const int k = (second ? kb - p.kb0 : kb) * p.kelems;
    const CUtensorMap *ma = &p.a[second || (p.mode == kBatchA && t.z) ? 1 : 0];
    const CUtensorMap *mb = &p.b[second ? 1 : 0];
    char *A = stage, *B = stage + kABytes;
    const int m0 = t.m * kBM, n0 = t.n * p.bcols;
    if (p.a_mn) {
        tma_load(A, ma, m0, k, bar);
        tma_load(A + kABytes / 2, ma, m0 + 64, k, bar);
    } else {
        tma_load(A, ma, k, m0, bar);
    }
    if (p.b_mn) {
        for (int j = 0; j < p.b_bytes; j += 8192) tma_load(B + j, mb, n0 + j / 128, k, bar);
    } else {
        tma_load(B, mb, k, n0, bar);
        if (p.mode == kDualB) tma_load(B + p.b_bytes / 2, &p.b[1], k, n0, bar);
    }
}

// A 32-column chunk of one warp's 32 rows of tile t, columns c0 ... of the tile.
template <int EPI>
__device__ __forceinline__ void epilogue_chunk(const GemmParams &p, const Tile &t, unsigned acc,
                                               int c0, int quarter, float scale_m,
                                               float *columns, float *trans) {
    const long long row0 = (long long)t.m * kBM + 32 * quarter;
    const long long left = (long long)p.M - row0;
    const int rows = left < 0 ? 0 : left > 32 ? 32 : (int)left;
    const int col0 = t.n * p.bcols + c0;
    const int cols = p.N - col0;
    // This chunk's bias and column scales, in the warp's own shared memory
    // (read back as broadcasts).
    const float *bias = columns, *scale = columns + kChunk, *scale2 = columns + 2 * kChunk;
    if (p.bias || p.fp8) {
        const int lane = threadIdx.x & 31, n = col0 + lane;
        const bool in = lane < cols;
        __syncwarp();
        if (p.bias) columns[lane] = in ? img_load(p.bias, n, p.bias_dtype) : 0.0f;
        if (p.fp8) columns[kChunk + lane] = in ? p.scale_n[n] : 0.0f;
        if (p.fp8 && p.scale_n2) columns[2 * kChunk + lane] = in ? p.scale_n2[n] : 0.0f;
        __syncwarp();
    }
    float v[kChunk];
    __syncwarp();
    tmem_load32(acc + c0, v);
    if constexpr (EPI == kEpiLinear) {
        float r[kChunk];
        if (p.in) read_block(p.in, p.ldi, p.in_dtype, p.in_vec, row0, rows, col0, cols, trans, r);
        tmem_load_wait();
        settled(v);
        if (p.fp8) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v[i] *= scale_m * scale[i];
        }
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v[i] += bias[i];
        }
        PDR_BY_ACT(p.act, apply_act, v);
        if (p.in) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v[i] += r[i];
        }
        const long long off = t.z * p.out_z + t.split * p.out_split;
        char *out = static_cast<char *>(p.out2 && t.z ? p.out2 : p.out) +
                    off * dtype_bytes(p.out_dtype);
        write_block(out, p.ldo, p.out_dtype, p.out_vec, row0, rows, col0, cols, trans, v);
    } else if constexpr (EPI == kEpiGated) {
        float u[kChunk];
        tmem_load32(acc + p.bcols + c0, u);
        tmem_load_wait();
        settled(v);
        settled(u);
        if (p.fp8) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
                v[i] *= scale_m * scale[i];
                u[i] *= scale_m * scale2[i];
            }
        }
        PDR_BY_ACT(p.act, apply_gated, v, u);
        write_block(p.out, p.ldo, p.out_dtype, p.out_vec, row0, rows, col0, cols, trans, v);
    } else if constexpr (EPI == kEpiSlope) {
        float dy[kChunk];
        read_block(p.in, p.ldi, p.in_dtype, p.in_vec, row0, rows, col0, cols, trans, dy);
        tmem_load_wait();
        settled(v);
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) v[i] += bias[i];
        }
        PDR_BY_ACT(p.act, apply_slope, v, dy);
        write_block(p.out, p.ldo, p.out_dtype, p.out_vec, row0, rows, col0, cols, trans, v);
        if (p.colsum) {
            // Rows outside count nothing, whatever act'(bias) is there.
            if ((int)(threadIdx.x & 31) >= rows) {
#pragma unroll
                for (int i = 0; i < kChunk; ++i) v[i] = 0.0f;
            }
            const float s = column_sums(v);
            const int lane = threadIdx.x & 31;
            if (lane < cols)
                p.colsum[((long long)t.m * 4 + quarter) * p.N + col0 + lane] = s;
        }
    } else {
        float u[kChunk], dh[kChunk];
        tmem_load32(acc + p.bcols + c0, u);
        read_block(p.in, p.ldi, p.in_dtype, p.in_vec, row0, rows, col0, cols, trans, dh);
        tmem_load_wait();
        settled(v);
        settled(u);
        PDR_BY_ACT(p.act, apply_gated_bwd, v, u, dh);
        write_block(p.out, p.ldo, p.out_dtype, p.out_vec, row0, rows, col0, cols, trans, v);
        write_block(p.out2, p.ldo, p.out_dtype, p.out_vec, row0, rows, col0, cols, trans, u);
    }
}

template <int EPI>
__global__ void __launch_bounds__(kThreads, 1) k_gemm(const __grid_constant__ GemmParams p) {
    extern __shared__ char raw[];
    // Stages first, at a 1024-byte boundary (the swizzle's period).
    char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    const int stage_bytes = kABytes + p.b_bytes;
    char *after = smem + p.stages * stage_bytes;
    Barriers *bars = reinterpret_cast<Barriers *>(after);
    float *columns_all = reinterpret_cast<float *>(after + 512);  // [8 warps][3][32]
    float *trans_all = columns_all + 8 * 3 * kChunk;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            bar_init(&bars->full[i], 1);
            bar_init(&bars->empty[i], 1);
        }
        for (int i = 0; i < p.nacc; ++i) {
            bar_init(&bars->acc_full[i], 1);
            bar_init(&bars->acc_empty[i], p.split_cols ? 8 : 4);
        }
        bar_init(&bars->drain, 1);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars->tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const unsigned tmem = bars->tmem;
    grid_dep_wait();

    if (warp == 0 && lane == 0) {
        int stage = 0, issued = 0;
        unsigned phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
            const Tile tile = tile_of(p, t);
            for (int kb = tile.k0; kb < tile.k1; ++kb) {
                ok = bar_wait(&bars->empty[stage], phase ^ 1, &bars->abort);
                if (!ok) break;
                bar_expect(&bars->full[stage], stage_bytes);
                load_stage(p, tile, kb, smem + stage * stage_bytes, &bars->full[stage]);
                ++issued;
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
        if (!ok) {
            // Copies in flight end before the block does (waits bounded).
            const int n = issued < p.stages ? issued : p.stages;
            for (int i = 0; i < n; ++i) {
                if (stage == 0) {
                    stage = p.stages;
                    phase ^= 1;
                }
                --stage;
                for (int j = 0; j < kWaitTries && !bar_try(&bars->full[stage], phase); ++j) {
                }
            }
        }
    } else if (warp == 1 && lane == 0) {
        int stage = 0, acc = 0;
        unsigned phase = 0, acc_phase = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < p.tiles && ok; t += gridDim.x) {
            const Tile tile = tile_of(p, t);
            ok = bar_wait(&bars->acc_empty[acc], acc_phase ^ 1, &bars->abort);
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const unsigned d = tmem + acc * p.bn;
            bool more = false;
            for (int kb = tile.k0; kb < tile.k1; ++kb) {
                ok = bar_wait(&bars->full[stage], phase, &bars->abort);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const unsigned at = smem_u32(smem + stage * stage_bytes);
                unsigned long long da = p.adesc | ((at >> 4) & 0x3fff);
                unsigned long long db = p.bdesc | (((at + kABytes) >> 4) & 0x3fff);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    mma(d, da, db, p.idesc, more, p.fp8);
                    more = true;
                    da += p.a_step;
                    db += p.b_step;
                }
                mma_commit(&bars->empty[stage]);
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!ok) break;
            mma_commit(&bars->acc_full[acc]);
            if (++acc == p.nacc) {
                acc = 0;
                acc_phase ^= 1;
            }
        }
        if (!ok) {
            mma_commit(&bars->drain);  // products in flight end before their memory is freed
            for (int j = 0; j < kWaitTries && !bar_try(&bars->drain, 0); ++j) {
            }
        }
    } else if (warp >= kEpiWarp) {
        const int ew = warp - kEpiWarp, group = ew >> 2, quarter = warp & 3;
        float *trans = trans_all + ew * (kTransBytes / 4);
        float *columns = columns_all + ew * 3 * kChunk;
        const int cols = p.split_cols ? p.bcols / 2 : p.bcols;
        const int cfirst = p.split_cols ? group * cols : 0;
        int acc = 0, it = 0;
        unsigned acc_phase = 0;
        for (int t = blockIdx.x; t < p.tiles; t += gridDim.x, ++it) {
            const bool mine = p.split_cols || (it & 1) == group;
            if (mine) {
                const Tile tile = tile_of(p, t);
                float scale_m = 1.0f;
                const long long row = (long long)tile.m * kBM + 32 * quarter + lane;
                if (p.fp8 && row < p.M) scale_m = p.scale_m[row];
                if (!bar_wait(&bars->acc_full[acc], acc_phase, &bars->abort)) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const unsigned d = tmem + ((unsigned)(32 * quarter) << 16) + acc * p.bn;
                for (int c = cfirst; c < cfirst + cols; c += kChunk)
                    if (tile.n * p.bcols + c < p.N)
                        epilogue_chunk<EPI>(p, tile, d, c, quarter, scale_m, columns, trans);
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) bar_arrive(&bars->acc_empty[acc]);
            }
            if (++acc == p.nacc) {
                acc = 0;
                acc_phase ^= 1;
            }
        }
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 2) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

// ---- small kernels -----------------------------------------------------------

// Row copy between row lengths, 16-bit or 8-bit elements.
template <typename T>
__global__ void __launch_bounds__(256) k_pack(const T *__restrict__ from, long long rows, int cols,
                                              T *__restrict__ to, long long ld) {
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (long long r = (long long)blockIdx.x * 8 + warp; r < rows; r += (long long)gridDim.x * 8)
        for (int c = lane; c < cols; c += 32) to[r * ld + c] = from[r * cols + c];
}

__global__ void __launch_bounds__(256) k_join(const float *__restrict__ part, int splits,
                                              long long stride, long long n, void *to, void *to2,
                                              int dtype) {
    grid_dep_wait();
    part += blockIdx.y * n;
    if (blockIdx.y) to = to2;
    const long long step = (long long)gridDim.x * 256;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += step) {
        float s = 0.0f;
        for (int j = 0; j < splits; ++j) s += part[j * stride + i];
        img_store(to, (size_t)i, dtype, s);
    }
}

// One block per 32 columns; thread row y adds rows y, y + 32, ..., then the 32
// partial sums are added in order.
__global__ void __launch_bounds__(1024) k_join_columns(const float *__restrict__ part,
                                                       long long rows, long long cols, void *to,
                                                       int dtype) {
    __shared__ float sums[32][33];
    grid_dep_wait();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + x;
    float s = 0.0f;
    if (c < cols)
        for (long long r = y; r < rows; r += 32) s += part[r * cols + c];
    sums[y][x] = s;
    __syncthreads();
    if (y == 0 && c < cols) {
        float v = 0.0f;
        for (int j = 0; j < 32; ++j) v += sums[j][x];
        img_store(to, (size_t)c, dtype, v);
    }
}

constexpr int kGroupRows = 512;  // rows whose column sums one block forms

// Threads walk over (row, column) of a group of rows; a thread keeps its
// column (cols <= 256: 256 / cols rows at once; else column after column).
__global__ void __launch_bounds__(256) k_cast_columns(const void *__restrict__ dy, int dy_dtype,
                                                      long long M, int N, void *__restrict__ dz,
                                                      int dz_dtype, long long ldz,
                                                      float *__restrict__ colsum) {
    __shared__ float sums[256];
    grid_dep_wait();
    const long long r0 = (long long)blockIdx.x * kGroupRows;
    const long long r1 = r0 + kGroupRows < M ? r0 + kGroupRows : M;
    const int per = N < 256 ? 256 / N : 1;  // rows at once
    for (int base = 0; base < N; base += 256) {
        const int width = N - base < 256 ? N - base : 256;
        const int sub = threadIdx.x / width, c = base + threadIdx.x % width;
        float s = 0.0f;
        if (sub < per)
            for (long long r = r0 + sub; r < r1; r += per) {
                const float v = img_load(dy, (size_t)(r * N + c), dy_dtype);
                s += v;
                if (dz) img_store(dz, (size_t)(r * ldz + c), dz_dtype, v);
            }
        if (colsum) {
            __syncthreads();
            sums[threadIdx.x] = s;
            __syncthreads();
            if ((int)threadIdx.x < width) {
                for (int j = 1; j < per; ++j) s += sums[threadIdx.x + j * width];
                colsum[(long long)blockIdx.x * N + c] = s;
            }
        }
    }
}

// ---- host ----------------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

bool make_map(CUtensorMap *m, const Operand &o, int bytes, int box_cols, int box_rows) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows};
    const cuuint64_t strides[1] = {(cuuint64_t)o.ld * bytes};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, unit[2] = {1, 1};
    return f(m, bytes == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
             const_cast<void *>(o.p), dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared-memory descriptor of an operand tile, without its address: 128-byte
// swizzle; 8-row (K-major) or 8-k (MN-major) groups 1024 bytes apart, and for
// MN-major the 64-wide blocks 8192 bytes apart.
unsigned long long smem_desc(bool mn) {
    return ((unsigned long long)(mn ? 8192 >> 4 : 1) << 16) |
           ((unsigned long long)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

template <int EPI>
cudaError_t launch(const GemmParams &p, int grid, size_t smem, cudaStream_t s) {
    const cudaError_t e = cudaFuncSetAttribute(
        k_gemm<EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    return launch_dependent(k_gemm<EPI>, dim3((unsigned)grid), dim3(kThreads), smem, s, p);
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

}  // namespace

int gemm_tile_columns(int epi, int M, int N, int nz) {
    const bool dual = epi == kEpiGated || epi == kEpiGatedBwd;
    const int least = 32, most = dual ? 128 : 256;
    int c = most;
    // No wider than the result, and narrower while the tiles do not fill the machine.
    while (c > least && c / 2 >= N) c /= 2;
    while (c > least && (long long)ceil_div(M, kBM) * ceil_div(N, c) * nz < kSMs) c /= 2;
    return c;
}

int gemm_splits(int M, int N, int nz, long long K) {
    const int cols = gemm_tile_columns(kEpiLinear, 1 << 30, N, nz);
    const long long tiles = (long long)ceil_div(M, kBM) * ceil_div(N, cols) * nz;
    const long long kb = (K + 63) / 64;
    long long s = kSMs / tiles;
    if (s > kb / 4) s = kb / 4;  // at least 4 stages of k each
    return s < 1 ? 1 : (int)s;
}

cudaError_t launch_gemm(const GemmArgs &g, cudaStream_t s) {
    const bool dual = g.mode == kDualB;
    const int bytes = g.dtype == PDR_E4M3 ? 1 : 2;
    const int kelems = kRowBytes / bytes;
    GemmParams p = {};
    p.mode = g.mode;
    p.a_mn = g.a_mn;
    p.b_mn = g.b_mn;
    p.act = g.act;
    p.M = g.M;
    p.N = g.N;
    p.nz = g.mode == kBatchA ? 2 : 1;
    p.splits = g.splits;
    p.bcols = gemm_tile_columns(g.epi, g.splits > 1 ? 1 << 30 : g.M, g.N, p.nz);
    p.bn = dual ? 2 * p.bcols : p.bcols;
    p.nm = ceil_div(g.M, kBM);
    p.nn = ceil_div(g.N, p.bcols);
    const long long tiles = (long long)p.nm * p.nn * p.nz * p.splits;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    p.tiles = (int)tiles;
    p.kb0 = ceil_div(g.K[0], kelems);
    p.kb = p.kb0 + (g.mode == kTwoSources ? ceil_div(g.K[1], kelems) : 0);
    p.kelems = kelems;
    p.b_bytes = g.b_mn ? ceil_div(p.bn, 64) * 8192 : p.bn * kRowBytes;
    p.nacc = p.bn >= 256 ? 2 : 4;
    p.split_cols = p.bcols >= 2 * kChunk;
    p.fp8 = bytes == 1;
    // D fp32 | A and B: f16 0, bf16 1 (kind::f16) or e4m3 0 (kind::f8f6f4) | majors | N / 8 | M / 16
    const unsigned t = g.dtype == PDR_BF16 ? 1 : 0;
    p.idesc = (1u << 4) | (t << 7) | (t << 10) | ((unsigned)g.a_mn << 15) |
              ((unsigned)g.b_mn << 16) | ((unsigned)(p.bn / 8) << 17) | ((unsigned)(kBM / 16) << 24);
    p.adesc = smem_desc(g.a_mn);
    p.bdesc = smem_desc(g.b_mn);
    p.a_step = g.a_mn ? 2048 >> 4 : 32 >> 4;  // 16 k of 128-byte rows, or 32 bytes along k
    p.b_step = g.b_mn ? 2048 >> 4 : 32 >> 4;
    const int na = g.mode == kTwoSources || g.mode == kBatchA ? 2 : 1;
    const int nb = g.mode == kTwoSources || dual ? 2 : 1;
    for (int i = 0; i < na; ++i)
        if (!make_map(&p.a[i], g.a[i], bytes, g.a_mn ? 64 : kelems, g.a_mn ? 64 : kBM))
            return cudaErrorInvalidValue;
    for (int i = 0; i < nb; ++i)
        if (!make_map(&p.b[i], g.b[i], bytes, g.b_mn ? 64 : kelems,
                      g.b_mn ? 64 : dual ? p.bn / 2 : p.bn))
            return cudaErrorInvalidValue;
    p.out = g.out;
    p.out2 = g.out2;
    p.out_dtype = g.out_dtype;
    p.ldo = g.ldo;
    p.out_z = g.out_z;
    p.out_split = g.out_split;
    const int ob = dtype_bytes(g.out_dtype), ib = dtype_bytes(g.in_dtype);
    p.out_vec = aligned_to(g.out, 32) && aligned_to(g.out2, 32) && g.ldo * ob % 32 == 0 &&
                g.out_z * ob % 32 == 0 && g.out_split * ob % 32 == 0;
    p.bias = g.bias;
    p.bias_dtype = g.bias_dtype;
    p.scale_m = g.scale_m;
    p.scale_n = g.scale_n;
    p.scale_n2 = g.scale_n2;
    p.in = g.in;
    p.in_dtype = g.in_dtype;
    p.ldi = g.ldi;
    p.in_vec = aligned_to(g.in, 32) && g.ldi * ib % 32 == 0;
    p.colsum = g.colsum;
    const size_t fixed = 1024 + 512 + 8 * 3 * kChunk * 4 + 8 * kTransBytes;
    const size_t stage = kABytes + p.b_bytes;
    p.stages = (int)((227 * 1024 - fixed) / stage);
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    const size_t smem = fixed + p.stages * stage;
    const int grid = p.tiles < kSMs ? p.tiles : kSMs;
    static_assert(sizeof(Barriers) <= 512, "barriers fit their place");
    switch (g.epi) {
        case kEpiGated: return launch<kEpiGated>(p, grid, smem, s);
        case kEpiSlope: return launch<kEpiSlope>(p, grid, smem, s);
        case kEpiGatedBwd: return launch<kEpiGatedBwd>(p, grid, smem, s);
        default: return launch<kEpiLinear>(p, grid, smem, s);
    }
}

cudaError_t launch_pack(const void *from, long long rows, long long cols, int bytes, void *to,
                        long long ld_to, cudaStream_t s) {
    const int grid = (int)(rows / 8 + 1 < 8 * kSMs ? rows / 8 + 1 : 8 * kSMs);
    if (bytes == 1)
        return launch_dependent(k_pack<unsigned char>, dim3(grid), dim3(256), 0, s,
                                static_cast<const unsigned char *>(from), rows, (int)cols,
                                static_cast<unsigned char *>(to), ld_to);
    return launch_dependent(k_pack<unsigned short>, dim3(grid), dim3(256), 0, s,
                            static_cast<const unsigned short *>(from), rows, (int)cols,
                            static_cast<unsigned short *>(to), ld_to);
}

cudaError_t launch_join(const float *part, int splits, long long stride, long long n, void *to,
                        void *to2, int dtype, cudaStream_t s) {
    const long long blocks = (n + 255) / 256;
    return launch_dependent(k_join, dim3((unsigned)(blocks < 8 * kSMs ? blocks : 8 * kSMs), to2 ? 2 : 1),
                            dim3(256), 0, s, part, splits, stride, n, to, to2, dtype);
}

cudaError_t launch_join_columns(const float *part, long long rows, long long cols, void *to,
                                int dtype, cudaStream_t s) {
    return launch_dependent(k_join_columns, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, s,
                            part, rows, cols, to, dtype);
}

long long column_groups(long long M) { return (M + kGroupRows - 1) / kGroupRows; }

cudaError_t launch_cast_columns(const void *dy, int dy_dtype, long long M, int N, void *dz,
                                int dz_dtype, long long ldz, float *colsum, cudaStream_t s) {
    return launch_dependent(k_cast_columns, dim3((unsigned)column_groups(M)), dim3(256), 0, s, dy,
                            dy_dtype, M, N, dz, dz_dtype, ldz, colsum);
}

cudaError_t read_wait_error(int *bits, cudaStream_t s) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(bits, g_wait_error, sizeof(int), 0,
                                              cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess || *bits == 0) return e;
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_wait_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace pdr
