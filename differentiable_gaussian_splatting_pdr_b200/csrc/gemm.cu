// The tensor-core product kernel behind linear.cu and gated.cu.
//
// Pairs of blocks (a cluster of two SMs) walk over 256 x BN tiles of the
// result, one persistent pair per two SMs.  Each block holds 128 rows of A, half
// of the BN rows of B and its 128 rows of the accumulator; tcgen05.mma with
// cta_group::2 multiplies over both blocks' shared memory, which reads a third
// less from L2 than single blocks with 128 x 256 tiles do.  A block's warps have
// fixed parts:
//   warp 0   copies its A rows and B half to shared memory with TMA (128-byte
//            swizzle, 64 16-bit or 128 8-bit k per stage, as many stages as
//            fit).  Where all k of a tile's B half leave room for three
//            stages of A, B stays in shared memory while the pair walks down a column
//            of tiles, and the stages hold A alone;
//   warp 1   owns the tensor memory, and in the first block issues the products
//            into one of the accumulators there (2 of 256 columns, 4 of fewer);
//   warps 4..19 take finished accumulators to registers and run the
//            epilogue, while the next tile's products run.
// What the four epilogues compute is in gemm.cuh (GemmEpi).  524288 x 256 to 8 columns: 49 us,
// 6.2 TB/s; 4096 x 4096 x 4096 in bf16: 109 us, 1260 TFLOP/s, bound by the operands' way
// from L2.
#include <stdint.h>
#include <string.h>

#include <atomic>

#include <cuda.h>

#include "gemm.cuh"

namespace pdr {
namespace {

constexpr int kBM = 128;              // tile rows
constexpr int kRowBytes = 128;        // k of a stage, in bytes (the swizzle's width)
constexpr int kABytes = kBM * kRowBytes;
constexpr int kMaxStages = 12;
constexpr int kGroups = 4, kEpiWarps = 4 * kGroups;  // epilogue warpgroups
constexpr int kThreads = 32 * (kEpiWarps + 4);
constexpr int kEpiRegs = 104, kOtherRegs = 64;  // per thread: 512 x 104 + 128 x 64 <= 640 x 96
constexpr int kCopyWarp = 0, kProductWarp = 1, kEpiWarp = 4;
constexpr int kSmemBytes = 227 * 1024;
constexpr int kMaxAcc = 4;            // accumulators in tensor memory
constexpr int kChunk = 16;            // columns an epilogue warp computes at once
constexpr int kStore = 2 * kChunk;    // columns that it stores at once
constexpr int kMaxCols = 64;          // most columns of a tile that an epilogue warp has
constexpr int kBufferBytes = 32 * kStore * 2;  // per epilogue warp: 32 rows of 16 floats or 32 halves
// Tries of a bounded wait.  A try that fails sleeps in hardware for 4.0 us (measured), so a
// wait gives up after 4 seconds, far beyond any product; what is under way when one did
// is waited for up to a quarter of a second each.
constexpr int kWaitTries = 1 << 20, kDrainTries = 1 << 16;
std::atomic<int> g_wait_tries{kWaitTries};

// A word per device that is set when a bounded wait gave up, in host memory that the
// kernels write: entry points read it without waiting for the device.
constexpr int kDevices = 64;
std::atomic<int *> g_wait_words{nullptr};

// Quotients by a divisor that is fixed for a launch, for dividends below 2^31:
// with l = ceil(log2 d) and mul = floor(2^(31 + l) / d) + 1, n / d = (n mul) >> (31 + l).
// (Integer divisions per tile held the products back: 5300 clocks for a tile of
// 2048 clocks of them.)
struct Divisor {
    unsigned d, mul, shift;
};

struct __align__(64) GemmParams {
    CUtensorMap a[2], b[2], o[2];     // operands, results
    int mode, a_mn, b_mn;
    int M, N, nz, splits, tiles;
    Divisor nm, nn;                   // tiles of 256 rows, of bcols columns
    // Where B stays: `share` pairs walk down the first na rows of each column of tiles
    // in turn (`main` tiles), the other pairs down the last nb rows, one column after another.
    Divisor na, nb;
    int share, main;
    int kb0, kb;                      // k blocks of the first source, of all
    int bn, bcols, stages, nacc;      // bcols: result columns of a tile
    int sharing;                      // epilogue groups that share a tile
    int stationary;                   // B of a column of tiles stays in shared memory
    int per_stage;                    // k blocks of a stage (2: where B stays only)
    int nbuf;                         // buffers of an epilogue warp (1 or 2)
    int columns;                      // floats of an epilogue warp's bias and column scales
    int b_bytes, kelems;              // a block's B bytes, and k, of a k block
    unsigned idesc;
    unsigned long long adesc, bdesc;  // smem descriptors without the address
    int a_step, b_step;               // descriptor advance (16-byte units) of one mma
    int fp8;
    void *out;
    int out_dtype, narrow;
    const void *bias;
    int bias_dtype;
    const float *scale_m, *scale_n, *scale_n2;
    const void *in;
    int in_dtype;
    long long ldi;
    float *colsum;
    Bound bound;
    int tries;                        // of a wait
    int *wait_word;                   // set when one gave up
};

// One product, or two that run one behind the other in the same launch: tiles of the
// same size, so that the pairs go from one to the other without a stop (no
// stationary B).
template <int NP>
struct GemmLaunch {
    GemmParams p[NP];
};

struct Barriers {
    unsigned long long full[kMaxStages], empty[kMaxStages], acc_full[kMaxAcc], acc_empty[kMaxAcc];
    unsigned long long b_full, b_empty, drain;
    unsigned tmem;
    int abort;                        // a wait of the pair gave up
    // In the first block: stages, and columns of stationary B, whose copies each block started.
    int stages_sent[2], columns_sent[2];
};

__device__ __forceinline__ unsigned smem_u32(const void *p) {
    return static_cast<unsigned>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void bar_init(unsigned long long *b, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(count) : "memory");
}
// The address of the same place in block `rank` of the cluster.
__device__ __forceinline__ unsigned at_rank(unsigned addr, unsigned rank) {
    unsigned r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrives at a barrier of the pair (its cluster address).  Relaxed: what it
// orders are reads of tensor memory, which tcgen05.wait::ld and the fence before
// it have ended; a release at this scope would also wait for the warp's stores
// to global memory (1.8 of an SM's epilogue warps stood there at any time).
__device__ __forceinline__ void bar_arrive_at(unsigned addr) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// One thread of a converged warp.  The copies and products are issued under this
// and not under a test of the lane: the compiler then knows that one thread is
// active, and puts their operands into uniform registers without a loop over the
// threads (which took some 100 clocks an instruction).
__device__ __forceinline__ bool elect_one() {
    unsigned p;
    asm volatile(
        "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void bar_expect(unsigned bar, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool bar_try(unsigned bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// An int of a block of the pair (its cluster address).
__device__ __forceinline__ void store_at(unsigned addr, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Waits for a phase of a barrier, at most p.tries tries; false (and the abort flags of
// both blocks and the library's error word set) if it gave up.  Nothing that waited in vain goes
// on to use what it waited for: the roles leave their loops, and the pair ends together.
__device__ __forceinline__ bool bar_wait(unsigned bar, unsigned parity, int *abort, const GemmParams &p) {
    for (int i = 0; i < p.tries; ++i) {
        if (bar_try(bar, parity)) return true;
        if ((i & 63) == 63 && *(volatile int *)abort) return false;
    }
    store_at(at_rank(smem_u32(abort), 0), 1);
    store_at(at_rank(smem_u32(abort), 1), 1);
    *(volatile int *)p.wait_word = 1;
    __threadfence_system();
    return false;
}
// Waits for what is under way, after a wait gave up.
__device__ __forceinline__ void bar_drain(unsigned bar, unsigned parity) {
    for (int i = 0; i < kDrainTries && !bar_try(bar, parity); ++i) {
    }
}
// A phase's bytes that never come count as come.
__device__ __forceinline__ void bar_complete(unsigned bar, unsigned bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// The copy reports to a barrier of the first block (`bar`: its cluster address).
__device__ __forceinline__ void tma_load(unsigned dst, const CUtensorMap *map, int x, int y,
                                         unsigned bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// One product of 32 bytes of k; the operands' descriptors in two words.
__device__ __forceinline__ void mma(unsigned d, unsigned al, unsigned ah, unsigned bl, unsigned bh,
                                    unsigned idesc, bool acc, bool fp8) {
    if (fp8)
        asm volatile(
            "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %6, 0;\n"
            " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
            " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %5, p;\n}" ::"r"(d),
            "r"(al), "r"(ah), "r"(bl), "r"(bh), "r"(idesc), "r"((unsigned)acc)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.u32 p, %6, 0;\n"
            " mov.b64 a, {%1, %2};\n mov.b64 b, {%3, %4};\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n}" ::"r"(d),
            "r"(al), "r"(ah), "r"(bl), "r"(bh), "r"(idesc), "r"((unsigned)acc)
            : "memory");
}
// Arrives at a barrier of both blocks when the products issued so far are done.
__device__ __forceinline__ void mma_commit(unsigned bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(bar), "h"((unsigned short)3)
        : "memory");
}

// 16 columns of the warp's 32 rows: lane l holds row l.
__device__ __forceinline__ void tmem_load(unsigned addr, float *v) {
    unsigned *r = reinterpret_cast<unsigned *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
// Waits for the warp's tensor-memory loads; `settled` then keeps the compiler
// from using their registers any earlier.
__device__ __forceinline__ void tmem_load_wait() {
    __syncwarp();
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
template <int C>
__device__ __forceinline__ void settled(float (&v)[C]) {
#pragma unroll
    for (int i = 0; i < C; ++i) asm volatile("" : "+f"(v[i]));
}

// ---- a row's 16 columns between registers and memory -------------------------
//
// Lane l of a warp holds row l of a block of 32 rows.

__device__ __forceinline__ void unpack_row(int dtype, const unsigned (&raw)[kChunk],
                                           float (&v)[kChunk]) {
    if (dtype == PDR_F32) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[i] = __uint_as_float(raw[i]);
    } else if (dtype == PDR_F16) {
#pragma unroll
        for (int i = 0; i < kChunk / 2; ++i) {
            const float2 f = unpack2(raw[i], PDR_F16);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kChunk / 2; ++i) {
            const float2 f = unpack2(raw[i], PDR_BF16);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
__device__ __forceinline__ void pack_row(int dtype, const float *v, unsigned (&w)[kChunk / 2]) {
    if (dtype == PDR_F16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = pack2(v[2 * j], v[2 * j + 1], PDR_F16);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = pack2(v[2 * j], v[2 * j + 1], PDR_BF16);
    }
}
// Results leave through the warp's buffer and TMA stores of 32 rows, which drop
// what is behind the last row and column: direct stores of 32 bytes a lane take 32
// turns of the load-store unit each, this way four.  A block in the buffer has
// rows of 64 bytes (32 columns of 16 bits or 16 of 32), their 16-byte pieces
// swizzled as the map says.
__device__ __forceinline__ void stage_half(char *buffer, int half, const unsigned (&w)[kChunk / 2]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        *reinterpret_cast<uint4 *>(buffer + lane * 64 + ((2 * half + j) ^ ((lane >> 1) & 3)) * 16) =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}
__device__ __forceinline__ void stage_floats(char *buffer, const float *v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4 *>(buffer + lane * 64 + (j ^ ((lane >> 1) & 3)) * 16) =
            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
// A warp's buffers in turn: the next one, when the stores before have read it.
struct Staging {
    char *base;
    int nbuf, turn;
    __device__ __forceinline__ char *next() {
        if (nbuf == 2) {
            if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            turn ^= kBufferBytes;
        } else {
            if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        __syncwarp();
        return base + turn;
    }
    __device__ __forceinline__ char *all() {
        if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        return base;
    }
};
__device__ __forceinline__ void tma_store(const CUtensorMap *map, const char *buffer, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
        "r"(x), "r"(y), "r"(z), "r"(smem_u32(buffer))
        : "memory");
}
// Stores one staged block, or two of neighbouring results.
__device__ __forceinline__ void store_buffer(const CUtensorMap *map, const CUtensorMap *map2,
                                             const char *buffer, int x, int y, int z) {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (elect_one()) {
        tma_store(map, buffer, x, y, z);
        if (map2) tma_store(map2, buffer + kBufferBytes, x, y, z);
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
}

// Sums of the 16 columns over the warp's 32 rows: lanes l and l + 16 return
// column l's.
__device__ __forceinline__ float column_sums(float (&v)[kChunk]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = kChunk / 2; w >= 1; w >>= 1) {
        const bool up = lane & w;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float mine = up ? v[i + w] : v[i], other = up ? v[i] : v[i + w];
            v[i] = mine + __shfl_xor_sync(0xffffffffu, other, w);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

template <int ACT, int C>
__device__ __forceinline__ void apply_act(float (&v)[C]) {
    float s;
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = act_both<ACT>(v[i], s);
}
template <int ACT, int C>
__device__ __forceinline__ void apply_gated(float (&g)[C], const float (&u)[C]) {
    float s;
#pragma unroll
    for (int i = 0; i < C; ++i) g[i] = act_both<ACT>(g[i], s) * u[i];
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

struct Tile {
    int m, n, z, split;  // m: this block's 128 rows
};
struct KRange {
    int first, end;
};
__device__ __forceinline__ int quotient(int n, const Divisor &d) {
    return d.d == 1 ? n : (int)(__umulhi((unsigned)n, d.mul) >> d.shift);
}
// Whether B stays in shared memory (of two products in a launch neither does).
template <int NP>
__device__ __forceinline__ bool stays(const GemmParams &p) {
    return NP == 1 && p.stationary;
}
template <int NP>
__device__ __forceinline__ Tile tile_of(const GemmParams &p, int t, int rank) {
    Tile r;
    if (stays<NP>(p)) {
        const bool last = t >= p.main;
        const Divisor &rows = last ? p.nb : p.na;
        if (last) t -= p.main;
        const int c = quotient(t, rows), z = quotient(c, p.nn);
        r.m = 2 * (t - c * (int)rows.d + (last ? (int)(p.nm.d - p.nb.d) : 0)) + rank;
        r.n = c - z * (int)p.nn.d;
        t = z;
    } else {  // along the rows: neighbouring pairs share A rows in L2
        const int q = quotient(t, p.nn), z = quotient(q, p.nm);
        r.n = t - q * (int)p.nn.d;
        r.m = 2 * (q - z * (int)p.nm.d) + rank;
        t = z;
    }
    r.z = 0;
    r.split = t;
    if (p.nz == 2) {
        r.z = t & 1;
        r.split = t >> 1;
    }
    return r;
}
__device__ __forceinline__ KRange k_range(const GemmParams &p, const Tile &t) {
    if (p.splits == 1) return {0, p.kb};
    return {(int)((unsigned)(p.kb * t.split) / (unsigned)p.splits),  // kb * splits < 2^31
            (int)((unsigned)(p.kb * (t.split + 1)) / (unsigned)p.splits)};
}
// The column of tiles of a tile (stationary B).
__device__ __forceinline__ int column_of(const GemmParams &p, int t) {
    return t < p.main ? quotient(t, p.na) : quotient(t - p.main, p.nb);
}
// The tiles of a pair: a contiguous run of the columns, or every so many.
struct Range {
    int first, end, step;
};
// (`before`: tiles of the product in front, after which the turn goes on.)
template <int NP>
__device__ __forceinline__ Range my_tiles(const GemmParams &p, int before) {
    const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
    if (stays<NP>(p)) {
        const int columns = p.nn.d * p.nz, sharing = columns * p.share;
        if (pair < sharing) {
            const int first = pair % columns * (int)p.na.d;
            return {first + pair / columns, first + (int)p.na.d, p.share};
        }
        const long long rest = p.tiles - p.main;
        return {p.main + (int)(rest * (pair - sharing) / (pairs - sharing)),
                p.main + (int)(rest * (pair - sharing + 1) / (pairs - sharing)), 1};
    }
    const int first = pair - before % pairs;
    return {first < 0 ? first + pairs : first, p.tiles, pairs};
}

__device__ __forceinline__ void load_a(const GemmParams &p, const Tile &t, int kb, unsigned A,
                                       unsigned bar) {
    const bool second = p.mode == kTwoSources && kb >= p.kb0;
    const int k = (second ? kb - p.kb0 : kb) * p.kelems;
    const CUtensorMap *map = &p.a[second || (p.mode == kBatchA && t.z) ? 1 : 0];
    const int m0 = t.m * kBM;
    if (p.a_mn) {
        tma_load(A, map, m0, k, bar);
        tma_load(A + kABytes / 2, map, m0 + 64, k, bar);
    } else {
        tma_load(A, map, k, m0, bar);
    }
}
// This block's half of the B rows (in the gated modes: all of Wg's or of Wu's).
__device__ __forceinline__ void load_b(const GemmParams &p, const Tile &t, int kb, int rank,
                                       unsigned B, unsigned bar) {
    const bool second = p.mode == kTwoSources && kb >= p.kb0;
    const int k = (second ? kb - p.kb0 : kb) * p.kelems;
    const bool dual = p.mode == kDualB;
    const CUtensorMap *map = &p.b[second || (dual && rank) ? 1 : 0];
    const int n0 = t.n * p.bcols + (dual ? 0 : rank * (p.bn / 2));
    if (p.b_mn) {
        for (int j = 0; j < p.b_bytes; j += 8192) tma_load(B + j, map, n0 + j / 128, k, bar);
    } else {
        tma_load(B, map, k, n0, bar);
    }
}

// One warp's 32 rows of a tile, from column c0 to c1 (32 columns or 64).
// `columns`: the warp's bias and column scales, up to [3][kMaxCols]; `have_n`: the
// column of tiles that they are of.  Here results leave by TMA, and rows of the
// input are full 32-byte sectors (a multiple of 16 16-bit, or 8 fp32, wide).
template <int EPI, int ACT>
__device__ __forceinline__ bool epilogue_tile(const GemmParams &p, const Tile &t, unsigned acc,
                                              unsigned ready, unsigned phase, int c0, int c1,
                                              int quarter, float *columns, int &have_n, float factor,
                                              Staging &staging, int *abort, unsigned release) {
    constexpr bool kTwo = EPI == kEpiGated || EPI == kEpiGatedBwd;  // g and u
    constexpr int C = EPI == kEpiGated ? 32 : 16;                   // columns at once
    const int lane = threadIdx.x & 31;
    const int row0 = t.m * kBM + 32 * quarter, n0 = t.n * p.bcols;
    char *stage = nullptr;
    c1 = min(c1, p.N - n0);
    // (A warp behind the last row of a tile still writes its column sums: zeros.)
    const bool any = (EPI == kEpiSlope ? t.m * kBM : row0) < p.M && c0 < c1, on = row0 + lane < p.M;
    const bool has_in = EPI != kEpiGated && p.in;
    unsigned raw[kChunk];
    const char *in_row = nullptr;
    auto fetch = [&](int c) {
        const int ib = p.in_dtype == PDR_F32 ? 4 : 2;
        load8(on, in_row + c * ib, raw);
        if (p.in_dtype == PDR_F32) load8(on && n0 + c + 8 < p.N, in_row + c * ib + 32, raw + 8);
    };
    float scale_m = 1.0f;
    if (any) {  // on their way while the products finish
        if (has_in) {
            in_row = static_cast<const char *>(p.in) +
                     ((long long)(row0 + lane) * p.ldi + n0) * (p.in_dtype == PDR_F32 ? 4 : 2);
            fetch(c0);
        }
        if (p.fp8 && on) scale_m = p.scale_m[row0 + lane];
        if ((p.bias || p.fp8) && have_n != t.n) {
            have_n = t.n;
            __syncwarp();
            for (int c = lane; c < c1 - c0; c += 32) {
                const int n = n0 + c0 + c;
                if (p.bias) columns[c] = img_load(p.bias, n, p.bias_dtype);
                if (p.fp8) columns[kMaxCols + c] = p.scale_n[n];
                if (p.fp8 && p.scale_n2) columns[2 * kMaxCols + c] = p.scale_n2[n];
            }
            __syncwarp();
        }
    }
    if (!__all_sync(0xffffffffu, bar_wait(ready, phase, abort, p))) return false;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    for (int c = c0; c < c1 && any; c += C) {
        float v[C], u[kTwo ? C : 1];
#pragma unroll
        for (int i = 0; i < C; i += kChunk) {
            tmem_load(acc + c + i, v + i);
            if constexpr (kTwo) tmem_load(acc + p.bcols + c + i, u + i);
        }
        tmem_load_wait();
        settled(v);
        if constexpr (kTwo) settled(u);
        if (c + C >= c1) {  // the accumulator is read: the next products may overwrite it
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) bar_arrive_at(release);
        }
        float x[kChunk];
        if (has_in) {
            unpack_row(p.in_dtype, raw, x);
            if (c + C < c1) fetch(c + C);
        }
        if (p.bound.part) {  // (a slope's or gated result has its input as a factor)
            if constexpr (EPI == kEpiLinear) {
#pragma unroll
                for (int i = 0; i < C; ++i) v[i] *= factor;
            } else {
#pragma unroll
                for (int i = 0; i < kChunk; ++i) x[i] *= factor;
            }
        }
        const float4 *column = reinterpret_cast<const float4 *>(columns + c - c0);
        if (p.fp8) {
#pragma unroll
            for (int i = 0; i < C; i += 4) {
                const float4 f = column[(kMaxCols + i) / 4];
                v[i] *= scale_m * f.x;
                v[i + 1] *= scale_m * f.y;
                v[i + 2] *= scale_m * f.z;
                v[i + 3] *= scale_m * f.w;
                if constexpr (EPI == kEpiGated) {
                    const float4 h = column[(2 * kMaxCols + i) / 4];
                    u[i] *= scale_m * h.x;
                    u[i + 1] *= scale_m * h.y;
                    u[i + 2] *= scale_m * h.z;
                    u[i + 3] *= scale_m * h.w;
                }
            }
        }
        if (!kTwo && p.bias) {
#pragma unroll
            for (int i = 0; i < C; i += 4) {
                const float4 f = column[i / 4];
                v[i] += f.x;
                v[i + 1] += f.y;
                v[i + 2] += f.z;
                v[i + 3] += f.w;
            }
        }
        if constexpr (EPI == kEpiLinear) {
            apply_act<ACT>(v);
            if (has_in) {
#pragma unroll
                for (int i = 0; i < C; ++i) v[i] += x[i];
            }
        } else if constexpr (EPI == kEpiGated) {
            apply_gated<ACT>(v, u);
        } else if constexpr (EPI == kEpiSlope) {
            apply_slope<ACT>(v, x);
        } else {
            apply_gated_bwd<ACT>(v, u, x);
        }
        unsigned w[kChunk / 2];
        const int half = C == 32 ? 0 : (c - c0) / kChunk & 1;
        const int slice = t.split * p.nz + t.z;
        if constexpr (EPI == kEpiGatedBwd) {  // dg in the first buffer, du in the second
            if (half == 0) stage = staging.all();
            pack_row(p.out_dtype, v, w);
            stage_half(stage, half, w);
            pack_row(p.out_dtype, u, w);
            stage_half(stage + kBufferBytes, half, w);
            if (half == 1 || c + C >= c1)
                store_buffer(&p.o[0], &p.o[1], stage, n0 + c - half * kChunk, row0, 0);
        } else if (EPI != kEpiSlope && p.out_dtype == PDR_F32) {
#pragma unroll
            for (int i = 0; i < C; i += kChunk) {
                if (n0 + c + i >= p.N) break;
                stage = staging.next();
                stage_floats(stage, v + i);
                store_buffer(&p.o[0], nullptr, stage, n0 + c + i, row0, slice);
            }
        } else {
            if (half == 0) stage = staging.next();
#pragma unroll
            for (int i = 0; i < C; i += kChunk) {
                pack_row(p.out_dtype, v + i, w);
                stage_half(stage, half + i / kChunk, w);
            }
            if ((C == 32 || half == 1 || c + C >= c1) && row0 < p.M)
                store_buffer(&p.o[p.mode == kBatchA && t.z], nullptr, stage, n0 + c - half * kChunk,
                             row0, p.mode == kBatchA ? 0 : slice);
        }
        if constexpr (EPI == kEpiSlope)
            if (p.colsum) {
#pragma unroll
                for (int i = 0; i < C; ++i) v[i] = on ? v[i] : 0.0f;  // rows outside count nothing
                const float s = column_sums(v);
                if (lane < kChunk && c + lane < c1)  // (1 / factor: a power of two)
                    p.colsum[((long long)t.m * 4 + quarter) * p.N + n0 + c + lane] = p.bound.part ? s / factor : s;
            }
    }
    if (!any && lane == 0) bar_arrive_at(release);
    return true;
}

// The same for results of at most 16 columns whose rows TMA cannot store (Gaussian
// parameters of 1, 2, 4, 5 ... channels): the warp's 32 rows are one run of memory,
// and go through its buffer in that order.
template <int ACT>
__device__ __forceinline__ bool epilogue_narrow(const GemmParams &p, const Tile &t, unsigned acc,
                                                unsigned ready, unsigned phase, int quarter,
                                                float *columns, int &have_n, float factor, float *buffer,
                                                int *abort, unsigned release) {
    const int lane = threadIdx.x & 31, N = p.N;
    const int row0 = t.m * kBM + 32 * quarter, rows = max(0, min(32, p.M - row0));
    const long long at = (long long)row0 * N + lane;
    const int run = rows * N;
    unsigned raw[kChunk];
    float scale_m = 1.0f;
    if (p.in) {
        if (p.in_dtype == PDR_F32) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
                if (lane + 32 * i < run) raw[i] = __ldg(static_cast<const unsigned *>(p.in) + at + 32 * i);
        } else {
#pragma unroll
            for (int i = 0; i < kChunk; ++i)
                if (lane + 32 * i < run) raw[i] = __ldg(static_cast<const unsigned short *>(p.in) + at + 32 * i);
        }
    }
    if (p.fp8 && lane < rows) scale_m = p.scale_m[row0 + lane];
    if (have_n < 0) {
        have_n = 0;
        if (lane < kChunk) {
            columns[lane] = p.bias && lane < N ? img_load(p.bias, lane, p.bias_dtype) : 0.0f;
            columns[kMaxCols + lane] = p.fp8 && lane < N ? p.scale_n[lane] : 1.0f;
        }
        __syncwarp();
    }
    if (!__all_sync(0xffffffffu, bar_wait(ready, phase, abort, p))) return false;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    float v[kChunk];
    tmem_load(acc, v);
    tmem_load_wait();
    settled(v);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncwarp();
    if (lane == 0) bar_arrive_at(release);
    if (p.fp8) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[i] *= scale_m * columns[kMaxCols + i];
    } else if (p.bound.part) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[i] *= factor;
    }
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] += columns[i];
    apply_act<ACT>(v);
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
        if (j < N) buffer[lane * N + j] = v[j];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        if (lane + 32 * i >= run) continue;
        float x = buffer[lane + 32 * i];
        if (p.in) x += p.in_dtype == PDR_F32 ? __uint_as_float(raw[i]) : unpack2(raw[i], p.in_dtype).x;
        img_store(p.out, (size_t)(at + 32 * i), p.out_dtype, x);
    }
    __syncwarp();
    return true;
}

// After a wait gave up: the copies that the two blocks started end, whose bytes the first
// block's barriers count.  A stage's n-th use is the (n / stages)-th phase of its barrier, and
// one use of a stage is under way at most: the next is started behind the products
// that read it, which waited for both blocks' copies.  So are the columns of stationary B.  Where one
// block alone started a use, the other's share is put right first: the first block announces
// the bytes of the second's copies, or counts those that it announced in vain.
__device__ __forceinline__ void drain_phase(unsigned bar, int n, const int (&sent)[2], unsigned bytes,
                                            unsigned parity) {
    if (n >= sent[0])
        bar_expect(bar, bytes);
    else if (n >= sent[1])
        bar_complete(bar, bytes);
    bar_drain(bar, parity);
}
template <int NP>
__device__ __forceinline__ void drain_copies(const GemmParams &p, const Barriers &bars, unsigned full,
                                             unsigned b_full, unsigned block_bytes) {
    const int sent[2] = {*(volatile const int *)&bars.stages_sent[0], *(volatile const int *)&bars.stages_sent[1]};
    const int last = max(sent[0], sent[1]), uses = (p.kb + p.per_stage - 1) / p.per_stage;  // (of a tile, where B stays)
    for (int n = max(0, last - p.stages); n < last; ++n) {
        const bool two = stays<NP>(p) && p.per_stage == 2 && 2 * (n % uses) + 1 < p.kb;
        drain_phase(full + 8 * (n % p.stages), n, sent, two ? 2 * block_bytes : block_bytes, n / p.stages & 1);
    }
    const int columns[2] = {*(volatile const int *)&bars.columns_sent[0], *(volatile const int *)&bars.columns_sent[1]};
    const int most = max(columns[0], columns[1]);
    if (most > 0) drain_phase(b_full, most - 1, columns, p.kb * p.b_bytes, (most - 1) & 1);
}

template <int EPI, int ACT, bool NARROW, int NP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_gemm(const __grid_constant__ GemmLaunch<NP> launch) {
    extern __shared__ char raw[];
    const GemmParams &p = launch.p[0];  // (both have the same tiles and shared memory)
    // Tiles first, at a 1024-byte boundary (the swizzle's period).
    char *smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    const int block_bytes = kABytes + (stays<NP>(p) ? 0 : p.b_bytes);  // of a k block
    const int stage_bytes = p.per_stage * block_bytes;
    char *held = smem + p.stages * stage_bytes;  // B of all k, where it stays
    char *after = held + (stays<NP>(p) ? p.kb * p.b_bytes : 0);
    char *buffers = after;  // nbuf per epilogue warp, 1024-byte aligned
    float *columns_all = reinterpret_cast<float *>(buffers + kEpiWarps * p.nbuf * kBufferBytes);  // [warp][columns]
    Barriers *bars = reinterpret_cast<Barriers *>(columns_all + kEpiWarps * p.columns);
    const int warp = threadIdx.x >> 5;
    const int rank = blockIdx.x & 1;  // in the pair; block 0 leads

    if (threadIdx.x == 0) {
        for (int i = 0; i < p.stages; ++i) {
            bar_init(&bars->full[i], 1);
            bar_init(&bars->empty[i], 1);
        }
        for (int i = 0; i < p.nacc; ++i) {
            bar_init(&bars->acc_full[i], 1);
            bar_init(&bars->acc_empty[i], 2 * 4 * p.sharing);
        }
        bar_init(&bars->b_full, 1);
        bar_init(&bars->b_empty, 1);
        bar_init(&bars->drain, 1);
        bars->abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kProductWarp) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&bars->tmem)),
                     "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const unsigned tmem = bars->tmem;
    const unsigned full = smem_u32(bars->full), empty = smem_u32(bars->empty);
    const unsigned acc_full = smem_u32(bars->acc_full), acc_empty = smem_u32(bars->acc_empty);
    const unsigned b_full = smem_u32(&bars->b_full), b_empty = smem_u32(&bars->b_empty);
    int *abort = &bars->abort;
    grid_dep_wait();

    // The launch gives each thread 96 registers; the epilogue's warps take
    // what the others do not need.
    if (warp >= kEpiWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        const int ew = warp - kEpiWarp, group = ew >> 2, quarter = warp & 3;
        Staging staging = {buffers + ew * p.nbuf * kBufferBytes, p.nbuf, 0};
        float *columns = columns_all + ew * p.columns;
        // `sharing` groups divide a tile's columns, sets of them take tiles in turn.
        const int cols = p.bcols / p.sharing, cfirst = group % p.sharing * cols;
        const int sets = kGroups / p.sharing, set = group / p.sharing;
        const unsigned release = at_rank(acc_empty, 0);
        const float factor = EPI != kEpiGated && p.bound.part ? bound_factor(p.bound, EPI == kEpiLinear) : 1.0f;
        int acc = 0, it = 0;
        unsigned acc_phase = 0;
        bool ok = true;
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const GemmParams &p = launch.p[q];
            const Range range = my_tiles<NP>(p, q ? launch.p[0].tiles : 0);
            int have_n = -1;
            Tile tile = tile_of<NP>(p, range.first, rank);
            for (int t = range.first; t < range.end && ok; t += range.step, ++it) {
                if ((it & (sets - 1)) == set) {
                    const unsigned d = tmem + ((unsigned)(32 * quarter) << 16) + acc * p.bn;
                    if constexpr (NARROW)
                        ok = epilogue_narrow<ACT>(p, tile, d, acc_full + 8 * acc, acc_phase, quarter,
                                                  columns, have_n, factor, reinterpret_cast<float *>(staging.base),
                                                  abort, release + 8 * acc);
                    else
                        ok = epilogue_tile<EPI, ACT>(p, tile, d, acc_full + 8 * acc, acc_phase, cfirst,
                                                     cfirst + cols, quarter, columns, have_n, factor,
                                                     staging, abort, release + 8 * acc);
                    if (!ok) break;
                }
                tile.m += 2 * range.step;  // down the column, or looked up
                if (!stays<NP>(p) || t >= p.main) tile = tile_of<NP>(p, t + range.step, rank);
                if (++acc == p.nacc) {
                    acc = 0;
                    acc_phase ^= 1;
                }
            }
        }
        if (!NARROW && elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        const unsigned stages0 = smem_u32(smem), held0 = smem_u32(held);
        if (warp == kCopyWarp && elect_one()) {
            const unsigned lead_full = at_rank(full, 0), lead_b_full = at_rank(b_full, 0);
            int stage = 0, issued = 0, column = -1, columns = 0;
            unsigned phase = 0, b_phase = 0;
            bool ok = true, ready = true;  // the first stages are empty
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                const GemmParams &p = launch.p[q];
                const Range range = my_tiles<NP>(p, q ? launch.p[0].tiles : 0);
                for (int t = range.first; t < range.end && ok; t += range.step) {
                    const Tile tile = tile_of<NP>(p, t, rank);
                    const KRange k = k_range(p, tile);
                    if (stays<NP>(p) && column != column_of(p, t)) {
                        column = column_of(p, t);
                        ok = bar_wait(b_empty, b_phase ^ 1, abort, p);
                        if (!ok) break;
                        b_phase ^= 1;
                        ++columns;
                        if (rank == 0) bar_expect(b_full, 2 * p.kb * p.b_bytes);
                        for (int kb = 0; kb < p.kb; ++kb)
                            load_b(p, tile, kb, rank, held0 + kb * p.b_bytes, lead_b_full);
                    }
                    for (int kb = k.first; kb < k.end; kb += p.per_stage) {
                        const bool two = stays<NP>(p) && p.per_stage == 2 && kb + 1 < k.end;
                        if (!ready) ok = bar_wait(empty + 8 * stage, phase ^ 1, abort, p);
                        if (!ok) break;
                        const unsigned bar = lead_full + 8 * stage, at = stages0 + stage * stage_bytes;
                        if (rank == 0) bar_expect(full + 8 * stage, two ? 4 * block_bytes : 2 * block_bytes);
                        ++issued;
                        if (++stage == p.stages) {
                            stage = 0;
                            phase ^= 1;
                        }
                        ready = bar_try(empty + 8 * stage, phase ^ 1);  // asked early: the answer takes a while
                        load_a(p, tile, kb, at, bar);
                        if (!stays<NP>(p)) load_b(p, tile, kb, rank, at + kABytes, bar);
                        if (two) load_a(p, tile, kb + 1, at + kABytes, bar);
                    }
                }
            }
            store_at(at_rank(smem_u32(&bars->stages_sent[rank]), 0), issued);
            store_at(at_rank(smem_u32(&bars->columns_sent[rank]), 0), columns);
        } else if (warp == kProductWarp && rank == 0 && elect_one()) {
            // Tiles left in the column of the first one (stationary B).
            int stage = 0, acc = 0, left = 0;
            unsigned phase = 0, acc_phase = 0, b_phase = 0;
            // Whether the next barriers were seen ready: asked before a block's
            // products are issued, so that the answer is there when they are.
            bool ok = true, full_ready = false, acc_ready = false;
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                const GemmParams &p = launch.p[q];
                const Range range = my_tiles<NP>(p, q ? launch.p[0].tiles : 0);
                const unsigned a_hi = (unsigned)(p.adesc >> 32), b_hi = (unsigned)(p.bdesc >> 32);
                const unsigned a_lo = (unsigned)p.adesc, b_lo = (unsigned)p.bdesc;
                if (!ok) break;
                for (int t = range.first; t < range.end; t += range.step) {
                    int nk = p.kb;
                    if (p.splits > 1) {
                        const KRange k = k_range(p, tile_of<NP>(p, t, rank));
                        nk = k.end - k.first;
                    }
                    if (stays<NP>(p) && left == 0) {
                        left = t < p.main ? p.tiles : p.nb.d;
                        if (t != range.first)
                            mma_commit(b_empty);  // the last column's B is free
                        else if (t >= p.main)
                            left -= t - p.main - column_of(p, t) * p.nb.d;
                        ok = bar_wait(b_full, b_phase, abort, p);
                        b_phase ^= 1;
                        if (!ok) break;
                    }
                    --left;
                    if (!acc_ready) ok = bar_wait(acc_empty + 8 * acc, acc_phase ^ 1, abort, p);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const unsigned d = tmem + acc * p.bn, this_full = acc_full + 8 * acc;
                    if (++acc == p.nacc) {
                        acc = 0;
                        acc_phase ^= 1;
                    }
                    bool more = false;
                    for (int kb = 0; kb < nk; kb += p.per_stage) {
                        if (!full_ready) ok = bar_wait(full + 8 * stage, phase, abort, p);
                        if (!ok) break;
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const unsigned at = stages0 + stage * stage_bytes, done = empty + 8 * stage;
                        const unsigned bt = stays<NP>(p) ? held0 + kb * p.b_bytes : at + kABytes;
                        if (++stage == p.stages) {
                            stage = 0;
                            phase ^= 1;
                        }
                        full_ready = bar_try(full + 8 * stage, phase);
                        if (kb + p.per_stage >= nk) acc_ready = bar_try(acc_empty + 8 * acc, acc_phase ^ 1);
                        auto block = [&](unsigned a, unsigned b) {
                            unsigned al = a_lo | (a >> 4), bl = b_lo | (b >> 4);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                mma(d, al, a_hi, bl, b_hi, p.idesc, more, p.fp8);
                                more = true;
                                al += p.a_step;
                                bl += p.b_step;
                            }
                        };
                        block(at, bt);
                        if (stays<NP>(p) && p.per_stage == 2 && kb + 1 < nk)
                            block(at + kABytes, bt + p.b_bytes);
                        mma_commit(done);
                    }
                    if (!ok) break;
                    mma_commit(this_full);
                }
            }
        }
    }
    // Neither block leaves, or gives up its memory, before both are done.
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_sync();
    if (*(volatile int *)abort) {  // (in both blocks or in neither)
        // A wait gave up.  No copy or product is started any more; those under way end first.
        if (warp == kProductWarp && elect_one()) {
            const unsigned drain = smem_u32(&bars->drain);
            if (rank == 0) mma_commit(drain);  // (of the thread that issued the products)
            bar_drain(drain, 0);
        } else if (warp == kCopyWarp && rank == 0 && elect_one()) {
            drain_copies<NP>(p, *bars, full, b_full, block_bytes);
        }
        __syncwarp();
        cluster_sync();
    }
    if (warp == kProductWarp) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

// ---- small kernels -----------------------------------------------------------

// Dense rows to padded rows, 16 bytes per thread, a row per warp; several matrices
// in one launch.
struct PackJobs {
    PackJob job[4];
    int n;
    unsigned first[5];  // block of each job
};
template <typename T>
__device__ __forceinline__ uint4 padded_vector(const T *row, int v, int cols) {
    constexpr int E = 16 / sizeof(T);
    if constexpr (sizeof(T) == 2)
        if (v * E + E <= cols) {  // by words of 4 bytes, whatever the row's parity
            const bool odd = reinterpret_cast<uintptr_t>(row) & 2;
            const unsigned *q = reinterpret_cast<const unsigned *>(row + v * E - odd);
            unsigned w[5];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __ldg(q + i);
            w[4] = odd ? __ldg(q + 4) : 0;  // (odd rows have no multiple of 8 elements: it is inside)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = odd ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
            return make_uint4(w[0], w[1], w[2], w[3]);
        }
    union {
        T e[E];
        uint4 u;
    } w;
#pragma unroll
    for (int i = 0; i < E; ++i) w.e[i] = v * E + i < cols ? __ldg(row + v * E + i) : T(0);
    return w.u;
}
template <typename T>
__device__ __forceinline__ void pack_rows(const PackJob &j, unsigned block, unsigned blocks) {
    constexpr int E = 16 / sizeof(T);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, vectors = (int)(j.ld / E);
    for (long long r = (long long)block * 8 + warp; r < j.rows; r += (long long)blocks * 8) {
        const T *row = static_cast<const T *>(j.from) + r * j.cols;
        uint4 *to = static_cast<uint4 *>(j.to) + r * vectors;
        for (int v = lane; v < vectors; v += 32) to[v] = padded_vector(row, v, (int)j.cols);
    }
}
__global__ void __launch_bounds__(256) k_pack(const PackJobs p) {
    grid_dep_wait();
    int i = 0;
    while (i + 1 < p.n && blockIdx.x >= p.first[i + 1]) ++i;
    const PackJob &j = p.job[i];
    const unsigned block = blockIdx.x - p.first[i], blocks = p.first[i + 1] - p.first[i];
    if (j.bytes == 1)
        pack_rows<unsigned char>(j, block, blocks);
    else if (j.bytes == 2)
        pack_rows<unsigned short>(j, block, blocks);
    else
        pack_rows<unsigned>(j, block, blocks);
}

// And back, a row per warp.  Rows of 16-bit elements: what a thread writes starts at 16
// bytes; it lies the same distance behind a vector of the padded row for the whole
// row, so that two aligned loads and a shift make it (linear 60000 x 128 -> 777 72 us, by
// pairs of elements 99).  32-bit elements go one by one, a warp's together (60000 x 128 -> 333
// 50 us; by shifted vectors 53).
template <typename T>
__global__ void __launch_bounds__(256) k_unpack(const T *__restrict__ from, long long rows, int cols,
                                                int ld, T *__restrict__ to) {
    grid_dep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (long long r = (long long)blockIdx.x * 8 + warp; r < rows; r += (long long)gridDim.x * 8) {
        const T *row = from + r * ld;
        T *out = to + r * cols;
        if constexpr (sizeof(T) == 4) {
            for (int c = lane; c < cols; c += 32) out[c] = __ldg(row + c);
            continue;
        }
        int head = (int)((0 - (reinterpret_cast<uintptr_t>(out) >> 1)) & 7);  // before the first vector
        if (head > cols) head = cols;
        const int vectors = (cols - head) / 8, tail = head + 8 * vectors;
        if (lane < head) out[lane] = __ldg(row + lane);
        const uint4 *in = reinterpret_cast<const uint4 *>(row);
        uint4 *whole = reinterpret_cast<uint4 *>(out + head);
#pragma unroll 2
        for (int v = lane; v < vectors; v += 32) {
            const uint4 a = __ldg(in + v), b = __ldg(in + v + (head != 0));  // (b's first element is in the row)
            unsigned w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 6; ++i) w[i] = head & 4 ? w[i + 2] : w[i];
#pragma unroll
            for (int i = 0; i < 5; ++i) w[i] = head & 2 ? w[i + 1] : w[i];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = head & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
            whole[v] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (lane < cols - tail) out[tail + lane] = __ldg(row + tail + lane);
    }
}

// A block per `W` columns: thread row y of 256 / W adds rows y, y + 256 / W, ... (eight
// loads under way at once), then the partial sums are added in order.
template <int W>
__device__ __forceinline__ void join_columns(const ColumnJob &j, unsigned block) {
    constexpr int Y = 256 / W;
    __shared__ float sums[Y][W + 1];
    const int x = threadIdx.x % W, y = threadIdx.x / W;
    const long long c = (long long)block * W + x;
    float s = 0.0f;
    if (c < j.cols)
        for (long long r = y; r < j.rows; r += Y * 8) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = r + Y * k < j.rows ? __ldg(j.part + (r + Y * k) * j.cols + c) : 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
    sums[y][x] = s;
    __syncthreads();
    if (y == 0 && c < j.cols) {
        float v = 0.0f;
        for (int k = 0; k < Y; ++k) v += sums[k][x];
        img_store(j.to, (size_t)c, j.dtype, v);
    }
}
__global__ void __launch_bounds__(256) k_join_columns(const ColumnJob j) {
    grid_dep_wait();
    join_columns<8>(j, blockIdx.x);
}

// Four neighbouring columns per thread.  Y rows of threads add a Y-th of the splits
// each, in order, and their sums are added in order: 8 where there are too few columns to
// fill the machine.
// Blocks behind the first `blocks` add up column sums (ColumnJob), 8 columns by 32
// rows of threads.
template <int Y>
__global__ void __launch_bounds__(256) k_join(const float *__restrict__ part, int splits, int rows,
                                              int cols, long long ld, long long slice, void *to, void *to2,
                                              int dtype, unsigned blocks, const ColumnJob job) {
    constexpr int X = 256 / Y;
    __shared__ float4 sums[Y][X];
    grid_dep_wait();
    if (blockIdx.x >= blocks) {
        if (blockIdx.y == 0) join_columns<8>(job, blockIdx.x - blocks);
        return;
    }
    const long long n = rows * ld, stride = slice * (to2 ? 2 : 1);
    part += blockIdx.y * slice;
    if (blockIdx.y) to = to2;
    const int x = threadIdx.x % X, y = threadIdx.x / X;
    const long long i = ((long long)blockIdx.x * X + x) * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int j1 = (y + 1) * splits / Y;
    if (i < n)
        for (int j = y * splits / Y; j < j1; j += 8) {
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (j + k < j1) v[k] = __ldg(reinterpret_cast<const float4 *>(part + (j + k) * stride + i));
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (j + k < j1) {
                    s.x += v[k].x;
                    s.y += v[k].y;
                    s.z += v[k].z;
                    s.w += v[k].w;
                }
        }
    if constexpr (Y > 1) {
        sums[y][x] = s;
        __syncthreads();
    }
    if (y || i >= n) return;
#pragma unroll
    for (int k = 1; k < Y; ++k) {
        s.x += sums[k][x].x;
        s.y += sums[k][x].y;
        s.z += sums[k][x].z;
        s.w += sums[k][x].w;
    }
    const long long r = i / ld;
    const int c = (int)(i - r * ld);
    const size_t at = (size_t)(r * cols + c);
    if (c + 4 <= cols && cols % 4 == 0 && dtype != PDR_F32) {  // (results start at 16 bytes)
        const uint2 w = make_uint2(pack2(s.x, s.y, dtype), pack2(s.z, s.w, dtype));
        *reinterpret_cast<uint2 *>(static_cast<unsigned short *>(to) + at) = w;
    } else {
        const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c + k < cols) img_store(to, at + k, dtype, v[k]);
    }
}

// The largest finite |v| of a job's arrays (blockIdx.y), a partial maximum per block of
// the kBoundParts across.  Maxima drop NaN by themselves; a thread that met an infinity
// looks again, element by element.  (16384 x 1024 in fp16: 8 us with the launch.)
struct BoundJobs {
    BoundJob job[3];
};
__device__ __forceinline__ unsigned larger2(unsigned m, unsigned w, int dtype) {
    w &= 0x7fff7fffu;
    if (dtype == PDR_F16) {
        const __half2 h = __hmax2(*reinterpret_cast<const __half2 *>(&m), *reinterpret_cast<const __half2 *>(&w));
        return *reinterpret_cast<const unsigned *>(&h);
    }
    const __nv_bfloat162 h =
        __hmax2(*reinterpret_cast<const __nv_bfloat162 *>(&m), *reinterpret_cast<const __nv_bfloat162 *>(&w));
    return *reinterpret_cast<const unsigned *>(&h);
}
__device__ __forceinline__ float larger(float m, float v) {
    const float a = fabsf(v);
    return a <= 3.402823466e38f ? fmaxf(m, a) : m;
}
constexpr int kLargestThreads = 256;
__global__ void __launch_bounds__(kLargestThreads)
    k_largest(const __grid_constant__ BoundJobs jobs, float *__restrict__ part) {
    __shared__ float warps[kLargestThreads / 32];
    grid_dep_wait();
    const BoundJob &j = jobs.job[blockIdx.y];
    const int E = j.dtype == PDR_F32 ? 4 : 8;
    const long long vectors = j.n / E, step = (long long)kBoundParts * kLargestThreads;
    const long long first = (long long)blockIdx.x * kLargestThreads + threadIdx.x;
    float m = 0.0f;
    for (int a = 0; a < (j.p2 ? 2 : 1); ++a) {
        const uint4 *p = static_cast<const uint4 *>(a ? j.p2 : j.p);
        float f = 0.0f;
        unsigned h = 0;
        for (long long i = first; i < vectors; i += 8 * step) {
            uint4 u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = i + k * step < vectors ? __ldg(p + i + k * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const unsigned w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (E == 4)
                        f = fmaxf(f, fabsf(__uint_as_float(w[i])));
                    else
                        h = larger2(h, w[i], j.dtype);
            }
        }
        if (E == 8) {
            const float2 two = unpack2(h, j.dtype);
            f = fmaxf(two.x, two.y);
        }
        if (f > 3.402823466e38f) {
            f = 0.0f;
            for (long long i = first; i < vectors; i += step)
                for (int k = 0; k < E; ++k) f = larger(f, img_load(p, (size_t)(i * E + k), j.dtype));
        }
        m = fmaxf(m, f);
        if (first < j.n - vectors * E) m = larger(m, img_load(p, (size_t)(vectors * E + first), j.dtype));
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x) return;
    for (int i = 1; i < kLargestThreads / 32; ++i) m = fmaxf(m, warps[i]);
    part[blockIdx.y * kBoundParts + blockIdx.x] = m;
}

// dy is taken in vectors of 16 bytes; a thread keeps its vector of the rows, and so its
// columns.
struct ColumnPlan {
    int vectors;              // of a row (the last one may lie behind its end in part)
    long long group;          // rows of a block
    unsigned blocks, across;  // down the rows, and across 256 vectors each
};
ColumnPlan column_plan(long long M, int N, int bytes) {
    const int E = 16 / bytes;
    ColumnPlan p = {};
    p.vectors = (N + E - 1) / E;
    p.across = (unsigned)((p.vectors + 255) / 256);
    // Four blocks an SM.
    const int per = p.vectors < 256 ? 256 / p.vectors : 1;
    long long blocks = 4 * kSMs / p.across;
    if (blocks > M / per) blocks = M / per;
    if (blocks < 1) blocks = 1;
    p.group = (M + blocks - 1) / blocks;
    p.blocks = M > 0 ? (unsigned)((M + p.group - 1) / p.group) : 0;
    return p;
}

// What rounding v to r leaves (an infinity stays one).
__device__ __forceinline__ float rest(float v, float r) { return fabsf(r) <= 3.402823466e38f ? v - r : 0.0f; }

// (Backward of 131072 x 256 to 256 columns, bf16 and a bias: 83 us with a cold L2, by single elements
// 180; of 30000 x 256 to 777 columns, whose rows start anywhere, 69 and 110.)
template <typename T>
__global__ void __launch_bounds__(256) k_cast_columns(const T *__restrict__ dy, int dy_dtype,
                                                      long long M, int N, ColumnPlan p,
                                                      void *__restrict__ dz, int dz_dtype,
                                                      long long ldz, int low, const TwiceJob two,
                                                      float *__restrict__ colsum, const Bound bound) {
    constexpr int E = 16 / sizeof(T);
    __shared__ float sums[256][E + 1];
    grid_dep_wait();
    const long long r0 = blockIdx.x * p.group, r1 = r0 + p.group < M ? r0 + p.group : M;
    const int base = blockIdx.y * 256, width = p.vectors - base < 256 ? p.vectors - base : 256;
    const int per = 256 / width;  // rows at once
    const int sub = threadIdx.x / width, j = base + threadIdx.x % width;
    const bool whole = N % E == 0;  // rows start at 16 bytes
    const float factor = bound.part ? bound_factor(bound, false) : 1.0f;
    if (E == 4 && two.to) {
        const int vectors = (int)(two.ld / 8), all = 2 * low * vectors;
        for (int i = (blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x; i < all; i += gridDim.x * gridDim.y * 256) {
            const int r = i / vectors, n = r < low ? r : r - low;
            static_cast<uint4 *>(two.to)[i] =
                n < N ? padded_vector(static_cast<const unsigned short *>(two.from) + (long long)n * two.cols,
                                      i - r * vectors, two.cols)
                      : make_uint4(0, 0, 0, 0);
        }
    }
    float s[E] = {};
    if (sub < per)
        for (long long r = r0 + sub; r < r1; r += 4 * per) {
            uint4 raw[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const T *row = dy + (r + k * per) * N;
                if (r + k * per >= r1 || j * E >= N)
                    raw[k] = make_uint4(0, 0, 0, 0);
                else if (whole)
                    raw[k] = __ldg(reinterpret_cast<const uint4 *>(row) + j);
                else
                    raw[k] = padded_vector(row, j, N);  // (zeros behind the row's end)
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const unsigned w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
                float v[E];
                if constexpr (E == 4) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = unpack2(w[i], dy_dtype);
                        v[2 * i] = f.x;
                        v[2 * i + 1] = f.y;
                    }
                }
#pragma unroll
                for (int i = 0; i < E; ++i) s[i] += v[i];
                if (!dz || r + k * per >= r1) continue;
                unsigned h[E / 2];
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] *= factor;
#pragma unroll
                for (int i = 0; i < E / 2; ++i) h[i] = pack2(v[2 * i], v[2 * i + 1], dz_dtype);
                // (Padded rows hold whole vectors.)
                unsigned short *to = static_cast<unsigned short *>(dz) + (r + k * per) * ldz + j * E;
                if constexpr (E == 4) {
                    *reinterpret_cast<uint2 *>(to) = make_uint2(h[0], h[1]);
                    if (low) {
                        const float2 a = unpack2(h[0], dz_dtype), b = unpack2(h[1], dz_dtype);
                        *reinterpret_cast<uint2 *>(to + low) = make_uint2(
                            pack2(rest(v[0], a.x), rest(v[1], a.y), dz_dtype), pack2(rest(v[2], b.x), rest(v[3], b.y), dz_dtype));
                    }
                } else
                    *reinterpret_cast<uint4 *>(to) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
    if (!colsum || blockIdx.x >= p.blocks) return;
    for (int half = 128; half >= 1; half /= 2) {  // the upper half of the rows to the lower, in turn
        if (half >= per) continue;
        if (sub >= half && sub < 2 * half && sub < per)
#pragma unroll
            for (int i = 0; i < E; ++i) sums[threadIdx.x][i] = s[i];
        __syncthreads();
        if (sub < half && sub + half < per)
#pragma unroll
            for (int i = 0; i < E; ++i) s[i] += sums[threadIdx.x + half * width][i];
    }
    if (sub == 0)
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (j * E + i < N) colsum[(long long)blockIdx.x * N + j * E + i] = s[i];
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

// The map of a result (`slices` of rows x cols, one behind the other) for the
// stores of 32 rows by 64 bytes.
bool make_store_map(CUtensorMap *m, void *to, int bytes, long long rows, long long cols,
                    long long ld, int slices) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)slices};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * bytes, (cuuint64_t)ld * bytes * rows};
    const cuuint32_t box[3] = {(cuuint32_t)(64 / bytes), 32, 1}, unit[3] = {1, 1, 1};
    return f(m, bytes == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, to,
             dims, strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared-memory descriptor of an operand tile, without its address: 128-byte
// swizzle; 8-row (K-major) or 8-k (MN-major) groups 1024 bytes apart, and for
// MN-major the 64-wide blocks 8192 bytes apart.
unsigned long long smem_desc(bool mn) {
    return ((unsigned long long)(mn ? 8192 >> 4 : 1) << 16) |
           ((unsigned long long)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

template <int EPI, int ACT, bool NARROW, int NP>
cudaError_t launch_as(const GemmLaunch<NP> &l, int grid, size_t smem, cudaStream_t s) {
    // The kernel's shared-memory limit, raised once per device.
    static std::atomic<unsigned long long> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev > 63 || !(raised.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(k_gemm<EPI, ACT, NARROW, NP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemBytes);
        if (e != cudaSuccess) return e;
        raised.fetch_or(bit, std::memory_order_release);
    }
    return launch_dependent(k_gemm<EPI, ACT, NARROW, NP>, dim3((unsigned)grid), dim3(kThreads), smem, s, l);
}
template <int EPI, int ACT>
cudaError_t launch_act(const GemmLaunch<1> &l, int grid, size_t smem, cudaStream_t s) {
    if constexpr (EPI == kEpiLinear)
        if (l.p[0].narrow) return launch_as<EPI, ACT, true, 1>(l, grid, smem, s);
    return launch_as<EPI, ACT, false, 1>(l, grid, smem, s);
}
template <int EPI>
cudaError_t launch(const GemmLaunch<1> &l, int act, int grid, size_t smem, cudaStream_t s) {
    switch (act) {
        case PDR_ACT_RELU: return launch_act<EPI, PDR_ACT_RELU>(l, grid, smem, s);
        case PDR_ACT_SILU: return launch_act<EPI, PDR_ACT_SILU>(l, grid, smem, s);
        case PDR_ACT_GELU: return launch_act<EPI, PDR_ACT_GELU>(l, grid, smem, s);
        case PDR_ACT_GELU_TANH: return launch_act<EPI, PDR_ACT_GELU_TANH>(l, grid, smem, s);
        default:
            if constexpr (EPI == kEpiSlope)
                return cudaErrorInvalidValue;  // (no activation, no slope: its callers read dy itself)
            else
                return launch_act<EPI, PDR_ACT_NONE>(l, grid, smem, s);
    }
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

Divisor divisor(int d) {
    unsigned l = 0;
    while ((1u << l) < (unsigned)d) ++l;
    return {(unsigned)d, (unsigned)((1ull << (31 + l)) / (unsigned)d + 1), l - 1};
}

}  // namespace

// (524288 x 256 to 6 fp32 columns with a residual: 50 us, through padded copies 143.)
bool gemm_narrow(int N, int out_dtype, bool has_in) {
    const int row = N * dtype_bytes(out_dtype);
    return N <= kChunk && (row % 16 || (has_in && row % 32));
}

// Columns of a tile of a result of M x N (x nz products) over kb k blocks.
static int gemm_tile_columns(int epi, int M, int N, int nz, long long kb) {
    const bool dual = epi == kEpiGated || epi == kEpiGatedBwd;
    // The width whose rounds of tiles over the pairs take least, in clocks as
    // measured: 560 + 4/3 per accumulator column and k block (the copies' way
    // from L2 bounds them), 300 + 16 per column in the epilogue beside the next tile's
    // products, and the first tile's start and the last one's end.  (Without the 300, short k
    // took narrow tiles: gated 49152 x 64 to 1024 62 against 42 us.)
    int best = 32;
    double least = -1;
    for (int c = dual ? 128 : 256; c >= 32; c /= 2) {
        const long long tiles = (long long)ceil_div(M, 2 * kBM) * ceil_div(N, c) * nz;
        const int bn = dual ? 2 * c : c;
        const double products = kb * (560 + 4 * bn / 3), ends = 300 + 16.0 * bn;
        const double cost = (tiles + kSMs / 2 - 1) / (kSMs / 2) * (products > ends ? products : ends) +
                            3000 + ends;
        if (least < 0 || cost < least) {
            least = cost;
            best = c;
        }
    }
    return best;
}

int gemm_splits(int M, int N, int nz, long long K) {
    const int cols = gemm_tile_columns(kEpiLinear, 1 << 30, N, nz, 32);
    const long long tiles = (long long)ceil_div(M, 2 * kBM) * ceil_div(N, cols) * nz;
    const long long kb = (K + 63) / 64;
    long long s = kSMs / 2 / tiles;
    if (s > kb / 4) s = kb / 4;  // at least 4 stages of k each
    return s < 1 ? 1 : (int)s;
}

namespace {
// The current device's word, null where there is no memory for it.
int *wait_word() {
    int *words = g_wait_words.load(std::memory_order_acquire);
    if (!words) {  // (relaxed: the first launch may be in a stream that is being captured)
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return nullptr;
        void *p = nullptr;
        const cudaError_t e = cudaHostAlloc(&p, kDevices * sizeof(int), cudaHostAllocPortable | cudaHostAllocMapped);
        if (e == cudaSuccess) {
            memset(p, 0, kDevices * sizeof(int));
            if (g_wait_words.compare_exchange_strong(words, static_cast<int *>(p)))
                words = static_cast<int *>(p);
            else
                cudaFreeHost(p);  // another thread was first: its words
        }
        cudaThreadExchangeStreamCaptureMode(&mode);
        if (e != cudaSuccess) return nullptr;
    }
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? words + dev % kDevices : nullptr;
}

int tile_columns(const GemmArgs &g) {
    const int kelems = g.dtype == PDR_E4M3 ? kRowBytes : kRowBytes / 2, nz = g.mode == kBatchA ? 2 : 1;
    if (g.splits > 1) return gemm_tile_columns(g.epi, 1 << 30, g.N, nz, 32);
    return gemm_tile_columns(g.epi, g.M, g.N, nz, ceil_div(g.K[0], kelems) + ceil_div(g.K[1], kelems));
}

// Everything of a product but its shared memory.
cudaError_t plan(const GemmArgs &g, int bcols, GemmParams &p) {
    const bool dual = g.mode == kDualB;
    const int bytes = g.dtype == PDR_E4M3 ? 1 : 2;
    const int kelems = kRowBytes / bytes;
    p = {};
    p.mode = g.mode;
    p.a_mn = g.a_mn;
    p.b_mn = g.b_mn;
    p.M = g.M;
    p.N = g.N;
    p.nz = g.mode == kBatchA ? 2 : 1;
    p.splits = g.splits;
    p.kb0 = ceil_div(g.K[0], kelems);
    p.kb = p.kb0 + (g.mode == kTwoSources ? ceil_div(g.K[1], kelems) : 0);
    p.kelems = kelems;
    p.bcols = bcols;
    p.bn = dual ? 2 * p.bcols : p.bcols;
    p.nm = divisor(ceil_div(g.M, 2 * kBM));
    p.nn = divisor(ceil_div(g.N, p.bcols));
    const long long tiles = (long long)p.nm.d * p.nn.d * p.nz * p.splits;
    if (tiles > 1 << 30) return cudaErrorInvalidValue;
    p.tiles = (int)tiles;
    p.b_bytes = g.b_mn ? ceil_div(p.bn / 2, 64) * 8192 : p.bn / 2 * kRowBytes;
    p.nacc = p.bn >= 256 ? 2 : 4;
    p.fp8 = bytes == 1;
    // D fp32 | A and B: f16 0, bf16 1 (kind::f16) or e4m3 0 (kind::f8f6f4) | majors | N / 8 | M / 16
    const unsigned t = g.dtype == PDR_BF16 ? 1 : 0;
    p.idesc = (1u << 4) | (t << 7) | (t << 10) | ((unsigned)g.a_mn << 15) |
              ((unsigned)g.b_mn << 16) | ((unsigned)(p.bn / 8) << 17) | ((unsigned)(2 * kBM / 16) << 24);
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
                      g.b_mn ? 64 : p.bn / 2))
            return cudaErrorInvalidValue;
    const int ob = dtype_bytes(g.out_dtype), ib = dtype_bytes(g.in_dtype);
    p.out = g.out;
    p.out_dtype = g.out_dtype;
    p.narrow = g.narrow;
    // Results and inputs as the callers lay them out: see GemmArgs.
    if (p.narrow ? g.epi != kEpiLinear || p.nz > 1 || g.splits > 1 || g.N > kChunk || g.ldo != g.N || (g.in && g.ldi != g.N)
                 : g.ldo * ob % 16 || !aligned_to(g.out, 16) || !aligned_to(g.out2, 16) ||
                       (g.in && (g.ldi * ib % 32 || !aligned_to(g.in, 32))))
        return cudaErrorInvalidValue;
    const int slices = g.out_split || g.out_z ? p.splits * p.nz : 1;
    for (int i = 0; !p.narrow && i < (g.out2 ? 2 : 1); ++i)
        if (!make_store_map(&p.o[i], i ? g.out2 : g.out, ob, g.M, g.N, g.ldo, slices))
            return cudaErrorInvalidValue;
    p.bias = g.bias;
    p.bias_dtype = g.bias_dtype;
    p.scale_m = g.scale_m;
    p.scale_n = g.scale_n;
    p.scale_n2 = g.scale_n2;
    p.in = g.in;
    p.in_dtype = g.in_dtype;
    p.ldi = g.ldi;
    p.colsum = g.colsum;
    p.bound = g.bound;
    p.tries = g_wait_tries.load(std::memory_order_relaxed);
    p.wait_word = wait_word();
    return p.wait_word ? cudaSuccess : cudaErrorMemoryAllocation;
}

// Divides the columns of tiles among the pairs (stationary B): neighbouring rows of
// tiles are under way at the same time, whole rows of the matrices together, which the
// memory serves faster than as many places a column apart (65536 x 256 to 1024 columns: 39
// against 43 us, with fp32 results and a residual 138 against 150, gated backward of
// 49152 x 64 to 1024 175 against 203).
void share_columns(GemmParams &p, int pairs) {
    const int rows = p.nm.d, columns = p.nn.d * p.nz, left = pairs % columns;
    p.share = pairs / columns;
    int last = 0;  // rows for the pairs that are left over
    if (left && p.share) {
        last = (int)((long long)left * rows / pairs);
        auto rounds = [&](int x) {
            const int a = ceil_div(rows - x, p.share), b = ceil_div((long long)x * columns, left);
            return a > b ? a : b;
        };
        if (rounds(last + 1) < rounds(last)) ++last;
    }
    if (!p.share || (left && !last)) {
        p.share = 0;
        last = rows;
    }
    p.main = (rows - last) * columns;
    p.na = divisor(rows - last > 0 ? rows - last : 1);
    p.nb = divisor(last > 0 ? last : 1);
}

// Shared memory of a product, or of two with `tiles` in all and the same tile sizes.
size_t plan_memory(GemmParams &p, int epi, int tiles, bool may_stay) {
    // Two or four groups share a tile, 64 columns a warp, and sets of groups take
    // tiles in turn (gated: 63 us, with 32 columns a warp 66; in 8 bits 72 and 78); a pair's
    // only tile is shared by all that it has 32 columns for.
    p.sharing = tiles <= kSMs / 2 ? p.bcols / kStore : p.bcols / kMaxCols;
    p.sharing = p.sharing < 1 ? 1 : p.sharing > kGroups ? kGroups : p.sharing;
    const size_t all_b = (size_t)p.kb * p.b_bytes;
    const int pairs = tiles < kSMs / 2 ? tiles : kSMs / 2;
    p.columns = p.fp8 ? 3 * kMaxCols : p.bias ? kMaxCols : 0;
    if (p.narrow) p.columns = 2 * kMaxCols;
    const size_t fixed = 1024 + 512 + kEpiWarps * p.columns * 4, buffers = kEpiWarps * kBufferBytes;
    const bool both = epi == kEpiGatedBwd;  // dg and du have a buffer each
    size_t room = kSmemBytes - fixed - (both ? 2 : 1) * buffers;
    // B stays where it leaves room for three stages of A and a pair has several
    // tiles to use it for (65536 x 256 to 1024 columns with silu: 62 against 67 us, gated in
    // 8 bits 72 against 76, to 8 columns 50 against 53).
    p.stationary = may_stay && p.splits == 1 && all_b + 3 * kABytes <= room && p.tiles >= 2 * pairs;
    if (p.stationary) share_columns(p, pairs);
    // A second buffer for each epilogue warp, where that takes no stage that is needed
    // (524288 x 256 to 8 columns: 50 against 51 us; 65536 x 256 to 1024 with gelu and a
    // residual 109 against 113).
    p.nbuf = both || (p.stationary && all_b + 4 * kABytes + buffers <= room) ? 2 : 1;
    if (!both) room -= (p.nbuf - 1) * buffers;
    // A stage of two k blocks, where there are as many and room for three stages,
    // halves the waits and counts beside the copies and products: one thread takes some 700
    // clocks for those of a stage beside a busy epilogue, as long as 16 KB take at
    // the memory's rate.
    const size_t left = room - (p.stationary ? all_b : 0);
    p.per_stage = p.stationary && p.kb > 1 && left >= 6 * kABytes ? 2 : 1;
    const size_t stage = p.per_stage * (kABytes + (p.stationary ? 0 : p.b_bytes));
    p.stages = (int)(left / stage);
    if (p.stages > kMaxStages) p.stages = kMaxStages;
    static_assert(sizeof(Barriers) <= 512, "barriers fit their place");
    return fixed + p.nbuf * buffers + p.stages * stage + (p.stationary ? all_b : 0);
}

int blocks_of(int tiles) { return 2 * (tiles < kSMs / 2 ? tiles : kSMs / 2); }
}  // namespace

cudaError_t launch_gemm(const GemmArgs &g, cudaStream_t s) {
    GemmLaunch<1> l;
    GemmParams &p = l.p[0];
    const cudaError_t e = plan(g, tile_columns(g), p);
    if (e != cudaSuccess) return e;
    const size_t smem = plan_memory(p, g.epi, p.tiles, true);
    const int grid = blocks_of(p.tiles);
    switch (g.epi) {
        case kEpiGated: return launch<kEpiGated>(l, g.act, grid, smem, s);
        case kEpiSlope: return launch<kEpiSlope>(l, g.act, grid, smem, s);
        case kEpiGatedBwd: return launch<kEpiGatedBwd>(l, g.act, grid, smem, s);
        default: return launch<kEpiLinear>(l, g.act, grid, smem, s);
    }
}

cudaError_t launch_gemm2(const GemmArgs &g0, const GemmArgs &g1, cudaStream_t s) {
    GemmLaunch<2> l;
    const int c0 = tile_columns(g0), c1 = tile_columns(g1);
    cudaError_t e = plan(g0, c0, l.p[0]);
    if (e != cudaSuccess) return e;
    // Together they took 26 us, one after the other 32 (dx and dW of 16384 x 256 to 1024;
    // the gated backward pass 68 and 74), and 33 against 39 where the first alone would
    // keep its B in shared memory (40722 x 440 to 8).  Apart where one is narrow.
    if (g0.narrow || g1.narrow) {
        e = launch_gemm(g0, s);
        return e == cudaSuccess ? launch_gemm(g1, s) : e;
    }
    const int c = c0 > c1 ? c0 : c1;
    if (c != c0) e = plan(g0, c, l.p[0]);
    if (e == cudaSuccess) e = plan(g1, c, l.p[1]);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)l.p[0].tiles + l.p[1].tiles;
    if (tiles > 1 << 30 || l.p[0].b_bytes != l.p[1].b_bytes) return cudaErrorInvalidValue;
    const size_t smem = plan_memory(l.p[0], g0.epi, (int)tiles, false);
    plan_memory(l.p[1], g1.epi, (int)tiles, false);
    return launch_as<kEpiLinear, PDR_ACT_NONE, false, 2>(l, blocks_of((int)tiles), smem, s);
}

namespace {
unsigned copy_blocks(long long rows) {
    return (unsigned)(rows / 8 + 1 < 16 * kSMs ? rows / 8 + 1 : 16 * kSMs);
}
template <typename T>
cudaError_t unpack_as(const void *from, long long rows, long long cols, long long ld, void *to, cudaStream_t s) {
    return launch_dependent(k_unpack<T>, dim3(copy_blocks(rows)), dim3(256), 0, s,
                            static_cast<const T *>(from), rows, (int)cols, (int)ld, static_cast<T *>(to));
}
}  // namespace

cudaError_t launch_pack(const PackJob *jobs, int n, cudaStream_t s) {
    PackJobs p = {};
    for (int i = 0; i < n; ++i)
        if (jobs[i].rows > 0) {
            p.job[p.n] = jobs[i];
            p.first[p.n + 1] = p.first[p.n] + copy_blocks(jobs[i].rows);
            ++p.n;
        }
    if (p.n == 0) return cudaSuccess;
    return launch_dependent(k_pack, dim3(p.first[p.n]), dim3(256), 0, s, p);
}
cudaError_t launch_unpack(const void *from, long long rows, long long cols, long long ld, int bytes,
                          void *to, cudaStream_t s) {
    return bytes == 2 ? unpack_as<unsigned short>(from, rows, cols, ld, to, s)
                      : unpack_as<unsigned>(from, rows, cols, ld, to, s);
}

cudaError_t launch_join(const float *part, int splits, int rows, int cols, long long ld, long long slice,
                        void *to, void *to2, int dtype, const ColumnJob &columns, cudaStream_t s) {
    const long long vectors = rows * ld / 4;
    // (Always Y = 8: gated backward with 1024 x 256 weights 75 against 68 us.  Always Y = 1:
    // backward of 131072 x 256 to 8 columns 60 against 57, to 256 columns 172 against 170.)
    const bool few = vectors < 256 * kSMs;
    const unsigned blocks = (unsigned)((vectors + (few ? 31 : 255)) / (few ? 32 : 256));
    const dim3 grid(blocks + (unsigned)((columns.cols + 7) / 8), to2 ? 2 : 1);
    return launch_dependent(few ? k_join<8> : k_join<1>, grid, dim3(256), 0, s, part, splits, rows, cols, ld,
                            slice, to, to2, dtype, blocks, columns);
}

cudaError_t launch_join_columns(const ColumnJob &columns, cudaStream_t s) {
    return launch_dependent(k_join_columns, dim3((unsigned)((columns.cols + 7) / 8)), dim3(256), 0, s, columns);
}

long long column_groups(long long M, int N, int dy_dtype, int low) {
    return column_plan(M, low ? low : N, dtype_bytes(dy_dtype)).blocks;
}

cudaError_t launch_cast_columns(const void *dy, int dy_dtype, long long M, int N, void *dz,
                                int dz_dtype, long long ldz, int low, const TwiceJob &two,
                                float *colsum, const Bound &bound, cudaStream_t s) {
    const ColumnPlan p = column_plan(M, low ? low : N, dtype_bytes(dy_dtype));
    // (Few rows: more blocks for the weight alone.)
    const long long copies = two.to ? (2 * low * two.ld / 8 + 255) / 256 : 0;
    const dim3 grid((unsigned)(copies > p.blocks ? (copies < 4 * kSMs ? copies : 4 * kSMs) : p.blocks), p.across);
    if (dy_dtype == PDR_F32)
        return launch_dependent(k_cast_columns<float>, grid, dim3(256), 0, s, static_cast<const float *>(dy),
                                dy_dtype, M, N, p, dz, dz_dtype, ldz, low, two, colsum, bound);
    return launch_dependent(k_cast_columns<unsigned short>, grid, dim3(256), 0, s,
                            static_cast<const unsigned short *>(dy), dy_dtype, M, N, p, dz, dz_dtype,
                            ldz, 0, two, colsum, bound);
}

cudaError_t launch_largest(const BoundJob *jobs, int n, float *part, cudaStream_t s) {
    BoundJobs j = {};
    for (int i = 0; i < n; ++i) j.job[i] = jobs[i];
    return launch_dependent(k_largest, dim3(kBoundParts, (unsigned)n), dim3(kLargestThreads), 0, s, j, part);
}

void set_wait_tries(int tries) {
    g_wait_tries.store(tries < 0 ? kWaitTries : tries, std::memory_order_relaxed);
}

bool wait_error_pending() {
    const int *words = g_wait_words.load(std::memory_order_acquire);
    int dev = 0;
    if (!words || cudaGetDevice(&dev) != cudaSuccess) return false;
    return *(volatile const int *)(words + dev % kDevices) != 0;
}

cudaError_t read_wait_error(int *bits, cudaStream_t s) {
    const cudaError_t e = cudaStreamSynchronize(s);
    *bits = wait_error_pending();
    if (*bits) *(volatile int *)wait_word() = 0;
    return e;
}

}  // namespace pdr
