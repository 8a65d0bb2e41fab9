// Orthogonalised update of a matrix by Newton-Schulz products, with the momentum step in front
// (spl_orthogonalize; declared in include/spl_local.h).
//
//   u = G, or M <- mu M + G and u = G + mu M (nesterov) or M
//   X = u / (|u|_F + eps), transposed if it has more rows than columns (m <= n below)
//   `steps` times:  A = X X^T,  B = b A + c A A,  X <- a X + B X
//
// which moves every singular value of X towards 1.  The three products run on the tensor cores
// (tcgen05, fp16 operands by TMA, fp32 accumulators in tensor memory).  A and A A are symmetric:
// only tiles that touch the lower triangle are computed, each value written to both places.
//
// Number formats.  Operands are fp16: 11 significant bits, against bf16's 8 (a bf16 operand
// would leave 1 % to 18 % of error in the result, growing with the spread of the singular
// values).  fp16's short range is met by fixed powers of two: X is held times x_scale =
// 2^round(log2(n) / 2), which brings its entries near 1 (they are near n^-1/2), A and B times
// 2^10 (diagonals near 1, off-diagonals down to 1e-6).  The state X itself keeps 22 bits, as
// the sum of two fp16 planes hi + lo 2^-11: rounding X to 11 bits in every step would feed noise
// of 2^-12 of the largest singular direction into the smallest ones, which the iteration then
// amplifies (2e-2 of error on steep spectra; with the two planes 1e-3 to 1.7e-3 on all of them,
// below the 1.7e-3 of the output's own rounding to bf16).  Only hi enters the products.
#include <cuda.h>
#include <cuda_fp16.h>

#include <cmath>
#include <mutex>
#include <type_traits>

#include "local_device.cuh"
#include "local_kernels.h"

namespace spl {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kGramScale = 1024.0f;    // of A and B
constexpr float kLoScale = 2048.0f;      // of the state's low plane

// ---- momentum, norm, state ------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr int kMaxPartials = 1216;  // sums of squares per matrix: eight CTAs per SM
constexpr int kMaxPhases = 160;     // of the run kernel below
constexpr int kMaxSlots = 32;       // of matrices with counters of their own

struct PrepArgs {
    const void* update;
    int64_t rows, cols, row_stride, batch_stride;
    float* momentum;
    float mu;
    bool nesterov;
    float eps, x_scale;
    double* partials;   // [batch][kMaxPartials]
    int num_partials;
    __half* hi;         // [batch][m][ld]
    __half* lo;
    int64_t ld, plane;  // plane = m * ld
    uint32_t* arrived;  // the run kernel's phase counters, cleared here
    uint32_t* flags;
};

// u of one entry once the momentum holds its new value.
__device__ __forceinline__ float step_value(float g, float m, const PrepArgs& p) {
    if (p.momentum == nullptr) return g;
    return p.nesterov ? __fmaf_rn(p.mu, m, g) : m;
}

// A matrix as a flat range of units (16-byte vectors of the update where its rows allow, single
// values otherwise): a CTA takes kPrepUnits per thread at a time, so that short rows share a CTA.
constexpr int kPrepUnits = 4;

template <bool kBf16, bool kVec>
struct PrepUnit {
    static constexpr int kN = kVec ? Vec16<kBf16>::kN : 1;
    float x[kN];

    __device__ __forceinline__ void load(const PrepArgs& p, int64_t b, int64_t r, int64_t u) {
        const unsigned char* row = static_cast<const unsigned char*>(p.update) +
                                   (b * p.batch_stride + r * p.row_stride) * Vec16<kBf16>::kBytes;
        if constexpr (kVec) Vec16<kBf16>::unpack(reinterpret_cast<const uint4*>(row)[u], x);
        else x[0] = Vec16<kBf16>::load1(row, u);
    }
    __device__ __forceinline__ void load_momentum(const float* m) {
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < kN; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(m + i);
                x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
            }
        } else {
            x[0] = *m;
        }
    }
    __device__ __forceinline__ void store_momentum(float* m) const {
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < kN; i += 4)
                *reinterpret_cast<float4*>(m + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        } else {
            *m = x[0];
        }
    }
};

// The momentum step and each CTA's share of |u|^2.
template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kPrepThreads) k_orth_norm(const __grid_constant__ PrepArgs p) {
    using U = PrepUnit<kBf16, kVec>;
    __shared__ double s_sum[kPrepThreads / 32];
    const int64_t b = blockIdx.y;
    if (blockIdx.x == 0 && b == 0)
        for (int i = threadIdx.x; i < kMaxPhases * kMaxSlots; i += kPrepThreads) p.arrived[i] = 0;
    const uint32_t per_row = static_cast<uint32_t>(p.cols / U::kN);
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kPrepThreads * kPrepUnits);
    double total = 0.0;
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * (kPrepThreads * kPrepUnits);
         first < p.rows * per_row; first += step) {
        const int64_t row0 = first / per_row;
        const uint32_t rem0 = static_cast<uint32_t>(first - row0 * per_row);
        U g[kPrepUnits], m[kPrepUnits];
        int64_t at[kPrepUnits];
#pragma unroll
        for (int k = 0; k < kPrepUnits; ++k) {
            const uint32_t i = rem0 + k * kPrepThreads + threadIdx.x;
            const int64_t r = row0 + i / per_row;
            at[k] = -1;
            if (r >= p.rows || !SPL_CHECK(r < p.rows, kSiteOrthIn, r)) continue;
            const uint32_t u = i % per_row;
            g[k].load(p, b, r, u);
            at[k] = (b * p.rows + r) * p.cols + static_cast<int64_t>(u) * U::kN;
            if (p.momentum != nullptr) m[k].load_momentum(p.momentum + at[k]);
        }
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kPrepUnits; ++k) {
            if (at[k] < 0) continue;
#pragma unroll
            for (int i = 0; i < U::kN; ++i) {
                if (p.momentum != nullptr) m[k].x[i] = __fmaf_rn(p.mu, m[k].x[i], g[k].x[i]);
                const float u = step_value(g[k].x[i], m[k].x[i], p);
                sum = __fmaf_rn(u, u, sum);
            }
            if (p.momentum != nullptr) m[k].store_momentum(p.momentum + at[k]);
        }
        total += static_cast<double>(sum);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(kAll, total, off);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kPrepThreads / 32; ++w) total += s_sum[w];
        p.partials[b * kMaxPartials + blockIdx.x] = total;
    }
}

// x_scale / (|u| + eps) of matrix b, the same in every thread of the CTA.
__device__ __forceinline__ float state_factor(const PrepArgs& p, int64_t b) {
    __shared__ double s_sum[kPrepThreads / 32];
    __shared__ float s_factor;
    double total = 0.0;
    for (int i = threadIdx.x; i < p.num_partials; i += kPrepThreads)
        total += p.partials[b * kMaxPartials + i];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(kAll, total, off);
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kPrepThreads / 32; ++w) total += s_sum[w];
        const float norm = static_cast<float>(sqrt(total));
        s_factor = __fdiv_rn(p.x_scale, __fadd_rn(norm, p.eps));
        if (!(norm <= 3.402823466e+38f)) {
            s_factor = __uint_as_float(0x7fc00000u);
            if (p.flags != nullptr) atomicOr(p.flags, kFlagNonFinite);
        }
    }
    __syncthreads();
    return s_factor;
}

__device__ __forceinline__ float nan_value() { return __uint_as_float(0x7fc00000u); }

__device__ __forceinline__ void split_state(float x, __half& hi, __half& lo) {
    hi = __float2half_rn(x);
    lo = __float2half_rn(__fmul_rn(__fsub_rn(x, __half2float(hi)), kLoScale));
}

// kN consecutive values of the state's two planes.
template <int kN>
__device__ __forceinline__ void store_state(const PrepArgs& p, int64_t at, const float* x) {
    __half h[kN], l[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) split_state(x[i], h[i], l[i]);
    if constexpr (kN == 8) {
        *reinterpret_cast<uint4*>(p.hi + at) = *reinterpret_cast<const uint4*>(h);
        *reinterpret_cast<uint4*>(p.lo + at) = *reinterpret_cast<const uint4*>(l);
    } else if constexpr (kN == 4) {
        *reinterpret_cast<uint2*>(p.hi + at) = *reinterpret_cast<const uint2*>(h);
        *reinterpret_cast<uint2*>(p.lo + at) = *reinterpret_cast<const uint2*>(l);
    } else {
        p.hi[at] = h[0];
        p.lo[at] = l[0];
    }
}

// X = u / (|u| + eps) in the state's format.
template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kPrepThreads) k_orth_state(const __grid_constant__ PrepArgs p) {
    using U = PrepUnit<kBf16, kVec>;
    const int64_t b = blockIdx.y;
    const float f = state_factor(p, b);
    const uint32_t per_row = static_cast<uint32_t>(p.cols / U::kN);
    const int64_t step = static_cast<int64_t>(gridDim.x) * (kPrepThreads * kPrepUnits);
    for (int64_t first = static_cast<int64_t>(blockIdx.x) * (kPrepThreads * kPrepUnits);
         first < p.rows * per_row; first += step) {
        const int64_t row0 = first / per_row;
        const uint32_t rem0 = static_cast<uint32_t>(first - row0 * per_row);
        U g[kPrepUnits], m[kPrepUnits];
        int64_t at[kPrepUnits];
#pragma unroll
        for (int k = 0; k < kPrepUnits; ++k) {
            const uint32_t i = rem0 + k * kPrepThreads + threadIdx.x;
            const int64_t r = row0 + i / per_row;
            at[k] = -1;
            if (r >= p.rows || !SPL_CHECK(r < p.rows, kSiteOrthIn, r)) continue;
            const uint32_t u = i % per_row;
            g[k].load(p, b, r, u);
            if (p.momentum != nullptr)
                m[k].load_momentum(p.momentum + (b * p.rows + r) * p.cols + static_cast<int64_t>(u) * U::kN);
            at[k] = b * p.plane + r * p.ld + static_cast<int64_t>(u) * U::kN;
        }
#pragma unroll
        for (int k = 0; k < kPrepUnits; ++k) {
            if (at[k] < 0) continue;
#pragma unroll
            for (int i = 0; i < U::kN; ++i) g[k].x[i] = __fmul_rn(step_value(g[k].x[i], m[k].x[i], p), f);
            store_state<U::kN>(p, at[k], g[k].x);
        }
    }
}

// The same for a tall matrix, whose state is its transpose: 64 x 64 tiles through shared memory.
template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kPrepThreads) k_orth_state_tall(const __grid_constant__ PrepArgs p) {
    using U = PrepUnit<kBf16, kVec>;
    constexpr int kAcross = 64 / U::kN, kDown = kPrepThreads / kAcross;
    __shared__ float s_tile[64][65];
    const int64_t b = blockIdx.y;
    const float f = state_factor(p, b);
    const int64_t tiles_r = (p.rows + 63) / 64, tiles = tiles_r * ((p.cols + 63) / 64);
    const int uc = threadIdx.x % kAcross, ur = threadIdx.x / kAcross;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t r0 = t % tiles_r * 64, c0 = t / tiles_r * 64;
#pragma unroll
        for (int k = 0; k < 64 / kDown; ++k) {
            const int64_t r = r0 + ur + k * kDown, c = c0 + uc * U::kN;
            if (r >= p.rows || c >= p.cols || !SPL_CHECK(r < p.rows, kSiteOrthIn, r)) continue;
            U g, m;
            g.load(p, b, r, c / U::kN);
            if (p.momentum != nullptr) m.load_momentum(p.momentum + (b * p.rows + r) * p.cols + c);
#pragma unroll
            for (int i = 0; i < U::kN; ++i)
                s_tile[ur + k * kDown][uc * U::kN + i] = __fmul_rn(step_value(g.x[i], m.x[i], p), f);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {   // 8 of the tile's rows per thread: the state's columns
            const int c = (threadIdx.x >> 3) + 32 * k, r = (threadIdx.x & 7) * 8;
            if (c0 + c >= p.cols || r0 + r >= p.rows) continue;
            // columns up to the row pitch, a multiple of 8, are this buffer's own
            if (!SPL_CHECK(r0 + r + 8 <= p.ld, kSiteOrthState, r0 + r)) continue;
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = s_tile[r + i][c];
            store_state<8>(p, b * p.plane + (c0 + c) * p.ld + r0 + r, x);
        }
        __syncthreads();
    }
}

template <bool kBf16, bool kVec>
cudaError_t launch_prep(PrepArgs p, int64_t batch, bool tall, int sms, cudaStream_t stream) {
    const int64_t per_cta = static_cast<int64_t>(kPrepThreads) * kPrepUnits;
    const int64_t ctas = (p.rows * (p.cols / PrepUnit<kBf16, kVec>::kN) + per_cta - 1) / per_cta;
    p.num_partials = static_cast<int>(ctas < kMaxPartials ? ctas : kMaxPartials);
    const unsigned b = static_cast<unsigned>(batch);
    k_orth_norm<kBf16, kVec><<<dim3(static_cast<unsigned>(p.num_partials), b), kPrepThreads, 0, stream>>>(p);
    const int64_t most = 8 * static_cast<int64_t>(sms);   // as many as are resident, then loop
    if (tall) {
        const int64_t tiles = (p.rows + 63) / 64 * ((p.cols + 63) / 64);
        k_orth_state_tall<kBf16, kVec><<<dim3(static_cast<unsigned>(tiles < most ? tiles : most), b), kPrepThreads,
                                         0, stream>>>(p);
    } else {
        k_orth_state<kBf16, kVec><<<dim3(static_cast<unsigned>(ctas < most ? ctas : most), b), kPrepThreads, 0,
                                    stream>>>(p);
    }
    return cudaGetLastError();
}

// ---- the products ---------------------------------------------------------------------------
// All products of a call run in one persistent cooperative kernel, as a list of phases.  A phase
// names the earlier ones it needs: a unit of work waits until all their units of the same matrix are
// in memory (counted per phase and slot of matrices in the workspace).  The matrices of a stack so
// follow one another through the phases, and one's waits are filled by the others' products.  A phase computes D = A B^T (B's rows along K) or D = A B
// (B's rows along N) tile by tile, and for each tile
//
//   value = f_acc * accumulator + f1 * source1 + f2 * source2
//
// written as one fp16 plane (a symmetric product also to its mirrored place), as the state's two
// planes, or as bf16 (in place or transposed).  Per CTA: one thread issues the operands' TMA loads
// into a ring of stages, one the MMAs, one the TMA loads of the sources' 128 x 64 slabs, two
// sets of four warps turn accumulators into results in the slabs' shared memory, a slab each, and
// one thread issues the TMA stores that take them from there.  Two accumulators in tensor memory let a tile's MMAs run under the previous tile's
// epilogue.
//
// kPair = 2: two CTAs form a 256 x 256 tile (cta_group::2: each loads its 128 rows of A and half
// of B, and holds 128 rows of the result), which halves the operand traffic into shared memory;
// kPair = 1: 128 x 128 tiles, four times as many, for problems too small to fill the GPU.
//
// Every wait is bounded; on a timeout a role leaves its loops after waiting (bounded) for what it
// has in flight, the others follow by their own timeouts, and the flags word says so.
constexpr int kBlock = 128;                  // rows of a CTA's part of a tile
constexpr int kTileK = 64;
constexpr int kSlab = 64;                    // columns of an epilogue slab
constexpr int kStages = 4;
constexpr int kOperandBytes = kBlock * kTileK * 2;
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kPlaneBytes = kBlock * kSlab * 2;
constexpr int kSlabBytes = 2 * kPlaneBytes;  // the sources, replaced by results; or one of each and
                                             // its mirror image
constexpr int kSlabs = 3;                    // one per set of epilogue warps, and one being filled
constexpr int kRunThreads = 384;
constexpr int kRunSmem = kStages * kStageBytes + kSlabs * kSlabBytes + 1024;
constexpr int kMaxMatrices = 10;   // X's planes twice, the output, five m x m matrices
constexpr uint8_t kNone = 255;

enum ResultKind : uint8_t { kPlane, kState, kBf16, kBf16Transposed, kPartial };

struct Phase {
    uint8_t a, b, src1, src2, dst, dst_lo;   // matrices, or kNone
    uint8_t result;                          // ResultKind
    bool b_along_n, sym;
    bool reduce;      // sum the previous phase's partial accumulators instead of a product
    uint8_t splits;   // parts of K (results are kPartial unless 1); of a reduce: partials per tile
    int16_t after[2]; // the phases that must be complete before this one, or -1
    int16_t first;    // the group of CTAs that takes the first unit
    int n, k;         // columns of the result, length of the product
    int tile_n;       // columns of a tile: kTile, or half of a pair's
    float f_acc, f1, f2;
};

struct OrthRun {
    CUtensorMap wide[kMaxMatrices];     // boxes of 64 columns x 128 rows
    CUtensorMap narrow[kMaxMatrices];   // 64 x 64
    Phase phases[kMaxPhases];
    int num_phases, m, batch, slots;
    float* partials;      // [unit][column / 4][row][4] of kPartial phases
    uint32_t* arrived;    // a counter per phase and slot, zero at launch
    uint32_t* flags;
};

// kCtas = 2: the copy is one of a pair's, counted on the barrier of the pair's first CTA.
template <int kCtas>
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int z,
                                         uint32_t bar) {
    if constexpr (kCtas == 2)
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];"
            ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
            "[%0], [%1, {%2, %3, %4}], [%5];"
            ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar) : "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(src)) : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle (rows of 64 fp16, groups of 8 rows 1,024
// bytes apart; `lead` is the distance of neighbouring 64-wide blocks of an operand whose rows
// run along the other dimension than K).
__device__ __forceinline__ uint64_t operand_desc(const void* p, uint32_t lead) {
    const uint64_t addr = smem_addr(p);
    return ((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

template <int kCtas>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if constexpr (kCtas == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u) : "memory");
}

// Arrives on the barrier (of both CTAs of a pair) once the MMAs issued so far are done.
template <int kCtas>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    if constexpr (kCtas == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
            ::"r"(smem_addr(bar)), "h"(static_cast<uint16_t>(3)) : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     ::"r"(smem_addr(bar)) : "memory");
}

// Address of a shared variable in the pair's first CTA.
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_addr(p)));
    return a;
}

__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
                 : "memory");
}

__device__ __forceinline__ void tmem_load_32(uint32_t addr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr));
}

__device__ __forceinline__ void fence_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// Waits until a counter has reached `count`; bounded.
__device__ __forceinline__ bool counter_wait(const uint32_t* counter, uint32_t count) {
    uint32_t v;
    uint64_t t0 = 0;
    for (;;) {
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
        if (v >= count) return true;
        const uint64_t now = global_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) return false;
    }
}

// ---- units of work --------------------------------------------------------------------------
struct UnitAt {
    int b, i, j;       // matrix, tile row, tile column
    int k0, k1;        // blocks of K
    int slab0, slab1;  // slabs of the tile
    int tile;          // index of the tile over all matrices
};

template <int kPair>
struct Tiling {
    static constexpr int kTile = kBlock * kPair;   // rows of a tile, and its columns at most

    // Tiles of a symmetric product are those that reach the diagonal of their last row: tile row i
    // has kTile / tile_n (i + 1) of them, the last one no more than there are.
    static __host__ __device__ __forceinline__ int tiles(int m, const Phase& p) {
        const int tm = (m + kTile - 1) / kTile, tn = (p.n + p.tile_n - 1) / p.tile_n, ratio = kTile / p.tile_n;
        if (!p.sym) return tm * tn;
        const int in_last = ratio * tm < tn ? ratio * tm : tn;
        return ratio * (tm * (tm - 1) / 2) + in_last;
    }
    static __host__ __device__ __forceinline__ int slabs(const Phase& p) { return p.tile_n / kSlab; }
    // A reduce phase deals out single slabs, a split product parts of K.
    static __host__ __device__ __forceinline__ int units(int m, int batch, const Phase& p) {
        return tiles(m, p) * batch * (p.reduce ? slabs(p) : p.splits);
    }
    // Whether a tile of a symmetric product holds its own mirror image (or its neighbour does).
    static __device__ __forceinline__ bool on_diagonal(const Phase& p, int i, int j) {
        return j * p.tile_n / kTile == i;
    }
    static __device__ __forceinline__ UnitAt at(int m, const Phase& p, int u) {
        UnitAt a;
        const int per = p.reduce ? slabs(p) : p.splits;
        a.tile = u / per;
        const int part = u - a.tile * per;
        const int tiles_b = tiles(m, p);
        a.b = a.tile / tiles_b;
        const int r = a.tile - a.b * tiles_b;
        if (p.sym) {   // tile row i starts at ratio i (i + 1) / 2
            const int ratio = kTile / p.tile_n;
            int i = static_cast<int>((sqrtf(1.0f + 8.0f * static_cast<float>(r) / ratio) - 1.0f) * 0.5f);
            while (ratio * (i * (i + 1) / 2) > r) --i;
            while (ratio * ((i + 1) * (i + 2) / 2) <= r) ++i;
            a.i = i;
            a.j = r - ratio * (i * (i + 1) / 2);
        } else {       // groups of 8 tile rows, so that the tiles in flight share both operands
            const int tm = (m + kTile - 1) / kTile, tn = (p.n + p.tile_n - 1) / p.tile_n;
            const int g = r / (8 * tn), h = min(8, tm - 8 * g), q = r - g * 8 * tn;
            a.i = 8 * g + q % h;
            a.j = q / h;
        }
        const int blocks = (p.k + kTileK - 1) / kTileK;
        a.k0 = p.reduce ? 0 : blocks * part / p.splits;
        a.k1 = p.reduce ? 0 : blocks * (part + 1) / p.splits;
        a.slab0 = p.reduce ? part : 0;
        a.slab1 = p.reduce ? part + 1 : slabs(p);
        return a;
    }
};

// Matrices b with b % slots = s share the counters of slot s.
__host__ __device__ __forceinline__ int matrices_of(int batch, int slots, int s) {
    return batch / slots + (s < batch % slots ? 1 : 0);
}

// A role's waits for the phases before its units: each (phase, slot) once.
template <int kPair>
struct Dependencies {
    int phase, slot;
    __device__ __forceinline__ Dependencies() : phase(-1), slot(-1) {}
    __device__ __forceinline__ bool wait(const OrthRun& run, const Phase& p, int ph, int b) {
        const int s = b % run.slots;
        if (ph == phase && s == slot) return true;
        phase = ph;
        slot = s;
        bool ok = true;
        for (int i = 0; i < 2; ++i) {
            const int q = p.after[i];
            if (q < 0) continue;
            const uint32_t units = Tiling<kPair>::units(run.m, matrices_of(run.batch, run.slots, s), run.phases[q]);
            ok = ok && counter_wait(run.arrived + q * run.slots + s, units * kPair);
        }
        fence_async_all();   // what other CTAs' copies wrote, before this one's read it
        return ok;
    }
};

// Byte offset of 16-byte chunk c of row r in a 128-byte-swizzled plane.
__device__ __forceinline__ int swizzled(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

__device__ __forceinline__ void unpack_half8(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack_half8(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A row's 16-byte chunk (8 results of 16 bits) of the transposed plane.  Neighbouring lanes hold
// neighbouring rows: the even lane takes the pair of rows of the chunk's first four columns, the
// odd lane of the last four, in words of two rows.  Columns four apart differ in the swizzle's
// bit 2, so the two lanes' words fall into different halves of the banks.
__device__ __forceinline__ void store_transposed(unsigned char* plane, int row, int chunk, const uint4& w) {
    const int r = row & 62;   // 64 rows per block; the pair's first row
    const bool odd = (row & 1) != 0;
    unsigned char* block = plane + (row >> 6) * (kSlab * 128);
    const uint32_t give0 = odd ? w.x : w.z, give1 = odd ? w.y : w.w;
    const uint32_t keep0 = odd ? w.z : w.x, keep1 = odd ? w.w : w.y;
    const uint32_t got0 = __shfl_xor_sync(kAll, give0, 1), got1 = __shfl_xor_sync(kAll, give1, 1);
    const uint32_t even_row[2] = {odd ? got0 : keep0, odd ? got1 : keep1};
    const uint32_t odd_row[2] = {odd ? keep0 : got0, odd ? keep1 : got1};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = chunk * 8 + (odd ? 4 : 0) + i;
        const uint32_t out = __byte_perm(even_row[i >> 1], odd_row[i >> 1], (i & 1) ? 0x7632 : 0x5410);
        *reinterpret_cast<uint32_t*>(block + swizzled(col, r >> 3) + (r & 7) * 2) = out;
    }
}

// A thread's row of a slab: accumulators v to results in the slab's planes.  Sources are read
// ahead of the stores that may alias them.  A mirror image takes the second source's plane, so
// every warp must have read that first (`all_read`).
template <int kSources, ResultKind kResult, bool kMirror, typename AllRead>
__device__ __forceinline__ void finish_row(unsigned char* slab, int row, float (&v)[kSlab], float f_acc,
                                           float f1, float f2, AllRead all_read) {
    constexpr int kChunks = kSlab / 8;
    constexpr bool kTranspose = kMirror || kResult == kBf16Transposed;
    // with the second plane reused, all of it first; otherwise in halves, for the registers' sake
    constexpr int kAhead = kSources == 2 && kTranspose ? kChunks : kChunks / 2;
#pragma unroll
    for (int c0 = 0; c0 < kChunks; c0 += kAhead) {
        uint4 r1[kAhead], r2[kAhead];
#pragma unroll
        for (int c = 0; c < kAhead; ++c) {
            if constexpr (kSources >= 1) r1[c] = *reinterpret_cast<const uint4*>(slab + swizzled(row, c0 + c));
            if constexpr (kSources == 2)
                r2[c] = *reinterpret_cast<const uint4*>(slab + kPlaneBytes + swizzled(row, c0 + c));
        }
#pragma unroll
        for (int c = 0; c < kAhead; ++c) {
            float* x = v + 8 * (c0 + c);
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __fmul_rn(x[i], f_acc);
            if constexpr (kSources == 2) {
                unpack_half8(r2[c], y);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __fmaf_rn(f2, y[i], x[i]);
            }
            if constexpr (kSources >= 1) {
                unpack_half8(r1[c], y);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __fmaf_rn(f1, y[i], x[i]);
            }
            uint4 w;
            if constexpr (kResult == kBf16 || kResult == kBf16Transposed) {
                const float z[8] = {x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
                w = Vec16<true>::pack(z);
            } else {
                w = pack_half8(x);
            }
            if constexpr (kSources == 2 && kTranspose) r1[c] = w;   // stored below
            else if constexpr (kResult != kBf16Transposed)
                *reinterpret_cast<uint4*>(slab + swizzled(row, c0 + c)) = w;
            if constexpr (kResult == kState) {
                unpack_half8(w, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(__fsub_rn(x[i], y[i]), kLoScale);
                *reinterpret_cast<uint4*>(slab + kPlaneBytes + swizzled(row, c0 + c)) = pack_half8(y);
            }
            if constexpr (kTranspose && kSources < 2) store_transposed(slab + kPlaneBytes, row, c0 + c, w);
        }
        if constexpr (kSources == 2 && kTranspose) {
            all_read();
#pragma unroll
            for (int c = 0; c < kAhead; ++c) {
                if constexpr (kResult != kBf16Transposed)
                    *reinterpret_cast<uint4*>(slab + swizzled(row, c0 + c)) = r1[c];
                store_transposed(slab + kPlaneBytes, row, c0 + c, r1[c]);
            }
        }
    }
}

template <int kCount>
using Count = std::integral_constant<int, kCount>;
template <ResultKind kResult>
using Result = std::integral_constant<ResultKind, kResult>;

template <int kPair>
__global__ void __launch_bounds__(kRunThreads, 1) k_orth_run(const __grid_constant__ OrthRun run) {
    using T = Tiling<kPair>;
    constexpr int kAccCols = T::kTile;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* stages = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char* slabs = stages + kStages * kStageBytes;
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2],
        src_full[kSlabs], src_empty[kSlabs], done[kSlabs], read[2], drain;
    __shared__ uint32_t s_tmem;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kPair == 2 ? static_cast<int>(blockIdx.x & 1) : 0;
    const int group = blockIdx.x / kPair, groups = gridDim.x / kPair;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], 8 * kPair);
            mbar_init(&read[s], 4);
        }
        for (int s = 0; s < kSlabs; ++s) {
            mbar_init(&src_full[s], 1);
            mbar_init(&src_empty[s], 1);
            mbar_init(&done[s], 4);
        }
        mbar_init(&drain, 1);
        fence_async_smem();
    }
    if (warp == 9) {
        if constexpr (kPair == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                         ::"r"(smem_addr(&s_tmem)), "n"(2 * kAccCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                         ::"r"(smem_addr(&s_tmem)), "n"(2 * kAccCols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if constexpr (kPair == 2) {   // the other CTA's barriers are set up too
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_tmem;
    bool late = false;

    if (warp == 8) {
        if (lane == 0) {   // operands
            Dependencies<kPair> deps;
            int stage = 0, used = 0;
            uint32_t phase = 0;
            for (int ph = 0; ph < run.num_phases && !late; ++ph) {
                const Phase p = run.phases[ph];
                if (p.reduce) continue;
                const int units = T::units(run.m, run.batch, p);
                for (int u = (group + groups - p.first % groups) % groups; u < units && !late; u += groups) {
                    const UnitAt at = T::at(run.m, p, u);
                    if (!deps.wait(run, p, ph, at.b)) {
                        late = true;
                        break;
                    }
                    for (int kb = at.k0; kb < at.k1; ++kb) {
                        if (!mbar_wait(&empty[stage], phase ^ 1u)) {
                            late = true;
                            break;
                        }
                        unsigned char* a = stages + stage * kStageBytes;
                        unsigned char* b = a + kOperandBytes;
                        const uint32_t bar = kPair == 2 ? leader_addr(&full[stage]) : smem_addr(&full[stage]);
                        const int cols = p.tile_n / kPair;   // of B per CTA: 128 or 64
                        if (rank == 0) mbar_expect_tx(&full[stage], kPair * (kOperandBytes + cols * kTileK * 2));
                        const int row = at.i * T::kTile + rank * kBlock, col = at.j * p.tile_n + rank * cols;
                        tma_load<kPair>(a, &run.wide[p.a], kb * kTileK, row, at.b, bar);
                        if (p.b_along_n) {
                            tma_load<kPair>(b, &run.narrow[p.b], col, kb * kTileK, at.b, bar);
                            if (cols > 64)
                                tma_load<kPair>(b + kOperandBytes / 2, &run.narrow[p.b], col + 64, kb * kTileK, at.b,
                                                bar);
                        } else {
                            tma_load<kPair>(b, cols > 64 ? &run.wide[p.b] : &run.narrow[p.b], kb * kTileK, col, at.b,
                                            bar);
                        }
                        if (used < kStages) ++used;
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
            if (late) {
                // the copies still in flight must land before the CTA leaves; a pair's are all
                // counted in its first CTA, and the second waits for that one before it exits
                bool pending = false;
                for (int q = 0; q < used && rank == 0; ++q) {
                    const int s = (stage + kStages - 1 - q) % kStages;
                    pending |= !mbar_wait(&full[s], s < stage ? phase : phase ^ 1u);
                }
                if (run.flags != nullptr)
                    atomicOr(run.flags, kFlagTimeout | (pending ? kFlagCopyPending : 0u));
            }
        }
        __syncwarp();
    } else if (warp == 9) {
        if (lane == 0 && rank == 0) {   // products
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            for (int ph = 0; ph < run.num_phases && !late; ++ph) {
                const Phase p = run.phases[ph];
                if (p.reduce) continue;
                // fp32 accumulators, fp16 operands, B transposed where its rows run along N
                const uint32_t idesc = (1u << 4) | ((p.b_along_n ? 1u : 0u) << 16) |
                                       (static_cast<uint32_t>(p.tile_n / 8) << 17) |
                                       (static_cast<uint32_t>(T::kTile / 16) << 24);
                const uint32_t lead = p.b_along_n ? kOperandBytes / 2 : 16;
                const uint32_t b_step = p.b_along_n ? 128 : 2;   // 16 of K: 16 rows, or 32 bytes
                const int units = T::units(run.m, run.batch, p);
                for (int u = (group + groups - p.first % groups) % groups; u < units && !late; u += groups) {
                    const UnitAt at = T::at(run.m, p, u);
                    if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u)) {
                        late = true;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    for (int kb = at.k0; kb < at.k1; ++kb) {
                        if (!mbar_wait(&full[stage], phase)) {
                            late = true;
                            break;
                        }
                        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                        const unsigned char* a = stages + stage * kStageBytes;
                        const uint64_t da = operand_desc(a, 16), db = operand_desc(a + kOperandBytes, lead);
#pragma unroll
                        for (int k = 0; k < kTileK / 16; ++k)
                            mma_f16<kPair>(tmem + acc * kAccCols, da + k * 2, db + k * b_step, idesc,
                                           kb > at.k0 || k > 0);
                        mma_commit<kPair>(&empty[stage]);
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    if (late) break;
                    mma_commit<kPair>(&acc_full[acc]);
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                }
            }
            if (late) {
                mma_commit<kPair>(&drain);
                mbar_wait(&drain, 0);
                if (run.flags != nullptr) atomicOr(run.flags, kFlagTimeout);
            }
        }
        __syncwarp();
    } else if (warp == 10) {
        if (lane == 0) {   // sources
            Dependencies<kPair> deps;
            int buf = 0, used = 0;
            uint32_t phase = 0;
            for (int ph = 0; ph < run.num_phases && !late; ++ph) {
                const Phase p = run.phases[ph];
                const int units = T::units(run.m, run.batch, p);
                for (int u = (group + groups - p.first % groups) % groups; u < units && !late; u += groups) {
                    const UnitAt at = T::at(run.m, p, u);
                    const int row = at.i * T::kTile + rank * kBlock;
                    if (row >= run.m) continue;
                    if (!deps.wait(run, p, ph, at.b)) {
                        late = true;
                        break;
                    }
                    for (int s = at.slab0; s < at.slab1; ++s) {
                        const int col = at.j * p.tile_n + s * kSlab;
                        if (col >= p.n) break;
                        if (!mbar_wait(&src_empty[buf], phase ^ 1u)) {
                            late = true;
                            break;
                        }
                        unsigned char* slab = slabs + buf * kSlabBytes;
                        const uint32_t bar = smem_addr(&src_full[buf]);
                        const int planes = (p.src1 != kNone) + (p.src2 != kNone);
                        if (planes > 0) mbar_expect_tx(&src_full[buf], planes * kPlaneBytes);
                        else mbar_arrive(&src_full[buf]);
                        if (p.src1 != kNone) tma_load<1>(slab, &run.wide[p.src1], col, row, at.b, bar);
                        if (p.src2 != kNone) tma_load<1>(slab + kPlaneBytes, &run.wide[p.src2], col, row, at.b, bar);
                        if (used < kSlabs) ++used;
                        if (++buf == kSlabs) {
                            buf = 0;
                            phase ^= 1u;
                        }
                    }
                }
            }
            if (late) {
                bool pending = false;
                for (int q = 0; q < used; ++q) {
                    const int s = (buf + kSlabs - 1 - q) % kSlabs;
                    pending |= !mbar_wait(&src_full[s], s < buf ? phase : phase ^ 1u);
                }
                if (run.flags != nullptr)
                    atomicOr(run.flags, kFlagTimeout | (pending ? kFlagCopyPending : 0u));
            }
        }
        __syncwarp();
    } else if (warp == 11) {
        if (lane == 0) {   // stores
            int buf = 0, leaving = -1;   // the buffer whose stores may still read it
            uint32_t phase = 0;
            for (int ph = 0; ph < run.num_phases && !late; ++ph) {
                const Phase p = run.phases[ph];
                const int units = T::units(run.m, run.batch, p);
                for (int u = (group + groups - p.first % groups) % groups; u < units && !late; u += groups) {
                    const UnitAt at = T::at(run.m, p, u);
                    const int row0 = at.i * T::kTile + rank * kBlock;
                    for (int s = at.slab0; s < at.slab1 && row0 < run.m; ++s) {
                        const int col0 = at.j * p.tile_n + s * kSlab;
                        if (col0 >= p.n) break;
                        if (!mbar_wait(&done[buf], phase)) {
                            late = true;
                            break;
                        }
                        const unsigned char* slab = slabs + buf * kSlabBytes;
                        if (p.result != kPartial) {
                            const bool transposed = p.result == kBf16Transposed;
                            if (!transposed) tma_store(&run.wide[p.dst], slab, col0, row0, at.b);
                            if (p.result == kState)
                                tma_store(&run.wide[p.dst_lo], slab + kPlaneBytes, col0, row0, at.b);
                            if (transposed || (p.sym && !T::on_diagonal(p, at.i, at.j))) {
                                tma_store(&run.narrow[p.dst], slab + kPlaneBytes, row0, col0, at.b);
                                if (row0 + 64 < run.m)
                                    tma_store(&run.narrow[p.dst], slab + kPlaneBytes + kSlab * 128,
                                              row0 + 64, col0, at.b);
                            }
                        }
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        // the slab before this one has left its buffer
                        asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                        if (leaving >= 0) mbar_arrive(&src_empty[leaving]);
                        leaving = buf;
                        if (++buf == kSlabs) {
                            buf = 0;
                            phase ^= 1u;
                        }
                    }
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    if (leaving >= 0) mbar_arrive(&src_empty[leaving]);
                    leaving = -1;
                    // once the stores are complete their results are visible to this thread, and
                    // to others through its release
                    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                    if (late) break;
                    asm volatile("red.release.gpu.global.add.u32 [%0], 1;"
                                 ::"l"(run.arrived + ph * run.slots + at.b % run.slots) : "memory");
                }
            }
            if (late && run.flags != nullptr) atomicOr(run.flags, kFlagTimeout);
        }
        __syncwarp();
    } else {   // results
        Dependencies<kPair> deps;
        // warps 0-3 take the even slabs in the order of the CTA's work, 4-7 the odd ones
        const int set = warp >> 2, quarter = warp & 3, row_in = quarter * 32 + lane;
        int acc = 0, slab_count = 0;
        uint32_t acc_phase = 0, read_phase = 0;
        for (int ph = 0; ph < run.num_phases && !late; ++ph) {
            const Phase p = run.phases[ph];
            const int units = T::units(run.m, run.batch, p);
            for (int u = (group + groups - p.first % groups) % groups; u < units && !late; u += groups) {
                const UnitAt at = T::at(run.m, p, u);
                const int row0 = at.i * T::kTile + rank * kBlock;
                if (p.reduce) {
                    const bool ok = deps.wait(run, p, ph, at.b);
                    if (__any_sync(kAll, !ok)) {
                        late = true;
                        break;
                    }
                } else {
                    const bool ok = mbar_wait(&acc_full[acc], acc_phase);
                    if (__any_sync(kAll, !ok)) {
                        late = true;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                }
                for (int s = at.slab0; s < at.slab1 && row0 < run.m; ++s) {
                    const int col0 = at.j * p.tile_n + s * kSlab;
                    if (col0 >= p.n) break;
                    const int buf = slab_count % kSlabs;
                    const uint32_t phase = slab_count / kSlabs & 1;
                    if ((slab_count++ & 1) != set) continue;
                    float v[kSlab];
                    if (!p.reduce) {
                        const uint32_t from = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                                              acc * kAccCols + s * kSlab;
                        tmem_load_32(from, reinterpret_cast<uint32_t*>(v));
                        tmem_load_32(from + 32, reinterpret_cast<uint32_t*>(v) + 32);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    }
                    const bool ok = mbar_wait(&src_full[buf], phase);
                    if (__any_sync(kAll, !ok)) {
                        late = true;
                        break;
                    }
                    unsigned char* slab = slabs + buf * kSlabBytes;
                    // where this thread's row of a unit's partial accumulators starts
                    auto partial = [&](int unit) {
                        return reinterpret_cast<float4*>(run.partials) +
                               ((static_cast<int64_t>(unit) * kPair + rank) * (T::kTile / 4) +
                                s * (kSlab / 4)) * kBlock + row_in;
                    };
                    if (p.result == kPartial) {
                        float4* to = partial(u);
#pragma unroll
                        for (int c = 0; c < kSlab / 4; ++c)
                            to[c * kBlock] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
                        __threadfence();
                    } else {
                        if (p.reduce) {
#pragma unroll
                            for (int c = 0; c < kSlab; ++c) v[c] = 0.0f;
                            for (int q = 0; q < p.splits; ++q) {   // in the order of K
                                const float4* from = partial(at.tile * p.splits + q);
#pragma unroll
                                for (int c = 0; c < kSlab / 4; ++c) {
                                    const float4 x = __ldcg(from + c * kBlock);
                                    v[4 * c] = __fadd_rn(v[4 * c], x.x);
                                    v[4 * c + 1] = __fadd_rn(v[4 * c + 1], x.y);
                                    v[4 * c + 2] = __fadd_rn(v[4 * c + 2], x.z);
                                    v[4 * c + 3] = __fadd_rn(v[4 * c + 3], x.w);
                                }
                            }
                        }
                        const bool mirror = p.sym && !T::on_diagonal(p, at.i, at.j);
                        // the four warps of the set have read this slab's sources
                        auto all_read = [&] {
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&read[set]);
                            late |= !mbar_wait(&read[set], read_phase);
                            read_phase ^= 1u;
                        };
                        auto finish = [&](auto sources, auto result, auto mirrored) {
                            finish_row<decltype(sources)::value, decltype(result)::value, decltype(mirrored)::value>(
                                slab, row_in, v, p.f_acc, p.f1, p.f2, all_read);
                        };
                        using Yes = std::true_type;
                        using No = std::false_type;
                        const Count<0> none;
                        const Count<1> one;
                        const Count<2> two;
                        const Result<kPlane> plane;
                        if (p.result == kState) finish(two, Result<kState>(), No());
                        else if (p.result == kBf16) finish(two, Result<kBf16>(), No());
                        else if (p.result == kBf16Transposed) finish(two, Result<kBf16Transposed>(), No());
                        else if (p.src1 == kNone) mirror ? finish(none, plane, Yes()) : finish(none, plane, No());
                        else if (p.src2 == kNone) mirror ? finish(one, plane, Yes()) : finish(one, plane, No());
                        else mirror ? finish(two, plane, Yes()) : finish(two, plane, No());
                        late = __any_sync(kAll, late);
                        fence_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&done[buf]);
                }
                if (late) break;
                if (!p.reduce) {
                    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (kPair == 2) arrive_at(leader_addr(&acc_empty[acc]));
                        else mbar_arrive(&acc_empty[acc]);
                    }
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                }
            }
        }
        if (late && lane == 0 && run.flags != nullptr) atomicOr(run.flags, kFlagTimeout);
    }
    __syncthreads();
    if constexpr (kPair == 2) {   // no copy, arrival or product of the pair is left
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    if (warp == 9) {
        if constexpr (kPair == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(2 * kAccCols));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(2 * kAccCols));
    }
}

// ---- small matrices: the whole call in one cluster -------------------------------------------
// A matrix whose short side is at most 128 (256: a pair of CTAs, for a long side up to 256) never
// leaves its cluster: X lies as fp16 operands in shared memory and as fp32 state in tensor memory,
// each CTA with 256 of its columns.  One launch does the momentum step, the norm, every product and
// the output, with three barriers a step instead of trips through L2 and waits across the grid.
//   kPair = 1: 128 rows of X per CTA, the cluster's CTAs side by side along the long side.  Each
//     multiplies its own columns, the partial Gram matrices are added up (in CTA order) and handed
//     round through distributed shared memory, and each CTA then forms B and its columns of B X.
//   kPair = 2: each CTA has 128 of the 256 rows.  Products are the pair's (cta_group::2); a
//     symmetric matrix's rows serve as both operands, and for B X the CTAs exchange the halves of
//     X that the other one's columns need.
// X by rows serves the Gram product (rows along K) and, the same bytes read the other way, B X
// (rows along N).
constexpr int kSmallThreads = 256;
constexpr int kSmallCols = 256;                    // of X per CTA
constexpr int kSmallClusters = 16;
constexpr int kStagePitch = kSmallCols + 1;        // floats; odd, so rows and columns both read freely
constexpr int kBlockBytes = kBlock * kTileK * 2;   // 64 columns of an operand

template <int kPair>
struct SmallShape {
    static constexpr int kGramCols = kBlock * kPair;
    static constexpr int kXBytes = kSmallCols / 64 * kBlockBytes;
    static constexpr int kABytes = kGramCols / 64 * kBlockBytes;
    // partial sums (kPair = 1), or the columns' half of X in all rows (kPair = 2)
    static constexpr int kOtherBytes = kPair == 1 ? kBlock * kBlock * 4 : 2 * 2 * kBlockBytes;
    static constexpr int kUsed = kXBytes + kABytes + kOtherBytes;
    static constexpr int kStaging = kBlock * kStagePitch * 4;
    static constexpr int kSmem = (kUsed > kStaging ? kUsed : kStaging) + 1024;
};

struct SmallArgs {
    PrepArgs p;
    uint16_t* out;
    int m, n, width;    // short and long side; columns of X per CTA (kPair = 1: a multiple of 64)
    int steps;
    bool tall;
    float a, b, c;      // coefficients
    uint32_t* flags;
};

__device__ __forceinline__ void tmem_store_32(uint32_t addr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
          "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]),
          "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]),
          "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
          "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t remote_addr(const void* p, uint32_t cta) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(cta));
    return a;
}

template <int kPair, bool kBf16, bool kVec>
__global__ void __launch_bounds__(kSmallThreads, 1) k_orth_small(const __grid_constant__ SmallArgs s) {
    using S = SmallShape<kPair>;
    using U = PrepUnit<kBf16, kVec>;
    constexpr int kGramCols = S::kGramCols;
    constexpr int kPerThread = kSmallCols / 2;   // columns of X per thread: two warps share a row
    extern __shared__ unsigned char smem_raw[];
    unsigned char* x_op = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    unsigned char* a_op = x_op + S::kXBytes;
    unsigned char* other = a_op + S::kABytes;
    float* staging = reinterpret_cast<float*>(x_op);   // before the operands exist, and after
    __shared__ __align__(8) uint64_t bar;
    __shared__ uint32_t s_tmem;
    __shared__ double s_sum[kSmallThreads / 32 + 1];
    const PrepArgs& p = s.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t ctas, cta;   // of the cluster
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(cta));
    const int64_t b = blockIdx.x / ctas;
    const int row0 = kPair == 2 ? static_cast<int>(cta) * kBlock : 0;        // this CTA's rows of X
    const int col0 = kPair == 2 ? 0 : static_cast<int>(cta) * s.width;       // and columns
    const int rows = min(kBlock, s.m - row0), cols = min(s.width, s.n - col0);   // may be <= 0
    bool late = false;

    if (tid == 0) {
        mbar_init(&bar, 1);
        fence_async_smem();
    }
    if (warp == 0) {
        if constexpr (kPair == 2) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                         ::"r"(smem_addr(&s_tmem)), "n"(512) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                         ::"r"(smem_addr(&s_tmem)), "n"(512) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        }
    }

    // the update with its momentum step, as fp32 [row][column] in shared memory: a warp per stored
    // line, kLines of them at a time for the loads in flight
    const int lines = s.tall ? cols : rows, length = s.tall ? rows : cols;   // as stored
    const int64_t line0 = s.tall ? col0 : row0, at0 = s.tall ? row0 : col0;
    constexpr int kWarps = kSmallThreads / 32, kLines = 4;
    float sum = 0.0f;
    for (int l0 = warp; l0 < lines; l0 += kWarps * kLines) {
        for (int at = lane * U::kN; at < length; at += 32 * U::kN) {
            U g[kLines], mom[kLines];
#pragma unroll
            for (int k = 0; k < kLines; ++k) {
                const int64_t line = line0 + l0 + k * kWarps;
                if (l0 + k * kWarps >= lines || !SPL_CHECK(line < p.rows, kSiteOrthIn, line)) continue;
                g[k].load(p, b, line, (at0 + at) / U::kN);
                if (p.momentum != nullptr) mom[k].load_momentum(p.momentum + (b * p.rows + line) * p.cols + at0 + at);
            }
#pragma unroll
            for (int k = 0; k < kLines; ++k) {
                const int line = l0 + k * kWarps;
                if (line >= lines) continue;
#pragma unroll
                for (int e = 0; e < U::kN; ++e) {
                    if (p.momentum != nullptr) mom[k].x[e] = __fmaf_rn(p.mu, mom[k].x[e], g[k].x[e]);
                    const float u = step_value(g[k].x[e], mom[k].x[e], p);
                    sum = __fmaf_rn(u, u, sum);
                    staging[s.tall ? (at + e) * kStagePitch + line : line * kStagePitch + at + e] = u;
                }
                if (p.momentum != nullptr)
                    mom[k].store_momentum(p.momentum + (b * p.rows + line0 + line) * p.cols + at0 + at);
            }
        }
    }
    double norm2 = static_cast<double>(sum);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) norm2 += __shfl_xor_sync(kAll, norm2, off);
    if (lane == 0) s_sum[warp] = norm2;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kSmallThreads / 32; ++w) norm2 += s_sum[w];
        s_sum[kSmallThreads / 32] = norm2;
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    cluster_barrier();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    norm2 = 0.0;
    for (uint32_t q = 0; q < ctas; ++q) {
        double v;
        asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(remote_addr(&s_sum[kSmallThreads / 32], q)));
        norm2 += v;
    }
    const float norm = static_cast<float>(sqrt(norm2));
    float factor = __fdiv_rn(p.x_scale, __fadd_rn(norm, p.eps));
    if (!(norm <= 3.402823466e+38f)) {
        factor = nan_value();
        if (tid == 0 && cta == 0 && s.flags != nullptr) atomicOr(s.flags, kFlagNonFinite);
    }

    // a thread's row, and its half of the columns
    const int quarter = warp & 3, half = warp >> 2, row = quarter * 32 + lane;
    const uint32_t lanes = s_tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t state = lanes + kSmallCols;   // X in columns 256 .. 511, accumulators in 0 .. 255
    // 8 columns of the operand X from column c, and in a pair their copy with the columns' owner
    auto put_x = [&](int c, const uint4& w) {
        *reinterpret_cast<uint4*>(x_op + c / 64 * kBlockBytes + swizzled(row, c % 64 / 8)) = w;
        if constexpr (kPair == 2) {
            const uint32_t to = remote_addr(other, c / 128) + cta * (2 * kBlockBytes) + c % 128 / 64 * kBlockBytes +
                                swizzled(row, c % 64 / 8);
            asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};"
                         ::"r"(to), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
        }
    };
    // what threads of the cluster wrote to shared memory, before the products read it
    auto publish = [&] {
        fence_async_all();
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        if (ctas > 1) cluster_barrier();
        else __syncthreads();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        fence_async_all();
    };
    uint32_t bar_phase = 0;
    // one product: `issue` runs in the thread that issues it; then all wait for it
    auto product = [&](auto issue) {
        if (tid == 0 && (kPair == 1 || cta == 0)) {
            issue();
            mma_commit<kPair>(&bar);
        }
        __syncwarp();
        if (!late) late = !mbar_wait(&bar, bar_phase);
        bar_phase ^= 1u;
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    };

    {
        float x[kPerThread];
#pragma unroll
        for (int c = 0; c < kPerThread; ++c) {
            const int col = half * kPerThread + c;
            x[c] = row < rows && col < cols ? __fmul_rn(staging[row * kStagePitch + col], factor) : 0.0f;
        }
        if (ctas > 1) cluster_barrier();   // a pair writes to the other's memory below
        else __syncthreads();
#pragma unroll
        for (int c = 0; c < kPerThread; c += 8) put_x(half * kPerThread + c, pack_half8(x + c));
#pragma unroll
        for (int c = 0; c < kPerThread; c += 32)
            tmem_store_32(state + half * kPerThread + c, reinterpret_cast<const uint32_t*>(x) + c);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    }
    publish();

    const float gram_scale = kGramScale / (p.x_scale * p.x_scale);
    const int k_x = (kPair == 2 ? s.n : s.width), k_a = s.m;   // lengths of the products
    constexpr uint32_t kInstr = (1u << 4) | (static_cast<uint32_t>(kGramCols / 16) << 24);   // fp32 sums, M
    for (int step = 0; step < s.steps; ++step) {
        // A = X X^T (this CTA's columns)
        product([&] {
            constexpr uint32_t idesc = kInstr | (static_cast<uint32_t>(kGramCols / 8) << 17);
            for (int k = 0; k < k_x; k += 16) {
                const uint64_t d = operand_desc(x_op + k / 64 * kBlockBytes, 16) + k % 64 / 16 * 2;
                mma_f16<kPair>(s_tmem, d, d, idesc, k > 0);
            }
        });
        {
            float v[kGramCols / 2];
#pragma unroll
            for (int c = 0; c < kGramCols / 2; c += 32)
                tmem_load_32(lanes + half * (kGramCols / 2) + c, reinterpret_cast<uint32_t*>(v) + c);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
            if (kPair == 2 || ctas == 1) {
#pragma unroll
                for (int c = 0; c < kGramCols / 2; c += 8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[c + i] = __fmul_rn(v[c + i], gram_scale);
                    const int col = half * (kGramCols / 2) + c;
                    *reinterpret_cast<uint4*>(a_op + col / 64 * kBlockBytes + swizzled(row, col % 64 / 8)) = pack_half8(v + c);
                }
            } else {   // partial sums: chunk c of row r at place c ^ (r & 31)
                float4* mine = reinterpret_cast<float4*>(other) + row * 32;
#pragma unroll
                for (int c = 0; c < kGramCols / 2; c += 4)
                    mine[((half * (kGramCols / 2) + c) / 4) ^ (row & 31)] = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
                cluster_barrier();
                // this CTA adds up its share of the rows and gives the result to all
                const int r0 = kBlock * static_cast<int>(cta) / static_cast<int>(ctas),
                          r1 = kBlock * (static_cast<int>(cta) + 1) / static_cast<int>(ctas);
                // kItems places at once from each of at most kMost CTAs: 16 loads in flight
                auto add_up = [&](auto items, auto most) {
                    constexpr int kItems = decltype(items)::value, kMost = decltype(most)::value;
                    const int total = (r1 - r0) * 32;
                    for (int i0 = tid; i0 < total; i0 += kSmallThreads * kItems) {
                        float4 q[kItems][kMost];
#pragma unroll
                        for (int j = 0; j < kItems; ++j) {
                            const int i = i0 + j * kSmallThreads, r = r0 + i / 32, c = i % 32;
                            if (i >= total) continue;
                            const float4* from = reinterpret_cast<const float4*>(other) + r * 32 + (c ^ (r & 31));
#pragma unroll
                            for (int k = 0; k < kMost; ++k)
                                if (k < static_cast<int>(ctas))
                                    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                                                 : "=f"(q[j][k].x), "=f"(q[j][k].y), "=f"(q[j][k].z), "=f"(q[j][k].w)
                                                 : "r"(remote_addr(from, k)));
                        }
#pragma unroll
                        for (int j = 0; j < kItems; ++j) {
                            const int i = i0 + j * kSmallThreads, r = r0 + i / 32, c = i % 32;
                            if (i >= total) continue;
                            float4 t = q[j][0];
#pragma unroll
                            for (int k = 1; k < kMost; ++k) {
                                if (k >= static_cast<int>(ctas)) continue;
                                t.x = __fadd_rn(t.x, q[j][k].x), t.y = __fadd_rn(t.y, q[j][k].y);
                                t.z = __fadd_rn(t.z, q[j][k].z), t.w = __fadd_rn(t.w, q[j][k].w);
                            }
                            const __half2 h0 = __floats2half2_rn(__fmul_rn(t.x, gram_scale), __fmul_rn(t.y, gram_scale));
                            const __half2 h1 = __floats2half2_rn(__fmul_rn(t.z, gram_scale), __fmul_rn(t.w, gram_scale));
                            const unsigned char* to =
                                a_op + c / 16 * kBlockBytes + swizzled(r, c % 16 / 2) + c % 2 * 8;
                            for (uint32_t k = 0; k < ctas; ++k)
                                asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};"
                                             ::"r"(remote_addr(to, k)), "r"(*reinterpret_cast<const uint32_t*>(&h0)),
                                               "r"(*reinterpret_cast<const uint32_t*>(&h1)) : "memory");
                        }
                    }
                };
                if (ctas <= 4) add_up(Count<4>(), Count<4>());
                else add_up(Count<1>(), Count<kSmallClusters>());
            }
        }
        publish();
        // B = b A + c A A, in A's place (the product has read A)
        product([&] {
            constexpr uint32_t idesc = kInstr | (static_cast<uint32_t>(kGramCols / 8) << 17);
            for (int k = 0; k < k_a; k += 16) {
                const uint64_t d = operand_desc(a_op + k / 64 * kBlockBytes, 16) + k % 64 / 16 * 2;
                mma_f16<kPair>(s_tmem, d, d, idesc, k > 0);
            }
        });
        {
            float v[kGramCols / 2];
#pragma unroll
            for (int c = 0; c < kGramCols / 2; c += 32)
                tmem_load_32(lanes + half * (kGramCols / 2) + c, reinterpret_cast<uint32_t*>(v) + c);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
            const float f = __fmul_rn(s.c, 1.0f / kGramScale);
            uint4 old[kGramCols / 16];
#pragma unroll
            for (int c = 0; c < kGramCols / 2; c += 8) {
                const int col = half * (kGramCols / 2) + c;
                old[c / 8] = *reinterpret_cast<const uint4*>(a_op + col / 64 * kBlockBytes + swizzled(row, col % 64 / 8));
            }
#pragma unroll
            for (int c = 0; c < kGramCols / 2; c += 8) {
                float y[8];
                unpack_half8(old[c / 8], y);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[c + i] = __fmaf_rn(s.b, y[i], __fmul_rn(f, v[c + i]));
                const int col = half * (kGramCols / 2) + c;
                *reinterpret_cast<uint4*>(a_op + col / 64 * kBlockBytes + swizzled(row, col % 64 / 8)) = pack_half8(v + c);
            }
        }
        publish();
        // X = a X + B X
        product([&] {
            const uint32_t n = kPair == 2 ? 256 : s.width;
            const uint32_t idesc = kInstr | (1u << 16) | (n / 8 << 17);
            for (int k = 0; k < k_a; k += 16) {
                const uint64_t d = operand_desc(a_op + k / 64 * kBlockBytes, 16) + k % 64 / 16 * 2;
                const unsigned char* x = kPair == 2 ? other + k / 128 * (2 * kBlockBytes) : x_op;
                const uint64_t e = operand_desc(x + k % 128 * 128, kBlockBytes);
                mma_f16<kPair>(s_tmem, d, e, idesc, k > 0);
            }
        });
        const bool last = step + 1 == s.steps;
        if (last) {   // no product reads shared memory any more: the result goes where it began
            if (ctas > 1) cluster_barrier();
            else __syncthreads();
        }
#pragma unroll 1
        for (int c0 = 0; c0 < kPerThread; c0 += 32) {
            const int col = half * kPerThread + c0;
            if (kPair == 1 && col >= s.width) break;
            float v[32], x[32];
            tmem_load_32(lanes + col, reinterpret_cast<uint32_t*>(v));
            tmem_load_32(state + col, reinterpret_cast<uint32_t*>(x));
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __fmaf_rn(s.a, x[i], __fmul_rn(v[i], 1.0f / kGramScale));
            if (last) {
                const float f = __fdiv_rn(1.0f, p.x_scale);
#pragma unroll
                for (int i = 0; i < 32; ++i) staging[row * kStagePitch + col + i] = __fmul_rn(x[i], f);
            } else {
                tmem_store_32(state + col, reinterpret_cast<const uint32_t*>(x));
#pragma unroll
                for (int i = 0; i < 32; i += 8) put_x(col + i, pack_half8(x + i));
            }
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        if (!last) publish();
    }
    __syncthreads();
    const int across = s.tall ? kStagePitch : 1, down = s.tall ? 1 : kStagePitch;   // along and between lines
    for (int line = warp; line < lines; line += kWarps) {
        uint16_t* out = s.out + (b * p.rows + line0 + line) * p.cols + at0;
        const float* from = staging + line * down;
        if ((p.cols & 1) == 0) {   // pairs of values stay on 4 bytes
            for (int at = 2 * lane; at < length; at += 64) {
                if (!SPL_CHECK(at < length, kSiteOrthOut, at)) continue;
                const float lo = from[at * across], hi = from[(at + 1) * across];
                uint32_t w;
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
                *reinterpret_cast<uint32_t*>(out + at) = w;
            }
        } else {
            for (int at = lane; at < length; at += 32)
                if (SPL_CHECK(at < length, kSiteOrthOut, at)) Vec16<true>::store1(out, at, from[at * across]);
        }
    }
    if (late && tid == 0 && s.flags != nullptr) atomicOr(s.flags, kFlagTimeout);
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    if (ctas > 1) cluster_barrier();
    else __syncthreads();
    if (warp == 0) {
        if constexpr (kPair == 2)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "n"(512));
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "n"(512));
    }
}

// Whether a matrix takes the small kernel.
bool is_small(int64_t m, int64_t n) {
    return (m <= kBlock && n <= kSmallCols * kSmallClusters) || (m <= 2 * kBlock && n <= kSmallCols);
}

template <int kPair, bool kBf16, bool kVec>
cudaError_t launch_small(const SmallArgs& s, int64_t batch, cudaStream_t stream) {
    const void* kern = reinterpret_cast<const void*>(&k_orth_small<kPair, kBf16, kVec>);
    const int ctas = kPair == 2 ? 2 : (s.n + s.width - 1) / s.width;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SmallShape<kPair>::kSmem);
    if (e == cudaSuccess && ctas > 8)   // beyond the portable cluster size
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(batch * ctas));
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = SmallShape<kPair>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_orth_small<kPair, kBf16, kVec>, s);
}

// The state's planes to bf16, transposed back where the matrix is tall: for outputs whose rows
// are no whole 16 bytes, which a TMA store cannot address.
__global__ void __launch_bounds__(256)
k_orth_finish(const __half* __restrict__ hi, const __half* __restrict__ lo, int64_t ld, int64_t plane,
              int64_t m, int64_t n, float f, uint16_t* __restrict__ out, bool tall) {
    __shared__ float s_tile[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t b = blockIdx.z, r0 = static_cast<int64_t>(blockIdx.y) * 32,
                  c0 = static_cast<int64_t>(blockIdx.x) * 32;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + warp + 8 * i, c = c0 + lane;
        if (r >= m || c >= n || !SPL_CHECK(c < ld, kSiteOrthState, c)) continue;
        const int64_t at = b * plane + r * ld + c;
        const float x = __fmul_rn(f, __fmaf_rn(__half2float(lo[at]), 1.0f / kLoScale, __half2float(hi[at])));
        if (tall) s_tile[warp + 8 * i][lane] = x;
        else Vec16<true>::store1(out, (b * m + r) * n + c, x);
    }
    if (!tall) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + lane, c = c0 + warp + 8 * i;
        if (r < m && c < n && SPL_CHECK(c < n, kSiteOrthOut, c))
            Vec16<true>::store1(out, (b * n + c) * m + r, s_tile[lane][warp + 8 * i]);
    }
}

// ---- host -----------------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

constexpr int kSquares = 5;      // m x m matrices: A, and the polynomials of a group of steps
constexpr int kSplitUnits = 320; // partial 128 x 128 accumulators a split product may leave
constexpr int kMaxSplits = 16;   // parts of a long K
constexpr int kSplitBlocks = 4;  // of at least 4 blocks each

// Whether a group of steps pays for a matrix of these sides (see group_steps).
bool may_group(int64_t m, int64_t n) { return 4 * n >= 5 * m && m >= 256; }

struct OrthLayout {
    int64_t m, n, ldx, ldm;   // short and long side, row pitches of X and of the square matrices
    size_t hi[2], lo[2], square[kSquares], arrived, partials, norms, bytes;
    size_t partial_bytes;
};

OrthLayout orth_layout(int64_t batch, int64_t rows, int64_t cols) {
    OrthLayout l;
    l.m = rows <= cols ? rows : cols;
    l.n = rows <= cols ? cols : rows;
    l.ldx = (l.n + 7) / 8 * 8;   // TMA wants row pitches of whole 16 bytes
    l.ldm = (l.m + 7) / 8 * 8;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round256(bytes);
        return here;
    };
    const size_t plane = static_cast<size_t>(batch * l.m * l.ldx) * 2;
    for (int i = 0; i < 2; ++i) {
        l.hi[i] = take(plane);
        l.lo[i] = take(plane);
    }
    const int squares = may_group(l.m, l.n) ? kSquares : 2;
    for (int i = 0; i < kSquares; ++i)
        l.square[i] = i < squares ? take(static_cast<size_t>(batch * l.m * l.ldm) * 2) : 0;
    l.arrived = take(kMaxPhases * kMaxSlots * 4);
    // partial accumulators of a split product: enough units for a few per SM, where its tiles
    // alone are fewer than that
    const int64_t blocks = (l.n + kTileK - 1) / kTileK, tm = (l.m + kBlock - 1) / kBlock;
    const int64_t tiles = tm * (tm + 1) / 2 * batch;
    const int64_t splits = blocks / kSplitBlocks < kMaxSplits ? blocks / kSplitBlocks : kMaxSplits;
    l.partial_bytes = 0;
    if (tiles < kSplitUnits && splits > 1)
        l.partial_bytes = static_cast<size_t>(tiles * splits < kSplitUnits ? tiles * splits : kSplitUnits) *
                          kBlock * kBlock * 4;
    l.partials = take(l.partial_bytes);
    l.norms = take(static_cast<size_t>(batch) * kMaxPartials * sizeof(double));
    l.bytes = at;
    return l;
}

// What a launch of the run kernel depends on beside its arguments, found once per device.
struct RunLimits {
    int single, pairs;   // CTAs, and pairs of CTAs, resident at once
};

template <int kPair>
cudaError_t prepare_run(int sms, int* groups) {
    const void* kern = reinterpret_cast<const void*>(&k_orth_run<kPair>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRunSmem);
    if (e != cudaSuccess) return e;
    if (kPair == 1) {
        *groups = sms;
        return cudaSuccess;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sms / 2 * 2));
    cfg.blockDim = dim3(kRunThreads);
    cfg.dynamicSmemBytes = kRunSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(groups, kern, &cfg);
}

cudaError_t run_limits(RunLimits* out) {
    static std::mutex mu;
    static RunLimits cached[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (cached[dev].single == 0) {
        int sms = 0;
        RunLimits l = {};
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = prepare_run<1>(sms, &l.single);
        if (e == cudaSuccess) e = prepare_run<2>(sms, &l.pairs);
        if (e != cudaSuccess) return e;
        cached[dev] = l;
    }
    *out = cached[dev];
    return cudaSuccess;
}

// How many of the first steps may be taken as one polynomial of A, applied to X once.  Per step X
// costs 3 m^2 n multiplications (the symmetric product counts half) and A m^3; a group of g costs
// 3 m^2 n + (4 g - 3) m^3, less as soon as n > m.  The iteration's last steps undo the roundings
// of its first ones, so only those are grouped, and at least two steps stay single: 64-bit
// simulations with these roundings give errors of 1.0e-3 to 1.8e-3 for steps one by one, the same
// for a group of 2, and for a group of 3 the same once m >= 1024 (at most 1.4e-3) but up to 2.1e-3
// at m = 512 and 5e-3 at 64; two groups of 2 would give up to 2.8e-3 at m = 512.
// The 28672 x 8192 matrix: 22.0 ms one by one.
int group_steps(int64_t m, int64_t n, int steps, float a) {
    if (!may_group(m, n)) return 1;
    int size = m >= 1024 ? 3 : 2;
    if (steps - 2 < size) size = steps - 2;
    // R is as large as the identity's factor a^size, and must fit fp16 times its scale
    while (size > 1 && std::pow(std::fabs(a), size) > 48.0f) --size;
    return size > 1 ? size : 1;
}

struct PhaseList {
    Phase phases[kMaxPhases];
    int num;

    int16_t last() const { return static_cast<int16_t>(num - 1); }
    void add(Phase ph) {
        ph.splits = 1;
        ph.after[0] = last();
        ph.after[1] = -1;
        phases[num++] = ph;
    }
    void after(int16_t first, int16_t second = -1) {
        phases[num - 1].after[0] = first;
        phases[num - 1].after[1] = second;
    }
    // A symmetric m x m product.
    void square(uint8_t a, uint8_t b, uint8_t src1, uint8_t src2, uint8_t dst, int m, int k, float f_acc,
                float f1, float f2) {
        Phase ph = {};
        ph.a = a;
        ph.b = b;
        ph.src1 = src1;
        ph.src2 = src2;
        ph.dst = dst;
        ph.dst_lo = kNone;
        ph.result = kPlane;
        ph.sym = true;
        ph.n = m;
        ph.k = k;
        ph.f_acc = f_acc;
        ph.f1 = f1;
        ph.f2 = f2;
        add(ph);
    }
};

// Estimated microseconds of a list of products on `groups` CTAs (or pairs), and with `out` the
// phases to run.  A pair's tiles have 256 or 128 columns, whichever the model prefers; a symmetric
// product with fewer tiles than groups and a long K is split along K where that pays, followed by
// a phase that sums the parts.  Measured: a block of 64 along K takes 0.28 us for a 128 x 128 tile
// alone on its SM (its 32 KB arrive from L2 no faster) and 0.44 us with all SMs at it (L2's own
// limit), 0.32 us for a pair's 256 x 256 tile and 0.2 us for 256 x 128; an epilogue 1 us and 0.8 us
// for each slab of 64 columns, two slabs at a time; and 5 us from a phase's last result to the
// next one's first product.  A stack's phases flow into one another, so that they take either the
// time of their work or one matrix's way through them.
template <int kPair>
double plan(const PhaseList& list, const OrthRun& run, int groups, size_t partial_bytes, OrthRun* out) {
    using T = Tiling<kPair>;
    const int slots = run.batch < kMaxSlots ? run.batch : kMaxSlots;
    constexpr double kBetween = 5.0;
    const size_t unit_bytes = static_cast<size_t>(T::kTile) * T::kTile * 4;
    double total = 0.0;
    int index[kMaxPhases], num = 0, taken = 0;   // where each listed phase ends up
    bool split = false, any_split = false;
    for (int i = 0; i < list.num; ++i) {
        Phase ph = list.phases[i];
        const int blocks = (ph.k + kTileK - 1) / kTileK;
        auto time = [&](int tile_n, int splits) {
            Phase q = ph;
            q.tile_n = tile_n;
            const int tiles = T::tiles(run.m, q) * run.batch, units = tiles * splits;
            const double full = units < groups ? static_cast<double>(units) / groups : 1.0;
            const double block = kPair == 1 ? 0.28 + 0.16 * full : tile_n == 256 ? 0.32 : 0.2;
            const double one = block * ((blocks + splits - 1) / splits), epilogue = 0.4 * (tile_n / kSlab);
            const double work = one > epilogue ? one : epilogue;
            const double through = one + 1.0 + epilogue + kBetween;   // one unit, alone
            double t = (units + groups - 1) / groups * work - work + through;
            if (slots > 1) {
                const double flow = static_cast<double>(units) / groups * work;
                t = flow > through ? flow : through;
            }
            if (splits > 1)
                t += (tiles * T::slabs(q) + groups - 1) / groups * (1.0 + 0.25 * splits) + kBetween;
            return t;
        };
        int best = 1;
        ph.tile_n = kPair == 2 && time(128, 1) < time(T::kTile, 1) ? 128 : T::kTile;
        if (ph.sym && T::tiles(run.m, ph) * run.batch < groups)
            for (int tile_n = T::kTile; tile_n >= 128; tile_n /= 2)
                for (int q = 2; q <= kMaxSplits && q <= blocks / kSplitBlocks; ++q) {
                    Phase half = ph;
                    half.tile_n = tile_n;
                    const size_t units = static_cast<size_t>(T::tiles(run.m, half)) * run.batch * q;
                    if (units * unit_bytes <= partial_bytes && num + 3 < kMaxPhases &&
                        time(tile_n, q) < time(ph.tile_n, best)) {
                        best = q;
                        ph.tile_n = tile_n;
                    }
                }
        total += time(ph.tile_n, best);
        const int tiles = T::tiles(run.m, ph) * run.batch;
        // the parts of two products beside each other would share the partials' memory
        if (i > 0 && (best > 1 || split)) ph.after[0] = static_cast<int16_t>(i - 1), ph.after[1] = -1;
        split = best > 1;
        any_split |= split;
        const bool beside = ph.after[0] >= 0 && ph.after[0] != i - 1;
        for (int q = 0; q < 2; ++q)
            ph.after[q] = static_cast<int16_t>(ph.after[q] < 0 ? -1 : index[ph.after[q]]);
        // work goes on where the phase before it left off, if the two overlap
        ph.first = static_cast<int16_t>(beside || slots > 1 ? taken % groups : 0);
        Phase sum = ph;
        if (best > 1) {
            ph.splits = static_cast<uint8_t>(best);
            ph.result = kPartial;
            ph.src1 = ph.src2 = kNone;
        }
        taken = ph.first + tiles * best;
        if (out != nullptr) out->phases[num] = ph;
        index[i] = num++;
        if (best > 1) {
            sum.reduce = true;
            sum.splits = static_cast<uint8_t>(best);
            sum.after[0] = static_cast<int16_t>(num - 1);
            sum.after[1] = -1;
            sum.first = 0;
            taken = tiles * T::slabs(sum);
            if (out != nullptr) out->phases[num] = sum;
            index[i] = num++;
        }
    }
    if (out != nullptr) {
        out->num_phases = num;
        // partials of one matrix may lie where another's lay in an earlier phase
        out->slots = any_split ? 1 : slots;
    }
    return total;
}

template <int kPair>
cudaError_t launch_run(const OrthRun& run, int groups, cudaStream_t stream) {
    using T = Tiling<kPair>;
    int most = 1;
    for (int i = 0; i < run.num_phases; ++i) {
        const int u = T::units(run.m, run.batch, run.phases[i]);
        if (u > most) most = u;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((most < groups ? most : groups) * kPair));
    cfg.blockDim = dim3(kRunThreads);
    cfg.dynamicSmemBytes = kRunSmem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = kPair;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_orth_run<kPair>, run);
}

}  // namespace

#if SPL_CHECKED
SPL_DEBUG_READER(debug_read_orthogonalize)
#endif

size_t orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols) {
    return orth_layout(batch, rows, cols).bytes;
}

cudaError_t launch_orthogonalize(const OrthogonalizeArgs& a, bool bf16, cudaStream_t stream) {
    const OrthLayout l = orth_layout(a.batch, a.rows, a.cols);
    unsigned char* ws = static_cast<unsigned char*>(a.workspace);
    const bool tall = a.rows > a.cols;
    RunLimits limits;
    cudaError_t e = run_limits(&limits);
    if (e != cudaSuccess) return e;
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return cudaErrorNotSupported;

    PrepArgs p = {};
    p.update = a.update;
    p.rows = a.rows;
    p.cols = a.cols;
    p.row_stride = a.row_stride;
    p.batch_stride = a.batch_stride;
    p.momentum = a.momentum;
    p.mu = a.mu;
    p.nesterov = a.nesterov;
    p.eps = a.eps;
    p.x_scale = std::ldexp(1.0f, static_cast<int>(std::lround(0.5 * std::log2(static_cast<double>(l.n)))));
    p.partials = reinterpret_cast<double*>(ws + l.norms);
    p.hi = reinterpret_cast<__half*>(ws + l.hi[0]);
    p.lo = reinterpret_cast<__half*>(ws + l.lo[0]);
    p.ld = l.ldx;
    p.plane = l.m * l.ldx;
    p.arrived = reinterpret_cast<uint32_t*>(ws + l.arrived);
    p.flags = a.flags;
    const int size = bf16 ? 2 : 4, lanes = 16 / size;
    const bool vec = reinterpret_cast<uintptr_t>(a.update) % 16 == 0 && a.cols % lanes == 0 &&
                     a.row_stride % lanes == 0 && (a.batch == 1 || a.batch_stride % lanes == 0) &&
                     reinterpret_cast<uintptr_t>(a.momentum) % 16 == 0;
    if (is_small(l.m, l.n)) {
        SmallArgs small = {};
        small.p = p;
        small.out = a.out;
        small.m = static_cast<int>(l.m);
        small.n = static_cast<int>(l.n);
        const int ctas = (small.n + kSmallCols - 1) / kSmallCols;
        small.width = l.m > kBlock ? kSmallCols : ((small.n + ctas - 1) / ctas + 63) / 64 * 64;
        small.steps = a.steps;
        small.tall = tall;
        small.a = a.coef[0];
        small.b = a.coef[1];
        small.c = a.coef[2];
        small.flags = a.flags;
        // a CTA's columns start at a multiple of 64, so its vectors are whole where the matrix's are
        if (l.m > kBlock) {
            if (bf16) return vec ? launch_small<2, true, true>(small, a.batch, stream)
                                 : launch_small<2, true, false>(small, a.batch, stream);
            return vec ? launch_small<2, false, true>(small, a.batch, stream)
                       : launch_small<2, false, false>(small, a.batch, stream);
        }
        if (bf16) return vec ? launch_small<1, true, true>(small, a.batch, stream)
                             : launch_small<1, true, false>(small, a.batch, stream);
        return vec ? launch_small<1, false, true>(small, a.batch, stream)
                   : launch_small<1, false, false>(small, a.batch, stream);
    }
    if (bf16) e = vec ? launch_prep<true, true>(p, a.batch, tall, limits.single, stream)
                      : launch_prep<true, false>(p, a.batch, tall, limits.single, stream);
    else e = vec ? launch_prep<false, true>(p, a.batch, tall, limits.single, stream)
                 : launch_prep<false, false>(p, a.batch, tall, limits.single, stream);
    if (e != cudaSuccess) return e;

    static thread_local OrthRun run;   // large for a stack frame; filled anew each call
    bool mapped = true;
    // Tensor maps of matrix `id`: 16-bit values [batch][rows][cols], row pitch ld.
    auto matrix = [&](int id, void* base, CUtensorMapDataType type, int64_t rows, int64_t cols, int64_t ld) {
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                    static_cast<cuuint64_t>(a.batch)};
        const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * 2), static_cast<cuuint64_t>(rows * ld * 2)};
        const cuuint32_t step[3] = {1, 1, 1};
        for (int i = 0; i < 2; ++i) {
            const cuuint32_t box[3] = {64, i == 0 ? 128u : 64u, 1};
            mapped &= encode(i == 0 ? &run.wide[id] : &run.narrow[id], type, 3, base, dims, strides, box, step,
                             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
        }
    };
    enum : uint8_t { kHi0, kHi1, kLo0, kLo1, kOut, kSquare0 };
    const auto f16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    for (int i = 0; i < 2; ++i) {
        matrix(kHi0 + i, ws + l.hi[i], f16, l.m, l.n, l.ldx);
        matrix(kLo0 + i, ws + l.lo[i], f16, l.m, l.n, l.ldx);
    }
    const int grouped = group_steps(l.m, l.n, a.steps, a.coef[0]);
    for (int i = 0; i < (grouped > 1 ? kSquares : 2); ++i)
        matrix(kSquare0 + i, ws + l.square[i], f16, l.m, l.m, l.ldm);
    const bool direct = a.cols % 8 == 0;   // the output's rows are whole 16 bytes
    if (direct) matrix(kOut, a.out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.rows, a.cols, a.cols);
    if (!mapped) return cudaErrorInvalidValue;

    run.m = static_cast<int>(l.m);
    run.batch = static_cast<int>(a.batch);
    run.partials = reinterpret_cast<float*>(ws + l.partials);
    run.arrived = p.arrived;
    run.flags = a.flags;

    // The list of products.  With f the identity's factor, X <- f X + R X where R is the rest of
    // the polynomial of one step (R = B, f = a) or of a group of them.
    const int m = run.m, n = static_cast<int>(l.n);
    const float ca = a.coef[0];
    auto build = [&](PhaseList& list, int grouped) {
        list.num = 0;
        uint8_t free_squares[kSquares];
        int num_free = 0;
        for (int i = (grouped > 1 ? kSquares : 2) - 1; i > 0; --i) free_squares[num_free++] = static_cast<uint8_t>(kSquare0 + i);
        auto take = [&] { return free_squares[--num_free]; };
        auto give = [&](uint8_t id) { free_squares[num_free++] = id; };
        const uint8_t A = kSquare0;
        int x = 0;
        for (int s = 0; s < a.steps; x ^= 1) {
            const int size = s == 0 ? grouped : 1;
            const uint8_t hi = static_cast<uint8_t>(kHi0 + x), lo = static_cast<uint8_t>(kLo0 + x);
            // A = X X^T
            list.square(hi, hi, kNone, kNone, A, m, n, kGramScale / (p.x_scale * p.x_scale), 0.0f, 0.0f);
            uint8_t R = kNone;
            float f = ca;
            for (int i = 0; i < size; ++i) {
                const bool more = i + 1 < size;
                const uint8_t B = take();   // B = b A + c A A
                list.square(A, A, A, kNone, B, m, m, a.coef[2] / kGramScale, a.coef[1], 0.0f);
                const int16_t poly = list.last();
                uint8_t next = B;
                int16_t rest = poly;
                if (R != kNone) {           // (a I + B) (f I + R) - a f I = a R + f B + B R
                    next = take();
                    list.square(B, R, R, B, next, m, m, 1.0f / kGramScale, ca, f);
                    f *= ca;
                    rest = list.last();
                }
                if (more) {                 // A <- (a I + B) A (a I + B); beside the product above
                    const uint8_t T = take();
                    list.square(B, A, A, kNone, T, m, m, 1.0f / kGramScale, ca, 0.0f);
                    list.after(poly);
                    list.square(T, B, T, kNone, A, m, m, 1.0f / kGramScale, ca, 0.0f);
                    list.after(static_cast<int16_t>(list.last() - 1), rest);
                    give(T);
                }
                if (R != kNone) {
                    give(R);
                    give(B);
                }
                R = next;
            }
            s += size;
            // X = f X + R X
            Phase ph = {};
            const bool last = s == a.steps && direct;
            const float out = last ? 1.0f / p.x_scale : 1.0f;
            ph.a = R;
            ph.b = ph.src1 = hi;
            ph.src2 = lo;
            ph.dst = last ? static_cast<uint8_t>(kOut) : static_cast<uint8_t>(kHi0 + (x ^ 1));
            ph.dst_lo = last ? kNone : static_cast<uint8_t>(kLo0 + (x ^ 1));
            ph.result = !last ? kState : tall ? kBf16Transposed : kBf16;
            ph.b_along_n = true;
            ph.n = n;
            ph.k = m;
            ph.f_acc = out / kGramScale;
            ph.f1 = out * f;
            ph.f2 = ph.f1 / kLoScale;
            list.add(ph);
            give(R);
        }
        return x;   // which of the state's two places holds the result
    };

    // The grouping and the tiles that the time model prefers
    static thread_local PhaseList lists[2];
    int best_list = 0, best_pair = 1, x = 0;
    double best = 0.0;
    for (int i = 0; i < (grouped > 1 ? 2 : 1); ++i) {
        const int end = build(lists[i], i == 0 ? 1 : grouped);
        const double t1 = plan<1>(lists[i], run, limits.single, l.partial_bytes, nullptr);
        const double t2 = plan<2>(lists[i], run, limits.pairs, l.partial_bytes, nullptr);
        const double t = t2 < t1 ? t2 : t1;
        if (i > 0 && t >= best) continue;
        best = t;
        best_list = i;
        best_pair = t2 < t1 ? 2 : 1;
        x = end;
    }
    if (best_pair == 2) {
        plan<2>(lists[best_list], run, limits.pairs, l.partial_bytes, &run);
        e = launch_run<2>(run, limits.pairs, stream);
    } else {
        plan<1>(lists[best_list], run, limits.single, l.partial_bytes, &run);
        e = launch_run<1>(run, limits.single, stream);
    }
    if (e != cudaSuccess || direct) return e;
    const dim3 grid(static_cast<unsigned>((l.n + 31) / 32), static_cast<unsigned>((l.m + 31) / 32),
                    static_cast<unsigned>(a.batch));
    k_orth_finish<<<grid, 256, 0, stream>>>(reinterpret_cast<const __half*>(ws + l.hi[x]),
                                            reinterpret_cast<const __half*>(ws + l.lo[x]), l.ldx,
                                            l.m * l.ldx, l.m, l.n, 1.0f / p.x_scale, a.out, tall);
    return cudaGetLastError();
}

}  // namespace spl
