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

#include "local_device.cuh"
#include "local_kernels.h"

namespace spl {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kGramScale = 1024.0f;    // of A and B
constexpr float kLoScale = 2048.0f;      // of the state's low plane

// ---- momentum, norm, state ------------------------------------------------------------------
constexpr int kPrepThreads = 256;
constexpr int kMaxPartials = 512;   // sums of squares per matrix

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
    uint32_t* flags;
};

// u of one entry once the momentum holds its new value.
__device__ __forceinline__ float step_value(float g, float m, const PrepArgs& p) {
    if (p.momentum == nullptr) return g;
    return p.nesterov ? __fmaf_rn(p.mu, m, g) : m;
}

// The momentum step and each CTA's share of |u|^2.
template <bool kBf16>
__global__ void __launch_bounds__(kPrepThreads) k_orth_norm(const __grid_constant__ PrepArgs p) {
    using V = Vec16<kBf16>;
    __shared__ double s_sum[kPrepThreads / 32];
    const int64_t b = blockIdx.y;
    double total = 0.0;
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const unsigned char* row = static_cast<const unsigned char*>(p.update) +
                                   (b * p.batch_stride + r * p.row_stride) * V::kBytes;
        float* mom = p.momentum == nullptr ? nullptr : p.momentum + (b * p.rows + r) * p.cols;
        float sum = 0.0f;
        for (int64_t c = threadIdx.x; c < p.cols; c += kPrepThreads) {
            if (!SPL_CHECK(c < p.cols, kSiteOrthIn, c)) continue;
            const float g = V::load1(row, c);
            float m = 0.0f;
            if (mom != nullptr) {
                m = __fmaf_rn(p.mu, mom[c], g);
                mom[c] = m;
            }
            const float u = step_value(g, m, p);
            sum = __fmaf_rn(u, u, sum);
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

__device__ __forceinline__ void store_state(__half* hi, __half* lo, int64_t at, float x) {
    const __half h = __float2half_rn(x);
    hi[at] = h;
    lo[at] = __float2half_rn(__fmul_rn(__fsub_rn(x, __half2float(h)), kLoScale));
}

// X = u / (|u| + eps) in the state's format, through a 32 x 32 tile in shared memory when the
// matrix is tall.
template <bool kBf16, bool kTall>
__global__ void __launch_bounds__(kPrepThreads) k_orth_state(const __grid_constant__ PrepArgs p) {
    using V = Vec16<kBf16>;
    __shared__ double s_sum[kPrepThreads / 32];
    __shared__ float s_factor;
    __shared__ float s_tile[32][33];
    const int64_t b = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    double total = 0.0;
    for (int i = threadIdx.x; i < p.num_partials; i += kPrepThreads)
        total += p.partials[b * kMaxPartials + i];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(kAll, total, off);
    if (lane == 0) s_sum[warp] = total;
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
    const float f = s_factor;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 32, c0 = static_cast<int64_t>(blockIdx.x) * 32;
    __half* hi = p.hi + b * p.plane;
    __half* lo = p.lo + b * p.plane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + warp + 8 * i, c = c0 + lane;
        if (r >= p.rows || c >= p.cols || !SPL_CHECK(r < p.rows, kSiteOrthIn, r)) continue;
        const float g = V::load1(static_cast<const unsigned char*>(p.update) +
                                     (b * p.batch_stride + r * p.row_stride) * V::kBytes, c);
        const float m = p.momentum == nullptr ? 0.0f : p.momentum[(b * p.rows + r) * p.cols + c];
        const float x = __fmul_rn(step_value(g, m, p), f);
        if constexpr (kTall)
            s_tile[warp + 8 * i][lane] = x;
        else
            store_state(hi, lo, r * p.ld + c, x);
    }
    if constexpr (kTall) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = r0 + lane, c = c0 + warp + 8 * i;   // the state's column and row
            if (r < p.rows && c < p.cols && SPL_CHECK(r < p.ld, kSiteOrthState, r))
                store_state(hi, lo, c * p.ld + r, s_tile[lane][warp + 8 * i]);
        }
    }
}

// ---- the products ---------------------------------------------------------------------------
enum Product { kGram = 0, kPoly = 1, kUpdate = 2, kLast = 3 };   // kLast: the update that ends it

constexpr int kTileM = 128, kTileK = 64;
constexpr int kGemmThreads = 192;          // four epilogue warps, one for TMA, one for the MMAs
constexpr int kEpiCols = 64;               // columns of a tile per epilogue step
constexpr int kEpiPitch = kEpiCols + 1;    // floats; odd: columns and rows both read without conflicts

template <int kTileN>
struct GemmShape {
    static constexpr int kBytesA = kTileM * kTileK * 2, kBytesB = kTileN * kTileK * 2;
    static constexpr int kStage = kBytesA + kBytesB;
    static constexpr int kEpilogue = 4 * 32 * kEpiPitch * 4;
    static constexpr int kStages = (227 * 1024 - 2048 - kEpilogue) / kStage;
    static constexpr int kSmem = kStages * kStage + kEpilogue + 1024 + 512;
    static constexpr int kTmemCols = 2 * kTileN;   // two accumulators
};

struct GemmArgs {
    int m, n, k;                 // of the product
    int tiles_m, tiles_n, tiles; // tiles per matrix
    int total_tiles;
    int batch;
    float fa, fb;                // value = fa * source + fb * accumulator
    const __half* src_hi;        // kPoly: A; kUpdate, kLast: X
    const __half* src_lo;
    int64_t src_ld, src_plane;
    __half* dst_hi;
    __half* dst_lo;
    int64_t dst_ld, dst_plane;
    uint16_t* out;               // kLast
    int64_t out_ld, out_plane;
    bool tall;                   // kLast: out holds X^T
    uint32_t* flags;
};

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle (rows of 64 fp16, groups of 8 rows 1,024
// bytes apart; `lead` is the distance of neighbouring 64-wide blocks of an operand whose rows
// run along the other dimension than K).
__device__ __forceinline__ uint64_t operand_desc(const void* p, uint32_t lead) {
    const uint64_t addr = smem_addr(p);
    return ((addr & 0x3ffffu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(add ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void tmem_load_32(uint32_t addr, uint32_t (&v)[32]) {
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

struct TileAt {
    int b, i, j;   // matrix, tile row, tile column
};

// Tiles of a symmetric product: tile row i (128 rows) has the columns' tiles that reach its last
// row's diagonal.  kRatio = kTileN / kTileM tile rows share a count.
template <bool kSym, int kTileN>
__device__ __forceinline__ TileAt tile_at(const GemmArgs& g, int t) {
    TileAt at;
    at.b = t / g.tiles;
    int r = t - at.b * g.tiles;
    if constexpr (kSym) {
        constexpr int kRatio = kTileN / kTileM;
        // the first p groups of kRatio tile rows hold kRatio p (p + 1) / 2 tiles
        const float q = static_cast<float>(2 * r) / kRatio;
        int p = static_cast<int>((sqrtf(1.0f + 4.0f * q) - 1.0f) * 0.5f);
        while (kRatio * p * (p + 1) / 2 > r) --p;
        while (kRatio * (p + 1) * (p + 2) / 2 <= r) ++p;
        r -= kRatio * p * (p + 1) / 2;
        at.i = p * kRatio + r / (p + 1);
        at.j = r % (p + 1);
    } else {
        at.i = r % g.tiles_m;
        at.j = r / g.tiles_m;
    }
    return at;
}

__device__ __forceinline__ void unpack_half8(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = *reinterpret_cast<const __half2*>(&w[i]);
        x[2 * i] = __low2float(h);
        x[2 * i + 1] = __high2float(h);
    }
}

__device__ __forceinline__ uint4 pack_half8(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint16_t half_bits(float x) {
    const __half h = __float2half_rn(x);
    return *reinterpret_cast<const uint16_t*>(&h);
}

__device__ __forceinline__ uint16_t bf16_bits(float x) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(0.0f), "f"(x));
    return static_cast<uint16_t>(w);
}

// One epilogue step of a warp: 32 rows from row0, kEpiCols columns from col0, accumulators in buf.
// Direct places take 8 columns per lane, 4 rows at a time; transposed ones 8 rows per lane, 8
// columns at a time.
template <int kMode>
__device__ __forceinline__ void epilogue_step(const GemmArgs& g, float* buf, int b, int row0,
                                              int col0, int lane) {
    constexpr bool kSym = kMode == kGram || kMode == kPoly;
    // values in place: buf becomes fa * source + fb * accumulator
#pragma unroll 2
    for (int it = 0; it < 8; ++it) {
        const int lr = it * 4 + (lane >> 3), lc = (lane & 7) * 8;
        const int r = row0 + lr, c = col0 + lc;
        if (r >= g.m || c >= g.n || (kSym && c > r)) continue;
        float v[8];
        float* at = buf + lr * kEpiPitch + lc;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(g.fb, at[i]);
        if constexpr (kMode != kGram) {
            float s[8];
            const int64_t from = b * g.src_plane + r * g.src_ld + c;
            if (!SPL_CHECK(c + 8 <= g.src_ld, kSiteOrthState, c)) continue;
            unpack_half8(*reinterpret_cast<const uint4*>(g.src_hi + from), s);
            if constexpr (kMode == kUpdate || kMode == kLast) {
                float l[8];
                unpack_half8(*reinterpret_cast<const uint4*>(g.src_lo + from), l);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] = __fmaf_rn(l[i], 1.0f / kLoScale, s[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fmaf_rn(g.fa, s[i], v[i]);
        }
        if constexpr (kMode == kLast) {
            if (!g.tall) {
                uint16_t* to = g.out + b * g.out_plane + static_cast<int64_t>(r) * g.out_ld + c;
                if (!SPL_CHECK(r < g.m, kSiteOrthOut, r)) continue;
                if (c + 8 <= g.n && (g.out_ld & 7) == 0) {
                    *reinterpret_cast<uint4*>(to) = Vec16<true>::pack(v);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c + i < g.n) to[i] = bf16_bits(v[i]);
                }
            }
        } else {
            __half* to = g.dst_hi + b * g.dst_plane + r * g.dst_ld + c;
            if (!SPL_CHECK(c + 8 <= g.dst_ld, kSiteOrthState, c)) continue;
            if (!kSym || c + 7 <= r) {   // columns up to the row pitch are this buffer's own
                const uint4 h = pack_half8(v);
                *reinterpret_cast<uint4*>(to) = h;
                if constexpr (kMode == kUpdate) {
                    float back[8], l[8];
                    unpack_half8(h, back);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        l[i] = __fmul_rn(__fsub_rn(v[i], back[i]), kLoScale);
                    *reinterpret_cast<uint4*>(g.dst_lo + b * g.dst_plane + r * g.dst_ld + c) = pack_half8(l);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i <= r) reinterpret_cast<uint16_t*>(to)[i] = half_bits(v[i]);
            }
        }
        if (kSym || (kMode == kLast && g.tall)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) at[i] = v[i];
        }
    }
    if (!(kSym || (kMode == kLast && g.tall))) return;
    __syncwarp();
#pragma unroll 2
    for (int it = 0; it < 8; ++it) {
        const int lc = it * 8 + (lane >> 2), lr = (lane & 3) * 8;
        const int r = row0 + lr, c = col0 + lc;
        if (r >= g.m || c >= g.n || (kSym && r + 7 <= c)) continue;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = buf[(lr + i) * kEpiPitch + lc];
        if constexpr (kMode == kLast) {
            uint16_t* to = g.out + b * g.out_plane + static_cast<int64_t>(c) * g.out_ld + r;
            if (!SPL_CHECK(c < g.n, kSiteOrthOut, c)) continue;
            if (r + 8 <= g.m && (g.out_ld & 7) == 0) {
                *reinterpret_cast<uint4*>(to) = Vec16<true>::pack(v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (r + i < g.m) to[i] = bf16_bits(v[i]);
            }
        } else {   // strictly above the diagonal; the diagonal is written in place above
            __half* to = g.dst_hi + b * g.dst_plane + c * g.dst_ld + r;
            if (!SPL_CHECK(r + 8 <= g.dst_ld, kSiteOrthState, r)) continue;
            if (r > c && r + 8 <= g.m) {
                *reinterpret_cast<uint4*>(to) = pack_half8(v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (r + i > c && r + i < g.m) reinterpret_cast<uint16_t*>(to)[i] = half_bits(v[i]);
            }
        }
    }
    __syncwarp();
}

// D = A B^T (B's rows run along K) for kGram and kPoly, D = A B (B's rows run along N) for the
// updates, tile by tile: one thread issues TMA loads into a ring of stages, one issues the MMAs,
// four warps turn finished accumulators into results while the next tile's MMAs run (two
// accumulators in tensor memory).  Every wait is bounded; on a timeout all roles leave their
// loops, wait (bounded) for what is in flight, and the flags word says so.
template <int kMode, int kTileN>
__global__ void __launch_bounds__(kGemmThreads, 1)
k_orth_product(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ GemmArgs g) {
    using S = GemmShape<kTileN>;
    constexpr bool kSym = kMode == kGram || kMode == kPoly;
    constexpr bool kBRowsAlongN = !kSym;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* stages = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    float* epi = reinterpret_cast<float*>(stages + S::kStages * S::kStage);
    uint64_t* bars = reinterpret_cast<uint64_t*>(stages + S::kStages * S::kStage + S::kEpilogue);
    uint64_t* full = bars;
    uint64_t* empty = bars + S::kStages;
    uint64_t* acc_full = bars + 2 * S::kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_full + 4;
    __shared__ uint32_t s_tmem, s_late;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int k_blocks = (g.k + kTileK - 1) / kTileK;

    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], 4);
        }
        mbar_init(drain, 1);
        s_late = 0;
        fence_async_smem();
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(&s_tmem)), "n"(S::kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = s_tmem;

    if (warp == 4) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int used = 0;   // stages ever filled, up to kStages
            bool late = false;
            for (int t = blockIdx.x; t < g.total_tiles && !late; t += gridDim.x) {
                const TileAt at = tile_at<kSym, kTileN>(g, t);
                for (int kb = 0; kb < k_blocks; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u)) {
                        late = true;
                        break;
                    }
                    unsigned char* a = stages + stage * S::kStage;
                    unsigned char* b = a + S::kBytesA;
                    mbar_expect_tx(&full[stage], S::kStage);
                    tma_load_3d(a, &map_a, kb * kTileK, at.i * kTileM, at.b, &full[stage]);
                    if constexpr (kBRowsAlongN) {
#pragma unroll
                        for (int q = 0; q < kTileN / 64; ++q)
                            tma_load_3d(b + q * 64 * kTileK * 2, &map_b, at.j * kTileN + q * 64,
                                        kb * kTileK, at.b, &full[stage]);
                    } else {
#pragma unroll
                        for (int q = 0; q < kTileN / 128; ++q)
                            tma_load_3d(b + q * 128 * kTileK * 2, &map_b, kb * kTileK,
                                        at.j * kTileN + q * 128, at.b, &full[stage]);
                    }
                    if (used < S::kStages) ++used;
                    if (++stage == S::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (late) {   // the copies still in flight must land before the CTA leaves
                bool pending = false;
                for (int q = 0; q < used; ++q) {
                    const int s = (stage + S::kStages - 1 - q) % S::kStages;
                    const uint32_t ph = s < stage ? phase : phase ^ 1u;
                    pending |= !mbar_wait(&full[s], ph);
                }
                if (g.flags != nullptr)
                    atomicOr(g.flags, kFlagTimeout | (pending ? kFlagCopyPending : 0u));
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        if (lane == 0) {
            // fp32 accumulators, fp16 operands, B transposed where its rows run along N
            constexpr uint32_t idesc = (1u << 4) | ((kBRowsAlongN ? 1u : 0u) << 16) |
                                       (static_cast<uint32_t>(kTileN / 8) << 17) |
                                       (static_cast<uint32_t>(kTileM / 16) << 24);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool late = false;
            for (int t = blockIdx.x; t < g.total_tiles && !late; t += gridDim.x) {
                if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1u)) {
                    late = true;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                for (int kb = 0; kb < k_blocks; ++kb) {
                    if (!mbar_wait(&full[stage], phase)) {
                        late = true;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const unsigned char* a = stages + stage * S::kStage;
                    const uint64_t da = operand_desc(a, 16);
                    const uint64_t db = operand_desc(a + S::kBytesA, kBRowsAlongN ? 64 * kTileK * 2 : 16);
#pragma unroll
                    for (int k = 0; k < kTileK / 16; ++k)   // 16 values of K: 32 bytes, or 16 rows
                        mma_f16(tmem + acc * kTileN, da + k * 2, db + k * (kBRowsAlongN ? 128 : 2),
                                idesc, kb > 0 || k > 0);
                    mma_commit(&empty[stage]);
                    if (++stage == S::kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (late) break;
                mma_commit(&acc_full[acc]);
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (late) {
                mma_commit(drain);
                mbar_wait(drain, 0);
                if (g.flags != nullptr) atomicOr(g.flags, kFlagTimeout);
            }
        }
        __syncwarp();
    } else {
        float* buf = epi + warp * 32 * kEpiPitch;
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int t = blockIdx.x; t < g.total_tiles; t += gridDim.x) {
            if (!mbar_wait(&acc_full[acc], acc_phase)) s_late = 1;
            __syncwarp();
            if (*static_cast<volatile uint32_t*>(&s_late) != 0) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const TileAt at = tile_at<kSym, kTileN>(g, t);
            const int row0 = at.i * kTileM + warp * 32;
            for (int c = 0; c < kTileN; c += kEpiCols) {
                const int col0 = at.j * kTileN + c;
                if (col0 >= g.n || row0 >= g.m || (kSym && col0 > row0 + 31)) break;
#pragma unroll
                for (int h = 0; h < kEpiCols / 32; ++h) {
                    uint32_t v[32];
                    tmem_load_32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + acc * kTileN + c + h * 32, v);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int i = 0; i < 32; ++i) buf[lane * kEpiPitch + h * 32 + i] = __uint_as_float(v[i]);
                }
                __syncwarp();
                epilogue_step<kMode>(g, buf, at.b, row0, col0, lane);
                __syncwarp();
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
            acc ^= 1;
            if (acc == 0) acc_phase ^= 1u;
        }
    }
    __syncthreads();
    if (warp == 5)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kTmemCols));
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

// Tensor map over fp16 [batch][rows][cols] with row pitch ld, boxes of 64 columns x box_rows.
bool make_map(CUtensorMap* map, __half* base, int64_t batch, int64_t rows, int64_t cols, int64_t ld,
              int box_rows) {
    const EncodeTiled enc = encode_tiled();
    if (enc == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * 2), static_cast<cuuint64_t>(rows * ld * 2)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t step[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, base, dims, strides, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

struct OrthLayout {
    int64_t m, n, ldx, ldm;   // short and long side, row pitches of X and of A and B
    size_t hi[2], lo[2], a, b, partials, bytes;
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
    l.a = take(static_cast<size_t>(batch * l.m * l.ldm) * 2);
    l.b = take(static_cast<size_t>(batch * l.m * l.ldm) * 2);
    l.partials = take(static_cast<size_t>(batch) * kMaxPartials * sizeof(double));
    l.bytes = at;
    return l;
}

template <int kMode, int kTileN>
cudaError_t launch_product(const CUtensorMap& a, const CUtensorMap& b, GemmArgs g, int sms,
                           cudaStream_t stream) {
    using S = GemmShape<kTileN>;
    constexpr bool kSym = kMode == kGram || kMode == kPoly;
    g.tiles_m = (g.m + kTileM - 1) / kTileM;
    g.tiles_n = (g.n + kTileN - 1) / kTileN;
    g.tiles = g.tiles_m * g.tiles_n;
    if (kSym) {
        g.tiles = 0;
        for (int i = 0; i < g.tiles_m; ++i) g.tiles += i / (kTileN / kTileM) + 1;
    }
    g.total_tiles = g.tiles * g.batch;
    const void* kern = reinterpret_cast<const void*>(&k_orth_product<kMode, kTileN>);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    const int grid = g.total_tiles < sms ? g.total_tiles : sms;
    k_orth_product<kMode, kTileN><<<grid, kGemmThreads, S::kSmem, stream>>>(a, b, g);
    return cudaGetLastError();
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
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    __half* hi[2] = {reinterpret_cast<__half*>(ws + l.hi[0]), reinterpret_cast<__half*>(ws + l.hi[1])};
    __half* lo[2] = {reinterpret_cast<__half*>(ws + l.lo[0]), reinterpret_cast<__half*>(ws + l.lo[1])};
    __half* gram = reinterpret_cast<__half*>(ws + l.a);
    __half* poly = reinterpret_cast<__half*>(ws + l.b);

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
    p.partials = reinterpret_cast<double*>(ws + l.partials);
    p.num_partials = static_cast<int>(a.rows < kMaxPartials ? a.rows : kMaxPartials);
    p.hi = hi[0];
    p.lo = lo[0];
    p.ld = l.ldx;
    p.plane = l.m * l.ldx;
    p.flags = a.flags;
    const dim3 norm_grid(static_cast<unsigned>(p.num_partials), static_cast<unsigned>(a.batch));
    const dim3 state_grid(static_cast<unsigned>((a.cols + 31) / 32), static_cast<unsigned>((a.rows + 31) / 32),
                          static_cast<unsigned>(a.batch));
    if (bf16) {
        k_orth_norm<true><<<norm_grid, kPrepThreads, 0, stream>>>(p);
        if (tall) k_orth_state<true, true><<<state_grid, kPrepThreads, 0, stream>>>(p);
        else k_orth_state<true, false><<<state_grid, kPrepThreads, 0, stream>>>(p);
    } else {
        k_orth_norm<false><<<norm_grid, kPrepThreads, 0, stream>>>(p);
        if (tall) k_orth_state<false, true><<<state_grid, kPrepThreads, 0, stream>>>(p);
        else k_orth_state<false, false><<<state_grid, kPrepThreads, 0, stream>>>(p);
    }
    if ((e = cudaGetLastError()) != cudaSuccess) return e;

    CUtensorMap x_k[2], x_n[2], gram_k, poly_k;   // operands with rows along K, and X along N
    for (int i = 0; i < 2; ++i)
        if (!make_map(&x_k[i], hi[i], a.batch, l.m, l.n, l.ldx, 128) ||
            !make_map(&x_n[i], hi[i], a.batch, l.m, l.n, l.ldx, 64))
            return cudaErrorInvalidValue;
    if (!make_map(&gram_k, gram, a.batch, l.m, l.m, l.ldm, 128) ||
        !make_map(&poly_k, poly, a.batch, l.m, l.m, l.ldm, 128))
        return cudaErrorInvalidValue;

    constexpr int kN = 256;
    for (int s = 0; s < a.steps; ++s) {
        const int x = s & 1;
        GemmArgs g = {};
        g.batch = static_cast<int>(a.batch);
        g.flags = a.flags;
        g.m = static_cast<int>(l.m);
        g.n = g.m;
        g.k = static_cast<int>(l.n);
        g.fb = kGramScale / (p.x_scale * p.x_scale);
        g.dst_hi = gram;
        g.dst_ld = l.ldm;
        g.dst_plane = l.m * l.ldm;
        if ((e = launch_product<kGram, kN>(x_k[x], x_k[x], g, sms, stream)) != cudaSuccess) return e;
        g.k = g.m;
        g.fa = a.coef[1];
        g.fb = a.coef[2] / kGramScale;
        g.src_hi = gram;
        g.src_ld = l.ldm;
        g.src_plane = l.m * l.ldm;
        g.dst_hi = poly;
        if ((e = launch_product<kPoly, kN>(gram_k, gram_k, g, sms, stream)) != cudaSuccess) return e;
        g.n = static_cast<int>(l.n);
        g.fa = a.coef[0];
        g.fb = 1.0f / kGramScale;
        g.src_hi = hi[x];
        g.src_lo = lo[x];
        g.src_ld = l.ldx;
        g.src_plane = l.m * l.ldx;
        g.dst_hi = hi[x ^ 1];
        g.dst_lo = lo[x ^ 1];
        g.dst_ld = l.ldx;
        g.dst_plane = l.m * l.ldx;
        if (s + 1 < a.steps) {
            e = launch_product<kUpdate, kN>(poly_k, x_n[x], g, sms, stream);
        } else {
            g.fa /= p.x_scale;
            g.fb /= p.x_scale;
            g.out = a.out;
            g.out_ld = a.cols;
            g.out_plane = a.rows * a.cols;
            g.tall = tall;
            e = launch_product<kLast, kN>(poly_k, x_n[x], g, sms, stream);
        }
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace spl
