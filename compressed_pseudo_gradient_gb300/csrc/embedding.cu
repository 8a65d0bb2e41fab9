// Embedding lookup with scaling and its gradient (spl_embedding, spl_embedding_grad; declared
// in include/spl_local.h).
//
//   out[t]     = scale table[id_t]
//   d_table[v] = scale (sum of d_out[t] over the tokens t with id_t = v, in ascending t)
//
// The gradient first sorts the tokens by id (up to kSmallSort of them in one CTA's shared memory,
// more by a stable radix sort: digit counts per tile, a scan, a ranked scatter), then sums over
// windows of consecutive sorted tokens: a run of
// equal ids inside one window is summed and written at once, a run that crosses window borders
// leaves one partial sum per window, joined in window order afterwards.  The work per CTA is
// thus the same however often an id repeats, no floating-point atomics are used, and every run
// gives the same bits.  Rows without tokens are zeroed by CTAs of the summing launch, found in a
// bitmap of the ids seen; beside a small sort, which leaves the GPU idle, the whole table is
// zeroed instead.
#include "local_device.cuh"
#include "local_kernels.h"

namespace spl {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---- lookup ---------------------------------------------------------------------------------
// Bound: HBM, each looked-up row read once and written once.  The output is taken as one flat
// range of units (16-byte vectors, or single values where a row is not 16-byte aligned); a CTA
// takes kThreads * kUnits consecutive ones, so short rows share a CTA and long ones split.
constexpr int kThreads = 256;
constexpr int kUnits = 4;

template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kThreads)
k_embedding(const __grid_constant__ EmbeddingArgs a, uint32_t units) {
    using V = Vec16<kBf16>;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads * kUnits);
    const int64_t row0 = first / units;
    const uint32_t rem0 = static_cast<uint32_t>(first - row0 * units);
    int64_t row[kUnits];
    uint32_t unit[kUnits];
    int64_t id[kUnits];
    uint4 raw[kUnits];
    float val[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const uint32_t at = rem0 + u * kThreads + threadIdx.x;
        row[u] = row0 + at / units;
        unit[u] = at % units;
        id[u] = row[u] < a.count ? token_at(a.ids, row[u]) : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        raw[u] = make_uint4(0, 0, 0, 0);
        val[u] = 0.0f;
        if (id[u] < 0 || id[u] >= a.vocab) continue;   // an id outside the table: zeros
        if (!SPL_CHECK(unit[u] < units, kSiteTable, unit[u])) continue;
        const unsigned char* src =
            static_cast<const unsigned char*>(a.table) + id[u] * a.stride * V::kBytes;
        if constexpr (kVec)
            raw[u] = reinterpret_cast<const uint4*>(src)[unit[u]];
        else
            val[u] = V::load1(src, unit[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        if (row[u] >= a.count || !SPL_CHECK(unit[u] < units, kSiteRowsOut, unit[u])) continue;
        if (unit[u] == 0 && (id[u] < 0 || id[u] >= a.vocab) && a.flags != nullptr)
            atomicOr(a.flags, kFlagBadToken);
        unsigned char* dst = static_cast<unsigned char*>(a.out) + row[u] * a.out_stride * V::kBytes;
        if constexpr (kVec) {
            float x[V::kN];
            V::unpack(raw[u], x);
#pragma unroll
            for (int i = 0; i < V::kN; ++i) x[i] = __fmul_rn(x[i], a.scale);
            __stcs(reinterpret_cast<uint4*>(dst) + unit[u], V::pack(x));
        } else {
            V::store1(dst, unit[u], __fmul_rn(val[u], a.scale));
        }
    }
}

// ---- sort by id -----------------------------------------------------------------------------
// Least-significant-digit radix sort of (id, position) with digits of up to 10 bits.  A tile is
// kTile consecutive entries, a warp's share of it consecutive too, so ranks by (tile, warp,
// round, lane) keep equal digits in order.  Ids that take no part (padding, out of range) get
// the key `vocab`, which sorts last.
constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = 8;
constexpr int kTile = kSortThreads * kSortRounds;
constexpr int kMaxDigits = 1024;

struct SortPass {
    TokenIds ids;               // first pass: the call's ids
    const uint32_t* keys_in;    // later passes
    const uint32_t* pos_in;
    uint32_t* keys_out;
    uint32_t* pos_out;
    uint32_t* counts;           // [digit][tile]
    uint32_t* seen;             // bitmap of the ids that take part (first pass)
    uint32_t* flags;
    int64_t padding_id;
    uint32_t n, vocab, tiles;
    int shift, bits;
    bool first;
};

__device__ __forceinline__ uint32_t sort_key(const SortPass& p, uint32_t i) {
    if (!p.first) return p.keys_in[i];
    const int64_t id = token_at(p.ids, i);
    return id < 0 || id >= p.vocab || id == p.padding_id ? p.vocab : static_cast<uint32_t>(id);
}

__global__ void __launch_bounds__(kSortThreads) k_sort_count(const __grid_constant__ SortPass p) {
    __shared__ uint32_t s_count[kMaxDigits];
    const int digits = 1 << p.bits;
    for (int d = threadIdx.x; d < digits; d += kSortThreads) s_count[d] = 0;
    __syncthreads();
    for (int r = 0; r < kSortRounds; ++r) {
        const uint32_t i = blockIdx.x * kTile + r * kSortThreads + threadIdx.x;
        if (i >= p.n || !SPL_CHECK(i < p.n, kSiteSorted, i)) continue;
        const uint32_t key = sort_key(p, i);
        atomicAdd(&s_count[(key >> p.shift) & (digits - 1)], 1u);
        if (p.first) {
            if (key < p.vocab) {
                atomicOr(&p.seen[key >> 5], 1u << (key & 31));
            } else if (p.flags != nullptr) {
                const int64_t id = token_at(p.ids, i);
                if (id != p.padding_id) atomicOr(p.flags, kFlagBadToken);
            }
        }
    }
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kSortThreads)
        p.counts[static_cast<size_t>(d) * p.tiles + blockIdx.x] = s_count[d];
}

// Exclusive prefix sums of n counts, in place, by one CTA.
__global__ void __launch_bounds__(1024) k_sort_scan(uint32_t* __restrict__ counts, uint32_t n) {
    __shared__ uint32_t s_warp[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t carry = 0;
    for (uint32_t base = 0; base < n; base += 4096) {
        const uint32_t i = base + threadIdx.x * 4;
        uint32_t v[4], sum = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k] = sum;
            sum += i + k < n ? counts[i + k] : 0u;
        }
        uint32_t scan = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t o = __shfl_up_sync(kAll, scan, off);
            if (lane >= off) scan += o;
        }
        if (lane == 31) s_warp[warp] = scan;
        __syncthreads();
        if (warp == 0) {
            uint32_t w = s_warp[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const uint32_t o = __shfl_up_sync(kAll, w, off);
                if (lane >= off) w += o;
            }
            s_warp[lane] = w;
        }
        __syncthreads();
        const uint32_t before = carry + (warp > 0 ? s_warp[warp - 1] : 0u) + scan - sum;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) counts[i + k] = before + v[k];
        carry += s_warp[31];
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSortThreads) k_sort_scatter(const __grid_constant__ SortPass p) {
    __shared__ uint32_t s_rank[kSortWarps][kMaxDigits];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int digits = 1 << p.bits;
    for (int d = threadIdx.x; d < kSortWarps * kMaxDigits; d += kSortThreads) (&s_rank[0][0])[d] = 0;
    __syncthreads();
    uint32_t key[kSortRounds], rank[kSortRounds];
    const uint32_t base = blockIdx.x * kTile + warp * (32 * kSortRounds) + lane;
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) key[r] = base + r * 32 < p.n ? sort_key(p, base + r * 32) : 0u;
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const bool ok = base + r * 32 < p.n;
        // entries past the end share a value no digit has and take no rank
        const uint32_t d = ok ? (key[r] >> p.shift) & (digits - 1) : 0xffffffffu;
        const unsigned peers = __match_any_sync(kAll, d);
        const int lead = __ffs(peers) - 1;
        uint32_t before = 0;
        if (lane == lead && ok) {
            before = s_rank[warp][d];
            s_rank[warp][d] = before + __popc(peers);
        }
        before = __shfl_sync(kAll, before, lead);
        rank[r] = before + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
    }
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kSortThreads) {   // start of each warp's share
        uint32_t at = p.counts[static_cast<size_t>(d) * p.tiles + blockIdx.x];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = s_rank[w][d];
            s_rank[w][d] = at;
            at += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
        const uint32_t i = base + r * 32;
        if (i >= p.n) continue;
        const uint32_t to = s_rank[warp][(key[r] >> p.shift) & (digits - 1)] + rank[r];
        if (!SPL_CHECK(to < p.n, kSiteSorted, to)) continue;
        p.keys_out[to] = key[r];
        p.pos_out[to] = p.first ? i : p.pos_in[i];
    }
}

// ---- small sorts ----------------------------------------------------------------------------
// Bitonic sort of (key, position) pairs in one CTA: positions are distinct, so the order is that
// of the stable sort above.  The other CTAs of the launch zero the table meanwhile.
constexpr int kSmallSort = 4096;
constexpr int kSmallThreads = 1024;

struct ZeroTable {
    float* base;
    int64_t rows, width, stride;   // rows = 0: nothing to zero
};

__global__ void __launch_bounds__(kSmallThreads)
k_sort_small(const __grid_constant__ SortPass p, const __grid_constant__ ZeroTable z, int padded) {
    const int tid = threadIdx.x;
    if (blockIdx.x > 0) {
        const int64_t ctas = gridDim.x - 1, cta = blockIdx.x - 1;
        if (z.stride == z.width) {   // one range of memory: 16-byte stores between its ends
            const int64_t n = z.rows * z.width;
            const RowSplit sp = split_row<false>(z.base, n);
            float4* v = reinterpret_cast<float4*>(z.base + sp.head);
            for (int64_t i = cta * kSmallThreads + tid; i < sp.vecs; i += ctas * kSmallThreads)
                if (SPL_CHECK(sp.head + 4 * (i + 1) <= n, kSiteRowsOut, i)) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int64_t done = sp.head + 4 * sp.vecs;
            if (cta == 0 && tid < sp.head) z.base[tid] = 0.0f;
            if (cta == 0 && tid < n - done) z.base[done + tid] = 0.0f;
        } else {
            for (int64_t r = cta; r < z.rows; r += ctas)
                for (int64_t i = tid; i < z.width; i += kSmallThreads) z.base[r * z.stride + i] = 0.0f;
        }
        return;
    }
    __shared__ uint64_t s[kSmallSort];
    for (int i = tid; i < padded; i += kSmallThreads) {
        uint64_t e = ~0ull;
        if (i < static_cast<int>(p.n)) {
            const uint32_t key = sort_key(p, i);
            if (key == p.vocab && p.flags != nullptr && token_at(p.ids, i) != p.padding_id)
                atomicOr(p.flags, kFlagBadToken);
            e = (static_cast<uint64_t>(key) << 32) | static_cast<uint32_t>(i);
        }
        s[i] = e;
    }
    __syncthreads();
    for (int size = 2; size <= padded; size <<= 1) {
        for (int off = size >> 1; off > 0; off >>= 1) {
            for (int q = tid; q < padded / 2; q += kSmallThreads) {
                const int i = (q / off) * 2 * off + q % off, j = i + off;   // off is a power of two
                const uint64_t a = s[i], b = s[j];
                if ((a > b) == ((i & size) == 0)) {
                    s[i] = b;
                    s[j] = a;
                }
            }
            __syncthreads();
        }
    }
    for (int i = tid; i < static_cast<int>(p.n); i += kSmallThreads) {
        p.keys_out[i] = static_cast<uint32_t>(s[i] >> 32);
        p.pos_out[i] = static_cast<uint32_t>(s[i]);
    }
}

// ---- sums -----------------------------------------------------------------------------------
// Sorted tokens per window.  Short windows give few tokens enough CTAs (2,000 tokens of width
// 1001: SMALLWIN us with 16, 6 us with 64); long ones leave fewer partial sums.
constexpr int kWindow = 64;
constexpr int kShortWindow = 16;
constexpr int kShortWindowTokens = 16384;   // up to this many tokens

int window_of(int64_t count) { return count <= kShortWindowTokens ? kShortWindow : kWindow; }

struct GradSums {
    const uint32_t* keys;   // sorted ids
    const uint32_t* pos;
    const uint32_t* seen;
    const void* d_out;
    int64_t d_out_stride;
    float* d_table;
    int64_t stride, width;
    float* partials;        // [window][head, tail][width]
    uint32_t n, vocab, windows, window;
    float scale;
    bool accumulate;
};

// The values of one unit: a 16-byte vector of the input, or one value.
template <bool kBf16, bool kVec>
struct Unit {
    static constexpr int kN = kVec ? Vec16<kBf16>::kN : 1;
    float x[kN];

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = 0.0f;
    }
    __device__ __forceinline__ void add(const Unit& o) {
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = __fadd_rn(x[i], o.x[i]);
    }
    __device__ __forceinline__ void load_in(const void* row, int64_t unit) {
        if constexpr (kVec)
            Vec16<kBf16>::unpack(__ldcs(static_cast<const uint4*>(row) + unit), x);
        else
            x[0] = Vec16<kBf16>::load1(row, unit);
    }
    __device__ __forceinline__ void load_f32(const float* p) {
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < kN; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(p + i);
                x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
            }
        } else {
            x[0] = *p;
        }
    }
    __device__ __forceinline__ void store_f32(float* p) const {
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < kN; i += 4)
                *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        } else {
            *p = x[0];
        }
    }
    // A finished sum into its row of the gradient.
    __device__ __forceinline__ void finish(float* p, float scale, bool accumulate) {
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = __fmul_rn(x[i], scale);
        if (accumulate) {
            Unit old;
            old.load_f32(p);
            add(old);
        }
        store_f32(p);
    }
};

// A run's sum within a window belongs to the row (both ends inside), to the window's head
// partial (it continues the previous window) or to its tail partial (it starts here and goes
// on).
template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kThreads)
k_grad_windows(const __grid_constant__ GradSums g, int col_blocks, uint32_t window_ctas,
               uint32_t zero_rows) {
    using U = Unit<kBf16, kVec>;
    // the zeroing CTAs are spread between the summing ones, so that reads and writes mix
    const uint64_t total = gridDim.x;
    const uint32_t summing = static_cast<uint32_t>(blockIdx.x * static_cast<uint64_t>(window_ctas) / total);
    if (static_cast<uint32_t>((blockIdx.x + 1ull) * window_ctas / total) == summing) {
        const uint32_t row0 = (blockIdx.x - summing) * zero_rows;
        for (uint32_t r = row0; r < row0 + zero_rows && r < g.vocab; ++r) {
            if ((g.seen[r >> 5] >> (r & 31)) & 1u) continue;
            float* dst = g.d_table + r * g.stride;
            if constexpr (kVec) {
                for (int64_t i = threadIdx.x; i < g.width / 4; i += blockDim.x)
                    reinterpret_cast<float4*>(dst)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            } else {
                for (int64_t i = threadIdx.x; i < g.width; i += blockDim.x) dst[i] = 0.0f;
            }
        }
        return;
    }
    __shared__ uint32_t s_key[kWindow + 2], s_pos[kWindow];
    const uint32_t win = summing / col_blocks;
    const int64_t unit = static_cast<int64_t>(summing % col_blocks) * blockDim.x + threadIdx.x;
    const uint32_t first = win * g.window;
    const int count = min(g.window, g.n - first);
    for (int i = threadIdx.x; i < count + 2; i += blockDim.x) {
        const int64_t at = static_cast<int64_t>(first) + i - 1;
        s_key[i] = at < 0 || at >= g.n ? 0xffffffffu : g.keys[at];   // one past each end
        if (i < count) s_pos[i] = g.pos[first + i];
    }
    __syncthreads();
    if (unit * U::kN >= g.width) return;
    const int64_t col = unit * U::kN;
    constexpr int kAhead = 8;
    U sum;
    sum.zero();
    int start = 0;   // of the current run
    for (int i0 = 0; i0 < count; i0 += kAhead) {
        U v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
            if (i0 + j < count && s_key[i0 + j + 1] < g.vocab)
                v[j].load_in(static_cast<const unsigned char*>(g.d_out) +
                                 static_cast<int64_t>(s_pos[i0 + j]) * g.d_out_stride *
                                     Vec16<kBf16>::kBytes, unit);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j;
            if (i >= count || s_key[i + 1] >= g.vocab) break;
            sum.add(v[j]);
            const uint32_t key = s_key[i + 1];
            const bool last = i + 1 == count;
            if (!last && s_key[i + 2] == key) continue;
            const bool from_left = start == 0 && s_key[0] == key;
            const bool to_right = last && s_key[i + 2] == key;
            if (from_left || to_right)
                sum.store_f32(g.partials + (2 * static_cast<int64_t>(win) + (from_left ? 0 : 1)) * g.width + col);
            else if (SPL_CHECK(key < g.vocab, kSiteRowsOut, key))
                sum.finish(g.d_table + key * g.stride + col, g.scale, g.accumulate);
            sum.zero();
            start = i + 1;
        }
    }
}

// Joins the partial sums of a run that crosses windows; the window it starts in owns it.
template <bool kBf16, bool kVec>
__global__ void __launch_bounds__(kThreads)
k_grad_join(const __grid_constant__ GradSums g, int col_blocks) {
    using U = Unit<kBf16, kVec>;
    const uint32_t win = blockIdx.x / col_blocks;
    const int64_t unit = static_cast<int64_t>(blockIdx.x % col_blocks) * blockDim.x + threadIdx.x;
    const uint32_t first = win * g.window, next = first + g.window;
    const uint32_t key = g.keys[next - 1];
    if (key >= g.vocab || g.keys[next] != key) return;           // no run leaves this window
    if (first > 0 && g.keys[first] == key && g.keys[first - 1] == key) return;   // not its first
    if (unit * U::kN >= g.width) return;
    const int64_t col = unit * U::kN;
    U sum;
    sum.load_f32(g.partials + (2 * static_cast<int64_t>(win) + 1) * g.width + col);
    for (uint32_t w = win + 1; w < g.windows && g.keys[w * g.window] == key; ++w) {
        U v;
        v.load_f32(g.partials + 2 * static_cast<int64_t>(w) * g.width + col);
        sum.add(v);
    }
    if (SPL_CHECK(key < g.vocab, kSiteRowsOut, key))
        sum.finish(g.d_table + key * g.stride + col, g.scale, g.accumulate);
}

constexpr size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

// Where each array of the gradient's workspace starts, and its size.
struct GradLayout {
    size_t keys[2], pos[2], counts, seen, partials, bytes;
    uint32_t tiles, windows;
};

GradLayout grad_layout(int64_t count, int64_t vocab, int64_t width) {
    GradLayout l;
    l.tiles = static_cast<uint32_t>((count + kTile - 1) / kTile);
    l.windows = static_cast<uint32_t>((count + window_of(count) - 1) / window_of(count));
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round16(bytes);
        return here;
    };
    for (int i = 0; i < 2; ++i) {
        l.keys[i] = take(static_cast<size_t>(count) * 4);
        l.pos[i] = take(static_cast<size_t>(count) * 4);
    }
    l.counts = take(static_cast<size_t>(l.tiles) * kMaxDigits * 4);
    l.seen = take((static_cast<size_t>(vocab) + 31) / 32 * 4);
    l.partials = take(static_cast<size_t>(l.windows) * 2 * static_cast<size_t>(width) * 4);
    l.bytes = at;
    return l;
}

template <bool kBf16, bool kVec>
cudaError_t launch_sums(const GradSums& g, cudaStream_t stream) {
    using U = Unit<kBf16, kVec>;
    const int64_t units = (g.width + U::kN - 1) / U::kN;
    const int threads = static_cast<int>(units >= kThreads ? kThreads : (units + 31) / 32 * 32);
    const int64_t col_blocks = (units + threads - 1) / threads;
    const uint32_t window_ctas = static_cast<uint32_t>(g.windows * col_blocks);
    // rows zeroed per CTA: about 128 KB of them
    uint32_t zero_rows = static_cast<uint32_t>(32768 / g.width);
    if (zero_rows < 1) zero_rows = 1;
    const uint32_t zero_ctas = g.seen == nullptr ? 0 : (g.vocab + zero_rows - 1) / zero_rows;
    if (window_ctas + zero_ctas > 0) {
        k_grad_windows<kBf16, kVec><<<window_ctas + zero_ctas, threads, 0, stream>>>(
            g, static_cast<int>(col_blocks), window_ctas, zero_rows);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (g.windows > 1) {
        k_grad_join<kBf16, kVec><<<static_cast<uint32_t>((g.windows - 1) * col_blocks), threads, 0, stream>>>(
            g, static_cast<int>(col_blocks));
    }
    return cudaGetLastError();
}

template <bool kBf16, bool kVec>
cudaError_t launch_lookup(const EmbeddingArgs& a, cudaStream_t stream) {
    const int64_t units = kVec ? a.width / Vec16<kBf16>::kN : a.width;
    const int64_t per_cta = static_cast<int64_t>(kThreads) * kUnits;
    const int64_t grid = (a.count * units + per_cta - 1) / per_cta;
    k_embedding<kBf16, kVec><<<static_cast<uint32_t>(grid), kThreads, 0, stream>>>(
        a, static_cast<uint32_t>(units));
    return cudaGetLastError();
}

bool on16(const void* p, int64_t stride, int bytes) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (stride * bytes) % 16 == 0;
}

}  // namespace

#if SPL_CHECKED
SPL_DEBUG_READER(debug_read_embedding)
#endif

cudaError_t launch_embedding(const EmbeddingArgs& a, bool bf16, cudaStream_t stream) {
    const int bytes = bf16 ? 2 : 4;
    const bool vec = on16(a.table, a.stride, bytes) && on16(a.out, a.out_stride, bytes) &&
                     (a.width * bytes) % 16 == 0;
    if (bf16) return vec ? launch_lookup<true, true>(a, stream) : launch_lookup<true, false>(a, stream);
    return vec ? launch_lookup<false, true>(a, stream) : launch_lookup<false, false>(a, stream);
}

size_t embedding_grad_workspace(int64_t count, int64_t vocab, int64_t width) {
    return grad_layout(count, vocab, width).bytes;
}

cudaError_t launch_embedding_grad(const EmbeddingGradArgs& a, bool bf16, cudaStream_t stream) {
    const GradLayout l = grad_layout(a.count, a.vocab, a.width);
    unsigned char* ws = static_cast<unsigned char*>(a.workspace);
    auto words = [&](size_t at) { return reinterpret_cast<uint32_t*>(ws + at); };
    cudaError_t e;
    const bool small = a.count <= kSmallSort;
    const bool zero = !a.accumulate;
    int bits = 1;
    while ((a.vocab >> bits) != 0) ++bits;   // keys 0 .. vocab
    const int passes = small ? 1 : (bits + 9) / 10;
    const int digit = (bits + passes - 1) / passes;
    int in = 1;
    if (!small && (e = cudaMemsetAsync(ws + l.seen, 0, (static_cast<size_t>(a.vocab) + 31) / 32 * 4, stream)) != cudaSuccess)
        return e;
    for (int pass = 0; pass < passes; ++pass) {
        SortPass p = {};
        p.ids = a.ids;
        p.first = pass == 0;
        p.keys_in = words(l.keys[in]);
        p.pos_in = words(l.pos[in]);
        p.keys_out = words(l.keys[in ^ 1]);
        p.pos_out = words(l.pos[in ^ 1]);
        p.counts = words(l.counts);
        p.seen = words(l.seen);
        p.flags = a.flags;
        p.padding_id = a.padding_id;
        p.n = static_cast<uint32_t>(a.count);
        p.vocab = static_cast<uint32_t>(a.vocab);
        p.tiles = l.tiles;
        p.shift = pass * digit;
        p.bits = digit;
        if (small) {
            int padded = 2, sms = 0, dev = 0;
            while (padded < a.count) padded *= 2;
            if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
                (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
                return e;
            // about 64 KB of the table per zeroing CTA, at most two per SM
            const int64_t want = (a.vocab * a.width + 16383) / 16384, most = 2 * static_cast<int64_t>(sms) - 1;
            const ZeroTable z = {a.d_table, zero ? a.vocab : 0, a.width, a.stride};
            const unsigned ctas = zero ? static_cast<unsigned>(want < most ? want : most) : 0;
            k_sort_small<<<1 + ctas, kSmallThreads, 0, stream>>>(p, z, padded);
        } else {
            k_sort_count<<<l.tiles, kSortThreads, 0, stream>>>(p);
            k_sort_scan<<<1, 1024, 0, stream>>>(p.counts, l.tiles << digit);
            k_sort_scatter<<<l.tiles, kSortThreads, 0, stream>>>(p);
        }
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        in ^= 1;
    }
    GradSums g = {};
    g.keys = words(l.keys[in]);
    g.pos = words(l.pos[in]);
    g.seen = zero && !small ? words(l.seen) : nullptr;   // rows to zero, by their absence
    g.d_out = a.d_out;
    g.d_out_stride = a.d_out_stride;
    g.d_table = a.d_table;
    g.stride = a.stride;
    g.width = a.width;
    g.partials = reinterpret_cast<float*>(ws + l.partials);
    g.n = static_cast<uint32_t>(a.count);
    g.vocab = static_cast<uint32_t>(a.vocab);
    g.windows = l.windows;
    g.window = static_cast<uint32_t>(window_of(a.count));
    g.scale = a.scale;
    g.accumulate = a.accumulate;
    const bool vec = on16(a.d_out, a.d_out_stride, bf16 ? 2 : 4) && on16(a.d_table, a.stride, 4) &&
                     a.width % (bf16 ? 8 : 4) == 0;
    if (bf16) return vec ? launch_sums<true, true>(g, stream) : launch_sums<true, false>(g, stream);
    return vec ? launch_sums<false, true>(g, stream) : launch_sums<false, false>(g, stream);
}

}  // namespace spl
