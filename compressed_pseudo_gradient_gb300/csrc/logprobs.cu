// Log-probabilities of given tokens with entropy and top alternatives, and their gradient
// (spl_token_logprobs, spl_token_logprobs_grad; declared in include/spl_local.h).
//
// With z = scale * x over a row x of logits, m = max x, e_j = exp(scale (x_j - m)):
//   S = sum e_j,  W = sum e_j (x_j - m)
//   lse = scale m + log S,  logp = scale (x_t - m) - log S,  H = log S - scale W / S
// and with p_j = exp(z_j - lse), for upstream gradients g of logp and h of H:
//   dx_j = scale (g (1[j = t] - p_j) - h p_j (z_j - lse + H)).
//
// Forward: every logit is read once.  A row goes to a cluster of CTAs (one CTA when there are
// enough rows), each thread keeps (m, S, W) of its vectors, rescaled when its maximum rises,
// and the triples are joined in a fixed tree (warp, CTA, cluster through distributed shared
// memory), so a call needs no workspace and gives the same bits each run.
// Top alternatives: each warp holds its k largest, sorted, one per lane, as 64-bit keys (the
// value's ordered bits, then the complement of its index: equal values rank by lower index);
// a vector is looked at again only if its maximum beats the warp's k-th entry.
#include <cooperative_groups.h>

#include "local_device.cuh"
#include "local_kernels.h"
#include "spl_kernels.h"

namespace cg = cooperative_groups;

namespace spl {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;
constexpr int kMaxParts = 8;
constexpr unsigned kAll = 0xffffffffu;

// ---- the running softmax statistics ---------------------------------------------------------
struct Stats {
    float m;   // largest logit so far (kLowest before the first)
    float s;   // sum of exp(scale (x - m))
    float w;   // sum of exp(scale (x - m)) (x - m)
};

// The statistics relative to another, not smaller, maximum: a vanishing factor drops them (its
// product with w's shift may be 0 times infinity), and -inf - m is held at the lowest number.
__device__ __forceinline__ void rescale(Stats& a, float m, float c) {
    const float delta = fmaxf(__fsub_rn(a.m, m), kLowest);
    const float f = ex2(__fmul_rn(delta, c));
    a.w = f > 0.0f ? __fmul_rn(f, __fmaf_rn(a.s, delta, a.w)) : 0.0f;
    a.s = __fmul_rn(f, a.s);
    a.m = m;
}

__device__ __forceinline__ Stats join(Stats a, Stats b, float c) {
    const float m = max_nan(a.m, b.m);
    rescale(a, m, c);
    rescale(b, m, c);
    a.s = __fadd_rn(a.s, b.s);
    a.w = __fadd_rn(a.w, b.w);
    return a;
}

template <int kN>
__device__ __forceinline__ float vector_max(const float (&x)[kN]) {
    float v = x[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) v = max_nan(v, x[i]);
    return v;
}

// Adds kN logits with the given maximum.  A masked logit (-inf, or one so low that the
// difference overflows) has e = 0 and adds nothing to either sum.
template <int kN>
__device__ __forceinline__ void add_values(Stats& a, const float (&x)[kN], float vmax, float c) {
    if (!(vmax <= a.m)) rescale(a, max_nan(vmax, a.m), c);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const float d = fmaxf(__fsub_rn(x[i], a.m), kLowest);
        const float e = ex2(__fmul_rn(d, c));
        a.s = __fadd_rn(a.s, e);
        a.w = __fmaf_rn(e, d, a.w);
    }
}

// ---- sorted lists of the largest ------------------------------------------------------------
__device__ __forceinline__ uint64_t rank_key(float x, uint32_t index) {
    const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));   // -0 ranks with +0
    const uint32_t hi = x != x ? 0xffffffffu : (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return (static_cast<uint64_t>(hi) << 32) | (0xffffffffu - index);
}

__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t hi = static_cast<uint32_t>(key >> 32);
    return __uint_as_float((hi & 0x80000000u) ? (hi == 0xffffffffu ? 0x7fc00000u : hi & 0x7fffffffu)
                                              : ~hi);
}

// A warp's list: lane l holds the l-th largest key so far (0: none yet).  `floor` is the value
// of entry k - 1; while there is none it is NaN, which no value is <= to.
struct TopList {
    uint64_t key;
    float floor;
};

__device__ __forceinline__ void top_insert(TopList& t, uint64_t key, int lane, int k) {
    const int at = __popc(__ballot_sync(kAll, t.key > key));
    const uint64_t up = __shfl_up_sync(kAll, t.key, 1);
    if (lane == at) t.key = key;
    if (lane > at) t.key = up;
    const uint64_t last = __shfl_sync(kAll, t.key, k - 1);
    t.floor = last == 0 ? __uint_as_float(0x7fc00000u) : key_value(last);
}

// Offers each lane's values (indices first, first + 1, ...) to the warp's list.  Called by all
// lanes; lanes without a vector pass ok = false.
template <int kN>
__device__ __noinline__ void top_offer(TopList& t, const float (&x)[kN], bool ok, uint32_t first,
                                       int lane, int k) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        // equal values are offered too: their keys decide (vectors interleave over the lanes)
        unsigned want = __ballot_sync(kAll, ok && !(x[i] < t.floor));
        while (want != 0) {
            const int src = __ffs(want) - 1;
            const float v = __shfl_sync(kAll, x[i], src);
            const uint32_t idx = __shfl_sync(kAll, first, src) + i;
            top_insert(t, rank_key(v, idx), lane, k);
            want &= want - 1;
            want &= __ballot_sync(kAll, ok && !(x[i] < t.floor));
        }
    }
}

// The 32 largest of two descending lists, descending: the larger of each entry and its mirror
// is a bitonic sequence of the 32 largest, sorted by five exchanges.
__device__ __forceinline__ uint64_t top_merge(uint64_t a, uint64_t b, int lane) {
    const uint64_t r = __shfl_sync(kAll, b, 31 - lane);
    uint64_t k = a > r ? a : r;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const uint64_t o = __shfl_xor_sync(kAll, k, off);
        k = ((lane & off) == 0) == (k > o) ? k : o;
    }
    return k;
}

// Bound: HBM.  Two CTAs of 512 threads per SM, four 16-byte loads in flight per thread.
template <bool kBf16, bool kTop>
__global__ void __launch_bounds__(kThreads, 2) k_logprobs(const __grid_constant__ LogprobsArgs a,
                                                          int parts) {
    using V = Vec16<kBf16>;
    constexpr int kN = V::kN;
    __shared__ Stats s_stats[kWarps];
    __shared__ uint64_t s_top[kTop ? kWarps : 1][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / parts;
    const int part = static_cast<int>(blockIdx.x % parts);
    const unsigned char* base =
        static_cast<const unsigned char*>(a.logits) + row * a.stride * V::kBytes;
    const RowSplit sp = split_row<kBf16>(base, a.vocab);
    const uint4* vecs = reinterpret_cast<const uint4*>(base + sp.head * V::kBytes);
    const int64_t begin = sp.vecs * part / parts, end = sp.vecs * (part + 1) / parts;
    const float c = __fmul_rn(a.scale, kLog2e);
    const float ninf = __uint_as_float(0xff800000u);

    Stats st = {kLowest, 0.0f, 0.0f};
    TopList top = {0, __uint_as_float(0x7fc00000u)};

    // one value per thread from index `first` on: the ends of a row around its whole vectors
    auto scalars = [&](int64_t first, int count) {
        const bool ok = tid < count && SPL_CHECK(first + tid < a.vocab, kSiteLogits, first + tid);
        const float x[1] = {ok ? V::load1(base, first + tid) : ninf};
        if (ok) add_values<1>(st, x, x[0], c);
        if constexpr (kTop)
            if (warp == 0) top_offer<1>(top, x, ok, static_cast<uint32_t>(first + tid), lane, a.top);
    };

    if (part == 0 && sp.head > 0) scalars(0, sp.head);
    for (int64_t b = begin; b < end; b += kThreads * kUnroll) {
        uint4 raw[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t v = b + u * kThreads + tid;
            const uint32_t fill = kBf16 ? 0xff80ff80u : 0xff800000u;   // -inf
            raw[u] = make_uint4(fill, fill, fill, fill);
            if (v < end && SPL_CHECK(sp.head + (v + 1) * kN <= a.vocab, kSiteLogits, v))
                raw[u] = __ldcs(vecs + v);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            float x[kN];
            V::unpack(raw[u], x);
            const float vmax = vector_max(x);
            if constexpr (kTop) {
                const int64_t v = b + u * kThreads + tid;
                const bool ok = v < end;
                if (__any_sync(kAll, ok && !(vmax <= top.floor)))
                    top_offer<kN>(top, x, ok, static_cast<uint32_t>(sp.head + v * kN), lane, a.top);
            }
            add_values<kN>(st, x, vmax, c);
        }
    }
    if (part == parts - 1) {
        const int64_t done = sp.head + sp.vecs * kN;
        if (done < a.vocab) scalars(done, static_cast<int>(a.vocab - done));
    }

    // join: warp, CTA
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        Stats o;
        o.m = __shfl_xor_sync(kAll, st.m, off);
        o.s = __shfl_xor_sync(kAll, st.s, off);
        o.w = __shfl_xor_sync(kAll, st.w, off);
        st = join(st, o, c);
    }
    if (lane == 0) s_stats[warp] = st;
    if constexpr (kTop) s_top[warp][lane] = top.key;
    __syncthreads();
    if constexpr (kTop) {
        for (int half = kWarps / 2; half > 0; half >>= 1) {
            if (warp < half) s_top[warp][lane] = top_merge(s_top[warp][lane], s_top[warp + half][lane], lane);
            __syncthreads();
        }
    }
    if (warp == 0) {
        st = lane < kWarps ? s_stats[lane] : Stats{kLowest, 0.0f, 0.0f};
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            Stats o;
            o.m = __shfl_xor_sync(kAll, st.m, off);
            o.s = __shfl_xor_sync(kAll, st.s, off);
            o.w = __shfl_xor_sync(kAll, st.w, off);
            st = join(st, o, c);
        }
    }
    if (parts > 1) {   // join the cluster's CTAs in the first one
        cg::cluster_group cluster = cg::this_cluster();
        if (tid == 0) s_stats[0] = st;
        cluster.sync();
        if (part == 0 && warp == 0) {
            st = Stats{kLowest, 0.0f, 0.0f};
            if (lane < parts) st = *cluster.map_shared_rank(&s_stats[0], lane);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                Stats o;
                o.m = __shfl_xor_sync(kAll, st.m, off);
                o.s = __shfl_xor_sync(kAll, st.s, off);
                o.w = __shfl_xor_sync(kAll, st.w, off);
                st = join(st, o, c);
            }
            if constexpr (kTop) {
                uint64_t k = s_top[0][lane];
                for (int p = 1; p < parts; ++p)
                    k = top_merge(k, *cluster.map_shared_rank(&s_top[0][lane], p), lane);
                s_top[0][lane] = k;
            }
        }
        cluster.sync();   // the other CTAs' shared memory has been read
    }
    if (part != 0 || warp != 0) return;

    const bool broken = !(fabsf(st.m) <= 3.402823466e+38f);   // NaN or infinite maximum
    const bool empty = !broken && st.s == 0.0f;               // every logit is -inf
    const float nan = __uint_as_float(0x7fc00000u);
    const float peak = __fmul_rn(st.m, a.scale);
    const float log_s = logf(st.s);
    auto logprob = [&](float x) {
        if (broken) return nan;
        if (empty) return ninf;
        return __fsub_rn(__fmul_rn(__fsub_rn(x, st.m), a.scale), log_s);
    };
    if (lane == 0) {
        if (a.lse != nullptr)
            a.lse[row] = broken ? nan : empty ? ninf : __fadd_rn(peak, log_s);
        if (a.entropy != nullptr)
            a.entropy[row] = broken ? nan
                             : empty ? 0.0f
                                     : __fsub_rn(log_s, __fdiv_rn(__fmul_rn(a.scale, st.w), st.s));
        if (a.targets.data != nullptr) {
            const int64_t t = token_at(a.targets, row);
            float lp = 0.0f;   // a negative target is outside the loss
            if (t >= a.vocab) {
                lp = nan;
                if (a.flags != nullptr) atomicOr(a.flags, kFlagBadToken);
            } else if (t >= 0 && SPL_CHECK(t < a.vocab, kSiteLogits, t)) {
                lp = logprob(V::load1(base, t));
            }
            a.logp[row] = lp;
        }
        if (broken && a.flags != nullptr) atomicOr(a.flags, kFlagNonFinite);
    }
    if constexpr (kTop) {
        if (lane < a.top && SPL_CHECK(row < a.rows, kSiteTop, row)) {
            const uint64_t k = s_top[0][lane];
            a.top_ids[row * a.top + lane] =
                static_cast<int64_t>(0xffffffffu - static_cast<uint32_t>(k));
            a.top_logp[row * a.top + lane] = logprob(key_value(k));
        }
    }
}

// ---- gradient -------------------------------------------------------------------------------
// Bound: HBM, every logit read once and every gradient written once.  A CTA takes kGradVecs
// vectors of a row per thread; rows whose input and output sit differently within 16 bytes are
// taken value by value.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;

struct GradRow {
    float scale, lse, g, h, entropy;
    int64_t target;   // -1: none
    bool empty;
};

template <bool kEntropy>
__device__ __forceinline__ float grad_value(float x, const GradRow& r) {
    const float d = __fsub_rn(__fmul_rn(x, r.scale), r.lse);
    const float p = ex2(__fmul_rn(d, kLog2e));
    float v = -__fmul_rn(p, r.g);
    if constexpr (kEntropy)   // p = 0: nothing (d may be -inf)
        if (p > 0.0f) v = __fsub_rn(v, __fmul_rn(__fmul_rn(r.h, p), __fadd_rn(d, r.entropy)));
    return v;
}

template <bool kBf16, bool kEntropy>
__global__ void __launch_bounds__(kGradThreads)
k_logprobs_grad(const __grid_constant__ LogprobsGradArgs a, int parts, bool vectors) {
    using V = Vec16<kBf16>;
    constexpr int kN = V::kN;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / parts;
    const int part = static_cast<int>(blockIdx.x % parts);
    const unsigned char* in = static_cast<const unsigned char*>(a.logits) + row * a.stride * V::kBytes;
    unsigned char* out = static_cast<unsigned char*>(a.out) + row * a.out_stride * V::kBytes;

    const RowSplit sp = split_row<kBf16>(in, a.vocab);
    const uint4* src = reinterpret_cast<const uint4*>(in + sp.head * V::kBytes);
    const int64_t b = static_cast<int64_t>(part) * kGradThreads * kGradVecs + tid;
    uint4 raw[kGradVecs];
    if (vectors) {
#pragma unroll
        for (int u = 0; u < kGradVecs; ++u) {
            const int64_t v = b + u * kGradThreads;
            if (v < sp.vecs) raw[u] = __ldcs(src + v);
        }
    }

    GradRow r;
    r.scale = a.scale;
    r.lse = a.lse[row];
    r.target = a.targets.data != nullptr ? token_at(a.targets, row) : -1;
    if (r.target >= a.vocab) {
        if (part == 0 && tid == 0 && a.flags != nullptr) atomicOr(a.flags, kFlagBadToken);
        r.target = -1;
    }
    r.g = r.target >= 0 && a.d_logp != nullptr ? a.d_logp[row] : 0.0f;
    r.h = kEntropy ? a.d_entropy[row] : 0.0f;
    r.entropy = kEntropy ? a.entropy[row] : 0.0f;
    r.empty = r.lse == __uint_as_float(0xff800000u);

    auto value = [&](float x, int64_t j) {
        if (r.empty) return 0.0f;
        float v = grad_value<kEntropy>(x, r);
        if (j == r.target) v = __fadd_rn(v, r.g);
        return __fmul_rn(v, r.scale);
    };

    if (!vectors) {
        for (int64_t j = static_cast<int64_t>(part) * kGradThreads + tid; j < a.vocab;
             j += static_cast<int64_t>(parts) * kGradThreads) {
            if (!SPL_CHECK(j < a.vocab, kSiteLogitsOut, j)) continue;
            V::store1(out, j, value(V::load1(in, j), j));
        }
        return;
    }
    uint4* dst = reinterpret_cast<uint4*>(out + sp.head * V::kBytes);
#pragma unroll
    for (int u = 0; u < kGradVecs; ++u) {
        const int64_t v = b + u * kGradThreads;
        if (v >= sp.vecs || !SPL_CHECK(sp.head + (v + 1) * kN <= a.vocab, kSiteLogitsOut, v)) continue;
        float x[kN];
        V::unpack(raw[u], x);
        const int64_t first = sp.head + v * kN;
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = value(x[i], first + i);
        __stcs(dst + v, V::pack(x));
    }
    if (part == 0) {   // the ends around the whole vectors
        const int64_t done = sp.head + sp.vecs * kN;
        const int ends = sp.head + static_cast<int>(a.vocab - done);
        if (tid < ends) {
            const int64_t j = tid < sp.head ? tid : done + (tid - sp.head);
            V::store1(out, j, value(V::load1(in, j), j));
        }
    }
}

template <bool kBf16, bool kTop>
cudaError_t launch_forward(const LogprobsArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    int parts = 1;
    while (parts < kMaxParts && a.rows * parts < 2 * sms && a.vocab / (2 * parts) >= 2048) parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(parts);
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_logprobs<kBf16, kTop>, a, parts);
}

template <bool kBf16, bool kEntropy>
cudaError_t launch_backward(const LogprobsGradArgs& a, cudaStream_t stream) {
    using V = Vec16<kBf16>;
    const uintptr_t in = reinterpret_cast<uintptr_t>(a.logits), out = reinterpret_cast<uintptr_t>(a.out);
    const bool vectors = (in - out) % 16 == 0 && ((a.stride - a.out_stride) * V::kBytes) % 16 == 0;
    const int64_t per_part = static_cast<int64_t>(kGradThreads) * kGradVecs;
    const int64_t parts = (a.vocab / V::kN + per_part) / per_part;
    const unsigned grid = static_cast<unsigned>(a.rows * parts);
    k_logprobs_grad<kBf16, kEntropy><<<grid, kGradThreads, 0, stream>>>(a, static_cast<int>(parts),
                                                                        vectors);
    return cudaGetLastError();
}

}  // namespace

#if SPL_CHECKED
SPL_DEBUG_READER(debug_read_logprobs)
#endif

cudaError_t launch_logprobs(const LogprobsArgs& a, bool bf16, cudaStream_t stream) {
    if (bf16) return a.top > 0 ? launch_forward<true, true>(a, stream) : launch_forward<true, false>(a, stream);
    return a.top > 0 ? launch_forward<false, true>(a, stream) : launch_forward<false, false>(a, stream);
}

cudaError_t launch_logprobs_grad(const LogprobsGradArgs& a, bool bf16, cudaStream_t stream) {
    const bool h = a.d_entropy != nullptr;
    if (bf16) return h ? launch_backward<true, true>(a, stream) : launch_backward<true, false>(a, stream);
    return h ? launch_backward<false, true>(a, stream) : launch_backward<false, false>(a, stream);
}

}  // namespace spl
