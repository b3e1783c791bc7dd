// kla_beam.cu -- beam search: selection over beams and vocabulary, and states following their beams.
//
// One pass over the logits: every CTA takes kChunk tokens of one beam and leaves that piece's
// maximum m, sum of e^{x - m} and its W best tokens in order. A beam's total is then
// sum_c s_c e^{m_c - M}, and since the score (x - M) - log(total) + score does not fall when x
// rises, the W best candidates of a request are among those lists: a second launch merges them by
// (score, lowest beam, logit, lowest token).
//
// Both launches pick the W best of many in the same way. The W-th best of the warps' best lanes (of eight
// warps: best and second best) is a threshold that W values or more reach, and not many more. They are
// gathered in shared memory and each counts those ahead of it, which is its place.
// Only where more reach the threshold than fit (long runs of equal values) the W best are taken one
// after the other. Taking them so everywhere cost 22.6 us for 64 rows of 100003 fp32 logits.
//
// Measured with cold caches, 8 requests of 8 such beams: 13 us for the pass (26 MB, 29 % of a copy's rate; bound by
// the latency of its loads and of the pieces' barriers, 2.1 of 4 instructions issued a cycle) and 9 us for the merge
// (eight CTAs, one after the other dependent steps behind barriers), whose launch overlaps the pass; 15 to 18 us
// together.
//
// Logits are ranked through an order-preserving map to 32-bit whole numbers (0 marks "nothing").
#include <cfloat>
#include <climits>

#include "layer_dev.cuh"
#include "../../include/kla_layer.h"

namespace kla {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kE = 16;                    // logits of one thread
constexpr int kChunk = kThreads * kE;     // tokens of one CTA
constexpr int kMaxW = 16;
constexpr int kMostV = 512 * kChunk;      // the merge numbers its entries in 32 bits

// Order-preserving map of floats (no NaN) to whole numbers above 0, and back.
__device__ __forceinline__ uint32_t rank_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t r) {
    return __uint_as_float(r & 0x80000000u ? r & 0x7fffffffu : ~r);
}
__device__ __forceinline__ float clean(float x) {   // NaN: -inf; +inf: the largest finite value
    return fminf(fmaxf(x, -INFINITY), FLT_MAX);
}

struct BeamScratch {   // per (beam, chunk): [B * W][nchunk] and the lists [..][W]
    float *m, *s;
    uint32_t *rank;
    int *token;
};

// Larger (a, b) first; pairs differ except where there is nothing (a = 0).
struct Pair {
    unsigned long long a, b;
};
__device__ __forceinline__ bool ahead(Pair x, Pair y) { return x.a > y.a || (x.a == y.a && x.b > y.b); }
__device__ __forceinline__ Pair larger(Pair x, Pair y) { return ahead(y, x) ? y : x; }
__device__ __forceinline__ Pair warp_best(Pair x) {
#pragma unroll
    for (int off = 16; off; off >>= 1)
        x = larger(x, Pair{__shfl_xor_sync(0xffffffffu, x.a, off), __shfl_xor_sync(0xffffffffu, x.b, off)});
    return x;
}

// The best value of the CTA, and a threshold that W <= 16 values or more reach: the W-th of its 32 warps'
// best lanes, or of 8 warps' best and second best (0 where there are fewer). One barrier.
template <int kCount>
__device__ __forceinline__ void thresholds(uint32_t mine, int W, uint32_t (&slot)[32], uint32_t &low, uint32_t &high) {
    static_assert(kCount == 32 || kCount == 8, "warps of the CTA");
    constexpr int kPer = kCount == 32 ? 1 : 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const uint32_t best = __reduce_max_sync(0xffffffffu, mine);
    uint32_t second = 0;
    if (kPer == 2) {
        const unsigned who = __ballot_sync(0xffffffffu, mine == best);
        second = __reduce_max_sync(0xffffffffu, lane == __ffs(who) - 1 ? 0u : mine);
    }
    if (lane < kPer) slot[warp * kPer + lane] = lane ? second : best;
    __syncthreads();
    const uint32_t v = lane < kPer * kCount ? slot[lane] : 0u;
    int ahead_of = 0;
#pragma unroll
    for (int k = 0; k < kPer * kCount; ++k) {
        const uint32_t o = __shfl_sync(0xffffffffu, v, k);
        ahead_of += o > v || (o == v && k < lane);
    }
    const unsigned at = __ballot_sync(0xffffffffu, lane < kPer * kCount && ahead_of == W - 1);
    low = __shfl_sync(0xffffffffu, v, __ffs(at) - 1);
    high = __reduce_max_sync(0xffffffffu, v);
}

constexpr int kGather = 256;   // values at or above the threshold that are ranked at once

template <typename T>
__global__ void __launch_bounds__(kThreads)
beam_scan_kernel(const T *logits, int64_t row_stride, const unsigned char *finished, int eos, BeamScratch sc, int W,
                 int V, int nchunk) {
    dependency_release();
    const int c = blockIdx.x, row = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int64_t at = static_cast<int64_t>(row) * nchunk + c;
    uint32_t *rank = sc.rank + at * W;
    int *token = sc.token + at * W;
    if (finished && finished[row]) {   // eos alone, at no cost; then the lowest other tokens
        if (tid < W) {
            uint32_t r = 0;
            int t = 0;
            if (c == 0) {
                t = tid == 0 ? eos : tid - 1 + (tid - 1 >= eos);
                r = tid == 0 ? rank_of(0.f) : t < V ? rank_of(-INFINITY) : 0;
            }
            rank[tid] = r;
            token[tid] = t;
        }
        if (tid == 0) {
            sc.m[at] = c == 0 ? 0.f : -INFINITY;
            sc.s[at] = c == 0 ? 1.f : 0.f;
        }
        return;
    }
    __shared__ uint32_t slot[32];
    __shared__ unsigned long long got[kGather];
    __shared__ float part[kWarps];
    __shared__ int count;
    if (tid == 0) count = 0;
    const T *x = logits + static_cast<int64_t>(row) * row_stride;   // V < 2^31: tokens in 32 bits
    const int first = c * kChunk + tid, left = V - first;   // this thread's tokens are first, first + kThreads, ..
    // sixteen loads on their way at once, of the last token where there is none (a condition on each had them
    // wait for one another: 31 us for 64 rows of 100003 fp32 logits)
    const bool whole = c * kChunk + kChunk <= V;
    T raw[kE];
    float e[kE];
    if (whole) {
#pragma unroll
        for (int u = 0; u < kE; ++u) raw[u] = x[first + u * kThreads];
#pragma unroll
        for (int u = 0; u < kE; ++u) e[u] = clean(to_f32(raw[u]));
    } else {
#pragma unroll
        for (int u = 0; u < kE; ++u) raw[u] = x[min(first + u * kThreads, V - 1)];
#pragma unroll
        for (int u = 0; u < kE; ++u) e[u] = u * kThreads < left ? clean(to_f32(raw[u])) : -INFINITY;
    }
    float own = e[0];
#pragma unroll
    for (int u = 1; u < kE; ++u) own = fmaxf(own, e[u]);
    uint32_t low, high;
    thresholds<kWarps>(left > 0 ? rank_of(own) : 0u, W, slot, low, high);
    const float m = value_of(high), from = low ? value_of(low) : -INFINITY;
    float s = 0.f;
    if (m > -INFINITY) {
#pragma unroll
        // e^(x - m), x - m rounded once; its error in units of the last place grows with m - x, as the term falls
        for (int u = 0; u < kE; ++u) s += __expf(e[u] - m);   // nothing: e^-inf
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) part[warp] = s;
    if (own >= from) {
#pragma unroll
        for (int u = 0; u < kE; ++u)
            if (e[u] >= from && u * kThreads < left) {
                const int k = atomicAdd(&count, 1);   // any order: places go by value and token
                if (k < kGather)
                    got[k] = (static_cast<unsigned long long>(rank_of(e[u])) << 32) |
                             (0xffffffffu - static_cast<uint32_t>(c * kChunk + u * kThreads + tid));
            }
    }
    __syncthreads();
    if (tid == 0) {
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += part[w];
        sc.m[at] = m;
        sc.s[at] = total;
    }
    const int n = count;
    if (n <= kGather) {
        if (tid < n) {
            const unsigned long long mine = got[tid];
            int place = 0;
            for (int k = 0; k < n; ++k) place += got[k] > mine;
            if (place < W) {
                rank[place] = static_cast<uint32_t>(mine >> 32);
                token[place] = static_cast<int>(0xffffffffu - static_cast<uint32_t>(mine));
            }
        }
        if (tid >= n && tid < W) rank[tid] = 0u;   // fewer than W tokens
        return;
    }
    // long runs of equal values: one after the other, the lowest token among equals
    unsigned taken = 0;   // of this thread's
    for (int k = 0; k < W; ++k) {
        unsigned long long mine = 0;
#pragma unroll
        for (int u = kE - 1; u >= 0; --u)
            if (u * kThreads < left && !(taken >> u & 1)) {
                const unsigned long long v = (static_cast<unsigned long long>(rank_of(e[u])) << 32) |
                                             (0xffffffffu - static_cast<uint32_t>(c * kChunk + u * kThreads + tid));
                mine = v > mine ? v : mine;
            }
        unsigned long long best = mine;
#pragma unroll
        for (int off = 16; off; off >>= 1) {
            const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, off);
            best = o > best ? o : best;
        }
        if (lane == 0) got[warp] = best;
        __syncthreads();
        best = got[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) best = got[w] > best ? got[w] : best;
        const int t = static_cast<int>(0xffffffffu - static_cast<uint32_t>(best));
        if (best && mine == best) taken |= 1u << ((t - c * kChunk) / kThreads);
        if (tid == 0) {
            rank[k] = static_cast<uint32_t>(best >> 32);
            token[k] = t;
        }
        __syncthreads();
    }
}

// One CTA per request: totals of the beams, then the W best of the lists' entries.
constexpr int kMerge = 1024;   // threads: 8192 entries are on their way at once

__global__ void __launch_bounds__(kMerge)
beam_merge_kernel(BeamScratch sc, const float *scores, const unsigned char *finished, int eos, float *new_scores,
                  int *parents, int *tokens, unsigned char *new_finished, int W, int nchunk) {
    __shared__ float Ms[kMaxW], logs[kMaxW], given[kMaxW];
    __shared__ uint32_t slot[32];
    __shared__ Pair got[kGather];
    __shared__ int count;
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int entries = W * nchunk * W;
    const int64_t base = static_cast<int64_t>(b) * W * nchunk;
    constexpr int kFirst = 8;   // entries of a thread that are on their way from the start
    uint32_t first[kFirst];
    if (tid == 0) count = 0;
    if (tid < W) given[tid] = scores[b * W + tid];
    dependency_wait();
#pragma unroll
    for (int u = 0; u < kFirst; ++u) first[u] = sc.rank[base * W + min(tid + u * kMerge, entries - 1)];
    for (int w = warp; w < W; w += kMerge / 32) {
        const float *m = sc.m + base + w * nchunk, *s = sc.s + base + w * nchunk;
        float M = -INFINITY, t = 0.f;
        for (int c = lane; c < nchunk; c += 32) M = fmaxf(M, m[c]);
#pragma unroll
        for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        for (int c = lane; c < nchunk; c += 32)
            if (m[c] > -INFINITY) t = fmaf(s[c], expf(m[c] - M), t);
#pragma unroll
        for (int off = 16; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
        if (lane == 0) {
            Ms[w] = M;
            logs[w] = logf(t);
        }
    }
    __syncthreads();
    auto score_of = [&](int w, uint32_t r) {
        const float key = ((value_of(r) - Ms[w]) - logs[w]) + given[w];
        return key == key ? key : -INFINITY;
    };
    const int per_beam = nchunk * W;
    auto key_of = [&](int i, uint32_t r) { return r ? rank_of(score_of(i / per_beam, r)) : 0u; };
    auto entry = [&](int i) {   // (score, lowest beam), (logit, lowest token); a = 0: nothing
        const uint32_t r = sc.rank[base * W + i];
        if (!r) return Pair{0, 0};
        const int w = i / per_beam;
        return Pair{(static_cast<unsigned long long>(rank_of(score_of(w, r))) << 32) | (0xffffffffu - w),
                    (static_cast<unsigned long long>(r) << 32) |
                        (0xffffffffu - static_cast<uint32_t>(sc.token[base * W + i]))};
    };
    auto put = [&](int k, Pair p) {
        const int w = static_cast<int>(0xffffffffu - static_cast<uint32_t>(p.a)), o = b * W + k;
        const int t = static_cast<int>(0xffffffffu - static_cast<uint32_t>(p.b));
        new_scores[o] = score_of(w, static_cast<uint32_t>(p.b >> 32));
        parents[o] = w;
        tokens[o] = t;
        if (new_finished) new_finished[o] = (finished && finished[b * W + w]) || t == eos;
    };
    uint32_t own = 0;
#pragma unroll
    for (int u = 0; u < kFirst; ++u) {
        const int i = tid + u * kMerge;
        first[u] = i < entries ? key_of(i, first[u]) : 0u;
        own = max(own, first[u]);
    }
    for (int i = tid + kFirst * kMerge; i < entries; i += kMerge)
        own = max(own, key_of(i, sc.rank[base * W + i]));
    uint32_t low, high;
    thresholds<kMerge / 32>(own, W, slot, low, high);
    auto gather = [&](int i, uint32_t key) {
        if (key && key >= low) {
            const int k = atomicAdd(&count, 1);
            if (k < kGather) got[k] = entry(i);
        }
    };
#pragma unroll
    for (int u = 0; u < kFirst; ++u) gather(tid + u * kMerge, first[u]);
    for (int i = tid + kFirst * kMerge; i < entries; i += kMerge) gather(i, key_of(i, sc.rank[base * W + i]));
    __syncthreads();
    const int n = count;
    if (n <= kGather) {
        if (tid < n) {
            const Pair mine = got[tid];
            int place = 0;
            for (int k = 0; k < n; ++k) place += ahead(got[k], mine);
            if (place < W) put(place, mine);
        }
        return;
    }
    // one after the other: the best of what lies behind the last one taken
    Pair last{~0ull, ~0ull};
    for (int k = 0; k < W; ++k) {
        Pair p{0, 0};
        for (int i = tid; i < entries; i += kMerge) {
            const Pair q = entry(i);
            if (q.a && ahead(last, q)) p = larger(p, q);
        }
        p = warp_best(p);
        if (lane == 0) got[warp] = p;
        __syncthreads();
        p = got[0];
#pragma unroll
        for (int w = 1; w < kMerge / 32; ++w) p = larger(p, got[w]);
        last = p;
        if (tid == 0) put(k, p);
        __syncthreads();
    }
}

// A copy through an index, bound by the memory: 64 beams of 8 MB, of which 42 are read, 132 us (6.8 TB/s).
constexpr int kCopy = 4;   // 16-byte words of one thread and turn

__global__ void __launch_bounds__(kThreads) reorder_kernel(const uint4 *S, const int *parents, uint4 *out, int W,
                                                           int64_t words) {
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kCopy) + threadIdx.x;
    const int row = blockIdx.y, from = parents[row];
    const bool live = from >= 0 && from < W;
    const uint4 *src = S + (static_cast<int64_t>(row / W) * W + (live ? from : 0)) * words;
    uint4 v[kCopy];
#pragma unroll
    for (int u = 0; u < kCopy; ++u) {
        const int64_t i = i0 + u * kThreads;
        v[u] = make_uint4(0, 0, 0, 0);
        if (live && i < words) v[u] = src[i];
    }
#pragma unroll
    for (int u = 0; u < kCopy; ++u) {
        const int64_t i = i0 + u * kThreads;
        if (i < words) out[static_cast<int64_t>(row) * words + i] = v[u];
    }
}

}  // namespace
}  // namespace kla

extern "C" {

size_t kla_beam_select_workspace_size(int B, int W, int V, kla_dtype dtype) {
    (void)dtype;
    if (B < 1 || W < 1 || W > kla::kMaxW || V < 1 || V > kla::kMostV) return 0;
    const size_t pieces = static_cast<size_t>(B) * W * ((V + kla::kChunk - 1) / kla::kChunk);
    return pieces * (2 + 2 * static_cast<size_t>(W)) * 4;
}

kla_status kla_beam_select(const void *logits, int64_t row_stride, const float *scores, const unsigned char *finished,
                           int eos, float *new_scores, int *parents, int *tokens, unsigned char *new_finished, int B,
                           int W, int V, kla_dtype dtype, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace kla;
    if (!logits || !scores || !new_scores || !parents || !tokens || !workspace) return KLA_ERR_INVALID_ARG;
    if (B < 1 || W < 1 || V < 1 || row_stride < V) return KLA_ERR_INVALID_ARG;
    if (dtype != KLA_DTYPE_F32 && dtype != KLA_DTYPE_BF16) return KLA_ERR_INVALID_ARG;
    if (eos < -1 || eos >= V || (finished && eos < 0)) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(logits, esz) || !aligned(scores, 4) || !aligned(new_scores, 4) || !aligned(parents, 4) ||
        !aligned(tokens, 4) || !aligned(workspace, 16))
        return KLA_ERR_INVALID_ARG;
    // the beams index the grid
    if (W > kMaxW || static_cast<int64_t>(B) * W > 65535 || V > kMostV) return KLA_ERR_UNSUPPORTED;
    const int nchunk = (V + kChunk - 1) / kChunk;
    const size_t need = kla_beam_select_workspace_size(B, W, V, dtype);
    if (workspace_bytes < need) return KLA_ERR_INVALID_ARG;
    const size_t n = static_cast<size_t>(B) * W;
    const Span outs[] = {span(new_scores, 4 * n), span(parents, 4 * n), span(tokens, 4 * n), span(new_finished, n),
                         span(workspace, need)};
    const Span ins[] = {span(logits, ((n - 1) * row_stride + V) * esz), span(scores, 4 * n), span(finished, n)};
    for (int i = 0; i < 5; ++i) {
        for (const Span &x : ins)
            if (overlaps(outs[i], x)) return KLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 5; ++j)
            if (overlaps(outs[i], outs[j])) return KLA_ERR_INVALID_ARG;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const size_t pieces = n * nchunk;
    BeamScratch sc;
    sc.m = static_cast<float *>(workspace);
    sc.s = sc.m + pieces;
    sc.rank = reinterpret_cast<uint32_t *>(sc.s + pieces);
    sc.token = reinterpret_cast<int *>(sc.rank + pieces * W);
    const dim3 grid(nchunk, static_cast<unsigned>(n));
    if (dtype == KLA_DTYPE_BF16)
        beam_scan_kernel<<<grid, kThreads, 0, cs>>>(static_cast<const __nv_bfloat16 *>(logits), row_stride, finished,
                                                    eos, sc, W, V, nchunk);
    else
        beam_scan_kernel<<<grid, kThreads, 0, cs>>>(static_cast<const float *>(logits), row_stride, finished, eos, sc,
                                                    W, V, nchunk);
    if (cudaGetLastError() != cudaSuccess) return KLA_ERR_CUDA;
    return launch_dependent(beam_merge_kernel, B, kMerge, 0, cs, sc, scores, finished, eos, new_scores, parents,
                            tokens, new_finished, W, nchunk) == cudaSuccess
               ? KLA_OK
               : KLA_ERR_CUDA;
}

kla_status kla_reorder_states(const void *S, const int *parents, void *out, int B, int W, size_t bytes, void *stream) {
    using namespace kla;
    if (!S || !parents || !out || B < 1 || W < 1 || bytes == 0 || bytes % 16) return KLA_ERR_INVALID_ARG;
    if (!aligned(S, 16) || !aligned(out, 16) || !aligned(parents, 4)) return KLA_ERR_INVALID_ARG;
    const size_t n = static_cast<size_t>(B) * W;
    if (overlaps(span(out, n * bytes), span(S, n * bytes)) || overlaps(span(out, n * bytes), span(parents, 4 * n)))
        return KLA_ERR_INVALID_ARG;
    const size_t words = bytes / 16, ctas = (words + kThreads * kCopy - 1) / (kThreads * kCopy);
    if (n > 65535 || ctas > INT_MAX) return KLA_ERR_UNSUPPORTED;
    reorder_kernel<<<dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(n)), kThreads, 0,
                     static_cast<cudaStream_t>(stream)>>>(static_cast<const uint4 *>(S), parents,
                                                          static_cast<uint4 *>(out), W, static_cast<int64_t>(words));
    return cudaGetLastError() == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // extern "C"
