// kla_beam.cu -- beam search: selection over beams and vocabulary, and states following their beams.
//
// One pass over the logits: every CTA takes kChunk tokens of one beam and leaves that piece's
// maximum m, sum of e^{x - m} and its W best tokens in order. A beam's total is then
// sum_c s_c e^{m_c - M}, and since the score (x - M) - log(total) + score does not fall when x
// rises, the W best candidates of a request are among those lists: a second launch merges them by
// (score, lowest beam, logit, lowest token).
//
// Logits are ranked through an order-preserving map to 32-bit whole numbers (0 marks "nothing").
#include <cfloat>
#include <climits>

#include "kla_internal.cuh"
#include "../../include/kla_layer.h"

namespace kla {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kE = 16;                    // logits of one thread
constexpr int kChunk = kThreads * kE;     // tokens of one CTA
constexpr int kMaxW = 16;

// Order-preserving map of floats (no NaN) to whole numbers above 0, and back.
__device__ __forceinline__ uint32_t rank_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 counts as 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t r) {
    return __uint_as_float(r & 0x80000000u ? r & 0x7fffffffu : ~r);
}
__device__ __forceinline__ float clean(float x) {   // NaN: -inf; +inf: the largest finite value
    return x == x ? fminf(x, FLT_MAX) : -INFINITY;
}

struct BeamScratch {   // per (beam, chunk): [B * W][nchunk] and the lists [..][W]
    float *m, *s;
    uint32_t *rank;
    int *token;
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
beam_scan_kernel(const T *logits, int64_t row_stride, const unsigned char *finished, int eos, BeamScratch sc, int W,
                 int V, int nchunk) {
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
    const T *x = logits + static_cast<int64_t>(row) * row_stride;
    const int v0 = c * kChunk;
    uint32_t e[kE];
    uint32_t best = 0;
    int where = 0;
#pragma unroll
    for (int u = 0; u < kE; ++u) {
        const int v = v0 + u * kThreads + tid;
        e[u] = v < V ? rank_of(clean(to_f32(x[v]))) : 0u;
    }
    auto own_best = [&]() {   // the lowest token among equals: u ascends with the token
        best = 0;
        where = 0;
#pragma unroll
        for (int u = 0; u < kE; ++u)
            if (e[u] > best) {
                best = e[u];
                where = u;
            }
    };
    own_best();
    __shared__ uint32_t top[kWarps], lr[kWarps][kMaxW];
    __shared__ int lt[kWarps][kMaxW];
    __shared__ float part[kWarps];
    const uint32_t wm = __reduce_max_sync(0xffffffffu, best);
    if (lane == 0) top[warp] = wm;
    __syncthreads();
    uint32_t cm = top[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) cm = max(cm, top[w]);
    const float m = value_of(cm);
    float s = 0.f;
    if (m > -INFINITY) {
#pragma unroll
        for (int u = 0; u < kE; ++u)
            if (e[u]) s += expf(value_of(e[u]) - m);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if (lane == 0) part[warp] = s;
    // the warp's W best
    for (int k = 0; k < W; ++k) {
        const uint32_t r = __reduce_max_sync(0xffffffffu, best);
        const int mine = best == r ? where * kThreads + tid : INT_MAX;
        const int t = __reduce_min_sync(0xffffffffu, mine);
        if (lane == 0) {
            lr[warp][k] = r;
            lt[warp][k] = v0 + t;
        }
        if (mine == t) {
#pragma unroll
            for (int u = 0; u < kE; ++u)
                if (u == where) e[u] = 0;
            own_best();
        }
    }
    __syncthreads();
    if (warp == 0) {   // lane w < 8 walks warp w's list
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) total += part[w];
        if (lane == 0) {
            sc.m[at] = m;
            sc.s[at] = total;
        }
        int head = 0;
        for (int k = 0; k < W; ++k) {
            const uint32_t r0 = lane < kWarps && head < W ? lr[lane][head] : 0u;
            const int t0 = r0 ? lt[lane][head] : INT_MAX;
            const uint32_t r = __reduce_max_sync(0xffffffffu, r0);
            const int t = __reduce_min_sync(0xffffffffu, r0 == r ? t0 : INT_MAX);
            if (lane == 0) {
                rank[k] = r;
                token[k] = t;
            }
            if (r && r0 == r && t0 == t) ++head;
        }
    }
}

// Larger (a, b) first; the lanes' pairs differ except where there is nothing (a = 0).
struct Pair {
    unsigned long long a, b;
};
__device__ __forceinline__ Pair larger(Pair x, Pair y) { return x.a > y.a || (x.a == y.a && x.b >= y.b) ? x : y; }
__device__ __forceinline__ Pair warp_best(Pair x) {
#pragma unroll
    for (int off = 16; off; off >>= 1)
        x = larger(x, Pair{__shfl_xor_sync(0xffffffffu, x.a, off), __shfl_xor_sync(0xffffffffu, x.b, off)});
    return x;
}

// One CTA per request: totals of the beams, then W rounds of the best list head.
__global__ void __launch_bounds__(kThreads)
beam_merge_kernel(BeamScratch sc, const float *scores, const unsigned char *finished, int eos, float *new_scores,
                  int *parents, int *tokens, unsigned char *new_finished, int W, int nchunk) {
    extern __shared__ int head[];   // [W * nchunk]
    __shared__ float Ms[kMaxW], logs[kMaxW];
    __shared__ Pair best[kWarps];
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid / 32, lists = W * nchunk;
    const int64_t base = static_cast<int64_t>(b) * lists;
    for (int w = warp; w < W; w += kWarps) {
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
    for (int i = tid; i < lists; i += kThreads) head[i] = 0;
    __syncthreads();
    auto score_of = [&](int w, uint32_t r) {
        const float key = ((value_of(r) - Ms[w]) - logs[w]) + scores[b * W + w];
        return key == key ? key : -INFINITY;
    };
    for (int k = 0; k < W; ++k) {
        Pair p{0, 0};
        for (int i = tid; i < lists; i += kThreads) {
            const int h = head[i];
            if (h >= W) continue;
            const int64_t e = (base + i) * W + h;
            const uint32_t r = sc.rank[e];
            if (!r) continue;
            const int w = i / nchunk;
            const unsigned long long key = rank_of(score_of(w, r));
            p = larger(p, Pair{(key << 32) | (0xffffffffu - static_cast<uint32_t>(w)),
                               (static_cast<unsigned long long>(r) << 32) |
                                   (0xffffffffu - static_cast<uint32_t>(sc.token[e]))});
        }
        p = warp_best(p);
        if (lane == 0) best[warp] = p;
        __syncthreads();
        p = best[0];
#pragma unroll
        for (int q = 1; q < kWarps; ++q) p = larger(p, best[q]);
        const int w = static_cast<int>(0xffffffffu - static_cast<uint32_t>(p.a));
        const uint32_t r = static_cast<uint32_t>(p.b >> 32);
        const int t = static_cast<int>(0xffffffffu - static_cast<uint32_t>(p.b));
        // the list that gave it: in a beam, its token's chunk (a finished beam's is chunk 0)
        const bool done = finished && finished[b * W + w];
        if (tid == 0) {
            const int o = b * W + k;
            new_scores[o] = score_of(w, r);
            parents[o] = w;
            tokens[o] = t;
            if (new_finished) new_finished[o] = done || t == eos;
            ++head[w * nchunk + (done ? 0 : t / kChunk)];
        }
        __syncthreads();
    }
}

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

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
struct Span {
    uintptr_t lo, hi;
};
Span span(const void *p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, p ? a + bytes : a};
}
bool overlaps(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

}  // namespace
}  // namespace kla

extern "C" {

size_t kla_beam_select_workspace_size(int B, int W, int V, kla_dtype dtype) {
    (void)dtype;
    if (B < 1 || W < 1 || W > kla::kMaxW || V < 1) return 0;
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
    const int nchunk = (V + kChunk - 1) / kChunk;
    // the beams index the grid; the merge keeps one list head per (beam, chunk) in shared memory
    if (W > kMaxW || static_cast<int64_t>(B) * W > 65535 || nchunk > 512) return KLA_ERR_UNSUPPORTED;
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
    beam_merge_kernel<<<B, kThreads, W * nchunk * sizeof(int), cs>>>(sc, scores, finished, eos, new_scores, parents,
                                                                     tokens, new_finished, W, nchunk);
    return cudaGetLastError() == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
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
