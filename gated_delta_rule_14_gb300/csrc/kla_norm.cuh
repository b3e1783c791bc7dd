// kla_norm.cuh -- what the two forms of the layer norm's kernels share (kla_norm_rows.cu: rows of up to
// kRowsMost values; kla_norm.cu: longer ones).
#pragma once

#include "layer_dev.cuh"
#include "../../include/kla_layer.h"

namespace kla {

constexpr int kRowsMost = 512;   // longest row that a part of a warp holds
constexpr int kMaxBlock = 1024;

// CTAs of the backward pass over rows of up to kRowsMost values: a multiple of the groups, and the same for
// every width of access, so that its scratch is.
int norm_rows_bwd_grid(int64_t rows, int groups);
// `width`: values of one access, that every row start allows. part: [grid][2][n] sums of dw and db, or NULL.
cudaError_t norm_rows_fwd(const void *x, const float *w, const float *b, void *y, float *mean, float *rstd,
                          int64_t rows, int groups, int n, kla_dtype dtype, int width, float eps, cudaStream_t s);
cudaError_t norm_rows_bwd(const void *dy, const void *x, const float *w, const float *mean, const float *rstd,
                          void *dx, float *part, int64_t rows, int groups, int n, kla_dtype dtype, int width,
                          cudaStream_t s);

namespace norm {

// kV consecutive values of type T, moved in one access.
template <typename T, int kV>
__device__ __forceinline__ void load(const T *p, T *x) {
    if constexpr (sizeof(T) * kV == 16) {
        *reinterpret_cast<uint4 *>(x) = *reinterpret_cast<const uint4 *>(p);
    } else if constexpr (sizeof(T) * kV == 4) {
        *reinterpret_cast<uint32_t *>(x) = *reinterpret_cast<const uint32_t *>(p);
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) x[i] = p[i];
    }
}
template <typename T, int kV>
__device__ __forceinline__ void store(T *p, const float *x) {
    if constexpr (sizeof(T) * kV == 16) {
        uint4 r;
        T *e = reinterpret_cast<T *>(&r);
#pragma unroll
        for (int i = 0; i < kV; ++i) e[i] = from_f32<T>(x[i]);
        *reinterpret_cast<uint4 *>(p) = r;
    } else if constexpr (kV == 2) {
        uint32_t r;
        T *e = reinterpret_cast<T *>(&r);
        e[0] = from_f32<T>(x[0]);
        e[1] = from_f32<T>(x[1]);
        *reinterpret_cast<uint32_t *>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) p[i] = from_f32<T>(x[i]);
    }
}

__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); }
__device__ __forceinline__ float across(float v, int off) { return __shfl_xor_sync(0xffffffffu, v, off); }
__device__ __forceinline__ float2 across(float2 v, int off) { return make_float2(across(v.x, off), across(v.y, off)); }

// Sum over the `lanes` lanes of a row's team.
template <int kLanes, typename V>
__device__ __forceinline__ V lane_sum(V v) {
#pragma unroll
    for (int off = kLanes / 2; off; off >>= 1) v = add(v, across(v, off));
    return v;
}
// Which rows a thread's team of `width` threads walks: rows first, first + step, .. of group g.
struct Walk {
    int lane, width, g;
    int64_t first, step;
    __device__ Walk(int groups, int threads) {
        g = blockIdx.x % groups;
        width = threads;
        lane = threadIdx.x % threads;
        const int teams = blockDim.x / threads;
        first = static_cast<int64_t>(blockIdx.x / groups) * teams + threadIdx.x / threads;
        step = static_cast<int64_t>(gridDim.x / groups) * teams;
    }
};

// Sum over kWarps warps that share a named barrier; calls alternate between two buffers, so that one
// barrier a sum does.
template <int kWarps>
struct WarpsSum {
    float2 (*part)[kMaxBlock / 32];   // [2][warps of the CTA]
    int first, bar, turn;             // the team's first warp and barrier
    template <typename V>
    __device__ __forceinline__ V operator()(V v) {
        v = lane_sum<32>(v);
        V *slot = reinterpret_cast<V *>(part[turn] + first);
        if ((threadIdx.x & 31) == 0) slot[(threadIdx.x / 32) % kWarps] = v;
        ptx::named_sync(bar, 32 * kWarps);
        v = slot[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = add(v, slot[w]);
        turn ^= 1;
        return v;
    }
};
// Whether a wait of the team has given up, which its threads decide alike: one that left alone would leave the
// others at a barrier that it never reaches. A thread notes its own time-out before the barrier of the turn's
// sum and reads the team's word after it. Turns alternate between two words: a thread may be on its way through
// the next turn while another still reads, but passes that turn's barrier only with it.
struct TeamLost {
    volatile int *word;   // [2]
    __device__ void init() const { word[0] = word[1] = 0; }
    __device__ __forceinline__ void note(int turn) const { word[turn & 1] = 1; }
    __device__ __forceinline__ bool read(int turn) const { return word[turn & 1] != 0; }
};

}  // namespace norm
}  // namespace kla
