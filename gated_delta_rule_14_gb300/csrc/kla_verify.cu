// kla_verify.cu -- verification of drafted tokens: which of them the target accepts, and the token after those.
//
// Comparisons are exact: u q of two 24-bit numbers fits the 53 bits of a double. Running sums are held to 2^-39 of the
// whole or better, so that a token's border is off by far less than what lies between two values of a 24-bit random
// number; sums in fp32 over 100000 tokens would move borders by whole tokens. The SM adds doubles at a 64th of the rate
// of floats, so 16 weights at a time are added as pairs of floats, a sum and what it has lost, and only those join as
// doubles. What 16 weights of sum S lose is 16 x 2^-24 S at most, each addition to it rounds by 2^-24 of that, and 16
// of them make 2^-40 S.
// Measured: 64 sequences of 8 drafts, 100003 tokens fp32, 25 us in a row of calls (floor 7.5), bf16 25 (3.8), 100000 tokens,
// whose rows fit 16 bytes, 23 either way; one of 4 drafts, 32000 tokens, 9.8 us on the GPU, bf16 13.9, which is a chain of
// trips: lengths and drafts, their probabilities, the rows, the sums across the cluster, the piece, the walk. Odd rows of a
// large vocabulary are single loads, a batch of which is asked for when the last one has been added up. With all sums in doubles, and every thread adding up all stretches, 156 and 62 us.
#include <cfloat>

#include "layer_dev.cuh"
#include "../../include/kla_block.h"

namespace kla {
namespace {

constexpr int kBlock = 512, kWarps = kBlock / 32, kMostCtas = 8;

struct VerifyArgs {
    const int *draft;
    const void *q, *p;
    int64_t qb, qr, pb, pr;   // batch and row strides
    const float *u;
    const int *lengths;
    int *accepted, *tokens;
    int B, K, V;
};

// A probability as a weight: nothing where it is not above zero, finite.
__device__ __forceinline__ double weight(float p) { return p > 0.f ? fminf(p, FLT_MAX) : 0.f; }

// What is left of a row for the draw. kRow: the target's own values; kRest: what the draft's do not cover; kAllBut:
// all but the token that the draft was sure of.
enum Rest { kRow, kRest, kAllBut };
__device__ __forceinline__ double left(Rest rest, float p, float q, bool drafted) {
    const double w = weight(p);
    if (rest == kRow) return w;
    if (rest == kAllBut) return drafted ? 0.0 : w;
    return fmax(w - weight(q), 0.0);
}
// A sum of floats that are not negative, with what its roundings have lost.
struct Pair {
    float hi, lo;
    __device__ __forceinline__ void add(float d, float e) {   // d + e, e far smaller
        const float t = hi + d, v = t - hi;
        lo += ((hi - (t - v)) + (d - v)) + e;
        hi = t;
    }
};
// The same as `left`, added to a pair: a difference and its rounding, which is exact.
template <Rest kKind>
__device__ __forceinline__ void add_left(Pair &s, float p, float q, bool drafted) {
    float a = fminf(fmaxf(p, 0.f), FLT_MAX), e = 0.f;   // NaN: 0
    if (kKind == kAllBut && drafted) a = 0.f;
    if (kKind == kRest) {
        const float b = fminf(fmaxf(q, 0.f), FLT_MAX), d = a - b, v = d - a;
        e = d > 0.f ? (a - (d - v)) - (b + v) : 0.f;
        a = fmaxf(d, 0.f);
    }
    s.add(a, e);
}
__device__ __forceinline__ bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// One access: 16 bytes, or a single value.
template <typename T, bool kWide>
struct Access {
    static constexpr int kV = kWide ? 16 / sizeof(T) : 1, kWords = kWide ? 4 : 1;
    uint32_t r[kWords];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kWide) {
            const uint4 q = *reinterpret_cast<const uint4 *>(p);
            r[0] = q.x, r[1] = q.y, r[2] = q.z, r[3] = q.w;
        } else {
            r[0] = __float_as_uint(to_f32(*p));
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (kWide && sizeof(T) == 2) return __uint_as_float(i & 1 ? r[i / 2] & 0xffff0000u : r[i / 2] << 16);
        else return __uint_as_float(r[i]);
    }
};

// What is left of tokens v0 .. v1 - 1, by a warp.
template <typename T, Rest kKind, bool kWide>
__device__ __forceinline__ double stretch_sum(const T *p, const T *q, int v0, int v1, int token) {
    using A = Access<T, kWide>;
    constexpr int kV = A::kV, kAtOnce = kWide ? (sizeof(T) == 4 ? 4 : 2) : 16, kStep = 32 * kV;
    const int lane = threadIdx.x & 31;
    double t = 0.0;
    for (int base = v0 + lane * kV; base - lane * kV < v1; base += kStep * kAtOnce) {
        A x[kAtOnce], y[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int v = base + j * kStep;
            x[j] = y[j] = A{};
            if (v + kV <= v1) {
                x[j].load(p + v);
                if (kKind == kRest) y[j].load(q + v);
            } else if (kWide) {   // the row's end within an access
                for (int i = 0; v + i < v1; ++i) {
                    const uint32_t a = __float_as_uint(to_f32(p[v + i]));
                    const uint32_t b = kKind == kRest ? __float_as_uint(to_f32(q[v + i])) : 0u;
                    if (sizeof(T) == 4) {
#pragma unroll
                        for (int k = 0; k < kV; ++k)
                            if (k == i) x[j].r[k % A::kWords] = a, y[j].r[k % A::kWords] = b;
                    } else {
#pragma unroll
                        for (int k = 0; k < kV; ++k)
                            if (k == i) {
                                x[j].r[k / 2 % A::kWords] |= k & 1 ? a : a >> 16;
                                y[j].r[k / 2 % A::kWords] |= k & 1 ? b : b >> 16;
                            }
                    }
                }
            }
        }
        Pair s{0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
            for (int i = 0; i < kV; ++i) add_left<kKind>(s, x[j][i], y[j][i], base + j * kStep + i == token);
        if (s.hi <= FLT_MAX) {
            t += static_cast<double>(s.hi) + static_cast<double>(s.lo);
        } else {   // more than a float holds
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
                for (int i = 0; i < kV; ++i) t += left(kKind, x[j][i], y[j][i], base + j * kStep + i == token);
        }
    }
    for (int off = 16; off; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    return t;
}
template <typename T>
__device__ __forceinline__ double stretch_sum(Rest rest, bool wide, const T *p, const T *q, int v0, int v1, int token) {
    if (rest == kRest)
        return wide ? stretch_sum<T, kRest, true>(p, q, v0, v1, token) : stretch_sum<T, kRest, false>(p, q, v0, v1, token);
    if (rest == kRow)
        return wide ? stretch_sum<T, kRow, true>(p, q, v0, v1, token) : stretch_sum<T, kRow, false>(p, q, v0, v1, token);
    return wide ? stretch_sum<T, kAllBut, true>(p, q, v0, v1, token) : stretch_sum<T, kAllBut, false>(p, q, v0, v1, token);
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(n));
    return n;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A double of another CTA of the cluster, at the address that it has in this one.
__device__ __forceinline__ double cluster_load(const double *p, uint32_t rank) {
    uint32_t at;
    double v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(at));
    return v;
}

// The stretch of the row that holds the mark, the sum of those before it, and the mark.
struct Draw {
    int stretch;   // -1: there is no weight
    double before, mark;
};
// By one warp, from kMine neighbouring sums a lane, `before` them all: the mark is `mark`, or u times their whole.
template <int kMine>
__device__ __forceinline__ void choose(const double (&w)[kMine], double before, bool of_whole, double mark, Draw &draw) {
    const int lane = threadIdx.x & 31;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) sum += w[i];
    double upto = sum;   // of this lane's and the lanes' before it
    for (int off = 1; off < 32; off <<= 1) {
        const double t = __shfl_up_sync(0xffffffffu, upto, off);
        if (lane >= off) upto += t;
    }
    if (of_whole) mark *= __shfl_sync(0xffffffffu, upto, 31);
    double run = before + (upto - sum), at = run;
    int hit = -1, some = -1;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        if (w[i] > 0.0) {
            some = lane * kMine + i;
            if (hit < 0 && run + w[i] > mark) {
                hit = some;
                at = run;
            }
        }
        run += w[i];
    }
    const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0), somes = __ballot_sync(0xffffffffu, some >= 0);
    if (hits) {
        if (lane == __ffs(hits) - 1) draw = Draw{hit, at, mark};
    } else if (somes) {   // rounding leaves none: the last token with any weight
        if (lane == 31 - __clz(somes)) draw = Draw{some, 0.0, DBL_MAX};
    } else if (lane == 0) {
        draw.stretch = -1;
    }
}

// A cluster of CTAs per sequence. Every warp of it has a stretch of the row and sums it; from those sums every CTA finds
// the stretch that holds the mark, the CTA that has it cuts it into one piece a warp, and the warp whose piece holds
// the mark walks that in 64 bits.
template <typename T>
__global__ void __launch_bounds__(kBlock, 2) verify_kernel(VerifyArgs a) {
    __shared__ int s_took;
    __shared__ double part[3][kWarps];
    __shared__ Draw draw, piece;
    const int ctas = cluster_size(), rank = cluster_rank(), b = blockIdx.x / ctas;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int n = a.lengths ? min(max(a.lengths[b], 0), a.K) : a.K;
    const T *p = static_cast<const T *>(a.p) + b * a.pb, *q = static_cast<const T *>(a.q) + b * a.qb;
    const int *draft = a.draft + static_cast<int64_t>(b) * a.K;
    const float *u = a.u + static_cast<int64_t>(b) * (a.K + 1);
    if (threadIdx.x == 0) s_took = n;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kBlock) {   // every CTA decides for itself
        const int token = draft[i];
        bool ok = token >= 0 && token < a.V;
        if (ok) {
            const double qt = a.q ? weight(to_f32(q[i * a.qr + token])) : 1.0;
            ok = static_cast<double>(u[i]) * qt < weight(to_f32(p[i * a.pr + token]));
        }
        if (!ok) atomicMin(&s_took, i);
    }
    __syncthreads();
    const int took = s_took;
    p += took * a.pr;
    if (a.q) q += took * a.qr;
    const int token = took < n ? draft[took] : -1;
    Rest rest = took == n ? kRow : a.q ? kRest : kAllBut;
    const bool wide = aligned16(p) && (rest != kRest || aligned16(q));
    // stretches and pieces start on whole accesses of a warp
    constexpr int kStep = 32 * 16 / sizeof(T);
    const int per = (a.V + ctas * kWarps * kStep - 1) / (ctas * kWarps * kStep) * kStep;
    auto start = [&](int stretch) { return static_cast<int>(min(static_cast<int64_t>(a.V), static_cast<int64_t>(stretch) * per)); };
    for (int turn = 0;; ++turn) {
        const int v0 = start(rank * kWarps + warp), v1 = start(rank * kWarps + warp + 1);
        const double t = stretch_sum<T>(rest, wide, p, q, v0, v1, token);
        if (lane == 0) part[turn][warp] = t;
        __syncwarp();
        cluster_sync();
        if (warp == 0) {
            constexpr int kMine = kMostCtas * kWarps / 32;
            double w[kMine];
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int at = lane * kMine + i;
                w[i] = at < ctas * kWarps ? cluster_load(&part[turn][at % kWarps], at / kWarps) : 0.0;
            }
            choose<kMine>(w, 0.0, true, u[a.K], draw);
        }
        __syncthreads();
        if (draw.stretch >= 0 || rest == kRow) break;
        rest = kRow;   // the draft covers the target: nothing is left but rounding
        __syncthreads();
    }
    cluster_sync();   // no CTA leaves while another reads its sums
    int *out = a.tokens + static_cast<int64_t>(b) * (a.K + 1);
    if (rank == 0) {
        if (threadIdx.x == 0) a.accepted[b] = took;
        for (int i = threadIdx.x; i <= a.K; i += kBlock)
            if (i != took) out[i] = i < took ? draft[i] : -1;
        if (draw.stretch < 0 && threadIdx.x == 0) out[took] = -1;   // no weight at all
    }
    if (draw.stretch < 0 || draw.stretch / kWarps != rank) return;
    const int from = start(draw.stretch), to = start(draw.stretch + 1);
    const int of_warp = ((to - from) + kWarps * kStep - 1) / (kWarps * kStep) * kStep;
    const int v0 = min(to, from + warp * of_warp), v1 = min(to, v0 + of_warp);
    const double t = stretch_sum<T>(rest, wide, p, q, v0, v1, token);
    if (lane == 0) part[2][warp] = t;
    __syncthreads();
    if (warp == 0) {
        const double w[1] = {lane < kWarps ? part[2][lane] : 0.0};
        choose<1>(w, draw.before, false, draw.mark, piece);
    }
    __syncthreads();
    if (warp != piece.stretch) return;
    constexpr int kWalk = 4;   // tokens a lane
    double run = piece.before;
    int found = -1, any = -1;
    for (int base = v0; base < v1 && found < 0; base += 32 * kWalk) {
        double w[kWalk], s = 0.0;
        int some = -1;
#pragma unroll
        for (int i = 0; i < kWalk; ++i) {
            const int v = base + lane * kWalk + i;
            w[i] = v < v1 ? left(rest, to_f32(p[v]), rest == kRest ? to_f32(q[v]) : 0.f, v == token) : 0.0;
            s += w[i];
            if (w[i] > 0.0) some = v;
        }
        double ahead = s;   // of this lane's and the lanes' before it
        for (int off = 1; off < 32; off <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, ahead, off);
            if (lane >= off) ahead += x;
        }
        double at = run + (ahead - s);
        int hit = -1;
#pragma unroll
        for (int i = 0; i < kWalk; ++i) {
            at += w[i];
            if (hit < 0 && w[i] > 0.0 && at > piece.mark) hit = base + lane * kWalk + i;
        }
        const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0), somes = __ballot_sync(0xffffffffu, some >= 0);
        if (somes) any = __shfl_sync(0xffffffffu, some, 31 - __clz(somes));
        if (hits) found = __shfl_sync(0xffffffffu, hit, __ffs(hits) - 1);
        run += __shfl_sync(0xffffffffu, ahead, 31);
    }
    if (lane == 0) out[took] = found >= 0 ? found : any;
}

template <typename T>
cudaError_t run(const VerifyArgs &a, cudaStream_t s) {
    // as many CTAs as a row fills with four accesses a thread, but no more in all than the SMs hold at once
    constexpr int kSms = 152, kPerSm = 2;
    const int per = kBlock * 4 * (16 / static_cast<int>(sizeof(T)));
    int ctas = 1;
    while (ctas < kMostCtas && ctas * per < a.V && 2 * ctas * static_cast<int64_t>(a.B) <= kSms * kPerSm) ctas *= 2;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = ctas;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ctas);
    cfg.blockDim = dim3(kBlock);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

}  // namespace
}  // namespace kla

extern "C" kla_status kla_verify_draft(const int *draft, const void *draft_probs, const void *target,
                                       const int64_t *strides, const float *uniforms, const int *lengths,
                                       int *accepted, int *tokens, int B, int K, int V, kla_dtype dtype,
                                       void *stream) {
    using namespace kla;
    if (B < 1 || K < 0 || V < 1) return KLA_ERR_INVALID_ARG;
    if (dtype != KLA_DTYPE_F32 && dtype != KLA_DTYPE_BF16) return KLA_ERR_INVALID_ARG;
    if (K > 1024 || V > (1 << 24) || B > 65535) return KLA_ERR_UNSUPPORTED;
    if (!target || !uniforms || !accepted || !tokens || (K > 0 && !draft)) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(draft_probs, esz) || !aligned(target, esz) || !aligned(draft, 4) || !aligned(uniforms, 4) ||
        !aligned(lengths, 4) || !aligned(accepted, 4) || !aligned(tokens, 4))
        return KLA_ERR_INVALID_ARG;
    const int64_t V64 = V;
    VerifyArgs a{draft, K > 0 ? draft_probs : nullptr, target, K * V64, V64, (K + 1) * V64, V64, uniforms, lengths,
                 accepted, tokens, B, K, V};
    if (strides) {
        for (int i = 0; i < 4; ++i)
            if (strides[i] < 0) return KLA_ERR_INVALID_ARG;
        a.qb = strides[0]; a.qr = strides[1]; a.pb = strides[2]; a.pr = strides[3];
    }
    const Span outs[] = {span(accepted, 4ull * B), span(tokens, 4ull * B * (K + 1))};
    const Span ins[] = {span(draft, 4ull * B * K),
                        span(a.q, K > 0 ? ((B - 1) * a.qb + (K - 1) * a.qr + V) * esz : 0),
                        span(target, ((B - 1) * a.pb + K * a.pr + V) * esz), span(uniforms, 4ull * B * (K + 1)),
                        span(lengths, 4ull * B)};
    for (const Span &o : outs)
        for (const Span &i : ins)
            if (overlaps(o, i)) return KLA_ERR_INVALID_ARG;
    if (overlaps(outs[0], outs[1])) return KLA_ERR_INVALID_ARG;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == KLA_DTYPE_BF16 ? run<__nv_bfloat16>(a, cs) : run<float>(a, cs);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}
