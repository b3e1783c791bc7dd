// kla_verify.cu -- verification of drafted tokens: which of them the target accepts, and the token after those.
//
// Comparisons are exact: u q of two 24-bit numbers fits the 53 bits of a double, and so does a draw's running sum but
// for the last of them, so that a token's border is off by 2^-50 of the whole at most, far less than what lies between
// two values of a 24-bit random number. Sums in fp32 over 100000 tokens would move borders by whole tokens.
#include <cfloat>

#include "layer_dev.cuh"
#include "../../include/kla_block.h"

namespace kla {
namespace {

constexpr int kBlock = 1024, kWarps = kBlock / 32;

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
template <typename T>
__device__ __forceinline__ double left(Rest rest, const T *p, const T *q, int token, int v) {
    const double w = weight(to_f32(p[v]));
    if (rest == kRow) return w;
    if (rest == kAllBut) return v == token ? 0.0 : w;
    const double d = w - weight(to_f32(q[v]));
    return d > 0.0 ? d : 0.0;
}

template <typename T>
__global__ void __launch_bounds__(kBlock) verify_kernel(VerifyArgs a) {
    __shared__ int s_took;
    __shared__ double part[kWarps];
    const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int n = a.lengths ? min(max(a.lengths[b], 0), a.K) : a.K;
    const T *p = static_cast<const T *>(a.p) + b * a.pb, *q = static_cast<const T *>(a.q) + b * a.qb;
    const int *draft = a.draft + static_cast<int64_t>(b) * a.K;
    const float *u = a.u + static_cast<int64_t>(b) * (a.K + 1);
    if (threadIdx.x == 0) s_took = n;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kBlock) {
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
    q += took * a.qr;
    const int token = took < n ? draft[took] : -1;
    Rest rest = took == n ? kRow : a.q ? kRest : kAllBut;
    // a warp's own stretch of the row
    const int per = (a.V + kWarps - 1) / kWarps, v0 = min(a.V, warp * per), v1 = min(a.V, v0 + per);
    double whole = 0.0;
    for (int turn = 0; turn < 2; ++turn) {
        double s = 0.0;
        for (int v = v0 + lane; v < v1; v += 32) s += left(rest, p, q, token, v);
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        __syncthreads();
        if (lane == 0) part[warp] = s;
        __syncthreads();
        whole = 0.0;
        for (int w = 0; w < kWarps; ++w) whole += part[w];
        if (whole > 0.0 || rest == kRow) break;
        rest = kRow;   // the draft covers the target: nothing is left but rounding
    }
    if (threadIdx.x == 0) a.accepted[b] = took;
    int *out = a.tokens + static_cast<int64_t>(b) * (a.K + 1);
    for (int i = threadIdx.x; i <= a.K; i += kBlock)
        if (i != took) out[i] = i < took ? draft[i] : -1;
    double mark = static_cast<double>(u[a.K]) * whole;
    // the warp whose stretch holds the mark; the last one with any weight where rounding leaves none
    double before = 0.0;
    int mine = -1, last = -1;
    double mine_before = 0.0;
    for (int w = 0; w < kWarps; ++w) {
        if (part[w] > 0.0) {
            last = w;
            if (mine < 0 && before + part[w] > mark) {
                mine = w;
                mine_before = before;
            }
        }
        before += part[w];
    }
    if (last < 0) {
        if (threadIdx.x == 0) out[took] = -1;
        return;
    }
    if (mine < 0) {
        mine = last;
        mark = DBL_MAX;   // above every sum: the last token with any weight
    }
    if (warp != mine) return;
    int found = -1, any = -1;
    double run = mine_before;
    for (int base = v0; base < v1 && found < 0; base += 32) {
        const int v = base + lane;
        const double w = v < v1 ? left(rest, p, q, token, v) : 0.0;
        double s = w;
        for (int off = 1; off < 32; off <<= 1) {
            const double t = __shfl_up_sync(0xffffffffu, s, off);
            if (lane >= off) s += t;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, w > 0.0 && run + s > mark);
        const unsigned some = __ballot_sync(0xffffffffu, w > 0.0);
        if (some) any = base + 31 - __clz(some);
        if (hit) found = base + __ffs(hit) - 1;
        run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) out[took] = found >= 0 ? found : any;
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
    if (dtype == KLA_DTYPE_BF16) verify_kernel<__nv_bfloat16><<<B, kBlock, 0, cs>>>(a);
    else verify_kernel<float><<<B, kBlock, 0, cs>>>(a);
    return cudaGetLastError() == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}
