// kla_rotary.cu -- rotary positions: pair i of a head's first `rot` values, (u, v), turned by position freqs[i].
//
// An angle counts as a 64-bit fraction of a turn: the frequency as turns a token, times 2^64, modulo 2^64; times the
// position in integers, whose overflow is whole turns. Its upper 32 bits, as a signed number of half turns, are what
// sine and cosine take. The product in fp32 would lose a bit with every doubling of the position, and one in fp64
// would cost tens of instructions of a pipe that does two a cycle and SM.
#include "layer_dev.cuh"
#include "../../include/kla_block.h"

namespace kla {
namespace {

struct RotaryArgs {
    const void *in[2];
    void *out[2];
    int64_t is[2][3], os[2][3];   // batch, token and head strides
    const float *freqs;
    const void *positions;
    int wide;                     // positions are int64
    int64_t tokens;
    int T, H[2], d, rot;
    float scale;
    int inverse;
};

// Turns a token, as a fraction of 2^64.
__device__ __forceinline__ unsigned long long turn_rate(float freq) {
    double t = static_cast<double>(freq) * 0.15915494309189533577;
    t -= floor(t);
    return static_cast<unsigned long long>(t * 18446744073709551616.0);
}
__device__ __forceinline__ void angle(unsigned long long rate, long long position, float &s, float &c) {
    const int half_turns = static_cast<int>((rate * static_cast<unsigned long long>(position)) >> 32);
    sincospif(static_cast<float>(half_turns) * 0x1p-31f, &s, &c);
}
__device__ __forceinline__ long long position_of(const RotaryArgs &p, int64_t token) {
    if (!p.positions) return token % p.T;
    return p.wide ? static_cast<const long long *>(p.positions)[token] : static_cast<const int *>(p.positions)[token];
}

// A CTA per token: every thread takes pairs of all heads.
template <typename T, bool kHalf>
__global__ void rotary_kernel(RotaryArgs p) {
    extern __shared__ float2 turn[];   // cos, sin
    const int64_t token = blockIdx.x;
    const int pairs = p.rot / 2;
    const long long at = position_of(p, token);
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
        float s, c;
        angle(turn_rate(p.freqs[i]), at, s, c);
        turn[i] = make_float2(p.scale * c, p.inverse ? -p.scale * s : p.scale * s);
    }
    __syncthreads();
    const int units = pairs + p.d - p.rot;   // pairs, then single values that are copied
    const int64_t b = token / p.T, t = token % p.T;
#pragma unroll
    for (int m = 0; m < 2; ++m)
        for (int i = threadIdx.x; i < p.H[m] * units; i += blockDim.x) {
            const int head = i / units, u = i % units;
            const T *x = static_cast<const T *>(p.in[m]) + b * p.is[m][0] + t * p.is[m][1] + head * p.is[m][2];
            T *y = static_cast<T *>(p.out[m]) + b * p.os[m][0] + t * p.os[m][1] + head * p.os[m][2];
            if (u < pairs) {
                const int i0 = kHalf ? u : 2 * u, i1 = kHalf ? u + pairs : 2 * u + 1;
                const float a = to_f32(x[i0]), v = to_f32(x[i1]);
                const float2 r = turn[u];
                y[i0] = from_f32<T>(fmaf(a, r.x, -v * r.y));
                y[i1] = from_f32<T>(fmaf(v, r.x, a * r.y));
            } else {
                y[u + pairs] = x[u + pairs];
            }
        }
}

template <typename T>
cudaError_t run(const RotaryArgs &p, bool half, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(p.tokens);
    const size_t smem = p.rot / 2 * sizeof(float2);
    if (half) rotary_kernel<T, true><<<grid, 256, smem, s>>>(p);
    else rotary_kernel<T, false><<<grid, 256, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace kla

extern "C" kla_status kla_rotary(const void *q, const void *k, void *q_out, void *k_out, const int64_t *strides,
                                 const float *freqs, const void *positions, int positions_are_64, int B, int T,
                                 int Hq, int Hk, int d, int rot, kla_rotary_layout layout, kla_dtype dtype,
                                 float scale, int inverse, void *stream) {
    using namespace kla;
    if (B < 0 || T < 0 || Hq < 1 || Hk < 0 || d < 1 || rot < 0 || rot > d || rot % 2) return KLA_ERR_INVALID_ARG;
    if (dtype != KLA_DTYPE_F32 && dtype != KLA_DTYPE_BF16) return KLA_ERR_INVALID_ARG;
    if (layout != KLA_ROTARY_HALF && layout != KLA_ROTARY_INTERLEAVED) return KLA_ERR_INVALID_ARG;
    if (scale - scale != 0.f) return KLA_ERR_INVALID_ARG;
    if (d > 1024 || Hq > 65535 || Hk > 65535 || static_cast<int64_t>(B) * T > 0x7fffffff) return KLA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(B) * T == 0) return KLA_OK;
    if (!q || !q_out || (rot > 0 && !freqs) || (Hk > 0 && (!k || !k_out))) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    const void *in[2] = {q, k};
    void *out[2] = {q_out, k_out};
    const int H[2] = {Hq, Hk};
    RotaryArgs p{};
    Span is[2], os[2];
    bool in_place[2] = {false, false};
    for (int m = 0; m < 2; ++m) {
        if (H[m] == 0) {
            is[m] = os[m] = span(nullptr, 0);
            continue;
        }
        if (!aligned(in[m], esz) || !aligned(out[m], esz)) return KLA_ERR_INVALID_ARG;
        const int64_t dense[3] = {static_cast<int64_t>(T) * H[m] * d, static_cast<int64_t>(H[m]) * d, d};
        size_t ri = d, ro = d;
        bool same = in[m] == out[m];
        for (int a = 0; a < 3; ++a) {
            p.is[m][a] = strides ? strides[3 * m + a] : dense[a];
            p.os[m][a] = strides ? strides[6 + 3 * m + a] : dense[a];
            if (p.is[m][a] < 0 || p.os[m][a] < 0) return KLA_ERR_INVALID_ARG;
            const size_t last = (a == 0 ? B : a == 1 ? T : H[m]) - 1;
            ri += last * p.is[m][a];
            ro += last * p.os[m][a];
            if (last && p.os[m][a] == 0) return KLA_ERR_INVALID_ARG;   // one place for several values
            if (last && p.is[m][a] != p.os[m][a]) same = false;
        }
        in_place[m] = same;
        is[m] = span(in[m], ri * esz);
        os[m] = span(out[m], ro * esz);
        p.in[m] = in[m];
        p.out[m] = out[m];
        p.H[m] = H[m];
    }
    const Span sf = span(freqs, rot / 2 * 4ull);
    const Span sp = span(positions, static_cast<size_t>(B) * T * (positions_are_64 ? 8 : 4));
    if (!aligned(freqs, 4) || !aligned(positions, positions_are_64 ? 8 : 4)) return KLA_ERR_INVALID_ARG;
    for (int m = 0; m < 2; ++m) {
        if (overlaps(os[m], sf) || overlaps(os[m], sp)) return KLA_ERR_INVALID_ARG;
        // slices of one packed tensor reach over each other: in place, an output covers what its input covers
        if (in_place[m]) continue;
        if (overlaps(os[m], is[0]) || overlaps(os[m], is[1]) || overlaps(os[m], os[1 - m])) return KLA_ERR_INVALID_ARG;
    }
    p.freqs = freqs;
    p.positions = positions;
    p.wide = positions_are_64 != 0;
    p.tokens = static_cast<int64_t>(B) * T;
    p.T = T;
    p.d = d;
    p.rot = rot;
    p.scale = scale;
    p.inverse = inverse != 0;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool half = layout == KLA_ROTARY_HALF;
    const cudaError_t e = dtype == KLA_DTYPE_BF16 ? run<__nv_bfloat16>(p, half, cs) : run<float>(p, half, cs);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}
