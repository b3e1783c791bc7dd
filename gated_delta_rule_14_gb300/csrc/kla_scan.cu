// kla_scan.cu -- the gated scan: h_t = a_t h_{t-1} + w_t x_t for every channel, forward, gradients and single tokens.
//
//   KLA_SCAN_SIGMOID   w = 1 / (1 + exp(gate)),  h = a h + w x,  dgate = a w (h_{t-1} - x) dh   with a = 1 - w
//   KLA_SCAN_LOG       a = exp(gate),            h = a h + x,    dgate = a h_{t-1} dh
//   both               dh_t = dy_t + a_{t+1} dh_{t+1},  dx = w dh
//
// The sigmoid's recurrence is taken as h + w (x - h) where w is the smaller of the two factors, as x + a (h - x) where
// a is: where a gate keeps its state for thousands of tokens a is within 2^-11 of 1 and its rounding to 24 bits would
// leave 12 of w, and where one drops a large state nothing of it may stay behind as a difference of roundings.
#include <climits>

#include "layer_dev.cuh"
#include "../../include/kla_block.h"

namespace kla {
namespace {

struct ScanArgs {
    const void *x, *gate, *dy;
    int64_t xb, xt, gb, gt, db, dt;   // batch and token strides
    const int *lengths;
    const float *h0;                  // backward: dh_T
    void *y, *dg;                     // backward: dx, dgate
    float *h_T;                       // backward: dh0
    float *states;
    int B, T, C;
};

__device__ __forceinline__ int valid_tokens(const ScanArgs &p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}

// The state's factor a and the input's w. exp(gate) is held below 2^100: w stays a normal number, a is 1.
template <bool kLog>
__device__ __forceinline__ void factors(float gate, float &a, float &w) {
    if (kLog) {
        a = expf(gate);
        w = 1.f;
    } else {
        float e = expf(gate);
        e = e > 0x1p100f ? 0x1p100f : e;
        w = 1.f / (1.f + e);
        a = e * w;
    }
}
template <bool kLog>
__device__ __forceinline__ float advance(float h, float x, float a, float w) {
    if (kLog) return fmaf(a, h, x);
    return w < 0.5f ? fmaf(w, x - h, h) : fmaf(a, h - x, x);
}

// A thread per channel walks all tokens.
template <typename T, bool kLog>
__global__ void scan_fwd_kernel(ScanArgs p) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
    if (c >= p.C) return;
    const T *x = static_cast<const T *>(p.x) + b * p.xb + c, *g = static_cast<const T *>(p.gate) + b * p.gb + c;
    T *y = static_cast<T *>(p.y) + static_cast<int64_t>(b) * p.T * p.C + c;
    const int n = valid_tokens(p, b);
    const int64_t spans = (p.T + KLA_SCAN_SPAN - 1) / KLA_SCAN_SPAN;
    float h = p.h0 ? p.h0[static_cast<int64_t>(b) * p.C + c] : 0.f;
    for (int t = 0; t < n; ++t) {
        if (p.states && t % KLA_SCAN_SPAN == 0) p.states[(b * spans + t / KLA_SCAN_SPAN) * p.C + c] = h;
        float a, w;
        factors<kLog>(to_f32(g[t * p.gt]), a, w);
        h = advance<kLog>(h, to_f32(x[t * p.xt]), a, w);
        y[static_cast<int64_t>(t) * p.C] = from_f32<T>(h);
    }
    for (int t = n; t < p.T; ++t) y[static_cast<int64_t>(t) * p.C] = from_f32<T>(0.f);
    if (p.h_T) p.h_T[static_cast<int64_t>(b) * p.C + c] = h;
}

template <typename T, bool kLog>
__global__ void scan_bwd_kernel(ScanArgs p) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
    if (c >= p.C) return;
    const T *x = static_cast<const T *>(p.x) + b * p.xb + c, *g = static_cast<const T *>(p.gate) + b * p.gb + c;
    const T *dy = static_cast<const T *>(p.dy) + b * p.db + c;
    const int64_t out0 = static_cast<int64_t>(b) * p.T * p.C + c;
    T *dx = static_cast<T *>(p.y) + out0, *dg = static_cast<T *>(p.dg) + out0;
    const int n = valid_tokens(p, b);
    const int64_t spans = (p.T + KLA_SCAN_SPAN - 1) / KLA_SCAN_SPAN;
    for (int t = n; t < p.T; ++t) {
        dx[static_cast<int64_t>(t) * p.C] = from_f32<T>(0.f);
        dg[static_cast<int64_t>(t) * p.C] = from_f32<T>(0.f);
    }
    float e = p.h0 ? p.h0[static_cast<int64_t>(b) * p.C + c] : 0.f;   // what reaches the state after token t
    float before[KLA_SCAN_SPAN];
    for (int s = (n + KLA_SCAN_SPAN - 1) / KLA_SCAN_SPAN - 1; s >= 0; --s) {
        const int t0 = s * KLA_SCAN_SPAN, m = min(n - t0, KLA_SCAN_SPAN);
        float h = p.states[(b * spans + s) * p.C + c], a, w;
        for (int i = 0; i < m; ++i) {
            before[i] = h;
            factors<kLog>(to_f32(g[(t0 + i) * p.gt]), a, w);
            h = advance<kLog>(h, to_f32(x[(t0 + i) * p.xt]), a, w);
        }
        for (int i = m - 1; i >= 0; --i) {
            const int64_t t = t0 + i;
            factors<kLog>(to_f32(g[t * p.gt]), a, w);
            const float dh = to_f32(dy[t * p.dt]) + e;
            dx[t * p.C] = from_f32<T>(w * dh);
            dg[t * p.C] = from_f32<T>(kLog ? a * before[i] * dh : a * w * (before[i] - to_f32(x[t * p.xt])) * dh);
            e = a * dh;
        }
    }
    if (p.h_T) p.h_T[static_cast<int64_t>(b) * p.C + c] = e;
}

template <typename T, bool kLog>
__global__ void scan_step_kernel(const T *x, int64_t xs, const T *gate, int64_t gs, float *h, T *y, int C) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
    if (c >= C) return;
    const int64_t at = static_cast<int64_t>(b) * C + c;
    float a, w;
    factors<kLog>(to_f32(gate[b * gs + c]), a, w);
    const float v = advance<kLog>(h[at], to_f32(x[b * xs + c]), a, w);
    h[at] = v;
    y[at] = from_f32<T>(v);
}

kla_status check(int B, int T, int C, kla_dtype dtype, kla_scan_mode mode) {
    if (B < 1 || T < 0 || C < 1) return KLA_ERR_INVALID_ARG;
    if (dtype != KLA_DTYPE_F32 && dtype != KLA_DTYPE_BF16) return KLA_ERR_INVALID_ARG;
    if (mode != KLA_SCAN_SIGMOID && mode != KLA_SCAN_LOG) return KLA_ERR_INVALID_ARG;
    if (T > INT_MAX - 65536 || B > 65535) return KLA_ERR_UNSUPPORTED;
    return KLA_OK;
}

// Bytes from a strided tensor's start to its last element's end.
size_t reach(int B, int T, int C, int64_t sb, int64_t st, size_t esz) {
    return T == 0 ? 0 : (static_cast<size_t>(B - 1) * sb + static_cast<size_t>(T - 1) * st + C) * esz;
}

template <typename F>
cudaError_t by_type(kla_dtype dtype, kla_scan_mode mode, F f) {
    if (dtype == KLA_DTYPE_BF16) {
        if (mode == KLA_SCAN_LOG) f(__nv_bfloat16{}, std::true_type{});
        else f(__nv_bfloat16{}, std::false_type{});
    } else {
        if (mode == KLA_SCAN_LOG) f(float{}, std::true_type{});
        else f(float{}, std::false_type{});
    }
    return cudaGetLastError();
}

}  // namespace
}  // namespace kla

extern "C" {

size_t kla_gated_scan_workspace_size(int B, int T, int C, kla_dtype dtype) {
    if (kla::check(B, T, C, dtype, KLA_SCAN_SIGMOID) != KLA_OK) return 0;
    return 0;
}

kla_status kla_gated_scan_fwd(const void *x, const void *gate, const int64_t *strides, const int *lengths,
                              const float *h0, void *y, float *h_T, float *states, int B, int T, int C,
                              kla_dtype dtype, kla_scan_mode mode, void *workspace, size_t workspace_bytes,
                              void *stream) {
    using namespace kla;
    const kla_status st = check(B, T, C, dtype, mode);
    if (st != KLA_OK) return st;
    if (T > 0 && (!x || !gate || !y)) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x, esz) || !aligned(gate, esz) || !aligned(y, esz) || !aligned(lengths, 4) || !aligned(h0, 4) ||
        !aligned(h_T, 4) || !aligned(states, 4) || !aligned(workspace, 16))
        return KLA_ERR_INVALID_ARG;
    const int64_t tc = static_cast<int64_t>(T) * C;
    ScanArgs p{x, gate, nullptr, tc, C, tc, C, 0, 0, lengths, h0, y, nullptr, h_T, states, B, T, C};
    if (strides) {
        for (int i = 0; i < 4; ++i)
            if (strides[i] < 0) return KLA_ERR_INVALID_ARG;
        p.xb = strides[0]; p.xt = strides[1]; p.gb = strides[2]; p.gt = strides[3];
    }
    const size_t need = kla_gated_scan_workspace_size(B, T, C, dtype);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KLA_ERR_INVALID_ARG;
    const size_t state = 4ull * B * C, spans = (T + KLA_SCAN_SPAN - 1) / KLA_SCAN_SPAN;
    const Span outs[] = {span(y, static_cast<size_t>(B) * tc * esz), span(h_T, state), span(states, state * spans),
                         span(workspace, need)};
    const Span ins[] = {span(x, reach(B, T, C, p.xb, p.xt, esz)), span(gate, reach(B, T, C, p.gb, p.gt, esz)),
                        span(lengths, 4ull * B), span(h0, state)};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 4; ++j)
            if (overlaps(outs[i], ins[j]) && !(i == 1 && j == 3 && h_T == h0)) return KLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(outs[i], outs[j])) return KLA_ERR_INVALID_ARG;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = by_type(dtype, mode, [&](auto t, auto log) {
        scan_fwd_kernel<decltype(t), decltype(log)::value><<<dim3((C + 31) / 32, B), 32, 0, cs>>>(p);
    });
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

kla_status kla_gated_scan_bwd(const void *x, const void *gate, const void *dy, const int64_t *strides,
                              const int *lengths, const float *states, const float *dh_T, void *dx, void *dgate,
                              float *dh0, int B, int T, int C, kla_dtype dtype, kla_scan_mode mode, void *workspace,
                              size_t workspace_bytes, void *stream) {
    using namespace kla;
    const kla_status st = check(B, T, C, dtype, mode);
    if (st != KLA_OK) return st;
    if (T > 0 && (!x || !gate || !dy || !dx || !dgate || !states)) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x, esz) || !aligned(gate, esz) || !aligned(dy, esz) || !aligned(dx, esz) || !aligned(dgate, esz) ||
        !aligned(lengths, 4) || !aligned(states, 4) || !aligned(dh_T, 4) || !aligned(dh0, 4) ||
        !aligned(workspace, 16))
        return KLA_ERR_INVALID_ARG;
    const int64_t tc = static_cast<int64_t>(T) * C;
    ScanArgs p{x, gate, dy, tc, C, tc, C, tc, C, lengths, dh_T, dx, dgate, dh0, const_cast<float *>(states), B, T, C};
    if (strides) {
        for (int i = 0; i < 6; ++i)
            if (strides[i] < 0) return KLA_ERR_INVALID_ARG;
        p.xb = strides[0]; p.xt = strides[1]; p.gb = strides[2]; p.gt = strides[3]; p.db = strides[4]; p.dt = strides[5];
    }
    const size_t need = kla_gated_scan_workspace_size(B, T, C, dtype);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KLA_ERR_INVALID_ARG;
    const size_t state = 4ull * B * C, spans = (T + KLA_SCAN_SPAN - 1) / KLA_SCAN_SPAN;
    const size_t all = static_cast<size_t>(B) * tc * esz;
    const Span outs[] = {span(dx, all), span(dgate, all), span(dh0, state), span(workspace, need)};
    const Span ins[] = {span(x, reach(B, T, C, p.xb, p.xt, esz)), span(gate, reach(B, T, C, p.gb, p.gt, esz)),
                        span(dy, reach(B, T, C, p.db, p.dt, esz)), span(lengths, 4ull * B),
                        span(states, state * spans), span(dh_T, state)};
    for (int i = 0; i < 4; ++i) {
        for (const Span &s : ins)
            if (overlaps(outs[i], s)) return KLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(outs[i], outs[j])) return KLA_ERR_INVALID_ARG;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = by_type(dtype, mode, [&](auto t, auto log) {
        scan_bwd_kernel<decltype(t), decltype(log)::value><<<dim3((C + 31) / 32, B), 32, 0, cs>>>(p);
    });
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

kla_status kla_gated_scan_step(const void *x, int64_t x_stride, const void *gate, int64_t gate_stride, float *h,
                               void *y, int B, int C, kla_dtype dtype, kla_scan_mode mode, void *stream) {
    using namespace kla;
    const kla_status st = check(B, 1, C, dtype, mode);
    if (st != KLA_OK) return st;
    if (!x || !gate || !h || !y || x_stride < C || gate_stride < C) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x, esz) || !aligned(gate, esz) || !aligned(y, esz) || !aligned(h, 4)) return KLA_ERR_INVALID_ARG;
    const Span sx = span(x, reach(B, 1, C, x_stride, 0, esz)), sg = span(gate, reach(B, 1, C, gate_stride, 0, esz));
    const Span sh = span(h, 4ull * B * C), sy = span(y, esz * B * C);
    if (overlaps(sh, sx) || overlaps(sh, sg) || overlaps(sy, sx) || overlaps(sy, sg) || overlaps(sy, sh))
        return KLA_ERR_INVALID_ARG;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = by_type(dtype, mode, [&](auto t, auto log) {
        using E = decltype(t);
        scan_step_kernel<E, decltype(log)::value><<<dim3((C + 255) / 256, B), 256, 0, cs>>>(
            static_cast<const E *>(x), x_stride, static_cast<const E *>(gate), gate_stride, h, static_cast<E *>(y), C);
    });
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // extern "C"
