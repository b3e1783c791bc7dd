// kla_block_norm.cu -- the norms of a block: after its heads, times the activation of a gate, and of the residual that
// the block's output is added to.
//
//   gated   y = xh w act(z)                 dx = N(dy w act(z)),  dz = dy xh w act'(z),  dw = sum dy act(z) xh
//   added   s = r + l x,  y = xh(s) w       dr = ds + N(dy w),  dx = l dr,  dw = sum dy xh,  dl = sum x dr
//   xh = (x - mean) rstd, N(u) = rstd (u - mean(u) - xh mean(u xh)); without the means' terms where mean = 0 (RMS)
#include <climits>

#include "kla_norm.cuh"
#include "../../include/kla_block.h"

namespace kla {
namespace {

using namespace norm;

struct NormArgs {
    const void *dy, *x, *z;   // added: z is the residual in the forward pass, dsum in the backward pass
    const void *sum;          // added, backward
    int64_t z_stride;         // between rows of `groups` of them
    const float *w, *l;
    int w_groups;             // weights [groups, n]
    void *y, *y2;             // gated: y; dx, dz. added: y, sum; dr, dx
    float *mean, *rstd;
    float *part;              // [parts][2][n]
    int64_t rows;             // of all groups
    int groups, n;
    float eps;
    int layer, silu;
};

template <typename V>
__device__ __forceinline__ V block_sum(V v, V *slots) {
    v = lane_sum<32>(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x / 32] = v;
    __syncthreads();
    v = slots[0];
    for (int i = 1; i < static_cast<int>(blockDim.x) / 32; ++i) v = add(v, slots[i]);
    return v;
}
__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + expf(-z)); }

// A CTA takes rows one after the other.
template <typename T, bool kGated>
__global__ void block_norm_fwd_kernel(NormArgs p) {
    __shared__ float slots[32];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t o = row * p.n;
        const T *x = static_cast<const T *>(p.x) + o;
        const T *z = static_cast<const T *>(p.z) +
                     (kGated ? row / p.groups * p.z_stride + row % p.groups * p.n : o);
        const float *w = p.w ? p.w + (p.w_groups ? row % p.groups * p.n : 0) : nullptr;
        auto value = [&](int c) {
            return kGated ? to_f32(x[c]) : fmaf(p.l ? p.l[c] : 1.f, to_f32(x[c]), to_f32(z[c]));
        };
        float mu = 0.f, q = 0.f;
        if (p.layer) {
            for (int c = threadIdx.x; c < p.n; c += blockDim.x) mu += value(c);
            mu = block_sum(mu, slots) / p.n;
        }
        for (int c = threadIdx.x; c < p.n; c += blockDim.x) {
            const float d = value(c) - mu;
            q = fmaf(d, d, q);
        }
        const float rs = 1.f / sqrtf(block_sum(q, slots) / p.n + p.eps);
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mu;
            if (p.rstd) p.rstd[row] = rs;
        }
        for (int c = threadIdx.x; c < p.n; c += blockDim.x) {
            const float v = value(c);
            float y = (v - mu) * rs * (w ? w[c] : 1.f);
            if (kGated) {
                const float g = to_f32(z[c]), s = sigmoid(g);
                y *= p.silu ? g * s : s;
            } else {
                static_cast<T *>(p.y2)[o + c] = from_f32<T>(v);
            }
            static_cast<T *>(p.y)[o + c] = from_f32<T>(y);
        }
    }
}

template <typename T, bool kGated>
__global__ void block_norm_bwd_kernel(NormArgs p) {
    __shared__ float2 slots[32];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const int64_t o = row * p.n;
        const T *v = static_cast<const T *>(kGated ? p.x : p.sum) + o, *dy = static_cast<const T *>(p.dy) + o;
        const T *z = static_cast<const T *>(p.z);
        if (z) z += kGated ? row / p.groups * p.z_stride + row % p.groups * p.n : o;
        const float *w = p.w ? p.w + (p.w_groups ? row % p.groups * p.n : 0) : nullptr;
        const float mu = p.mean ? p.mean[row] : 0.f, rs = p.rstd[row];
        auto part = [&](int c, float &xh, float &u, float &slope) {   // u = dL/dxh
            xh = (to_f32(v[c]) - mu) * rs;
            u = to_f32(dy[c]) * (w ? w[c] : 1.f);
            if (kGated) {
                const float g = to_f32(z[c]), s = sigmoid(g);
                slope = (p.silu ? s * fmaf(g, 1.f - s, 1.f) : s * (1.f - s)) * u;
                u *= p.silu ? g * s : s;
            }
        };
        float2 s = make_float2(0.f, 0.f);
        float xh, u, slope;
        for (int c = threadIdx.x; c < p.n; c += blockDim.x) {
            part(c, xh, u, slope);
            s.x += u;
            s.y = fmaf(u, xh, s.y);
        }
        s = block_sum(s, slots);
        const float m1 = p.layer ? s.x / p.n : 0.f, m2 = s.y / p.n;
        for (int c = threadIdx.x; c < p.n; c += blockDim.x) {
            part(c, xh, u, slope);
            float d = rs * (u - m1 - xh * m2);
            if (kGated) {
                static_cast<T *>(p.y)[o + c] = from_f32<T>(d);
                static_cast<T *>(p.y2)[o + c] = from_f32<T>(slope * xh);
            } else {
                if (z) d += to_f32(z[c]);
                static_cast<T *>(p.y)[o + c] = from_f32<T>(d);
                if (p.y2) static_cast<T *>(p.y2)[o + c] = from_f32<T>(d * p.l[c]);
            }
        }
    }
}

// Sums over the rows of one group (or of all, where they share weights): a CTA per 32 columns, its lanes along them.
template <typename T, bool kGated>
__global__ void block_norm_sums_kernel(NormArgs p, float *dw, float *dl) {
    __shared__ float2 slots[32][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), warp = threadIdx.x / 32;
    const int64_t step = p.w_groups ? p.groups : 1;
    float2 s = make_float2(0.f, 0.f);
    for (int64_t row = blockIdx.y + warp * step; c < p.n && row < p.rows; row += 32 * step) {
        const int64_t o = row * p.n + c;
        const float mu = p.mean ? p.mean[row] : 0.f, rs = p.rstd[row];
        const float xh = (to_f32(static_cast<const T *>(kGated ? p.x : p.sum)[o]) - mu) * rs;
        float d = to_f32(static_cast<const T *>(p.dy)[o]);
        if (kGated) {
            const float g =
                to_f32(static_cast<const T *>(p.z)[row / p.groups * p.z_stride + row % p.groups * p.n + c]);
            d *= p.silu ? g * sigmoid(g) : sigmoid(g);
        }
        s.x = fmaf(d, xh, s.x);
        if (!kGated && dl) s.y = fmaf(to_f32(static_cast<const T *>(p.x)[o]), to_f32(static_cast<const T *>(p.y)[o]), s.y);
    }
    slots[warp][threadIdx.x & 31] = s;
    __syncthreads();
    if (warp == 0 && c < p.n) {
        for (int i = 1; i < 32; ++i) s = add(s, slots[i][threadIdx.x & 31]);
        if (dw) dw[blockIdx.y * static_cast<int64_t>(p.n) + c] = s.x;
        if (!kGated && dl) dl[c] = s.y;
    }
}

kla_status check(int64_t rows, int groups, int n, kla_dtype dtype) {
    if (rows < 0 || groups < 1 || n < 1) return KLA_ERR_INVALID_ARG;
    if (dtype != KLA_DTYPE_F32 && dtype != KLA_DTYPE_BF16) return KLA_ERR_INVALID_ARG;
    if (n < 3 || n > 65536 || groups > 65535 || rows > INT_MAX / groups) return KLA_ERR_UNSUPPORTED;
    return KLA_OK;
}

template <int kOuts, int kIns>
bool apart(const Span (&outs)[kOuts], const Span (&ins)[kIns]) {
    for (int i = 0; i < kOuts; ++i) {
        for (const Span &s : ins)
            if (overlaps(outs[i], s)) return false;
        for (int j = i + 1; j < kOuts; ++j)
            if (overlaps(outs[i], outs[j])) return false;
    }
    return true;
}

template <typename T, bool kGated>
cudaError_t fwd(const NormArgs &p, cudaStream_t s) {
    const int grid = static_cast<int>(p.rows < 152 * 8 ? p.rows : 152 * 8);
    block_norm_fwd_kernel<T, kGated><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}
template <typename T, bool kGated>
cudaError_t bwd(const NormArgs &p, float *dw, float *dl, cudaStream_t s) {
    const int grid = static_cast<int>(p.rows < 152 * 8 ? p.rows : 152 * 8);
    block_norm_bwd_kernel<T, kGated><<<grid, 256, 0, s>>>(p);
    if (dw || dl)
        block_norm_sums_kernel<T, kGated><<<dim3((p.n + 31) / 32, p.w_groups ? p.groups : 1), 1024, 0, s>>>(p, dw, dl);
    return cudaGetLastError();
}

}  // namespace
}  // namespace kla

extern "C" {

kla_status kla_gated_norm_fwd(const void *x, const void *gate, int64_t gate_stride, const float *weight,
                              int weight_groups, void *y, float *mean, float *rstd, int64_t rows, int groups, int n,
                              kla_dtype dtype, kla_norm_kind norm, kla_activation act, float eps, void *stream) {
    using namespace kla;
    const kla_status st = check(rows, groups, n, dtype);
    if (st != KLA_OK) return st;
    if (!(eps >= 0.f) || eps - eps != 0.f) return KLA_ERR_INVALID_ARG;
    if ((norm != KLA_NORM_RMS && norm != KLA_NORM_LAYER) || (act != KLA_ACT_SILU && act != KLA_ACT_SIGMOID))
        return KLA_ERR_INVALID_ARG;
    if (norm == KLA_NORM_RMS && mean) return KLA_ERR_INVALID_ARG;
    if (gate_stride < static_cast<int64_t>(groups) * n) return KLA_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !gate || !y)) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x, esz) || !aligned(gate, esz) || !aligned(y, esz) || !aligned(weight, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return KLA_ERR_INVALID_ARG;
    if (rows == 0) return KLA_OK;
    const size_t row = static_cast<size_t>(groups) * n, all = rows * row * esz, stat = 4ull * rows * groups;
    const Span outs[] = {span(y, all), span(mean, stat), span(rstd, stat)};
    const Span ins[] = {span(x, all), span(gate, ((rows - 1) * gate_stride + row) * esz),
                        span(weight, 4ull * (weight_groups ? row : n))};
    if (!apart(outs, ins)) return KLA_ERR_INVALID_ARG;
    NormArgs p{};
    p.x = x; p.z = gate; p.z_stride = gate_stride; p.w = weight; p.w_groups = weight_groups != 0; p.y = y;
    p.mean = mean; p.rstd = rstd; p.rows = rows * groups; p.groups = groups; p.n = n; p.eps = eps;
    p.layer = norm == KLA_NORM_LAYER; p.silu = act == KLA_ACT_SILU;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == KLA_DTYPE_BF16 ? fwd<__nv_bfloat16, true>(p, cs) : fwd<float, true>(p, cs);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

size_t kla_gated_norm_bwd_workspace_size(int64_t rows, int groups, int n, kla_dtype dtype, int weight_groups) {
    if (kla::check(rows, groups, n, dtype) != KLA_OK || rows == 0) return 0;
    return 0;
}

kla_status kla_gated_norm_bwd(const void *dy, const void *x, const void *gate, int64_t gate_stride,
                              const float *weight, int weight_groups, const float *mean, const float *rstd, void *dx,
                              void *dgate, float *dweight, int64_t rows, int groups, int n, kla_dtype dtype,
                              kla_activation act, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace kla;
    const kla_status st = check(rows, groups, n, dtype);
    if (st != KLA_OK) return st;
    if (act != KLA_ACT_SILU && act != KLA_ACT_SIGMOID) return KLA_ERR_INVALID_ARG;
    if (gate_stride < static_cast<int64_t>(groups) * n) return KLA_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !x || !gate || !rstd || !dx || !dgate)) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(dy, esz) || !aligned(x, esz) || !aligned(gate, esz) || !aligned(dx, esz) || !aligned(dgate, esz) ||
        !aligned(weight, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dweight, 4) ||
        !aligned(workspace, 16))
        return KLA_ERR_INVALID_ARG;
    const size_t row = static_cast<size_t>(groups) * n, par = 4ull * (weight_groups ? row : n);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (rows == 0)   // no rows: the sums are empty
        return !dweight || cudaMemsetAsync(dweight, 0, par, cs) == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
    const size_t need = dweight ? kla_gated_norm_bwd_workspace_size(rows, groups, n, dtype, weight_groups) : 0;
    if (workspace_bytes < need || (need > 0 && !workspace)) return KLA_ERR_INVALID_ARG;
    const size_t all = rows * row * esz, stat = 4ull * rows * groups;
    const Span outs[] = {span(dx, all), span(dgate, all), span(dweight, par), span(workspace, need)};
    const Span ins[] = {span(dy, all), span(x, all), span(gate, ((rows - 1) * gate_stride + row) * esz),
                        span(weight, par), span(mean, stat), span(rstd, stat)};
    if (!apart(outs, ins)) return KLA_ERR_INVALID_ARG;
    NormArgs p{};
    p.dy = dy; p.x = x; p.z = gate; p.z_stride = gate_stride; p.w = weight; p.w_groups = weight_groups != 0;
    p.y = dx; p.y2 = dgate; p.mean = const_cast<float *>(mean); p.rstd = const_cast<float *>(rstd);
    p.rows = rows * groups; p.groups = groups; p.n = n; p.layer = mean != nullptr; p.silu = act == KLA_ACT_SILU;
    const cudaError_t e = dtype == KLA_DTYPE_BF16 ? bwd<__nv_bfloat16, true>(p, dweight, nullptr, cs)
                                                  : bwd<float, true>(p, dweight, nullptr, cs);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

kla_status kla_add_norm_fwd(const void *x, const void *residual, const float *weight, const float *scale, void *y,
                            void *sum, float *mean, float *rstd, int64_t rows, int n, kla_dtype dtype,
                            kla_norm_kind norm, float eps, void *stream) {
    using namespace kla;
    const kla_status st = check(rows, 1, n, dtype);
    if (st != KLA_OK) return st;
    if (!(eps >= 0.f) || eps - eps != 0.f) return KLA_ERR_INVALID_ARG;
    if (norm != KLA_NORM_RMS && norm != KLA_NORM_LAYER) return KLA_ERR_INVALID_ARG;
    if (norm == KLA_NORM_RMS && mean) return KLA_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !residual || !y || !sum)) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x, esz) || !aligned(residual, esz) || !aligned(y, esz) || !aligned(sum, esz) || !aligned(weight, 4) ||
        !aligned(scale, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
        return KLA_ERR_INVALID_ARG;
    if (rows == 0) return KLA_OK;
    const size_t all = static_cast<size_t>(rows) * n * esz, stat = 4ull * rows, par = 4ull * n;
    const Span outs[] = {span(y, all), span(sum, all), span(mean, stat), span(rstd, stat)};
    const Span ins[] = {span(x, all), span(weight, par), span(scale, par),
                        sum == residual ? span(nullptr, 0) : span(residual, all)};
    if (!apart(outs, ins)) return KLA_ERR_INVALID_ARG;
    NormArgs p{};
    p.x = x; p.z = residual; p.w = weight; p.l = scale; p.y = y; p.y2 = sum; p.mean = mean; p.rstd = rstd;
    p.rows = rows; p.groups = 1; p.n = n; p.eps = eps; p.layer = norm == KLA_NORM_LAYER;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == KLA_DTYPE_BF16 ? fwd<__nv_bfloat16, false>(p, cs) : fwd<float, false>(p, cs);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

size_t kla_add_norm_bwd_workspace_size(int64_t rows, int n, kla_dtype dtype) {
    if (kla::check(rows, 1, n, dtype) != KLA_OK || rows == 0) return 0;
    return 0;
}

kla_status kla_add_norm_bwd(const void *dy, const void *dsum, const void *x, const void *sum, const float *weight,
                            const float *scale, const float *mean, const float *rstd, void *dx, void *dresidual,
                            float *dweight, float *dscale, int64_t rows, int n, kla_dtype dtype, void *workspace,
                            size_t workspace_bytes, void *stream) {
    using namespace kla;
    const kla_status st = check(rows, 1, n, dtype);
    if (st != KLA_OK) return st;
    if (!scale && (dx || dscale)) return KLA_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !sum || !rstd || !dresidual || (scale && !dx) || (dscale && !x))) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(dy, esz) || !aligned(dsum, esz) || !aligned(x, esz) || !aligned(sum, esz) || !aligned(dx, esz) ||
        !aligned(dresidual, esz) || !aligned(weight, 4) || !aligned(scale, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dscale, 4) || !aligned(workspace, 16))
        return KLA_ERR_INVALID_ARG;
    const size_t par = 4ull * n;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if ((dweight && cudaMemsetAsync(dweight, 0, par, cs) != cudaSuccess) ||
            (dscale && cudaMemsetAsync(dscale, 0, par, cs) != cudaSuccess))
            return KLA_ERR_CUDA;
        return KLA_OK;
    }
    const size_t need = dweight || dscale ? kla_add_norm_bwd_workspace_size(rows, n, dtype) : 0;
    if (workspace_bytes < need || (need > 0 && !workspace)) return KLA_ERR_INVALID_ARG;
    const size_t all = static_cast<size_t>(rows) * n * esz, stat = 4ull * rows;
    const Span outs[] = {span(dx, all), span(dresidual, all), span(dweight, par), span(dscale, par),
                         span(workspace, need)};
    const Span ins[] = {span(dy, all), span(dsum, all), span(dscale ? x : nullptr, all), span(sum, all),
                        span(weight, par), span(scale, par), span(mean, stat), span(rstd, stat)};
    if (!apart(outs, ins)) return KLA_ERR_INVALID_ARG;
    NormArgs p{};
    p.dy = dy; p.x = x; p.z = dsum; p.sum = sum; p.w = weight; p.l = scale; p.y = dresidual; p.y2 = dx;
    p.mean = const_cast<float *>(mean); p.rstd = const_cast<float *>(rstd);
    p.rows = rows; p.groups = 1; p.n = n; p.layer = mean != nullptr;
    const cudaError_t e = dtype == KLA_DTYPE_BF16 ? bwd<__nv_bfloat16, false>(p, dweight, dscale, cs)
                                                  : bwd<float, false>(p, dweight, dscale, cs);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // extern "C"
