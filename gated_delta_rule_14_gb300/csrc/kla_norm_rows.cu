// kla_norm_rows.cu -- layer norm over rows of up to 512 values, forward and gradients (the formulas are at the
// head of kla_norm.cu).
//
// A row belongs to a team of kL lanes (a power of two that fits it), each with kNV accesses of kV values at
// fixed columns. A team takes kR rows at a time, whose loads are on their way together: short rows are
// bound by how many bytes are in flight, and with one row of 64 bf16 values a turn on half-empty teams of 16
// lanes a fifth of the memory's rate was reached. CTAs are persistent and keep to one group, so that
// weight, bias and the sums of dw and db stay in registers.
// Measured, 29296 x 16 heads of 64 bf16: forward 34 us (52 % of a copy's rate), backward 41 us (64 %); 100000 x 300
// fp32: 46 and 75 us. Warps wait for their loads most (4.5 of them a cycle, 3.3 in the backward pass), at 2.4 of 4
// instructions issued a cycle (2.1): the loads' latency bounds it. 64 x 16 heads of 128 take 2.5 us, a launch's.
#include "kla_norm.cuh"

namespace kla {
namespace {

using namespace norm;

constexpr int kThreads = 256;

// A team's columns of one thread: access k covers columns (k * kL + lane) * kV ..
template <typename T, int kV, int kL, int kNV>
__device__ __forceinline__ void take(const T *row, int lane, int n, bool live, T (&v)[kV * kNV]) {
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
        const int c = (k * kL + lane) * kV;
        if (live && c < n) {
            load<T, kV>(row + c, v + k * kV);
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) v[k * kV + i] = from_f32<T>(0.f);
        }
    }
}

template <int kE>
constexpr int rows_at_once() { return kE <= 8 ? 4 : 2; }

constexpr int fwd_ctas(int e) { return e <= 8 ? 4 : 3; }   // an SM's registers hold

template <typename T, int kV, int kL, int kNV>
__global__ void __launch_bounds__(kThreads, fwd_ctas(kV * kNV))
rows_fwd_kernel(const T *x, const float *w, const float *b, T *y, float *mean, float *rstd, int64_t rows, int groups,
                int n, float eps) {
    constexpr int kE = kV * kNV, kR = rows_at_once<kE>();
    const Walk at(groups, kL);
    float wr[kE], br[kE];
#pragma unroll
    for (int u = 0; u < kE; ++u) {
        const int c = (u / kV * kL + at.lane) * kV + u % kV;
        wr[u] = w && c < n ? w[static_cast<int64_t>(at.g) * n + c] : 1.f;
        br[u] = b && c < n ? b[static_cast<int64_t>(at.g) * n + c] : 0.f;
    }
    const float inv = 1.f / n;
    // every lane of a warp takes the same number of turns (the sums use whole warps)
    const int64_t block0 = at.first - threadIdx.x / kL;
    for (int64_t r0 = at.first; r0 - at.first + block0 < rows; r0 += kR * at.step) {
        alignas(16) T raw[kR][kE];
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            const int64_t r = r0 + j * at.step;
            take<T, kV, kL, kNV>(x + (r * groups + at.g) * n, at.lane, n, r < rows, raw[j]);
        }
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            const int64_t r = r0 + j * at.step, row = r * groups + at.g;
            float v[kE], s = 0.f, q = 0.f;
#pragma unroll
            for (int u = 0; u < kE; ++u) {
                v[u] = to_f32(raw[j][u]);
                s += v[u];
            }
            const float mu = lane_sum<kL>(s) * inv;
#pragma unroll
            for (int u = 0; u < kE; ++u) {
                v[u] -= mu;
                const float e = (u / kV * kL + at.lane) * kV < n ? v[u] : 0.f;
                q = fmaf(e, e, q);
            }
            const float rs = 1.f / sqrtf(lane_sum<kL>(q) * inv + eps);
            if (r < rows) {
                if (at.lane == 0) {
                    if (mean) mean[row] = mu;
                    if (rstd) rstd[row] = rs;
                }
#pragma unroll
                for (int u = 0; u < kE; ++u) v[u] = fmaf(v[u] * rs, wr[u], br[u]);
#pragma unroll
                for (int k = 0; k < kNV; ++k) {
                    const int c = (k * kL + at.lane) * kV;
                    if (c < n) store<T, kV>(y + row * n + c, v + k * kV);
                }
            }
        }
    }
}

template <typename T, int kV, int kL, int kNV>
__global__ void __launch_bounds__(kThreads, 2)
rows_bwd_kernel(const T *dy, const T *x, const float *w, const float *mean, const float *rstd, T *dx, float *part,
                int64_t rows, int groups, int n) {
    dependency_release();
    constexpr int kE = kV * kNV, kR = rows_at_once<kE>();
    const Walk at(groups, kL);
    float wr[kE], dw[kE], db[kE];
#pragma unroll
    for (int u = 0; u < kE; ++u) {
        const int c = (u / kV * kL + at.lane) * kV + u % kV;
        wr[u] = w && c < n ? w[static_cast<int64_t>(at.g) * n + c] : 1.f;
        dw[u] = db[u] = 0.f;
    }
    const float inv = 1.f / n;
    const int64_t block0 = at.first - threadIdx.x / kL;
    for (int64_t r0 = at.first; r0 - at.first + block0 < rows; r0 += kR * at.step) {
        alignas(16) T rx[kR][kE], rd[kR][kE];
        float mu[kR], rs[kR];
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            const int64_t r = r0 + j * at.step, row = r * groups + at.g;
            const bool live = r < rows;
            take<T, kV, kL, kNV>(x + row * n, at.lane, n, live, rx[j]);
            take<T, kV, kL, kNV>(dy + row * n, at.lane, n, live, rd[j]);
            mu[j] = live ? mean[row] : 0.f;
            rs[j] = live ? rstd[row] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            const int64_t r = r0 + j * at.step, row = r * groups + at.g;
            float xh[kE], d[kE];
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int u = 0; u < kE; ++u) {   // columns past n, and rows past the last, have d = 0 and add nothing
                xh[u] = (to_f32(rx[j][u]) - mu[j]) * rs[j];
                d[u] = to_f32(rd[j][u]);
                dw[u] = fmaf(d[u], xh[u], dw[u]);
                db[u] += d[u];
                d[u] *= wr[u];
                s.x += d[u];
                s.y = fmaf(d[u], xh[u], s.y);
            }
            s = lane_sum<kL>(s);
            if (r < rows) {
                const float p1 = -rs[j] * s.x * inv, p2 = -rs[j] * s.y * inv;
#pragma unroll
                for (int u = 0; u < kE; ++u) xh[u] = fmaf(rs[j], d[u], fmaf(p2, xh[u], p1));
#pragma unroll
                for (int k = 0; k < kNV; ++k) {
                    const int c = (k * kL + at.lane) * kV;
                    if (c < n) store<T, kV>(dx + row * n + c, xh + k * kV);
                }
            }
        }
    }
    if (!part) return;
    // one partial row of dw and of db per CTA
    float *pw = part + static_cast<int64_t>(blockIdx.x) * 2 * n;
    __shared__ float acc[kThreads * kE];   // [team][column]
    constexpr int kTeams = kThreads / kL, kCols = kL * kE;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kE; ++u)
            acc[threadIdx.x / kL * kCols + (u / kV * kL + at.lane) * kV + u % kV] = pass ? db[u] : dw[u];
        __syncthreads();
        for (int c = threadIdx.x; c < n; c += kThreads) {
            float s = 0.f;
#pragma unroll 8
            for (int q = 0; q < kTeams; ++q) s += acc[q * kCols + c];
            pw[pass * n + c] = s;
        }
    }
}

// Calls f with the narrowest team that holds n values, kV at a time.
template <int kV_, int kL_, int kNV_>
struct Shape {
    static constexpr int kV = kV_, kL = kL_, kNV = kNV_;
};
template <typename T, typename F>
void by_shape(int n, int width, F f) {
    constexpr int kFull = 16 / sizeof(T);
    const int need = (n + width - 1) / width;   // accesses
    if (width == kFull) {
        if (need <= 2) f(Shape<kFull, 2, 1>{});
        else if (need <= 4) f(Shape<kFull, 4, 1>{});
        else if (need <= 8) f(Shape<kFull, 8, 1>{});
        else if (need <= 16) f(Shape<kFull, 16, 1>{});
        else if (need <= 32) f(Shape<kFull, 32, 1>{});
        else if (sizeof(T) == 2 || need <= 64) f(Shape<kFull, 32, 2>{});
        else if constexpr (sizeof(T) == 4) f(Shape<4, 32, 4>{});
    } else if (sizeof(T) == 2 && width == 2) {
        if constexpr (sizeof(T) == 2) {
            if (need <= 16) f(Shape<2, 16, 1>{});
            else if (need <= 64) f(Shape<2, 32, 2>{});
            else if (need <= 128) f(Shape<2, 32, 4>{});
            else f(Shape<2, 32, 8>{});
        }
    } else {
        if (need <= 16) f(Shape<1, 16, 1>{});
        else if (need <= 64) f(Shape<1, 32, 2>{});
        else if (need <= 128) f(Shape<1, 32, 4>{});
        else if (need <= 256) f(Shape<1, 32, 8>{});
        else f(Shape<1, 32, 16>{});
    }
}

}  // namespace

static int grid_of(int64_t rows, int groups, int per_sm) {
    constexpr int kSms = 152;
    const int64_t most = (rows + 7) / 8;   // of a group: the widest teams, eight a CTA, have a row each
    int64_t want = (static_cast<int64_t>(kSms) * per_sm + groups - 1) / groups;
    if (want > most) want = most;
    if (want < 1) want = 1;
    return static_cast<int>(want * groups);
}
int norm_rows_bwd_grid(int64_t rows, int groups) { return grid_of(rows, groups, 2); }

template <typename T>
static cudaError_t fwd_typed(const void *x, const float *w, const float *b, void *y, float *mean, float *rstd,
                             int64_t rows, int groups, int n, int width, float eps, cudaStream_t s) {
    by_shape<T>(n, width, [&](auto shape) {
        using S = decltype(shape);
        const int grid = grid_of(rows, groups, fwd_ctas(S::kV * S::kNV));
        rows_fwd_kernel<T, S::kV, S::kL, S::kNV><<<grid, kThreads, 0, s>>>(
            static_cast<const T *>(x), w, b, static_cast<T *>(y), mean, rstd, rows, groups, n, eps);
    });
    return cudaGetLastError();
}
template <typename T>
static cudaError_t bwd_typed(const void *dy, const void *x, const float *w, const float *mean, const float *rstd,
                             void *dx, float *part, int64_t rows, int groups, int n, int width, cudaStream_t s) {
    const int grid = norm_rows_bwd_grid(rows, groups);
    by_shape<T>(n, width, [&](auto shape) {
        using S = decltype(shape);
        rows_bwd_kernel<T, S::kV, S::kL, S::kNV><<<grid, kThreads, 0, s>>>(
            static_cast<const T *>(dy), static_cast<const T *>(x), w, mean, rstd, static_cast<T *>(dx), part, rows,
            groups, n);
    });
    return cudaGetLastError();
}

cudaError_t norm_rows_fwd(const void *x, const float *w, const float *b, void *y, float *mean, float *rstd,
                          int64_t rows, int groups, int n, kla_dtype dtype, int width, float eps, cudaStream_t s) {
    return dtype == KLA_DTYPE_BF16
               ? fwd_typed<__nv_bfloat16>(x, w, b, y, mean, rstd, rows, groups, n, width, eps, s)
               : fwd_typed<float>(x, w, b, y, mean, rstd, rows, groups, n, width, eps, s);
}
cudaError_t norm_rows_bwd(const void *dy, const void *x, const float *w, const float *mean, const float *rstd,
                          void *dx, float *part, int64_t rows, int groups, int n, kla_dtype dtype, int width,
                          cudaStream_t s) {
    return dtype == KLA_DTYPE_BF16
               ? bwd_typed<__nv_bfloat16>(dy, x, w, mean, rstd, dx, part, rows, groups, n, width, s)
               : bwd_typed<float>(dy, x, w, mean, rstd, dx, part, rows, groups, n, width, s);
}

}  // namespace kla
