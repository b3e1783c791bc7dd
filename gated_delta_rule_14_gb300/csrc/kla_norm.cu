// kla_norm.cu -- layer norm over the last axis of [rows, groups, n], forward and gradients.
//
//   forward    y = xh w[g] + b[g],  xh = (x - mean) rstd
//   backward   dx = rstd (u - mean(u) - xh mean(u xh)),  u = dy w[g];  dw[g] = sum dy xh;  db[g] = sum dy
//
// Every value is read once and stays in registers: a row belongs to one team of threads (16 or 32
// lanes, or a whole CTA), each with kE values at fixed columns. Teams are persistent and keep to one
// group, so that weight and bias, and in the backward pass the sums of dw and db, stay in registers
// too; the sums leave as one partial row per CTA and a second launch adds those in a fixed order.
// Rows longer than a CTA's registers (n > 16384) are walked in pieces of that size.
#include <climits>

#include "kla_internal.cuh"
#include "../../include/kla_layer.h"

namespace kla {
namespace {

constexpr int kSms = 152;
constexpr int kE = 16;                 // values of one thread
constexpr int kMaxBlock = 1024;
constexpr int kHeld = kE * kMaxBlock;  // longest row held in registers

// kV consecutive values of type T at p as fp32; one access.
template <typename T, int kV>
__device__ __forceinline__ void load(const T *p, float *x) {
    if constexpr (sizeof(T) * kV == 16) {
        const uint4 r = *reinterpret_cast<const uint4 *>(p);
        const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
        for (int i = 0; i < kV; ++i) x[i] = to_f32(e[i]);
    } else if constexpr (sizeof(T) * kV == 4 && kV == 2) {
        const uint32_t r = *reinterpret_cast<const uint32_t *>(p);
        const T *e = reinterpret_cast<const T *>(&r);
        x[0] = to_f32(e[0]);
        x[1] = to_f32(e[1]);
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) x[i] = to_f32(p[i]);
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
    } else if constexpr (sizeof(T) * kV == 4 && kV == 2) {
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

// Sum over the row's team: kTeam lanes of a warp, or the CTA (kTeam = 0), where two buffers let
// one barrier a sum do.
template <int kTeam>
struct TeamSum {
    int turn = 0;
    __device__ __forceinline__ float2 operator()(float2 v) {
        constexpr int kLanes = kTeam ? kTeam : 32;
#pragma unroll
        for (int off = kLanes / 2; off; off >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
        }
        if constexpr (kTeam == 0) {
            __shared__ float2 part[2][kMaxBlock / 32];
            const int nw = blockDim.x / 32;
            if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x / 32] = v;
            __syncthreads();
            v = make_float2(0.f, 0.f);
            for (int w = 0; w < nw; ++w) {
                v.x += part[turn][w].x;
                v.y += part[turn][w].y;
            }
            turn ^= 1;
        }
        return v;
    }
};

// Which rows a thread's team walks: rows first, first + step, .. of group g.
template <int kTeam>
struct Walk {
    int lane, width, g;
    int64_t first, step;
    __device__ Walk(int groups) {
        const int parts = gridDim.x / groups;
        g = blockIdx.x % groups;
        width = kTeam ? kTeam : blockDim.x;
        lane = kTeam ? threadIdx.x % kTeam : threadIdx.x;
        const int teams = kTeam ? blockDim.x / kTeam : 1;
        first = static_cast<int64_t>(blockIdx.x / groups) * teams + (kTeam ? threadIdx.x / kTeam : 0);
        step = static_cast<int64_t>(parts) * teams;
    }
};

template <typename T, int kV, int kTeam>
__global__ void __launch_bounds__(kTeam ? 256 : kMaxBlock)
norm_fwd_kernel(const T *x, const float *w, const float *b, T *y, float *mean, float *rstd, int64_t rows, int groups,
                int n, float eps) {
    constexpr int kK = kE / kV;
    const Walk<kTeam> at(groups);
    TeamSum<kTeam> sum;
    float wr[kE], br[kE];
#pragma unroll
    for (int k = 0; k < kK; ++k)
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int c = (k * at.width + at.lane) * kV + i;
            wr[k * kV + i] = w && c < n ? w[static_cast<int64_t>(at.g) * n + c] : 1.f;
            br[k * kV + i] = b && c < n ? b[static_cast<int64_t>(at.g) * n + c] : 0.f;
        }
    // every lane of a warp takes the same number of turns (the sums use whole warps)
    const int64_t turns = (rows + at.step - 1) / at.step;
    const float inv = 1.f / n;
    for (int64_t t = 0; t < turns; ++t) {
        const int64_t r = at.first + t * at.step;
        const bool live = r < rows;
        const int64_t row = r * groups + at.g;
        const T *xr = x + row * n;
        float v[kE];
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const int c = (k * at.width + at.lane) * kV;
#pragma unroll
            for (int i = 0; i < kV; ++i) v[k * kV + i] = 0.f;
            if (live && c < n) load<T, kV>(xr + c, v + k * kV);
        }
#pragma unroll
        for (int i = 0; i < kE; ++i) s += v[i];
        const float mu = sum(make_float2(s, 0.f)).x * inv;
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < kK; ++k)
            if ((k * at.width + at.lane) * kV < n)
#pragma unroll
                for (int i = 0; i < kV; ++i) {
                    const float d = v[k * kV + i] - mu;
                    q = fmaf(d, d, q);
                }
        const float rs = 1.f / sqrtf(sum(make_float2(q, 0.f)).x * inv + eps);
        if (!live) continue;
        if (at.lane == 0) {
            if (mean) mean[row] = mu;
            if (rstd) rstd[row] = rs;
        }
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const int c = (k * at.width + at.lane) * kV;
            if (c < n) {
                float o[kV];
#pragma unroll
                for (int i = 0; i < kV; ++i) o[i] = fmaf((v[k * kV + i] - mu) * rs, wr[k * kV + i], br[k * kV + i]);
                store<T, kV>(y + row * n + c, o);
            }
        }
    }
}

template <typename T, int kV, int kTeam>
__global__ void __launch_bounds__(kTeam ? 256 : kMaxBlock)
norm_bwd_kernel(const T *dy, const T *x, const float *w, const float *mean, const float *rstd, T *dx, float *part,
                int64_t rows, int groups, int n) {
    constexpr int kK = kE / kV;
    const Walk<kTeam> at(groups);
    TeamSum<kTeam> sum;
    float wr[kE], dw[kE], db[kE];
#pragma unroll
    for (int k = 0; k < kK; ++k)
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int c = (k * at.width + at.lane) * kV + i;
            wr[k * kV + i] = w && c < n ? w[static_cast<int64_t>(at.g) * n + c] : 1.f;
            dw[k * kV + i] = db[k * kV + i] = 0.f;
        }
    const int64_t turns = (rows + at.step - 1) / at.step;
    const float inv = 1.f / n;
    for (int64_t t = 0; t < turns; ++t) {
        const int64_t r = at.first + t * at.step;
        const bool live = r < rows;
        const int64_t row = r * groups + at.g;
        float xh[kE], d[kE];
#pragma unroll
        for (int i = 0; i < kE; ++i) xh[i] = d[i] = 0.f;
        float mu = 0.f, rs = 0.f;
        if (live) {
            mu = mean[row];
            rs = rstd[row];
        }
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const int c = (k * at.width + at.lane) * kV;
            if (live && c < n) {
                load<T, kV>(x + row * n + c, xh + k * kV);
                load<T, kV>(dy + row * n + c, d + k * kV);
            }
        }
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kK; ++k)
            if ((k * at.width + at.lane) * kV < n)
#pragma unroll
                for (int i = k * kV; i < k * kV + kV; ++i) {
                    xh[i] = (xh[i] - mu) * rs;
                    dw[i] = fmaf(d[i], xh[i], dw[i]);
                    db[i] += d[i];
                    d[i] *= wr[i];
                    s.x += d[i];
                    s.y = fmaf(d[i], xh[i], s.y);
                }
        s = sum(s);
        if (!live) continue;
        s.x *= inv;
        s.y *= inv;
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const int c = (k * at.width + at.lane) * kV;
            if (c < n) {
                float o[kV];
#pragma unroll
                for (int i = 0; i < kV; ++i) o[i] = rs * (d[k * kV + i] - s.x - xh[k * kV + i] * s.y);
                store<T, kV>(dx + row * n + c, o);
            }
        }
    }
    if (!part) return;
    // one partial row of dw and of db per CTA
    float *pw = part + static_cast<int64_t>(blockIdx.x) * 2 * n, *pb = pw + n;
    if constexpr (kTeam == 0) {
#pragma unroll
        for (int k = 0; k < kK; ++k)
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const int c = (k * at.width + at.lane) * kV + i;
                if (c < n) {
                    pw[c] = dw[k * kV + i];
                    pb[c] = db[k * kV + i];
                }
            }
    } else {
        __shared__ float acc[256 * kE];   // [team][column]
        constexpr int kTeams = 256 / kTeam, kCols = kTeam * kE;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kK; ++k)
#pragma unroll
                for (int i = 0; i < kV; ++i)
                    acc[threadIdx.x / kTeam * kCols + (k * kTeam + at.lane) * kV + i] =
                        pass ? db[k * kV + i] : dw[k * kV + i];
            __syncthreads();
            for (int c = threadIdx.x; c < n; c += 256) {
                float s = 0.f;
#pragma unroll
                for (int q = 0; q < kTeams; ++q) s += acc[q * kCols + c];
                (pass ? pb : pw)[c] = s;
            }
        }
    }
}

// dweight and dbias of group blockIdx.y, 32 columns a CTA: 8 rows of threads walk the partial rows
// in a fixed order.
__global__ void __launch_bounds__(256) norm_sum_kernel(const float *part, float *dw, float *db, int parts, int groups,
                                                       int n) {
    __shared__ float sw[8][33], sb[8][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x / 32, g = blockIdx.y;
    float a = 0.f, b = 0.f;
    if (c < n)
        for (int p = r; p < parts; p += 8) {
            const float *row = part + (static_cast<int64_t>(p) * groups + g) * 2 * n;
            a += row[c];
            b += row[n + c];
        }
    sw[r][threadIdx.x & 31] = a;
    sb[r][threadIdx.x & 31] = b;
    __syncthreads();
    if (r == 0 && c < n) {
        for (int q = 1; q < 8; ++q) {
            a += sw[q][threadIdx.x];
            b += sb[q][threadIdx.x];
        }
        if (dw) dw[static_cast<int64_t>(g) * n + c] = a;
        if (db) db[static_cast<int64_t>(g) * n + c] = b;
    }
}

// ---- rows longer than kHeld: pieces of the row per thread, read again for each use
template <typename T>
__global__ void __launch_bounds__(kMaxBlock) norm_fwd_long_kernel(const T *x, const float *w, const float *b, T *y,
                                                                  float *mean, float *rstd, int groups, int n,
                                                                  float eps) {
    TeamSum<0> sum;
    const int64_t row = blockIdx.x;
    const int64_t g = row % groups;
    const T *xr = x + row * n;
    float s = 0.f, q = 0.f;
    for (int c = threadIdx.x; c < n; c += kMaxBlock) s += to_f32(xr[c]);
    const float mu = sum(make_float2(s, 0.f)).x / n;
    for (int c = threadIdx.x; c < n; c += kMaxBlock) {
        const float d = to_f32(xr[c]) - mu;
        q = fmaf(d, d, q);
    }
    const float rs = 1.f / sqrtf(sum(make_float2(q, 0.f)).x / n + eps);
    if (threadIdx.x == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
    }
    for (int c = threadIdx.x; c < n; c += kMaxBlock) {
        const float o = (to_f32(xr[c]) - mu) * rs;
        y[row * n + c] = from_f32<T>(fmaf(o, w ? w[g * n + c] : 1.f, b ? b[g * n + c] : 0.f));
    }
}

template <typename T>
__global__ void __launch_bounds__(kMaxBlock) norm_bwd_long_kernel(const T *dy, const T *x, const float *w,
                                                                  const float *mean, const float *rstd, T *dx,
                                                                  float *part, int64_t rows, int groups, int n) {
    TeamSum<0> sum;
    const Walk<0> at(groups);
    float *pw = part ? part + static_cast<int64_t>(blockIdx.x) * 2 * n : nullptr;
    if (pw)
        for (int c = threadIdx.x; c < 2 * n; c += kMaxBlock) pw[c] = 0.f;
    __syncthreads();
    for (int64_t r = at.first; r < rows; r += at.step) {
        const int64_t row = r * groups + at.g;
        const float mu = mean[row], rs = rstd[row];
        float2 s = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < n; c += kMaxBlock) {
            const float d = to_f32(dy[row * n + c]), xh = (to_f32(x[row * n + c]) - mu) * rs;
            const float u = d * (w ? w[static_cast<int64_t>(at.g) * n + c] : 1.f);
            s.x += u;
            s.y = fmaf(u, xh, s.y);
            if (pw) {   // a column belongs to one thread
                pw[c] = fmaf(d, xh, pw[c]);
                pw[n + c] += d;
            }
        }
        s = sum(s);
        s.x /= n;
        s.y /= n;
        for (int c = threadIdx.x; c < n; c += kMaxBlock) {
            const float d = to_f32(dy[row * n + c]), xh = (to_f32(x[row * n + c]) - mu) * rs;
            const float u = d * (w ? w[static_cast<int64_t>(at.g) * n + c] : 1.f);
            dx[row * n + c] = from_f32<T>(rs * (u - s.x - xh * s.y));
        }
    }
}

// ------------------------------------------------------------------------------------ host side
struct Plan {
    int team;      // 16, 32, or 0 for the CTA
    int block, grid;
    bool held;
};

// The smallest team whose registers hold the row; CTAs for every SM a few times over, a multiple of
// the groups, none without a row.
Plan plan(int64_t rows, int groups, int n) {
    Plan p{};
    p.held = n <= kHeld;
    p.team = n <= 16 * kE ? 16 : n <= 32 * kE ? 32 : 0;
    p.block = p.team ? 256 : p.held ? (((n + kE - 1) / kE + 31) / 32) * 32 : kMaxBlock;
    const int64_t per_cta = p.team ? 256 / p.team : 1;
    const int64_t most = (rows + per_cta - 1) / per_cta;   // CTAs of one group
    int64_t want = (static_cast<int64_t>(kSms) * 1024 / p.block + groups - 1) / groups;
    if (want > most) want = most;
    if (want < 1) want = 1;
    p.grid = static_cast<int>(want * groups);
    return p;
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

kla_status check(int64_t rows, int groups, int n, kla_dtype dtype) {
    if (rows < 0 || groups < 1 || n < 1) return KLA_ERR_INVALID_ARG;
    if (dtype != KLA_DTYPE_F32 && dtype != KLA_DTYPE_BF16) return KLA_ERR_INVALID_ARG;
    // rows of one or two values: dx is eps alone, left over from terms that cancel in fp32
    if (n < 3 || n > 65536 || groups > 65535 || rows * groups > INT_MAX) return KLA_ERR_UNSUPPORTED;
    return KLA_OK;
}

// The widest access that every row start allows: 16 bytes, a bf16 pair, or one value.
template <typename T>
int width(int n, const void *a, const void *b, const void *c) {
    constexpr int kFull = 16 / sizeof(T);
    auto fits = [&](int v) {
        const uintptr_t bytes = v * sizeof(T);
        return n % v == 0 && aligned(a, bytes) && aligned(b, bytes) && aligned(c, bytes);
    };
    return fits(kFull) ? kFull : sizeof(T) == 2 && fits(2) ? 2 : 1;
}

template <typename T, int kV>
void run_fwd(const Plan &p, const T *x, const float *w, const float *b, T *y, float *mean, float *rstd, int64_t rows,
             int groups, int n, float eps, cudaStream_t s) {
    if (p.team == 16)
        norm_fwd_kernel<T, kV, 16><<<p.grid, p.block, 0, s>>>(x, w, b, y, mean, rstd, rows, groups, n, eps);
    else if (p.team == 32)
        norm_fwd_kernel<T, kV, 32><<<p.grid, p.block, 0, s>>>(x, w, b, y, mean, rstd, rows, groups, n, eps);
    else
        norm_fwd_kernel<T, kV, 0><<<p.grid, p.block, 0, s>>>(x, w, b, y, mean, rstd, rows, groups, n, eps);
}
template <typename T, int kV>
void run_bwd(const Plan &p, const T *dy, const T *x, const float *w, const float *mean, const float *rstd, T *dx,
             float *part, int64_t rows, int groups, int n, cudaStream_t s) {
    if (p.team == 16)
        norm_bwd_kernel<T, kV, 16><<<p.grid, p.block, 0, s>>>(dy, x, w, mean, rstd, dx, part, rows, groups, n);
    else if (p.team == 32)
        norm_bwd_kernel<T, kV, 32><<<p.grid, p.block, 0, s>>>(dy, x, w, mean, rstd, dx, part, rows, groups, n);
    else
        norm_bwd_kernel<T, kV, 0><<<p.grid, p.block, 0, s>>>(dy, x, w, mean, rstd, dx, part, rows, groups, n);
}

template <typename T>
void fwd_as(const void *xv, const float *w, const float *b, void *yv, float *mean, float *rstd, int64_t rows,
            int groups, int n, float eps, cudaStream_t s) {
    const T *x = static_cast<const T *>(xv);
    T *y = static_cast<T *>(yv);
    const Plan p = plan(rows, groups, n);
    const int v = width<T>(n, x, y, y);
    if (!p.held)
        norm_fwd_long_kernel<T><<<static_cast<int>(rows * groups), kMaxBlock, 0, s>>>(x, w, b, y, mean, rstd, groups,
                                                                                     n, eps);
    else if (v == 16 / sizeof(T))
        run_fwd<T, 16 / sizeof(T)>(p, x, w, b, y, mean, rstd, rows, groups, n, eps, s);
    else if (sizeof(T) == 2 && v == 2)
        run_fwd<T, sizeof(T) == 2 ? 2 : 1>(p, x, w, b, y, mean, rstd, rows, groups, n, eps, s);
    else
        run_fwd<T, 1>(p, x, w, b, y, mean, rstd, rows, groups, n, eps, s);
}
template <typename T>
void bwd_as(const void *dyv, const void *xv, const float *w, const float *mean, const float *rstd, void *dxv,
            float *part, int64_t rows, int groups, int n, cudaStream_t s) {
    const T *dy = static_cast<const T *>(dyv), *x = static_cast<const T *>(xv);
    T *dx = static_cast<T *>(dxv);
    const Plan p = plan(rows, groups, n);
    const int v = width<T>(n, x, dy, dx);
    if (!p.held)
        norm_bwd_long_kernel<T><<<p.grid, kMaxBlock, 0, s>>>(dy, x, w, mean, rstd, dx, part, rows, groups, n);
    else if (v == 16 / sizeof(T))
        run_bwd<T, 16 / sizeof(T)>(p, dy, x, w, mean, rstd, dx, part, rows, groups, n, s);
    else if (sizeof(T) == 2 && v == 2)
        run_bwd<T, sizeof(T) == 2 ? 2 : 1>(p, dy, x, w, mean, rstd, dx, part, rows, groups, n, s);
    else
        run_bwd<T, 1>(p, dy, x, w, mean, rstd, dx, part, rows, groups, n, s);
}

}  // namespace
}  // namespace kla

extern "C" {

kla_status kla_layer_norm_fwd(const void *x, const float *weight, const float *bias, void *y, float *mean,
                              float *rstd, int64_t rows, int groups, int n, kla_dtype dtype, float eps,
                              void *stream) {
    using namespace kla;
    const kla_status st = check(rows, groups, n, dtype);
    if (st != KLA_OK) return st;
    if (!(eps >= 0.f) || eps - eps != 0.f) return KLA_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !y)) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x, esz) || !aligned(y, esz) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return KLA_ERR_INVALID_ARG;
    const size_t stat = static_cast<size_t>(rows) * groups * 4, all = stat / 4 * n * esz, par = 4ull * groups * n;
    const Span outs[] = {span(y, all), span(mean, stat), span(rstd, stat)};
    const Span ins[] = {span(x, all), span(weight, par), span(bias, par)};
    for (int i = 0; i < 3; ++i) {
        for (const Span &s : ins)
            if (overlaps(outs[i], s)) return KLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(outs[i], outs[j])) return KLA_ERR_INVALID_ARG;
    }
    if (rows == 0) return KLA_OK;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (dtype == KLA_DTYPE_BF16)
        fwd_as<__nv_bfloat16>(x, weight, bias, y, mean, rstd, rows, groups, n, eps, cs);
    else
        fwd_as<float>(x, weight, bias, y, mean, rstd, rows, groups, n, eps, cs);
    return cudaGetLastError() == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

size_t kla_layer_norm_bwd_workspace_size(int64_t rows, int groups, int n, kla_dtype dtype) {
    if (kla::check(rows, groups, n, dtype) != KLA_OK || rows == 0) return 0;
    return static_cast<size_t>(kla::plan(rows, groups, n).grid) * 2 * n * sizeof(float);
}

kla_status kla_layer_norm_bwd(const void *dy, const void *x, const float *weight, const float *mean,
                              const float *rstd, void *dx, float *dweight, float *dbias, int64_t rows, int groups,
                              int n, kla_dtype dtype, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace kla;
    const kla_status st = check(rows, groups, n, dtype);
    if (st != KLA_OK) return st;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x, esz) || !aligned(dy, esz) || !aligned(dx, esz) || !aligned(weight, 4) || !aligned(mean, 4) ||
        !aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(workspace, 16))
        return KLA_ERR_INVALID_ARG;
    const bool sums = dweight || dbias;
    const size_t need = sums ? kla_layer_norm_bwd_workspace_size(rows, groups, n, dtype) : 0;
    if (workspace_bytes < need || (need > 0 && !workspace)) return KLA_ERR_INVALID_ARG;
    const size_t stat = static_cast<size_t>(rows) * groups * 4, all = stat / 4 * n * esz, par = 4ull * groups * n;
    const Span outs[] = {span(dx, all), span(dweight, par), span(dbias, par), span(workspace, need)};
    const Span ins[] = {span(x, all), span(dy, all), span(weight, par), span(mean, stat), span(rstd, stat)};
    for (int i = 0; i < 4; ++i) {
        for (const Span &s : ins)
            if (overlaps(outs[i], s)) return KLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(outs[i], outs[j])) return KLA_ERR_INVALID_ARG;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (rows == 0) {   // no rows: the sums are empty
        if ((dweight && cudaMemsetAsync(dweight, 0, par, cs) != cudaSuccess) ||
            (dbias && cudaMemsetAsync(dbias, 0, par, cs) != cudaSuccess))
            return KLA_ERR_CUDA;
        return KLA_OK;
    }
    float *part = sums ? static_cast<float *>(workspace) : nullptr;
    if (dtype == KLA_DTYPE_BF16)
        bwd_as<__nv_bfloat16>(dy, x, weight, mean, rstd, dx, part, rows, groups, n, cs);
    else
        bwd_as<float>(dy, x, weight, mean, rstd, dx, part, rows, groups, n, cs);
    if (cudaGetLastError() != cudaSuccess) return KLA_ERR_CUDA;
    if (!sums) return KLA_OK;
    norm_sum_kernel<<<dim3((n + 31) / 32, groups), 256, 0, cs>>>(part, dweight, dbias,
                                                                 plan(rows, groups, n).grid / groups, groups, n);
    return cudaGetLastError() == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // extern "C"
