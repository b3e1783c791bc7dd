// kla_linear.cu -- linear attention with one decay per head: the C entry points, the fp32 scan for
// every size, type and stride, and the single-token step.
//
// The recurrence S_t = g S_{t-1} + k_t v_t^T needs no solve: a chunk's own contribution to the
// state and its products among its own tokens do not depend on the state that enters it, so chunks
// only meet in S' = g^n S + Z. Long sequences with few heads are therefore cut into segments: one
// launch takes each segment's own Z from a zero state, an elementwise pass turns the Z into start
// states, and the second launch writes the outputs. All powers of g have exponents >= 0.
#include <climits>

#include "kla_linear.cuh"

namespace kla {

namespace {

constexpr int kC = 64;        // tokens per chunk
constexpr int kThreads = 256;
constexpr int kPitch = kC + 4;   // rows of 64 floats, 16-byte aligned, one bank group apart

struct Scans {   // up to three scans of one shape in one launch, by blockIdx.z
    LinScan s[3];
};

__device__ __forceinline__ size_t s_index(const LinScan &p, int chain, int d, int z) {
    return static_cast<size_t>(chain) * p.dx * p.dz +
           (p.s_t ? static_cast<size_t>(z) * p.dx + d : static_cast<size_t>(d) * p.dz + z);
}

// Four consecutive values as fp32, in one access where `whole`.
__device__ __forceinline__ void four(const float *p, bool whole, float (&x)[4]) {
    if (whole) {
        const float4 v = *reinterpret_cast<const float4 *>(p);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = p[u];
    }
}
__device__ __forceinline__ void four(const __nv_bfloat16 *p, bool whole, float (&x)[4]) {
    if (whole) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = to_f32(p[u]);
    }
}
// Whether every row of a tensor can be read four values at a time.
template <typename T>
__device__ __forceinline__ bool fours(const T *p, const int64_t (&st)[3]) {
    return ((reinterpret_cast<uintptr_t>(p) / sizeof(T)) | st[0] | st[1] | st[2]) % 4 == 0;
}

// kN consecutive floats of shared memory.
template <int kN>
__device__ __forceinline__ void take(const float *p, float (&x)[kN]) {
    if constexpr (kN % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kN; i += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + i);
            x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i] = p[i];
    }
}

// fp32 scan of one segment of one (sequence, head) and kZ value channels, chunk by chunk. Bound by the
// fp32 pipe: each of the products (X Y^T, P Z, X S and Y^T Z) is a 16 x 16 grid of threads with a tile of
// registers each, fed with 16-byte loads from operands laid out along the tile (X and Y transposed; P takes Y's
// place), one load for eight to eleven multiply-adds. `states`: only the segment's own contribution, from zero.
// Measured, 2 x 1000 tokens of 4 heads of 64, cut into one chunk a CTA: forward 32 us, backward 62 us, in three
// launches each that are one chunk's chain of loads and barriers long; 8 x 1024 tokens of 16 heads of 128: 575 and
// 1680 us, a third of the fp32 pipe's rate. Y in both orders, P beside it, X read once for each of its products and the
// last chunk's state always taken took 34, 64, 653 and 1932; registers for three CTAs an SM of the 64 x 64 tiles
// (80, some spilled) 593 for 8 x 2048 tokens of 16 heads, which took 443 then and take 410 now.
template <int kX, int kZ>
constexpr int kScanFloats = (kX + (kX > kC ? kX : kC)) * kPitch + (kC + kX) * (kZ + 4) + kC + 1;

constexpr int scan_ctas(int x, int z) { return x < 128 || z < 64 ? 2 : 1; }   // an SM's shared memory holds

template <typename T, int kX, int kZ>
__global__ void __launch_bounds__(kThreads, scan_ctas(kX, kZ)) lin_scan_kernel(const __grid_constant__ Scans all, const int states) {
    constexpr int kR = kX / 16, kU = kZ / 16;   // state rows and columns of a thread
    constexpr int kZp = kZ + 4;
    extern __shared__ __align__(16) float sm[];
    float *Xt = sm;                    // [x][token]
    float *Yt = Xt + kX * kPitch;      // [x][token]
    float *Pt = Yt;                    // [column][row], once Y is used up
    float *Z = Yt + (kX > kC ? kX : kC) * kPitch;   // [token][z]
    float *S = Z + kC * kZp;           // [x][z]
    float *gp = S + kX * kZp;          // g^0 .. g^kC
    const LinScan &p = all.s[blockIdx.z];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, nz = p.dz / kZ;
    const int chain = blockIdx.x / nz, z0 = (blockIdx.x % nz) * kZ, seg = blockIdx.y;
    const int b = chain / p.H, h = chain % p.H;
    const int n = lin_length(p.lengths, b, p.T);
    int t_begin;
    const int valid = lin_segment(p, seg, n, t_begin);
    const int t_stop = min(p.T, t_begin + p.seg_len);   // outputs past `valid` are zeros
    const bool reverse = p.reverse;
    if (tid <= kC) gp[tid] = powf(p.decay[h], static_cast<float>(tid));
    dependency_release();
    dependency_wait();   // the start states

    float s[kR][kU];   // state rows ty * kR .., columns tx * kU ..
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int d = ty * kR + r, z = z0 + tx * kU + u;
            s[r][u] = 0.f;
            if (!states && p.nseg > 1)
                s[r][u] = p.seg_states[lin_slot(p, chain, lin_start_slot(p, seg)) + d * p.dz + z];
            else if (!states && p.S0)
                s[r][u] = p.S0[s_index(p, chain, d, z)];
        }
    const T *xg = static_cast<const T *>(p.x) + b * p.xs[0] + h * p.xs[2];
    const T *yg = static_cast<const T *>(p.y) + b * p.ys[0] + h * p.ys[2];
    const T *zg = static_cast<const T *>(p.z) + b * p.zs[0] + h * p.zs[2] + z0;
    T *og = static_cast<T *>(p.out) + (static_cast<size_t>(b) * p.T * p.H + h) * p.dz + z0;
    const bool xw = fours(static_cast<const T *>(p.x), p.xs), yw = fours(static_cast<const T *>(p.y), p.ys);
    const bool zw = fours(static_cast<const T *>(p.z), p.zs);
    const int64_t x_step = p.xs[1], y_step = p.ys[1], z_step = p.zs[1], o_step = static_cast<int64_t>(p.H) * p.dz;
    const float a_intra = p.a_intra, a_inter = p.a_inter, a_upd = p.a_upd;

    const int nchunk = (t_stop - t_begin + kC - 1) / kC;
    const bool wanted = p.ST && seg == p.nseg - 1;
    for (int ci = 0; ci < nchunk; ++ci) {
        const int c = reverse ? nchunk - 1 - ci : ci;
        const int t0 = t_begin + c * kC;
        const int cnt = max(0, min(kC, t_begin + valid - t0));   // valid tokens of the chunk
        if (states && cnt == 0) continue;
        __syncthreads();
        // Masked tokens become zeros. Every load is made, of a valid token where there is any, so that all of a
        // thread's are on their way at once (with a condition on each, 15 us went by for one chunk's state).
        const int most = cnt - 1;
        constexpr int kNx = kC * kX / 4 / kThreads, kNz = kC * kZ / 4 / kThreads;
        float x[kNx][4] = {}, y[kNx][4] = {}, v[kNz][4] = {};
        if (cnt > 0) {
            if (!states)
#pragma unroll
                for (int q = 0; q < kNx; ++q) {
                    const int i = tid + q * kThreads, t = i % kC, d = i / kC * 4;
                    four(xg + (t0 + min(t, most)) * x_step + d, xw, x[q]);
                }
#pragma unroll
            for (int q = 0; q < kNx; ++q) {
                const int i = tid + q * kThreads, t = i % kC, d = i / kC * 4;
                four(yg + (t0 + min(t, most)) * y_step + d, yw, y[q]);
            }
#pragma unroll
            for (int q = 0; q < kNz; ++q) {
                const int i = tid + q * kThreads, t = i / (kZ / 4), z = i % (kZ / 4) * 4;
                four(zg + (t0 + min(t, most)) * z_step + z, zw, v[q]);
            }
        }
#pragma unroll
        for (int q = 0; q < kNx; ++q) {
            const int i = tid + q * kThreads, t = i % kC, d = i / kC * 4;
            const bool ok = t < cnt;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[q][u] = ok ? x[q][u] : 0.f;
                y[q][u] = ok ? y[q][u] : 0.f;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) Yt[(d + u) * kPitch + t] = y[q][u];
            if (!states)
#pragma unroll
                for (int u = 0; u < 4; ++u) Xt[(d + u) * kPitch + t] = x[q][u];
        }
#pragma unroll
        for (int q = 0; q < kNz; ++q) {
            const int i = tid + q * kThreads, t = i / (kZ / 4), z = i % (kZ / 4) * 4;
            const bool ok = t < cnt;
            *reinterpret_cast<float4 *>(Z + t * kZp + z) =
                make_float4(ok ? v[q][0] : 0.f, ok ? v[q][1] : 0.f, ok ? v[q][2] : 0.f, ok ? v[q][3] : 0.f);
        }
        if (!states)
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int u = 0; u < kU; ++u) S[(ty * kR + r) * kZp + tx * kU + u] = s[r][u];
        __syncthreads();
        float a[4][4] = {}, e[4][kU] = {};   // X Y^T and X S, which take the same values of X
        if (!states) {
#pragma unroll 4
            for (int d = 0; d < kX; ++d) {
                float x[4], y[4], z[kU];
                take<4>(Xt + d * kPitch + 4 * ty, x);
                take<4>(Yt + d * kPitch + 4 * tx, y);
                take<kU>(S + d * kZp + kU * tx, z);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) a[i][q] = fmaf(x[i], y[q], a[i][q]);
#pragma unroll
                    for (int u = 0; u < kU; ++u) e[i][u] = fmaf(x[i], z[u], e[i][u]);
                }
            }
        }
        // the state moves on, where it is taken up again: a segment's last one only at the sequence's end
        if (cnt > 0 && (states || wanted || ci + 1 < nchunk)) {
            const float gn = gp[cnt];
            float upd[kR][kU] = {};
#pragma unroll 2
            for (int q0 = 0; q0 < kC; q0 += 4) {
                float y[kR][4];
#pragma unroll
                for (int r = 0; r < kR; ++r) take<4>(Yt + (kR * ty + r) * kPitch + q0, y[r]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int q = q0 + j;
                    float z[kU];
                    take<kU>(Z + q * kZp + kU * tx, z);
                    const float w = q < cnt ? gp[reverse ? q + 1 : cnt - 1 - q] : 0.f;
#pragma unroll
                    for (int u = 0; u < kU; ++u) z[u] *= w;
#pragma unroll
                    for (int r = 0; r < kR; ++r)
#pragma unroll
                        for (int u = 0; u < kU; ++u) upd[r][u] = fmaf(y[r][j], z[u], upd[r][u]);
                }
            }
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
                for (int u = 0; u < kU; ++u) s[r][u] = fmaf(gn, s[r][u], a_upd * upd[r][u]);
        }
        if (states) continue;
        __syncthreads();   // Y is used up
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int dist = reverse ? 4 * tx + q - 4 * ty - i : 4 * ty + i - 4 * tx - q;
                w[i] = dist >= 0 ? a_intra * gp[dist] * a[i][q] : 0.f;
            }
            *reinterpret_cast<float4 *>(Pt + (4 * tx + q) * kPitch + 4 * ty) = make_float4(w[0], w[1], w[2], w[3]);
        }
        __syncthreads();
        float o[4][kU] = {};
        // a warp's eight rows: columns on the mask's side only
        const int row0 = (tid >> 5) * 8, j0 = reverse ? row0 : 0, j1 = reverse ? kC : row0 + 8;
#pragma unroll 4
        for (int q = j0; q < j1; ++q) {
            float w[4], z[kU];
            take<4>(Pt + q * kPitch + 4 * ty, w);
            take<kU>(Z + q * kZp + kU * tx, z);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int u = 0; u < kU; ++u) o[i][u] = fmaf(w[i], z[u], o[i][u]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
            if (t0 + t < t_stop) {
                const bool ok = t < cnt;
                const float w = ok ? a_inter * gp[reverse ? cnt - 1 - t : t + 1] : 0.f;
                T *dst = og + (t0 + t) * o_step + kU * tx;
#pragma unroll
                for (int u = 0; u < kU; ++u) dst[u] = from_f32<T>(ok ? fmaf(w, e[i][u], o[i][u]) : 0.f);
            }
        }
    }
    if (!states && !wanted) return;
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int d = ty * kR + r, z = z0 + tx * kU + u;
            if (states)
                p.seg_states[lin_slot(p, chain, seg) + d * p.dz + z] = s[r][u];
            else
                p.ST[s_index(p, chain, d, z)] = s[r][u];
        }
}

// Start states of a chain's segments, S' = g^n S + Z, one element a thread: the loads of a chain do not depend on one
// another. 8 us for nine segments of 16 heads of 128 x 128.
__global__ void __launch_bounds__(kThreads) lin_combine_kernel(const __grid_constant__ Scans all) {
    const LinScan &p = all.s[blockIdx.z];
    dependency_release();
    dependency_wait();
    const int chain = blockIdx.x, b = chain / p.H, h = chain % p.H;
    const int i = blockIdx.y * kThreads + threadIdx.x, elems = p.dx * p.dz;
    if (i >= elems) return;
    const int n = lin_length(p.lengths, b, p.T);
    const float g = p.decay[h];
    const int d = p.seg_t ? i % p.dx : i / p.dz, z = p.seg_t ? i / p.dx : i % p.dz;
    float s = p.S0 ? p.S0[s_index(p, chain, d, z)] : 0.f;
    float *slot = p.seg_states + lin_slot(p, chain, 0) + i;
    const float g_full = powf(g, static_cast<float>(p.seg_len));
    slot[static_cast<size_t>(p.nseg - 1) * elems] = s;
    constexpr int kAhead = 8;   // slots read before the first of them is replaced
    for (int k = 0; k < p.nseg - 1; k += kAhead) {
        float v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            v[u] = k + u < p.nseg - 1 ? slot[static_cast<size_t>(k + u) * elems] : 0.f;
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (k + u < p.nseg - 1) {
                int t0;
                const int m = lin_segment(p, k + u, n, t0);
                s = fmaf(m == p.seg_len ? g_full : powf(g, static_cast<float>(m)), s, v[u]);
                slot[static_cast<size_t>(k + u) * elems] = s;
            }
    }
}

template <typename T, int kX, int kZ>
cudaError_t launch_scan_as(const LinScan *p, int scans, cudaStream_t stream) {
    constexpr int kBytes = kScanFloats<kX, kZ> * 4;
    auto kern = lin_scan_kernel<T, kX, kZ>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    Scans all;
    for (int i = 0; i < scans; ++i) all.s[i] = p[i];
    const int ctas = p->B * p->H * (p->dz / kZ);
    if (p->nseg > 1) {
        kern<<<dim3(ctas, p->nseg - 1, scans), kThreads, kBytes, stream>>>(all, 1);
        if ((e = cudaGetLastError()) != cudaSuccess || (e = launch_lin_combine(p, scans, stream)) != cudaSuccess)
            return e;
        return launch_dependent(kern, dim3(ctas, p->nseg, scans), kThreads, kBytes, stream, all, 0);
    }
    kern<<<dim3(ctas, 1, scans), kThreads, kBytes, stream>>>(all, 0);
    return cudaGetLastError();
}
template <typename T, int kX>
cudaError_t launch_scan_x(const LinScan *p, int scans, cudaStream_t stream) {
    return p->dz >= 64   ? launch_scan_as<T, kX, 64>(p, scans, stream)
           : p->dz == 32 ? launch_scan_as<T, kX, 32>(p, scans, stream)
                         : launch_scan_as<T, kX, 16>(p, scans, stream);
}
template <typename T>
cudaError_t launch_scan(const LinScan *p, int scans, cudaStream_t stream) {
    switch (p->dx) {
        case 128: return launch_scan_x<T, 128>(p, scans, stream);
        case 64: return launch_scan_x<T, 64>(p, scans, stream);
        case 32: return launch_scan_x<T, 32>(p, scans, stream);
        default: return launch_scan_x<T, 16>(p, scans, stream);
    }
}

// ---------------------------------------------------------------------------- single-token step
// One CTA per (sequence, head) and kZ value channels: every state element is read once, decayed,
// written to and reduced against the query on the way out. Bound by the memory: 128 x 24 states of 128 x 128 take
// 59 us (6.8 TB/s, a copy's rate). 64 x 16 (67 MB) in place, again and again: 14 us, since L2 holds them; from one
// buffer to another and back, which together it does not hold: 19 us (7.0 TB/s, a part of it from L2). 1 x 16: 2 us,
// a launch's latency.
template <typename T, int kZ>
__global__ void __launch_bounds__(kThreads) lin_step_kernel(const T *q, const T *k, const T *v, const float *decay,
                                                            const int *parent, const float *S, float *S_out, T *o,
                                                            int H, int dk, int dv, int n_states, float q_scale) {
    constexpr int kVec = kZ / 4, kRows = kThreads / kVec;   // float4 of a row, rows in flight
    __shared__ float qs[128], ks[128], part[kThreads / 32][kZ];
    const int tid = threadIdx.x, nz = dv / kZ;
    const int bh = blockIdx.x / nz, z0 = (blockIdx.x % nz) * kZ;
    const int b = bh / H, h = bh % H;
    const int from = parent ? parent[b] : b;
    const bool live = from >= 0 && from < n_states;
    const int c = tid % kVec, r = tid / kVec;
    const float *src = S + ((static_cast<size_t>(live ? from : 0) * H + h) * dk) * dv + z0 + 4 * c;
    float *dst = S_out + (static_cast<size_t>(bh) * dk) * dv + z0 + 4 * c;
    constexpr int kMost = 128 / kRows > 0 ? 128 / kRows : 1;
    float4 s[kMost];
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
        const int d = r + u * kRows;
        s[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (d < dk && live) s[u] = *reinterpret_cast<const float4 *>(src + static_cast<size_t>(d) * dv);
    }
    for (int d = tid; d < dk; d += kThreads) {
        qs[d] = to_f32(q[static_cast<size_t>(bh) * dk + d]) * q_scale;
        ks[d] = to_f32(k[static_cast<size_t>(bh) * dk + d]);
    }
    const float g = decay[h];
    float vv[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < 4; ++u) vv[u] = to_f32(v[static_cast<size_t>(bh) * dv + z0 + 4 * c + u]);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
        const int d = r + u * kRows;
        if (d < dk) {
            const float kd = ks[d], qd = qs[d];
            s[u].x = fmaf(kd, vv[0], g * s[u].x);
            s[u].y = fmaf(kd, vv[1], g * s[u].y);
            s[u].z = fmaf(kd, vv[2], g * s[u].z);
            s[u].w = fmaf(kd, vv[3], g * s[u].w);
            *reinterpret_cast<float4 *>(dst + static_cast<size_t>(d) * dv) = s[u];
            acc[0] = fmaf(qd, s[u].x, acc[0]);
            acc[1] = fmaf(qd, s[u].y, acc[1]);
            acc[2] = fmaf(qd, s[u].z, acc[2]);
            acc[3] = fmaf(qd, s[u].w, acc[3]);
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int off = kVec; off < 32; off <<= 1) acc[u] += __shfl_xor_sync(0xffffffffu, acc[u], off);
    if ((tid & 31) < kVec)
#pragma unroll
        for (int u = 0; u < 4; ++u) part[tid / 32][4 * c + u] = acc[u];
    __syncthreads();
    if (tid < kZ) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) sum += part[w][tid];
        o[static_cast<size_t>(bh) * dv + z0 + tid] = from_f32<T>(sum);
    }
}

template <typename T>
cudaError_t launch_step(const void *q, const void *k, const void *v, const float *decay, const int *parent,
                        const float *S, float *S_out, void *o, int B, int H, int dk, int dv, int n_states,
                        float q_scale, cudaStream_t stream) {
    const T *qq = static_cast<const T *>(q), *kk = static_cast<const T *>(k), *vv = static_cast<const T *>(v);
    if (dv % 32 == 0)
        lin_step_kernel<T, 32><<<B * H * (dv / 32), kThreads, 0, stream>>>(
            qq, kk, vv, decay, parent, S, S_out, static_cast<T *>(o), H, dk, dv, n_states, q_scale);
    else
        lin_step_kernel<T, 16><<<B * H * (dv / 16), kThreads, 0, stream>>>(
            qq, kk, vv, decay, parent, S, S_out, static_cast<T *>(o), H, dk, dv, n_states, q_scale);
    return cudaGetLastError();
}

// ------------------------------------------------------------------------------------ host side
bool supported_d(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool finite(float x) { return x - x == 0.0f; }

// The bytes that a strided [B, T, H, d] tensor reaches over.
Span reach(const void *p, const int64_t *st, int B, int T, int H, int d, size_t esz) {
    if (B < 1 || T < 1 || H < 1) return span(p, 0);
    return span(p, (static_cast<size_t>(B - 1) * st[0] + static_cast<size_t>(T - 1) * st[1] +
                    static_cast<size_t>(H - 1) * st[2] + d) * esz);
}

constexpr int kSms = 152;
// Tokens are numbered in 32 bits up to the end of the last segment's last chunk. At most 2 kSms segments are
// asked for, each a whole number of chunks of up to 128 tokens: they reach less than 2 kSms chunks past T.
constexpr int kMostTokens = INT_MAX - 65536;
static_assert((2 * kSms + 1) * 128 < 65536, "segments past the last token");

size_t seg_bytes(const LinScan &p) {
    return p.nseg > 1 ? static_cast<size_t>(p.B) * p.H * p.nseg * p.dx * p.dz * sizeof(float) : 0;
}

// Segments of the fp32 scan: CTAs for every SM twice, down to one chunk a segment.
void plan_scan(LinScan &p, kla_dtype dtype, int scans) {
    if (dtype == KLA_DTYPE_BF16 && p.dx == 128 && p.dz == 128) return lin_tc_plan(p, scans);   // one scratch size
    const int nchunk = (p.T + kC - 1) / kC;
    const long ctas = static_cast<long>(p.B) * p.H * (p.dz < 64 ? 1 : p.dz / 64) * scans;
    long n = 2 * kSms / ctas;
    n = n > nchunk ? nchunk : n < 1 ? 1 : n;
    const int len = n > 0 ? static_cast<int>((nchunk + n - 1) / n) : 1;
    p.seg_len = len * kC;
    p.nseg = nchunk > 0 ? (nchunk + len - 1) / len : 1;
}

// Scratch of `scans` scans of these sizes, which run side by side.
size_t scratch(LinScan p, kla_dtype dtype, int scans) {
    plan_scan(p, dtype, scans);
    return scans * seg_bytes(p);
}

void set_strides(int64_t (&to)[3], const int64_t *from, int T, int H, int d) {
    to[0] = from ? from[0] : static_cast<int64_t>(T) * H * d;
    to[1] = from ? from[1] : static_cast<int64_t>(H) * d;
    to[2] = from ? from[2] : d;
}

// Sizes, type and scale common to both directions; `ntens` strided tensors.
kla_status check_sizes(int B, int T, int H, int d_k, int d_v, kla_dtype dtype, float q_scale, const int64_t *strides,
                       int ntens) {
    if (B < 1 || T < 0 || H < 1 || d_k < 1 || d_v < 1) return KLA_ERR_INVALID_ARG;
    if (dtype != KLA_DTYPE_F32 && dtype != KLA_DTYPE_BF16) return KLA_ERR_INVALID_ARG;
    if (!finite(q_scale)) return KLA_ERR_INVALID_ARG;
    for (int i = 0; strides && i < 3 * ntens; ++i)
        if (strides[i] < 0) return KLA_ERR_INVALID_ARG;
    if (!supported_d(d_k) || !supported_d(d_v) || T > kMostTokens) return KLA_ERR_UNSUPPORTED;
    // chains times value tiles index the grid
    if (static_cast<int64_t>(B) * H * 8 > INT_MAX) return KLA_ERR_UNSUPPORTED;
    return KLA_OK;
}

}  // namespace

cudaError_t launch_lin_combine(const LinScan *p, int scans, cudaStream_t stream) {
    Scans all;
    for (int i = 0; i < scans; ++i) all.s[i] = p[i];
    return launch_dependent(lin_combine_kernel, dim3(p->B * p->H, (p->dx * p->dz + kThreads - 1) / kThreads, scans),
                            kThreads, 0, stream, all);
}

cudaError_t launch_lin_scan(const LinScan *p, int scans, kla_dtype dtype, cudaStream_t stream) {
    return dtype == KLA_DTYPE_BF16 ? launch_scan<__nv_bfloat16>(p, scans, stream)
                                   : launch_scan<float>(p, scans, stream);
}

}  // namespace kla

using kla::LinScan;

extern "C" {

size_t kla_linear_fwd_workspace_size(int B, int T, int H, int d_k, int d_v, kla_dtype dtype) {
    if (B < 1 || T < 1 || T > kla::kMostTokens || H < 1 || !kla::supported_d(d_k) || !kla::supported_d(d_v)) return 0;
    LinScan p{};
    p.B = B; p.T = T; p.H = H; p.dx = d_k; p.dz = d_v;
    return kla::scratch(p, dtype, 1);
}

size_t kla_linear_bwd_workspace_size(int B, int T, int H, int d_k, int d_v, kla_dtype dtype) {
    if (B < 1 || T < 1 || T > kla::kMostTokens || H < 1 || !kla::supported_d(d_k) || !kla::supported_d(d_v)) return 0;
    LinScan p{}, q{};
    p.B = q.B = B; p.T = q.T = T; p.H = q.H = H;
    p.dx = q.dz = d_k;
    p.dz = q.dx = d_v;
    const size_t a = kla::scratch(p, dtype, 3), b = kla::scratch(q, dtype, 3);
    const size_t fwd = kla::scratch(p, dtype, 1);   // one buffer serves both directions
    return a > b ? (a > fwd ? a : fwd) : (b > fwd ? b : fwd);
}

kla_status kla_linear_fwd(const void *q, const void *k, const void *v, const int64_t *strides, const float *decay,
                          const int *lengths, const float *S0, void *o, float *S_T, int B, int T, int H, int d_k,
                          int d_v, kla_dtype dtype, float q_scale, void *workspace, size_t workspace_bytes,
                          void *stream) {
    using namespace kla;
    kla_status st = check_sizes(B, T, H, d_k, d_v, dtype, q_scale, strides, 3);
    if (st != KLA_OK) return st;
    if (!decay || (T > 0 && (!q || !k || !v || !o))) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(q, esz) || !aligned(k, esz) || !aligned(v, esz) || !aligned(o, esz) || !aligned(decay, 4) ||
        !aligned(lengths, 4) || !aligned(S0, 16) || !aligned(S_T, 16) || !aligned(workspace, 16))
        return KLA_ERR_INVALID_ARG;
    const size_t need = kla_linear_fwd_workspace_size(B, T, H, d_k, d_v, dtype);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KLA_ERR_INVALID_ARG;
    LinScan p{};
    p.x = q; p.y = k; p.z = v;
    set_strides(p.xs, strides, T, H, d_k);
    set_strides(p.ys, strides ? strides + 3 : nullptr, T, H, d_k);
    set_strides(p.zs, strides ? strides + 6 : nullptr, T, H, d_v);
    const size_t sbytes = static_cast<size_t>(B) * H * d_k * d_v * 4;
    const size_t obytes = static_cast<size_t>(B) * T * H * d_v * esz;
    const Span outs[] = {span(o, obytes), span(S_T, sbytes), span(workspace, need)};
    const Span ins[] = {reach(q, p.xs, B, T, H, d_k, esz), reach(k, p.ys, B, T, H, d_k, esz),
                        reach(v, p.zs, B, T, H, d_v, esz), span(decay, 4ull * H), span(lengths, 4ull * B),
                        span(S0, sbytes)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 6; ++j)
            if (overlaps(outs[i], ins[j]) && !(i == 1 && j == 5 && S0 == S_T)) return KLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(outs[i], outs[j])) return KLA_ERR_INVALID_ARG;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (T == 0) {   // no tokens: the final state is the initial one
        if (!S_T || S_T == S0) return KLA_OK;
        const cudaError_t e = S0 ? cudaMemcpyAsync(S_T, S0, sbytes, cudaMemcpyDeviceToDevice, cs)
                                 : cudaMemsetAsync(S_T, 0, sbytes, cs);
        return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
    }
    p.out = o; p.decay = decay; p.lengths = lengths; p.S0 = S0; p.ST = S_T;
    p.B = B; p.T = T; p.H = H; p.dx = d_k; p.dz = d_v;
    p.a_intra = p.a_inter = q_scale;
    p.a_upd = 1.0f;
    p.seg_states = static_cast<float *>(workspace);
    cudaError_t e;
    plan_scan(p, dtype, 1);
    e = lin_tc_supports(p, dtype) ? launch_lin_tc(&p, 1, cs) : launch_lin_scan(&p, 1, dtype, cs);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

kla_status kla_linear_bwd(const void *q, const void *k, const void *v, const void *dO, const int64_t *strides,
                          const float *decay, const int *lengths, const float *S0, const float *dS_T, void *dq,
                          void *dk, void *dv, float *dS0, int B, int T, int H, int d_k, int d_v, kla_dtype dtype,
                          float q_scale, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace kla;
    kla_status st = check_sizes(B, T, H, d_k, d_v, dtype, q_scale, strides, 4);
    if (st != KLA_OK) return st;
    if (!decay || (T > 0 && (!q || !k || !v || !dO || !dq || !dk || !dv))) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(q, esz) || !aligned(k, esz) || !aligned(v, esz) || !aligned(dO, esz) || !aligned(dq, esz) ||
        !aligned(dk, esz) || !aligned(dv, esz) || !aligned(decay, 4) || !aligned(lengths, 4) || !aligned(S0, 16) ||
        !aligned(dS_T, 16) || !aligned(dS0, 16) || !aligned(workspace, 16))
        return KLA_ERR_INVALID_ARG;
    const size_t need = kla_linear_bwd_workspace_size(B, T, H, d_k, d_v, dtype);
    if (workspace_bytes < need || (need > 0 && !workspace)) return KLA_ERR_INVALID_ARG;
    int64_t qs[3], ks[3], vs[3], os[3];
    set_strides(qs, strides, T, H, d_k);
    set_strides(ks, strides ? strides + 3 : nullptr, T, H, d_k);
    set_strides(vs, strides ? strides + 6 : nullptr, T, H, d_v);
    set_strides(os, strides ? strides + 9 : nullptr, T, H, d_v);
    const size_t sbytes = static_cast<size_t>(B) * H * d_k * d_v * 4;
    const size_t n = static_cast<size_t>(B) * T * H;
    const Span outs[] = {span(dq, n * d_k * esz), span(dk, n * d_k * esz), span(dv, n * d_v * esz), span(dS0, sbytes),
                         span(workspace, need)};
    const Span ins[] = {reach(q, qs, B, T, H, d_k, esz), reach(k, ks, B, T, H, d_k, esz),
                        reach(v, vs, B, T, H, d_v, esz), reach(dO, os, B, T, H, d_v, esz), span(decay, 4ull * H),
                        span(lengths, 4ull * B), span(S0, sbytes), span(dS_T, sbytes)};
    for (int i = 0; i < 5; ++i) {
        for (const Span &x : ins)
            if (overlaps(outs[i], x)) return KLA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 5; ++j)
            if (overlaps(outs[i], outs[j])) return KLA_ERR_INVALID_ARG;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (T == 0) {   // no tokens: dL/dS0 = dL/dS_T
        if (!dS0) return KLA_OK;
        const cudaError_t e = dS_T ? cudaMemcpyAsync(dS0, dS_T, sbytes, cudaMemcpyDeviceToDevice, cs)
                                   : cudaMemsetAsync(dS0, 0, sbytes, cs);
        return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
    }
    auto set = [&](const void *x, const int64_t *xs, const void *y, const int64_t *ys, const void *z,
                    const int64_t *zs, void *out, const float *s0, float *sT, int s_t, int dx, int dz, int reverse) {
        LinScan p{};
        p.x = x; p.y = y; p.z = z;
        for (int i = 0; i < 3; ++i) { p.xs[i] = xs[i]; p.ys[i] = ys[i]; p.zs[i] = zs[i]; }
        p.out = out; p.decay = decay; p.lengths = lengths; p.S0 = s0; p.ST = sT; p.s_t = s_t;
        p.B = B; p.T = T; p.H = H; p.dx = dx; p.dz = dz; p.reverse = reverse;
        p.a_intra = q_scale;
        p.a_inter = reverse ? 1.0f : q_scale;
        p.a_upd = reverse ? q_scale : 1.0f;
        return p;
    };
    LinScan p[3] = {set(k, ks, q, qs, dO, os, dv, dS_T, dS0, 0, d_k, d_v, 1),
                    set(v, vs, dO, os, q, qs, dk, dS_T, nullptr, 1, d_v, d_k, 1),
                    set(dO, os, v, vs, k, ks, dq, S0, nullptr, 1, d_v, d_k, 0)};
    const bool tc = lin_tc_supports(p[0], dtype) && lin_tc_supports(p[1], dtype) && lin_tc_supports(p[2], dtype);
    float *scratch = static_cast<float *>(workspace);
    for (int i = 0; i < 3; ++i) {
        plan_scan(p[i], dtype, 3);
        p[i].seg_states = scratch;
        scratch += seg_bytes(p[i]) / sizeof(float);
    }
    cudaError_t e;
    if (tc) {
        e = launch_lin_tc(p, 3, cs);
    } else if (d_k == d_v) {
        e = launch_lin_scan(p, 3, dtype, cs);
    } else {   // dv's state is the transpose of the others'
        e = launch_lin_scan(p, 1, dtype, cs);
        if (e == cudaSuccess) e = launch_lin_scan(p + 1, 2, dtype, cs);
    }
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

kla_status kla_linear_step(const void *q, const void *k, const void *v, const float *decay, const int *parent,
                           const float *S, float *S_out, void *o, int B, int H, int d_k, int d_v, int n_states,
                           kla_dtype dtype, float q_scale, void *stream) {
    using namespace kla;
    kla_status st = check_sizes(B, 1, H, d_k, d_v, dtype, q_scale, nullptr, 0);
    if (st != KLA_OK) return st;
    if (!q || !k || !v || !decay || !S || !S_out || !o || n_states < 1 || (!parent && n_states != B))
        return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(q, esz) || !aligned(k, esz) || !aligned(v, esz) || !aligned(o, esz) || !aligned(decay, 4) ||
        !aligned(parent, 4) || !aligned(S, 16) || !aligned(S_out, 16))
        return KLA_ERR_INVALID_ARG;
    const size_t nh = static_cast<size_t>(B) * H, one = static_cast<size_t>(H) * d_k * d_v * 4;
    const Span outs[] = {span(S_out, B * one), span(o, nh * d_v * esz)};
    const Span ins[] = {span(S, n_states * one), span(q, nh * d_k * esz), span(k, nh * d_k * esz),
                        span(v, nh * d_v * esz), span(decay, 4ull * H), span(parent, 4ull * B)};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 6; ++j)
            if (overlaps(outs[i], ins[j]) && !(i == 0 && j == 0 && !parent && S == S_out)) return KLA_ERR_INVALID_ARG;
    if (overlaps(outs[0], outs[1])) return KLA_ERR_INVALID_ARG;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        dtype == KLA_DTYPE_BF16
            ? launch_step<__nv_bfloat16>(q, k, v, decay, parent, S, S_out, o, B, H, d_k, d_v, n_states, q_scale, cs)
            : launch_step<float>(q, k, v, decay, parent, S, S_out, o, B, H, d_k, d_v, n_states, q_scale, cs);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // extern "C"
