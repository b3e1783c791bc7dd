// kla_block_norm.cu -- the norms of a block: after its heads, times the activation of a gate, and of the residual that
// the block's output is added to.
//
//   gated   y = xh w act(z)                 dx = N(dy w act(z)),  dz = dy xh w act'(z),  dw = sum dy act(z) xh
//   added   s = r + l x,  y = xh(s) w       dr = ds + N(dy w),  dx = l dr,  dw = sum dy xh,  dl = sum x dr
//   xh = (x - mean) rstd, N(u) = rstd (u - mean(u) - xh mean(u xh)); without the means' terms where mean = 0 (RMS)
//
// What bounds them is the memory: 3 and 5 elements a value for the gated norm, 4 and 6 for the residual's (5 where it is
// not scaled). Backward, the residual's sum is formed again from x and the residual: read back as it was rounded to bf16
// it would leave 9 bits of dw.
// Measured, bf16: 32768 x 16 heads of 128 gated forward 72 us (5.6 TB/s, 82 % of a copy's rate), backward with dw 122 us
// (5.5 TB/s), in fp32 146 and 221 us (5.5 and 6.1 TB/s); 16397 x 2048 residual forward 50 us (5.4 TB/s), backward with dw
// and dl 75 us (5.4 TB/s), in fp32 92 and 141 us (5.8 and 5.7 TB/s). By the counters (16384 rows of the same) 19 to 20
// instructions a value forward and 31 to 33 backward at 2.0 to 2.7 of 4 a cycle with 16 warps an SM: arithmetic and memory
// each fill about two thirds of the time. Rows of 100 to 300 values fill their teams by three quarters, and a team has one
// short row at hand, whose sums, addresses and loop are spread over few values: 65536 x 3 heads of 100 bf16 49 and 75 us
// (2.4 and 2.6 TB/s). CTAs that add up row by row with barriers and read twice took 3650 us for the first, 709 for the
// second.
#include <atomic>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "layer_dev.cuh"
#include "../../include/kla_block.h"

namespace kla {
namespace {

enum Op { kGatedFwd, kGatedBwd, kAddFwd, kAddBwd };
constexpr bool gated(Op op) { return op == kGatedFwd || op == kGatedBwd; }
constexpr bool backward(Op op) { return op == kGatedBwd || op == kAddBwd; }
// What a row is read of, in this order: gated x, z, dy; added x, residual, dy, dsum.
constexpr int inputs(Op op) { return op == kAddBwd ? 4 : op == kGatedBwd ? 3 : 2; }

struct NormArgs {
    const void *in[4];        // added, backward: dsum may be NULL
    int64_t z_stride;         // gated: between rows of `groups` of z
    const float *w, *l;
    int w_groups;             // weights [groups, n]
    void *out[2];             // gated: y; dx, dz. added: y, sum; dresidual, dx (or NULL)
    float *mean, *rstd;
    float *part;              // [parts][sums][n] of dw (and dl), or NULL
    int64_t rows;             // of all groups
    int groups, n;
    int classes;              // a CTA has rows of one remainder by this: of equal weights, and kLie: of equal start
    float eps;
    int layer, silu;
};

__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return add2(a, b); }
__device__ __forceinline__ float across(float v, int off) { return __shfl_xor_sync(0xffffffffu, v, off); }
__device__ __forceinline__ float2 across(float2 v, int off) { return make_float2(across(v.x, off), across(v.y, off)); }

// The sigmoid, and exp(-z).
template <typename T>
__device__ __forceinline__ float2 sigmoid(float2 z, float2 &e) {
    if (sizeof(T) == 4) {
        e = make_float2(expf(-z.x), expf(-z.y));
        return make_float2(1.f / (1.f + e.x), 1.f / (1.f + e.y));
    }
    // bf16: the hardware's exponential and reciprocal, off by 2^-21 at z of 10, far below z's own 2^-9
    e = mul2(z, both(-1.4426950408889634f));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
    float2 s = add2(e, both(1.f));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s.y));
    return s;
}
// act(z), and act'(z). The sigmoid's slope is s (1 - s), where 1 - s is taken as exp(-z) s: as a difference it would have
// lost 2^-10 of itself at z of 10 and all at 17. (At most 1: an infinite exponential and s = 0 make a NaN, which is not
// the smaller.)
template <typename T>
__device__ __forceinline__ float2 activation(float2 z, int silu) {
    float2 e;
    const float2 s = sigmoid<T>(z, e);
    return silu ? mul2(z, s) : s;
}
template <typename T>
__device__ __forceinline__ float2 activation(float2 z, int silu, float2 &slope) {
    float2 e;
    const float2 s = sigmoid<T>(z, e);
    e = mul2(e, s);
    const float2 rest = make_float2(fminf(e.x, 1.f), fminf(e.y, 1.f));
    slope = mul2(s, silu ? fma2(z, rest, both(1.f)) : rest);
    return silu ? mul2(z, s) : s;
}
// 1 / sqrt(v): the hardware's, off by 2^-22, and one step of Newton's iteration
__device__ __forceinline__ float reciprocal_root(float v) {
    const float r = rsqrtf(v);
    return v > 0.f && v <= FLT_MAX ? fmaf(r * fmaf(-v * r, r, 1.f), 0.5f, r) : r;
}

template <int kBytes>
__device__ __forceinline__ void copy_in(void *to, const void *from) {
    if constexpr (kBytes == 2) return;
    else if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(to)), "l"(from) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(to)), "l"(from) : "memory");
}
// The first `size` of 16 bytes, the rest zeros.
__device__ __forceinline__ void copy_start(void *to, const void *from, int size) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(to)), "l"(from), "r"(size) : "memory");
}
template <int kGroups>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kGroups) : "memory");
}

__device__ __forceinline__ void set(float2 &v, int i, float x) { (i ? v.y : v.x) = x; }
__device__ __forceinline__ float part(const float2 &v, int i) { return i ? v.y : v.x; }

// kBytes of a row as values, and back
template <int kBytes>
struct alignas(kBytes) Raw {
    typename std::conditional<kBytes == 2, uint16_t, uint32_t>::type r[kBytes == 2 ? 1 : kBytes / 4];
};
template <typename T, int kBytes>
__device__ __forceinline__ void unpack(const Raw<kBytes> &raw, float *v) {
    if constexpr (kBytes == 2) {
        v[0] = __uint_as_float(static_cast<uint32_t>(raw.r[0]) << 16);
    } else {
#pragma unroll
        for (int i = 0; i < kBytes / 4; ++i) {
            if (sizeof(T) == 4) {
                v[i] = __uint_as_float(raw.r[i]);
            } else {
                v[2 * i] = __uint_as_float(raw.r[i] << 16);
                v[2 * i + 1] = __uint_as_float(raw.r[i] & 0xffff0000u);
            }
        }
    }
}
template <typename T, int kBytes>
__device__ __forceinline__ void pack(void *p, const float *v) {
    uint32_t r[(kBytes + 2) / 4];
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i)
        r[i] = sizeof(T) == 4 ? __float_as_uint(v[i]) : ptx::pack_bf16(v[2 * i], v[2 * i + 1]);
    if constexpr (kBytes == 16) *static_cast<uint4 *>(p) = make_uint4(r[0], r[1], r[2], r[3]);
    else if constexpr (kBytes == 4) *static_cast<uint32_t *>(p) = r[0];
    else *static_cast<T *>(p) = from_f32<T>(v[0]);
}

// ---- rows that a team of threads holds in registers
// A row belongs to a team of `width` threads (4 to 32 lanes of a warp, or whole warps up to the CTA), each with kNV
// accesses of kBytes at fixed columns, so that weights and the sums of dw and dl stay in registers. Every thread
// copies its own values of the next kStages - 1 rows into shared memory and takes them from there: no barrier stands
// between copy and use, and what is on its way does not cost registers. CTAs are persistent. Rows whose length is no
// multiple of 16 bytes start in the middle of 16, every second, fourth or eighth at the same place: a CTA has rows of one
// place, and so a thread the same columns of all of them, those of the 16 bytes as they lie (kLie). Where the tensors' rows
// start differently that leaves accesses of 4 bytes; of odd bf16 those too are none, and values are loaded as they are
// needed (kDirect), as are rows of which shared memory holds no two. 16384 x 1001 bf16 by single values, 4 bytes and 16, us
// forward and backward: gated 44 and 64, 37 and 59, 29 and 44; residual 50 and 120, 41 and 71, 31 and 54.
enum Rows { kRing, kLie, kDirect };
constexpr int kMostBlock = 512;
// Of the operation and the values of a thread: how many CTAs an SM's registers and shared memory hold.
constexpr int ctas(Op op, int values, int block) {
    const int of_256 = values <= 8 ? (backward(op) ? 3 : 4) : 2;
    return block == 256 ? of_256 : of_256 / 2;
}
constexpr int stages(Op op, int values, int bytes, int block) {   // bytes: of a thread's row of one input
    const int most = 200 * 1024 / (ctas(op, values, block) * block) / (inputs(op) * bytes + (backward(op) ? 8 : 0));
    return most > 6 ? 6 : most < 2 ? 2 : most;
}

template <typename T, int kBytes, int kNV, Op kOp, int kBlock, Rows kBy>
__global__ void __launch_bounds__(kBlock, ctas(kOp, kNV *kBytes / static_cast<int>(sizeof(T)), kBlock))
block_norm_kernel(NormArgs p, int width) {
    constexpr int kV = kBytes / sizeof(T), kE = kV * kNV, kP = kE / 2, kIns = inputs(kOp);
    constexpr int kStages = stages(kOp, kE, kNV * kBytes, kBlock);
    constexpr bool kGated = gated(kOp), kBwd = backward(kOp), kLoad = kBy == kDirect;
    dependency_release();
    extern __shared__ __align__(16) uint8_t ring[];   // [stage][input][access][thread], then [stage][2][thread] of stats
    __shared__ float2 sums[2][kBlock / 32];
    const int team = threadIdx.x / width, lane = threadIdx.x % width, teams = kBlock / width;
    const int classes = p.classes, g = blockIdx.x % classes, group = p.w_groups ? g % p.groups : 0;
    // 64 bits: sums pass the last row
    const int64_t first = blockIdx.x / classes * teams, mine = (p.rows - g + classes - 1) / classes;
    const int step = gridDim.x / classes * teams;
    const int turns = first < mine ? static_cast<int>((mine - first + step - 1) / step) : 0;
    const bool four = kOp == kAddBwd && p.in[3] != nullptr;
    float *const stats = reinterpret_cast<float *>(ring + kStages * kIns * kNV * kBlock * kBytes);
    auto slot = [&](int stage, int i, int k) {
        return ring + (((stage * kIns + i) * kNV + k) * kBlock + threadIdx.x) * kBytes;
    };
    // the next row to be copied, and the one at hand: their index, and the first of their values of this thread
    const int64_t row0 = (first + team) * classes + g, rows = p.rows;
    const int hop = step * classes;
    const int before = kBy == kLie ? static_cast<int>(row0 * p.n % kV) : 0;   // values in front of the row's in its first access
    const int64_t off0 = row0 * p.n + lane * kV - before, off_hop = static_cast<int64_t>(hop) * p.n;
    int64_t ahead = row0, ahead_off = off0;
    // columns of this thread; kLie: which of its accesses are the row's first and last, of which it has a part
    bool there[kNV];
#pragma unroll
    for (int k = 0; k < kNV; ++k) there[k] = (k * width + lane) * kV - before < p.n;
    const int end = (p.n - 1 + before) / kV, of_end = p.n + before - end * kV;
    const int head = kBy == kLie && before > 0 && lane == 0 ? 0 : -1;
    const int tail = kBy == kLie && of_end < kV && end % width == lane ? end / width : -1;
    uint32_t keep[kBy == kLie ? 4 : 1];   // of the first access
#pragma unroll
    for (int i = 0; i < (kBy == kLie ? 4 : 1); ++i) {
        const int gone = head == 0 ? before * static_cast<int>(sizeof(T)) - 4 * i : 0;
        keep[i] = gone >= 4 ? 0u : gone == 2 ? 0xffff0000u : ~0u;
    }
    auto column = [&](int u) { return (u / kV * width + lane) * kV + u % kV - before; };
    auto inside = [&](int u) { return kBy == kLie ? column(u) >= 0 && column(u) < p.n : there[u / kV]; };
    auto source = [&](int i, int64_t row, int64_t off) {   // this thread's first values of a row
        if (kGated && i == 1 && p.z_stride) {
            const unsigned r = static_cast<unsigned>(row), outer = r / static_cast<unsigned>(p.groups);
            off = outer * p.z_stride + static_cast<int64_t>(r - outer * p.groups) * p.n + lane * kV - before;
        }
        return static_cast<const T *>(p.in[i]) + off;
    };
    auto fetch = [&](int stage) {
        if (kLoad) return;
        if (ahead < rows) {
#pragma unroll
            for (int i = 0; i < kIns; ++i) {
                if (i == 3 && !four) break;
                const T *from = source(i, ahead, ahead_off);
#pragma unroll
                for (int k = 0; k < kNV; ++k)
                    if (kBy == kLie && k == tail)
                        copy_start(slot(stage, i, k), from + k * width * kV, of_end * static_cast<int>(sizeof(T)));
                    else if (there[k]) copy_in<kBytes>(slot(stage, i, k), from + k * width * kV);
            }
            if (kBwd) {
                copy_in<4>(stats + (stage * 2) * kBlock + threadIdx.x, p.rstd + ahead);
                if (p.layer) copy_in<4>(stats + (stage * 2 + 1) * kBlock + threadIdx.x, p.mean + ahead);
            }
        }
        ahead += hop;
        ahead_off += off_hop;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    float2 w[kP], l[kGated ? 1 : kP], dw[kBwd ? kP : 1], dl[kOp == kAddBwd ? kP : 1];
#pragma unroll
    for (int u = 0; u < kE; ++u) {
        const int c = column(u);
        const bool in = c >= 0 && c < p.n;
        set(w[u / 2], u % 2, p.w && in ? p.w[static_cast<int64_t>(group) * p.n + c] : 1.f);
        if (!kGated) set(l[u / 2], u % 2, p.l && in ? p.l[c] : 1.f);
    }
#pragma unroll
    for (int u = 0; u < kP; ++u) {
        if (kBwd) dw[u] = both(0.f);
        if (kOp == kAddBwd) dl[u] = both(0.f);
    }
    const float inv = 1.f / p.n;
    int turn_sum = 0;
    auto sum = [&](auto v) {   // over the team; all of the CTA's threads take part in the same calls
        for (int off = width < 32 ? width / 2 : 16; off; off >>= 1) v = add(v, across(v, off));
        if (width > 32) {
            using V = decltype(v);
            const int warps = width / 32, at = team * warps;
            if ((threadIdx.x & 31) == 0) reinterpret_cast<V &>(sums[turn_sum][threadIdx.x / 32]) = v;
            ptx::named_sync(1 + team, width);
            v = reinterpret_cast<const V &>(sums[turn_sum][at]);
            for (int i = 1; i < warps; ++i) v = add(v, reinterpret_cast<const V &>(sums[turn_sum][at + i]));
            turn_sum ^= 1;   // the next sum's words, while others still read these
        }
        return v;
    };
    int64_t row = row0, off = off0;
    for (int t = 0, stage = 0; t < turns; ++t, row += hop, off += off_hop) {
        fetch(stage == 0 ? kStages - 1 : stage - 1);
        copies_wait<kStages - 1>();
        const bool live = row < rows;
        auto get = [&](int i, float2 (&v)[kP]) {   // zeros past the row's end
            Raw<kBytes> raw[kNV];
            const T *from = kLoad ? source(i, row, off) : nullptr;
#pragma unroll
            for (int k = 0; k < kNV; ++k) {   // all loads before the first use
                raw[k] = Raw<kBytes>{};
                if (live && there[k])
                    raw[k] = kLoad ? *reinterpret_cast<const Raw<kBytes> *>(from + k * width * kV)
                                   : *reinterpret_cast<const Raw<kBytes> *>(slot(stage, i, k));
            }
            if constexpr (kBy == kLie)   // what is in front is another row's
#pragma unroll
                for (int q = 0; q < 4; ++q) raw[0].r[q] &= keep[q];
#pragma unroll
            for (int k = 0; k < kNV; ++k) {
                float e[kV];
                unpack<T, kBytes>(raw[k], e);
#pragma unroll
                for (int j = 0; j < kV; ++j) set(v[(k * kV + j) / 2], (k * kV + j) % 2, e[j]);
            }
        };
        auto put = [&](int i, const float2 (&v)[kP]) {
            T *to = static_cast<T *>(p.out[i]) + off;
#pragma unroll
            for (int k = 0; k < kNV; ++k) {
                float e[kV];
#pragma unroll
                for (int j = 0; j < kV; ++j) e[j] = part(v[(k * kV + j) / 2], (k * kV + j) % 2);
                if (kBy == kLie && live && (k == head || k == tail)) {
#pragma unroll
                    for (int j = 0; j < kV; ++j)
                        if (inside(k * kV + j)) to[k * width * kV + j] = from_f32<T>(e[j]);
                } else if (live && there[k]) {
                    pack<T, kBytes>(to + k * width * kV, e);
                }
            }
        };
        float2 x[kP];   // what the norm is of, then xh
        get(0, x);
        if (!kGated) {
            float2 r[kP];
            get(1, r);
#pragma unroll
            for (int u = 0; u < kP; ++u) x[u] = fma2(l[u], x[u], r[u]);
        }
        if constexpr (!kBwd) {
            float2 z[kP];
            if (kGated && kLoad) get(1, z);   // its trip beside the first sum's
            if (kOp == kAddFwd) put(1, x);
            float mu = 0.f;
            if (p.layer) {
                float2 s = both(0.f);
#pragma unroll
                for (int u = 0; u < kP; ++u) s = add2(s, x[u]);
                mu = sum(s.x + s.y) * inv;
#pragma unroll
                for (int u = 0; u < kP; ++u) {
                    x[u] = add2(x[u], both(-mu));
                    if (!inside(2 * u)) x[u].x = 0.f;
                    if (!inside(2 * u + 1)) x[u].y = 0.f;
                }
            }
            float2 q = both(0.f);
#pragma unroll
            for (int u = 0; u < kP; ++u) q = fma2(x[u], x[u], q);
            const float rs = reciprocal_root(sum(q.x + q.y) * inv + p.eps);
            if (live && lane == 0) {
                if (p.mean) p.mean[row] = mu;
                if (p.rstd) p.rstd[row] = rs;
            }
            if (kGated && !kLoad) get(1, z);
#pragma unroll
            for (int u = 0; u < kP; ++u) {
                x[u] = mul2(mul2(x[u], both(rs)), w[u]);
                if (kGated) x[u] = mul2(x[u], activation<T>(z[u], p.silu));
            }
            put(0, x);
        } else {
            const float rs = !live ? 0.f : kLoad ? p.rstd[row] : stats[(stage * 2) * kBlock + threadIdx.x];
            const float mu =
                !live || !p.layer ? 0.f : kLoad ? p.mean[row] : stats[(stage * 2 + 1) * kBlock + threadIdx.x];
            constexpr bool kEarly = kOp == kAddBwd && kLoad && kE <= 8;   // what is used after the sums, asked for here
            float2 x0[kEarly ? kP : 1], ds[kEarly ? kP : 1];
            if constexpr (kEarly) {
                get(0, x0);
                if (four) get(3, ds);
            }
            float2 d[kP];   // dL/dxh; zero past the row's end, where nothing is added to any sum then
            float2 s0 = both(0.f), s1 = s0;
            get(2, d);
            if (kGated) {
                float2 z[kP];
                get(1, z);
#pragma unroll
                for (int u = 0; u < kP; ++u) {
                    float2 slope;
                    const float2 a = activation<T>(z[u], p.silu, slope);
                    x[u] = mul2(add2(x[u], both(-mu)), both(rs));
                    const float2 dyx = mul2(d[u], x[u]);
                    dw[u] = fma2(dyx, a, dw[u]);
                    z[u] = mul2(mul2(dyx, w[u]), slope);
                    d[u] = mul2(mul2(d[u], w[u]), a);
                    s0 = add2(s0, d[u]);
                    s1 = fma2(d[u], x[u], s1);
                }
                put(1, z);
            } else {
#pragma unroll
                for (int u = 0; u < kP; ++u) {
                    x[u] = mul2(add2(x[u], both(-mu)), both(rs));
                    dw[u] = fma2(d[u], x[u], dw[u]);
                    d[u] = mul2(d[u], w[u]);
                    s0 = add2(s0, d[u]);
                    s1 = fma2(d[u], x[u], s1);
                }
            }
            float m1 = 0.f, m2;
            if (p.layer) {
                const float2 m = sum(make_float2(s0.x + s0.y, s1.x + s1.y));
                m1 = m.x * inv;
                m2 = m.y * inv;
            } else {
                m2 = sum(s1.x + s1.y) * inv;
            }
            const float2 c0 = both(rs), c1 = both(-rs * m1), c2 = both(-rs * m2);
#pragma unroll
            for (int u = 0; u < kP; ++u) d[u] = fma2(c0, d[u], fma2(c2, x[u], c1));
            if (four) {
                if constexpr (!kEarly) get(3, x);
#pragma unroll
                for (int u = 0; u < kP; ++u) d[u] = add2(d[u], kEarly ? ds[kEarly ? u : 0] : x[u]);
            }
            put(0, d);
            if (kOp == kAddBwd && p.l) {
                if constexpr (!kEarly) get(0, x);
#pragma unroll
                for (int u = 0; u < kP; ++u) {
                    dl[u] = fma2(d[u], kEarly ? x0[kEarly ? u : 0] : x[u], dl[u]);
                    d[u] = mul2(d[u], l[u]);
                }
                put(1, d);
            }
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    if constexpr (kBwd) {
        copies_wait<0>();
        if (!p.part) return;
        // one row of each sum a CTA: first over the teams of a warp, which have the same columns, then over the rest
        constexpr int kSums = kOp == kAddBwd ? 2 : 1;
        const int owners = width < 32 ? kBlock / 32 : teams, owner = width < 32 ? threadIdx.x / 32 : team;
        float *const acc = reinterpret_cast<float *>(ring);   // [owners][n]
        float *to = p.part + static_cast<int64_t>(blockIdx.x) * kSums * p.n;
#pragma unroll
        for (int which = 0; which < kSums; ++which, to += p.n) {
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kE; ++u) {
                const float2 &pair = which ? dl[kOp == kAddBwd ? u / 2 : 0] : dw[u / 2];
                float v = part(pair, u % 2);
                for (int off = width; off < 32; off *= 2) v += across(v, off);
                const int c = column(u);
                if (c >= 0 && c < p.n && (threadIdx.x & 31) == lane % 32) acc[owner * p.n + c] = v;
            }
            __syncthreads();
            for (int c = threadIdx.x; c < p.n; c += kBlock) {
                float v = acc[c];
                for (int q = 1; q < owners; ++q) v += acc[q * p.n + c];
                to[c] = v;
            }
        }
    }
}

// ---- any other row, of any length and alignment: bf16 above 8192 values, fp32 above 8192 (4096 where rows fit no 16 bytes: by
// single loads above, without a ring). A CTA takes rows one after the other, value by value, and reads each twice, three
// times with a mean; backward twice, and a third time for dw and dl. From memory and then from L1 or L2: 8192 x 12288 bf16
// gated 450 and 712 us, residual 273 and 1274, where the bytes of one pass take 89, 148, 119 and 178.
constexpr int kAnyBlock = 512;
template <typename V>
__device__ __forceinline__ V block_sum(V v, float2 *slots) {
    for (int off = 16; off; off >>= 1) v = add(v, across(v, off));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) reinterpret_cast<V &>(slots[threadIdx.x / 32]) = v;
    __syncthreads();
    v = reinterpret_cast<const V &>(slots[0]);
    for (int i = 1; i < kAnyBlock / 32; ++i) v = add(v, reinterpret_cast<const V &>(slots[i]));
    return v;
}

// One column of a row: what the norm is of; and dL/dxh with what else the gate's gradient takes.
template <typename T, Op kOp>
struct Column {
    const NormArgs &p;
    int64_t o, oz;
    const float *w;
    __device__ __forceinline__ Column(const NormArgs &a, int64_t row) : p(a), o(row * a.n), oz(o), w(a.w) {
        if (gated(kOp) && p.z_stride) oz = row / p.groups * p.z_stride + row % p.groups * p.n;
        if (w && p.w_groups) w += row % p.groups * p.n;
    }
    __device__ __forceinline__ float in(int i, int64_t at) const { return to_f32(static_cast<const T *>(p.in[i])[at]); }
    __device__ __forceinline__ float value(int c) const {
        return gated(kOp) ? in(0, o + c) : fmaf(p.l ? p.l[c] : 1.f, in(0, o + c), in(1, o + c));
    }
    __device__ __forceinline__ float weight(int c) const { return w ? w[c] : 1.f; }
    __device__ __forceinline__ float act(int c, float &slope) const {
        slope = 0.f;
        if (!gated(kOp)) return 1.f;
        float2 both_slopes;
        const float a = activation<T>(both(in(1, oz + c)), p.silu, both_slopes).x;
        slope = both_slopes.x;
        return a;
    }
    __device__ __forceinline__ void put(int i, int c, float v) const {
        static_cast<T *>(p.out[i])[o + c] = from_f32<T>(v);
    }
};

template <typename T, Op kOp>
__global__ void __launch_bounds__(kAnyBlock) block_norm_any_fwd_kernel(NormArgs p) {
    __shared__ float2 slots[32];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const Column<T, kOp> at(p, row);
        float mu = 0.f, q = 0.f, slope;
        if (p.layer) {
            for (int c = threadIdx.x; c < p.n; c += kAnyBlock) mu += at.value(c);
            mu = block_sum(mu, slots) / p.n;
        }
        for (int c = threadIdx.x; c < p.n; c += kAnyBlock) {
            const float d = at.value(c) - mu;
            q = fmaf(d, d, q);
        }
        const float rs = reciprocal_root(block_sum(q, slots) / p.n + p.eps);
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mu;
            if (p.rstd) p.rstd[row] = rs;
        }
        for (int c = threadIdx.x; c < p.n; c += kAnyBlock) {
            const float v = at.value(c);
            if (kOp == kAddFwd) at.put(1, c, v);
            at.put(0, c, (v - mu) * rs * at.weight(c) * at.act(c, slope));
        }
    }
}

template <typename T, Op kOp>
__global__ void __launch_bounds__(kAnyBlock) block_norm_any_bwd_kernel(NormArgs p) {
    __shared__ float2 slots[32];
    dependency_release();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const Column<T, kOp> at(p, row);
        const float mu = p.mean ? p.mean[row] : 0.f, rs = p.rstd[row];
        float2 s = make_float2(0.f, 0.f);
        float slope;
        for (int c = threadIdx.x; c < p.n; c += kAnyBlock) {
            const float d = at.in(2, at.o + c) * at.weight(c) * at.act(c, slope);
            s.x += d;
            s.y = fmaf(d, (at.value(c) - mu) * rs, s.y);
        }
        s = block_sum(s, slots);
        const float m1 = p.layer ? s.x / p.n : 0.f, m2 = s.y / p.n;
        for (int c = threadIdx.x; c < p.n; c += kAnyBlock) {
            const float xh = (at.value(c) - mu) * rs, dyw = at.in(2, at.o + c) * at.weight(c);
            const float d = dyw * at.act(c, slope);
            float o = rs * (d - m1 - xh * m2);
            if (kOp == kAddBwd) {
                if (p.in[3]) o += at.in(3, at.o + c);
                at.put(0, c, o);
                if (p.l) at.put(1, c, o * p.l[c]);
            } else {
                at.put(0, c, o);
                at.put(1, c, dyw * xh * slope);
            }
        }
        if (kOp == kAddBwd && threadIdx.x == 0 && p.part)   // the means, for dl
            reinterpret_cast<float2 *>(p.part)[row] = make_float2(m1, m2);
    }
}

// dw and dl of those: a CTA's lanes along 32 columns, its warps along the rows of one part of them.
template <typename T, Op kOp>
__global__ void __launch_bounds__(1024) block_norm_any_sums_kernel(NormArgs p, const float2 *means, float *part) {
    constexpr int kSums = kOp == kAddBwd ? 2 : 1;
    __shared__ float2 slots[32][33];
    dependency_release();
    dependency_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    const int groups = p.w_groups ? p.groups : 1;
    const int64_t each = (p.rows / groups + gridDim.z - 1) / gridDim.z, r0 = blockIdx.z * each;
    const int64_t r1 = r0 + each < p.rows / groups ? r0 + each : p.rows / groups;
    float2 s = make_float2(0.f, 0.f);
    for (int64_t r = r0 + warp; c < p.n && r < r1; r += 32) {
        const int64_t row = r * groups + blockIdx.y;
        const Column<T, kOp> at(p, row);
        const float mu = p.mean ? p.mean[row] : 0.f, rs = p.rstd[row], xh = (at.value(c) - mu) * rs;
        const float dy = at.in(2, at.o + c);
        float slope;
        s.x = fmaf(dy * xh, at.act(c, slope), s.x);
        if (kSums == 2 && p.l) {
            const float2 m = means[row];
            float o = rs * (dy * at.weight(c) - m.x - xh * m.y);
            if (p.in[3]) o += at.in(3, at.o + c);
            s.y = fmaf(o, at.in(0, at.o + c), s.y);
        }
    }
    slots[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < p.n) {
        for (int i = 1; i < 32; ++i) s = add(s, slots[i][lane]);
        float *to = part + (static_cast<int64_t>(blockIdx.z) * groups + blockIdx.y) * kSums * p.n + c;
        to[0] = s.x;
        if (kSums == 2) to[p.n] = s.y;
    }
}

// The parts' rows added up in their order: part i of group g is row i * groups + g.
__global__ void __launch_bounds__(1024) block_norm_join_kernel(const float *part, float *dw, float *dl, int parts,
                                                               int groups, int n, int sums) {
    __shared__ float2 slots[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    dependency_wait();
    float2 s = make_float2(0.f, 0.f);
    if (c < n)
#pragma unroll 4
        for (int i = warp; i < parts; i += 32) {
            const float *from = part + (static_cast<int64_t>(i) * groups + blockIdx.y) * sums * n + c;
            s.x += from[0];
            if (sums == 2) s.y += from[n];
        }
    slots[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < n) {
        for (int i = 1; i < 32; ++i) s = add(s, slots[i][lane]);
        if (dw) dw[static_cast<int64_t>(blockIdx.y) * n + c] = s.x;
        if (dl) dl[c] = s.y;
    }
}

// ------------------------------------------------------------------------------------ host side
constexpr int kSms = 152;

// Groups with weights of their own are a grid's axis; others are the gate's rows between two strides, as many as there are
// tokens.
kla_status check(int64_t rows, int groups, int n, kla_dtype dtype, bool own) {
    if (rows < 0 || groups < 1 || n < 1) return KLA_ERR_INVALID_ARG;
    if (dtype != KLA_DTYPE_F32 && dtype != KLA_DTYPE_BF16) return KLA_ERR_INVALID_ARG;
    if (n < 3 || n > 65536 || (own && groups > 65535) || rows > INT_MAX / groups) return KLA_ERR_UNSUPPORTED;
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

// Rows as they lie: how many start differently, and of how many accesses one is at most.
int starts_of(int n, int esz) {
    int m = 1;
    while (static_cast<int64_t>(n) * esz * m % 16) m *= 2;
    return m;
}
int most_of(int n, int esz) { return (n * esz + 2 * (16 - esz)) / 16; }
// Classes of rows: of groups with weights of their own, and of those that start alike.
int classes_of(int groups, int starts) {
    int m = groups;
    while (m % starts) m *= 2;
    return m;
}
// Whether rows are taken as they lie, given that all of a row's tensors start alike: where a team holds them, and a part
// of the sums for each class is not too many.
bool lies(int groups, int n, int esz) {
    const int starts = starts_of(n, esz);
    return starts > 1 && most_of(n, esz) <= 2 * kMostBlock && classes_of(groups, starts) <= 4 * kSms;
}
// How rows are taken: `bytes` of an access (0: by block_norm_any_*), accesses of a thread, threads of a team and of a
// CTA.
struct Plan {
    int bytes, nv, width, block;
    int grid;   // CTAs, a multiple of the classes of rows
    bool direct() const { return bytes == 2 || nv > (bytes == 16 ? 2 : 8); }
};
// Rows start on `bytes` bytes, or as they lie (`lie`, 16). A thread takes 32 bytes of a row, so that a row's share of the sums, the addresses and
// the loop is spread over many values (with 16 bytes 32768 x 16 heads of 128 took 85 us instead of 78, and 124
// instead of 120), or 64 of rows of fp32 that shared memory holds no two of.
Plan plan(int64_t rows, int classes, int n, int esz, int bytes, bool lie, Op op) {
    Plan p{bytes, bytes == 16 ? 2 : 8, 4, 256, 0};
    const int accesses = lie ? most_of(n, esz) : n * esz / bytes;
    if ((esz == 4 || bytes == 2) && accesses > kMostBlock * p.nv) p.nv *= 2;
    if (accesses > kMostBlock * p.nv) {
        p.bytes = 0;
        const int64_t most = kSms * 4;
        p.grid = static_cast<int>(rows < most ? rows : most);
        return p;
    }
    while (p.width * p.nv < accesses) p.width *= 2;
    if (p.width > p.block || p.nv == (bytes == 16 ? 4 : 16)) p.block = kMostBlock;
    const int64_t teams = p.block / p.width, of_class = (rows / classes + teams - 1) / teams;
    int64_t want = (static_cast<int64_t>(kSms) * ctas(op, p.nv * bytes / esz, p.block) + classes - 1) / classes;
    if (want > of_class) want = of_class;
    p.grid = static_cast<int>((want < 1 ? 1 : want) * classes);
    return p;
}
// Parts of the rows that block_norm_any_sums_kernel takes side by side.
int any_parts(int64_t rows, int groups, int n) {
    const int64_t tiles = static_cast<int64_t>((n + 31) / 32) * groups, most = (rows / groups + 255) / 256;
    int64_t parts = 2 * kSms / tiles;
    if (parts > most) parts = most;
    return static_cast<int>(parts < 1 ? 1 : parts);
}
size_t any_means_bytes(int64_t rows) { return (static_cast<size_t>(rows) * sizeof(float2) + 15) / 16 * 16; }
// Scratch of the backward pass, for whatever alignment the call has.
size_t workspace_bytes_of(int64_t rows, int groups, int n, int esz, Op op) {
    const int sums = op == kAddBwd ? 2 : 1;
    size_t most = any_means_bytes(rows) + static_cast<size_t>(any_parts(rows, groups, n)) * groups * sums * n * 4;
    for (int bytes : {16, 4, 2}) {
        if (bytes < esz) continue;
        const bool lie = bytes == 16 && lies(groups, n, esz);
        const Plan p = plan(rows, lie ? classes_of(groups, starts_of(n, esz)) : groups, n, esz, bytes, lie, op);
        const size_t need = p.bytes ? static_cast<size_t>(p.grid) * sums * n * 4 : 0;
        if (need > most) most = need;
    }
    return most;
}

template <typename T, int kBytes, int kNV, Op kOp, int kBlock, Rows kBy>
cudaError_t run_rows(const NormArgs &a, const Plan &p, cudaStream_t s) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> done[kMaxDevices];
    constexpr int kS = stages(kOp, kNV * kBytes / static_cast<int>(sizeof(T)), kNV * kBytes, kBlock);
    constexpr int kSums = backward(kOp) ? kBlock * kNV * kBytes / static_cast<int>(sizeof(T)) * 4 : 0;
    constexpr int kRing =
        kBy == kDirect ? kSums : kS * kBlock * (inputs(kOp) * kNV * kBytes + (backward(kOp) ? 8 : 0));
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    auto kernel = block_norm_kernel<T, kBytes, kNV, kOp, kBlock, kBy>;
    if (!done[dev].load(std::memory_order_acquire)) {   // once per device and kernel: the attribute outlasts the call
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing)) != cudaSuccess)
            return e;
        done[dev].store(true, std::memory_order_release);
    }
    static_assert(kRing >= kSums, "a CTA's sums are joined there");
    kernel<<<p.grid, kBlock, kRing, s>>>(a, p.width);
    return cudaGetLastError();
}

// The rows' kernel, and in the backward pass the sums over its parts. `workspace` is NULL where no sum is wanted.
template <typename T, Op kOp>
cudaError_t run(NormArgs a, float *dw, float *dl, void *workspace, cudaStream_t s) {
    constexpr int kSums = kOp == kAddBwd ? 2 : 1;
    const int groups = a.w_groups ? a.groups : 1, esz = sizeof(T);
    auto start = [&](int bytes) {
        for (const void *q : {a.in[0], a.in[1], a.in[2], a.in[3], static_cast<const void *>(a.out[0]),
                              static_cast<const void *>(a.out[1])})
            if (!aligned(q, bytes)) return false;
        return true;
    };
    auto fits = [&](int bytes) { return a.n * esz % bytes == 0 && (a.z_stride * esz) % bytes == 0 && start(bytes); };
    // the gate's rows start as x's do
    const bool alike = a.z_stride == 0 || (a.z_stride - static_cast<int64_t>(a.groups) * a.n) * esz % 16 == 0;
    const bool lie = alike && start(16) && lies(groups, a.n, esz);
    a.classes = lie ? classes_of(groups, starts_of(a.n, esz)) : groups;
    const Plan p = plan(a.rows, a.classes, a.n, esz, lie || fits(16) ? 16 : fits(4) ? 4 : 2, lie, kOp);
    cudaError_t e;
    if (p.bytes) {
        a.part = static_cast<float *>(workspace);
        const bool large = p.block == 512;
        if constexpr (sizeof(T) == 4) {
            if (p.direct())
                e = p.bytes == 16 ? run_rows<T, 16, 4, kOp, 512, kDirect>(a, p, s)
                                  : run_rows<T, 4, 16, kOp, 512, kDirect>(a, p, s);
        } else {
            if (p.direct())
                e = !large      ? run_rows<T, 2, 8, kOp, 256, kDirect>(a, p, s)
                    : p.nv == 8 ? run_rows<T, 2, 8, kOp, 512, kDirect>(a, p, s)
                                : run_rows<T, 2, 16, kOp, 512, kDirect>(a, p, s);
        }
        if (p.direct()) {
        } else if (lie) {
            e = large ? run_rows<T, 16, 2, kOp, 512, kLie>(a, p, s) : run_rows<T, 16, 2, kOp, 256, kLie>(a, p, s);
        } else if (large) {
            e = p.bytes == 16 ? run_rows<T, 16, 2, kOp, 512, kRing>(a, p, s) : run_rows<T, 4, 8, kOp, 512, kRing>(a, p, s);
        } else {
            e = p.bytes == 16 ? run_rows<T, 16, 2, kOp, 256, kRing>(a, p, s) : run_rows<T, 4, 8, kOp, 256, kRing>(a, p, s);
        }
        if (e != cudaSuccess || !workspace) return e;
        return launch_dependent(block_norm_join_kernel, dim3((a.n + 31) / 32, groups), 1024, 0, s, a.part, dw, dl,
                                p.grid / groups, groups, a.n, kSums);
    }
    if constexpr (!backward(kOp)) {
        block_norm_any_fwd_kernel<T, kOp><<<p.grid, kAnyBlock, 0, s>>>(a);
        return cudaGetLastError();
    } else {
        float *part = workspace ? reinterpret_cast<float *>(static_cast<char *>(workspace) + any_means_bytes(a.rows))
                                : nullptr;
        a.part = static_cast<float *>(workspace);
        block_norm_any_bwd_kernel<T, kOp><<<p.grid, kAnyBlock, 0, s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess || !workspace) return e;
        const int parts = any_parts(a.rows, groups, a.n);
        e = launch_dependent(block_norm_any_sums_kernel<T, kOp>, dim3((a.n + 31) / 32, groups, parts), 1024, 0, s, a,
                             static_cast<const float2 *>(workspace), part);
        if (e != cudaSuccess) return e;
        return launch_dependent(block_norm_join_kernel, dim3((a.n + 31) / 32, groups), 1024, 0, s, part, dw, dl, parts,
                                groups, a.n, kSums);
    }
}
template <Op kOp>
kla_status run(const NormArgs &a, kla_dtype dtype, float *dw, float *dl, void *workspace, void *stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == KLA_DTYPE_BF16 ? run<__nv_bfloat16, kOp>(a, dw, dl, workspace, s)
                                                  : run<float, kOp>(a, dw, dl, workspace, s);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // namespace
}  // namespace kla

extern "C" {

kla_status kla_gated_norm_fwd(const void *x, const void *gate, int64_t gate_stride, const float *weight,
                              int weight_groups, void *y, float *mean, float *rstd, int64_t rows, int groups, int n,
                              kla_dtype dtype, kla_norm_kind norm, kla_activation act, float eps, void *stream) {
    using namespace kla;
    const kla_status st = check(rows, groups, n, dtype, weight_groups != 0);
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
    p.in[0] = x; p.in[1] = gate; p.w = weight; p.w_groups = weight_groups != 0; p.out[0] = y;
    p.z_stride = gate_stride == static_cast<int64_t>(row) ? 0 : gate_stride;
    p.mean = mean; p.rstd = rstd; p.rows = rows * groups; p.groups = groups; p.n = n; p.eps = eps;
    p.layer = norm == KLA_NORM_LAYER; p.silu = act == KLA_ACT_SILU;
    return run<kGatedFwd>(p, dtype, nullptr, nullptr, nullptr, stream);
}

size_t kla_gated_norm_bwd_workspace_size(int64_t rows, int groups, int n, kla_dtype dtype, int weight_groups) {
    if (kla::check(rows, groups, n, dtype, weight_groups != 0) != KLA_OK || rows == 0) return 0;
    return kla::workspace_bytes_of(rows * groups, weight_groups ? groups : 1, n, dtype == KLA_DTYPE_BF16 ? 2 : 4,
                                   kla::kGatedBwd);
}

kla_status kla_gated_norm_bwd(const void *dy, const void *x, const void *gate, int64_t gate_stride,
                              const float *weight, int weight_groups, const float *mean, const float *rstd, void *dx,
                              void *dgate, float *dweight, int64_t rows, int groups, int n, kla_dtype dtype,
                              kla_activation act, void *workspace, size_t workspace_bytes, void *stream) {
    using namespace kla;
    const kla_status st = check(rows, groups, n, dtype, weight_groups != 0);
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
    p.in[0] = x; p.in[1] = gate; p.in[2] = dy; p.w = weight; p.w_groups = weight_groups != 0;
    p.z_stride = gate_stride == static_cast<int64_t>(row) ? 0 : gate_stride;
    p.out[0] = dx; p.out[1] = dgate; p.mean = const_cast<float *>(mean); p.rstd = const_cast<float *>(rstd);
    p.rows = rows * groups; p.groups = groups; p.n = n; p.layer = mean != nullptr; p.silu = act == KLA_ACT_SILU;
    return run<kGatedBwd>(p, dtype, dweight, nullptr, dweight ? workspace : nullptr, stream);
}

kla_status kla_add_norm_fwd(const void *x, const void *residual, const float *weight, const float *scale, void *y,
                            void *sum, float *mean, float *rstd, int64_t rows, int n, kla_dtype dtype,
                            kla_norm_kind norm, float eps, void *stream) {
    using namespace kla;
    const kla_status st = check(rows, 1, n, dtype, false);
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
    p.in[0] = x; p.in[1] = residual; p.w = weight; p.l = scale; p.out[0] = y; p.out[1] = sum; p.mean = mean;
    p.rstd = rstd; p.rows = rows; p.groups = 1; p.n = n; p.eps = eps; p.layer = norm == KLA_NORM_LAYER;
    return run<kAddFwd>(p, dtype, nullptr, nullptr, nullptr, stream);
}

size_t kla_add_norm_bwd_workspace_size(int64_t rows, int n, kla_dtype dtype) {
    if (kla::check(rows, 1, n, dtype, false) != KLA_OK || rows == 0) return 0;
    return kla::workspace_bytes_of(rows, 1, n, dtype == KLA_DTYPE_BF16 ? 2 : 4, kla::kAddBwd);
}

kla_status kla_add_norm_bwd(const void *dy, const void *dsum, const void *x, const void *residual,
                            const float *weight, const float *scale, const float *mean, const float *rstd, void *dx,
                            void *dresidual, float *dweight, float *dscale, int64_t rows, int n, kla_dtype dtype,
                            void *workspace, size_t workspace_bytes, void *stream) {
    using namespace kla;
    const kla_status st = check(rows, 1, n, dtype, false);
    if (st != KLA_OK) return st;
    if (!scale && (dx || dscale)) return KLA_ERR_INVALID_ARG;
    if (rows > 0 && (!dy || !x || !residual || !rstd || !dresidual || (scale && !dx))) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(dy, esz) || !aligned(dsum, esz) || !aligned(x, esz) || !aligned(residual, esz) ||
        !aligned(dx, esz) || !aligned(dresidual, esz) || !aligned(weight, 4) || !aligned(scale, 4) || !aligned(mean, 4) ||
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
    const Span ins[] = {span(dy, all), span(dsum, all), span(x, all), span(residual, all),
                        span(weight, par), span(scale, par), span(mean, stat), span(rstd, stat)};
    if (!apart(outs, ins)) return KLA_ERR_INVALID_ARG;
    NormArgs p{};
    p.in[0] = x; p.in[1] = residual; p.in[2] = dy; p.in[3] = dsum; p.w = weight; p.l = scale; p.out[0] = dresidual;
    p.out[1] = dx; p.mean = const_cast<float *>(mean); p.rstd = const_cast<float *>(rstd);
    p.rows = rows; p.groups = 1; p.n = n; p.layer = mean != nullptr;
    return run<kAddBwd>(p, dtype, dweight, dscale, dweight || dscale ? workspace : nullptr, stream);
}

}  // extern "C"
