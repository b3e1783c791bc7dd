// kla_rotary.cu -- rotary positions: pair i of a head's first `rot` values, (u, v), turned by position freqs[i].
//
// An angle counts as a 64-bit fraction of a turn: the frequency as turns a token, times 2^64, modulo 2^64; times the
// position in integers, whose overflow is whole turns. Its upper 32 bits, as a signed number of half turns, are what
// sine and cosine take. The product in fp32 would lose a bit with every doubling of the position, and one in fp64
// would cost tens of instructions of a pipe that does two a cycle and SM.
// What bounds it is the memory, one read and one write of every value. Measured: 8 x 4096 tokens of 32 heads of 128
// bf16, slices of one projection, 88 us in a row of calls (6.1 TB/s, 90 % of a copy's rate), 93 after other work; 40 heads
// in fp32 212 us (6.3 TB/s). Of heads whose pairs fit no wide accesses single values in shared memory bound it: 126 of 128
// values turned 130 us, 20 of 80 95 (floors 79 and 49); in fp32 179 and 114 (158 and 99).
#include <type_traits>

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

// Turns a token, as a fraction of 2^64. Of f / 2 pi two roundings of 2^-53 are lost, 2^-54.6 f of a turn, and the position
// times as much of the angle; of its sign and upper 32 bits fp32 keeps 2^-26 of a turn.
__device__ __forceinline__ unsigned long long turn_rate(float freq) {
    double t = static_cast<double>(freq) * 0.15915494309189533577;
    t -= floor(t);
    return static_cast<unsigned long long>(t * 18446744073709551616.0);
}
// Sine and cosine of the angle at a position. bf16 takes the hardware's, whose 2^-20 of error in [-pi, pi] is far
// below the values' 2^-9.
template <typename T>
__device__ __forceinline__ void turned(unsigned long long rate, long long position, float &s, float &c) {
    const float half_turns =
        static_cast<float>(static_cast<int>((rate * static_cast<unsigned long long>(position)) >> 32)) * 0x1p-31f;
    if (sizeof(T) == 4) {
        sincospif(half_turns, &s, &c);
    } else {
        const float a = half_turns * 3.14159265358979f;
        asm("sin.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(a));
        asm("cos.approx.ftz.f32 %0, %1;" : "=f"(c) : "f"(a));
    }
}

// kV neighbouring values, moved in one access.
template <typename T, int kV>
struct alignas(sizeof(T) * kV) Values {
    static constexpr int kBytes = sizeof(T) * kV;
    typename std::conditional<kBytes == 2, uint16_t, uint32_t>::type r[kBytes == 2 ? 1 : kBytes / 4];
    __device__ __forceinline__ void get(float *v) const {
        if constexpr (kBytes == 2) {
            v[0] = __uint_as_float(static_cast<uint32_t>(r[0]) << 16);
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < kBytes / 4; ++i) {
                v[2 * i] = __uint_as_float(r[i] << 16);
                v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) v[i] = __uint_as_float(r[i]);
        }
    }
    __device__ __forceinline__ void set(const float *v) {
        if constexpr (kBytes == 2) {
            r[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
        } else if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < kBytes / 4; ++i) r[i] = ptx::pack_bf16(v[2 * i], v[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < kV; ++i) r[i] = __float_as_uint(v[i]);
        }
    }
};

// A warp takes tokens one after the other (or, where tokens are few, a part of one's heads). A lane has one unit of a
// head, two accesses of kV values: kV pairs, whose sines and cosines it takes once for all of its heads, or values that
// are copied. kAtOnce heads are on their way at once, the first of them while the sines are taken. Where a warp's
// lanes hold all heads of a token (kTokens), it is as many tokens that are on their way at once, each with sines of its
// own. Of the 64-bit rates the CTA makes one table, as fp64 is slow.
constexpr int kBlock = 256;
constexpr int at_once(int bytes, bool tokens) { return bytes == 16 || tokens ? 4 : 8; }
constexpr int ctas(int bytes) { return bytes >= 8 ? 3 : 4; }   // an SM's registers hold
// The units of a head, lanes of it and heads side by side in a warp.
struct Units {
    int turning, rest, all, across, side;
    __host__ __device__ Units(int d, int rot, int v) {
        turning = rot / 2 / v;
        rest = (d - rot) / v;
        all = turning + (rest + 1) / 2;
        across = all < 32 ? all : 32;
        side = 32 / across;
    }
};
template <typename T, int kV, bool kHalf, bool kTokens>
__global__ void __launch_bounds__(kBlock, ctas(sizeof(T) * kV)) rotary_kernel(RotaryArgs p, int parts) {
    using X = Values<T, kV>;
    constexpr int kAtOnce = at_once(sizeof(T) * kV, kTokens);
    extern __shared__ unsigned long long rates[];
    const int pairs = p.rot / 2, lane = threadIdx.x & 31, heads = p.H[0] + p.H[1];
    for (int i = threadIdx.x; i < pairs; i += kBlock) rates[i] = turn_rate(p.freqs[i]);
    __syncthreads();
    const Units n(p.d, p.rot, kV);
    const int lane_u = lane % n.across, lane_h = lane / n.across;
    // kTokens: `side` of a warp's tokens side by side, and this lane's head and place among them
    const int side = kTokens ? n.side / heads : n.side, head = lane_h % heads, place = lane_h / heads;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * (kBlock / 32);
    const int64_t first_job = static_cast<int64_t>(blockIdx.x) * (kBlock / 32) + threadIdx.x / 32;
    // of a token and a head: position, and element offsets of its values
    auto position = [&](unsigned token) -> long long {
        if (!p.positions) return token % static_cast<unsigned>(p.T);
        return p.wide ? static_cast<const long long *>(p.positions)[token] : static_cast<const int *>(p.positions)[token];
    };
    auto angles = [&](int u, long long at, float (&c)[kV], float (&s)[kV]) {
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            turned<T>(rates[u * kV + j], at, s[j], c[j]);
            c[j] *= p.scale;
            s[j] *= p.inverse ? -p.scale : p.scale;
        }
    };
    auto turn = [&](X &x0, X &x1, const float (&c)[kV], const float (&s)[kV]) {
        float v[2 * kV];
        x0.get(v);
        x1.get(v + kV);
#pragma unroll
        for (int j = 0; j < kV; ++j) {   // pair j: values j and kV + j, or 2 j and 2 j + 1
            float &a = v[kHalf ? j : 2 * j], &e = v[kHalf ? kV + j : 2 * j + 1];
            const float old = a;
            a = fmaf(old, c[j], -e * s[j]);
            e = fmaf(e, c[j], old * s[j]);
        }
        x0.set(v);
        x1.set(v + kV);
    };
    struct Unit {   // its two accesses
        bool turns, two;
        int i0, i1;
    };
    auto unit = [&](int u) {
        Unit r;
        r.turns = u < n.turning;
        r.i0 = r.turns ? (kHalf ? 1 : 2) * u * kV : p.rot + 2 * (u - n.turning) * kV;
        r.i1 = r.turns && kHalf ? r.i0 + pairs : r.i0 + kV;
        r.two = r.turns || 2 * (u - n.turning) + 1 < n.rest;
        return r;
    };
    if constexpr (kTokens) {
        const int m = head < p.H[0] ? 0 : 1;
        const int64_t per = static_cast<int64_t>(side) * kAtOnce, jobs = (p.tokens + per - 1) / per;
        const T *in = static_cast<const T *>(p.in[m]) + (m ? head - p.H[0] : head) * p.is[m][2];
        T *out = static_cast<T *>(p.out[m]) + (m ? head - p.H[0] : head) * p.os[m][2];
        if (place >= side) return;
        const Unit w = unit(lane_u);
        for (int64_t job = first_job; job < jobs; job += warps) {
            X x0[kAtOnce], x1[kAtOnce];
            long long at[kAtOnce];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const int64_t token = job * per + q * side + place;
                if (token >= p.tokens) continue;
                const unsigned b = static_cast<unsigned>(token) / static_cast<unsigned>(p.T);
                const unsigned t = static_cast<unsigned>(token) - b * p.T;
                const T *f = in + b * p.is[m][0] + t * p.is[m][1];
                at[q] = position(static_cast<unsigned>(token));
                x0[q] = *reinterpret_cast<const X *>(f + w.i0);
                if (w.two) x1[q] = *reinterpret_cast<const X *>(f + w.i1);
            }
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const int64_t token = job * per + q * side + place;
                if (token >= p.tokens) continue;
                if (w.turns) {
                    float c[kV], s[kV];
                    angles(lane_u, at[q], c, s);
                    turn(x0[q], x1[q], c, s);
                }
                const unsigned b = static_cast<unsigned>(token) / static_cast<unsigned>(p.T);
                const unsigned t = static_cast<unsigned>(token) - b * p.T;
                T *o = out + b * p.os[m][0] + t * p.os[m][1];
                *reinterpret_cast<X *>(o + w.i0) = x0[q];
                if (w.two) *reinterpret_cast<X *>(o + w.i1) = x1[q];
            }
        }
    } else {
        const int64_t jobs = p.tokens * parts;
        if (lane_h >= side) return;
        for (int64_t job = first_job; job < jobs; job += warps) {
            const unsigned token = static_cast<unsigned>(job / parts), slice = static_cast<unsigned>(job % parts);
            const unsigned b = token / static_cast<unsigned>(p.T), t = token - b * p.T;
            const long long at = position(token);
            const T *in0 = static_cast<const T *>(p.in[0]) + b * p.is[0][0] + t * p.is[0][1];
            const T *in1 = static_cast<const T *>(p.in[1]) + b * p.is[1][0] + t * p.is[1][1] - p.H[0] * p.is[1][2];
            T *out0 = static_cast<T *>(p.out[0]) + b * p.os[0][0] + t * p.os[0][1];
            T *out1 = static_cast<T *>(p.out[1]) + b * p.os[1][0] + t * p.os[1][1] - p.H[0] * p.os[1][2];
            const int h0 = slice * side + lane_h, hop = side * parts;   // this lane's heads
            for (int u = lane_u; u < n.all; u += n.across) {
                const Unit w = unit(u);
                X x0[kAtOnce], x1[kAtOnce];
                auto load = [&](int h) {
#pragma unroll
                    for (int q = 0; q < kAtOnce; ++q, h += hop) {
                        const bool first = h < p.H[0];
                        const T *f = (first ? in0 : in1) + h * (first ? p.is[0][2] : p.is[1][2]);
                        if (h < heads) x0[q] = *reinterpret_cast<const X *>(f + w.i0);
                        if (h < heads && w.two) x1[q] = *reinterpret_cast<const X *>(f + w.i1);
                    }
                };
                if (h0 < heads) load(h0);
                float c[kV], s[kV];
                if (w.turns) angles(u, at, c, s);
                for (int h = h0; h < heads; h += hop * kAtOnce) {
                    if (h != h0) load(h);
#pragma unroll
                    for (int q = 0; q < kAtOnce; ++q) {
                        const int hq = h + q * hop;
                        if (w.turns) turn(x0[q], x1[q], c, s);
                        const bool first = hq < p.H[0];
                        T *o = (first ? out0 : out1) + hq * (first ? p.os[0][2] : p.os[1][2]);
                        if (hq < heads) *reinterpret_cast<X *>(o + w.i0) = x0[q];
                        if (hq < heads && w.two) *reinterpret_cast<X *>(o + w.i1) = x1[q];
                    }
                }
            }
        }
    }
}

// Heads that start on 16 bytes but whose pairs fit no such accesses (126 of 128 values turned, 20 of 80): a warp takes
// whole heads of a token into shared memory, as many as 4 KB hold, turns them there value by value, a lane the same
// pairs of all of them, and sends them on.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kBlock, 5) rotary_rows_kernel(RotaryArgs p, int at_once) {
    constexpr int kV = 16 / sizeof(T), kLoads = 4, kRows = 4;
    extern __shared__ __align__(16) unsigned char shared[];
    const int pairs = p.rot / 2, lane = threadIdx.x & 31, heads = p.H[0] + p.H[1], per_row = p.d / kV;
    unsigned long long *const rates = reinterpret_cast<unsigned long long *>(shared);
    for (int i = threadIdx.x; i < pairs; i += kBlock) rates[i] = turn_rate(p.freqs[i]);
    __syncthreads();
    T *const buf = reinterpret_cast<T *>(shared + (pairs + 1) / 2 * 16) + (threadIdx.x / 32) * at_once * p.d;
    uint4 *const wide = reinterpret_cast<uint4 *>(buf);
    const int slices = (heads + at_once - 1) / at_once;
    const int row_hop = 32 / per_row, col_hop = 32 % per_row;   // of a lane's next access
    const int64_t jobs = p.tokens * slices, warps = static_cast<int64_t>(gridDim.x) * (kBlock / 32);
    for (int64_t job = static_cast<int64_t>(blockIdx.x) * (kBlock / 32) + threadIdx.x / 32; job < jobs; job += warps) {
        const unsigned token = static_cast<unsigned>(job / slices), slice = static_cast<unsigned>(job - static_cast<int64_t>(token) * slices);
        const unsigned b = token / static_cast<unsigned>(p.T), t = token - b * p.T;
        const int first = slice * at_once, here = min(heads - first, at_once), accesses = here * per_row;
        const long long at = !p.positions ? t
                             : p.wide     ? static_cast<const long long *>(p.positions)[token]
                                          : static_cast<const int *>(p.positions)[token];
        const T *in0 = static_cast<const T *>(p.in[0]) + b * p.is[0][0] + t * p.is[0][1];
        const T *in1 = static_cast<const T *>(p.in[1]) + b * p.is[1][0] + t * p.is[1][1] - p.H[0] * p.is[1][2];
        T *out0 = static_cast<T *>(p.out[0]) + b * p.os[0][0] + t * p.os[0][1];
        T *out1 = static_cast<T *>(p.out[1]) + b * p.os[1][0] + t * p.os[1][1] - p.H[0] * p.os[1][2];
        int head = first + lane / per_row, col = lane % per_row;
        for (int i = lane; i < accesses; i += 32 * kLoads) {
            uint4 x[kLoads];
#pragma unroll
            for (int q = 0; q < kLoads; ++q) {
                const bool q0 = head < p.H[0];
                if (i + 32 * q < accesses)
                    x[q] = *reinterpret_cast<const uint4 *>((q0 ? in0 : in1) + head * (q0 ? p.is[0][2] : p.is[1][2]) + col * kV);
                col += col_hop;
                head += row_hop + (col >= per_row);
                if (col >= per_row) col -= per_row;
            }
#pragma unroll
            for (int q = 0; q < kLoads; ++q)
                if (i + 32 * q < accesses) wide[i + 32 * q] = x[q];
        }
        __syncwarp();
        for (int u = lane; u < pairs; u += 32) {
            const int i0 = kHalf ? u : 2 * u, i1 = kHalf ? u + pairs : 2 * u + 1;
            float s, c;
            turned<T>(rates[u], at, s, c);
            c *= p.scale;
            s *= p.inverse ? -p.scale : p.scale;
            T *x = buf;
            for (int row = 0; row < here; row += kRows, x += kRows * p.d) {
                float a[kRows], e[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    if (row + r < here) {
                        a[r] = to_f32(x[r * p.d + i0]);
                        e[r] = to_f32(x[r * p.d + i1]);
                    }
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    if (row + r < here) {
                        x[r * p.d + i0] = from_f32<T>(fmaf(a[r], c, -e[r] * s));
                        x[r * p.d + i1] = from_f32<T>(fmaf(e[r], c, a[r] * s));
                    }
            }
        }
        __syncwarp();
        head = first + lane / per_row;
        col = lane % per_row;
        for (int i = lane; i < accesses; i += 32) {
            const bool q0 = head < p.H[0];
            *reinterpret_cast<uint4 *>((q0 ? out0 : out1) + head * (q0 ? p.os[0][2] : p.os[1][2]) + col * kV) = wide[i];
            col += col_hop;
            head += row_hop + (col >= per_row);
            if (col >= per_row) col -= per_row;
        }
        __syncwarp();
    }
}
template <typename T>
cudaError_t run_rows(const RotaryArgs &p, bool half, cudaStream_t s) {
    constexpr int kSms = 152, kWarps = kBlock / 32, kCtas = 5;
    const int row = p.d * static_cast<int>(sizeof(T)), heads = p.H[0] + p.H[1];
    int at_once = row < 4096 ? 4096 / row : 1;
    if (at_once > heads) at_once = heads;
    // few tokens: fewer heads at once, as long as there are warps without any
    const int64_t each = (p.tokens * heads + kSms * kWarps - 1) / (kSms * kWarps);
    if (at_once > each) at_once = static_cast<int>(each);
    int64_t grid = (p.tokens * ((heads + at_once - 1) / at_once) + kWarps - 1) / kWarps;
    if (grid > kSms * kCtas) grid = kSms * kCtas;
    const size_t smem = (p.rot / 2 + 1) / 2 * 16 + static_cast<size_t>(kWarps) * at_once * row;   // 36 KB at most
    const unsigned g = static_cast<unsigned>(grid);
    if (half) rotary_rows_kernel<T, true><<<g, kBlock, smem, s>>>(p, at_once);
    else rotary_rows_kernel<T, false><<<g, kBlock, smem, s>>>(p, at_once);
    return cudaGetLastError();
}

template <typename T, int kV, bool kHalf>
cudaError_t run(const RotaryArgs &p, cudaStream_t s) {
    constexpr int kSms = 152, kWarps = kBlock / 32, kCtas = ctas(sizeof(T) * kV), kAtOnce = 4;
    const Units n(p.d, p.rot, kV);
    const int heads = p.H[0] + p.H[1];
    // A warp's lanes hold all of a token's heads, and there are tokens enough for every warp to have several: 32 x 1024
    // tokens of 2 heads of 128 bf16 took 31 us with one token at a time.
    const bool tokens = n.all <= 32 && heads <= n.side &&
                        p.tokens >= static_cast<int64_t>(kSms) * kWarps * (n.side / heads) * kAtOnce / 2;
    // few tokens: a token's heads over several warps, as long as there are SMs without one
    int64_t parts = static_cast<int64_t>(kSms) * kWarps / p.tokens, jobs;
    const int most = (heads + n.side - 1) / n.side;
    parts = parts < 1 ? 1 : parts > most ? most : parts;
    if (tokens) jobs = (p.tokens + n.side / heads * kAtOnce - 1) / (n.side / heads * kAtOnce);
    else jobs = p.tokens * parts;
    int64_t grid = (jobs + kWarps - 1) / kWarps;
    if (grid > kSms * kCtas) grid = kSms * kCtas;
    const size_t smem = p.rot / 2 * sizeof(unsigned long long);
    const unsigned g = static_cast<unsigned>(grid);
    if (tokens) rotary_kernel<T, kV, kHalf, true><<<g, kBlock, smem, s>>>(p, 1);
    else rotary_kernel<T, kV, kHalf, false><<<g, kBlock, smem, s>>>(p, static_cast<int>(parts));
    return cudaGetLastError();
}
template <typename T, int kV>
cudaError_t run(const RotaryArgs &p, bool half, cudaStream_t s) {
    return half ? run<T, kV, true>(p, s) : run<T, kV, false>(p, s);
}
// By the widest access that every head's start, and both parts of it, allow.
template <typename T>
cudaError_t run(const RotaryArgs &p, int B, bool half, cudaStream_t s) {
    constexpr int kFull = 16 / sizeof(T);
    auto starts = [&](int v) {
        const int size[2][3] = {{B, p.T, p.H[0]}, {B, p.T, p.H[1]}};
        for (int m = 0; m < 2; ++m) {
            if (!aligned(p.in[m], v * sizeof(T)) || !aligned(p.out[m], v * sizeof(T))) return false;
            for (int a = 0; a < 3; ++a)
                if (size[m][a] > 1 && (p.is[m][a] % v || p.os[m][a] % v)) return false;
        }
        return true;
    };
    auto fits = [&](int v) { return p.rot / 2 % v == 0 && (p.d - p.rot) % v == 0 && starts(v); };
    if (fits(kFull)) return run<T, kFull>(p, half, s);
    if (sizeof(T) == 2 && fits(4)) return run<T, sizeof(T) == 2 ? 4 : 1>(p, half, s);
    // through shared memory, but where accesses of 4 bytes fit heads of less than 48 bf16: 8 x 4096 x 32 heads took, by those
    // and through shared memory, 29 and 49 us of 16 values with 4 or 12 turned, 38 and 54 of 32, 54 and 60 of 40, 74 and 62
    // of 48 (12 or 44), 75 and 64 of 56, 75 and 66 of 64, 152 and 95 of 80 (pairs "interleaved": 2 to 6 us less, in the same
    // order); of single values 222 and 132 (126 of 128)
    if (p.rot > 0 && p.d % kFull == 0 && starts(kFull) && !(sizeof(T) == 2 && fits(2) && p.d < 48))
        return run_rows<T>(p, half, s);
    if (sizeof(T) == 2 && fits(2)) return run<T, sizeof(T) == 2 ? 2 : 1>(p, half, s);
    return run<T, 1>(p, half, s);
}

// Whether two tensors of equal strides share an element: whether `apart`, the distance of their starts in values, is a sum
// of strides times differences of indexes, which lie within lo and hi. Axes come in the order of their strides, so that
// those behind one reach a little further than its stride at most, and leave two or three differences to try.
struct Axis {
    int64_t stride, lo, hi;
};
bool meet(const Axis *axes, int n, int64_t apart) {
    int64_t least = 0, most = 0;
    for (int i = 0; i < n; ++i) {
        least += axes[i].stride * axes[i].lo;
        most += axes[i].stride * axes[i].hi;
    }
    if (apart < least || apart > most) return false;
    if (n == 0) return true;
    const Axis &a = axes[0];
    if (a.stride == 0) return meet(axes + 1, n - 1, apart);
    least -= a.stride * a.lo;
    most -= a.stride * a.hi;
    // stride * i within apart - most .. apart - least
    auto below = [&](int64_t v) { return v >= 0 ? v / a.stride : -((-v + a.stride - 1) / a.stride); };   // rounded down
    int64_t i = -below(most - apart), last = below(apart - least);
    if (i < a.lo) i = a.lo;
    if (last > a.hi) last = a.hi;
    if (last - i > 8) return true;   // strides that overlap among themselves
    for (; i <= last; ++i)
        if (meet(axes + 1, n - 1, apart - a.stride * i)) return true;
    return false;
}
// The same of an output and an input, or another output: slices of a packed projection reach over each other without
// sharing anything. Those have equal strides; of others it is not asked.
bool share(const void *q, const int64_t *qs, int Hq, const void *k, const int64_t *ks, int Hk, int B, int T, int d, int esz) {
    const int64_t bytes = static_cast<const char *>(k) - static_cast<const char *>(q);
    if (bytes % esz) return true;
    const int64_t size[2][4] = {{B, T, Hq, d}, {B, T, Hk, d}};
    Axis axes[4];
    for (int a = 0; a < 4; ++a) {   // k's index less q's, times the stride, is minus their distance
        const int64_t sq = a < 3 ? qs[a] : 1, sk = a < 3 ? ks[a] : 1;
        if (size[0][a] > 1 && size[1][a] > 1 && sq != sk) return true;
        axes[a] = {size[0][a] > 1 ? sq : sk, 1 - size[1][a], size[0][a] - 1};
    }
    for (int a = 0; a < 4; ++a)
        for (int b = a + 1; b < 4; ++b)
            if (axes[b].stride > axes[a].stride) {
                const Axis t = axes[a];
                axes[a] = axes[b];
                axes[b] = t;
            }
    return meet(axes, 4, bytes / esz);
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
    for (int m = 0; m < 2; ++m)
        if (overlaps(os[m], sf) || overlaps(os[m], sp)) return KLA_ERR_INVALID_ARG;
    auto apart = [&](const Span &a, const void *pa, const int64_t *sa, int ha, const Span &b, const void *pb,
                     const int64_t *sb, int hb) {
        return !overlaps(a, b) || !share(pa, sa, ha, pb, sb, hb, B, T, d, static_cast<int>(esz));
    };
    for (int m = 0; m < 2; ++m)
        for (int j = 0; j < 2; ++j)   // in place: its own input apart, and what the other reads later is not written over
            if (!(m == j && in_place[m]) && !apart(os[m], out[m], p.os[m], H[m], is[j], in[j], p.is[j], H[j]))
                return KLA_ERR_INVALID_ARG;
    if (!apart(os[0], out[0], p.os[0], H[0], os[1], out[1], p.os[1], H[1])) return KLA_ERR_INVALID_ARG;
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
    const cudaError_t e = dtype == KLA_DTYPE_BF16 ? run<__nv_bfloat16>(p, B, half, cs) : run<float>(p, B, half, cs);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}
