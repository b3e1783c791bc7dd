// kla_norm.cu -- layer norm over the last axis of [rows, groups, n], forward and gradients.
//
//   forward    y = xh w[g] + b[g],  xh = (x - mean) rstd
//   backward   dx = rstd (u - mean(u) - xh mean(u xh)),  u = dy w[g];  dw[g] = sum dy xh;  db[g] = sum dy
//
// Here rows of more than 512 values; shorter ones are in kla_norm_rows.cu. Every value is read once: a row
// belongs to a team of threads, each with values at fixed columns. Teams are persistent and keep to one
// group, so that weight and bias, and in the backward pass the sums of dw and db, stay in registers; the sums
// leave as one partial row per CTA and a second launch adds those in a fixed order.
// What bounds it is the memory, and to keep it busy ~70 KB have to be on the way to every SM. Rows of a
// CTA therefore come and go through shared memory by bulk copies, one to four rows ahead of every team (what
// shared memory holds: of 2048 values in the forward pass four in bf16, one in fp32), which cost no registers
// and take rows of any width and alignment: a copy takes the 16-byte granules that the row touches, and
// threads pick their columns from there. (Loads one row ahead into registers reached half of that.)
// Measured, 16397 x 2048 bf16: forward 27 us (5.0 TB/s, 74 % of a copy's rate), backward 40 us (5.0 TB/s) and 7 us
// for the sums of dw and db. What is left above the memory is latency: a row's chain of shared-memory accesses,
// shuffles and barriers, at 800 instructions a row in the forward pass and 1280 in the backward, of which 1.85 of 4
// are issued a cycle. The same rows in fp32, with twice the bytes to the same chain: 45 and 68 us (88 and 87 %), so
// one row ahead does; 16397 x 8192 fp32 167 and 249 us (95 and 96 %).
#include <atomic>
#include <climits>

#include "kla_norm.cuh"

namespace kla {
cudaError_t device_error_word(unsigned **out);   // kla_api.cu
namespace {

using namespace norm;

constexpr int kSms = 152;
constexpr int kRingMostN = 8192;       // longest row that goes through shared memory
constexpr int kRingMost = 4;           // rows on the way to a team, at most
// Values of one thread: the backward pass keeps five arrays of them, the forward pass three. The more, the
// less the sums and hand-overs of a row weigh.
constexpr int ring_values(bool bwd) { return bwd ? 16 : 32; }
// Threads of a CTA: the backward pass takes one CTA an SM, so that an SM leaves one partial row; the
// forward pass two.
constexpr int ring_block(bool bwd) { return bwd ? 512 : 256; }

// ---- rows of a CTA, through shared memory
// A row's buffer mirrors the memory around it: the 16-byte granules that the row touches, copied in one
// bulk copy. Granules that reach past the tensor's ends are left out; their few values are read directly.
template <typename T>
struct Row {
    const T *base;
    int shift;          // values from the buffer's start to the row's
    int skip, have;     // columns [skip, have) are in the buffer
    uint32_t lead, bytes;   // what the copy leaves out at the front, and brings
    __device__ __forceinline__ Row(const T *tensor, const T *end, const T *row, int n) : base(row) {
        constexpr int kSize = sizeof(T), kG = 16 / kSize;
        shift = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15) / kSize;
        int lo = 0, hi = (shift + n + kG - 1) / kG;   // granules
        if (row - tensor < shift) ++lo;
        if (end - row < hi * kG - shift) --hi;
        if (hi < lo) hi = lo;
        skip = lo * kG - shift;
        have = hi * kG - shift;
        lead = lo * 16;
        bytes = (hi - lo) * 16;
    }
};
// Whether the columns of a thread's k-th access exist for every lane: a row has more than half of the
// values that its team holds (the narrowest team: more than kRowsMost).
__device__ __forceinline__ constexpr bool always(int k, int width, int v, int e) {
    return (k + 1) * width * v <= kRowsMost || 2 * (k + 1) * v <= e;
}
// kN values, kV at a time, of a thread; zero from column n on. Accesses of 16 bytes: every row starts and
// ends on 16 bytes, and its buffer starts with it.
template <typename T, int kV>
constexpr bool whole_rows() { return sizeof(T) * kV == 16; }
template <typename T, int kV, int kWidth, int kN>
__device__ __forceinline__ void get_row(const T *tensor, const T *end, const T *row, const uint8_t *buf, int lane,
                                        int n, float2 (&x)[kN / 2]) {
    float *f = reinterpret_cast<float *>(x);
    if constexpr (whole_rows<T, kV>()) {
        const T *v = reinterpret_cast<const T *>(buf) + lane * kV;
#pragma unroll
        for (int k = 0; k < kN / kV; ++k) {
            alignas(16) T e[kV];
            if (always(k, kWidth, kV, kN) || (k * kWidth + lane) * kV < n) {
                load<T, kV>(v + k * kWidth * kV, e);
            } else {
#pragma unroll
                for (int i = 0; i < kV; ++i) e[i] = from_f32<T>(0.f);
            }
#pragma unroll
            for (int i = 0; i < kV; ++i) f[k * kV + i] = to_f32(e[i]);
        }
    } else {
        const Row<T> r(tensor, end, row, n);
        const T *v = reinterpret_cast<const T *>(buf) + r.shift + lane * kV;
#pragma unroll
        for (int k = 0; k < kN / kV; ++k) {
            T e[kV];
#pragma unroll
            for (int i = 0; i < kV; ++i) e[i] = from_f32<T>(0.f);
            if (always(k, kWidth, kV, kN) || (k * kWidth + lane) * kV < n) load<T, kV>(v + k * kWidth * kV, e);
#pragma unroll
            for (int i = 0; i < kV; ++i) f[k * kV + i] = to_f32(e[i]);
        }
        if (r.skip > 0 || r.have < n)   // the tensor's first or last row, off the 16-byte grid
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                const int c = (k / kV * kWidth + lane) * kV + k % kV;
                if (c < n && (c < r.skip || c >= r.have)) f[k] = to_f32(row[c]);
            }
    }
}

// A row on its way out: whole granules inside the row leave by one bulk store from a buffer that
// mirrors the memory, the few values at its ends directly.
template <typename T>
struct OutRow {
    T *row;
    int shift, lo, hi;   // columns [lo, hi) leave by the bulk store
    __device__ __forceinline__ OutRow(T *r, int n) : row(r) {
        constexpr int kSize = sizeof(T), kG = 16 / kSize;
        shift = static_cast<int>(reinterpret_cast<uintptr_t>(r) & 15) / kSize;
        lo = (kG - shift) % kG;
        hi = (shift + n) / kG * kG - shift;
        if (hi < lo) hi = lo;
    }
};

__device__ __forceinline__ void bulk_in(uint32_t to, const void *from, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
                 "l"(from), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void bulk_out(void *to, uint32_t from, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(from), "r"(bytes)
                 : "memory");
}

// kBwd: x and dy in, dx out, else x in, y out. A CTA holds one or more teams of `width` threads, each
// with buffers and a named barrier of its own. The barrier of a sum over the row also tells that the
// row's buffer is read and that the last row's output is written.
template <typename T, int kV, int kWidth, bool kBwd>
__global__ void __launch_bounds__(ring_block(kBwd), kBwd ? 1 : 2)
norm_ring_kernel(const T *x, const T *dy, const float *w, const float *b, T *out, float *mean, float *rstd,
                 float *part, int64_t rows, int groups, int n, float eps, int stages, int pitch, unsigned *err) {
    using namespace ptx;
    dependency_release();
    constexpr int kN = ring_values(kBwd), kK = kN / kV, kIns = kBwd ? 2 : 1;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ uint64_t full[ring_block(kBwd) / kWidth][kRingMost];
    __shared__ float2 sums[2][kMaxBlock / 32];
    __shared__ int lost[ring_block(kBwd) / kWidth][2];
    const Walk at(groups, kWidth);
    const int team = threadIdx.x / kWidth, lane = at.lane;
    const TeamLost gave_up{lost[team]};
    WarpsSum<kWidth / 32> sum{sums, team * (kWidth / 32), 1 + team, 0};
    const bool lead = lane == 0;
    uint8_t *ring = sm + team * (stages * kIns + 2) * pitch, *outs = ring + stages * kIns * pitch;
    const uint32_t s_ring = smem_u32(ring), s_outs = smem_u32(outs), bar0 = smem_u32(full[team]);
    const T *end_x = x + rows * groups * n, *end_d = kBwd ? dy + rows * groups * n : nullptr;
    const int turns = at.first < rows ? static_cast<int>((rows - at.first + at.step - 1) / at.step) : 0;
    const int64_t o0 = (at.first * groups + at.g) * n, hop = at.step * groups * n;   // values between rows
    // one thread of the team
    auto fetch = [&](int64_t o, int st) {
        const uint32_t bar = bar0 + 8 * st, buf = s_ring + st * kIns * pitch;
        if constexpr (whole_rows<T, kV>()) {
            const uint32_t bytes = n * static_cast<uint32_t>(sizeof(T));
            mbar_arrive_expect_tx(bar, kIns * bytes);
            bulk_in(buf, x + o, bytes, bar);
            if constexpr (kBwd) bulk_in(buf + pitch, dy + o, bytes, bar);
        } else {
            const Row<T> rx(x, end_x, x + o, n), rd(kBwd ? dy : x, kBwd ? end_d : end_x, (kBwd ? dy : x) + o, n);
            mbar_arrive_expect_tx(bar, rx.bytes + (kBwd ? rd.bytes : 0u));
            if (rx.bytes)
                bulk_in(buf + rx.lead, reinterpret_cast<const char *>(rx.base - rx.shift) + rx.lead, rx.bytes, bar);
            if (kBwd && rd.bytes)
                bulk_in(buf + pitch + rd.lead, reinterpret_cast<const char *>(rd.base - rd.shift) + rd.lead, rd.bytes,
                        bar);
        }
    };
    auto send = [&](T *to, uint32_t buf) {
        if constexpr (whole_rows<T, kV>()) {
            bulk_out(to, buf, n * static_cast<uint32_t>(sizeof(T)));
        } else {
            const OutRow<T> r(to, n);
            if (r.hi > r.lo)
                bulk_out(r.row + r.lo, buf + (r.shift + r.lo) * static_cast<uint32_t>(sizeof(T)),
                         (r.hi - r.lo) * static_cast<uint32_t>(sizeof(T)));
        }
        tma_store_commit();
    };
    if (lead) {
        gave_up.init();
        for (int i = 0; i < stages; ++i) mbar_init(bar0 + 8 * i, 1);
        fence_mbar_init();
        for (int i = 0; i < stages && i < turns; ++i) fetch(o0 + i * hop, i);
    }
    float2 wr[kN / 2], acc_w[kN / 2], acc_b[kN / 2];   // forward: acc_b is the bias
#pragma unroll
    for (int k = 0; k < kK; ++k)
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int c = (k * kWidth + lane) * kV + i, u = k * kV + i;
            reinterpret_cast<float *>(wr)[u] = w && c < n ? w[static_cast<int64_t>(at.g) * n + c] : 1.f;
            reinterpret_cast<float *>(acc_w)[u] = 0.f;
            reinterpret_cast<float *>(acc_b)[u] =
                !kBwd && b && c < n ? b[static_cast<int64_t>(at.g) * n + c] : 0.f;
        }
    __syncthreads();
    const float inv = 1.f / n;
    int64_t row = at.first * groups + at.g, o = o0;
    float nmu = 0.f, nrs = 0.f;   // backward: the next row's mean and rstd
    if (kBwd && turns > 0) {
        nmu = mean[row];
        nrs = rstd[row];
    }
    int t = 0, st = 0;
    uint32_t phase = 0;
    for (; t < turns; ++t, row += at.step * groups, o += hop) {
        float mu = nmu, rs = nrs;
        if (kBwd && t + 1 < turns) {
            nmu = mean[row + at.step * groups];
            nrs = rstd[row + at.step * groups];
        }
        if (!mbar_wait_bounded(bar0 + 8 * st, phase, 100000u)) gave_up.note(t);
        const uint8_t *buf = ring + st * kIns * pitch;
        float2 v[kN / 2], d[kN / 2];
        get_row<T, kV, kWidth, kN>(x, end_x, x + o, buf, lane, n, v);
        if constexpr (kBwd) get_row<T, kV, kWidth, kN>(dy, end_d, dy + o, buf + pitch, lane, n, d);
        float2 s = make_float2(0.f, 0.f);
        if constexpr (kBwd) {
            float2 s0 = s, s1 = s;
#pragma unroll
            for (int i = 0; i < kN / 2; ++i) {   // columns past n have d = 0 and add nothing
                v[i] = mul2(add2(v[i], both(-mu)), both(rs));
                acc_w[i] = fma2(d[i], v[i], acc_w[i]);
                acc_b[i] = add2(acc_b[i], d[i]);
                d[i] = mul2(d[i], wr[i]);
                s0 = add2(s0, d[i]);
                s1 = fma2(d[i], v[i], s1);
            }
            s = make_float2(s0.x + s0.y, s1.x + s1.y);
        } else {
#pragma unroll
            for (int i = 0; i < kN / 2; ++i) s = add2(s, v[i]);
            s.x += s.y;
        }
        fence_proxy_async_smem();   // this thread's part of the last output row, before the barrier
        if (lead)                   // the output buffer of two rows ago is read
            tma_store_wait_read_all();
        if constexpr (kBwd) s = sum(s);
        else s.x = sum(s.x);
        if (gave_up.read(t)) break;
        if (lead) {
            if (t > 0) send(out + o - hop, s_outs + ((t - 1) & 1) * pitch);
            if (t + stages < turns) fetch(o + stages * hop, st);
        }
        if (++st == stages) {
            st = 0;
            phase ^= 1;
        }
        if constexpr (kBwd) {
            s.x *= inv;
            s.y *= inv;
        } else {
            mu = s.x * inv;
            float2 q = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kN / 2; ++i) {
                v[i] = add2(v[i], both(-mu));
                float2 e = v[i];   // columns past n are no part of the sum
                const int c0 = ((2 * i) / kV * kWidth + lane) * kV, c1 = ((2 * i + 1) / kV * kWidth + lane) * kV;
                if (!always((2 * i) / kV, kWidth, kV, kN) && c0 >= n) e.x = 0.f;
                if (!always((2 * i + 1) / kV, kWidth, kV, kN) && c1 >= n) e.y = 0.f;
                q = fma2(e, e, q);
            }
            rs = 1.f / sqrtf(sum(q.x + q.y) * inv + eps);
            if (lead) {
                if (mean) mean[row] = mu;
                if (rstd) rstd[row] = rs;
            }
        }
        uint8_t *to = outs + (t & 1) * pitch;
        const OutRow<T> ro(out + o, n);   // of whole rows not used
        T *line = reinterpret_cast<T *>(to) + (whole_rows<T, kV>() ? 0 : ro.shift) + lane * kV;
        const float2 p0 = both(rs), p1 = both(-rs * s.x), p2 = both(-rs * s.y);
#pragma unroll
        for (int i = 0; i < kN / 2; ++i)
            v[i] = kBwd ? fma2(p0, d[i], fma2(p2, v[i], p1)) : fma2(mul2(v[i], p0), wr[i], acc_b[i]);
        const float *f = reinterpret_cast<const float *>(v);
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const int c = (k * kWidth + lane) * kV;
            if (always(k, kWidth, kV, kN) || c < n) {
                if (whole_rows<T, kV>() || (c >= ro.lo && c < ro.hi)) {
                    store<T, kV>(line + k * kWidth * kV, f + k * kV);
                } else {
#pragma unroll
                    for (int i = 0; i < kV; ++i) ro.row[c + i] = from_f32<T>(f[k * kV + i]);
                }
            }
        }
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (lead) {
        if (turns > 0 && t == turns) send(out + o - hop, s_outs + ((turns - 1) & 1) * pitch);
        if (t < turns) {   // a wait gave up in turn t
            atomicOr(err, kErrTimeout);
            for (int u = t; u < turns && u < t + stages; ++u) {   // nothing may land after the CTA has ended
                mbar_wait_bounded(bar0 + 8 * st, phase, 100000u);
                if (++st == stages) {
                    st = 0;
                    phase ^= 1;
                }
            }
        }
        tma_store_wait_all();
    }
    if (kBwd && part) {   // one partial row of dw and of db per CTA: the teams add up one after the other
        float *fw = reinterpret_cast<float *>(sm), *fb = fw + n;
        for (int q = 0; q < static_cast<int>(blockDim.x) / kWidth; ++q) {
            __syncthreads();
            if (team == q)
#pragma unroll
                for (int k = 0; k < kK; ++k)
#pragma unroll
                    for (int i = 0; i < kV; ++i) {
                        const int c = (k * kWidth + lane) * kV + i, u = k * kV + i;
                        const float aw = reinterpret_cast<const float *>(acc_w)[u];
                        const float ab = reinterpret_cast<const float *>(acc_b)[u];
                        if (c < n) {
                            fw[c] = q ? fw[c] + aw : aw;
                            fb[c] = q ? fb[c] + ab : ab;
                        }
                    }
        }
        __syncthreads();
        float *p = part + static_cast<int64_t>(blockIdx.x) * 2 * n;
        for (int c = threadIdx.x; c < 2 * n; c += blockDim.x) p[c] = fw[c];
    }
}

// dweight and dbias of group blockIdx.y, 32 columns a CTA: 32 rows of threads walk the partial rows, eight
// loads in flight each (one at a time took 43 us for 1216 partial rows of 2048 columns), in a fixed order.
__global__ void __launch_bounds__(1024) norm_sum_kernel(const float *part, float *dw, float *db, int parts, int groups,
                                                        int n) {
    __shared__ float sw[32][33], sb[32][33];
    dependency_wait();
    const int x = threadIdx.x & 31, c = blockIdx.x * 32 + x, r = threadIdx.x / 32, g = blockIdx.y;
    float a = 0.f, b = 0.f;
    if (c < n) {
        const float *row = part + (static_cast<int64_t>(r) * groups + g) * 2 * n + c;
        const int64_t step = static_cast<int64_t>(32) * groups * 2 * n;
#pragma unroll 8
        for (int p = r; p < parts; p += 32, row += step) {
            a += row[0];
            b += row[n];
        }
    }
    sw[r][x] = a;
    sb[r][x] = b;
    __syncthreads();
    // warp r takes column r: lane x holds the sum of its row of threads
    a = sw[x][r];
    b = sb[x][r];
#pragma unroll
    for (int off = 16; off; off >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, off);
        b += __shfl_xor_sync(0xffffffffu, b, off);
    }
    const int col = blockIdx.x * 32 + r;
    if (x == 0 && col < n) {
        if (dw) dw[static_cast<int64_t>(g) * n + col] = a;
        if (db) db[static_cast<int64_t>(g) * n + col] = b;
    }
}

// ---- rows longer than kRingMostN: more than a CTA holds
// The forward pass reads a row once for its statistics and again, from L1 or L2, for its output. A thread
// takes pieces of kP accesses whose loads are on their way together; a piece's mean and squared deviations
// join the thread's by the pairwise update of Chan, Golub and LeVeque, (N, M, Q) + (c, m, q) = (N + c,
// M + d c / (N + c), Q + q + d^2 N c / (N + c)), d = m - M, which subtracts the mean before it squares as two
// passes would. The backward pass cannot keep a row's columns
// and their sums in one CTA's registers either: it reads x and dy twice, by rows and then by columns.
// Measured, 8000 x 12288 bf16: forward 111 us (3.5 TB/s), backward 162 us (3.7 TB/s of one read, 6.1 of the two);
// walking the row value by value, with sums of dw and db in memory, took 172 and 565.
constexpr int kLongBlock = 512, kLongTile = 2048, kLongRows = 4;
// Weights and biases of a piece come in 16-byte accesses too: one value at a time, 32 bytes from lane to lane, took
// 237 us for 8000 x 12288 bf16.
template <int kV>
constexpr int kLongPiece = kV >= 4 ? 4 : 8;   // accesses of a piece

// kV floats, all `otherwise` without a pointer.
template <int kV>
__device__ __forceinline__ void load_floats(const float *p, int64_t at, float otherwise, float (&v)[kV]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = otherwise;
    } else if constexpr (kV % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kV; i += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(p + at + i);
            v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i) v[i] = p[at + i];
    }
}

template <typename T, int kV>
__global__ void __launch_bounds__(kLongBlock, 2)
norm_fwd_long_kernel(const T *x, const float *w, const float *b, T *y, float *mean, float *rstd, int groups, int n,
                     float eps) {
    __shared__ float2 sums[2][kMaxBlock / 32];
    WarpsSum<kLongBlock / 32> sum{sums, 0, 1, 0};
    constexpr int kP = kLongPiece<kV>, kStep = kLongBlock * kV;
    const int64_t row = blockIdx.x;
    const T *xr = x + row * n;
    float N = 0.f, M = 0.f, Q = 0.f;
    for (int c0 = threadIdx.x * kV; c0 < n; c0 += kP * kStep) {
        alignas(16) T v[kP * kV];
#pragma unroll
        for (int k = 0; k < kP; ++k) load<T, kV>(xr + min(c0 + k * kStep, n - kV), v + k * kV);
        float s = 0.f, q = 0.f, count = 0.f;
#pragma unroll
        for (int k = 0; k < kP; ++k)
            if (c0 + k * kStep < n) {
                count += kV;
#pragma unroll
                for (int i = 0; i < kV; ++i) s += to_f32(v[k * kV + i]);
            }
        const float m = s / count;
#pragma unroll
        for (int k = 0; k < kP; ++k)
            if (c0 + k * kStep < n)
#pragma unroll
                for (int i = 0; i < kV; ++i) {
                    const float d = to_f32(v[k * kV + i]) - m;
                    q = fmaf(d, d, q);
                }
        const float d = m - M, part = count / (N + count);
        M = fmaf(d, part, M);
        Q += fmaf(d * d, N * part, q);
        N += count;
    }
    const float mu = sum(N * M) / n;
    const float rs = 1.f / sqrtf(sum(fmaf(N * (M - mu), M - mu, Q)) / n + eps);
    if (threadIdx.x == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
    }
    const int64_t at = row % groups * n;
    for (int c0 = threadIdx.x * kV; c0 < n; c0 += kP * kStep) {
        alignas(16) T v[kP * kV];
#pragma unroll
        for (int k = 0; k < kP; ++k) load<T, kV>(xr + min(c0 + k * kStep, n - kV), v + k * kV);
#pragma unroll
        for (int k = 0; k < kP; ++k) {
            const int c = c0 + k * kStep;
            if (c >= n) break;
            float o[kV], wv[kV], bv[kV];
            load_floats<kV>(w, at + c, 1.f, wv);
            load_floats<kV>(b, at + c, 0.f, bv);
#pragma unroll
            for (int i = 0; i < kV; ++i) o[i] = fmaf((to_f32(v[k * kV + i]) - mu) * rs, wv[i], bv[i]);
            store<T, kV>(y + row * n + c, o);
        }
    }
}

// Backward pass, first launch: mean(u) and mean(u xh) of every row.
template <typename T, int kV>
__global__ void __launch_bounds__(kLongBlock, 2)
norm_bwd_long_sums_kernel(const T *dy, const T *x, const float *w, const float *mean, const float *rstd,
                          float2 *row_sums, int groups, int n) {
    dependency_release();
    __shared__ float2 sums[2][kMaxBlock / 32];
    WarpsSum<kLongBlock / 32> sum{sums, 0, 1, 0};
    constexpr int kP = kLongPiece<kV> / 2, kStep = kLongBlock * kV;
    const int64_t row = blockIdx.x, at = row % groups * n;
    const float mu = mean[row], rs = rstd[row];
    float2 s = make_float2(0.f, 0.f);
    for (int c0 = threadIdx.x * kV; c0 < n; c0 += kP * kStep) {
        alignas(16) T xv[kP * kV];
        alignas(16) T dv[kP * kV];
#pragma unroll
        for (int k = 0; k < kP; ++k) {
            const int c = min(c0 + k * kStep, n - kV);
            load<T, kV>(x + row * n + c, xv + k * kV);
            load<T, kV>(dy + row * n + c, dv + k * kV);
        }
#pragma unroll
        for (int k = 0; k < kP; ++k) {
            const int c = c0 + k * kStep;
            if (c >= n) break;
            float wv[kV];
            load_floats<kV>(w, at + c, 1.f, wv);
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const float u = to_f32(dv[k * kV + i]) * wv[i];
                s.x += u;
                s.y = fmaf(u, (to_f32(xv[k * kV + i]) - mu) * rs, s.y);
            }
        }
    }
    s = sum(s);
    if (threadIdx.x == 0) row_sums[row] = make_float2(s.x / n, s.y / n);
}

// Second launch: a CTA keeps to kLongTile columns of a group, whose weights and sums of dw and db stay in
// registers, and walks rows from the last, which L2 still holds, kLongRows at a time.
template <typename T, int kV>
__global__ void __launch_bounds__(256, 2)
norm_bwd_long_kernel(const T *dy, const T *x, const float *w, const float *mean, const float *rstd,
                     const float2 *row_sums, T *dx, float *part, int64_t rows, int groups, int n) {
    dependency_release();
    constexpr int kNV = kLongTile / 256 / kV, kE = kNV * kV, kR = kLongRows;
    const int g = blockIdx.y % groups, split = blockIdx.y / groups, splits = gridDim.y / groups;
    int col[kNV];
    float wv[kE], aw[kE], ab[kE];
#pragma unroll
    for (int k = 0; k < kNV; ++k) {
        col[k] = blockIdx.x * kLongTile + (k * 256 + threadIdx.x) * kV;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            wv[k * kV + i] = w && col[k] < n ? w[static_cast<int64_t>(g) * n + col[k] + i] : 1.f;
            aw[k * kV + i] = ab[k * kV + i] = 0.f;
        }
    }
    dependency_wait();
    for (int64_t r = rows - 1 - split; r >= 0; r -= static_cast<int64_t>(splits) * kR) {
        alignas(16) T xv[kR][kE];
        alignas(16) T dv[kR][kE];
        float mu[kR], rs[kR];
        float2 s[kR];
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            const int64_t mine = r - static_cast<int64_t>(j) * splits, row = (mine < 0 ? 0 : mine) * groups + g;
#pragma unroll
            for (int k = 0; k < kNV; ++k) {
                const int c = min(col[k], n - kV);
                load<T, kV>(x + row * n + c, xv[j] + k * kV);
                load<T, kV>(dy + row * n + c, dv[j] + k * kV);
            }
            mu[j] = mean[row], rs[j] = rstd[row], s[j] = row_sums[row];
        }
#pragma unroll
        for (int j = 0; j < kR; ++j) {
            const int64_t mine = r - static_cast<int64_t>(j) * splits;
            if (mine < 0) break;
            float o[kE];
#pragma unroll
            for (int i = 0; i < kE; ++i) {
                const float d = to_f32(dv[j][i]), xh = (to_f32(xv[j][i]) - mu[j]) * rs[j];
                o[i] = rs[j] * (fmaf(d, wv[i], -s[j].x) - xh * s[j].y);
                aw[i] = fmaf(d, xh, aw[i]);
                ab[i] += d;
            }
#pragma unroll
            for (int k = 0; k < kNV; ++k)
                if (col[k] < n) store<T, kV>(dx + (mine * groups + g) * n + col[k], o + k * kV);
        }
    }
    if (!part) return;
    float *p = part + static_cast<int64_t>(blockIdx.y) * 2 * n;
#pragma unroll
    for (int k = 0; k < kNV; ++k)
        if (col[k] < n)
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                p[col[k] + i] = aw[k * kV + i];
                p[n + col[k] + i] = ab[k * kV + i];
            }
}

// ------------------------------------------------------------------------------------ host side
enum Form { kRows, kRing, kLong };
struct Plan {
    Form form;
    int width;           // kRing: threads of a row's team
    int block, grid;     // grid: also the partial rows of dw and db
    int stages, pitch, smem;   // kRing: rows on the way to a team, bytes of a row's buffer, bytes of a CTA
};

// kRing: the smallest team that holds the row; persistent CTAs as many as the SMs hold at once, a multiple of
// the groups, none without a row.
Plan plan(int64_t rows, int groups, int n, kla_dtype dtype, bool bwd) {
    Plan p{};
    p.form = n <= kRowsMost ? kRows : n <= kRingMostN ? kRing : kLong;
    if (p.form == kRows) {
        if (bwd) p.grid = norm_rows_bwd_grid(rows, groups);   // the forward pass launches by itself
        return p;
    }
    if (p.form == kLong) {   // only the backward pass asks: CTAs along the rows
        const int64_t tiles = (n + kLongTile - 1) / kLongTile;
        int64_t splits = 2 * kSms / (tiles * groups);
        const int64_t most = (rows + kLongRows - 1) / kLongRows;
        splits = splits > most ? most : splits;
        p.grid = static_cast<int>(splits < 1 ? 1 : splits) * groups;
        return p;
    }
    int per_sm = 1;
    {
        const int least = 32 * ring_values(bwd);   // what a warp holds
        p.width = n <= 2 * least ? (n <= least ? 32 : 64) : n <= 4 * least ? 128 : n <= 8 * least ? 256 : 512;
        const int most = ring_block(bwd);
        int teams = most / p.width;
        // teams that would have no row only cost shared memory
        if (teams > rows) teams = static_cast<int>(rows);
        p.block = teams * p.width;
        per_sm = bwd ? 1 : 2;
        p.pitch = (n * (dtype == KLA_DTYPE_BF16 ? 2 : 4) + 31) / 16 * 16;
        const int bytes = 216 * 1024 / per_sm - 4096;
        p.stages = (bytes / teams / p.pitch - 2) / (bwd ? 2 : 1);
        p.stages = p.stages > kRingMost ? kRingMost : p.stages < 1 ? 1 : p.stages;
        p.smem = teams * (p.stages * (bwd ? 2 : 1) + 2) * p.pitch;
        if (bwd && p.smem < 8 * n) p.smem = 8 * n;   // the sums of dw and db at the end
    }
    const int64_t per_cta = p.block / p.width;
    const int64_t most = (rows + per_cta - 1) / per_cta;   // CTAs of one group
    int64_t want = (static_cast<int64_t>(kSms) * per_sm + groups - 1) / groups;
    if (want > most) want = most;
    if (want < 1) want = 1;
    p.grid = static_cast<int>(want * groups);
    return p;
}

kla_status check(int64_t rows, int groups, int n, kla_dtype dtype) {
    if (rows < 0 || groups < 1 || n < 1) return KLA_ERR_INVALID_ARG;
    if (dtype != KLA_DTYPE_F32 && dtype != KLA_DTYPE_BF16) return KLA_ERR_INVALID_ARG;
    // rows of one or two values: dx is eps alone, left over from terms that cancel in fp32
    if (n < 3 || n > 65536 || groups > 65535 || rows * groups > INT_MAX) return KLA_ERR_UNSUPPORTED;
    return KLA_OK;
}

// Scratch of the backward pass over long rows, in front of the partial sums.
size_t row_sums_bytes(int64_t rows, int groups, int n) {
    return n > kRingMostN ? (static_cast<size_t>(rows) * groups * sizeof(float2) + 15) / 16 * 16 : 0;
}

// The widest access that every row start allows: 16 bytes, a bf16 pair, or one value. The kernels of long rows take
// weights w1 and w2 at that width too.
template <typename T>
int width(int n, const void *a, const void *b, const void *c, const float *w1, const float *w2) {
    constexpr int kFull = 16 / sizeof(T);
    auto fits = [&](int v) {
        const uintptr_t bytes = v * sizeof(T);
        return n % v == 0 && aligned(a, bytes) && aligned(b, bytes) && aligned(c, bytes);
    };
    const bool weights = n <= kRingMostN || (aligned(w1, 16) && aligned(w2, 16));
    return fits(kFull) && weights ? kFull : sizeof(T) == 2 && fits(2) ? 2 : 1;
}

template <typename T, int kV, int kWidth, bool kBwd>
cudaError_t run_ring_as(const Plan &p, const T *x, const T *dy, const float *w, const float *b, T *out, float *mean,
                        float *rstd, float *part, int64_t rows, int groups, int n, float eps, cudaStream_t s) {
    unsigned *err = nullptr;
    cudaError_t e = device_error_word(&err);
    if (e != cudaSuccess) return e;
    auto kern = norm_ring_kernel<T, kV, kWidth, kBwd>;
    if (p.smem > 48 * 1024) {   // asked for once per device and kernel: the attribute outlasts the call
        constexpr int kMaxDevices = 64;
        static std::atomic<bool> done[kMaxDevices];
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
        if (!done[dev].load(std::memory_order_acquire)) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 222 * 1024);
            if (e != cudaSuccess) return e;
            done[dev].store(true, std::memory_order_release);
        }
    }
    kern<<<p.grid, p.block, p.smem, s>>>(x, dy, w, b, out, mean, rstd, part, rows, groups, n, eps, p.stages, p.pitch,
                                         err);
    return cudaGetLastError();
}
template <typename T, int kV, bool kBwd, typename... A>
cudaError_t run_ring(const Plan &p, A... a) {
    constexpr int kLeast = kBwd ? 64 : 32;   // 16 or 32 values a thread, rows from 513 values
    if (p.width == kLeast) return run_ring_as<T, kV, kLeast, kBwd>(p, a...);
    if (p.width == 2 * kLeast) return run_ring_as<T, kV, 2 * kLeast, kBwd>(p, a...);
    if (p.width == 4 * kLeast) return run_ring_as<T, kV, 4 * kLeast, kBwd>(p, a...);
    return run_ring_as<T, kV, 8 * kLeast, kBwd>(p, a...);
}

template <typename T, int kV>
cudaError_t fwd_as(const Plan &p, const T *x, const float *w, const float *b, T *y, float *mean, float *rstd,
                   int64_t rows, int groups, int n, float eps, cudaStream_t s) {
    if (p.form == kRing)
        return run_ring<T, kV, false>(p, x, static_cast<const T *>(nullptr), w, b, y, mean,
                                                                  rstd, static_cast<float *>(nullptr), rows, groups,
                                                                  n, eps, s);
    norm_fwd_long_kernel<T, kV><<<static_cast<int>(rows * groups), kLongBlock, 0, s>>>(x, w, b, y, mean, rstd, groups,
                                                                                      n, eps);
    return cudaGetLastError();
}
template <typename T, int kV>
cudaError_t bwd_as(const Plan &p, const T *dy, const T *x, const float *w, const float *mean, const float *rstd,
                   T *dx, float *part, float2 *row_sums, int64_t rows, int groups, int n, cudaStream_t s) {
    if (p.form == kRing)
        return run_ring<T, kV, true>(p, x, dy, w, static_cast<const float *>(nullptr), dx,
                                                                 const_cast<float *>(mean),
                                                                 const_cast<float *>(rstd), part, rows, groups, n,
                                                                 0.f, s);
    norm_bwd_long_sums_kernel<T, kV><<<static_cast<int>(rows * groups), kLongBlock, 0, s>>>(dy, x, w, mean, rstd,
                                                                                           row_sums, groups, n);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_dependent(norm_bwd_long_kernel<T, kV>, dim3((n + kLongTile - 1) / kLongTile, p.grid), 256, 0, s, dy,
                            x, w, mean, rstd, static_cast<const float2 *>(row_sums), dx, part, rows, groups, n);
}

// By type and width of access.
template <typename T>
cudaError_t fwd_typed(const void *xv, const float *w, const float *b, void *yv, float *mean, float *rstd,
                      int64_t rows, int groups, int n, float eps, kla_dtype dtype, cudaStream_t s) {
    const T *x = static_cast<const T *>(xv);
    T *y = static_cast<T *>(yv);
    const Plan p = plan(rows, groups, n, dtype, false);
    const int v = width<T>(n, x, y, y, w, b);
    if (p.form == kRows) return norm_rows_fwd(x, w, b, y, mean, rstd, rows, groups, n, dtype, v, eps, s);
    if (v == 16 / sizeof(T)) return fwd_as<T, 16 / sizeof(T)>(p, x, w, b, y, mean, rstd, rows, groups, n, eps, s);
    if (sizeof(T) == 2 && v == 2)
        return fwd_as<T, sizeof(T) == 2 ? 2 : 1>(p, x, w, b, y, mean, rstd, rows, groups, n, eps, s);
    return fwd_as<T, 1>(p, x, w, b, y, mean, rstd, rows, groups, n, eps, s);
}
template <typename T>
cudaError_t bwd_typed(const void *dyv, const void *xv, const float *w, const float *mean, const float *rstd,
                      void *dxv, float *part, float2 *row_sums, int64_t rows, int groups, int n, kla_dtype dtype,
                      cudaStream_t s) {
    const T *dy = static_cast<const T *>(dyv), *x = static_cast<const T *>(xv);
    T *dx = static_cast<T *>(dxv);
    const Plan p = plan(rows, groups, n, dtype, true);
    const int v = width<T>(n, x, dy, dx, w, w);
    if (p.form == kRows) return norm_rows_bwd(dy, x, w, mean, rstd, dx, part, rows, groups, n, dtype, v, s);
    if (v == 16 / sizeof(T))
        return bwd_as<T, 16 / sizeof(T)>(p, dy, x, w, mean, rstd, dx, part, row_sums, rows, groups, n, s);
    if (sizeof(T) == 2 && v == 2)
        return bwd_as<T, sizeof(T) == 2 ? 2 : 1>(p, dy, x, w, mean, rstd, dx, part, row_sums, rows, groups, n, s);
    return bwd_as<T, 1>(p, dy, x, w, mean, rstd, dx, part, row_sums, rows, groups, n, s);
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
    const cudaError_t e =
        dtype == KLA_DTYPE_BF16
            ? fwd_typed<__nv_bfloat16>(x, weight, bias, y, mean, rstd, rows, groups, n, eps, dtype, cs)
            : fwd_typed<float>(x, weight, bias, y, mean, rstd, rows, groups, n, eps, dtype, cs);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

size_t kla_layer_norm_bwd_workspace_size(int64_t rows, int groups, int n, kla_dtype dtype) {
    if (kla::check(rows, groups, n, dtype) != KLA_OK || rows == 0) return 0;
    return kla::row_sums_bytes(rows, groups, n) +
           static_cast<size_t>(kla::plan(rows, groups, n, dtype, true).grid) * 2 * n * sizeof(float);
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
    const size_t lead = row_sums_bytes(rows, groups, n);
    const size_t need = sums ? kla_layer_norm_bwd_workspace_size(rows, groups, n, dtype) : lead;
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
    float *part = sums ? reinterpret_cast<float *>(static_cast<char *>(workspace) + lead) : nullptr;
    float2 *row_sums = static_cast<float2 *>(workspace);
    const cudaError_t e =
        dtype == KLA_DTYPE_BF16
            ? bwd_typed<__nv_bfloat16>(dy, x, weight, mean, rstd, dx, part, row_sums, rows, groups, n, dtype, cs)
            : bwd_typed<float>(dy, x, weight, mean, rstd, dx, part, row_sums, rows, groups, n, dtype, cs);
    if (e != cudaSuccess) return KLA_ERR_CUDA;
    if (!sums) return KLA_OK;
    return launch_dependent(norm_sum_kernel, dim3((n + 31) / 32, groups), 1024, 0, cs, part, dweight, dbias,
                            plan(rows, groups, n, dtype, true).grid / groups, groups, n) == cudaSuccess
               ? KLA_OK
               : KLA_ERR_CUDA;
}

}  // extern "C"
