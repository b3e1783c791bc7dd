// kla_scan.cu -- the gated scan: h_t = a_t h_{t-1} + w_t x_t for every channel, forward, gradients and single tokens.
//
//   KLA_SCAN_SIGMOID   w = 1 / (1 + exp(gate)),  h = a h + w x,  dgate = a w (h_{t-1} - x) dh   with a = 1 - w
//   KLA_SCAN_LOG       a = exp(gate),            h = a h + x,    dgate = a h_{t-1} dh
//   both               dh_t = dy_t + a_{t+1} dh_{t+1},  dx = w dh
//
// In fp32 the sigmoid's recurrence is taken as h + w (x - h) where w is the smaller of the two factors, as x + a (h - x)
// where a is: where a gate keeps its state for thousands of tokens a is within 2^-11 of 1 and its rounding to 24 bits
// would leave 12 of w, and where one drops a large state nothing of it may stay behind as a difference of roundings.
// In bf16 as a h + w x with a = 1 - w in paired arithmetic, whose rounding of 2^-23 is far below the values' own 2^-8 as
// long as a is not small; a warp with gates below -6 takes its tokens as in fp32 (`Exact`), as a gate that forgets leaves
// nothing but a of the state, and of the gradient.
//
// Every value is read once: 6 bytes a value forward and 10 backward in bf16, which at a copy's rate is 237 us for a
// prompt of 131072 x 2048. Time is therefore cut into tiles that are worked on side by side and joined by what they
// tell each other through the workspace, in one pass; a pass for the tiles' maps and one for the outputs would move 10
// bytes forward. Backward, the states are walked again from one kept every 128 tokens (0.03 bytes a value), which is
// exact and cheaper than reading the outputs back.
// Measured, calls in a row: 131072 x 2048 forward 277 us (5.8 TB/s, 86 % of a copy's rate), backward 513 us (5.2 TB/s); 8 x
// 4096 x 2048 forward 67 us (6.0 TB/s), backward 110 us (6.1 TB/s); in fp32 8 x 2048 x 2048 81 us (5.0 TB/s) and 129 us
// (5.2 TB/s), log gates 65 and 104. Where channels are few the chain of tiles is what is waited for, four or eight of them a
// trip to L2, 0.7 us: 131072 x 512 111 and 234 us, 131072 x 64 67 and 149. A thread per channel that walks all tokens took
// 120 ms for the first. By the counters (8 x 2048 x 2048 bf16) 19 instructions a value forward and 31 backward, both at 2.0
// of 4 a cycle; warps wait for the chain (forward) and for tiles on their way: registers hold 16 warps an SM, whose tiles
// and those that follow are what is under way at once. In fp32, with its own exponential and reciprocal and a channel a
// lane, they are 56 and 90 a value, at 2.5 and 2.4 a cycle: these bound it, at 73 and 77 % of the memory's time.
#include <cuda.h>

#include <atomic>
#include <cfloat>
#include <climits>

#include "layer_dev.cuh"
#include "../../include/kla_block.h"

namespace kla {
cudaError_t device_error_word(unsigned **out);   // kla_api.cu
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
    int blocks, tiles;                // channel blocks of a sequence, tiles along its tokens
    struct Head *head;                // of the workspace; NULL with one tile along the tokens
    uint2 *carry;                     // [B][tiles][C]
    unsigned *err;
    unsigned first, polls;            // the first ticket given out, and how often a tile asks for the state that enters it
};
// The workspace: this, then what tiles tell each other. All bits set before the kernel starts.
struct Head {
    unsigned ticket, abort;
    unsigned pad[2];
};

__device__ __forceinline__ int valid_tokens(const ScanArgs &p, int b) {
    return p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
}

// exp(gate), for the sigmoid held below 2^100: w stays a normal number then, and a is 1. bf16 gates take the
// hardware's exponential and reciprocal, off by 2^-21 at gates of 10, far below the gate's own 2^-9.
template <typename T, bool kLog>
__device__ __forceinline__ float gate_exp(float gate) {
    float e;
    if (sizeof(T) == 2) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(gate * 1.4426950408889634f));
    else e = expf(gate);
    return !kLog && e > 0x1p100f ? 0x1p100f : e;
}
// The state's factor a and the input's w.
template <typename T, bool kLog>
__device__ __forceinline__ void factors(float e, float &a, float &w) {
    if (kLog) {
        a = e;
        w = 1.f;
    } else {
        if (sizeof(T) == 2) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(1.f + e));
        else w = __frcp_rn(1.f + e);
        a = e * w;
    }
}
// 1 - a to its own last bits. The logarithm's near 0 by the exponential's series, whose next term is 2^-29 of it.
template <typename T, bool kLog>
__device__ __forceinline__ float loss(float gate) {
    float a, w;
    factors<T, kLog>(gate_exp<T, kLog>(gate), a, w);
    if (!kLog) return w;
    float s = fmaf(gate, 0.2f, 1.f);
    s = fmaf(gate * 0.25f, s, 1.f);
    s = fmaf(gate * 0.33333334f, s, 1.f);
    s = fmaf(gate * 0.5f, s, 1.f);
    return fabsf(gate) < 0.0625f ? -gate * s : 1.f - a;
}
// The product A of a channel's m factors, where that is close to 1. Every factor is off by up to 2^-22 (the hardware's
// exponential) or 2^-24 (a = 1 - w and the product's rounding), and with gates that are alike always to the same side: the
// state after 100000 tokens of constant gates of -1e-5 was 2.6e-3 off in bf16 and 1.9e-3 in fp32. There 1 - A is added up
// from the losses (9e-6 and 2.3e-5 off), up to mean losses of 2^-9, from which on the factors' errors are 2^-15 (bf16's
// exponential: 2^-13) of theirs. States do not drift within a stretch, as its tokens are few; what is told of it is what
// adds up.
__device__ __forceinline__ bool keeps(float A, int m) { return fabsf(1.f - A) < m * 0x1p-9f; }
template <typename T, bool kLog>
__device__ __forceinline__ float lose(float lost, float gate) { return fmaf(loss<T, kLog>(gate), 1.f - lost, lost); }
// One number that says both: a where KLA_SCAN_LOG; else the smaller of w and a, the latter with its sign set.
template <bool kLog>
__device__ __forceinline__ float coefficient(float a, float w) {
    return kLog ? a : w < 0.5f ? w : -a;
}
template <bool kLog>
__device__ __forceinline__ float advance(float h, float x, float c) {
    return kLog ? fmaf(c, h, x) : fmaf(c, x - h, c > 0.f ? h : x);
}
// prod a, one factor on
template <bool kLog>
__device__ __forceinline__ float shrink(float A, float c) {
    return kLog ? c * A : fmaf(-c, A, c > 0.f ? A : 0.f);
}

template <typename T>
__device__ __forceinline__ void put(T *p, const float (&v)[1]) { *p = from_f32<T>(v[0]); }

// What a tile tells the next ones of a channel, in one 64-bit word (whose two halves arrive together, so that no
// fences are needed): first how it maps the state that enters it, {A, H}: h -> A h + H; then, once that state is
// known, {kWhole, the state that leaves it}. A workspace of set bits says nothing yet. A lane's words of two channels are
// told and heard by one access where they lie on 16 bytes (kPairs), of which each is whole by itself.
constexpr unsigned kEmpty = 0xffffffffu, kWhole = 0xfffffffeu, kNan = 0x7fffffffu;
__device__ __forceinline__ unsigned factor_bits(float a) { return a == a ? __float_as_uint(a) : kNan; }
__device__ __forceinline__ unsigned long long bits(uint2 v) { return static_cast<unsigned long long>(v.y) << 32 | v.x; }
template <int kV, bool kPairs>
__device__ __forceinline__ void tell(uint2 *p, int count, const uint2 (&v)[kV]) {   // of the first `count` channels
    if constexpr (kPairs) {
        if (count > 0)
            asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(p), "l"(bits(v[0])), "l"(bits(v[1])) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i < count) asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p + i), "l"(bits(v[i])) : "memory");
    }
}
template <int kV, bool kPairs = false>
__device__ __forceinline__ void tell_map(uint2 *p, int count, const float (&A)[kV], const float (&H)[kV]) {
    uint2 w[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) w[v] = make_uint2(factor_bits(A[v]), __float_as_uint(H[v]));
    tell<kV, kPairs>(p, count, w);
}
template <int kV, bool kPairs = false>
__device__ __forceinline__ void tell_state(uint2 *p, int count, const float (&h)[kV]) {
    uint2 w[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) w[v] = make_uint2(kWhole, __float_as_uint(h[v]));
    tell<kV, kPairs>(p, count, w);
}
// Gates that grow: a product of factors that fp32 does not hold makes a NaN of a state of zero, and is reported; one that has
// become a NaN by a factor of zero, too. `a` is the product of a channel's neighbouring tokens.
template <bool kLog>
__device__ __forceinline__ void watch(const ScanArgs &p, bool live, float a) {
    if (kLog && live && !(a <= FLT_MAX)) atomicOr(p.err, kErrGateRange);
}
template <bool kLog>
__device__ __forceinline__ void watch(const ScanArgs &p, int count, float2 a) {
    if (kLog && ((count > 0 && !(a.x <= FLT_MAX)) || (count > 1 && !(a.y <= FLT_MAX)))) atomicOr(p.err, kErrGateRange);
}
// The state at the chain's start (zeros where none is given), and at its end where that is wanted.
template <int kV>
__device__ __forceinline__ void start(const ScanArgs &p, int b, int c, int count, float (&h)[kV]) {
#pragma unroll
    for (int v = 0; v < kV; ++v) h[v] = p.h0 && v < count ? p.h0[static_cast<int64_t>(b) * p.C + c + v] : 0.f;
}
template <int kV>
__device__ __forceinline__ void finish(const ScanArgs &p, int b, int c, int count, const float (&h)[kV]) {
    if (p.h_T)
#pragma unroll
        for (int v = 0; v < kV; ++v)
            if (v < count) p.h_T[static_cast<int64_t>(b) * p.C + c + v] = h[v];
}
__device__ __forceinline__ void give_up(const ScanArgs &p) {
    if ((threadIdx.x & 31) == 0) {
        atomicOr(p.err, kErrTimeout);
        if (p.head) *const_cast<volatile unsigned *>(&p.head->abort) = 0u;
    }
}
template <int kV, bool kPairs>
__device__ __forceinline__ void hear(const uint2 *p, int count, uint2 (&v)[kV]) {
    unsigned long long w[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) w[i] = kEmpty;
    if constexpr (kPairs) {
        if (count > 0) asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(w[0]), "=l"(w[1]) : "l"(p) : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
            if (i < count) asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(w[i]) : "l"(p + i) : "memory");
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = make_uint2(static_cast<unsigned>(w[i]), static_cast<unsigned>(w[i] >> 32));
}

constexpr unsigned kPolls = 1u << 21;   // of the wait of below: a second or two

// The state that enters a tile, from what the `left` tiles before it told: `p` is the nearest one's word of this
// thread's first channel, `hop` leads to the next further one. Of the nearest kAhead tiles one has to know the state
// that leaves it, and the maps of those in between are applied to that in their order, as they apply them
// themselves: whatever is known when, the bits are the same. The chain's first tile tells kWhole at once. Tiles are
// taken by ticket in the order of the chain, so that all of those are running or done and none of them waits for a
// later one: the wait ends. Its limit is for what cannot be foreseen. Run by a whole warp; false where it gave up.
template <int kV, bool kPairs, int kAhead>
__device__ __forceinline__ bool hear_state(const uint2 *p, int64_t hop, int left, int count, const Head *head,
                                         unsigned limit, float (&h)[kV]) {
#pragma unroll
    for (int v = 0; v < kV; ++v) h[v] = 0.f;
    for (unsigned polls = 0; polls < limit; ++polls) {
        uint2 w[kAhead][kV];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) hear<kV, kPairs>(p + j * hop, j < left ? count : 0, w[j]);
        int found[kV];
        bool known = true;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            found[v] = -1;
            bool told = true;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (told && found[v] < 0 && w[j][v].x == kWhole) found[v] = j;
                told &= w[j][v].x != kEmpty;
            }
            known &= found[v] >= 0 || v >= count;
        }
        if (__all_sync(0xffffffffu, known)) {
#pragma unroll
            for (int j = kAhead - 1; j >= 0; --j)
#pragma unroll
                for (int v = 0; v < kV; ++v) {
                    const float y = __uint_as_float(w[j][v].y);
                    if (j == found[v]) h[v] = y;
                    else if (j < found[v]) h[v] = fmaf(__uint_as_float(w[j][v].x), h[v], y);
                }
            return true;
        }
        if ((polls & 63u) == 63u && *reinterpret_cast<const volatile unsigned *>(&head->abort) == 0u) return false;
    }
    return false;
}

// How far away that may be: four tiles, or kFar where chains are few. Then the SMs hold many tiles of each, and the chain
// is what is waited for, a trip to L2 every so many tiles; with more chains hearing from further costs more than it gives.
// us, of 4 and 8: forward 131072 x 64 97 and 74, x 512 134 and 117, x 1024 (16 chains) 174 and 175, x 2048 (32) 286 and 316;
// fp32 x 128 172 and 122, x 512 (16) 259 and 230. Backward fp32 x 128 180 and 146, x 512 345 and 349; bf16, whose words
// are two a lane, x 64 158 and 168, x 512 232 and 292, so that it stays at four. (3 and 6 tiles instead of four: x 1024 181
// and 171 forward, 337 and 377 backward, four 172 and 312; x 2048 279 and 298, 509 and 610, four 281 and 508.)
template <int kV, bool kPairs, int kFar>
__device__ __forceinline__ bool entering(const ScanArgs &p, const uint2 *from, int64_t hop, int left, int count,
                                         float (&h)[kV]) {
    constexpr int kFew = 16;
    if (kFar > 4 && p.B * p.blocks <= kFew) return hear_state<kV, kPairs, kFar>(from, hop, left, count, p.head, p.polls, h);
    return hear_state<kV, kPairs, 4>(from, hop, left, count, p.head, p.polls, h);
}

// The tile of a ticket: `at` tiles along the chain, of channels c0 ..
struct Tile {
    int b, c0, at;
    __device__ __forceinline__ Tile(const ScanArgs &p, unsigned ticket, int width) {
        const unsigned chains = static_cast<unsigned>(p.B) * p.blocks, rest = ticket % chains;
        at = ticket / chains;
        b = rest / p.blocks;
        c0 = rest % p.blocks * width;
    }
};
// One ticket for a whole CTA: tiles start in the order of the tickets.
__device__ __forceinline__ unsigned take_ticket(const ScanArgs &p) {
    if (!p.head) return blockIdx.x;
    __shared__ unsigned mine;
    if (threadIdx.x == 0) mine = atomicAdd(&p.head->ticket, 1u) + 1u;   // from all bits set
    __syncthreads();
    return mine;
}

// ---- bf16 tensors that start in the middle of 4 bytes, of which no asynchronous copy takes all rows
// A tile is kWarps x kTok tokens of 32 channels; a thread holds kTok tokens of one channel in registers, all of its
// loads on their way at once. Every warp finds how its tokens map a state, the last one joins those maps, tells
// the tile's own, hears the state that enters the tile and tells the one that leaves it; then every warp walks its tokens.
template <typename T, bool kLog, int kTok, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) scan_fwd_kernel(ScanArgs p) {
    constexpr int kTile = kTok * kWarps, kV = 1;
    __shared__ float2 maps[kWarps][32];
    __shared__ float enter[kV][32];
    const Tile at(p, take_ticket(p), 32);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int b = at.b, c = at.c0 + lane * kV, n = valid_tokens(p, b);
    const bool live = c < p.C;
    const int first = at.at * kTile, t0 = first + warp * kTok;
    const int64_t row = static_cast<int64_t>(b) * p.T + t0;
    T *y = static_cast<T *>(p.y) + row * p.C + c;
    const int last = n > 0 ? (n - 1) / kTile : 0;
    if (at.at > last) {   // nothing but masked tokens
        const float zero[kV] = {};
        if (live)
            for (int i = 0; i < kTok && t0 + i < p.T; ++i) put<T>(y + static_cast<int64_t>(i) * p.C, zero);
        return;
    }
    const int m = min(max(n - t0, 0), kTok);   // of this warp's tokens, how many are valid
    T x[kTok], g[kTok];
    {
        const T *px = static_cast<const T *>(p.x) + b * p.xb + t0 * p.xt + c;
        const T *pg = static_cast<const T *>(p.gate) + b * p.gb + t0 * p.gt + c;
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (live && i < m) {
                x[i] = *(px + i * p.xt);
                g[i] = *(pg + i * p.gt);
            }
    }
    float co[kTok][kV], A[kV], H[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) A[v] = 1.f, H[v] = 0.f;
#pragma unroll
    for (int i = 0; i < kTok; ++i)
        if (i < m) {
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                float a, w;
                factors<T, kLog>(gate_exp<T, kLog>(to_f32(g[i])), a, w);
                co[i][v] = coefficient<kLog>(a, w);
                A[v] = shrink<kLog>(A[v], co[i][v]);
                H[v] = advance<kLog>(H[v], to_f32(x[i]), co[i][v]);
            }
        }
    if (keeps(A[0], m)) {
        float lost = 0.f;
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (i < m) lost = lose<T, kLog>(lost, to_f32(g[i]));
        A[0] = 1.f - lost;
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) maps[warp][v * 32 + lane] = make_float2(A[v], H[v]);
    __syncthreads();
    // the map of the tile's tokens before this warp's
    float pa[kV], ph[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) pa[v] = 1.f, ph[v] = 0.f;
    for (int w = 0; w < warp; ++w)
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const float2 f = maps[w][v * 32 + lane];
            ph[v] = fmaf(f.x, ph[v], f.y);
            pa[v] *= f.x;
        }
    watch<kLog>(p, live, A[0]);
    watch<kLog>(p, live, pa[0] * A[0]);
    float in[kV];
    if (warp == kWarps - 1) {
        uint2 *here = p.carry + (static_cast<int64_t>(b) * p.tiles + at.at) * p.C + c;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            H[v] = fmaf(A[v], ph[v], H[v]);
            A[v] *= pa[v];
        }
        if (at.at > 0 && at.at < last) tell_map<kV>(here, live, A, H);
        if (at.at == 0) start<kV>(p, b, c, live, in);
        else if (!entering<kV, false, 4>(p, here - p.C, -static_cast<int64_t>(p.C), at.at, live, in)) give_up(p);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            enter[v][lane] = in[v];
            H[v] = fmaf(A[v], in[v], H[v]);
        }
        if (at.at < last) tell_state<kV>(here, live, H);
        else finish<kV>(p, b, c, live, H);
    }
    __syncthreads();
    if (!live) return;
    float h[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) h[v] = fmaf(pa[v], enter[v][lane], ph[v]);
    if (p.states && m > 0 && t0 % KLA_SCAN_SPAN == 0) {
        const int64_t spans = (p.T + KLA_SCAN_SPAN - 1) / KLA_SCAN_SPAN;
        float *s = p.states + (b * spans + t0 / KLA_SCAN_SPAN) * p.C + c;
#pragma unroll
        for (int v = 0; v < kV; ++v) s[v] = h[v];
    }
#pragma unroll
    for (int i = 0; i < kTok; ++i)
        if (i < m) {
#pragma unroll
            for (int v = 0; v < kV; ++v) h[v] = advance<kLog>(h[v], to_f32(x[i]), co[i][v]);
            put<T>(y + static_cast<int64_t>(i) * p.C, h);
        } else if (t0 + i < p.T) {
            const float zero[kV] = {};
            put<T>(y + static_cast<int64_t>(i) * p.C, zero);
        }
}

// The same against time: what reaches the state behind a token's is e_{t-1} = a_t (dy_t + e_t), and a tile's map
// {A, D} is e -> A e + D with D = sum of dy_t times the product of the tile's gates up to t. A tile is one span, whose
// entering state the forward pass has kept; h_{t-1} is walked from it again.
template <typename T, bool kLog, int kTok, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) scan_bwd_kernel(ScanArgs p) {
    constexpr int kTile = kTok * kWarps, kV = 1;
    static_assert(kTile == KLA_SCAN_SPAN, "");
    __shared__ float2 maps[kWarps][32];
    __shared__ float backs[kWarps][32], enter[kV][32];
    const Tile at(p, take_ticket(p), 32);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int b = at.b, c = at.c0 + lane * kV, n = valid_tokens(p, b), tile = p.tiles - 1 - at.at;
    const bool live = c < p.C;
    const int t0 = tile * kTile + warp * kTok;
    const int64_t row = static_cast<int64_t>(b) * p.T + t0;
    T *dx = static_cast<T *>(p.y) + row * p.C + c, *dg = static_cast<T *>(p.dg) + row * p.C + c;
    const float zero[kV] = {};
    const int last = n > 0 ? (n - 1) / kTile : 0;
    if (tile > last) {
        if (live)
            for (int i = 0; i < kTok && t0 + i < p.T; ++i) {
                put<T>(dx + static_cast<int64_t>(i) * p.C, zero);
                put<T>(dg + static_cast<int64_t>(i) * p.C, zero);
            }
        return;
    }
    const int m = min(max(n - t0, 0), kTok);
    T x[kTok], d[kTok];
    float e[kTok][kV], h[kV];   // e: exp(gate)
    {
        T g[kTok];
        const T *px = static_cast<const T *>(p.x) + b * p.xb + t0 * p.xt + c;
        const T *pg = static_cast<const T *>(p.gate) + b * p.gb + t0 * p.gt + c;
        const T *pd = static_cast<const T *>(p.dy) + b * p.db + t0 * p.dt + c;
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (live && i < m) {
                g[i] = *(pg + i * p.gt);
                x[i] = *(px + i * p.xt);
                d[i] = *(pd + i * p.dt);
            }
        const float *s = p.states + (static_cast<int64_t>(b) * p.tiles + tile) * p.C + c;
#pragma unroll
        for (int v = 0; v < kV; ++v) h[v] = live && n > 0 ? s[v] : 0.f;
#pragma unroll
        for (int i = 0; i < kTok; ++i)
#pragma unroll
            for (int v = 0; v < kV; ++v) e[i][v] = i < m ? gate_exp<T, kLog>(to_f32(g[i])) : 0.f;
    }
    float A[kV], H[kV], D[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) A[v] = 1.f, H[v] = D[v] = 0.f;
#pragma unroll
    for (int i = 0; i < kTok; ++i)
        if (i < m) {
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                float a, w;
                factors<T, kLog>(e[i][v], a, w);
                const float co = coefficient<kLog>(a, w);
                A[v] = shrink<kLog>(A[v], co);
                H[v] = advance<kLog>(H[v], to_f32(x[i]), co);
                D[v] = fmaf(A[v], to_f32(d[i]), D[v]);
            }
        }
    if (live && keeps(A[0], m)) {
        const T *pg = static_cast<const T *>(p.gate) + b * p.gb + t0 * p.gt + c;
        float lost = 0.f;
        for (int i = 0; i < m; ++i) lost = lose<T, kLog>(lost, to_f32(*(pg + i * p.gt)));
        A[0] = 1.f - lost;
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        maps[warp][v * 32 + lane] = make_float2(A[v], H[v]);
        backs[warp][v * 32 + lane] = D[v];
    }
    __syncthreads();
    float sa[kV], sd[kV];   // the map of the tile's tokens after this warp's
#pragma unroll
    for (int v = 0; v < kV; ++v) sa[v] = 1.f, sd[v] = 0.f;
    for (int w = kWarps - 1; w > warp; --w)
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const float f = maps[w][v * 32 + lane].x;
            sd[v] = fmaf(f, sd[v], backs[w][v * 32 + lane]);
            sa[v] *= f;
        }
    watch<kLog>(p, live, A[0]);
    watch<kLog>(p, live, sa[0] * A[0]);
    if (warp == 0) {
        float in[kV];
        uint2 *here = p.carry + (static_cast<int64_t>(b) * p.tiles + tile) * p.C + c;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            D[v] = fmaf(A[v], sd[v], D[v]);
            A[v] *= sa[v];
        }
        if (tile > 0 && tile < last) tell_map<kV>(here, live, A, D);
        if (tile == last) start<kV>(p, b, c, live, in);
        else if (!entering<kV, false, 4>(p, here + p.C, p.C, last - tile, live, in)) give_up(p);
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            enter[v][lane] = in[v];
            D[v] = fmaf(A[v], in[v], D[v]);
        }
        if (tile > 0) tell_state<kV>(here, live, D);
        else finish<kV>(p, b, c, live, D);
    }
    // the states before this warp's tokens
    for (int w = 0; w < warp; ++w)
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const float2 f = maps[w][v * 32 + lane];
            h[v] = fmaf(f.x, h[v], f.y);
        }
    float before[kTok][kV];
#pragma unroll
    for (int i = 0; i < kTok; ++i)
        if (i < m) {
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                float a, w;
                factors<T, kLog>(e[i][v], a, w);
                before[i][v] = h[v];
                h[v] = advance<kLog>(h[v], to_f32(x[i]), coefficient<kLog>(a, w));
            }
        }
    __syncthreads();
    if (!live) return;
#pragma unroll
    for (int v = 0; v < kV; ++v) h[v] = fmaf(sa[v], enter[v][lane], sd[v]);   // now what reaches the state
#pragma unroll
    for (int i = kTok - 1; i >= 0; --i)
        if (i < m) {
            float ox[kV], og[kV];
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                float a, w;
                factors<T, kLog>(e[i][v], a, w);
                const float dh = to_f32(d[i]) + h[v];
                h[v] = a * dh;
                ox[v] = w * dh;
                og[v] = kLog ? before[i][v] * h[v] : w * (before[i][v] - to_f32(x[i])) * h[v];
            }
            put<T>(dx + static_cast<int64_t>(i) * p.C, ox);
            put<T>(dg + static_cast<int64_t>(i) * p.C, og);
        } else if (t0 + i < p.T) {
            put<T>(dx + static_cast<int64_t>(i) * p.C, zero);
            put<T>(dg + static_cast<int64_t>(i) * p.C, zero);
        }
}

// Tokens of a thread, warps at them and CTAs of an SM. Each side of the choice at 8 x 4096 x 2048 bf16 and, in fp32, 8 x
// 2048 x 2048, us: forward 32 tokens x 8 warps x 2 CTAs 82 and 102, 16 x 8 x 3 89 and 95; backward 16 x 8 x 2 138 and 181,
// 16 x 4 x 4 134 and 179, but 609 instead of 525 at 1 x 131072 x 2048, whose chain gets twice as long (all by copies of the
// warps' own, and before the backward pass had its warp for the chain: 71 and 85, 105 and 128 since).
struct Shape {
    int tok, warps, ctas;
    constexpr int tile() const { return tok * warps; }
};
constexpr Shape fwd_shape(int esz, bool ring) { return ring && esz == 2 ? Shape{32, 8, 2} : Shape{16, 8, 3}; }
constexpr Shape bwd_shape() { return Shape{16, 8, 2}; }

// ---- tiles through shared memory: rows of 128 bytes (64 channels of bf16, 32 of fp32), 4 bytes a lane; of bf16 rows that
// start in the middle of 4 bytes, or end there, 132
constexpr int kEvenRow = 128, kOddRow = 132;
// How rows get there: one instruction of the tensor memory accelerator a tile and tensor, asynchronous copies by the warps
// that need them, or those of rows as they lie.
enum Copies { kTma, kEven, kOdd };
struct Maps {
    CUtensorMap x, gate, dy;
};
__device__ __forceinline__ void load_tile(uint32_t to, const CUtensorMap *map, uint32_t bar, int c, int t, int b) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(to),
        "l"(map), "r"(bar), "r"(c), "r"(t), "r"(b)
        : "memory");
}

// What a lane has of a row: two channels of bf16, whose arithmetic is paired, or one of fp32. A gate is kept as one
// number: bf16: w, or a where KLA_SCAN_LOG, with h = a h + w x and a = 1 - w, whose rounding of 2^-25 is that of a
// itself where it is near 1 (and whose exponential and reciprocal are the hardware's, off by 2^-21 at gates of 10; where a
// is small Exact takes the warp's tokens). fp32: the coefficient of above in the forward pass; exp(gate) in the backward pass, from
// which both factors come to their last bits.
template <typename T, bool kLog, bool kBwd>
struct Lane;
template <bool kLog, bool kBwd>
struct Lane<__nv_bfloat16, kLog, kBwd> {
    static constexpr int kV = 2;
    using V = float2;
    static __device__ __forceinline__ V unpack(uint32_t r) {
        return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    }
    static __device__ __forceinline__ V load(const uint8_t *p) { return unpack(*reinterpret_cast<const uint32_t *>(p)); }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, V v) {
        *reinterpret_cast<uint32_t *>(p) = ptx::pack_bf16(v.x, v.y);
    }
    static __device__ __forceinline__ V all(float x) { return both(x); }
    static __device__ __forceinline__ V fma(V a, V b, V c) { return fma2(a, b, c); }
    static __device__ __forceinline__ V mul(V a, V b) { return mul2(a, b); }
    static __device__ __forceinline__ V add(V a, V b) { return add2(a, b); }
    static __device__ __forceinline__ V keep(V gate) {
        V e = mul2(gate, both(1.4426950408889634f));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
        if (kLog) return e;
        e = add2(e, both(1.f));
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
        asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
        return e;
    }
    static __device__ __forceinline__ V a(V k) { return kLog ? k : fma2(k, both(-1.f), both(1.f)); }
    static __device__ __forceinline__ V w(V k) { return kLog ? both(1.f) : k; }
    // h, a token on; prod a, a token on
    static __device__ __forceinline__ V advance(V h, V x, V k) { return fma2(a(k), h, kLog ? x : mul2(k, x)); }
    static __device__ __forceinline__ V shrink(V A, V k) { return mul2(A, a(k)); }
    static __device__ __forceinline__ V reach(V dh, V k) { return mul2(a(k), dh); }   // a dh
    static __device__ __forceinline__ V loss(V k) { return k; }                       // 1 - a, of KLA_SCAN_SIGMOID
};
template <bool kLog, bool kBwd>
struct Lane<float, kLog, kBwd> {
    static constexpr int kV = 1;
    using V = float;
    static __device__ __forceinline__ V load(const uint8_t *p) { return *reinterpret_cast<const float *>(p); }
    static __device__ __forceinline__ void store(float *p, V v) { *p = v; }
    static __device__ __forceinline__ V all(float x) { return x; }
    static __device__ __forceinline__ V fma(V a, V b, V c) { return fmaf(a, b, c); }
    static __device__ __forceinline__ V mul(V a, V b) { return a * b; }
    static __device__ __forceinline__ V add(V a, V b) { return a + b; }
    static __device__ __forceinline__ V keep(V gate) {
        const float e = gate_exp<float, kLog>(gate);
        return kBwd ? e : coefficient<kLog>(a(e), w(e));
    }
    static __device__ __forceinline__ V a(V e) { return kLog ? e : e * w(e); }
    static __device__ __forceinline__ V w(V e) { return kLog ? 1.f : __frcp_rn(1.f + e); }
    static __device__ __forceinline__ V advance(V h, V x, V k) {
        return kla::advance<kLog>(h, x, kBwd ? coefficient<kLog>(a(k), w(k)) : k);
    }
    static __device__ __forceinline__ V shrink(V A, V k) {
        return kla::shrink<kLog>(A, kBwd ? coefficient<kLog>(a(k), w(k)) : k);
    }
    static __device__ __forceinline__ V reach(V dh, V k) { return a(k) * dh; }
    static __device__ __forceinline__ V loss(V k) { return kBwd ? w(k) : k > 0.f ? k : 1.f + k; }
};
// The bf16 sigmoid of a warp with gates that Lane does not hold: a gate kept as its coefficient, of which both factors come
// to their last bits.
struct Exact {
    using V = float2;
    static __device__ __forceinline__ float keep(float gate) {
        float a, w;
        factors<__nv_bfloat16, false>(gate_exp<__nv_bfloat16, false>(gate), a, w);
        return coefficient<false>(a, w);
    }
    static __device__ __forceinline__ V keep(V gate) { return make_float2(keep(gate.x), keep(gate.y)); }
    static __device__ __forceinline__ float w(float c) { return c > 0.f ? c : 1.f + c; }
    static __device__ __forceinline__ V w(V k) { return make_float2(w(k.x), w(k.y)); }
    static __device__ __forceinline__ V advance(V h, V x, V k) {
        return make_float2(kla::advance<false>(h.x, x.x, k.x), kla::advance<false>(h.y, x.y, k.y));
    }
    static __device__ __forceinline__ V shrink(V A, V k) {
        return make_float2(kla::shrink<false>(A.x, k.x), kla::shrink<false>(A.y, k.y));
    }
    static __device__ __forceinline__ V reach(V dh, V k) { return shrink(dh, k); }
};
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float2 larger(float2 a, float2 b) { return make_float2(fmaxf(a.x, b.x), fmaxf(a.y, b.y)); }
__device__ __forceinline__ float part(float v, int) { return v; }
__device__ __forceinline__ float part(float2 v, int i) { return i ? v.y : v.x; }
template <int kV>
__device__ __forceinline__ auto whole(const float (&v)[kV]) {
    if constexpr (kV == 1) return v[0];
    else return make_float2(v[0], v[1]);
}
// A lane's product of m factors, once more where it is close to 1, from the gates: log gates, or those of Exact. Few lanes need
// it, and its loop unrolled costs the others 2 % of the backward pass. 8 x 4096 x 2048 bf16 with log gates that are all
// such, of -softplus(N(-10, 1)), 86 and 132 us, others 65 and 105.
template <typename T, bool kLog, typename V, typename F>
__device__ __forceinline__ V kept_product(V A, int count, int m, F gate) {
    constexpr int kV = sizeof(V) / sizeof(float);
    bool any = false;
#pragma unroll
    for (int v = 0; v < kV; ++v) any |= v < count && keeps(part(A, v), m);   // past the last channel there is anything
    if (any) {
        float lost[kV] = {}, a[kV];
#pragma unroll 1
        for (int i = 0; i < m; ++i) {
            const V g = gate(i);
#pragma unroll
            for (int v = 0; v < kV; ++v) lost[v] = lose<T, kLog>(lost[v], part(g, v));
        }
#pragma unroll
        for (int v = 0; v < kV; ++v) a[v] = keeps(part(A, v), m) ? 1.f - lost[v] : part(A, v);
        A = whole<kV>(a);
    }
    return A;
}
// The same from the losses that a sigmoid's tokens are kept by: with gates of N(10, 1) 70 and 114 us, others 67 and 109 (from
// the gates 93 and 132).
template <typename L, int kTok, typename V>
__device__ __forceinline__ V kept_product(V A, int count, int m, const V (&k)[kTok]) {
    constexpr int kV = sizeof(V) / sizeof(float);
    bool any = false;
#pragma unroll
    for (int v = 0; v < kV; ++v) any |= v < count && keeps(part(A, v), m);
    if (any) {
        V lost = L::all(0.f);
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (i < m) lost = L::fma(L::loss(k[i]), L::fma(lost, L::all(-1.f), L::all(1.f)), lost);
        float a[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) a[v] = keeps(part(A, v), m) ? 1.f - part(lost, v) : part(A, v);
        A = whole<kV>(a);
    }
    return A;
}
// The largest w of a lane's tokens, where it matters: bf16, sigmoid.
template <typename T, bool kLog>
struct Most {
    static constexpr bool kAsks = sizeof(T) == 2 && !kLog;
    float w = 0.f;
    template <typename V>
    __device__ __forceinline__ void see(V k) {
        if (kAsks) w = fmaxf(fmaxf(w, part(k, 0)), part(k, 1));
    }
    // Whether the warp's tokens are Exact's: of any lane a gate below -6 among its `count` channels. There 1 - w is off by
    // 2^-23, 2^-14 of a (from -5 on, gates of N(0, 1) have one such in 2000 warps, and 8 x 4096 x 2048 took 70 us, not 67).
    // In other channels there may be anything: where there is one, the gates are looked at once more.
    // A warp as a whole, as lanes that go apart cost the others more: 8 x 4096 x 2048 66.7 and 109.1 us without Exact, 67.1
    // and 109.6 with it, 119.8 and 171 where all warps take it; lane by lane 66.7 and 113.6.
    template <typename F>
    __device__ __forceinline__ bool any(int count, int m, F gate) const {
        if (!kAsks) return false;
        bool here = count > 0 && w > 0.9975274f;   // sigmoid(6)
        if (here && count == 1) {
            here = false;
#pragma unroll 1
            for (int i = 0; i < m; ++i) here |= part(gate(i), 0) < -6.f;
        }
        return __any_sync(0xffffffffu, here);
    }
};
using One = float[1];
using Two = float[2];
__device__ __forceinline__ const One &parts(const float &v) { return reinterpret_cast<const One &>(v); }
__device__ __forceinline__ const Two &parts(const float2 &v) { return reinterpret_cast<const Two &>(v); }
__device__ __forceinline__ void copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void *from, int size) {   // the rest zeros
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(size) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
// Rows 0 .. m - 1 of kTok, `pitch` values apart, into this warp's part of a buffer; `left` channels there are from the
// rows' first on. kOdd: rows of bf16 that start in the middle of 4 bytes or end there. Their words are copied as they lie,
// so that a row may take 33 of them; the word that a row starts in the middle of begins with a value of the tensor's too,
// as the tensor starts on 4 bytes, and of the one that a row ends in the middle of only that half is read.
template <typename T, int kTok, Copies kBy>
__device__ __forceinline__ void copy_rows(uint8_t *to, const T *from, int64_t pitch, int m, int left, bool wide) {
    const int lane = threadIdx.x & 31;
    const uint32_t s = ptx::smem_u32(to);
    const char *f = reinterpret_cast<const char *>(from);
    pitch *= sizeof(T);
    if constexpr (kBy == kOdd) {
        static_assert(kTok <= 32, "");
        // even and odd rows: where the lane's word is, whether and how much of it is there
        const uint32_t odd = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(f) >> 1) & 1;
        const char *at[2];
        int size[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int half = r ? (odd ^ (static_cast<uint32_t>(pitch) >> 1)) & 1 : odd, first = 2 * lane - half;
            at[r] = f + r * pitch + 2 * first;
            size[r] = first >= left ? 0 : first + 1 < left ? 4 : 2;
        }
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            if (i < m && size[i & 1]) copy4(s + i * kOddRow + lane * 4, at[i & 1], size[i & 1]);
            at[i & 1] += 2 * pitch;
        }
        // the 33rd words, a row a lane
        const char *row = f + lane * pitch;
        if (lane < m && (reinterpret_cast<uintptr_t>(row) & 2) && left > 63)
            copy4(s + lane * kOddRow + 128, row + 126, left > 64 ? 4 : 2);
    } else if (wide) {
        const int off = (lane & 7) * 16;
        const bool in = off < left * static_cast<int64_t>(sizeof(T));
#pragma unroll
        for (int i = 0; i < kTok; i += 4) {
            const int r = i + lane / 8;
            if (r < m && in) copy16(s + r * kEvenRow + off, f + r * pitch + off);
        }
    } else {
        const int off = lane * 4;
        const bool in = off < left * static_cast<int64_t>(sizeof(T));
#pragma unroll
        for (int i = 0; i < kTok; ++i)
            if (i < m && in) copy4(s + i * kEvenRow + off, f + i * pitch + off);
    }
}
// A lane's two values of a row that starts in the middle of 4 bytes, or not: rows of one tensor alternate, or none does.
template <Copies kBy>
struct Parity {
    uint32_t shift[2];   // of even and odd rows, in bits
    template <typename T>
    __device__ __forceinline__ Parity(const T *first, int64_t pitch) {
        if (kBy == kOdd) {
            const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(first) >> 1) & 1;
            shift[0] = 16 * at;
            shift[1] = 16 * (at ^ (static_cast<uint32_t>(pitch) & 1));
        }
    }
    template <typename L>
    __device__ __forceinline__ typename L::V load(const uint8_t *p, int row) const {
        if constexpr (kBy != kOdd) {
            return L::load(p);
        } else {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(p);
            return L::unpack(__funnelshift_r(w[0], w[1], row & 1 ? shift[1] : shift[0]));
        }
    }
    template <typename L, typename T>
    __device__ __forceinline__ void store(T *p, typename L::V v, int row, int count) const {
        if constexpr (kBy != kOdd) {
            L::store(p, v);
        } else if (shift[row & 1] == 0 && count == 2) {
            L::store(p, v);
        } else {
            p[0] = from_f32<T>(part(v, 0));
            if (count == 2) p[1] = from_f32<T>(part(v, 1));
        }
    }
};

// Tiles one after the other. A CTA takes a ticket for its next tile while it works on one, not earlier, so that where
// tiles are few no CTA has two of them and another none.
struct Turns {
    const ScanArgs &p;
    unsigned total, now;
    __device__ __forceinline__ Turns(const ScanArgs &a) : p(a) {
        total = static_cast<unsigned>(a.B) * a.blocks * a.tiles;
        now = blockIdx.x;
    }
    __device__ __forceinline__ unsigned ask() const {   // one thread
        return p.head ? atomicAdd(&p.head->ticket, 1u) + 1u : now + gridDim.x;
    }
};

constexpr uint32_t kWaits = 400000;   // of 20 us at most, more than `entering` takes to give up

// How many channels a lane has from c on: kV or none where rows have an even number.
template <Copies kBy, int kV>
__device__ __forceinline__ int channels(const ScanArgs &p, int c) {
    return kBy == kOdd ? min(max(p.C - c, 0), kV) : c < p.C ? kV : 0;
}

// Runs f with whether all of a warp's kTok tokens are valid, as the loops over them have no conditions then, and by which
// functions the warp takes them.
template <typename L, typename X, typename F>
__device__ __forceinline__ void by_case(bool full, bool exact, F f) {
    if (exact) f(std::false_type{}, X{});
    else if (full) f(std::true_type{}, L{});
    else f(std::false_type{}, L{});
}

// As above, with tiles one after the other: while a CTA waits for the state that enters one and writes its outputs, the
// next one's rows are on their way.
template <typename T, bool kLog, Copies kBy, int kTok, int kWarps, int kCtas>
__global__ void __launch_bounds__(32 * kWarps, kCtas) scan_fwd_ring_kernel(ScanArgs p, bool wide, const __grid_constant__ Maps maps) {
    using L = Lane<T, kLog, false>;
    using X = typename std::conditional<Most<T, kLog>::kAsks, Exact, L>::type;
    using V = typename L::V;
    constexpr int kTile = kTok * kWarps, kV = L::kV, kWidth = 32 * kV, kRow = kBy == kOdd ? kOddRow : kEvenRow;
    constexpr bool kPairs = kV == 2 && kBy != kOdd;
    extern __shared__ __align__(128) uint8_t buf[];   // x twice, gate once: kTile rows each
    __shared__ V map_a[kWarps][32], map_h[kWarps][32], enter[32];
    __shared__ unsigned s_next;
    __shared__ uint64_t full[2];   // kTma: the rows of an even or odd turn's tile are there
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    uint8_t *const mine = buf + warp * kTok * kRow;
    uint8_t *const gates = mine + 2 * kTile * kRow;
    Turns turns(p);
    if (p.head) dependency_wait();
    const uint32_t b_full = ptx::smem_u32(full);
    if (kBy == kTma && threadIdx.x == 0) {
        ptx::mbar_init(b_full, 1);
        ptx::mbar_init(b_full + 8, 1);
        ptx::fence_mbar_init();
    }
    if (kBy == kTma) __syncthreads();
    // every warp its own rows, or one thread the tile (after a barrier: all warps are done with what it replaces)
    auto fetch = [&](unsigned ticket, int stage) {
        const Tile at(p, ticket, kWidth);
        if constexpr (kBy == kTma) {
            if (threadIdx.x == 0 && at.at * kTile < valid_tokens(p, at.b)) {
                const uint32_t bar = b_full + 8 * stage, to = ptx::smem_u32(buf);
                ptx::mbar_arrive_expect_tx(bar, 2 * kTile * kRow);
                load_tile(to + 2 * kTile * kRow, &maps.gate, bar, at.c0, at.at * kTile, at.b);
                load_tile(to + stage * kTile * kRow, &maps.x, bar, at.c0, at.at * kTile, at.b);
            } else if (threadIdx.x == 0) {
                ptx::mbar_arrive(b_full + 8 * stage);
            }
            return;
        }
        const int t0 = at.at * kTile + warp * kTok, m = min(valid_tokens(p, at.b) - t0, kTok);
        const int left = p.C - at.c0;
        copy_rows<T, kTok, kBy>(gates, static_cast<const T *>(p.gate) + at.b * p.gb + t0 * p.gt + at.c0, p.gt, m, left,
                                 wide);
        copy_rows<T, kTok, kBy>(mine + stage * kTile * kRow,
                                 static_cast<const T *>(p.x) + at.b * p.xb + t0 * p.xt + at.c0, p.xt, m, left, wide);
        copies_commit();
    };
    unsigned ticket = blockIdx.x;
    if (p.head) {
        if (threadIdx.x == 0) s_next = turns.ask();
        __syncthreads();
        ticket = s_next;
        __syncthreads();
    }
    if (ticket < turns.total) fetch(ticket, 0);
    for (unsigned turn = 0; ticket < turns.total; ++turn) {
        const int stage = turn & 1;
        const Tile at(p, ticket, kWidth);
        turns.now = ticket;
        unsigned asked = 0;
        const int b = at.b, c = at.c0 + lane * kV, n = valid_tokens(p, b), t0 = at.at * kTile + warp * kTok;
        const int count = channels<kBy, kV>(p, c);
        const int last = n > 0 ? (n - 1) / kTile : 0;
        const int m = min(max(n - t0, 0), kTok);   // of this warp's tokens, how many are valid
        const uint8_t *xs = mine + stage * kTile * kRow + lane * 4, *gs = gates + lane * 4;
        const Parity<kBy> of_x(static_cast<const T *>(p.x) + b * p.xb + t0 * p.xt + at.c0, p.xt);
        const Parity<kBy> of_g(static_cast<const T *>(p.gate) + b * p.gb + t0 * p.gt + at.c0, p.gt);
        V k[kTok], A = L::all(1.f), H = L::all(0.f);
        if constexpr (kBy == kTma) {
            if (!__all_sync(0xffffffffu, ptx::mbar_wait_bounded(b_full + 8 * stage, turn >> 1 & 1, kWaits)))
                give_up(p);   // and on, with whatever is there: the other warps meet this one at their barriers
        } else {
            copies_wait();
            __syncwarp();
        }
        if (threadIdx.x == 0) asked = turns.ask();
        Most<T, kLog> most;
        auto map_tokens = [&](auto full, auto by) {
            using K = decltype(by);
            A = L::all(1.f);
            H = L::all(0.f);
#pragma unroll
            for (int i = 0; i < kTok; ++i)
                if (full || i < m) {
                    k[i] = K::keep(of_g.template load<L>(gs + i * kRow, i));
                    if (std::is_same<K, L>::value) most.see(k[i]);
                    A = K::shrink(A, k[i]);
                    H = K::advance(H, of_x.template load<L>(xs + i * kRow, i), k[i]);
                }
        };
        by_case<L, L>(m == kTok, false, map_tokens);
        const bool exact = most.any(count, m, [&](int i) { return of_g.template load<L>(gs + i * kRow, i); });
        if (exact) map_tokens(std::false_type{}, X{});
        if (kLog || exact) A = kept_product<T, kLog>(A, count, m, [&](int i) { return of_g.template load<L>(gs + i * kRow, i); });
        else A = kept_product<L>(A, count, m, k);
        __syncwarp();
        map_a[warp][lane] = A;
        map_h[warp][lane] = H;
        if (threadIdx.x == 0) s_next = asked;
        __syncthreads();
        const unsigned next = s_next;
        // the map of the tile's tokens before this warp's: all loads on their way at once, as the chain waits for the last warp
        V pa = L::all(1.f), ph = L::all(0.f);
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w)
            if (w < warp) {
                ph = L::fma(map_a[w][lane], ph, map_h[w][lane]);
                pa = L::mul(pa, map_a[w][lane]);
            }
        watch<kLog>(p, count, A);
        watch<kLog>(p, count, L::mul(A, pa));
        const bool teller = warp == kWarps - 1 && at.at <= last;
        uint2 *here = p.carry + (static_cast<int64_t>(b) * p.tiles + at.at) * p.C + c;
        if (teller) {
            H = L::fma(A, ph, H);
            A = L::mul(A, pa);
            if (at.at > 0 && at.at < last) tell_map<kV, kPairs>(here, count, parts(A), parts(H));
        }
        if (next < turns.total && (kBy == kTma || !teller)) fetch(next, stage ^ 1);
        if (teller) {
            float in[kV];
            if (at.at == 0) start<kV>(p, b, c, count, in);
            else if (!entering<kV, kPairs, 8>(p, here - p.C, -static_cast<int64_t>(p.C), at.at, count, in)) give_up(p);
            const V e = whole<kV>(in);
            H = L::fma(A, e, H);
            if (at.at < last) tell_state<kV, kPairs>(here, count, parts(H));
            else finish<kV>(p, b, c, count, parts(H));
            enter[lane] = e;
            if (kBy != kTma && next < turns.total) fetch(next, stage ^ 1);   // which nobody waits for
        }
        __syncthreads();
        if (count > 0) {
            V h = L::fma(pa, enter[lane], ph);
            if (p.states && m > 0 && t0 % KLA_SCAN_SPAN == 0) {
                const int64_t spans = (p.T + KLA_SCAN_SPAN - 1) / KLA_SCAN_SPAN;
                float *s = p.states + (b * spans + t0 / KLA_SCAN_SPAN) * p.C + c;
#pragma unroll
                for (int v = 0; v < kV; ++v)
                    if (v < count) s[v] = part(h, v);
            }
            T *y = static_cast<T *>(p.y) + (static_cast<int64_t>(b) * p.T + t0) * p.C + c;
            const Parity<kBy> of_y(y, p.C);
            by_case<L, X>(m == kTok, exact, [&](auto full, auto by) {
                using K = decltype(by);
#pragma unroll
                for (int i = 0; i < kTok; ++i, y += p.C)
                    if (full || i < m) {
                        h = K::advance(h, of_x.template load<L>(xs + i * kRow, i), k[i]);
                        of_y.template store<L>(y, h, i, count);
                    } else if (t0 + i < p.T) {
                        of_y.template store<L>(y, L::all(0.f), i, count);
                    }
            });
        }
        __syncwarp();
        ticket = next;
    }
}

// The backward pass has a warp for the chain beside those for the tokens (138 -> 122 us at 8 x 4096 x 2048, before tiles
// came by tensor maps; the forward pass needs its registers more and lost by it, 82 -> 87). Barriers: `maps` completes when every warp has left the map of
// its tokens, `carry` when what enters them is there; next[i] when the ticket of the tile after one of parity i is.
template <typename V, int kWarps>
struct Shared {
    V a[2][kWarps][32], h[2][kWarps][32], d[kWarps][32];
    V enter[kWarps][32];
    unsigned ticket[2];
    uint64_t maps, carry, next[2], full[2];
};

template <typename L, bool kLog, Copies kBy, int kWarps, typename F>
__device__ __forceinline__ void carry_warp(const ScanArgs &p, Shared<typename L::V, kWarps> &sh, Turns &turns,
                                           unsigned ticket, int tile_tokens, F fetch_tile) {
    using V = typename L::V;
    constexpr int kV = L::kV;
    constexpr bool kPairs = kV == 2 && kBy != kOdd;
    using namespace ptx;
    const int lane = threadIdx.x & 31;
    const uint32_t b_maps = smem_u32(&sh.maps), b_carry = smem_u32(&sh.carry), b_next = smem_u32(sh.next);
    for (unsigned i = 0; ticket < turns.total; ++i) {
        const Tile at(p, ticket, 32 * kV);
        const int b = at.b, c = at.c0 + lane * kV, n = valid_tokens(p, b), tile = p.tiles - 1 - at.at;
        const int last = n > 0 ? (n - 1) / tile_tokens : 0;
        const int count = channels<kBy, kV>(p, c);
        uint2 *here = p.carry + (static_cast<int64_t>(b) * p.tiles + tile) * p.C + c;
        turns.now = ticket;
        unsigned next = 0;
        auto ask = [&] {   // and let the others fetch that tile
            if (lane == 0) {
                next = turns.ask();
                sh.ticket[i & 1] = next;
                mbar_arrive(b_next + 8 * (i & 1));
            }
            next = __shfl_sync(0xffffffffu, next, 0);
        };
        if (i > 0) ask();   // of a CTA's first tile later: other CTAs may not have one yet
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(b_maps, i & 1, kWaits))) {
            give_up(p);
            return;
        }
        if (i == 0) ask();
        if (kBy == kTma && next < turns.total) fetch_tile(next, (i + 1) & 1);   // the gates' rows and that half are read
        if (tile <= last) {
            V pa = L::all(1.f), pd = L::all(0.f), most = pa;   // the tile's map, and the largest product on the way to it
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                const V a = sh.a[i & 1][w][lane];
                pd = L::fma(a, pd, sh.d[w][lane]);
                pa = L::mul(pa, a);
                if (kLog) most = larger(most, pa);
            }
            float in[kV];
            if (tile == last) {
                start<kV>(p, b, c, count, in);
            } else {
                if (tile > 0) tell_map<kV, kPairs>(here, count, parts(pa), parts(pd));
                if (!entering<kV, kPairs, kV == 1 ? 8 : 4>(p, here + p.C, p.C, last - tile, count, in)) give_up(p);
            }
            V e = whole<kV>(in);
            const V out = L::fma(pa, e, pd);
            if (tile > 0) tell_state<kV, kPairs>(here, count, parts(out));
            else finish<kV>(p, b, c, count, parts(out));
            watch<kLog>(p, count, most);
#pragma unroll
            for (int w = kWarps - 1; w >= 0; --w) {
                sh.enter[w][lane] = e;
                e = L::fma(sh.a[i & 1][w][lane], e, sh.d[w][lane]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(b_carry);
        ticket = next;
    }
}

template <typename T, bool kLog, Copies kBy, int kTok, int kWarps, int kCtas>
__global__ void __launch_bounds__(32 * (kWarps + 1), kCtas) scan_bwd_ring_kernel(ScanArgs p, bool wide, const __grid_constant__ Maps maps) {
    using namespace ptx;
    using L = Lane<T, kLog, true>;
    using X = typename std::conditional<Most<T, kLog>::kAsks, Exact, L>::type;
    using V = typename L::V;
    constexpr int kTile = kTok * kWarps, kV = L::kV, kWidth = 32 * kV, kRow = kBy == kOdd ? kOddRow : kEvenRow;
    static_assert(kTile == KLA_SCAN_SPAN, "");
    extern __shared__ __align__(128) uint8_t buf[];   // x and dy twice, gate once: kTile rows each
    __shared__ Shared<V, kWarps> sh;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    Turns turns(p);
    if (p.head) dependency_wait();
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&sh.maps), kWarps);
        mbar_init(smem_u32(&sh.carry), 1);
        mbar_init(smem_u32(&sh.next[0]), 1);
        mbar_init(smem_u32(&sh.next[1]), 1);
        mbar_init(smem_u32(&sh.full[0]), 1);
        mbar_init(smem_u32(&sh.full[1]), 1);
        fence_mbar_init();
        sh.ticket[1] = p.head ? turns.ask() : blockIdx.x;
    }
    __syncthreads();
    unsigned ticket = sh.ticket[1];
    const uint32_t b_full = smem_u32(sh.full);
    auto fetch_tile = [&](unsigned of, int stage) {   // kTma: by one lane of the chain's warp
        const Tile at(p, of, kWidth);
        const int t0 = (p.tiles - 1 - at.at) * kTile;
        const uint32_t bar = b_full + 8 * stage, to = smem_u32(buf);
        if (lane != 0) return;
        if (t0 >= valid_tokens(p, at.b)) {
            mbar_arrive(bar);
            return;
        }
        mbar_arrive_expect_tx(bar, 3 * kTile * kRow);
        load_tile(to + 4 * kTile * kRow, &maps.gate, bar, at.c0, t0, at.b);
        load_tile(to + 2 * stage * kTile * kRow, &maps.x, bar, at.c0, t0, at.b);
        load_tile(to + (2 * stage + 1) * kTile * kRow, &maps.dy, bar, at.c0, t0, at.b);
    };
    if (warp == kWarps) {
        if (kBy == kTma && ticket < turns.total) fetch_tile(ticket, 0);
        carry_warp<L, kLog, kBy, kWarps>(p, sh, turns, ticket, kTile, fetch_tile);
        return;
    }
    const uint32_t b_maps = smem_u32(&sh.maps), b_carry = smem_u32(&sh.carry), b_next = smem_u32(sh.next);
    uint8_t *const mine = buf + warp * kTok * kRow;
    uint8_t *const gates = mine + 4 * kTile * kRow;
    auto fetch = [&](unsigned of, int stage) {
        const Tile at(p, of, kWidth);
        const int t0 = (p.tiles - 1 - at.at) * kTile + warp * kTok, m = min(valid_tokens(p, at.b) - t0, kTok);
        const int left = p.C - at.c0;
        uint8_t *to = mine + 2 * stage * kTile * kRow;
        copy_rows<T, kTok, kBy>(gates, static_cast<const T *>(p.gate) + at.b * p.gb + t0 * p.gt + at.c0, p.gt, m, left,
                                 wide);
        copy_rows<T, kTok, kBy>(to, static_cast<const T *>(p.x) + at.b * p.xb + t0 * p.xt + at.c0, p.xt, m, left, wide);
        copy_rows<T, kTok, kBy>(to + kTile * kRow, static_cast<const T *>(p.dy) + at.b * p.db + t0 * p.dt + at.c0, p.dt,
                                 m, left, wide);
        copies_commit();
    };
    if (kBy != kTma && ticket < turns.total) fetch(ticket, 0);
    for (unsigned turn = 0; ticket < turns.total; ++turn) {
        const Tile at(p, ticket, kWidth);
        const int stage = turn & 1, b = at.b, c = at.c0 + lane * kV, n = valid_tokens(p, b), tile = p.tiles - 1 - at.at;
        const int t0 = tile * kTile + warp * kTok, m = min(max(n - t0, 0), kTok);
        const int count = channels<kBy, kV>(p, c);
        const uint8_t *xs = mine + 2 * stage * kTile * kRow + lane * 4, *ds = xs + kTile * kRow, *gs = gates + lane * 4;
        const Parity<kBy> of_x(static_cast<const T *>(p.x) + b * p.xb + t0 * p.xt + at.c0, p.xt);
        const Parity<kBy> of_g(static_cast<const T *>(p.gate) + b * p.gb + t0 * p.gt + at.c0, p.gt);
        const Parity<kBy> of_d(static_cast<const T *>(p.dy) + b * p.db + t0 * p.dt + at.c0, p.dt);
        V k[kTok], A = L::all(1.f), H = L::all(0.f), D = H, h;
        {
            const float *s = p.states + (static_cast<int64_t>(b) * p.tiles + tile) * p.C + c;
            float in[kV];
#pragma unroll
            for (int v = 0; v < kV; ++v) in[v] = v < count && m > 0 ? s[v] : 0.f;
            h = whole<kV>(in);
        }
        bool ok = true;
        if constexpr (kBy == kTma) {
            ok = mbar_wait_bounded(b_full + 8 * stage, turn >> 1 & 1, kWaits);
        } else {
            copies_wait();
            __syncwarp();
        }
        Most<T, kLog> most;
        auto map_tokens = [&](auto full, auto by) {
            using K = decltype(by);
            A = L::all(1.f);
            H = D = L::all(0.f);
#pragma unroll
            for (int i = 0; i < kTok; ++i)
                if (full || i < m) {
                    k[i] = K::keep(of_g.template load<L>(gs + i * kRow, i));
                    if (std::is_same<K, L>::value) most.see(k[i]);
                    A = K::shrink(A, k[i]);
                    H = K::advance(H, of_x.template load<L>(xs + i * kRow, i), k[i]);
                    D = L::fma(A, of_d.template load<L>(ds + i * kRow, i), D);
                }
        };
        by_case<L, L>(m == kTok, false, map_tokens);
        const bool exact = most.any(count, m, [&](int i) { return of_g.template load<L>(gs + i * kRow, i); });
        if (exact) map_tokens(std::false_type{}, X{});
        if (kLog || exact) A = kept_product<T, kLog>(A, count, m, [&](int i) { return of_g.template load<L>(gs + i * kRow, i); });
        else A = kept_product<L>(A, count, m, k);
        __syncwarp();
        watch<kLog>(p, count, A);
        sh.a[turn & 1][warp][lane] = A;
        sh.h[turn & 1][warp][lane] = H;
        sh.d[warp][lane] = D;
        __syncwarp();
        if (lane == 0) mbar_arrive(b_maps);
        ok = ok && mbar_wait_bounded(b_next + 8 * (turn & 1), turn >> 1 & 1, kWaits);
        const unsigned next = ok ? sh.ticket[turn & 1] : turns.total;
        if (kBy != kTma && next < turns.total) fetch(next, stage ^ 1);
        ok = ok && mbar_wait_bounded(b_maps, turn & 1, kWaits);
        // the states before this warp's tokens, while the chain's are on their way
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w)
            if (w < warp) h = L::fma(sh.a[turn & 1][w][lane], h, sh.h[turn & 1][w][lane]);
        V lead[kTok];   // h_{t-1}, of which the sigmoid's gradient takes x_t
        by_case<L, X>(m == kTok, exact, [&](auto full, auto by) {
            using K = decltype(by);
#pragma unroll
            for (int i = 0; i < kTok; ++i)
                if (full || i < m) {
                    const V x = of_x.template load<L>(xs + i * kRow, i);
                    lead[i] = kLog ? h : L::fma(x, L::all(-1.f), h);
                    h = K::advance(h, x, k[i]);
                }
        });
        ok = ok && mbar_wait_bounded(b_carry, turn & 1, kWaits);
        if (!__all_sync(0xffffffffu, ok)) {   // not before what is on its way here has come
            copies_wait();
            if (kBy == kTma) {
                mbar_wait_bounded(b_full + 8 * stage, turn >> 1 & 1, kWaits);
                mbar_wait_bounded(b_full + 8 * (stage ^ 1), (turn + 1) >> 1 & 1, kWaits);
            }
            give_up(p);
            return;
        }
        if (count > 0) {
            V e = sh.enter[warp][lane];   // what reaches the state behind the token
            const int64_t out = (static_cast<int64_t>(b) * p.T + t0) * p.C + c;
            const Parity<kBy> of_dx(static_cast<T *>(p.y) + out, p.C), of_dg(static_cast<T *>(p.dg) + out, p.C);
            T *dx = static_cast<T *>(p.y) + out + (kTok - 1) * static_cast<int64_t>(p.C);
            T *dg = static_cast<T *>(p.dg) + out + (kTok - 1) * static_cast<int64_t>(p.C);
            by_case<L, X>(m == kTok, exact, [&](auto full, auto by) {
                using K = decltype(by);
#pragma unroll
                for (int i = kTok - 1; i >= 0; --i, dx -= p.C, dg -= p.C)
                    if (full || i < m) {
                        const V dh = L::add(of_d.template load<L>(ds + i * kRow, i), e), w = K::w(k[i]);
                        e = K::reach(dh, k[i]);
                        of_dx.template store<L>(dx, kLog ? dh : L::mul(w, dh), i, count);
                        of_dg.template store<L>(dg, L::mul(kLog ? lead[i] : L::mul(w, lead[i]), e), i, count);
                    } else if (t0 + i < p.T) {
                        of_dx.template store<L>(dx, L::all(0.f), i, count);
                        of_dg.template store<L>(dg, L::all(0.f), i, count);
                    }
            });
        }
        __syncwarp();
        ticket = next;
    }
}

// A workspace that says nothing yet, with the ticket before the first. A kernel of the library, that the scan's CTAs may be
// set up while it runs.
__global__ void __launch_bounds__(256) clear_kernel(uint4 *p, size_t words, unsigned first) {
    dependency_release();
    for (size_t i = blockIdx.x * 256 + threadIdx.x; i < words; i += gridDim.x * 256)
        p[i] = make_uint4(i == 0 ? first - 1u : kEmpty, kEmpty, kEmpty, kEmpty);
}

template <typename T, bool kLog>
__global__ void scan_step_kernel(const T *x, int64_t xs, const T *gate, int64_t gs, float *h, T *y, int C) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
    if (c >= C) return;
    const int64_t at = static_cast<int64_t>(b) * C + c;
    const float u = to_f32(x[b * xs + c]), g = to_f32(gate[b * gs + c]);
    float a, w;
    factors<T, kLog>(gate_exp<T, kLog>(g), a, w);
    float v = advance<kLog>(h[at], u, coefficient<kLog>(a, w));
    // thousands of steps of gates near 0 add up: by the loss there, as `kept_product` does
    if (kLog && fabsf(g) < 0.0625f) v = fmaf(-loss<T, kLog>(g), h[at], h[at] + u);
    h[at] = v;
    y[at] = from_f32<T>(v);
}

int tiles_of(int T, int tile) { return T > tile ? (T + tile - 1) / tile : 1; }

kla_status check(int B, int T, int C, kla_dtype dtype, kla_scan_mode mode) {
    if (B < 1 || T < 0 || C < 1) return KLA_ERR_INVALID_ARG;
    if (dtype != KLA_DTYPE_F32 && dtype != KLA_DTYPE_BF16) return KLA_ERR_INVALID_ARG;
    if (mode != KLA_SCAN_SIGMOID && mode != KLA_SCAN_LOG) return KLA_ERR_INVALID_ARG;
    if (T > INT_MAX - 65536 || C > INT_MAX - 65536 || B > 65535) return KLA_ERR_UNSUPPORTED;
    // a ticket for every tile of 32 channels
    if (static_cast<int64_t>(B) * ((C + 31) / 32) > INT_MAX / tiles_of(T, KLA_SCAN_SPAN)) return KLA_ERR_UNSUPPORTED;
    return KLA_OK;
}

// Bytes from a strided tensor's start to its last element's end.
size_t reach(int B, int T, int C, int64_t sb, int64_t st, size_t esz) {
    return T == 0 ? 0 : (static_cast<size_t>(B - 1) * sb + static_cast<size_t>(T - 1) * st + C) * esz;
}

// Bytes of the words between tiles of `tile` tokens, and in front of them the tickets.
size_t carry_bytes(int B, int T, int C, int tile) {
    const int tiles = tiles_of(T, tile);
    return tiles == 1 ? 0 : sizeof(Head) + (static_cast<size_t>(B) * tiles * C * sizeof(uint2) + 15) / 16 * 16;
}

// Whether every row starts on `bytes` bytes and has a multiple of them.
bool rows_fit(const ScanArgs &p, size_t esz, int bytes) {
    for (const void *a : {p.x, p.gate, p.dy, static_cast<const void *>(p.y), static_cast<const void *>(p.dg)})
        if (!aligned(a, bytes)) return false;
    return (p.C | p.xb | p.xt | p.gb | p.gt | p.db | p.dt) % (bytes / static_cast<int>(esz)) == 0;
}

// Sets up the tiles of 32 kV channels and `tile` tokens, and what they tell each other.
cudaError_t lay_out(ScanArgs &p, int tile, int width, void *workspace, cudaStream_t s) {
    p.blocks = (p.C + width - 1) / width;
    p.tiles = tiles_of(p.T, tile);
    const cudaError_t e = device_error_word(&p.err);
    if (e != cudaSuccess || p.tiles == 1) return e;
    p.head = static_cast<Head *>(workspace);
    p.carry = reinterpret_cast<uint2 *>(p.head + 1);
    const size_t words = carry_bytes(p.B, p.T, p.C, tile) / sizeof(uint4), ctas = (words + 1023) / 1024;
    clear_kernel<<<static_cast<unsigned>(ctas < 608 ? ctas : 608), 256, 0, s>>>(static_cast<uint4 *>(workspace), words, p.first);
    return cudaGetLastError();
}
unsigned tiles_in_all(const ScanArgs &p) { return static_cast<unsigned>(p.B) * p.blocks * p.tiles; }
// CTAs of a kernel that takes one ticket each
unsigned tickets(const ScanArgs &p) { return tiles_in_all(p) - (p.head ? p.first : 0); }

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = []() -> EncodeTiledFn {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}
// A strided [B, T, C] tensor; box = 128 bytes of channels x `tokens` tokens of one sequence.
bool make_map(CUtensorMap *m, const void *base, int64_t sb, int64_t st, const ScanArgs &p, size_t esz, int tokens) {
    const EncodeTiledFn fn = encode_fn();
    constexpr int64_t kMost = int64_t(1) << 38;   // of a stride in bytes: 2^40
    if (!fn || st <= 0 || st > kMost || (p.B > 1 && (sb <= 0 || sb > kMost))) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(p.C), static_cast<cuuint64_t>(p.T), static_cast<cuuint64_t>(p.B)};
    // the stride of an axis of one element is never used
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(st) * esz, p.B > 1 ? static_cast<cuuint64_t>(sb) * esz : 256};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(kEvenRow / esz), static_cast<cuuint32_t>(tokens), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, esz == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(base),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// By tensor maps where rows fit 16 bytes, none is broadcast, and there are tiles enough for the maps' making (a
// microsecond of the host's) to be worth it: more than the SMs take at once. 8 x 4096 x 2048 by the warps' copies and by
// maps: forward 79 and 72 us, backward 120 and 111; fp32 8 x 2048 x 2048 97 and 85, 146 and 130.
bool by_maps(Maps &m, const ScanArgs &p, bool wide, size_t esz, int tile, int ctas) {
    if (!wide || tiles_in_all(p) <= 152u * ctas) return false;
    return make_map(&m.x, p.x, p.xb, p.xt, p, esz, tile) && make_map(&m.gate, p.gate, p.gb, p.gt, p, esz, tile) &&
           (!p.dy || make_map(&m.dy, p.dy, p.db, p.dt, p, esz, tile));
}

// kBuffers of `tile` rows a CTA; as many CTAs as the SMs hold at once.
template <int kBuffers, int kCtas, auto kKernel>
cudaError_t run_ring(const ScanArgs &p, bool wide, const Maps &maps, int row, int tile, int block, cudaStream_t s) {
    constexpr int kMaxDevices = 64, kSms = 152;
    static std::atomic<bool> done[kMaxDevices];
    const int smem = kBuffers * tile * row;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!done[dev].load(std::memory_order_acquire)) {   // once per device and kernel
        if ((e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess)
            return e;
        done[dev].store(true, std::memory_order_release);
    }
    const unsigned most = kCtas * kSms, tiles = tiles_in_all(p);
    const unsigned grid = tiles < most ? tiles : most;
    if (p.head) return launch_dependent(kKernel, dim3(grid), dim3(block), smem, s, p, wide, maps);
    kKernel<<<grid, block, smem, s>>>(p, wide, maps);
    return cudaGetLastError();
}

template <typename F>
cudaError_t by_type(kla_dtype dtype, kla_scan_mode mode, F f) {
    if (dtype == KLA_DTYPE_BF16)
        return mode == KLA_SCAN_LOG ? f(__nv_bfloat16{}, std::true_type{}) : f(__nv_bfloat16{}, std::false_type{});
    return mode == KLA_SCAN_LOG ? f(float{}, std::true_type{}) : f(float{}, std::false_type{});
}

// What the self-test sets otherwise: a first ticket of 1 leaves out the tile that all others of its chain wait for.
struct Trial {
    unsigned first, polls;
};
constexpr Trial kInEarnest{0, kPolls};

}  // namespace
}  // namespace kla

extern "C" size_t kla_gated_scan_workspace_size(int B, int T, int C, kla_dtype dtype) {
    using namespace kla;
    if (check(B, T, C, dtype, KLA_SCAN_SIGMOID) != KLA_OK) return 0;
    return carry_bytes(B, T, C, KLA_SCAN_SPAN);   // no kernel has a shorter tile
}

namespace kla {
namespace {

kla_status scan_fwd(const void *x, const void *gate, const int64_t *strides, const int *lengths,
                              const float *h0, void *y, float *h_T, float *states, int B, int T, int C,
                              kla_dtype dtype, kla_scan_mode mode, void *workspace, size_t workspace_bytes,
                              void *stream, Trial trial) {
    const kla_status st = check(B, T, C, dtype, mode);
    if (st != KLA_OK) return st;
    if (T > 0 && (!x || !gate || !y)) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x, esz) || !aligned(gate, esz) || !aligned(y, esz) || !aligned(lengths, 4) || !aligned(h0, 4) ||
        !aligned(h_T, 4) || !aligned(states, 4) || !aligned(workspace, 16))
        return KLA_ERR_INVALID_ARG;
    const int64_t tc = static_cast<int64_t>(T) * C;
    ScanArgs p{x, gate, nullptr, tc, C, tc, C, 0, 0, lengths, h0, y, nullptr, h_T, states, B, T, C,
               0, 0, nullptr, nullptr, nullptr, trial.first, trial.polls};
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
    const bool even = rows_fit(p, esz, 4), wide = rows_fit(p, esz, 16);
    const bool ring = even || (aligned(x, 4) && aligned(gate, 4));
    if (lay_out(p, fwd_shape(static_cast<int>(esz), ring).tile(), ring ? kEvenRow / static_cast<int>(esz) : 32, workspace, cs) != cudaSuccess)
        return KLA_ERR_CUDA;
    const cudaError_t e = by_type(dtype, mode, [&](auto t, auto log) {
        using E = decltype(t);
        constexpr bool kLog = decltype(log)::value;
        constexpr Shape r = fwd_shape(sizeof(E), true), o = fwd_shape(sizeof(E), false);
        static_assert(r.tile() % KLA_SCAN_SPAN == 0 && o.tile() % KLA_SCAN_SPAN == 0 && KLA_SCAN_SPAN % r.tok == 0, "");
        Maps maps{};
        if (even && by_maps(maps, p, wide, esz, r.tile(), r.ctas))
            return run_ring<3, r.ctas, scan_fwd_ring_kernel<E, kLog, kTma, r.tok, r.warps, r.ctas>>(
                p, wide, maps, kEvenRow, r.tile(), 32 * r.warps, cs);
        if (even)
            return run_ring<3, r.ctas, scan_fwd_ring_kernel<E, kLog, kEven, r.tok, r.warps, r.ctas>>(
                p, wide, maps, kEvenRow, r.tile(), 32 * r.warps, cs);
        if constexpr (sizeof(E) == 2) {
            if (ring)
                return run_ring<3, r.ctas, scan_fwd_ring_kernel<E, kLog, kOdd, r.tok, r.warps, r.ctas>>(
                    p, false, maps, kOddRow, r.tile(), 32 * r.warps, cs);
            scan_fwd_kernel<E, kLog, o.tok, o.warps><<<tickets(p), 32 * o.warps, 0, cs>>>(p);
        }
        return cudaGetLastError();
    });
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

kla_status scan_bwd(const void *x, const void *gate, const void *dy, const int64_t *strides,
                              const int *lengths, const float *states, const float *dh_T, void *dx, void *dgate,
                              float *dh0, int B, int T, int C, kla_dtype dtype, kla_scan_mode mode, void *workspace,
                              size_t workspace_bytes, void *stream, Trial trial) {
    const kla_status st = check(B, T, C, dtype, mode);
    if (st != KLA_OK) return st;
    if (T > 0 && (!x || !gate || !dy || !dx || !dgate || !states)) return KLA_ERR_INVALID_ARG;
    const size_t esz = dtype == KLA_DTYPE_BF16 ? 2 : 4;
    if (!aligned(x, esz) || !aligned(gate, esz) || !aligned(dy, esz) || !aligned(dx, esz) || !aligned(dgate, esz) ||
        !aligned(lengths, 4) || !aligned(states, 4) || !aligned(dh_T, 4) || !aligned(dh0, 4) ||
        !aligned(workspace, 16))
        return KLA_ERR_INVALID_ARG;
    const int64_t tc = static_cast<int64_t>(T) * C;
    ScanArgs p{x, gate, dy, tc, C, tc, C, tc, C, lengths, dh_T, dx, dgate, dh0, const_cast<float *>(states), B, T, C,
               0, 0, nullptr, nullptr, nullptr, trial.first, trial.polls};
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
    const bool even = rows_fit(p, esz, 4), wide = rows_fit(p, esz, 16);
    const bool ring = even || (aligned(x, 4) && aligned(gate, 4) && aligned(dy, 4));
    if (lay_out(p, bwd_shape().tile(), ring ? kEvenRow / static_cast<int>(esz) : 32, workspace, cs) != cudaSuccess)
        return KLA_ERR_CUDA;
    const cudaError_t e = by_type(dtype, mode, [&](auto t, auto log) {
        using E = decltype(t);
        constexpr bool kLog = decltype(log)::value;
        constexpr Shape r = bwd_shape(), o = r;
        static_assert(r.tile() % KLA_SCAN_SPAN == 0 && o.tile() % KLA_SCAN_SPAN == 0 && KLA_SCAN_SPAN % r.tok == 0, "");
        Maps maps{};
        if (even && by_maps(maps, p, wide, esz, r.tile(), r.ctas))
            return run_ring<5, r.ctas, scan_bwd_ring_kernel<E, kLog, kTma, r.tok, r.warps, r.ctas>>(
                p, wide, maps, kEvenRow, r.tile(), 32 * (r.warps + 1), cs);
        if (even)
            return run_ring<5, r.ctas, scan_bwd_ring_kernel<E, kLog, kEven, r.tok, r.warps, r.ctas>>(
                p, wide, maps, kEvenRow, r.tile(), 32 * (r.warps + 1), cs);
        if constexpr (sizeof(E) == 2) {
            if (ring)
                return run_ring<5, r.ctas, scan_bwd_ring_kernel<E, kLog, kOdd, r.tok, r.warps, r.ctas>>(
                    p, false, maps, kOddRow, r.tile(), 32 * (r.warps + 1), cs);
            scan_bwd_kernel<E, kLog, o.tok, o.warps><<<tickets(p), 32 * o.warps, 0, cs>>>(p);
        }
        return cudaGetLastError();
    });
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // namespace
}  // namespace kla

extern "C" {

kla_status kla_gated_scan_fwd(const void *x, const void *gate, const int64_t *strides, const int *lengths,
                              const float *h0, void *y, float *h_T, float *states, int B, int T, int C,
                              kla_dtype dtype, kla_scan_mode mode, void *workspace, size_t workspace_bytes,
                              void *stream) {
    return kla::scan_fwd(x, gate, strides, lengths, h0, y, h_T, states, B, T, C, dtype, mode, workspace,
                         workspace_bytes, stream, kla::kInEarnest);
}

kla_status kla_gated_scan_bwd(const void *x, const void *gate, const void *dy, const int64_t *strides,
                              const int *lengths, const float *states, const float *dh_T, void *dx, void *dgate,
                              float *dh0, int B, int T, int C, kla_dtype dtype, kla_scan_mode mode, void *workspace,
                              size_t workspace_bytes, void *stream) {
    return kla::scan_bwd(x, gate, dy, strides, lengths, states, dh_T, dx, dgate, dh0, B, T, C, dtype, mode, workspace,
                         workspace_bytes, stream, kla::kInEarnest);
}

kla_status kla_selftest_scan_timeout(unsigned limit_polls, int backward, const void *x, float *states, void *out,
                                     void *out2, int B, int T, int C, kla_dtype dtype, void *workspace,
                                     size_t workspace_bytes, void *stream) {
    using namespace kla;
    if (limit_polls < 1 || limit_polls > kPolls) return KLA_ERR_INVALID_ARG;
    const kla_status st = check(B, T, C, dtype, KLA_SCAN_SIGMOID);
    if (st != KLA_OK) return st;
    if (tiles_of(T, fwd_shape(2, true).tile()) < 2) return KLA_ERR_INVALID_ARG;   // nothing would wait
    const Trial trial{1, limit_polls};
    if (backward)
        return scan_bwd(x, x, x, nullptr, nullptr, states, nullptr, out, out2, nullptr, B, T, C, dtype,
                        KLA_SCAN_SIGMOID, workspace, workspace_bytes, stream, trial);
    return scan_fwd(x, x, nullptr, nullptr, nullptr, out, nullptr, states, B, T, C, dtype, KLA_SCAN_SIGMOID, workspace,
                    workspace_bytes, stream, trial);
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
        return cudaGetLastError();
    });
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // extern "C"
