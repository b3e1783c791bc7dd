// kla_linear_tc.cu -- tensor-core (tcgen05) scan of the decayed linear attention for sm_103a.
//
// Scope: bf16, dx = dz = 128, chunks of C = 128 tokens, fp32 state; see kla_linear.cuh for the roles
// x, y, z and the four directions. Per chunk with n valid tokens and entering state S (dx x dz):
//   D = X Y^T                         -> P_ij = a_intra g^{|i-j|} D_ij on the mask's side, else 0
//   O = diag(r) X S,  O += P Z        r_i = a_inter g^{i+1} (against time: a_inter g^{n-1-i})
//   U = (diag(w) Y)^T Z               w_j = a_upd g^{n-1-j} (against time: a_upd g^{j+1})
//   S <- g^n S + U
// No power of g has a negative exponent, so nothing overflows for any g in [0, 1]. U does not depend
// on S: the only chain from chunk to chunk is one fp32 multiply-add per state element.
//
// One CTA per (sequence, head, segment) walks its chunks; all products are M = N = 128 on tcgen05:
//   D   A = X (smem, K-major)         B = Y (smem, K-major)
//   O   A = X (smem, K-major)         B = S (bf16, smem, MN-major)
//   O   A = P (TMEM, over D)          B = Z (smem, MN-major)
//   U   A = (diag(w) Y)^T (TMEM)      B = Z (smem, MN-major)
// Operands that threads compute and that would be read from shared memory once per product sit in
// TMEM instead: P replaces D column by column, and the weighted keys are written transposed. So does
// the fp32 state: U accumulates onto g^n S in place.
// (diag(w) Y)^T is kept as two bf16 terms (hi + lo, up to 2^-16 off, a third of that on average): the fp32 state
// is an output of its own, and one term (2^-8) would be its error. S as an operand and P are rounded to one bf16
// term: they only enter O, which is stored with 8 bits itself. Against 64 bits O is off by 2.3e-3 (its own
// rounding alone: 1.7e-3) and the state by 4e-6 (dS0 of a few tokens, whose weights share one error, by 7e-6, up
// to 1.1e-5); a third term of the keys took the 4096-token prompt below from 94 to 136 us. Weighing in fp32 and
// splitting the product leaves 2.5e-6, for 2 % more time there and 4 % more on 131072 tokens: not taken.
//
// Warps: 0-7 turn D into P; 8-15 copy and decay the state, scale the first half of O and send the
// outputs out through the Z tile; 16-23 weigh the keys; 24 loads (TMA, two stages of X, Y, Z tiles, each
// tile refilled as soon as its own readers are done: Y first, Z, which is needed last, last);
// 25 issues the products, in the order D, X S, U, P Z, which leaves P's conversion the time of X S
// and U. They hand over through mbarriers that complete once per chunk, on which whole warps wait and give up
// as one (the votes that this takes cost 0.5 to 1 %). Eight warps per role: with four, and keys and state on the
// same eight, the chain of conversions took 6900 cycles a chunk.
//
// Measured, 16 heads: outputs of 8 x 4096 tokens 92 us (537 MB, 5.8 TB/s, 86 % of a copy's rate, the tensor pipe
// active in 49 % of the cycles): the memory. The three scans of that shape's backward pass 250 us: 384 CTAs go
// over 152 SMs in three rounds of 32 chunks, so ~2.6 us a chunk, where the memory's share would be ~1.9 (1.22 GB of
// traffic); by count ~3900 of a chunk's ~5000 cycles move operands and tiles through shared memory. The states
// of 131072 tokens in eight segments 148 us (6.4 TB/s), their outputs 320 us (6.7 TB/s).
#include <cuda.h>

#include <atomic>

#include "kla_linear.cuh"
#include "warp_mma.cuh"

namespace kla {
namespace {

using namespace ptx;

constexpr int kC = 128, kD = 128;
constexpr int kThreads = 26 * 32;
constexpr uint32_t kWaitLimit = 100000;   // x 20 us: a stuck wait gives up after ~2 s
constexpr uint32_t kTile = 32768, kHalf = 16384;   // a 128 x 128 bf16 tile: two blocks of 64 channels
constexpr uint32_t OFF_S = 6 * kTile;   // after two stages of X, Y, Z tiles, or three of Y, Z
constexpr uint32_t OFF_SMALL = OFF_S + kTile;
constexpr uint32_t SMEM_BYTES = OFF_SMALL + 2048 + 1024;   // + alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory");
constexpr uint32_t TM_D = 0, TM_P = 0, TM_O = 128, TM_U = 256, TM_YH = 384;   // keys: hi, then lo 64 columns on

struct Small {
    // by stage: a tile has landed, and may be filled again
    uint64_t fy[3], yfree[3];   // Y: D is computed and the keys are weighed
    uint64_t fx[2], xfree[2];   // X: X S is computed
    uint64_t fz[3], zfree[3];   // Z: U and P Z are computed; the outputs, which leave through it, are out
    uint64_t end;       // after an abort: the products that were issued are done
    uint64_t d, p;      // D computed, P written
    uint64_t xs, sc;    // X S computed, scaled
    uint64_t o, ord;    // O computed, O read
    uint64_t y, u;      // weighted keys written, U added
    uint64_t s;         // operand copy of S written, S decayed
    uint32_t tmem_base;
    volatile int abort;
    float gp[kC + 1];              // g^0 .. g^128
    float diag[64];                // a_intra g^distance at 32 + column - row of a diagonal 32 x 32 block, 0 off the mask
    uint32_t keep[64];             // the mask of that column and its right neighbour, as bf16 pairs
    alignas(16) float near[32];    // g^distance of a block's columns from its side near the diagonal
};
static_assert(sizeof(Small) <= 2048, "small area");

struct Job {
    CUtensorMap x, y, z, o;
    LinScan p;
};
struct TcParams {
    Job job[3];
    int scans, first_seg, states;
    unsigned *err;
};

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

template <bool kStates>   // only the segment's own contribution to the state
__global__ void __launch_bounds__(kThreads, 1) lin_tc_kernel(const __grid_constant__ TcParams tp) {
    const Job &job = tp.job[blockIdx.x % tp.scans];
    const LinScan &p = job.p;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    Small &sm = *reinterpret_cast<Small *>(smem + OFF_SMALL);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = (warp & 3) * 32 + lane;   // TMEM lane of this thread
    const int chain = blockIdx.x / tp.scans, b = chain / p.H, h = chain % p.H, seg = blockIdx.y;
    const int n = lin_length(p.lengths, b, p.T);
    int t_begin;
    const int valid = lin_segment(p, seg, n, t_begin);
    const int t_stop = min(p.T, t_begin + p.seg_len);
    const int nchunk = (valid + kC - 1) / kC;
    const float g = p.decay[h];
    const bool have = !kStates && (seg > 0 || p.S0 != nullptr);   // S is not zero at the start
    const bool want_s = kStates || (p.ST && seg == p.nseg - 1);

    const uint32_t b_fy = smem_u32(&sm.fy[0]), b_fx = smem_u32(&sm.fx[0]), b_fz = smem_u32(&sm.fz[0]);
    const uint32_t b_yfree = smem_u32(&sm.yfree[0]), b_xfree = smem_u32(&sm.xfree[0]);
    const uint32_t b_zfree = smem_u32(&sm.zfree[0]), b_end = smem_u32(&sm.end);
    const uint32_t b_d = smem_u32(&sm.d), b_p = smem_u32(&sm.p), b_xs = smem_u32(&sm.xs), b_sc = smem_u32(&sm.sc);
    const uint32_t b_o = smem_u32(&sm.o), b_ord = smem_u32(&sm.ord), b_y = smem_u32(&sm.y), b_u = smem_u32(&sm.u);
    const uint32_t b_s = smem_u32(&sm.s);
    const bool back = p.reverse;
    auto chunk_of = [&](int c) { return back ? nchunk - 1 - c : c; };
    auto count_of = [&](int c) { return min(kC, valid - chunk_of(c) * kC); };
    // stages: two of X, Y, Z tiles, or three of Y, Z where only the state is wanted
    constexpr int kNs = kStates ? 3 : 2;
    constexpr uint32_t kY = kStates ? 0 : kTile, kZt = kY + kTile;
    // Where only the state is wanted, the columns of D hold a second set of weighted keys, so that those of
    // the next chunk are written while this chunk's product runs; each set has barriers of its own.
    auto keys_at = [&](int c) { return kStates && (c & 1) ? TM_D : TM_YH; };
    auto keys_ready = [&](int c) { return kStates && (c & 1) ? b_p : b_y; };
    auto keys_phase = [&](int c) { return kStates ? c >> 1 : c; };
    auto stage_of = [&](int c) { return sbase + (c % kNs) * (kZt + kTile); };
    auto load = [&](const CUtensorMap &map, uint32_t tile, uint32_t full, int c) {   // one thread
        const uint32_t to = stage_of(c) + tile, bar = full + 8 * (c % kNs);
        const int t0 = t_begin + chunk_of(c) * kC;
        mbar_arrive_expect_tx(bar, kTile);
        for (int i = 0; i < 2; ++i) tma_load_4d(to + i * kHalf, &map, bar, 64 * i, h, t0, b);
    };
    if (warp == 24 && lane == 0) {   // the first loads leave before the rest of the CTA is set up
        for (int i = 0; i < kNs; ++i) {
            mbar_init(b_fy + 8 * i, 1);
            mbar_init(b_fz + 8 * i, 1);
            mbar_init(b_yfree + 8 * i, kStates ? 8 : 9);   // the warps that weigh, and the product D
            if (i < 2) {
                mbar_init(b_fx + 8 * i, 1);
                mbar_init(b_xfree + 8 * i, 1);
            }
            mbar_init(b_zfree + 8 * i, kStates ? 1 : 8);   // the products, or the warps that send O out
        }
        mbar_init(b_end, 1);
        mbar_init(b_d, 1);
        mbar_init(b_p, 8);
        mbar_init(b_xs, 1);
        mbar_init(b_sc, 8);
        mbar_init(b_o, 1);
        mbar_init(b_ord, 8);
        mbar_init(b_y, 8);
        mbar_init(b_u, 1);
        mbar_init(b_s, 8);
        sm.abort = 0;
        fence_mbar_init();
        for (int c = 0; c < kNs && c < nchunk; ++c) {
            load(job.y, kY, b_fy, c);
            if (!kStates) load(job.x, 0, b_fx, c);
            load(job.z, kZt, b_fz, c);
        }
    }
    dependency_release();
    if (tid <= kC) sm.gp[tid] = powf(g, static_cast<float>(tid));
    if (tid < 64) {
        const int dist = p.reverse ? tid - 32 : 32 - tid;
        sm.diag[tid] = dist >= 0 ? p.a_intra * powf(g, static_cast<float>(dist)) : 0.f;
        const int next = p.reverse ? dist + 1 : dist - 1;
        sm.keep[tid] = (dist >= 0 ? 0xFFFFu : 0u) | (next >= 0 ? 0xFFFF0000u : 0u);
        if (tid < 32) sm.near[tid] = powf(g, static_cast<float>(p.reverse ? tid : 31 - tid));
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&sm.tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    dependency_wait();   // the start states; inputs were there before the call's first launch
    const uint32_t tbase = sm.tmem_base;
    const uint32_t tlane = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16);

    // False once any wait of the CTA has given up: every loop then ends. By whole warps.
    auto wait = [&](uint32_t bar, int phase) { return warp_wait(bar, phase & 1, kWaitLimit, &sm.abort); };
    auto wait_alone = [&](uint32_t bar, int phase) {   // one thread, with nobody to agree with
        for (uint32_t i = 0; i < kWaitLimit; ++i) {
            if (mbar_try_wait_sleep(bar, phase & 1, 20000u)) return true;
            if (sm.abort) return false;
        }
        sm.abort = 1;
        return false;
    };
    auto arrive = [&](uint32_t bar) {   // one arrival for the warp
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    // warps 8-15: O of chunk c leaves through the Z tile, the last that its products read and the last that
    // the next chunk needs; each warp's 32 rows x 64 channels are one box, and rows past T are cut off by the
    // tensor's bounds
    auto put_out = [&](int c) {
        const int half = (warp - 8) >> 2, cnt = count_of(c);
        const uint32_t tile = stage_of(c) + kZt + half * kHalf;
        tc_fence_after();
        uint32_t pk[32];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t r[32];
            tmem_ld32(tlane + TM_O + 64 * half + 32 * k, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                pk[16 * k + i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        }
        tc_fence_before();
        arrive(b_ord);   // the next X S may go: shared memory, which the products keep busy, comes after
        if (row >= cnt)  // masked: zero whatever the products left
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            st_shared_v4(tile + sw128_off(row, 16 * i), pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            const int t = t_begin + chunk_of(c) * kC + 32 * (warp & 3);
            if (t < p.T) tma_store_4d(&job.o, tile + (warp & 3) * 4096, 64 * half, h, t, b);
            tma_store_commit();
            tma_store_wait_read_all();
            mbar_arrive(b_zfree + 8 * (c % kNs));
        }
        __syncwarp();
    };

    if (warp == 24) {
        // ---------------------------------------------------------------- loads
        if (lane == 0) {
            int last[3] = {nchunk, nchunk, nchunk};   // loads issued of each kind
            for (int c = kNs; c < nchunk; ++c) {
                const int before = c / kNs - 1, at = 8 * (c % kNs);
                last[0] = last[1] = last[2] = c;
                if (!wait_alone(b_yfree + at, before)) break;
                load(job.y, kY, b_fy, c);
                last[0] = c + 1;
                if (!kStates) {
                    if (!wait_alone(b_xfree + at, before)) break;
                    load(job.x, 0, b_fx, c);
                    last[1] = c + 1;
                }
                if (!wait_alone(b_zfree + at, before)) break;
                load(job.z, kZt, b_fz, c);
                last[2] = c + 1;
            }
            // nothing of this CTA's may be in flight when it ends, an abort included
            for (int i = 0; i < 3; ++i)
                for (int c = max(0, last[i] - kNs); c < last[i]; ++c)
                    if (i != 1 || !kStates)
                        mbar_wait_bounded((i == 0 ? b_fy : i == 1 ? b_fx : b_fz) + 8 * (c % kNs), (c / kNs) & 1,
                                          kWaitLimit);
        }
    } else if (warp == 25) {
        // ---------------------------------------------------------------- products
        const bool lead = elect_one();
        const uint32_t id_kk = idesc_bf16(128, 128, 0, 0), id_km = idesc_bf16(128, 128, 0, 1);
        const uint64_t ds = sw128_desc(sbase + OFF_S, kHalf, 1024);
        for (int c = 0; c < nchunk; ++c) {
            const uint32_t st = stage_of(c), at = 8 * (c % kNs);
            const uint64_t dx = sw128_desc(st, 16, 1024), dy = sw128_desc(st + kY, 16, 1024);
            const uint64_t dz = sw128_desc(st + kZt, kHalf, 1024);
            const bool update = c < nchunk - 1 || want_s;
            const bool inter = !kStates && (c > 0 || have);
            if (!kStates) {
                if (!wait(b_fy + at, c / kNs) || !wait(b_fx + at, c / kNs)) break;
                if (c > 0 && !wait(b_o, c - 1)) break;   // P of the last chunk, which lies over D, is done with
                tc_fence_after();
                if (lead) {
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t off = (s >> 2) * kHalf + (s & 3) * 32;
                        mma_bf16(tbase + TM_D, desc_add(dx, off), desc_add(dy, off), id_kk, s);
                    }
                    mma_commit(b_d);
                    mma_commit(b_yfree + at);
                }
            }
            if (!wait(b_s, c)) break;
            if (!kStates) {
                if (c > 0 && !wait(b_ord, c - 1)) break;
                tc_fence_after();
                if (lead) {
                    if (inter) {
#pragma unroll
                        for (int s = 0; s < 8; ++s)
                            mma_bf16(tbase + TM_O, desc_add(dx, (s >> 2) * kHalf + (s & 3) * 32),
                                     desc_add(ds, s * 2048), id_km, s);
                    }
                    mma_commit(b_xs);
                    mma_commit(b_xfree + at);
                }
            }
            if (!wait(b_fz + at, c / kNs) || !wait(keys_ready(c), keys_phase(c))) break;
            tc_fence_after();
            if (lead) {
                const uint32_t keys = tbase + keys_at(c);
                if (update) {
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_bf16_ta(tbase + TM_U, keys + 8 * s, desc_add(dz, s * 2048), id_km, c > 0 || have || s > 0);
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_bf16_ta(tbase + TM_U, keys + 64 + 8 * s, desc_add(dz, s * 2048), id_km, 1);
                }
                mma_commit(b_u);
                if (kStates) {
                    mma_commit(b_zfree + at);
                    mma_commit(b_xfree + 8 * (c & 1));   // this set of keys is read
                }
            }
            __syncwarp();
            if (kStates) continue;
            if (!wait(b_p, c) || !wait(b_sc, c)) break;
            tc_fence_after();
            if (lead) {
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_bf16_ta(tbase + TM_O, tbase + TM_P + 64 * (s >> 2) + 8 * (s & 3),
                                desc_add(dz, s * 2048), id_km, inter || s > 0);
                mma_commit(b_o);
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        // ---------------------------------------------------------------- D -> P
        const int w = warp & 3, half = warp >> 2;   // rows 32 w .., columns 64 half ..
        const bool reverse = p.reverse;
        const float a_intra = p.a_intra;
        const float *diag = sm.diag + 32 - lane;
        const uint32_t *keep = sm.keep + 32 - lane;
        for (int c = 0; !kStates && c < nchunk; ++c) {
            const int cnt = count_of(c);
            if (!wait(b_d, c)) break;
            tc_fence_after();
            // ascending: P's columns lie over columns of D already read
#pragma unroll 1
            for (int k = 2 * half; k < 2 * half + 2; ++k) {
                uint32_t pk[16];
                if (reverse ? k < w : k > w) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) pk[i] = 0u;
                } else {
                    uint32_t r[32];
                    tmem_ld32(tlane + TM_D + 32 * k, r);
                    tmem_ld_wait();
                    const float2 *d2 = reinterpret_cast<const float2 *>(r);
                    if (k == w) {   // the diagonal block: every distance from the table
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 v = mul2(make_float2(diag[2 * i], diag[2 * i + 1]), d2[i]);
                            // off the mask the table's 0 would leave NaN where D overflows
                            pk[i] = pack_bf16(v.x, v.y) & keep[2 * i];
                        }
                    } else {        // distance to the block's near side times distance within the block
                        const float2 f = both(a_intra * sm.gp[reverse ? 32 * k - row : row - 32 * k - 31]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 e = *reinterpret_cast<const float4 *>(&sm.near[4 * i]);
                            const float2 v0 = mul2(mul2(make_float2(e.x, e.y), f), d2[2 * i]);
                            const float2 v1 = mul2(mul2(make_float2(e.z, e.w), f), d2[2 * i + 1]);
                            pk[2 * i] = pack_bf16(v0.x, v0.y);
                            pk[2 * i + 1] = pack_bf16(v1.x, v1.y);
                        }
                    }
                    if (32 * k + 32 > cnt) {   // masked tokens: whatever D holds there, P is zero
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            if (32 * k + 2 * i >= cnt) pk[i] = 0u;
                            else if (32 * k + 2 * i + 1 >= cnt) pk[i] &= 0xFFFFu;
                        }
                    }
                }
                tmem_st16(tlane + TM_P + 64 * half + 16 * (k & 1), pk);
            }
            tmem_st_wait();
            tc_fence_before();
            arrive(b_p);
        }
    } else if (warp < 16) {
        // ---------------------------------------------------------------- S and O
        const int half = (warp - 8) >> 2, T = p.T;   // columns 64 half ..
        const bool reverse = p.reverse;
        const float a_inter = p.a_inter;
        const size_t sdd = static_cast<size_t>(kD) * kD;
        const float *src = !have ? nullptr
                           : p.nseg > 1 ? p.seg_states + lin_slot(p, chain, lin_start_slot(p, seg))
                                        : p.S0 + chain * sdd;
        const bool src_t = p.nseg > 1 || p.s_t;   // [z][d]: a warp's lanes are neighbours; the scratch is kept so
        float *dst = !want_s ? nullptr
                     : kStates ? p.seg_states + lin_slot(p, chain, seg)
                               : p.ST + chain * sdd;
        const bool dst_t = kStates || p.s_t;
        auto get = [&](uint32_t (&r)[32], int z) {   // 32 z channels from z of this thread's x channel
            if (src_t) {
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(src[(z + i) * kD + row]);
            } else if ((reinterpret_cast<uintptr_t>(src) & 31) == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) ld_global_v8(src + row * kD + z + 8 * i, r + 8 * i);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + row * kD + z + 4 * i);
                    r[4 * i] = v.x;
                    r[4 * i + 1] = v.y;
                    r[4 * i + 2] = v.z;
                    r[4 * i + 3] = v.w;
                }
            }
        };
        const uint32_t t_s = tlane + TM_U + 64 * half;
        const uint32_t copy = sbase + OFF_S + half * kHalf;
        if (have || (want_s && nchunk == 0)) {   // the start state; the first U replaces it where it is zero
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                uint32_t r[32];
                if (have) {
                    get(r, 64 * half + 32 * k);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = 0u;
                }
                tmem_st32(t_s + 32 * k, r);
            }
            tmem_st_wait();
        }

        for (int c = 0; c < nchunk; ++c) {
            const int cnt = count_of(c);
            const bool update = c < nchunk - 1 || want_s;
            if (c > 0 && !wait(b_u, c - 1)) break;   // X S of the last chunk, issued before U, is done as well
            tc_fence_after();
            if (c > 0 || have) {
                const float gn = sm.gp[cnt];
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    uint32_t r[32];
                    tmem_ld32(t_s + 32 * k, r);
                    tmem_ld_wait();
                    if (!kStates) {   // operand copy: row = x channel, 128-byte swizzled rows of 64 z channels
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t pk[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                pk[u] = pack_bf16(__uint_as_float(r[8 * i + 2 * u]),
                                                  __uint_as_float(r[8 * i + 2 * u + 1]));
                            st_shared_v4(copy + sw128_off(row, 64 * k + 16 * i), pk[0], pk[1], pk[2], pk[3]);
                        }
                    }
                    if (update) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 &v = reinterpret_cast<float2 *>(r)[i];
                            v = mul2(v, both(gn));
                        }
                        tmem_st32(t_s + 32 * k, r);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                fence_proxy_async_smem();
            }
            arrive(b_s);
            if (kStates) continue;
            if (c > 0) {   // outputs of the last chunk
                if (!wait(b_o, c - 1)) break;
                put_out(c - 1);
            }
            if (c > 0 || have) {
                if (!wait(b_xs, c)) break;
                tc_fence_after();
                const float f = a_inter * sm.gp[reverse ? max(0, cnt - 1 - row) : row + 1];
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    uint32_t r[32];
                    tmem_ld32(tlane + TM_O + 64 * half + 32 * k, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 &v = reinterpret_cast<float2 *>(r)[i];
                        v = mul2(v, both(f));
                    }
                    tmem_st32(tlane + TM_O + 64 * half + 32 * k, r);
                }
                tmem_st_wait();
                tc_fence_before();
            }
            arrive(b_sc);
        }
        if (!kStates && nchunk > 0 && wait(b_o, nchunk - 1)) put_out(nchunk - 1);
        if (want_s && (nchunk == 0 || wait(b_u, nchunk - 1))) {
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                uint32_t r[32];
                tmem_ld32(t_s + 32 * k, r);
                tmem_ld_wait();
                const int z = 64 * half + 32 * k;
                if (dst_t) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) dst[(z + i) * kD + row] = __uint_as_float(r[i]);
                } else if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {   // whole sectors of a row
#pragma unroll
                    for (int i = 0; i < 4; ++i) st_global_v8(dst + row * kD + z + 8 * i, r + 8 * i);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(dst + row * kD + z + 4 * i) =
                            make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                }
            }
        }
        if (!kStates) {
            if (lane == 0) tma_store_wait_all();
            // outputs of tokens past the valid chunks
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + (static_cast<size_t>(b) * T * p.H + h) * kD;
            for (int t = t_begin + nchunk * kC + row; t < t_stop; t += kC) {
                uint4 *to = reinterpret_cast<uint4 *>(out + static_cast<size_t>(t) * p.H * kD + 64 * half);
#pragma unroll
                for (int i = 0; i < 8; ++i) to[i] = make_uint4(0u, 0u, 0u, 0u);
            }
        }
    } else {
        // ---------------------------------------------------------------- keys
        const int half = (warp - 16) >> 2, gt = tid - 512, T = p.T;   // tokens 64 half .. of the chunk
        const bool reverse = p.reverse;
        const float a_upd = p.a_upd;
        int wcnt = -1;
        uint2 w[8];   // of this thread's token pairs: 4 q + lane % 4 of the half, q < 8
        for (int c = 0; c < nchunk; ++c) {
            const int cnt = count_of(c);
            const bool update = c < nchunk - 1 || want_s;
            if (cnt != wcnt) {
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    float f[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int t = 64 * half + 8 * q + 2 * (lane & 3) + u;
                        f[u] = t < cnt ? a_upd * sm.gp[reverse ? t + 1 : cnt - 1 - t] : 0.f;
                    }
                    w[q].x = pack_bf16(f[0], f[1]);
                    w[q].y = pack_bf16(f[0] - __uint_as_float(w[q].x << 16),
                                       f[1] - __uint_as_float(w[q].x & 0xFFFF0000u));
                }
                wcnt = cnt;
            }
            const uint32_t st = stage_of(c), stage = 8 * (c % kNs);
            if (!wait(b_fy + stage, c / kNs)) break;
            const int t0 = t_begin + chunk_of(c) * kC;
            if (cnt < kC && t0 + cnt < T) {
                // masked tokens that the tile holds: a zero weight does not silence a NaN in Z
                if (!wait(b_fz + stage, c / kNs)) break;
                for (int i = gt; i < (kC - cnt) * 16; i += 256) {
                    const int r = cnt + (i >> 4), k = i & 15;
                    st_shared_v4(st + kZt + (k >> 3) * kHalf + r * 128 + (k & 7) * 16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            bool ok = true;
            if (update) {   // weighted keys, transposed: lane = x channel, columns = tokens of this half
                // ldmatrix turns 8 x 8 blocks around: thread t gets channel t / 4 and token pair t % 4 of each,
                // which is how tensor memory takes 16 lanes x 4 columns. 16 channels x 64 tokens at a time.
#pragma unroll 1
                for (int g16 = 0; g16 < 2; ++g16) {
                    const int ch = (warp & 3) * 32 + 16 * g16;
                    // lane l gives the address of one row of block l / 8: tokens +8 for blocks 2 and 3,
                    // channels +8 for blocks 1 and 3
                    const int tok = 64 * half + (lane & 7) + ((lane >> 4) << 3), c8 = ch + ((lane >> 3) & 1) * 8;
                    const uint32_t from = st + kY + (c8 >> 6) * kHalf + sw128_off(tok, (c8 & 63) * 2);
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {   // 16 tokens
                        uint32_t y[4];
                        wmma16::ldsm4t(from + i * 16 * 128, y);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            if (cnt < kC) {   // masked tokens: zero whatever the keys hold
                                const int t = 64 * half + 16 * i + 8 * (u >> 1) + 2 * (lane & 3);
                                if (t >= cnt) y[u] = 0u;
                                else if (t + 1 >= cnt) y[u] &= 0xFFFFu;
                            }
                            // w y = hi + lo: hi rounds w1 y, lo takes its exact rest and w2 y (w = w1 + w2)
                            const uint2 f = w[2 * i + (u >> 1)];
                            const uint32_t a = mul_bf16x2(f.x, y[u]);
                            hi[4 * i + u] = a;
                            lo[4 * i + u] = fma_bf16x2(f.y, y[u], fma_bf16x2(f.x, y[u], a ^ 0x80008000u));
                        }
                    }
                    // the keys that these replace are read
                    if (g16 == 0)
                        ok = kStates ? c < 2 || wait(b_xfree + 8 * (c & 1), (c - 2) >> 1) : c == 0 || wait(b_u, c - 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t to = tlane + (static_cast<uint32_t>(16 * g16) << 16) + keys_at(c) + 32 * half;
                    tmem_st_frag16(to, hi);
                    tmem_st_frag16(to + 64, lo);
                }
                tmem_st_wait();
                tc_fence_before();
            } else if (!kStates && c > 0) {
                ok = wait(b_u, c - 1);
            }
            if (!ok) break;
            arrive(keys_ready(c));
            arrive(b_yfree + stage);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (sm.abort && warp == 25) {   // products of an aborted pass: wait for what was issued
        if (elect_one()) {
            mma_commit(b_end);
            mbar_wait_bounded(b_end, 0, kWaitLimit);
        }
    }
    if (sm.abort && tid == 0) atomicOr(tp.err, kErrTimeout);
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// ---------------------------------------------------------------------------- host side
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

// Strided [B, T, H, 128] bf16 tensor; box = 64 channels x `tokens` tokens of one (b, h).
bool make_map(CUtensorMap *m, const void *base, const int64_t (&st)[3], int B, int T, int H, int tokens) {
    const EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {kD, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(B)};
    // the stride of an axis of one element is never used
    const cuuint64_t strides[3] = {H > 1 ? static_cast<cuuint64_t>(st[2]) * 2 : 256,
                                   T > 1 ? static_cast<cuuint64_t>(st[1]) * 2 : 256,
                                   B > 1 ? static_cast<cuuint64_t>(st[0]) * 2 : 256};
    const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(tokens), 1}, estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tma_rows(const void *base, const int64_t (&st)[3], int B, int T, int H) {
    const int size[3] = {B, T, H};
    for (int i = 0; i < 3; ++i)
        if (size[i] > 1 && (st[i] <= 0 || st[i] % 8 != 0 || st[i] >= (int64_t(1) << 38))) return false;
    return (reinterpret_cast<uintptr_t>(base) & 15) == 0;
}

// The kernels' shared memory, asked for once per device: the attribute outlasts the call.
cudaError_t allow_smem() {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return e != cudaSuccess ? e : cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    for (const void *k : {reinterpret_cast<const void *>(lin_tc_kernel<true>),
                          reinterpret_cast<const void *>(lin_tc_kernel<false>)})
        if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM_BYTES))) !=
            cudaSuccess)
            return e;
    done[dev].store(true, std::memory_order_release);
    return cudaSuccess;
}

}  // namespace

bool lin_tc_supports(const LinScan &p, kla_dtype dtype) {
    return dtype == KLA_DTYPE_BF16 && p.dx == kD && p.dz == kD && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 &&
           tma_rows(p.x, p.xs, p.B, p.T, p.H) && tma_rows(p.y, p.ys, p.B, p.T, p.H) &&
           tma_rows(p.z, p.zs, p.B, p.T, p.H);
}

// Segments by their cost in microseconds, as measured: a launch starts and ends in ~8 and the three launches
// of a cut sequence in ~17; a chunk takes 1.9, or its share of the memory's rate (128 KB, of which the
// segment's own state takes half, in 0.95; four fifths where the scans of a backward pass share tiles in L2).
// 48 chains of 1000 tokens: 25 in one piece, 38 in two; 16 of 2000: 36 in one, 27 in eight; backward, 8
// chains of 16384: 136 in four, 105 in six.
void lin_tc_plan(LinScan &p, int scans) {
    constexpr int kSms = 152;
    const int nchunk = (p.T + kC - 1) / kC;
    const long ctas = static_cast<long>(p.B) * p.H * scans;
    auto chunk_us = [scans](double least, double kb, long on) {
        const double fed = (scans > 1 ? 0.8 : 1.0) * kb * 1e-3 * static_cast<double>(on) / 6.78;
        return fed > least ? fed : least;
    };
    int best = nchunk > 0 ? nchunk : 1;
    double least = 8 + chunk_us(1.9, 131, ctas) * nchunk;
    for (int n = 2; n <= nchunk && n * ctas <= kSms; ++n) {
        const int len = (nchunk + n - 1) / n;
        const double cost = 17 + (chunk_us(1.9, 131, n * ctas) + chunk_us(0.95, 66, n * ctas)) * len;
        if (cost < 1.02 * least) {   // of equals the one on more SMs
            if (cost < least) least = cost;
            best = len;
        }
    }
    p.seg_len = best * kC;
    p.nseg = nchunk > 0 ? (nchunk + best - 1) / best : 1;
}

cudaError_t launch_lin_tc(const LinScan *p, int scans, cudaStream_t stream) {
    TcParams tp;
    tp.scans = scans;
    for (int i = 0; i < scans; ++i) {
        tp.job[i].p = p[i];
        tp.job[i].p.seg_t = 1;
        const LinScan &q = p[i];
        const int64_t dense[3] = {static_cast<int64_t>(q.T) * q.H * kD, static_cast<int64_t>(q.H) * kD, kD};
        auto tile = [&](CUtensorMap *m, const void *base, const int64_t (&st)[3]) {
            for (int k = 0; k < i; ++k) {   // the directions of a backward pass share their inputs
                const LinScan &o = p[k];
                const void *had[3] = {o.x, o.y, o.z};
                const int64_t *hs[3] = {o.xs, o.ys, o.zs};
                const CUtensorMap *hm[3] = {&tp.job[k].x, &tp.job[k].y, &tp.job[k].z};
                for (int u = 0; u < 3; ++u)
                    if (had[u] == base && hs[u][0] == st[0] && hs[u][1] == st[1] && hs[u][2] == st[2]) {
                        *m = *hm[u];
                        return true;
                    }
            }
            return make_map(m, base, st, q.B, q.T, q.H, kC);
        };
        if (!tile(&tp.job[i].x, q.x, q.xs) || !tile(&tp.job[i].y, q.y, q.ys) || !tile(&tp.job[i].z, q.z, q.zs) ||
            !make_map(&tp.job[i].o, q.out, dense, q.B, q.T, q.H, 32))
            return cudaErrorInvalidValue;
    }
    cudaError_t e;
    if ((e = device_error_word(&tp.err)) != cudaSuccess || (e = allow_smem()) != cudaSuccess) return e;
    const int chains = p[0].B * p[0].H, nseg = p[0].nseg;
    if (nseg > 1) {
        lin_tc_kernel<true><<<dim3(chains * scans, nseg - 1), kThreads, SMEM_BYTES, stream>>>(tp);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        LinScan all[3];
        for (int i = 0; i < scans; ++i) all[i] = tp.job[i].p;
        if ((e = launch_lin_combine(all, scans, stream)) != cudaSuccess) return e;
    }
    if (nseg > 1)
        return launch_dependent(lin_tc_kernel<false>, dim3(chains * scans, nseg), kThreads, SMEM_BYTES, stream, tp);
    lin_tc_kernel<false><<<chains * scans, kThreads, SMEM_BYTES, stream>>>(tp);
    return cudaGetLastError();
}

}  // namespace kla
