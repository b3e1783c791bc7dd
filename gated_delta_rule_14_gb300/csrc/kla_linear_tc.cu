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
// TMEM instead: P replaces D column by column, and the weighted keys are written transposed.
// (diag(w) Y)^T is kept as two bf16 terms (hi + lo, 2^-17 relative): the fp32 state is an output of
// its own, and one term (2^-9) would be its error. S as an operand and P are rounded to one bf16
// term: they only enter O, which is stored with 8 bits itself.
//
// Warps: 0-3 turn D into P; 4-7 scale the first half of O and write the outputs; 8-15 own S in fp32
// registers (thread = one x channel, 64 z channels), weigh the keys and update S; 16 loads (TMA, two
// stages of X, Y, Z tiles); 17 issues the products. They hand over through mbarriers that complete
// once per chunk.
#include <cuda.h>

#include "kla_linear.cuh"
#include "sm103_ptx.cuh"

namespace kla {
namespace {

using namespace ptx;

constexpr int kC = 128, kD = 128;
constexpr int kThreads = 18 * 32;
constexpr uint32_t kWaitLimit = 100000;   // x 20 us: a stuck wait gives up after ~2 s
constexpr uint32_t kTile = 32768, kHalf = 16384;   // a 128 x 128 bf16 tile: two blocks of 64 channels
constexpr uint32_t OFF_STAGE = 0, STAGE = 3 * kTile;
constexpr uint32_t OFF_S = 2 * STAGE;
constexpr uint32_t OFF_SMALL = OFF_S + kTile;
constexpr uint32_t SMEM_BYTES = OFF_SMALL + 2048 + 1024;   // + alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory");
constexpr uint32_t TM_D = 0, TM_P = 0, TM_O = 128, TM_U = 256, TM_YH = 384, TM_YL = 448;
constexpr uint32_t kBarKeys = 1;   // named barrier of warps 8-15

struct Small {
    uint64_t full[2];   // X, Y, Z tiles landed, by stage
    uint64_t free[2];   // every product that reads the stage is done
    uint64_t end;       // after an abort: the products that were issued are done
    uint64_t d, p;      // D computed, P written
    uint64_t xs, sc;    // X S computed, scaled
    uint64_t o, ord;    // O computed, O read
    uint64_t y, u, urd; // weighted keys written, U computed, U read
    uint64_t s;         // operand copy of S written
    uint32_t tmem_base;
    volatile int abort;
    float gp[kC + 1];   // g^0 .. g^128
    float gb[32];       // g of the distance within a 32-column block, from its near side
    alignas(16) float w[kC];
};
static_assert(sizeof(Small) <= 2048, "small area");

struct Job {
    CUtensorMap x, y, z;
    LinScan p;
};
struct TcParams {
    Job job[3];
    int scans, first_seg, states;
    unsigned *err;
};

__device__ __forceinline__ void st_global_v8(void *p, const uint32_t *r) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
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

    const uint32_t b_full = smem_u32(&sm.full[0]), b_free = smem_u32(&sm.free[0]), b_end = smem_u32(&sm.end);
    const uint32_t b_d = smem_u32(&sm.d), b_p = smem_u32(&sm.p), b_xs = smem_u32(&sm.xs), b_sc = smem_u32(&sm.sc);
    const uint32_t b_o = smem_u32(&sm.o), b_ord = smem_u32(&sm.ord), b_y = smem_u32(&sm.y), b_u = smem_u32(&sm.u);
    const uint32_t b_urd = smem_u32(&sm.urd), b_s = smem_u32(&sm.s);
    if (tid == 0) {
        mbar_init(b_full, 1);
        mbar_init(b_full + 8, 1);
        mbar_init(b_free, 1);
        mbar_init(b_free + 8, 1);
        mbar_init(b_end, 1);
        mbar_init(b_d, 1);
        mbar_init(b_p, 4);
        mbar_init(b_xs, 1);
        mbar_init(b_sc, 4);
        mbar_init(b_o, 1);
        mbar_init(b_ord, 4);
        mbar_init(b_y, 8);
        mbar_init(b_u, 1);
        mbar_init(b_urd, 8);
        mbar_init(b_s, 8);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (tid <= kC) sm.gp[tid] = powf(g, static_cast<float>(tid));
    if (warp == 5) sm.gb[lane] = powf(g, static_cast<float>(p.reverse ? lane : 31 - lane));
    if (warp == 0) {
        tmem_alloc(smem_u32(&sm.tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = sm.tmem_base;
    const uint32_t tlane = tbase + (static_cast<uint32_t>((warp & 3) * 32) << 16);

    // False once any wait of the CTA has given up: every loop then ends.
    auto wait = [&](uint32_t bar, int phase) {
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
    auto chunk_of = [&](int c) { return p.reverse ? nchunk - 1 - c : c; };
    auto count_of = [&](int c) { return min(kC, valid - chunk_of(c) * kC); };

    if (warp == 16) {
        // ---------------------------------------------------------------- loads
        int issued = 0, seen = 0;
        if (lane == 0) {
            for (int c = 0; c < nchunk; ++c) {
                if (c >= 2 && !wait(b_free + 8 * (c & 1), (c - 2) >> 1)) break;
                const uint32_t st = sbase + OFF_STAGE + (c & 1) * STAGE, bar = b_full + 8 * (c & 1);
                const int t0 = t_begin + chunk_of(c) * kC;
                mbar_arrive_expect_tx(bar, (kStates ? 2 : 3) * kTile);
                for (int i = 0; i < 2; ++i) {
                    if (!kStates) tma_load_4d(st + i * kHalf, &job.x, bar, 64 * i, h, t0, b);
                    tma_load_4d(st + kTile + i * kHalf, &job.y, bar, 64 * i, h, t0, b);
                }
                for (int i = 0; i < 2; ++i) tma_load_4d(st + 2 * kTile + i * kHalf, &job.z, bar, 64 * i, h, t0, b);
                ++issued;
            }
            // nothing of this CTA's may be in flight when it ends, an abort included
            for (seen = issued > 2 ? issued - 2 : 0; seen < issued; ++seen)
                mbar_wait_bounded(b_full + 8 * (seen & 1), (seen >> 1) & 1, kWaitLimit);
        }
    } else if (warp == 17) {
        // ---------------------------------------------------------------- products
        const bool lead = elect_one();
        const uint32_t id_kk = idesc_bf16(128, 128, 0, 0), id_km = idesc_bf16(128, 128, 0, 1);
        const uint64_t ds = sw128_desc(sbase + OFF_S, kHalf, 1024);
        for (int c = 0; c < nchunk; ++c) {
            const uint32_t st = sbase + OFF_STAGE + (c & 1) * STAGE;
            const uint64_t dx = sw128_desc(st, 16, 1024), dy = sw128_desc(st + kTile, 16, 1024);
            const uint64_t dz = sw128_desc(st + 2 * kTile, kHalf, 1024);
            const bool update = c < nchunk - 1 || want_s;
            const bool inter = !kStates && (c > 0 || have);
            if (!wait(b_full + 8 * (c & 1), c >> 1)) break;
            if (!kStates) {
                if (c > 0 && !wait(b_o, c - 1)) break;   // P of the last chunk, which lies over D, is done with
                tc_fence_after();
                if (lead) {
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t off = (s >> 2) * kHalf + (s & 3) * 32;
                        mma_bf16(tbase + TM_D, desc_add(dx, off), desc_add(dy, off), id_kk, s);
                    }
                    mma_commit(b_d);
                }
            }
            if (!wait(b_y, c) || (c > 0 && !wait(b_urd, c - 1))) break;
            tc_fence_after();
            if (lead) {
                if (update) {
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_bf16_ta(tbase + TM_U, tbase + TM_YH + 8 * s, desc_add(dz, s * 2048), id_km, s);
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_bf16_ta(tbase + TM_U, tbase + TM_YL + 8 * s, desc_add(dz, s * 2048), id_km, 1);
                }
                mma_commit(b_u);
                if (kStates) mma_commit(b_free + 8 * (c & 1));
            }
            __syncwarp();
            if (kStates) continue;
            if (!wait(b_s, c) || (c > 0 && !wait(b_ord, c - 1))) break;
            tc_fence_after();
            if (lead) {
                if (inter) {
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_bf16(tbase + TM_O, desc_add(dx, (s >> 2) * kHalf + (s & 3) * 32), desc_add(ds, s * 2048),
                                 id_km, s);
                }
                mma_commit(b_xs);
            }
            if (!wait(b_p, c) || !wait(b_sc, c)) break;
            tc_fence_after();
            if (lead) {
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_bf16_ta(tbase + TM_O, tbase + TM_P + 8 * s, desc_add(dz, s * 2048), id_km, inter || s > 0);
                mma_commit(b_o);
                mma_commit(b_free + 8 * (c & 1));
            }
            __syncwarp();
        }
    } else if (warp < 4) {
        // ---------------------------------------------------------------- D -> P
        const int w = warp;
        for (int c = 0; !kStates && c < nchunk; ++c) {
            const int cnt = count_of(c);
            if (!wait(b_d, c)) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k) {   // ascending: P's columns lie over columns of D already read
                uint32_t pk[16];
                if (p.reverse ? k < w : k > w) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) pk[i] = 0u;
                } else {
                    uint32_t r[32];
                    tmem_ld32(tlane + TM_D + 32 * k, r);
                    tmem_ld_wait();
                    if (k == w) {   // the diagonal block: every distance from the table
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const int dist = p.reverse ? i - lane : lane - i;
                            const float f = dist >= 0 ? p.a_intra * sm.gp[dist & 31] : 0.f;
                            const float v = f * __uint_as_float(r[i]);
                            r[i] = __float_as_uint(dist >= 0 && 32 * k + i < cnt ? v : 0.f);
                        }
                    } else {        // distance to the block's near side times distance within the block
                        const float f = p.a_intra * sm.gp[p.reverse ? 32 * k - row : row - 32 * k - 31];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float v = (f * sm.gb[i]) * __uint_as_float(r[i]);
                            r[i] = __float_as_uint(32 * k + i < cnt ? v : 0.f);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        pk[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                }
                tmem_st16(tlane + TM_P + 16 * k, pk);
            }
            tmem_st_wait();
            tc_fence_before();
            arrive(b_p);
        }
    } else if (warp < 8) {
        // ---------------------------------------------------------------- O
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
        const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
        for (int c = 0; !kStates && c < nchunk; ++c) {
            const int cnt = count_of(c);
            if (c > 0 || have) {
                if (!wait(b_xs, c)) break;
                tc_fence_after();
                const float f = p.a_inter * sm.gp[p.reverse ? max(0, cnt - 1 - row) : row + 1];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint32_t r[16];
                    tmem_ld16(tlane + TM_O + 16 * k, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(f * __uint_as_float(r[i]));
                    tmem_st16(tlane + TM_O + 16 * k, r);
                }
                tmem_st_wait();
                tc_fence_before();
            }
            arrive(b_sc);
            if (!wait(b_o, c)) break;
            tc_fence_after();
            const int t = t_begin + chunk_of(c) * kC + row;
            __nv_bfloat16 *dst = out + ((static_cast<size_t>(b) * p.T + t) * p.H + h) * kD;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t r[32], pk[16];
                tmem_ld32(tlane + TM_O + 32 * k, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    pk[i] = row < cnt ? pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])) : 0u;
                if (t < t_stop) {
                    if (wide) {
                        st_global_v8(dst + 32 * k, pk);
                        st_global_v8(dst + 32 * k + 16, pk + 8);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            reinterpret_cast<uint4 *>(dst + 32 * k)[i] =
                                make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
            arrive(b_ord);
        }
        // outputs of tokens past the valid chunks
        for (int t = t_begin + nchunk * kC + row; !kStates && t < t_stop; t += kC) {
            uint4 *dst = reinterpret_cast<uint4 *>(out + ((static_cast<size_t>(b) * p.T + t) * p.H + h) * kD);
#pragma unroll
            for (int i = 0; i < 16; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
        }
    } else {
        // ---------------------------------------------------------------- keys and state
        const int half = (warp - 8) >> 2, gt = tid - 256;
        float s[64];
        const size_t sdd = static_cast<size_t>(kD) * kD;
        {
            const float *src = nullptr;
            bool tr = false;
            if (have) {
                src = seg > 0 ? p.seg_states + (static_cast<size_t>(chain) * (p.nseg - 1) + seg - 1) * sdd
                              : p.S0 + chain * sdd;
                tr = seg == 0 && p.s_t;
            }
#pragma unroll
            for (int i = 0; i < 64; ++i)
                s[i] = !src ? 0.f : tr ? src[(64 * half + i) * kD + row] : src[row * kD + 64 * half + i];
        }
        auto put_s = [&]() {   // bf16 copy of S: row = x channel, 128-byte swizzled rows of 64 z channels
            const uint32_t base = sbase + OFF_S + half * kHalf;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                st_shared_v4(base + sw128_off(row, 16 * i), pack_bf16(s[8 * i], s[8 * i + 1]),
                             pack_bf16(s[8 * i + 2], s[8 * i + 3]), pack_bf16(s[8 * i + 4], s[8 * i + 5]),
                             pack_bf16(s[8 * i + 6], s[8 * i + 7]));
            fence_proxy_async_smem();
        };
        if (!kStates) {
            if (have) put_s();
            arrive(b_s);
        }
        int wcnt = -1;
        for (int c = 0; c < nchunk; ++c) {
            const int cnt = count_of(c);
            const bool update = c < nchunk - 1 || want_s;
            if (cnt != wcnt) {
                named_sync(kBarKeys, 256);
                if (gt < kC)
                    sm.w[gt] = gt < cnt ? p.a_upd * sm.gp[p.reverse ? gt + 1 : cnt - 1 - gt] : 0.f;
                named_sync(kBarKeys, 256);
                wcnt = cnt;
            }
            if (!wait(b_full + 8 * (c & 1), c >> 1)) break;
            const uint32_t st = sbase + OFF_STAGE + (c & 1) * STAGE;
            const int t0 = t_begin + chunk_of(c) * kC;
            if (cnt < kC && t0 + cnt < p.T) {
                // masked tokens that the tile holds: a zero weight does not silence a NaN in Z
                for (int i = gt; i < (kC - cnt) * 16; i += 256) {
                    const int r = cnt + (i >> 4), k = i & 15;
                    st_shared_v4(st + 2 * kTile + (k >> 3) * kHalf + r * 128 + (k & 7) * 16, 0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            if (update) {   // weighted keys, transposed: lane = x channel, columns = tokens of this half
                const uint32_t yb = st + kTile + (row >> 6) * kHalf;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int j = 64 * half + 16 * q + 2 * i;
                        const float2 w = *reinterpret_cast<const float2 *>(&sm.w[j]);
                        float a = ld_shared_bf16(yb + sw128_off(j, (row & 63) * 2));
                        float e = ld_shared_bf16(yb + sw128_off(j + 1, (row & 63) * 2));
                        a = j < cnt ? a * w.x : 0.f;
                        e = j + 1 < cnt ? e * w.y : 0.f;
                        hi[i] = pack_bf16(a, e);
                        lo[i] = pack_bf16(a - __uint_as_float(hi[i] << 16), e - __uint_as_float(hi[i] & 0xFFFF0000u));
                    }
                    tmem_st8(tlane + TM_YH + 32 * half + 8 * q, hi);
                    tmem_st8(tlane + TM_YL + 32 * half + 8 * q, lo);
                }
                tmem_st_wait();
                tc_fence_before();
            }
            arrive(b_y);
            if (!wait(b_u, c)) break;
            tc_fence_after();
            if (update) {
                const float gn = sm.gp[cnt];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t r[16];
                    tmem_ld16(tlane + TM_U + 64 * half + 16 * k, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[16 * k + i] = fmaf(gn, s[16 * k + i], __uint_as_float(r[i]));
                }
                tc_fence_before();
            }
            arrive(b_urd);
            if (!kStates && c < nchunk - 1) {
                if (!wait(b_xs, c)) break;   // the copy in use is read
                put_s();
                arrive(b_s);
            }
        }
        if (want_s && !sm.abort) {
            float *dst = kStates ? p.seg_states + (static_cast<size_t>(chain) * (p.nseg - 1) + seg) * sdd
                                 : p.ST + chain * sdd;
            const bool tr = !kStates && p.s_t;
#pragma unroll
            for (int i = 0; i < 64; ++i)
                dst[tr ? (64 * half + i) * kD + row : row * kD + 64 * half + i] = s[i];
        }
    }
    tc_fence_before();
    __syncthreads();
    if (sm.abort && warp == 17) {   // products of an aborted pass: wait for what was issued
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

// Strided [B, T, H, 128] bf16 tensor; box = 64 channels x 128 tokens of one (b, h).
bool make_map(CUtensorMap *m, const void *base, const int64_t (&st)[3], int B, int T, int H) {
    const EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {kD, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T), static_cast<cuuint64_t>(B)};
    // the stride of an axis of one element is never used
    const cuuint64_t strides[3] = {H > 1 ? static_cast<cuuint64_t>(st[2]) * 2 : 256,
                                   T > 1 ? static_cast<cuuint64_t>(st[1]) * 2 : 256,
                                   B > 1 ? static_cast<cuuint64_t>(st[0]) * 2 : 256};
    const cuuint32_t box[4] = {64, 1, kC, 1}, estr[4] = {1, 1, 1, 1};
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

}  // namespace

bool lin_tc_supports(const LinScan &p, kla_dtype dtype) {
    return dtype == KLA_DTYPE_BF16 && p.dx == kD && p.dz == kD && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0 &&
           tma_rows(p.x, p.xs, p.B, p.T, p.H) && tma_rows(p.y, p.ys, p.B, p.T, p.H) &&
           tma_rows(p.z, p.zs, p.B, p.T, p.H);
}

void lin_tc_plan(LinScan &p, int scans) {
    constexpr int kSms = 152;
    const int nchunk = (p.T + kC - 1) / kC;
    const long ctas = static_cast<long>(p.B) * p.H * scans;
    long n = ctas >= kSms ? 1 : kSms / ctas;
    if (n > nchunk / 4) n = nchunk / 4;
    if (n < 1) n = 1;
    const int len = static_cast<int>((nchunk + n - 1) / n);
    p.seg_len = (len > 0 ? len : 1) * kC;
    p.nseg = nchunk > 0 ? (nchunk + len - 1) / len : 1;
}

cudaError_t launch_lin_tc(const LinScan *p, int scans, cudaStream_t stream) {
    TcParams tp;
    tp.scans = scans;
    for (int i = 0; i < scans; ++i) {
        tp.job[i].p = p[i];
        if (!make_map(&tp.job[i].x, p[i].x, p[i].xs, p[i].B, p[i].T, p[i].H) ||
            !make_map(&tp.job[i].y, p[i].y, p[i].ys, p[i].B, p[i].T, p[i].H) ||
            !make_map(&tp.job[i].z, p[i].z, p[i].zs, p[i].B, p[i].T, p[i].H))
            return cudaErrorInvalidValue;
    }
    cudaError_t e;
    if ((e = device_error_word(&tp.err)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(lin_tc_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(SMEM_BYTES))) != cudaSuccess ||
        (e = cudaFuncSetAttribute(lin_tc_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  static_cast<int>(SMEM_BYTES))) != cudaSuccess)
        return e;
    const int chains = p[0].B * p[0].H, nseg = p[0].nseg;
    if (nseg > 1) {
        lin_tc_kernel<true><<<dim3(chains * scans, nseg - 1), kThreads, SMEM_BYTES, stream>>>(tp);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        for (int i = 0; i < scans; ++i)
            if ((e = launch_lin_combine(p[i], stream)) != cudaSuccess) return e;
    }
    lin_tc_kernel<false><<<dim3(chains * scans, nseg), kThreads, SMEM_BYTES, stream>>>(tp);
    return cudaGetLastError();
}

}  // namespace kla
