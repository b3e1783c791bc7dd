// kla_linear.cuh -- the scan that every direction of the decayed linear attention is made of.
//
// With roles x (query), y (key), z (value) and a state S (dx x dz) the scan computes, along time,
//     out_i = sum_{j <= i} a_intra g^{i-j} (x_i.y_j) z_j + a_inter g^{i+1} S0^T x_i
//     S_end = g^n S0 + a_upd sum_j g^{n-1-j} y_j z_j^T
// and against time (j >= i, g^{j-i}; the entering state undecayed at the last token: g^{n-1-i} in
// the read, g^{j+1} in the update, so that S_end is the gradient of the state before the first
// token). The four directions, with s the query scale:
//     o  = scan(q, k, v, S0)            intra s, inter s, update 1        S_end = S_T
//     dq = scan(dO, v, k, S0^T)         intra s, inter s, update 1
//     dk = back(v, dO, q, dS_T^T)       intra s, inter 1, update s
//     dv = back(k, q, dO, dS_T)         intra s, inter 1, update s        S_end = dS0
#pragma once

#include "layer_dev.cuh"
#include "../../include/kla_layer.h"

namespace kla {

struct LinScan {
    const void *x, *y, *z;
    int64_t xs[3], ys[3], zs[3];   // element strides of batch, token, head
    void *out;                     // [B, T, H, dz] contiguous, the inputs' dtype
    const float *decay;
    const int *lengths;            // or NULL
    const float *S0;               // or NULL (zeros)
    float *ST;                     // or NULL
    int s_t;                       // 1: S0 and ST are stored [dz][dx]
    int B, T, H, dx, dz;
    int reverse;
    float a_intra, a_inter, a_upd;
    float *seg_states;             // scratch of nseg > 1 segments: [chains][nseg][dx][dz], or [dz][dx]; the
    int seg_t;                     // 1: the latter                 start state of segment s at lin_slot(s)
    int nseg, seg_len;             // segments in processing order, tokens each
};

// Valid tokens of sequence b.
__device__ __forceinline__ int lin_length(const int *lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : n < T ? n : T;
}
// Valid tokens of the segment that is s-th in processing order, and its first token.
__device__ __forceinline__ int lin_segment(const LinScan &p, int s, int n, int &t0) {
    const int at = p.reverse ? p.nseg - 1 - s : s;
    t0 = at * p.seg_len;
    const int left = n - t0;
    return left < 0 ? 0 : left < p.seg_len ? left : p.seg_len;
}

// Slot k < nseg - 1 holds segment k's own contribution to the state, then the state after segment k;
// the last slot holds S0, which the last segment may overwrite (S_T in place) while the first reads it.
__device__ __forceinline__ size_t lin_slot(const LinScan &p, int chain, int k) {
    return (static_cast<size_t>(chain) * p.nseg + k) * p.dx * p.dz;
}
__device__ __forceinline__ int lin_start_slot(const LinScan &p, int seg) { return seg > 0 ? seg - 1 : p.nseg - 1; }

// Turns the contributions into start states.
cudaError_t launch_lin_combine(const LinScan *p, int scans, cudaStream_t stream);
// Tensor-core form: bf16, dx = dz = 128, rows that TMA can read (kla_linear_tc.cu). Runs up to three
// scans of the same sizes side by side in one launch, each with segments (and a scratch) of its own.
bool lin_tc_supports(const LinScan &p, kla_dtype dtype);
void lin_tc_plan(LinScan &p, int scans);
cudaError_t launch_lin_tc(const LinScan *p, int scans, cudaStream_t stream);
cudaError_t device_error_word(unsigned **out);   // kla_api.cu
// Any size, type, stride and alignment, fp32 arithmetic (kla_linear.cu).
cudaError_t launch_lin_scan(const LinScan *p, int scans, kla_dtype dtype, cudaStream_t stream);

}  // namespace kla
