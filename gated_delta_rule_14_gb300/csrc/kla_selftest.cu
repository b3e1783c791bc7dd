// kla_selftest.cu -- exercises the bounded-wait failure path without a GPU fault.
//
// Every wait of the library's kernels on an mbarrier is bounded: after its poll limit the wait
// gives up, the kernel records kErrTimeout in the device error word, skips its remaining work
// and exits cleanly, so the context stays usable and kla_device_status reports
// KLA_ERR_TIMEOUT. These kernels run that path on purpose: one thread waits, with the same
// bounded wait, on a barrier phase that nothing completes; one team of a CTA does, beside teams that
// go on; and one warp does, which calls the CTA's other warps out of waits of their own.
#include "kla_internal.cuh"
#include "kla_norm.cuh"
#include "sm103_ptx.cuh"

namespace {

__global__ void selftest_wait_kernel(unsigned *err, uint32_t limit) {
    __shared__ uint64_t bar;
    const uint32_t b = kla::ptx::smem_u32(&bar);
    if (threadIdx.x == 0) {
        kla::ptx::mbar_init(b, 1);
        kla::ptx::fence_mbar_init();
    }
    __syncthreads();
    // a freshly initialised barrier sits in phase 0 and nobody arrives: the wait must give up
    if (threadIdx.x == 0 && !kla::ptx::mbar_wait_bounded(b, 0, limit)) atomicOr(err, kla::kErrTimeout);
}

// Teams that walk turns as those of the layer norm do (kla_norm.cu): a wait, a sum with the team's barrier,
// the decision whether to leave. The first team's phase of turn 1 is never completed.
constexpr int kTeamWidth = 64, kTeams = 4, kTurns = 20000;

__global__ void __launch_bounds__(kTeamWidth *kTeams) selftest_teams_kernel(unsigned *err, int *done, uint32_t limit) {
    using namespace kla;
    __shared__ uint64_t bars[kTeams];
    __shared__ float2 sums[2][kMaxBlock / 32];
    __shared__ int lost[kTeams][2];
    const int team = threadIdx.x / kTeamWidth;
    const bool lead = threadIdx.x % kTeamWidth == 0;
    const norm::TeamLost gave_up{lost[team]};
    norm::WarpsSum<kTeamWidth / 32> sum{sums, team * (kTeamWidth / 32), 1 + team, 0};
    const uint32_t bar = ptx::smem_u32(&bars[team]);
    if (lead) {
        gave_up.init();
        ptx::mbar_init(bar, 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    int t = 0;
    for (; t < kTurns; ++t) {
        if (lead && !(team == 0 && t > 0)) ptx::mbar_arrive(bar);
        if (!ptx::mbar_wait_bounded(bar, t & 1, limit)) gave_up.note(t);
        const float all = sum(1.f);
        if (gave_up.read(t) || all != kTeamWidth) break;
    }
    __syncthreads();
    if (lead && t < kTurns) atomicOr(err, kErrTimeout);
    done[threadIdx.x] = t;
}

// Warps that wait as those of the tensor-core scan do (kla_linear_tc.cu). Each completes its own phases up to
// turn kWarpTurns; the first warp none but that of turn 0, and it alone has the short limit.
constexpr int kWarps = 8, kWarpTurns = 100;

__global__ void __launch_bounds__(32 * kWarps) selftest_warps_kernel(unsigned *err, int *done, uint32_t limit) {
    using namespace kla;
    __shared__ uint64_t bars[kWarps];
    __shared__ int abort;
    const int warp = threadIdx.x / 32, last = warp ? kWarpTurns : 1;
    const bool lead = threadIdx.x % 32 == 0;
    const uint32_t bar = ptx::smem_u32(&bars[warp]);
    if (threadIdx.x == 0) abort = 0;
    if (lead) {
        ptx::mbar_init(bar, 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    int t = 0;
    for (; t < 2 * kWarpTurns; ++t) {
        if (lead && t < last) ptx::mbar_arrive(bar);
        if (!ptx::warp_wait(bar, t & 1, warp ? 100000u : limit, &abort)) break;
        __syncwarp();
    }
    __syncthreads();
    if (threadIdx.x == 0 && abort) atomicOr(err, kErrTimeout);
    done[threadIdx.x] = t;
}

}  // namespace

namespace kla {

cudaError_t launch_selftest_wait(unsigned *err, unsigned limit, cudaStream_t stream) {
    selftest_wait_kernel<<<1, 32, 0, stream>>>(err, limit);
    return cudaGetLastError();
}

cudaError_t launch_selftest_teams(unsigned *err, int *turns, unsigned limit, cudaStream_t stream) {
    selftest_teams_kernel<<<1, kTeamWidth * kTeams, 0, stream>>>(err, turns, limit);
    return cudaGetLastError();
}

cudaError_t launch_selftest_warps(unsigned *err, int *turns, unsigned limit, cudaStream_t stream) {
    selftest_warps_kernel<<<1, 32 * kWarps, 0, stream>>>(err, turns, limit);
    return cudaGetLastError();
}

}  // namespace kla
