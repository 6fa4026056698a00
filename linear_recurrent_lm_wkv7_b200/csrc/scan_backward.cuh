// scan_backward.cuh — what the launches of the selective scan's backward share
// (wkv7_scan_backward.cu, and wkv7_scan_tc.cu for the states of bf16 with N = 128).
#pragma once
#include "scan_common.cuh"

namespace wkv7 {

struct BwdDev {
    const void *x, *Bm, *Cm, *dy;
    long ldx, ldb, ldc, lddy;
    const float *A, *D, *s0, *dsT;
    void *dx, *ddt, *dB, *dC;
    long lddx, ldddt, lddb, lddc;
    float *dA, *dD, *dbias, *ds0;
    int H, G, softplus, dt_bf16;
    SegMap seg, chunk;   // segments, and the same cut at 64 tokens
    long seg_count, chunk_count;
    // workspace
    const Decays* dec;      // [chunk][H]
    __nv_bfloat16* states;  // [2][chunk][H] StateTile: S_0 and dS
    float* seg_state;       // [2][seg][H][64][N]
    float* seg_decay;       // [seg][H]
    float* part;            // [2][share][row][G N]: dB and dC of a share of the heads
    float* scalars;         // [chunk][H][4]: dA, d dt_bias, dD
    int shares;
    long rows;
    int* status;
};

// The tcgen05 kernel holds a state column per lane and writes the states transposed.
template <typename IO, int N>
constexpr bool kStatesT = sizeof(IO) == 2 && N == 128;
// A state as it lies in memory, and in shared memory after one bulk copy.
template <typename IO, int N>
using StateTile = SwizzledTile<kStatePlanes, kStatesT<IO, N> ? N : kScanP, kStatesT<IO, N> ? kScanP : N>;

// One pass of the states in both directions on tcgen05: as scan_states_kernel.
cudaError_t launch_states_tc(const BwdDev& d, bool write, bool whole, cudaStream_t stream);

}  // namespace wkv7
