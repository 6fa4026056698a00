// wkv7_scan.cu — selective state-space scan: prompts and single tokens.
//
// The recurrence and its chunk form are in scan_common.cuh.  A block carries the state
// of one head through the chunks of one segment of a sequence.  It works on transposed
// outputs, Y^T = S C^T and X^T M^T, so that the rows of S (and of X^T) are the rows of
// the warp-level products: warp w holds rows 16 (w % 4) .. of the state and one half
// (w / 4) of its N columns in fp32 registers for the whole segment, and the state
// never passes through shared memory.  Per chunk
//   G = C B^T (lower triangle, ten 16 x 16 pieces over the eight warps),
//   M_ts = G_ts exp(l_t - l_s) delta_s, rounded to planes in shared memory,
//   Y^T = exp(l_t) (S C^T) + X^T M^T  (each half of the warps sums half of the terms;
//         the two partial sums meet in shared memory),
//   S <- exp(l_64) S + (X^T delta exp(l_64 - l)) B.
// Few heads and long sequences leave most SMs idle, so then sequences are cut into
// segments: a first pass takes every segment's state from zero, a join walks the
// segments of a head (S <- decay S + segment's state), and a second pass starts each
// segment from its true state.
//
// What bounds it: no more than two blocks fit an SM, and their
// warps wait for each other's results more than the tensor pipe is busy.  fp32, packed
// [5003] rows in nine sequences, H12 N64 G4: 86 us; of the outputs' 59 (ncu) the tensor pipe is
// busy for 40 % (three planes of an operand: six products for one), of the states' 25 for 32 %.
#include <algorithm>

#include "scan_common.cuh"

namespace wkv7 {

// wkv7_scan_tc.cu: one pass of the tcgen05 kernel, over the outputs or the segments' states
cudaError_t launch_scan_tc(const ScanArgs& p, const SegMap& map, bool whole, bool out, float* seg_state,
                           float* seg_decay, cudaStream_t stream);

namespace {

template <typename IO, int N>
struct FwdLayout {
    static constexpr int PI = kInPlanes<IO>, PC = kCalcPlanes<IO>;
    using TX = Tile<PI, kChunk, kScanP>;
    using TB = Tile<PI, kChunk, N>;
    using TM = Tile<PC, kChunk, kChunk>;
    // bf16: the next chunk is copied while this one is worked on
    static constexpr int stages = sizeof(IO) == 2 ? 2 : 1;
    static constexpr int stage_bytes = TX::bytes + 2 * TB::bytes;
    static constexpr int off_m = stages * stage_bytes;
    static constexpr int xchg_bytes = kScanThreads * 16 * 4;
    static constexpr int m_bytes = TM::bytes > xchg_bytes ? TM::bytes : xchg_bytes;
    // fp32 rows of Y, one area per warp: over B and C, which have been used by then, where
    // they are large enough
    static constexpr int y_pitch = 20;  // floats: 16 rows p of a token and 4 of padding
    static constexpr int y_bytes = sizeof(IO) == 2 ? 0 : 8 * 32 * y_pitch * 4;
    static constexpr bool y_over = 2 * TB::bytes >= y_bytes;
    static constexpr int off_d = off_m + m_bytes + (y_over ? 0 : y_bytes);
    static constexpr int off_y = y_over ? TX::bytes : off_m + m_bytes;
    static_assert(off_y + y_bytes <= off_d, "rows of Y");
    // Blocks per SM: two where shared memory has room.  (fp32 N = 64 with one block, the
    // next chunk's rows ahead in registers: 57 us and 23 for the states of the segments,
    // against 51 and 22; with no more blocks than SMs 112 us against 123.)
    static constexpr int resident = sizeof(IO) == 2 || N <= 64 ? 2 : 1;
    static constexpr int bytes = off_d + 2 * static_cast<int>(sizeof(Decays));
};

__global__ void __launch_bounds__(256) decays_kernel(const DecayArgs a) {
    chain_next();
    const long u = static_cast<long>(blockIdx.x) * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (u >= seg_slots(a.map) * a.H) return;
    const long slot = u / a.H;
    const int h = static_cast<int>(u % a.H);
    int n;
    long r0, r1, lo, hi;
    if (!seg_rows(a.map, slot, n, r0, r1, lo, hi, a.status)) return;
    const long r = r0 + 2 * lane;
    const float dt0 = r < r1 ? load_dt(a.dt, r * a.lddt + h, a.dt_bf16) : 0.f;
    const float dt1 = r + 1 < r1 ? load_dt(a.dt, (r + 1) * a.lddt + h, a.dt_bf16) : 0.f;
    chunk_decays(a.out[u], dt0, dt1, static_cast<int>(r1 - r0), a.A[h], a.bias ? a.bias[h] : 0.f, a.softplus, lane);
}

struct ScanDev {
    const void *x, *Bm, *Cm;
    long ldx, ldb, ldc, ldy;
    const float *D, *s0;
    void* y;
    float *sT, *seg_state, *seg_decay;
    int H, G;
    SegMap map, chunk;  // segments, and the same cut at 64 tokens
    const Decays* dec;  // [chunk][H]
    int* status;
};

// OUT: write y (and C, G, M are formed); otherwise only the segment's end state.
// One segment per sequence (spb == 1 and seg >= T): s0 in, sT out.  Otherwise the
// start state is the slot's in seg_state (OUT) or zero (!OUT, which then writes the
// end state and the decay of the slot).
template <typename IO, int N, bool OUT>
__global__ void __launch_bounds__(kScanThreads, FwdLayout<IO, N>::resident)
    scan_kernel(const ScanDev a, bool whole) {
    chain_wait();
    if constexpr (!OUT) chain_next();
    using LY = FwdLayout<IO, N>;
    using TX = typename LY::TX;
    using TB = typename LY::TB;
    using TM = typename LY::TM;
    constexpr int PI = LY::PI, PC = LY::PC;
    constexpr int NH = N / 2 >= 16 ? N / 2 : 16;  // state columns per warp half (N = 16: the second half has none)
    constexpr int NT = NH / 8;                    // tiles of 8 columns
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    Decays* dec = reinterpret_cast<Decays*>(smem + LY::off_d);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pg = warp & 3, half = warp >> 2;
    const int g8 = lane >> 2, q2 = (lane & 3) * 2;
    const bool has_n = half * NH < N;  // this half has state columns
    const int n0 = has_n ? half * NH : 0;
    const int h = blockIdx.x % a.H, grp = h / (a.H / a.G);  // neighbouring blocks share B and C
    const long slot = blockIdx.x / a.H;

    int n;
    long r0, r1, lo, hi;
    const bool used = seg_rows(a.map, slot, n, r0, r1, lo, hi, a.status);
    if (!used) {
        if (!whole || !a.sT) return;  // an empty sequence passes its state on
        const long e = (static_cast<long>(n) * a.H + h) * kScanP * N;
        for (int i = tid; i < kScanP * N; i += kScanThreads) a.sT[e + i] = a.s0 ? a.s0[e + i] : 0.f;
        return;
    }
    const long seq_state = (static_cast<long>(n) * a.H + h) * kScanP * N;
    const long slot_state = (slot * a.H + h) * kScanP * N;

    const IO* xg = static_cast<const IO*>(a.x) + r0 * a.ldx + h * kScanP;
    const IO* bg = static_cast<const IO*>(a.Bm) + r0 * a.ldb + static_cast<long>(grp) * N;
    const IO* cg = static_cast<const IO*>(a.Cm) + r0 * a.ldc + static_cast<long>(grp) * N;
    const int rows = static_cast<int>(r1 - r0);
    const int chunks = (rows + kChunk - 1) / kChunk;
    const float Dh = a.D ? a.D[h] : 0.f;
    const Decays* dg = a.dec + (seg_first(a.chunk, n, lo) + (r0 - lo) / kChunk) * a.H + h;

    auto stage = [&](int c) { return sb + (c % LY::stages) * LY::stage_bytes; };
    auto count = [&](int c) { return rows - c * kChunk < kChunk ? rows - c * kChunk : kChunk; };
    auto load = [&](int c) {
        const int nr = count(c);
        const uint32_t s = stage(c);
        load_tile<TX, kScanP>(s, xg + static_cast<long>(c) * kChunk * a.ldx, a.ldx, nr, tid, kScanThreads);
        load_tile<TB, N>(s + TX::bytes, bg + static_cast<long>(c) * kChunk * a.ldb, a.ldb, nr, tid, kScanThreads);
        if constexpr (OUT)
            load_tile<TB, N>(s + TX::bytes + TB::bytes, cg + static_cast<long>(c) * kChunk * a.ldc, a.ldc, nr, tid,
                             kScanThreads);
    };
    auto load_decays = [&](int c) {
        cp_decays(sb + LY::off_d + (c & 1) * static_cast<uint32_t>(sizeof(Decays)), dg + static_cast<long>(c) * a.H, tid);
        cp_async_commit();
    };
    if constexpr (LY::stages == 2) load(0);
    load_decays(0);

    // state: S[i] = tile of columns n0 + 8 i; rows 16 pg + g8 (0, 1) and + 8 (2, 3)
    float S[NT][4];
    {
        const float* src = nullptr;
        if (whole)
            src = a.s0 ? a.s0 + seq_state : nullptr;
        else if (OUT)
            src = a.seg_state + slot_state;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float2 u = make_float2(0.f, 0.f), v = u;
            if (src && has_n) {
                const float* p = src + (pg * 16 + g8) * N + n0 + i * 8 + q2;
                u = *reinterpret_cast<const float2*>(p);
                v = *reinterpret_cast<const float2*>(p + 8 * N);
            }
            S[i][0] = u.x, S[i][1] = u.y, S[i][2] = v.x, S[i][3] = v.y;
        }
    }
    float run = 1.f;  // decay of the segment so far

    for (int c = 0; c < chunks; ++c) {
        if constexpr (LY::stages == 2) {
            cp_async_wait<0>();
            __syncthreads();
            if (c + 1 < chunks) {
                load(c + 1);
                load_decays(c + 1);
            }
        } else {
            __syncthreads();  // the last chunk's readers are done
            load(c);
            cp_async_wait<0>();
            __syncthreads();
            if (c + 1 < chunks) load_decays(c + 1);
        }
        const Decays& d = dec[c & 1];
        const uint32_t sx = stage(c), sB = sx + TX::bytes, sC = sB + TB::bytes, sM = sb + LY::off_m;

        if constexpr (OUT) {
            // ---- M: 16 x 16 pieces (tb, ts), ts <= tb
            for (int u = warp; u < 10; u += 8) {
                const int tb = u < 1 ? 0 : u < 3 ? 1 : u < 6 ? 2 : 3, ts = u - tb * (tb + 1) / 2;
                float acc[2][4] = {};
#pragma unroll
                for (int k = 0; k < N; k += 16) {
                    uint32_t fa[PI][4], fb[2][PI][2];
                    frag_a<TB>(fa, sC, tb * 16, k, lane);
                    frag_b<TB>(fb, sB, ts * 16, k, lane);
                    mma_planes<PI, PI>(acc[0], fa, fb[0]);
                    mma_planes<PI, PI>(acc[1], fa, fb[1]);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int t = tb * 16 + g8 + 8 * r, s = ts * 16 + j * 8 + q2;
                        const float m0 = t >= s ? acc[j][2 * r] * decay_between(d, t, s) * d.delta[s] : 0.f;
                        const float m1 =
                            t >= s + 1 ? acc[j][2 * r + 1] * decay_between(d, t, s + 1) * d.delta[s + 1] : 0.f;
                        uint32_t pl[PC];
                        split_pair<PC, PI == 1>(pl, m0, m1);
#pragma unroll
                        for (int p = 0; p < PC; ++p) sts32(sM + p * TM::plane + t * TM::pitch + s * 2, pl[p]);
                    }
            }
        }
        // ---- inter-chunk part of Y^T, from the state before this chunk
        float Y[8][4];
        if constexpr (OUT) {
#pragma unroll
            for (int j = 0; j < 8; ++j) Y[j][0] = Y[j][1] = Y[j][2] = Y[j][3] = 0.f;
            if (has_n) {
#pragma unroll
                for (int kk = 0; kk < NH / 16; ++kk) {
                    uint32_t fa[PC][4], u[PC];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float* s = &S[2 * kk + (r >> 1)][2 * (r & 1)];
                        split_pair<PC, PI == 1>(u, s[0], s[1]);
#pragma unroll
                        for (int p = 0; p < PC; ++p) fa[p][r] = u[p];
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t fb[2][PI][2];
                        frag_b<TB>(fb, sC, j * 16, n0 + kk * 16, lane);
                        mma_planes<PC, PI>(Y[2 * j], fa, fb[0]);
                        mma_planes<PC, PI>(Y[2 * j + 1], fa, fb[1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 f = *reinterpret_cast<const float2*>(&d.from[j * 8 + q2]);
                    Y[j][0] *= f.x, Y[j][1] *= f.y, Y[j][2] *= f.x, Y[j][3] *= f.y;
                }
            }
        }
        // ---- S <- exp(l_64) S + (X^T delta exp(l_64 - l)) B, the product from zero: the tensor cores
        // cut their sums, and a state that was their accumulator lost 2^-23 at every step (1.4e-4
        // of it after 8192 tokens of fp32, 2e-4 of bf16, where little decays)
        run *= d.total;
        if (has_n) {
            float add[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i) add[i][0] = add[i][1] = add[i][2] = add[i][3] = 0.f;
#pragma unroll
            for (int k = 0; k < kChunk; k += 16) {
                uint32_t fx[PI][4], fa[kStatePlanes][4];
                frag_a_t<TX>(fx, sx, pg * 16, k, lane);
                const float2 d0 = *reinterpret_cast<const float2*>(&d.delta[k + q2]);
                const float2 d8 = *reinterpret_cast<const float2*>(&d.delta[k + 8 + q2]);
                const float2 e0 = *reinterpret_cast<const float2*>(&d.to[k + q2]);
                const float2 e8 = *reinterpret_cast<const float2*>(&d.to[k + 8 + q2]);
                scale_frag<PI, kStatePlanes>(fa, fx, d0.x * e0.x, d0.y * e0.y, d8.x * e8.x, d8.y * e8.y);
#pragma unroll
                for (int i = 0; i < NT; i += 2) {
                    uint32_t fb[2][PI][2];
                    frag_b_t<TB>(fb, sB, n0 + i * 8, k, lane);
                    mma_planes<kStatePlanes, PI>(add[i], fa, fb[0]);
                    mma_planes<kStatePlanes, PI>(add[i + 1], fa, fb[1]);
                }
            }
            const float tot = d.total;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[i][e] = fmaf(tot, S[i][e], add[i][e]);
        }
        if constexpr (OUT) {
            __syncthreads();  // M is complete
            // ---- intra-chunk part: token pieces s of 16; the halves take {0, 3} and {1, 2}
#pragma unroll
            for (int kq = 0; kq < 2; ++kq) {
                const int ks = half ? 1 + kq : 3 * kq;
                uint32_t fx[PI][4];
                frag_a_t<TX>(fx, sx, pg * 16, ks * 16, lane);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j < ks) continue;
                    uint32_t fb[2][PC][2];
                    frag_b<TM>(fb, sM, j * 16, ks * 16, lane);
                    mma_planes<PI, PC>(Y[2 * j], fx, fb[0]);
                    mma_planes<PI, PC>(Y[2 * j + 1], fx, fb[1]);
                }
            }
            __syncthreads();  // M has been read: its space takes the exchange
            // ---- the halves meet: each keeps 32 tokens and passes the other 32 on
            float* xc = reinterpret_cast<float*>(smem + LY::off_m);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float4 v;
                v.x = half ? Y[j][0] : Y[4 + j][0], v.y = half ? Y[j][1] : Y[4 + j][1];
                v.z = half ? Y[j][2] : Y[4 + j][2], v.w = half ? Y[j][3] : Y[4 + j][3];
                reinterpret_cast<float4*>(xc)[(warp * 4 + j) * 32 + lane] = v;
            }
            asm volatile("bar.sync %0, 64;" ::"r"(1 + pg) : "memory");
            float Z[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 v = reinterpret_cast<const float4*>(xc)[((warp ^ 4) * 4 + j) * 32 + lane];
                Z[j][0] = v.x + (half ? Y[4 + j][0] : Y[j][0]), Z[j][1] = v.y + (half ? Y[4 + j][1] : Y[j][1]);
                Z[j][2] = v.z + (half ? Y[4 + j][2] : Y[j][2]), Z[j][3] = v.w + (half ? Y[4 + j][3] : Y[j][3]);
            }
            // ---- + D x, and out: rows of 16 channels of this warp's 32 tokens
            const int t0 = half * 32, left = rows - c * kChunk;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t fx[PI][4];
                frag_a_t<TX>(fx, sx, pg * 16, t0 + k * 16, lane);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float xl = 0.f, xh = 0.f;
#pragma unroll
                    for (int p = PI - 1; p >= 0; --p) {
                        xl += bf_lo(fx[p][r]);
                        xh += bf_hi(fx[p][r]);
                    }
                    float* z = &Z[2 * k + (r >> 1)][2 * (r & 1)];
                    z[0] = fmaf(Dh, xl, z[0]);
                    z[1] = fmaf(Dh, xh, z[1]);
                }
            }
            IO* yg = static_cast<IO*>(a.y) + (r0 + static_cast<long>(c) * kChunk + t0) * a.ldy + h * kScanP + pg * 16;
            if constexpr (sizeof(IO) == 2) {
                // transposed into this pair's rows of the exchange area that only this warp has read
                const uint32_t st = sb + LY::off_m + (warp ^ 4) * 2048;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    // rows t of tile j: 16 channels = 32 bytes each, at a pitch of 48
                    stsm2t(st + (j * 8 + (lane & 7)) * 48 + ((lane >> 3) & 1) * 16, pack_bf16(Z[j][0], Z[j][1]),
                           pack_bf16(Z[j][2], Z[j][3]));
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = i * 16 + (lane >> 1);
                    uint4 v;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(st + t * 48 + (lane & 1) * 16)
                                 : "memory");
                    if (t0 + t < left) *reinterpret_cast<uint4*>(yg + t * a.ldy + (lane & 1) * 8) = v;
                }
            } else {
                float* st = reinterpret_cast<float*>(smem + LY::off_y) + warp * 32 * LY::y_pitch;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        st[(j * 8 + q2 + (e & 1)) * LY::y_pitch + g8 + 8 * (e >> 1)] = Z[j][e];
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = i * 8 + (lane >> 2);
                    if (t0 + t < left)
                        *reinterpret_cast<float4*>(yg + t * a.ldy + (lane & 3) * 4) =
                            *reinterpret_cast<const float4*>(st + t * LY::y_pitch + (lane & 3) * 4);
                }
            }
        }
    }

    // ---- the end state
    float* dst = nullptr;
    if (whole)
        dst = a.sT ? a.sT + seq_state : nullptr;
    else if (!OUT)
        dst = a.seg_state + slot_state;
    if (dst && has_n) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float* p = dst + (pg * 16 + g8) * N + n0 + i * 8 + q2;
            *reinterpret_cast<float2*>(p) = make_float2(S[i][0], S[i][1]);
            *reinterpret_cast<float2*>(p + 8 * N) = make_float2(S[i][2], S[i][3]);
        }
    }
    if (!OUT && !whole && tid == 0) a.seg_decay[slot * a.H + h] = run;
}

// Start states of the segments from their end states (from zero) and decays, in place,
// and the final states: thread = 4 elements of a head's state, walking its segments.
__global__ void __launch_bounds__(256) scan_join_kernel(const ScanDev a, int elems) {
    chain_wait();
    chain_next();
    const int h = blockIdx.x % a.H;
    const long n = blockIdx.x / a.H;
    const int e = (blockIdx.y * 256 + threadIdx.x) * 4;
    if (e >= elems) return;
    long lo, hi;
    seq_span(a.map.offs, static_cast<int>(n), a.map.T, lo, hi, a.status);
    const long first = seg_first(a.map, static_cast<int>(n), lo), cnt = (hi - lo + a.map.seg - 1) / a.map.seg;
    const long st = (n * a.H + h) * elems + e;
    float4 S = a.s0 ? *reinterpret_cast<const float4*>(a.s0 + st) : make_float4(0.f, 0.f, 0.f, 0.f);
    auto at = [&](long i) { return reinterpret_cast<float4*>(a.seg_state + ((first + i) * a.H + h) * elems + e); };
    for (long i = 0; i < cnt; i += 4) {  // four segments' loads before the first is used
        float4 v[4];
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < cnt) {
                v[k] = *at(i + k);
                f[k] = a.seg_decay[(first + i + k) * a.H + h];
            }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < cnt) {
                *at(i + k) = S;
                S.x = fmaf(f[k], S.x, v[k].x), S.y = fmaf(f[k], S.y, v[k].y);
                S.z = fmaf(f[k], S.z, v[k].z), S.w = fmaf(f[k], S.w, v[k].w);
            }
    }
    if (a.sT) *reinterpret_cast<float4*>(a.sT + st) = S;
}

// ---------------------------------------------------------------- single tokens
// Block = one (sequence, head): N / 4 lanes hold one row of the state, four columns
// each; every element is read once, updated, used for y and written.  s_out may be s_in.
// Bound by the states' traffic: B256 H40 N128 (671 MB) 99.9 us, 6.7 TB/s; of one sequence
// (H32) 2.8 us, a launch and the latency of two dependent loads.
template <typename IO, int N>
__global__ void __launch_bounds__(256)
    scan_step_kernel(const IO* __restrict__ x, long ldx, const void* __restrict__ dt, long lddt, int dt_bf16,
                     const float* __restrict__ A, const IO* __restrict__ Bm, long ldb, const IO* __restrict__ Cm,
                     long ldc, const float* __restrict__ D, const float* __restrict__ bias, const float* s_in,
                     IO* __restrict__ y, long ldy, float* s_out, int H, int G, int softplus) {
    constexpr int LR = N / 4, RW = 32 / LR, ROWS = 8 * RW, PASS = kScanP / ROWS > 0 ? kScanP / ROWS : 1;
    const int h = blockIdx.x % H;
    const long n = blockIdx.x / H;
    const int tid = threadIdx.x, sub = tid / LR, col = (tid % LR) * 4;
    const long base = (n * H + h) * static_cast<long>(kScanP) * N;
    float4 S[PASS];
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
        const int p = i * ROWS + sub;
        S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (s_in && p < kScanP) S[i] = *reinterpret_cast<const float4*>(s_in + base + p * N + col);
    }
    const int grp = h / (H / G);
    float b[4], c[4];
    load_vec<4>(b, Bm + n * ldb + static_cast<long>(grp) * N + col);
    load_vec<4>(c, Cm + n * ldc + static_cast<long>(grp) * N + col);
    float delta = load_dt(dt, n * lddt + h, dt_bf16) + (bias ? bias[h] : 0.f);
    if (softplus) delta = softplus_f32(delta);
    const float da = expf(delta * A[h]), Dh = D ? D[h] : 0.f;
#pragma unroll
    for (int i = 0; i < PASS; ++i) {
        const int p = i * ROWS + sub;
        const float xp = p < kScanP ? to_f32(x[n * ldx + h * kScanP + p]) : 0.f;
        const float u = delta * xp;
        S[i].x = fmaf(da, S[i].x, u * b[0]), S[i].y = fmaf(da, S[i].y, u * b[1]);
        S[i].z = fmaf(da, S[i].z, u * b[2]), S[i].w = fmaf(da, S[i].w, u * b[3]);
        float o = fmaf(S[i].x, c[0], fmaf(S[i].y, c[1], fmaf(S[i].z, c[2], S[i].w * c[3])));
#pragma unroll
        for (int m = LR / 2; m >= 1; m >>= 1) o += __shfl_xor_sync(0xffffffffu, o, m);
        if (p < kScanP) {
            *reinterpret_cast<float4*>(s_out + base + p * N + col) = S[i];
            if (tid % LR == 0) y[n * ldy + h * kScanP + p] = from_f32<IO>(fmaf(Dh, xp, o));
        }
    }
}

// The kernels: this file's on warp-level products, one block per SM for fp32 with N = 128
// and two otherwise, and wkv7_scan_tc.cu's.  (At B1 T16384 H40 N128 a chunk of 128 tokens
// takes the latter 3.8 us with its outputs and 1.8 without.)
constexpr CutCost kCutWarp{kChunk, 2, 1.4, 0.5, 0.5, 2.0};
constexpr CutCost kCutTc{128, 1, 1.0, 0.5, 1.5, 2.0};
constexpr CutCost kCutWarpF32{kChunk, 2, 1.7, 0.5, 0.5, 1.0}, kCutWarpF32Large{kChunk, 1, 1.0, 0.5, 1.0, 1.0};  // large: N = 128
const CutCost& cut_cost(int io_dtype, int N) {
    return io_dtype == WKV7_BF16 ? N == 128 ? kCutTc : kCutWarp : N == 128 ? kCutWarpF32Large : kCutWarpF32;
}
// bf16 with N = 128 runs on the tcgen05 kernel: B4 T1024 H32 takes 35 us there and took 114 on this
// file's.  It is written for tiles of 128 columns.  N = 64 takes 64 us here (96 with the L2
// flushed), so even half-empty tiles of it would be faster there, which is not built; fp32 rows
// would be three planes of each operand in its shared memory.
bool uses_tc(int io_dtype, int N) { return io_dtype == WKV7_BF16 && N == 128; }

template <typename IO, int N>
cudaError_t scan_typed(const ScanArgs& p, const SegMap& map, bool whole, ScanDev& d, cudaStream_t st) {
    using LY = FwdLayout<IO, N>;
    static std::atomic<unsigned long long> cfg_out{0}, cfg_state{0};
    cudaError_t e = configure_smem_once(scan_kernel<IO, N, true>, LY::bytes, cfg_out);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(seg_slots(map) * p.H);
    if (!whole) {
        e = configure_smem_once(scan_kernel<IO, N, false>, LY::bytes, cfg_state);
        if (e != cudaSuccess) return e;
        launch_next(scan_kernel<IO, N, false>, grid, kScanThreads, LY::bytes, st, d, false);
        constexpr int elems = kScanP * N;
        launch_next(scan_join_kernel, dim3(static_cast<unsigned>(p.B) * p.H, (elems / 4 + 255) / 256), 256, 0, st, d, elems);
    }
    launch_next(scan_kernel<IO, N, true>, grid, kScanThreads, LY::bytes, st, d, whole);
    return cudaGetLastError();
}

}  // namespace

// Sequences are cut into segments where that is faster: blocks of one segment each run in
// waves, and a cut needs a pass over the states and the join first.  Of packed sequences
// only the mean length is known here; the longest is taken to have twice that.  (fp32
// packed [5003] rows in nine sequences, H12 N64: 86 us in segments of four chunks, 145 whole.
// bf16 B4 T1024 H32 N64: 64 us whole, 74 in two segments; B1 T4096 H40 N64: 90 us in seven,
// 115 in three.)
SegMap scan_segments(int B, int T, int H, const int32_t* offs, bool packed, const CutCost& k) {
    SegMap m{offs, B, T, 0, 1};
    const long total = (static_cast<long>(T) + k.chunk - 1) / k.chunk, units = static_cast<long>(B) * H;
    const long mean = packed ? (total + B - 1) / B : total, chunks = std::min(total, packed && B > 1 ? 2 * mean : mean);
    const long sms = 148, resident = sms * k.per_sm;
    const auto waves = [&](long blocks) { return blocks <= sms ? 1.0 : (blocks + resident - 1) / resident * k.share; };
    long best = 1;
    double least = std::max(waves(units) * (mean + k.start), chunks + k.start);
    for (long s = 2; s <= chunks && s <= 64 && units * s <= 8 * resident; ++s) {
        const long c = (chunks + s - 1) / s;
        // half of the sequences' last segments count as full ones
        const double w = waves(packed ? (2 * total + c * B) * H / (2 * c) : units * s);
        const double t = w * (c * (1.0 + k.states) + 2 * k.start) + k.join;
        if (t < least) {
            least = t;
            best = s;
        }
    }
    if (best == 1) {
        m.seg = total * k.chunk;
        if (m.seg == 0) m.seg = k.chunk;
        return m;
    }
    m.seg = (chunks + best - 1) / best * k.chunk;
    m.spb = static_cast<int>((T + m.seg - 1) / m.seg);
    return m;
}

cudaError_t launch_decays(const DecayArgs& a, cudaStream_t stream) {
    const long warps = seg_slots(a.map) * a.H;
    if (warps > 0) decays_kernel<<<static_cast<unsigned>((warps + 7) / 8), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

SegMap chunk_map(int B, int T, const int32_t* offs) { return SegMap{offs, B, T, kChunk, (T + kChunk - 1) / kChunk}; }
long chunk_slots(int B, int T, bool packed) {
    return packed && T > kChunk ? T / kChunk + B : static_cast<long>(B) * ((static_cast<long>(T) + kChunk - 1) / kChunk);
}

// The segments' states and decays of either kernel (the size query does not know the io
// type), and the chunks' decays of this file's.
static size_t cut_floats(int B, int T, int H, int N, bool packed, const CutCost& cost) {
    const SegMap m = scan_segments(B, T, H, nullptr, packed, cost);
    if (m.seg >= T) return 0;
    const long slots = packed ? T / m.seg + B : static_cast<long>(B) * m.spb;
    return static_cast<size_t>(slots) * H * (static_cast<size_t>(kScanP) * N + 4);
}
static size_t decays_bytes(int B, int T, int H, bool packed) {
    return static_cast<size_t>(chunk_slots(B, T, packed)) * H * sizeof(Decays);
}
size_t scan_workspace_bytes(int B, int T, int H, int N, bool packed) {
    const size_t b = cut_floats(B, T, H, N, packed, cut_cost(WKV7_BF16, N));
    const size_t f = cut_floats(B, T, H, N, packed, cut_cost(WKV7_F32, N));
    return (b > f ? b : f) * sizeof(float) + decays_bytes(B, T, H, packed);
}

cudaError_t launch_scan(const ScanArgs& p, int io_dtype, cudaStream_t stream) {
    const bool packed = p.seq_offsets != nullptr;
    const bool tc = uses_tc(io_dtype, p.N);
    const SegMap map = scan_segments(p.B, p.T, p.H, p.seq_offsets, packed, cut_cost(io_dtype, p.N));
    const bool whole = map.seg >= p.T;
    uint8_t* ws = static_cast<uint8_t*>(p.ws);
    Decays* dec = reinterpret_cast<Decays*>(ws);
    if (!tc) ws += decays_bytes(p.B, p.T, p.H, packed);
    float* seg_state = reinterpret_cast<float*>(ws);
    float* seg_decay = whole ? nullptr : seg_state + static_cast<size_t>(seg_slots(map)) * p.H * kScanP * p.N;
    ScanDev d{p.x, p.Bm, p.Cm, p.ldx, p.ldb, p.ldc, p.ldy, p.D, p.s0, p.y, p.sT, seg_state, seg_decay, p.H, p.G,
              map, chunk_map(p.B, p.T, p.seq_offsets), dec, p.status};
    if (tc) {
        cudaError_t e = cudaSuccess;
        if (!whole) {
            e = launch_scan_tc(p, map, false, false, seg_state, seg_decay, stream);
            if (e != cudaSuccess) return e;
            constexpr int elems = kScanP * 128;
            launch_next(scan_join_kernel, dim3(static_cast<unsigned>(p.B) * p.H, elems / 4 / 256), 256, 0, stream, d, elems);
        }
        return launch_scan_tc(p, map, whole, true, seg_state, seg_decay, stream);
    }
    const cudaError_t e = launch_decays(DecayArgs{p.dt, p.lddt, p.A, p.dt_bias, dec, p.H, p.softplus,
                                                  p.dt_dtype == WKV7_BF16, d.chunk, p.status},
                                        stream);
    if (e != cudaSuccess) return e;
    if (io_dtype == WKV7_BF16) switch (p.N) {
            case 16: return scan_typed<__nv_bfloat16, 16>(p, map, whole, d, stream);
            case 32: return scan_typed<__nv_bfloat16, 32>(p, map, whole, d, stream);
            default: return scan_typed<__nv_bfloat16, 64>(p, map, whole, d, stream);
        }
    switch (p.N) {
        case 16: return scan_typed<float, 16>(p, map, whole, d, stream);
        case 32: return scan_typed<float, 32>(p, map, whole, d, stream);
        case 64: return scan_typed<float, 64>(p, map, whole, d, stream);
        default: return scan_typed<float, 128>(p, map, whole, d, stream);
    }
}

template <typename IO, int N>
static void step_typed(const ScanArgs& p, cudaStream_t st) {
    scan_step_kernel<IO, N><<<static_cast<unsigned>(static_cast<long>(p.B) * p.H), 256, 0, st>>>(
        static_cast<const IO*>(p.x), p.ldx, p.dt, p.lddt, p.dt_dtype == WKV7_BF16, p.A,
        static_cast<const IO*>(p.Bm), p.ldb, static_cast<const IO*>(p.Cm), p.ldc, p.D, p.dt_bias, p.s0,
        static_cast<IO*>(p.y), p.ldy, p.sT, p.H, p.G, p.softplus);
}

cudaError_t launch_scan_step(const ScanArgs& p, int io_dtype, cudaStream_t stream) {
    const bool bf = io_dtype == WKV7_BF16;
    switch (p.N) {
        case 16: bf ? step_typed<__nv_bfloat16, 16>(p, stream) : step_typed<float, 16>(p, stream); break;
        case 32: bf ? step_typed<__nv_bfloat16, 32>(p, stream) : step_typed<float, 32>(p, stream); break;
        case 64: bf ? step_typed<__nv_bfloat16, 64>(p, stream) : step_typed<float, 64>(p, stream); break;
        default: bf ? step_typed<__nv_bfloat16, 128>(p, stream) : step_typed<float, 128>(p, stream); break;
    }
    return cudaGetLastError();
}

}  // namespace wkv7
