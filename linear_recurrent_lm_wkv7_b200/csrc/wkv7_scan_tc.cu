// wkv7_scan_tc.cu — selective scan of bf16 prompts with N = 128 on the tcgen05 tensor
// cores.  The recurrence, its chunk form and the decays: scan_common.cuh; here a chunk
// has 128 tokens.
//
// A block carries the state of one head through the chunks of one segment.  Per chunk:
//   (1) G  = C B^T                      128 t x 128 s, K = 128
//       M_ts = G_ts exp(l_t - l_s) delta_s, rounded to two bf16 planes in tensor memory
//   (2) D1 = C S^T                      128 t x 2 x 64 p, K = 128, S as two bf16 planes side by side
//   (3) D2 = M X                        128 t x 64 p, K = 128, A operand M from tensor memory
//       y_t = exp(l_t) D1_t + D2_t + D x_t
//   (4) D3 = B^T (X delta exp(l_128 - l))   128 n x 64 p, K = 128, the scaled x as three planes
//       S <- exp(l_128) S + D3, in fp32 registers (lane n, 64 rows p)
// Only (2) waits for the state, and the state only for (4): G, M and (4) of the next
// chunk run ahead of it.  The outputs round to bf16, so two planes (2^-16) do for M and
// the S of (2); the state stays fp32 and takes three.  D3 starts from zero at every chunk
// and is added in fp32: the tensor cores cut their sums, and a state that was their
// accumulator would lose 2^-23 at every step of a long sequence.
//
// 24 warps, each on one job, in step through mbarriers:
//   0-7   M from G (row t per lane; the 32 x 32 blocks of the lower triangle, shared by two warps)
//   8-15  the state (lane n, half of p each), its planes, and y (lane t)
//   16-18, 20  the scaled x, in pieces of 32 tokens through a ring of two
//   19    loads (TMA);   21 issues every product;   22, 23 the decays of every other chunk
//         (thousands of cycles of dependent steps each, hence two, and three chunks' room)
// Lanes 32 (w % 4) .. of tensor memory belong to warps w, and so does the SM's quarter that
// they issue on: warps 3 and 7 make four blocks of M, warps 0 and 4 one.  The jobs that
// touch no tensor memory are therefore put on the first quarters.
//
// Measured: B4 T1024 H32 35.3 us (128 blocks of eight chunks), B1 T16384 H40 145 us + 69 for
// the states of its segments.  Per chunk the products alone take some 3000 cycles of 8000:
// tensor pipe 31 %, issue slots 45 %; the rest is the chain state -> planes -> (2) -> y, whose
// warps also round and store, and instructions fetched again (24 warps on six programs).
#include <cuda.h>

#include "scan_backward.cuh"
#include "tma_host.cuh"

namespace wkv7 {
namespace {

constexpr int kL = 128;         // tokens per chunk
constexpr int kN = 128;         // columns of the state
constexpr int kWarpS = 8, kWarpX = 16, kWarpLoad = 19, kWarpMma = 21, kWarpDec = 22;
constexpr int kTcThreads = 24 * 32;
constexpr int kDecs = 3;  // chunks whose decays are kept
constexpr int kHalf = kScanP / 2;
// A wait gives up after kPolls polls of kPollNs: two seconds and more.  (A loop of its own,
// and not the timed wait of sm100_ptx.cuh: there are dozens of waits, and with the clock's
// reading in each the kernel's loops outgrew the instruction cache.)
constexpr uint32_t kPollNs = 1000, kPolls = 1u << 21;

constexpr uint32_t kTile = kL * 128;         // 128 rows of 128 bytes (64 bf16): one atom column
constexpr uint32_t kStage = kTile + 4 * kTile;  // X, B (two atoms), C (two atoms)
constexpr uint32_t kOffS = 2 * kStage;       // two planes of S^T: rows n, 64 p
constexpr uint32_t kPiece = 32 * 128;        // 32 tokens of scaled x, one plane
constexpr uint32_t kOffXw = kOffS + 2 * kTile;
// the pass that only makes states has no planes of S: its ring starts there and holds four
constexpr uint32_t kOffXwStates = kOffS;
constexpr uint32_t kOffDec = kOffXw + 2 * 3 * kPiece;
static_assert(kOffXwStates + 4 * 3 * kPiece <= kOffDec, "the ring of four");

struct Decays128 {
    float delta[kL], hi[kL], lo[kL];  // hi + lo = -l_t log2(e): negated, to be added
    float from[kL];                   // exp(l_t)
    float w[kL];                      // delta_t exp(l_128 - l_t)
    float total, pad[3];
};
constexpr uint32_t kOffBar = kOffDec + kDecs * sizeof(Decays128);
struct Bars {
    uint64_t full[3], empty[3], dec_full[kDecs], dec_empty[kDecs], xw_full[4], xw_empty[4];
    uint64_t d3_full[2], d3_empty[2], g_full, m_full, s_full, d1_full, d2_full, d_empty, fin;
    uint32_t tmem;
};
constexpr uint32_t kTcSmem = kOffBar + sizeof(Bars) + 1024;  // + alignment of the tiles
static_assert(kTcSmem <= 227 * 1024, "shared memory of an SM");

// tensor memory columns
constexpr uint32_t kColG = 0, kColM = 128, kColD1 = 256, kColD2 = 384, kColD3 = 448;  // D1: one half per plane of S

constexpr uint32_t kIdG = idesc_f32acc(1, 128, 128, 0, 0);
constexpr uint32_t kId1 = idesc_f32acc(1, 128, 128, 0, 1);  // A K-major, B rows are K: both planes of S
constexpr uint32_t kIdY = idesc_f32acc(1, 128, 64, 0, 1);   // A from tensor memory, B rows are K
constexpr uint32_t kIdS = idesc_f32acc(1, 128, 64, 1, 1);   // both rows are K

__device__ __forceinline__ void tma_load_2d(void* dst, const void* map, uint64_t* bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// One lane of the warp, always the same.  The products' warp runs converged and only the
// instructions themselves are that lane's: their descriptors then stay in uniform
// registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(p));
    return p != 0;
}
// d (+)= a b: A from shared memory, or from tensor memory
__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)));
}
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)));
}
// 16 columns of this lane; several loads, then one wait that their results go through.
__device__ __forceinline__ void tmem_load16(uint32_t taddr, float (&f)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]),
          "=f"(f[8]), "=f"(f[9]), "=f"(f[10]), "=f"(f[11]), "=f"(f[12]), "=f"(f[13]), "=f"(f[14]), "=f"(f[15])
        : "r"(taddr)
        : "memory");
}
// Waits for the loads; the values may only be used behind it.
__device__ __forceinline__ void tmem_wait(float (&f)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(f[0]), "+f"(f[1]), "+f"(f[2]), "+f"(f[3]), "+f"(f[4]), "+f"(f[5]), "+f"(f[6]), "+f"(f[7]),
                   "+f"(f[8]), "+f"(f[9]), "+f"(f[10]), "+f"(f[11]), "+f"(f[12]), "+f"(f[13]), "+f"(f[14]),
                   "+f"(f[15])::"memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t taddr, const uint32_t (&f)[8]) {
    __syncwarp();
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(f[0]),
        "r"(f[1]), "r"(f[2]), "r"(f[3]), "r"(f[4]), "r"(f[5]), "r"(f[6]), "r"(f[7]), "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptors of a tile: K-major (rows are M or N, two atom columns), or with K as rows and
// `lbo` bytes between the atom columns.  The address field counts 16 bytes, so K-step k
// (16 elements) is an addition of a constant: the one thread that issues the products has
// no time to build descriptors.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) { return sdesc_sw128(addr, 16, 1024); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t lbo) { return sdesc_sw128(addr, lbo, 1024); }
// from K-step k to the next: 32 bytes on, or from the first atom column's last to the second's first
__host__ __device__ constexpr uint64_t next_k(int k) { return k == 3 ? (kTile >> 4) - 6 : 2; }
__host__ __device__ constexpr uint64_t step_mn(int k) { return k * 128; }
__host__ __device__ constexpr uint64_t at(uint32_t bytes) { return bytes >> 4; }  // further on in shared memory

struct TcMaps {
    CUtensorMap x, b, c;
};
struct TcArgs {
    const void* dt;
    long lddt, ldy;
    const float *A, *D, *bias, *s0;
    __nv_bfloat16* y;
    float *sT, *seg_state, *seg_decay;
    int H, G, softplus, dt_bf16;
    SegMap map;
    int* status;
};

// Warp: the decays of a chunk from the raw dt of tokens 4 lane .. 4 lane + 3.
__device__ __forceinline__ void chunk_decays128(Decays128& d, const float (&dt)[4], int n, float A, float bias,
                                                bool softplus, int lane) {
    const Pair rate = log2_rate(A);
    float e[4];
    Pair l[4], run{0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        e[i] = dt[i] + bias;
        if (softplus) e[i] = softplus_f32(e[i]);
        if (4 * lane + i >= n) e[i] = 0.f;
        run = pair_add(run, pair_mul(e[i], rate));
        l[i] = run;
    }
    run = pair_scan(run, lane);
    Pair before{__shfl_up_sync(0xffffffffu, run.h, 1), __shfl_up_sync(0xffffffffu, run.l, 1)};
    if (lane == 0) before = {0.f, 0.f};
    const Pair end{__shfl_sync(0xffffffffu, run.h, 31), __shfl_sync(0xffffffffu, run.l, 31)};
    float hi[4], lo[4], from[4], w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Pair c = pair_add(before, l[i]);
        hi[i] = c.h;
        lo[i] = c.l;
        from[i] = exp2_pair(c.h, c.l);
        w[i] = e[i] * exp2_diff(end.h, end.l, c.h, c.l);
    }
    *reinterpret_cast<float4*>(&d.delta[4 * lane]) = make_float4(e[0], e[1], e[2], e[3]);
    *reinterpret_cast<float4*>(&d.hi[4 * lane]) = make_float4(-hi[0], -hi[1], -hi[2], -hi[3]);
    *reinterpret_cast<float4*>(&d.lo[4 * lane]) = make_float4(-lo[0], -lo[1], -lo[2], -lo[3]);
    *reinterpret_cast<float4*>(&d.from[4 * lane]) = make_float4(from[0], from[1], from[2], from[3]);
    *reinterpret_cast<float4*>(&d.w[4 * lane]) = make_float4(w[0], w[1], w[2], w[3]);
    if (lane == 31) d.total = exp2_pair(end.h, end.l);
}

// OUT, whole: as in scan_kernel (wkv7_scan.cu).
template <bool OUT>
__global__ void __launch_bounds__(kTcThreads, 1)
    scan_tc_kernel(const TcArgs a, bool whole, const __grid_constant__ TcMaps maps) {
    if constexpr (OUT)
        chain_wait();
    else
        chain_next();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    Bars& bar = *reinterpret_cast<Bars*>(sm + kOffBar);
    Decays128* dec = reinterpret_cast<Decays128*>(sm + kOffDec);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same for all lanes, and known to be
    const int h = blockIdx.x % a.H, grp = h / (a.H / a.G);
    const long slot = blockIdx.x / a.H;
    constexpr long kState = static_cast<long>(kScanP) * kN;
    // the pass over states loads less and keeps less: deeper rings
    constexpr int kStages = OUT ? 2 : 3, kRing = OUT ? 2 : 4, kD3s = OUT ? 1 : 2;
    constexpr uint32_t kStageBytes = OUT ? kStage : 3 * kTile;
    static_assert(kStages * kStageBytes <= kOffS, "the stages");
    constexpr uint32_t kXw = OUT ? kOffXw : kOffXwStates;

    int n;
    long r0, r1, lo, hi;
    if (!seg_rows(a.map, slot, n, r0, r1, lo, hi, a.status)) {
        if (!whole || !a.sT) return;  // an empty sequence passes its state on
        const long e = (static_cast<long>(n) * a.H + h) * kState;
        for (int i = tid; i < kState; i += kTcThreads) a.sT[e + i] = a.s0 ? a.s0[e + i] : 0.f;
        return;
    }
    const long seq_state = (static_cast<long>(n) * a.H + h) * kState;
    const long slot_state = (slot * a.H + h) * kState;
    const int rows = static_cast<int>(r1 - r0), chunks = (rows + kL - 1) / kL;
    auto count = [&](int c) { return rows - c * kL < kL ? rows - c * kL : kL; };

    if (warp == kWarpMma) {
        if (lane == 0) {
            for (int i = 0; i < kStages; ++i) {
                mbar_init(&bar.full[i], 1);
                mbar_init(&bar.empty[i], OUT ? 9 : 1);
            }
            for (int i = 0; i < kD3s; ++i) {
                mbar_init(&bar.d3_full[i], 1);
                mbar_init(&bar.d3_empty[i], 8);
            }
            for (int i = 0; i < kRing; ++i) {
                mbar_init(&bar.xw_full[i], 4);
                mbar_init(&bar.xw_empty[i], 1);
            }
            for (int i = 0; i < kDecs; ++i) {
                mbar_init(&bar.dec_full[i], 1);
                mbar_init(&bar.dec_empty[i], 20);  // every warp of M, S and x
            }
            mbar_init(&bar.g_full, 1);
            mbar_init(&bar.m_full, 8);
            mbar_init(&bar.s_full, 8);
            mbar_init(&bar.d1_full, 1);
            mbar_init(&bar.d2_full, 1);
            mbar_init(&bar.d_empty, 8);
            mbar_init(&bar.fin, 1);
            fence_mbar_init();
        }
        tmem_alloc(&bar.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = bar.tmem;
    const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // lanes 32 (warp % 4) ..
    bool ok = true;
    // Waits for phase number `k` (0, 1, ..) of a barrier: the warp goes on or gives up as one.
    auto wait = [&](uint64_t& b, int k) {
        for (uint32_t i = 0; ok && !__all_sync(0xffffffffu, mbar_try_wait_sleep(&b, k & 1, kPollNs)); ++i)
            ok = i < kPolls;
    };
    auto signal = [&](uint64_t& b) {  // once per warp
        __syncwarp();
        if (lane == 0) arrive(&b);
    };

    if (OUT && warp < kWarpS) {
        // ------------------------------------------------------------ M from G
        if constexpr (OUT) {
            const int q = warp & 3, half = warp >> 2;
            const int t = 32 * q + lane;
            const uint32_t tG = tm + lane_base + kColG, tM = tm + lane_base + kColM;
            {  // the blocks above the diagonal are zero for good
                const uint32_t z[8] = {};
                for (int j = half; j < 4; j += 2)
                    if (j > q)
                        for (int i = 0; i < 16; i += 8) {
                            tmem_store8(tM + 16 * j + i, z);
                            tmem_store8(tM + 64 + 16 * j + i, z);
                        }
                tmem_store_wait();
            }
            for (int c = 0; c < chunks && ok; ++c) {
                wait(bar.dec_full[c % kDecs], c / kDecs);
                // G of this chunk comes after (3) of the last one on the tensor cores, so M is free too
                wait(bar.g_full, c);
                if (!ok) break;
                tc_fence_after();
                const Decays128& d = dec[c % kDecs];
                // the columns' parts are stored negated
                const float2 ht = make_float2(-d.hi[t], -d.hi[t]), lt = make_float2(-d.lo[t], -d.lo[t]);
                // pieces of 16 columns: two to a block of 32, blocks half, half + 2 up to q
                const int pieces = q >= half ? 2 * ((q - half) / 2 + 1) : 0;
                auto col = [&](int i) { return 32 * (half + 2 * (i >> 1)) + 16 * (i & 1); };
                float g[16], nx[16];
                __syncwarp();
                if (pieces) tmem_load16(tG + col(0), nx);
#pragma unroll 1
                for (int i = 0; i < pieces; ++i) {
                    const int s0 = col(i);
                    tmem_wait(nx);
#pragma unroll
                    for (int e = 0; e < 16; ++e) g[e] = nx[e];
                    if (i + 1 < pieces) tmem_load16(tG + col(i + 1), nx);
                    uint32_t p0[8], p1[8];
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const int s = s0 + k;
                        const float4 hs = *reinterpret_cast<const float4*>(&d.hi[s]);
                        const float4 ls = *reinterpret_cast<const float4*>(&d.lo[s]);
                        const float4 ds = *reinterpret_cast<const float4*>(&d.delta[s]);
                        float m[4];
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float2 x = add2(add2(ht, e ? make_float2(hs.z, hs.w) : make_float2(hs.x, hs.y)),
                                                  add2(lt, e ? make_float2(ls.z, ls.w) : make_float2(ls.x, ls.y)));
                            const float2 v = mul2(mul2(make_float2(ex2_ftz(x.x), ex2_ftz(x.y)),
                                                       e ? make_float2(ds.z, ds.w) : make_float2(ds.x, ds.y)),
                                                  make_float2(g[k + e], g[k + e + 1]));
                            m[e] = v.x, m[e + 1] = v.y;
                        }
                        if (s0 + 16 > 32 * q) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) m[e] = s + e <= t ? m[e] : 0.f;
                        }
                        uint32_t u[2];
                        split_pair<2>(u, m[0], m[1]);
                        p0[k / 2] = u[0], p1[k / 2] = u[1];
                        split_pair<2>(u, m[2], m[3]);
                        p0[k / 2 + 1] = u[0], p1[k / 2 + 1] = u[1];
                    }
                    tmem_store8(tM + s0 / 2, p0);
                    tmem_store8(tM + 64 + s0 / 2, p1);
                }
                tmem_store_wait();
                tc_fence_before();
                signal(bar.m_full);
                signal(bar.dec_empty[c % kDecs]);
            }
        }
    } else if (warp >= kWarpS && warp < kWarpX) {
        // ------------------------------------------------------------ the state and y
        const int row = 32 * (warp & 3) + lane;       // column n of the state; token t of y
        const int p0 = warp >= kWarpS + 4 ? kHalf : 0;  // this warp's rows p of the state and channels of y
        float S[kHalf];
        {
            const float* src = whole ? (a.s0 ? a.s0 + seq_state : nullptr) : OUT ? a.seg_state + slot_state : nullptr;
#pragma unroll
            for (int p = 0; p < kHalf; ++p) S[p] = src ? src[(p0 + p) * kN + row] : 0.f;
        }
        auto write_planes = [&]() {  // S^T: row n, 64 p, swizzled, for (2)
#pragma unroll
            for (int i = 0; i < kHalf; i += 8) {
                uint32_t u[4][2];
#pragma unroll
                for (int e = 0; e < 4; ++e) split_pair<2>(u[e], S[i + 2 * e], S[i + 2 * e + 1]);
                const uint32_t o = swz(row, (p0 + i) * 2, kN);
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    *reinterpret_cast<uint4*>(sm + kOffS + p * kTile + o) = make_uint4(u[0][p], u[1][p], u[2][p], u[3][p]);
            }
            fence_proxy_async_smem();
            signal(bar.s_full);
        };
        if constexpr (OUT) write_planes();
        const float Dh = OUT && a.D ? a.D[h] : 0.f;
        float run = 1.f;
        for (int c = 0; c < chunks && ok; ++c) {
            const Decays128& d = dec[c % kDecs];
            wait(bar.dec_full[c % kDecs], c / kDecs);
            wait(bar.d3_full[c % kD3s], c / kD3s);
            if (!ok) break;
            tc_fence_after();
            const float tot = d.total, f = d.from[row];
            signal(bar.dec_empty[c % kDecs]);
            run *= tot;
            {
                const uint32_t d3 = tm + lane_base + kColD3 - (c % kD3s) * 64;
                float v[2][16];
                __syncwarp();
                tmem_load16(d3 + p0, v[0]);
                tmem_load16(d3 + p0 + 16, v[1]);
                tmem_wait(v[0]);
                tmem_wait(v[1]);
#pragma unroll
                for (int e = 0; e < kHalf; e += 2) {
                    const float2 r = fma2(make_float2(tot, tot), make_float2(S[e], S[e + 1]),
                                          make_float2(v[e / 16][e % 16], v[e / 16][e % 16 + 1]));
                    S[e] = r.x, S[e + 1] = r.y;
                }
            }
            tc_fence_before();
            signal(bar.d3_empty[c % kD3s]);
            if constexpr (OUT) {
                wait(bar.d1_full, c);  // (2) has read the planes
                if (!ok) break;
                if (c + 1 < chunks) write_planes();
                wait(bar.d2_full, c);
                if (!ok) break;
                tc_fence_after();
                const uint8_t* xs = sm + (c % kStages) * kStageBytes;
                __nv_bfloat16* dst = a.y + (r0 + static_cast<long>(c) * kL + row) * a.ldy + h * kScanP + p0;
                const bool live = row < count(c);
#pragma unroll 1
                for (int i = 0; i < kHalf; i += 16) {
                    float u[16], v[16];
                    {
                        float w[16];
                        __syncwarp();
                        tmem_load16(tm + lane_base + kColD1 + p0 + i, u);
                        tmem_load16(tm + lane_base + kColD1 + 64 + p0 + i, w);
                        tmem_load16(tm + lane_base + kColD2 + p0 + i, v);
                        tmem_wait(u);
                        tmem_wait(w);
                        tmem_wait(v);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 r = fma2(make_float2(f, f),
                                                  add2(make_float2(u[e], u[e + 1]), make_float2(w[e], w[e + 1])),
                                                  make_float2(v[e], v[e + 1]));
                            u[e] = r.x, u[e + 1] = r.y;
                        }
                    }
                    if (i == kHalf - 16) {
                        tc_fence_before();
                        signal(bar.d_empty);
                    }
#pragma unroll
                    for (int k = 0; k < 16; k += 8) {
                        const uint4 xv = *reinterpret_cast<const uint4*>(xs + swz(row, (p0 + i + k) * 2, kL));
                        const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 r = fma2(make_float2(Dh, Dh), make_float2(bf_lo(xw[e]), bf_hi(xw[e])),
                                                  make_float2(u[k + 2 * e], u[k + 2 * e + 1]));
                            o[e] = pack_bf16(r.x, r.y);
                        }
                        if (live) *reinterpret_cast<uint4*>(dst + i + k) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
                signal(bar.empty[c % kStages]);
            }
        }
        float* dst = whole ? (a.sT ? a.sT + seq_state : nullptr) : OUT ? nullptr : a.seg_state + slot_state;
        if (ok && dst) {
#pragma unroll
            for (int p = 0; p < kHalf; ++p) dst[(p0 + p) * kN + row] = S[p];
        }
        if (!OUT && !whole && warp == kWarpS && lane == 0) a.seg_decay[slot * a.H + h] = run;
    } else if (warp < kWarpMma && warp != kWarpLoad) {
        // ------------------------------------------------------------ the scaled x
        // One group of four warps; without outputs the warps of M are two more, and the
        // groups take the pieces in turn.
        const int group = warp < kWarpS ? 1 + (warp >> 2) : 0, groups = OUT ? 1 : 3;
        const int w = (warp < kWarpS ? warp & 3 : warp == 20 ? 3 : warp - kWarpX) * 32 + lane;
        const int r = w >> 2, part = (w & 3) * 32;  // row of a piece; bytes part .. of it
        int now = -1;                               // the chunk at hand
        for (int piece = group; piece < 4 * chunks && ok; piece += groups) {
            const int c = piece >> 2, s = 32 * (piece & 3) + r, ring = piece % kRing;
            const Decays128& d = dec[c % kDecs];
            uint8_t* st = sm + (c % kStages) * kStageBytes;
            if (c != now) {
                for (; now < c; ++now)
                    if (now >= 0) signal(bar.dec_empty[now % kDecs]);
                wait(bar.full[c % kStages], c / kStages);
                wait(bar.dec_full[c % kDecs], c / kDecs);
            }
            if (piece >= kRing) wait(bar.xw_empty[ring], piece / kRing - 1);
            if (!ok) break;
            const bool live = s < count(c);
            const float f = d.w[s];
            uint8_t* out = sm + kXw + ring * 3 * kPiece;
#pragma unroll
            for (int b = 0; b < 32; b += 16) {
                uint4 xv = *reinterpret_cast<const uint4*>(st + swz(s, part + b, kL));
                if (!live) {
                    // Rows of the next sequence: their x and B meet factors of zero in (3) and (4),
                    // which an infinity or NaN would not survive.
                    xv = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(st + swz(s, part + b, kL)) = xv;
                    *reinterpret_cast<uint4*>(st + kTile + swz(s, part + b, kL)) = xv;
                    *reinterpret_cast<uint4*>(st + 2 * kTile + swz(s, part + b, kL)) = xv;
                }
                const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
                uint32_t u[4][3];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = mul2(make_float2(f, f), make_float2(bf_lo(xw[e]), bf_hi(xw[e])));
                    split_pair<3>(u[e], v.x, v.y);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    *reinterpret_cast<uint4*>(out + p * kPiece + swz(r, part + b, 32)) =
                        make_uint4(u[0][p], u[1][p], u[2][p], u[3][p]);
            }
            fence_proxy_async_smem();
            signal(bar.xw_full[ring]);
        }
        for (; ok && now < chunks; ++now)
            if (now >= 0) signal(bar.dec_empty[now % kDecs]);
    } else if (warp == kWarpLoad) {
        // ------------------------------------------------------------ loads
        int issued = 0;
        for (int c = 0; c < chunks && ok; ++c) {
            const int st = c % kStages;
            if (c >= kStages) wait(bar.empty[st], c / kStages - 1);
            if (!ok) break;
            if (lane == 0) {
                uint8_t* p = sm + st * kStageBytes;
                const int row = static_cast<int>(r0 + static_cast<long>(c) * kL);
                mbar_arrive_expect_tx(&bar.full[st], kStageBytes);
                tma_load_2d(p + kTile, &maps.b, &bar.full[st], grp * kN, row);
                tma_load_2d(p + 2 * kTile, &maps.b, &bar.full[st], grp * kN + 64, row);
                if constexpr (OUT) {
                    tma_load_2d(p + 3 * kTile, &maps.c, &bar.full[st], grp * kN, row);
                    tma_load_2d(p + 4 * kTile, &maps.c, &bar.full[st], grp * kN + 64, row);
                }
                tma_load_2d(p, &maps.x, &bar.full[st], h * kScanP, row);
            }
            __syncwarp();
            issued = c + 1;
        }
        // nothing may still be on its way into shared memory when the block ends, also
        // where other warps gave up
        for (int c = issued < kStages ? 0 : issued - kStages; c < issued; ++c)
            mbar_wait(&bar.full[c % kStages], static_cast<uint32_t>(c / kStages) & 1u, 2000000000ull);
    } else if (warp >= kWarpDec) {
        // ------------------------------------------------------------ decays
        const float Ah = a.A[h], bias = a.bias ? a.bias[h] : 0.f;
        float dt[4];
        auto fetch = [&](int c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const long r = r0 + static_cast<long>(c) * kL + 4 * lane + i;
                dt[i] = r < r1 ? load_dt(a.dt, r * a.lddt + h, a.dt_bf16) : 0.f;
            }
        };
        fetch(warp - kWarpDec);
        for (int c = warp - kWarpDec; c < chunks && ok; c += 2) {
            if (c >= kDecs) wait(bar.dec_empty[c % kDecs], c / kDecs - 1);
            if (!ok) break;
            chunk_decays128(dec[c % kDecs], dt, count(c), Ah, bias, a.softplus, lane);
            fetch(c + 2);
            signal(bar.dec_full[c % kDecs]);
        }
    } else {
        // ------------------------------------------------------------ products
        const uint64_t dX = desc_mn(sb, kTile), dBk = desc_k(sb + kTile), dBn = desc_mn(sb + kTile, kTile),
                       dC = desc_k(sb + 3 * kTile), dS = desc_mn(sb + kOffS, kTile), dXw = desc_mn(sb + kXw, kPiece);
        auto products_g = [&](int c) {
            const uint64_t st = (c % kStages) * at(kStageBytes);
            if (elect_one()) {
                uint64_t p = dC + st, q = dBk + st;
#pragma unroll 1
                for (int k = 0; k < 8; ++k) {
                    mma_smem(tm + kColG, p, q, kIdG, k > 0);
                    const uint64_t d = next_k(k);
                    p += d;
                    q += d;
                }
                mma_commit(&bar.g_full);
            }
            __syncwarp();
        };
        for (int c = 0; c < chunks && ok; ++c) {
            const int st = c % kStages;
            const uint64_t so = st * at(kStageBytes);
            const uint32_t d3 = tm + kColD3 - (c % kD3s) * 64;
            if (!OUT || c == 0) {
                wait(bar.full[st], c / kStages);
                if (!ok) break;
                tc_fence_after();
                if constexpr (OUT) products_g(0);
            }
            // (4), half of its pieces at a time: the ring is filled again while (2) runs
            if (c >= kD3s) wait(bar.d3_empty[c % kD3s], c / kD3s - 1);
            auto products_s = [&](int k) {
                const int ring = k % kRing;
                wait(bar.xw_full[ring], (4 * c + k) / kRing);
                if (!ok) return;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t p = dBn + so + step_mn(2 * k);
                    uint64_t q = dXw + ring * at(3 * kPiece);
#pragma unroll 1
                    for (int i = 0; i < 3; ++i, q += at(kPiece)) {
                        mma_smem(d3, p, q, kIdS, k > 0 || i > 0);
                        mma_smem(d3, p + step_mn(1), q + step_mn(1), kIdS, true);
                    }
                    mma_commit(&bar.xw_empty[ring]);
                    if (k == 3) {
                        mma_commit(&bar.d3_full[c % kD3s]);
                        if constexpr (!OUT) mma_commit(&bar.empty[st]);
                    }
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int k = 0; k < 2; ++k) products_s(k);
            if constexpr (OUT) {
                // (2)
                wait(bar.s_full, c);
                if (c > 0) wait(bar.d_empty, c - 1);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    uint64_t p = dC + so, q = dS;
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        mma_smem(tm + kColD1, p, q, kId1, k > 0);
                        p += next_k(k);
                        q += step_mn(1);
                    }
                    mma_commit(&bar.d1_full);
                }
                __syncwarp();
            }
#pragma unroll 1
            for (int k = 2; k < 4; ++k) products_s(k);
            if (!ok) break;
            if constexpr (OUT) {
                // (3)
                wait(bar.m_full, c);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    uint32_t p = tm + kColM;
                    uint64_t q = dX + so;
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        mma_tmem(tm + kColD2, p, q, kIdY, k > 0);
                        mma_tmem(tm + kColD2, p + 64, q, kIdY, true);
                        p += 8;
                        q += step_mn(1);
                    }
                    mma_commit(&bar.d2_full);
                    mma_commit(&bar.empty[st]);
                }
                __syncwarp();
                // (1) of the next chunk: M of this one has been made, so G is free
                if (c + 1 < chunks) {
                    wait(bar.full[(c + 1) % kStages], (c + 1) / kStages);
                    if (!ok) break;
                    tc_fence_after();
                    products_g(c + 1);
                }
            }
        }
        // every product is complete before tensor memory is given back
        if (elect_one()) mma_commit(&bar.fin);
        __syncwarp();
        const bool before = ok;
        ok = true;
        wait(bar.fin, 0);
        ok = ok && before;
    }
    __syncwarp();
    if (!ok && lane == 0) report_status(a.status, WKV7_ERR_DEVICE_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ---------------------------------------------------------------- states of the backward
// As scan_states_kernel (wkv7_scan_backward.cu): blockIdx.y 0 walks the states forwards from
// x and B, 1 their gradients backwards from dy and C, in chunks of 64 tokens, and with
// WRITE leaves each at every chunk.  Product (4) alone, K = 64, with the chunks' decays
// loaded like the rows.  19 warps: 0-7 the state (lane n, half of p each), 8-15 the scaled
// rows in two groups that take pieces of 32 tokens in turn, 16 loads, 17 products, 18 stores.
// A state leaves as one bulk copy of its 48 KB out of two buffers.  At B4 T1024 H32 (201 MB
// written) 49.7 us, 4.0 TB/s: 256 blocks in two waves of 148; 59.9 us with one buffer,
// 93 us stored from the registers, 74 us in scan_states_kernel's form on mma.sync.
constexpr int kStStages = 3, kStRing = 4, kStOuts = 2, kStThreads = 19 * 32;
constexpr uint32_t kStTile = kChunk * 128;  // 64 rows of 128 bytes
constexpr uint32_t kStStage = 3 * kStTile;
constexpr uint32_t kStOffXw = kStStages * kStStage;
constexpr uint32_t kStOffOut = kStOffXw + kStRing * 3 * kPiece;
constexpr uint32_t kStOut = 3 * kScanP * kN * 2;  // a state in planes
constexpr uint32_t kStOffDec = kStOffOut + kStOuts * kStOut;
constexpr uint32_t kStOffBar = kStOffDec + kStStages * static_cast<uint32_t>(sizeof(Decays));
struct StBars {
    uint64_t full[kStStages], empty[kStStages], xw_full[kStRing], xw_empty[kStRing], d_full[2], d_empty[2], out_full[kStOuts], out_empty[kStOuts], fin;
    uint32_t tmem;
};
constexpr uint32_t kStSmem = kStOffBar + sizeof(StBars) + 1024;
static_assert(kStOffBar % 8 == 0 && kStSmem <= 227 * 1024, "shared memory of an SM");

struct StMaps {
    CUtensorMap x, b, dy, c;
};

template <bool WRITE>
__global__ void __launch_bounds__(kStThreads, 1)
    states_tc_kernel(const BwdDev a, bool whole, const __grid_constant__ StMaps maps) {
    chain_wait();
    chain_next();
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(sm);
    StBars& bar = *reinterpret_cast<StBars*>(sm + kStOffBar);
    const Decays* dec = reinterpret_cast<const Decays*>(sm + kStOffDec);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int back = blockIdx.y, h = blockIdx.x % a.H, grp = h / (a.H / a.G);
    const long slot = blockIdx.x / a.H;
    constexpr long kState = static_cast<long>(kScanP) * kN;

    int n;
    long r0, r1, lo, hi;
    if (!seg_rows(a.seg, slot, n, r0, r1, lo, hi, a.status)) {
        if (!whole || !back || !a.ds0) return;
        const long e = (static_cast<long>(n) * a.H + h) * kState;  // no tokens: ds0 = dsT
        for (int i = tid; i < kState; i += kStThreads) a.ds0[e + i] = a.dsT ? a.dsT[e + i] : 0.f;
        return;
    }
    const long seq_state = (static_cast<long>(n) * a.H + h) * kState;
    float* slot_state = a.seg_state + ((back ? a.seg_count : 0) + slot) * a.H * kState + h * kState;
    const int rows = static_cast<int>(r1 - r0), chunks = (rows + kChunk - 1) / kChunk;
    const long chunk0 = seg_first(a.chunk, n, lo) + (r0 - lo) / kChunk;
    auto at_chunk = [&](int i) { return back ? chunks - 1 - i : i; };  // the i-th of the walk

    if (warp == 17) {
        if (lane == 0) {
            for (int i = 0; i < kStStages; ++i) {
                mbar_init(&bar.full[i], 1);
                mbar_init(&bar.empty[i], 17);  // the products, and the warps that read decays and rows
            }
            for (int i = 0; i < kStRing; ++i) {
                mbar_init(&bar.xw_full[i], 4);
                mbar_init(&bar.xw_empty[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&bar.d_full[i], 1);
                mbar_init(&bar.d_empty[i], 8);
            }
            for (int i = 0; i < kStOuts; ++i) {
                mbar_init(&bar.out_full[i], 8);
                mbar_init(&bar.out_empty[i], 1);
            }
            mbar_init(&bar.fin, 1);
            fence_mbar_init();
        }
        tmem_alloc(&bar.tmem, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = bar.tmem;
    bool ok = true;
    auto wait = [&](uint64_t& b, int k) {
        for (uint32_t i = 0; ok && !__all_sync(0xffffffffu, mbar_try_wait_sleep(&b, k & 1, kPollNs)); ++i)
            ok = i < kPolls;
    };
    auto signal = [&](uint64_t& b) {  // once per warp
        __syncwarp();
        if (lane == 0) arrive(&b);
    };

    if (warp < 8) {
        // ------------------------------------------------------------ the state
        const int row = 32 * (warp & 3) + lane, p0 = warp >= 4 ? kHalf : 0;
        const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;
        float S[kHalf];
        {
            const float* first = back ? a.dsT : a.s0;
            const float* src = whole ? (first ? first + seq_state : nullptr) : WRITE ? slot_state : nullptr;
#pragma unroll
            for (int p = 0; p < kHalf; ++p) S[p] = src ? src[(p0 + p) * kN + row] : 0.f;
        }
        float run = 1.f;
        for (int i = 0; i < chunks && ok; ++i) {
            if constexpr (WRITE) {
                const int o = i % kStOuts;
                if (i >= kStOuts) wait(bar.out_empty[o], i / kStOuts - 1);
                if (!ok) break;
#pragma unroll
                for (int p = 0; p < kHalf; p += 8) {
                    uint32_t u[4][3];
#pragma unroll
                    for (int e = 0; e < 4; ++e) split_pair<3>(u[e], S[p + 2 * e], S[p + 2 * e + 1]);
#pragma unroll
                    for (int w = 0; w < 3; ++w)
                        *reinterpret_cast<uint4*>(sm + kStOffOut + o * kStOut + w * (kState * 2) +
                                                  swz(row, (p0 + p) * 2, kN)) =
                            make_uint4(u[0][w], u[1][w], u[2][w], u[3][w]);
                }
                fence_proxy_async_smem();
                signal(bar.out_full[o]);
            }
            wait(bar.full[i % kStStages], i / kStStages);
            const float tot = dec[i % kStStages].total;
            signal(bar.empty[i % kStStages]);
            wait(bar.d_full[i & 1], i >> 1);
            if (!ok) break;
            tc_fence_after();
            run *= tot;
            float v[2][16];
            __syncwarp();
            tmem_load16(tm + lane_base + 64 * (i & 1) + p0, v[0]);
            tmem_load16(tm + lane_base + 64 * (i & 1) + p0 + 16, v[1]);
            tmem_wait(v[0]);
            tmem_wait(v[1]);
            tc_fence_before();
            signal(bar.d_empty[i & 1]);
#pragma unroll
            for (int e = 0; e < kHalf; e += 2) {
                const float2 r = fma2(make_float2(tot, tot), make_float2(S[e], S[e + 1]),
                                      make_float2(v[e / 16][e % 16], v[e / 16][e % 16 + 1]));
                S[e] = r.x, S[e + 1] = r.y;
            }
        }
        float* dst = !WRITE ? slot_state : whole && back && a.ds0 ? a.ds0 + seq_state : nullptr;
        if (ok && dst) {
#pragma unroll
            for (int p = 0; p < kHalf; ++p) dst[(p0 + p) * kN + row] = S[p];
        }
        if (!WRITE && !back && warp == 0 && lane == 0) a.seg_decay[slot * a.H + h] = run;
    } else if (warp < 16) {
        // ------------------------------------------------------------ the scaled rows
        const int group = (warp - 8) >> 2, w = (warp & 3) * 32 + lane, r = w >> 2, part = (w & 3) * 32;
        for (int i = 0; i < chunks && ok; ++i) {  // piece `group` of every chunk
            const int s = 32 * group + r, ring = (2 * i + group) % kStRing, left = rows - at_chunk(i) * kChunk;
            const Decays& d = dec[i % kStStages];
            uint8_t* st = sm + (i % kStStages) * kStStage;
            wait(bar.full[i % kStStages], i / kStStages);
            if (2 * i + group >= kStRing) wait(bar.xw_empty[ring], (2 * i + group) / kStRing - 1);
            if (!ok) break;
            const bool live = s < left;
            const float f = back ? d.from[s] : d.delta[s] * d.to[s];
            uint8_t* out = sm + kStOffXw + ring * 3 * kPiece;
#pragma unroll
            for (int b = 0; b < 32; b += 16) {
                uint4 xv = *reinterpret_cast<const uint4*>(st + swz(s, part + b, kChunk));
                if (!live) {  // rows of the next sequence, as in scan_tc_kernel
                    xv = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(st + kStTile + swz(s, part + b, kChunk)) = xv;
                    *reinterpret_cast<uint4*>(st + 2 * kStTile + swz(s, part + b, kChunk)) = xv;
                }
                const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
                uint32_t u[4][3];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 v = mul2(make_float2(f, f), make_float2(bf_lo(xw[e]), bf_hi(xw[e])));
                    split_pair<3>(u[e], v.x, v.y);
                }
#pragma unroll
                for (int p = 0; p < 3; ++p)
                    *reinterpret_cast<uint4*>(out + p * kPiece + swz(r, part + b, 32)) =
                        make_uint4(u[0][p], u[1][p], u[2][p], u[3][p]);
            }
            fence_proxy_async_smem();
            signal(bar.xw_full[ring]);
            signal(bar.empty[i % kStStages]);
        }
    } else if (warp == 16) {
        // ------------------------------------------------------------ loads
        int issued = 0;
        for (int i = 0; i < chunks && ok; ++i) {
            const int st = i % kStStages;
            if (i >= kStStages) wait(bar.empty[st], i / kStStages - 1);
            if (!ok) break;
            if (lane == 0) {
                uint8_t* p = sm + st * kStStage;
                const int row = static_cast<int>(r0 + static_cast<long>(at_chunk(i)) * kChunk);
                const CUtensorMap *mx = back ? &maps.dy : &maps.x, *mb = back ? &maps.c : &maps.b;
                mbar_arrive_expect_tx(&bar.full[st], kStStage + static_cast<uint32_t>(sizeof(Decays)));
                tma_load_2d(p, mx, &bar.full[st], h * kScanP, row);
                tma_load_2d(p + kStTile, mb, &bar.full[st], grp * kN, row);
                tma_load_2d(p + 2 * kStTile, mb, &bar.full[st], grp * kN + 64, row);
                bulk_load(sm + kStOffDec + st * sizeof(Decays), a.dec + (chunk0 + at_chunk(i)) * a.H + h,
                          sizeof(Decays), &bar.full[st]);
            }
            __syncwarp();
            issued = i + 1;
        }
        // nothing may still be on its way into shared memory when the block ends
        for (int i = issued < kStStages ? 0 : issued - kStStages; i < issued; ++i)
            mbar_wait(&bar.full[i % kStStages], static_cast<uint32_t>(i / kStStages) & 1u, 2000000000ull);
    } else if (warp == 18) {
        // ------------------------------------------------------------ stores
        if constexpr (WRITE) {
            for (int i = 0; i < chunks && ok; ++i) {
                const int o = i % kStOuts;
                wait(bar.out_full[o], i / kStOuts);
                if (!ok) break;
                if (lane == 0) {
                    bulk_store(a.states + (((back ? a.chunk_count : 0) + chunk0 + at_chunk(i)) * a.H + h) *
                                              (kStatePlanes * kState),
                               sm + kStOffOut + o * kStOut, kStOut);
                    bulk_commit();
                    bulk_wait_read<kStOuts - 1>();
                    if (i >= kStOuts - 1) arrive(&bar.out_empty[(i + 1) % kStOuts]);
                }
                __syncwarp();
            }
            if (lane == 0) bulk_wait_all();
            __syncwarp();
        }
    } else {
        // ------------------------------------------------------------ products
        const uint64_t dB = desc_mn(sb + kStTile, kStTile), dXw = desc_mn(sb + kStOffXw, kPiece);
        for (int i = 0; i < chunks && ok; ++i) {
            const int st = i % kStStages;
            wait(bar.full[st], i / kStStages);
            if (i >= 2) wait(bar.d_empty[i & 1], (i >> 1) - 1);
#pragma unroll 1
            for (int k = 0; k < 2; ++k) {
                const int piece = 2 * i + k, ring = piece % kStRing;
                wait(bar.xw_full[ring], piece / kStRing);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t p = dB + st * at(kStStage) + step_mn(2 * k);
                    uint64_t q = dXw + ring * at(3 * kPiece);
#pragma unroll 1
                    for (int w = 0; w < 3; ++w, q += at(kPiece)) {
                        mma_smem(tm + 64 * (i & 1), p, q, kIdS, k > 0 || w > 0);
                        mma_smem(tm + 64 * (i & 1), p + step_mn(1), q + step_mn(1), kIdS, true);
                    }
                    mma_commit(&bar.xw_empty[ring]);
                    if (k == 1) {
                        mma_commit(&bar.d_full[i & 1]);
                        mma_commit(&bar.empty[st]);
                    }
                }
                __syncwarp();
            }
        }
        if (elect_one()) mma_commit(&bar.fin);
        __syncwarp();
        const bool before = ok;
        ok = true;
        wait(bar.fin, 0);
        ok = ok && before;
    }
    __syncwarp();
    if (!ok && lane == 0) report_status(a.status, WKV7_ERR_DEVICE_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tm, 128);
    }
}

// rows x width matrix of bf16 at a row stride, box 64 columns x `box_rows`
bool make_map(CUtensorMap* m, const void* base, uint64_t width, uint64_t rows, uint64_t ld, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {width, rows};
    const cuuint64_t strides[1] = {ld * 2};
    const cuuint32_t box[2] = {64, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_scan_tc(const ScanArgs& p, const SegMap& map, bool whole, bool out, float* seg_state,
                           float* seg_decay, cudaStream_t stream) {
    TcMaps maps;
    const uint64_t rows = p.seq_offsets ? p.T : static_cast<uint64_t>(p.B) * p.T;
    if (!make_map(&maps.x, p.x, static_cast<uint64_t>(p.H) * kScanP, rows, p.ldx, kL) ||
        !make_map(&maps.b, p.Bm, static_cast<uint64_t>(p.G) * kN, rows, p.ldb, kL) ||
        !make_map(&maps.c, p.Cm, static_cast<uint64_t>(p.G) * kN, rows, p.ldc, kL))
        return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> cfg_out{0}, cfg_state{0};
    const TcArgs a{p.dt, p.lddt, p.ldy, p.A, p.D, p.dt_bias, p.s0, static_cast<__nv_bfloat16*>(p.y), p.sT, seg_state,
                   seg_decay, p.H, p.G, p.softplus, p.dt_dtype == WKV7_BF16, map, p.status};
    const unsigned grid = static_cast<unsigned>(seg_slots(map) * p.H);
    cudaError_t e;
    if (out) {
        e = configure_smem_once(scan_tc_kernel<true>, kTcSmem, cfg_out);
        if (e != cudaSuccess) return e;
        if (whole)
            scan_tc_kernel<true><<<grid, kTcThreads, kTcSmem, stream>>>(a, whole, maps);
        else
            e = launch_next(scan_tc_kernel<true>, grid, kTcThreads, kTcSmem, stream, a, whole, maps);
    } else {
        e = configure_smem_once(scan_tc_kernel<false>, kTcSmem, cfg_state);
        if (e == cudaSuccess) scan_tc_kernel<false><<<grid, kTcThreads, kTcSmem, stream>>>(a, whole, maps);
    }
    return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_states_tc(const BwdDev& d, bool write, bool whole, cudaStream_t stream) {
    StMaps maps;
    const uint64_t rows = static_cast<uint64_t>(d.rows), wx = static_cast<uint64_t>(d.H) * kScanP,
                   wb = static_cast<uint64_t>(d.G) * kN;
    if (!make_map(&maps.x, d.x, wx, rows, d.ldx, kChunk) || !make_map(&maps.dy, d.dy, wx, rows, d.lddy, kChunk) ||
        !make_map(&maps.b, d.Bm, wb, rows, d.ldb, kChunk) || !make_map(&maps.c, d.Cm, wb, rows, d.ldc, kChunk))
        return cudaErrorInvalidValue;
    static std::atomic<unsigned long long> cfg_w{0}, cfg_s{0};
    const dim3 grid(static_cast<unsigned>(d.seg_count * d.H), 2);
    cudaError_t e;
    if (write) {
        e = configure_smem_once(states_tc_kernel<true>, kStSmem, cfg_w);
        if (e == cudaSuccess) launch_next(states_tc_kernel<true>, grid, kStThreads, kStSmem, stream, d, whole, maps);
    } else {
        e = configure_smem_once(states_tc_kernel<false>, kStSmem, cfg_s);
        if (e == cudaSuccess) launch_next(states_tc_kernel<false>, grid, kStThreads, kStSmem, stream, d, whole, maps);
    }
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace wkv7
