// wkv7_scan_backward.cu — gradient of <dy, y> + <dsT, sT> of the selective scan.
//
// Notation of scan_common.cuh; per chunk, with S_0 the state at its start, dS the
// gradient of the state at its end, L_ts = exp(l_t - l_s) for s <= t, G = C B^T,
// M_ts = dy_t . x_s, f_t = exp(l_t), e_s = exp(l_64 - l_s):
//   dS_0   = exp(l_64) dS + sum_t f_t dy_t C_t^T          (walking the chunks backwards)
//   dx_s   = delta_s (sum_{t>=s} G_ts L_ts dy_t + e_s dS B_s) + D dy_s
//   dB_s   = sum_{t>=s} Q_ts C_t + e_s delta_s dS^T x_s,   Q_ts = M_ts L_ts delta_s
//   dC_t   = sum_{s<=t} Q_ts B_s + f_t S_0^T dy_t          (dB, dC summed over a group's heads)
// and through the decays, with W_ts = G_ts Q_ts, E_t = f_t C_t . S_0^T dy_t and
// F_s = e_s delta_s x_s . dS B_s, the gradient of A delta_i sums what passes token i:
//   sum_{s<i<=t} W_ts + sum_{t>=i} E_t + sum_{s<i} F_s + exp(l_64) <S_0, dS>.
// The first sum is taken as it stands (row prefixes V = W U with U_si = 1 for s < i, a
// product of its own, then columns over t >= i): the shorter way, sums over rows minus
// sums over columns, cancels, and left errors of 1e-5 where a strong decay lies between
// tokens that act on each other.  Last, d delta_s has the term
// x_s . (sum G L dy + e dS B_s), and d softplus(u) / du = 1 - exp(-softplus(u)).
//
// Launches: the decays; (1) the states S_0 and the gradients dS at every chunk boundary,
// forwards and backwards side by side, written as bf16 planes (over segments where
// sequences and heads are few, as in wkv7_scan.cu; on tcgen05 in wkv7_scan_tc.cu for bf16
// and N = 128); (2) one block per chunk, group and share of
// the group's heads, which keeps the sums over heads in registers: warps 0-3 hold 16
// tokens t each (dC, E, sums over s), warps 4-7 16 tokens s each (dx, dB, F, sums over
// t); (3) sums over the shares and over chunks, in a fixed order.
//
// Measured at B4 T1024 H32 N128 bf16: decays 3.6 us, (1) 49.7, (2) 133, (3) 4.  (2) has eight
// warps an SM, all their registers in use.  Half of a head's 14000 cycles are the products
// with the states, which shared memory bounds (every warp of a side reads the whole state in
// three planes, 7700 of the cycles; the tensor pipe is busy for 5500); the rest is the chain of
// products, exponentials and row sums within a warp.
#include "scan_backward.cuh"
#include "sm100_ptx.cuh"

namespace wkv7 {
namespace {

// ---------------------------------------------------------------- (1) states
template <typename IO, int N>
struct StateLayout {
    using TX = Tile<kInPlanes<IO>, kChunk, kScanP>;
    using TB = Tile<kInPlanes<IO>, kChunk, N>;
    static constexpr int stages = sizeof(IO) == 2 ? 2 : 1;
    static constexpr int stage_bytes = TX::bytes + TB::bytes;
    static constexpr int off_d = stages * stage_bytes;
    // a warp's 16 rows of one plane of the state, for its way out in whole rows
    static constexpr int cols = N / 2 >= 16 ? N / 2 : 16;
    using TO = Tile<1, 16, cols>;
    static constexpr int off_o = off_d + 2 * static_cast<int>(sizeof(Decays));
    static constexpr int bytes = off_o + 8 * TO::bytes;
};

// blockIdx.y: 0 the states from x and B, forwards; 1 their gradients from dy and C,
// backwards.  WRITE: start from the true state and write it at every chunk; otherwise
// from zero, and only the segment's end and decay are wanted.
template <typename IO, int N, bool WRITE>
__global__ void __launch_bounds__(kScanThreads, sizeof(IO) == 2 || N <= 64 ? 2 : 1)
    scan_states_kernel(const BwdDev a, bool whole) {
    chain_wait();
    chain_next();
    using LY = StateLayout<IO, N>;
    using TX = typename LY::TX;
    using TB = typename LY::TB;
    constexpr int PI = kInPlanes<IO>, PC = kStatePlanes;
    constexpr int NH = N / 2 >= 16 ? N / 2 : 16, NT = NH / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    Decays* dec = reinterpret_cast<Decays*>(smem + LY::off_d);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pg = warp & 3, half = warp >> 2, g8 = lane >> 2, q2 = (lane & 3) * 2;
    const bool has_n = half * NH < N;
    const int n0 = has_n ? half * NH : 0;
    const int back = blockIdx.y;
    const int h = blockIdx.x % a.H, grp = h / (a.H / a.G);
    const long slot = blockIdx.x / a.H;
    constexpr long kState = static_cast<long>(kScanP) * N;

    int n;
    long r0, r1, lo, hi;
    if (!seg_rows(a.seg, slot, n, r0, r1, lo, hi, a.status)) {
        if (!whole || !back || !a.ds0) return;
        const long e = (static_cast<long>(n) * a.H + h) * kState;  // no tokens: ds0 = dsT
        for (int i = tid; i < kState; i += kScanThreads) a.ds0[e + i] = a.dsT ? a.dsT[e + i] : 0.f;
        return;
    }
    const long seq_state = (static_cast<long>(n) * a.H + h) * kState;
    float* slot_state = a.seg_state + ((back ? a.seg_count : 0) + slot) * a.H * kState + h * kState;
    const IO* xg = back ? static_cast<const IO*>(a.dy) : static_cast<const IO*>(a.x);
    const IO* bg = back ? static_cast<const IO*>(a.Cm) : static_cast<const IO*>(a.Bm);
    const long ldx = back ? a.lddy : a.ldx, ldb = back ? a.ldc : a.ldb;
    xg += r0 * ldx + h * kScanP;
    bg += r0 * ldb + static_cast<long>(grp) * N;
    const int rows = static_cast<int>(r1 - r0), chunks = (rows + kChunk - 1) / kChunk;
    const long chunk0 = seg_first(a.chunk, n, lo) + (r0 - lo) / kChunk;
    const Decays* dg = a.dec + chunk0 * a.H + h;

    // i-th chunk of the walk
    auto at = [&](int i) { return back ? chunks - 1 - i : i; };
    auto count = [&](int c) { return rows - c * kChunk < kChunk ? rows - c * kChunk : kChunk; };
    auto stage = [&](int i) { return sb + (i % LY::stages) * LY::stage_bytes; };
    auto load = [&](int i) {
        const int c = at(i), nr = count(c);
        load_tile<TX, kScanP>(stage(i), xg + static_cast<long>(c) * kChunk * ldx, ldx, nr, tid, kScanThreads);
        load_tile<TB, N>(stage(i) + TX::bytes, bg + static_cast<long>(c) * kChunk * ldb, ldb, nr, tid, kScanThreads);
        cp_decays(sb + LY::off_d + (i & 1) * static_cast<uint32_t>(sizeof(Decays)), dg + static_cast<long>(c) * a.H, tid);
        cp_async_commit();
    };
    if constexpr (LY::stages == 2) load(0);
    float S[NT][4];
    {
        const float* src = nullptr;
        if (whole) {
            const float* first = back ? a.dsT : a.s0;
            src = first ? first + seq_state : nullptr;
        } else if (WRITE) {
            src = slot_state;
        }
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
    float run = 1.f;
    for (int i = 0; i < chunks; ++i) {
        if constexpr (LY::stages == 2) {
            cp_async_wait<0>();
            __syncthreads();
            if (i + 1 < chunks) load(i + 1);
        } else {
            __syncthreads();
            load(i);
            cp_async_wait<0>();
            __syncthreads();
        }
        const Decays& d = dec[i & 1];
        if (WRITE && has_n) {
            __nv_bfloat16* dst =
                a.states + (((back ? a.chunk_count : 0) + chunk0 + at(i)) * a.H + h) * (PC * kState);
            // Plane by plane through shared memory: rows of NH columns in 16-byte pieces
            // (stored from the fragments, 4 bytes a lane, they took 71 % of the L1's time).
            using TO = typename LY::TO;
            const uint32_t so = sb + LY::off_o + warp * TO::bytes;
            float rest[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) rest[j][e] = S[j][e];
#pragma unroll
            for (int p = 0; p < PC; ++p) {
                __syncwarp();
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t u[4];  // (rows 0-7, tile j) (rows 8-15, tile j) (0-7, j + 1) (8-15, j + 1)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float* v = &rest[j + (k >> 1)][2 * (k & 1)];
                        u[k] = PI == 1 ? __byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x7632)
                                       : pack_bf16(v[0], v[1]);
                        v[0] -= bf_lo(u[k]);
                        v[1] -= bf_hi(u[k]);
                    }
                    stsm4(addr_a<TO>(so, 0, j * 8, lane), u);
                }
                __syncwarp();
                constexpr int per = NH / 8;
#pragma unroll
                for (int k = 0; k < 16 * per / 32; ++k) {
                    const int i = lane + k * 32, r = i / per, c = i % per;
                    uint4 v;
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(so + r * TO::pitch + c * 16)
                                 : "memory");
                    *reinterpret_cast<uint4*>(dst + p * kState + StateTile<IO, N>::at(pg * 16 + r, n0 + c * 8) / 2) = v;
                }
            }
        }
        run *= d.total;
        if (has_n) {  // the product from zero, as in scan_kernel (wkv7_scan.cu)
            float add[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) add[j][0] = add[j][1] = add[j][2] = add[j][3] = 0.f;
            const uint32_t sx = stage(i), sB = sx + TX::bytes;
#pragma unroll
            for (int k = 0; k < kChunk; k += 16) {
                uint32_t fx[PI][4], fa[PC][4];
                frag_a_t<TX>(fx, sx, pg * 16, k, lane);
                float2 w0, w8;
                if (back) {
                    w0 = *reinterpret_cast<const float2*>(&d.from[k + q2]);
                    w8 = *reinterpret_cast<const float2*>(&d.from[k + 8 + q2]);
                } else {
                    const float2 d0 = *reinterpret_cast<const float2*>(&d.delta[k + q2]);
                    const float2 d8 = *reinterpret_cast<const float2*>(&d.delta[k + 8 + q2]);
                    const float2 e0 = *reinterpret_cast<const float2*>(&d.to[k + q2]);
                    const float2 e8 = *reinterpret_cast<const float2*>(&d.to[k + 8 + q2]);
                    w0 = make_float2(d0.x * e0.x, d0.y * e0.y);
                    w8 = make_float2(d8.x * e8.x, d8.y * e8.y);
                }
                scale_frag<PI, PC>(fa, fx, w0.x, w0.y, w8.x, w8.y);
#pragma unroll
                for (int j = 0; j < NT; j += 2) {
                    uint32_t fb[2][PI][2];
                    frag_b_t<TB>(fb, sB, n0 + j * 8, k, lane);
                    mma_planes<PC, PI>(add[j], fa, fb[0]);
                    mma_planes<PC, PI>(add[j + 1], fa, fb[1]);
                }
            }
            const float tot = d.total;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[j][e] = fmaf(tot, S[j][e], add[j][e]);
        }
    }
    float* dst = nullptr;
    if (!WRITE)
        dst = slot_state;
    else if (whole && back)
        dst = a.ds0 ? a.ds0 + seq_state : nullptr;
    if (dst && has_n) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float* p = dst + (pg * 16 + g8) * N + n0 + j * 8 + q2;
            *reinterpret_cast<float2*>(p) = make_float2(S[j][0], S[j][1]);
            *reinterpret_cast<float2*>(p + 8 * N) = make_float2(S[j][2], S[j][3]);
        }
    }
    if (!WRITE && !back && tid == 0) a.seg_decay[slot * a.H + h] = run;
}

// The segments' true starts (forwards) and end gradients (backwards, blockIdx.z = 1), in
// place of what each gives from zero; ds0.
__global__ void __launch_bounds__(256) scan_states_join_kernel(const BwdDev a, int elems) {
    chain_wait();
    chain_next();
    const int h = blockIdx.x % a.H, back = blockIdx.z;
    const long n = blockIdx.x / a.H;
    const int e = (blockIdx.y * 256 + threadIdx.x) * 4;
    if (e >= elems) return;
    long lo, hi;
    seq_span(a.seg.offs, static_cast<int>(n), a.seg.T, lo, hi, a.status);
    const long first = seg_first(a.seg, static_cast<int>(n), lo), cnt = (hi - lo + a.seg.seg - 1) / a.seg.seg;
    const long st = (n * a.H + h) * elems + e;
    const float* start = back ? a.dsT : a.s0;
    float4 S = start ? *reinterpret_cast<const float4*>(start + st) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (long i = 0; i < cnt; ++i) {
        const long s = first + (back ? cnt - 1 - i : i);
        float4* p = reinterpret_cast<float4*>(a.seg_state + (((back ? a.seg_count : 0) + s) * a.H + h) * elems + e);
        const float4 v = *p;
        const float f = a.seg_decay[s * a.H + h];
        *p = S;
        S.x = fmaf(f, S.x, v.x), S.y = fmaf(f, S.y, v.y), S.z = fmaf(f, S.z, v.z), S.w = fmaf(f, S.w, v.w);
    }
    if (back && a.ds0) *reinterpret_cast<float4*>(a.ds0 + st) = S;
}

// ---------------------------------------------------------------- (2) gradients of a chunk
template <typename IO, int N>
struct GradLayout {
    static constexpr int PI = kInPlanes<IO>, PC = kCalcPlanes<IO>;
    using TX = Tile<PI, kChunk, kScanP>;
    using TB = Tile<PI, kChunk, N>;
    static constexpr bool transposed = kStatesT<IO, N>;
    using TS = StateTile<IO, N>;
    // bf16: the next head's rows of x and dy are copied while this one is worked on, its
    // states once this one's have been used.  fp32: one stage, in which S_0 and dS take
    // turns in one place.
    static constexpr bool shared_state = sizeof(IO) == 4;
    static constexpr int stages = sizeof(IO) == 2 ? 2 : 1;
    static constexpr int stage_bytes = 2 * TX::bytes;
    static constexpr int off_s0 = stages * stage_bytes, off_ds = off_s0 + (shared_state ? 0 : TS::bytes);
    static constexpr int off_b = off_ds + TS::bytes, off_c = off_b + TB::bytes;
    static constexpr int off_d = off_c + TB::bytes;
    static constexpr int off_sc = off_d + 3 * static_cast<int>(sizeof(Decays));  // the last head's until its end
    static constexpr int sc_floats = 7 * kChunk + 16;  // per head, twice
    static constexpr int off_x = off_sc + 2 * sc_floats * 4;  // half of e dS B, by fragments
    static constexpr int off_bar = off_x + 4 * 4 * 32 * 16;
    static constexpr int bytes = off_bar + 16;
};
static_assert(GradLayout<__nv_bfloat16, 128>::bytes <= 227 * 1024 && GradLayout<float, 128>::bytes <= 227 * 1024,
              "shared memory of an SM");

// Sums of a head by token: E; over t >= s of G L M; x . e dS B; over the rows t >= i of each
// block of 16 of V.  And the warps' parts of the diagonal of M and of <S_0, dS>.
struct HeadSums {
    float *e, *u, *f, *v, *diag, *dot;
};

// Value pair (c, c + 1) of row r of a tile.
template <typename TL>
__device__ __forceinline__ float2 tile_pair(const uint8_t* smem, int off, int r, int c) {
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int p = TL::planes - 1; p >= 0; --p) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(smem + off + p * TL::plane + r * TL::pitch + c * 2);
        v.x += bf_lo(u);
        v.y += bf_hi(u);
    }
    return v;
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}
// Two neighbouring accumulator tiles [16][16] as planes of an A fragment.
template <int P, bool CUT>
__device__ __forceinline__ void acc_to_a(uint32_t (&f)[P][4], const float (&t0)[4], const float (&t1)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float* s = (r < 2 ? t0 : t1) + 2 * (r & 1);
        uint32_t u[P];
        split_pair<P, CUT>(u, s[0], s[1]);
#pragma unroll
        for (int p = 0; p < P; ++p) f[p][r] = u[p];
    }
}
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float a, float b) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(a, b);
}
__device__ __forceinline__ void store_pair(float* p, float a, float b) {
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
}
__device__ __forceinline__ void store_dt(void* p, long i, float v, bool bf16) {
    if (bf16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(p)[i] = v;
}

template <typename IO, int N>
__global__ void __launch_bounds__(kScanThreads, 1) scan_grad_kernel(const BwdDev a) {
    chain_wait();
    chain_next();
    using LY = GradLayout<IO, N>;
    using TX = typename LY::TX;
    using TB = typename LY::TB;
    using TS = typename LY::TS;
    constexpr int PI = LY::PI, PC = LY::PC, NT = N / 8;
    constexpr int NB = N < 32 ? N : 32;  // state columns worked on at a time
    constexpr int kState = kScanP * N;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    Decays* dec = reinterpret_cast<Decays*>(smem + LY::off_d);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blk = warp & 3, g8 = lane >> 2, q2 = (lane & 3) * 2;
    const bool s_side = warp >= 4;

    const int HG = a.H / a.G;
    const int share = blockIdx.x % a.shares;
    const int grp = static_cast<int>(blockIdx.x / a.shares % a.G);
    const long slot = blockIdx.x / a.shares / a.G;
    const int h0 = grp * HG + static_cast<int>(static_cast<long>(HG) * share / a.shares);
    const int heads = grp * HG + static_cast<int>(static_cast<long>(HG) * (share + 1) / a.shares) - h0;

    int n;
    long r0, r1, lo, hi;
    if (!seg_rows(a.chunk, slot, n, r0, r1, lo, hi, a.status)) {
        if (tid < heads * 4) a.scalars[(slot * a.H + h0) * 4 + tid] = 0.f;
        for (int i = tid + kScanThreads; i < heads * 4; i += kScanThreads)
            a.scalars[(slot * a.H + h0) * 4 + i] = 0.f;
        return;
    }
    const int nr = static_cast<int>(r1 - r0);
    const IO* xg = static_cast<const IO*>(a.x) + r0 * a.ldx;
    const IO* yg = static_cast<const IO*>(a.dy) + r0 * a.lddy;

    auto stage = [&](int i) { return (i % LY::stages) * LY::stage_bytes; };
    // The states come by bulk copies, the rows by every thread's own (16 bytes each, the
    // states took 2500 of a head's 16000 cycles, N = 128).
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + LY::off_bar);
    if (tid == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    auto load_state = [&](int off, int back, int h) {
        bulk_load(smem + off, a.states + (((back ? a.chunk_count : 0) + slot) * a.H + h) * (kStatePlanes * kState),
                  TS::bytes, bar);
    };
    // A wait that gives up is reported and is the last: it waits once more, so that no copy is on
    // its way into shared memory when the block ends, and thread 0 starts no further one.
    bool ok = true;
    uint32_t phase = 0;
    auto wait_states = [&]() {
        if (ok && !mbar_wait(bar, phase & 1, 2000000000ull)) {
            ok = false;
            report_status(a.status, WKV7_ERR_DEVICE_TIMEOUT);
            mbar_wait(bar, phase & 1, 2000000000ull);
        }
        ++phase;
    };
    auto load = [&](int i) {
        const int h = h0 + i, s = stage(i);
        load_tile<TX, kScanP>(sb + s, xg + h * kScanP, a.ldx, nr, tid, kScanThreads);
        load_tile<TX, kScanP>(sb + s + TX::bytes, yg + h * kScanP, a.lddy, nr, tid, kScanThreads);
        cp_decays(sb + LY::off_d + (i % 3) * static_cast<uint32_t>(sizeof(Decays)), a.dec + slot * a.H + h, tid);
        cp_async_commit();
    };
    auto load_states = [&](int i) {
        if (tid != 0 || !ok) return;
        mbar_arrive_expect_tx(bar, (LY::shared_state ? 1 : 2) * TS::bytes);
        load_state(LY::off_s0, 0, h0 + i);
        if constexpr (!LY::shared_state) load_state(LY::off_ds, 1, h0 + i);
    };
    auto sums = [&](int i) {
        float* p = reinterpret_cast<float*>(smem + LY::off_sc) + (i & 1) * LY::sc_floats;
        return HeadSums{p, p + 64, p + 128, p + 192, p + 448, p + 456};
    };
    // Warp 0: from the row sums of head i to d dt and the chunk's part of dA, d dt_bias, dD.
    auto finish = [&](int i) {
        const HeadSums s = sums(i);
        const Decays& d = dec[i % 3];
        const int h = h0 + i;
        float E[2], F[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            E[k] = s.e[2 * lane + k];
            F[k] = d.delta[2 * lane + k] * s.f[2 * lane + k];
        }
        float diag = 0.f, dot = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) diag += s.diag[k];
#pragma unroll
        for (int k = 0; k < 8; ++k) dot += s.dot[k];
        // sums over this lane's tokens and those behind (E) or before (F)
        float se = E[0] + E[1], sf = F[0] + F[1];
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const float oe = __shfl_down_sync(0xffffffffu, se, m), of = __shfl_up_sync(0xffffffffu, sf, m);
            if (lane + m < 32) se += oe;
            if (lane >= m) sf += of;
        }
        float after = __shfl_down_sync(0xffffffffu, se, 1), before = __shfl_up_sync(0xffffffffu, sf, 1);
        if (lane == 31) after = 0.f;
        if (lane == 0) before = 0.f;
        float dA = 0.f, db = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int t = 2 * lane + k;
            float ga = fmaf(d.total, dot, after + E[1] + (k ? before + F[0] : E[0] + before));  // of A delta_t
#pragma unroll
            for (int b = 0; b < 4; ++b)
                if (b >= t / 16) ga += s.v[b * kChunk + t];
            float v = fmaf(a.A[h], ga, s.u[t] + s.f[t]);
            if (a.softplus) v *= -expm1f(-d.delta[t]);
            if (t < nr) {
                dA = fmaf(d.delta[t], ga, dA);
                db += v;
                store_dt(a.ddt, (r0 + t) * a.ldddt + h, v, a.dt_bf16);
            }
        }
        dA = warp_sum(dA);
        db = warp_sum(db);
        if (lane == 0) *reinterpret_cast<float4*>(a.scalars + (slot * a.H + h) * 4) = make_float4(dA, db, diag, 0.f);
    };

    load_tile<TB, N>(sb + LY::off_b, static_cast<const IO*>(a.Bm) + r0 * a.ldb + static_cast<long>(grp) * N, a.ldb, nr,
                     tid, kScanThreads);
    load_tile<TB, N>(sb + LY::off_c, static_cast<const IO*>(a.Cm) + r0 * a.ldc + static_cast<long>(grp) * N, a.ldc, nr,
                     tid, kScanThreads);
    load(0);
    load_states(0);
    cp_async_wait<0>();
    __syncthreads();

    // Pieces of 16 x 16 of this warp's rows: k = 0 .. 3 are the columns' token blocks; on
    // the t side those up to blk count, on the s side those from blk on.
    auto in_tri = [&](int k) { return s_side ? k >= blk : k <= blk; };
    const uint32_t mine = sb + (s_side ? LY::off_b : LY::off_c), theirs = sb + (s_side ? LY::off_c : LY::off_b);
    float G[8][4], Q[8][4], acc[NT][4];  // G of the group; sums over heads: Q and the inter-chunk part of dC or dB
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) G[j][e] = Q[j][e] = 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
#pragma unroll
    for (int k = 0; k < N; k += 16) {
        uint32_t fa[PI][4];
        frag_a<TB>(fa, mine, blk * 16, k, lane);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (!in_tri(c)) continue;
            uint32_t fb[2][PI][2];
            frag_b<TB>(fb, theirs, c * 16, k, lane);
            mma_planes<PI, PI>(G[2 * c], fa, fb[0]);
            mma_planes<PI, PI>(G[2 * c + 1], fa, fb[1]);
        }
    }

    for (int i = 0; i < heads; ++i) {
        if (i > 0) {
            if constexpr (LY::stages == 1) {
                __syncthreads();
                load(i);
                load_states(i);
            }
            cp_async_wait<0>();
            __syncthreads();
        }
        wait_states();
        const Decays& d = dec[i % 3];
        const HeadSums hs = sums(i);
        const int ox = stage(i), oy = ox + TX::bytes;
        constexpr int os0 = LY::off_s0, ods = LY::off_ds;
        const int row0 = blk * 16 + g8;  // this lane's rows: row0 and row0 + 8

        // ---- rows times a state: dy S_0 (t side), x dS (s side); sums over the state's
        // rows p.  Adds to acc, and on the t side E = f C . (dy S_0)
        auto times_state = [&](int orow, int ostate, const float (&scale)[2], float (&e_sum)[2]) {
#pragma unroll
            for (int nb = 0; nb < N; nb += NB) {
                float v[NB / 8][4];
#pragma unroll
                for (int j = 0; j < NB / 8; ++j) v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0.f;
#pragma unroll
                for (int k = 0; k < kScanP; k += 16) {
                    uint32_t fa[PI][4];
                    frag_a<TX>(fa, sb + orow, blk * 16, k, lane);
#pragma unroll
                    for (int j = 0; j < NB / 8; j += 2) {
                        uint32_t fb[2][kStatePlanes][2];
                        if constexpr (LY::transposed)
                            frag_b<TS>(fb, sb + ostate, nb + j * 8, k, lane);
                        else
                            frag_b_t<TS>(fb, sb + ostate, nb + j * 8, k, lane);
                        mma_planes<PI, kStatePlanes>(v[j], fa, fb[0]);
                        mma_planes<PI, kStatePlanes>(v[j + 1], fa, fb[1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < NB / 8; ++j)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        if (!s_side) {
                            const float2 c = tile_pair<TB>(smem, LY::off_c, row0 + 8 * r, nb + j * 8 + q2);
                            e_sum[r] = fmaf(c.x, v[j][2 * r], fmaf(c.y, v[j][2 * r + 1], e_sum[r]));
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            acc[nb / 8 + j][2 * r + e] = fmaf(scale[r], v[j][2 * r + e], acc[nb / 8 + j][2 * r + e]);
                    }
            }
        };
        if (!s_side) {
            const float scale[2] = {d.from[row0], d.from[row0 + 8]};
            float es[2] = {0.f, 0.f};
            times_state(oy, os0, scale, es);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                es[r] = quad_sum(es[r]);
                if ((lane & 3) == 0) hs.e[row0 + 8 * r] = scale[r] * es[r];
            }
        }
        if constexpr (LY::shared_state) {
            __syncthreads();  // S_0 has been read
            if (tid == 0 && ok) {
                mbar_arrive_expect_tx(bar, TS::bytes);
                load_state(ods, 1, h0 + i);
            }
            wait_states();
        }
        // ---- <S_0, dS>
        {
            float dot = 0.f;
            const __nv_bfloat16* g = a.states + (slot * a.H + h0 + i) * (kStatePlanes * kState);
#pragma unroll
            for (int k = 0; k < kState / 8 / kScanThreads + (kState / 8 % kScanThreads ? 1 : 0); ++k) {
                const int p = tid + k * kScanThreads;  // eight columns of a row
                if (kState / 8 % kScanThreads && p >= kState / 8) continue;
                uint4 u[kStatePlanes], v[kStatePlanes];
#pragma unroll
                for (int w = 0; w < kStatePlanes; ++w) {
                    u[w] = *reinterpret_cast<const uint4*>(smem + ods + w * TS::plane + p * 16);
                    if constexpr (LY::shared_state)
                        v[w] = *reinterpret_cast<const uint4*>(g + w * kState + p * 8);
                    else
                        v[w] = *reinterpret_cast<const uint4*>(smem + os0 + w * TS::plane + p * 16);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 x = make_float2(0.f, 0.f), y = x;
#pragma unroll
                    for (int w = kStatePlanes - 1; w >= 0; --w) {
                        const uint32_t a1 = (&u[w].x)[e], b1 = (&v[w].x)[e];
                        x = add2(x, make_float2(bf_lo(a1), bf_hi(a1)));
                        y = add2(y, make_float2(bf_lo(b1), bf_hi(b1)));
                    }
                    const float2 z = mul2(x, y);
                    dot += z.x + z.y;
                }
            }
            dot = warp_sum(dot);
            if (lane == 0) hs.dot[warp] = dot;
        }
        // ---- e dS B, the first part of dx: the s side takes 32 columns p, the t side (which has
        // no product with dS of its own) the others, and hands them over
        float X[8][4];
        {
            const int p0 = s_side ? 0 : 32;
#pragma unroll
            for (int j = 0; j < 8; ++j) X[j][0] = X[j][1] = X[j][2] = X[j][3] = 0.f;
#pragma unroll
            for (int k = 0; k < N; k += 16) {
                uint32_t fa[PI][4];
                frag_a<TB>(fa, sb + LY::off_b, blk * 16, k, lane);
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    uint32_t fb[2][kStatePlanes][2];
                    if constexpr (LY::transposed)
                        frag_b_t<TS>(fb, sb + ods, p0 + j * 8, k, lane);
                    else
                        frag_b<TS>(fb, sb + ods, p0 + j * 8, k, lane);
                    mma_planes<PI, kStatePlanes>(X[j], fa, fb[0]);
                    mma_planes<PI, kStatePlanes>(X[j + 1], fa, fb[1]);
                }
            }
        }
        float4* xc = reinterpret_cast<float4*>(smem + LY::off_x) + blk * 4 * 32 + lane;
        if (s_side) {
            const float scale[2] = {d.to[row0] * d.delta[row0], d.to[row0 + 8] * d.delta[row0 + 8]};
            float unused[2];
            times_state(ox, ods, scale, unused);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) xc[j * 32] = make_float4(X[j][0], X[j][1], X[j][2], X[j][3]);
        }
        __syncthreads();  // the states have been used, e dS B is complete
        if constexpr (LY::stages == 2) {
            if (i + 1 < heads) {
                load(i + 1);
                load_states(i + 1);
            }
        }
        if (s_side) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 v = xc[j * 32];
                X[4 + j][0] = v.x, X[4 + j][1] = v.y, X[4 + j][2] = v.z, X[4 + j][3] = v.w;
            }
            float fs[2] = {0.f, 0.f};
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float to = d.to[row0 + 8 * r];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 x = tile_pair<TX>(smem, ox, row0 + 8 * r, j * 8 + q2);
                    X[j][2 * r] *= to;
                    X[j][2 * r + 1] *= to;
                    fs[r] = fmaf(x.x, X[j][2 * r], fmaf(x.y, X[j][2 * r + 1], fs[r]));
                }
                fs[r] = quad_sum(fs[r]);
                if ((lane & 3) == 0) hs.f[row0 + 8 * r] = fs[r];
            }
        }
        // ---- M (t side) or its transpose, and everything that is made of it
        float M[8][4];
#pragma unroll
        for (int j = 0; j < 8; ++j) M[j][0] = M[j][1] = M[j][2] = M[j][3] = 0.f;
#pragma unroll
        for (int k = 0; k < kScanP; k += 16) {
            uint32_t fa[PI][4];
            frag_a<TX>(fa, sb + (s_side ? ox : oy), blk * 16, k, lane);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (!in_tri(c)) continue;
                uint32_t fb[2][PI][2];
                frag_b<TX>(fb, sb + (s_side ? oy : ox), c * 16, k, lane);
                mma_planes<PI, PI>(M[2 * c], fa, fb[0]);
                mma_planes<PI, PI>(M[2 * c + 1], fa, fb[1]);
            }
        }
        float sum[2] = {0.f, 0.f}, diag = 0.f;
        {
            // l of this lane's two rows, and pairs of columns; on the t side rows are t
            const float sign = s_side ? -1.f : 1.f;
            const float2 neg = make_float2(-sign, -sign);
            float2 rh[2], rl[2], rd[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = row0 + 8 * r;
                rh[r] = make_float2(sign * d.hi[row], sign * d.hi[row]);
                rl[r] = make_float2(sign * d.lo[row], sign * d.lo[row]);
                rd[r] = make_float2(d.delta[row], d.delta[row]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!in_tri(j >> 1)) continue;
                const int col = j * 8 + q2;
                const float2 ch = *reinterpret_cast<const float2*>(&d.hi[col]);
                const float2 cl = *reinterpret_cast<const float2*>(&d.lo[col]);
                const float2 cd = *reinterpret_cast<const float2*>(&d.delta[col]);
                const bool edge = (j >> 1) == blk;  // the block on the diagonal
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = row0 + 8 * r;
                    const float2 x = add2(fma2(neg, ch, rh[r]), fma2(neg, cl, rl[r]));
                    float2 l = make_float2(ex2_ftz(x.x), ex2_ftz(x.y));
                    float2 mm = make_float2(M[j][2 * r], M[j][2 * r + 1]);
                    const float2 g = make_float2(G[j][2 * r], G[j][2 * r + 1]);
                    if (edge) {  // t >= s
                        if (!s_side && row == col) diag += mm.x;
                        if (!s_side && row == col + 1) diag += mm.y;
                        if (s_side ? col < row : row < col) l.x = 0.f, mm.x = 0.f;
                        if (s_side ? col + 1 < row : row < col + 1) l.y = 0.f, mm.y = 0.f;
                    }
                    const float2 m = mul2(mm, l);
                    const float2 q = mul2(m, s_side ? rd[r] : cd);
                    const float2 qs = add2(make_float2(Q[j][2 * r], Q[j][2 * r + 1]), q);
                    Q[j][2 * r] = qs.x, Q[j][2 * r + 1] = qs.y;
                    float2 w;
                    if (s_side) {
                        sum[r] = fmaf(g.x, m.x, fmaf(g.y, m.y, sum[r]));
                        w = mul2(g, l);  // the weights of dy in dx
                    } else {
                        w = mul2(g, q);  // W; off the diagonal, which no sum takes
                        if (edge && row == col) w.x = 0.f;
                        if (edge && row == col + 1) w.y = 0.f;
                    }
                    M[j][2 * r] = w.x, M[j][2 * r + 1] = w.y;
                }
            }
        }
        if (s_side) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                sum[r] = quad_sum(sum[r]);
                if ((lane & 3) == 0) hs.u[row0 + 8 * r] = sum[r];
            }
        } else {
            diag = warp_sum(diag);
            if (lane == 0) hs.diag[blk] = diag;
            // V = W U of this warp's rows: U_si = 1 for s < i, as B fragments made in place
            float V[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j) V[j][0] = V[j][1] = V[j][2] = V[j][3] = 0.f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c > blk) continue;
                uint32_t fa[kStatePlanes][4];
                acc_to_a<kStatePlanes, true>(fa, M[2 * c], M[2 * c + 1]);
#pragma unroll
                for (int j = 2 * c; j < 8; ++j) {
                    if (j > 2 * blk + 1) continue;
                    uint32_t ub[1][2];
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const int at = (j - 2 * c) * 8 - w * 8;  // of the tile's first i behind the fragment's first s
                        ub[0][w] = at >= 8 ? 0x3f803f80u
                                           : at <= -8 ? 0u
                                                      : (q2 < g8 + at ? 0x3f80u : 0u) | (q2 + 1 < g8 + at ? 0x3f800000u : 0u);
                    }
                    mma_planes<kStatePlanes, 1>(V[j], fa, ub);
                }
            }
            // Column sums over t >= i, lanes g8 holding rows: halves of the columns are passed on
            // at every step, so that each lane ends with two columns' sums.
            float v[16];
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i2 = j * 8 + q2 + e;
                    v[2 * j + e] = j > 2 * blk + 1 ? 0.f
                                                   : (row0 >= i2 ? V[j][e] : 0.f) + (row0 + 8 >= i2 ? V[j][2 + e] : 0.f);
                }
#pragma unroll
            for (int n2 = 8; n2 >= 2; n2 >>= 1) {  // lanes 4 n2 / 2 apart swap halves
                const int far = 2 * n2;
                const bool up = lane & far;
#pragma unroll
                for (int k = 0; k < n2; ++k) {
                    const float give = up ? v[k] : v[n2 + k];
                    const float got = __shfl_xor_sync(0xffffffffu, give, far);
                    v[k] = (up ? v[n2 + k] : v[k]) + got;
                }
            }
            // lane bits 4, 3, 2 chose 8, 4, 2 of the 16 columns 2 j + e
            const int k0 = ((lane >> 4) & 1) * 8 + ((lane >> 3) & 1) * 4 + ((lane >> 2) & 1) * 2;
            *reinterpret_cast<float2*>(&hs.v[blk * kChunk + (k0 / 2) * 8 + q2]) = make_float2(v[0], v[1]);
        }

        if (s_side) {
            // ---- dx: + (G L)^T dy
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (!in_tri(c)) continue;
                uint32_t fa[PC][4];
                acc_to_a<PC, PI == 1>(fa, M[2 * c], M[2 * c + 1]);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    uint32_t fb[2][PI][2];
                    frag_b_t<TX>(fb, sb + oy, j * 8, c * 16, lane);
                    mma_planes<PC, PI>(X[j], fa, fb[0]);
                    mma_planes<PC, PI>(X[j + 1], fa, fb[1]);
                }
            }
            const float Dh = a.D ? a.D[h0 + i] : 0.f;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = row0 + 8 * r;
                const float delta = d.delta[row];
                IO* dst = static_cast<IO*>(a.dx) + (r0 + row) * a.lddx + (h0 + i) * kScanP + q2;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 y = tile_pair<TX>(smem, oy, row, j * 8 + q2);
                    if (row < nr)
                        store_pair(dst + j * 8, fmaf(delta, X[j][2 * r], Dh * y.x),
                                   fmaf(delta, X[j][2 * r + 1], Dh * y.y));
                }
            }
        }
        if (warp == 0 && i > 0) finish(i - 1);
    }

    // ---- + Q B (t side) or Q^T C (s side), and out
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (!in_tri(c)) continue;
        uint32_t fa[PC][4];
        acc_to_a<PC, PI == 1>(fa, Q[2 * c], Q[2 * c + 1]);
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
            uint32_t fb[2][PI][2];
            frag_b_t<TB>(fb, theirs, j * 8, c * 16, lane);
            mma_planes<PC, PI>(acc[j], fa, fb[0]);
            mma_planes<PC, PI>(acc[j + 1], fa, fb[1]);
        }
    }
    const int width = a.G * N;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int row = blk * 16 + g8 + 8 * r;
        if (row >= nr) continue;
        const int col = grp * N + q2;
        if (a.shares > 1) {
            float* dst = a.part + (static_cast<long>((s_side ? 0 : a.shares) + share) * a.rows + r0 + row) * width + col;
#pragma unroll
            for (int j = 0; j < NT; ++j) store_pair(dst + j * 8, acc[j][2 * r], acc[j][2 * r + 1]);
        } else {
            IO* dst = s_side ? static_cast<IO*>(a.dB) + (r0 + row) * a.lddb + col
                             : static_cast<IO*>(a.dC) + (r0 + row) * a.lddc + col;
#pragma unroll
            for (int j = 0; j < NT; ++j) store_pair(dst + j * 8, acc[j][2 * r], acc[j][2 * r + 1]);
        }
    }
    __syncthreads();  // the last head's row sums
    if (warp == 0) finish(heads - 1);
}

// ---------------------------------------------------------------- (3) sums
// Blocks [0, sum_blocks): dB and dC of every row from the shares, 4 columns a thread.
// The H blocks after them: dA, d dt_bias and dD of a head from its chunks.
template <typename IO>
__global__ void __launch_bounds__(256) scan_sum_kernel(const BwdDev a, int width, unsigned sum_blocks) {
    chain_wait();
    if (blockIdx.x < sum_blocks) {
        const long per = width / 4, total = 2 * a.rows * per;
        const long i = static_cast<long>(blockIdx.x) * 256 + threadIdx.x;
        if (i >= total) return;
        const bool c_side = i >= a.rows * per;
        const long k = c_side ? i - a.rows * per : i, row = k / per, col = k % per * 4;
        if (a.chunk.offs) {  // rows of no sequence have no partial sums and no gradients
            const int n = seq_of_row(a.chunk.offs, a.chunk.B, row);
            long lo, hi;
            seq_span(a.chunk.offs, n, a.chunk.T, lo, hi, a.status);
            if (row < lo || row >= hi) return;
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        for (int sh = 0; sh < a.shares; ++sh) {
            const float4 v = *reinterpret_cast<const float4*>(
                a.part + (static_cast<long>((c_side ? a.shares : 0) + sh) * a.rows + row) * width + col);
            s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
        }
        IO* dst = c_side ? static_cast<IO*>(a.dC) + row * a.lddc + col : static_cast<IO*>(a.dB) + row * a.lddb + col;
        store_vec<4>(dst, s);
        return;
    }
    const int h = blockIdx.x - sum_blocks;
    __shared__ float red[3][8];
    float s[3] = {0.f, 0.f, 0.f};
    for (long c = threadIdx.x; c < a.chunk_count; c += 256) {
        const float4 v = *reinterpret_cast<const float4*>(a.scalars + (c * a.H + h) * 4);
        s[0] += v.x, s[1] += v.y, s[2] += v.z;
    }
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        s[k] = warp_sum(s[k]);
        if (threadIdx.x % 32 == 0) red[k][threadIdx.x / 32] = s[k];
    }
    __syncthreads();
    if (threadIdx.x >= 3) return;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[threadIdx.x][w];
    float* dst = threadIdx.x == 0 ? a.dA : threadIdx.x == 1 ? a.dbias : a.dD;
    if (dst) dst[h] = v;
}

// Shares of a group's heads per chunk: as many as make the blocks fill the device's
// SMs in waves with the least idle time, a block costing its heads and some two heads'
// time for what it does once.
int shares_of(long chunks, int G, int HG) {
    constexpr long kSms = 148;
    int best = 1;
    long cost = -1;
    for (int s = 1; s <= HG; ++s) {
        const long waves = (chunks * G * s + kSms - 1) / kSms, c = waves * ((HG + s - 1) / s + 2);
        if (cost < 0 || c < cost) {
            cost = c;
            best = s;
        }
    }
    return best;
}

struct Plan {
    SegMap seg, chunk;
    bool whole;
    long seg_count, chunk_count, rows;
    int shares;
    size_t off_dec, off_seg, off_decay, off_part, off_scalars, bytes;
};
Plan plan_of(int B, int T, int H, int N, int G, int io_dtype, const int32_t* offs, bool packed) {
    Plan p;
    // both directions run at once; without segments the one pass makes states anyway
    p.seg = scan_segments(B, T, 2 * H, offs, packed, io_dtype == WKV7_BF16 && N != 128 ? CutCost{kChunk, 2, 1.4, 1.0, 1.0, 2.0}
                                                        : CutCost{kChunk, 1, 1.0, 1.0, 1.0, 2.0});
    p.whole = p.seg.seg >= T;
    p.chunk = chunk_map(B, T, offs);
    p.seg_count = packed && !p.whole ? T / p.seg.seg + B : static_cast<long>(B) * p.seg.spb;
    p.chunk_count = chunk_slots(B, T, packed);
    p.rows = packed ? T : static_cast<long>(B) * T;
    p.shares = shares_of(p.chunk_count, G, H / G);
        const size_t state = static_cast<size_t>(kScanP) * N;
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    p.off_dec = up(2 * static_cast<size_t>(p.chunk_count) * H * kStatePlanes * state * 2);
    p.off_seg = p.off_dec + up(static_cast<size_t>(p.chunk_count) * H * sizeof(Decays));
    p.off_decay = p.off_seg + (p.whole ? 0 : up(2 * static_cast<size_t>(p.seg_count) * H * state * 4));
    p.off_part = p.off_decay + (p.whole ? 0 : up(static_cast<size_t>(p.seg_count) * H * 4));
    p.off_scalars = p.off_part +
                    (p.shares > 1 ? up(2 * static_cast<size_t>(p.shares) * p.rows * G * N * 4) : 0);
    p.bytes = p.off_scalars + up(static_cast<size_t>(p.chunk_count) * H * 16);
    return p;
}

template <typename IO, int N>
cudaError_t bwd_typed(const BwdDev& d, const Plan& p, cudaStream_t st) {
    using SL = StateLayout<IO, N>;
    using GL = GradLayout<IO, N>;
    static std::atomic<unsigned long long> cfg_w{0}, cfg_s{0}, cfg_g{0};
    cudaError_t e = configure_smem_once(scan_grad_kernel<IO, N>, GL::bytes, cfg_g);
    if constexpr (!kStatesT<IO, N>) {
        if (e == cudaSuccess) e = configure_smem_once(scan_states_kernel<IO, N, true>, SL::bytes, cfg_w);
        if (e == cudaSuccess && !p.whole) e = configure_smem_once(scan_states_kernel<IO, N, false>, SL::bytes, cfg_s);
    }
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(p.seg_count * d.H), 2);
    constexpr bool tc = kStatesT<IO, N>;
    auto states = [&](bool write) {
        if constexpr (tc) {
            e = launch_states_tc(d, write, write && p.whole, st);
        } else if (write) {
            launch_next(scan_states_kernel<IO, N, true>, grid, kScanThreads, SL::bytes, st, d, p.whole);
        } else {
            launch_next(scan_states_kernel<IO, N, false>, grid, kScanThreads, SL::bytes, st, d, false);
        }
    };
    if (!p.whole) {
        states(false);
        if (e != cudaSuccess) return e;
        constexpr int elems = kScanP * N;
        launch_next(scan_states_join_kernel, dim3(static_cast<unsigned>(p.seg.B) * d.H, (elems / 4 + 255) / 256, 2), 256, 0,
                    st, d, elems);
    }
    states(true);
    if (e != cudaSuccess) return e;
    launch_next(scan_grad_kernel<IO, N>, static_cast<unsigned>(p.chunk_count * d.G * d.shares), kScanThreads, GL::bytes, st, d);
    const int width = d.G * N;
    const unsigned sum_blocks =
        d.shares > 1 ? static_cast<unsigned>((2 * p.rows * (width / 4) + 255) / 256) : 0;
    launch_next(scan_sum_kernel<IO>, sum_blocks + d.H, 256, 0, st, d, width, sum_blocks);
    return cudaGetLastError();
}

}  // namespace

size_t scan_backward_workspace_bytes(int B, int T, int H, int N, int G, int io_dtype, bool packed) {
    return plan_of(B, T, H, N, G, io_dtype, nullptr, packed).bytes;
}

cudaError_t launch_scan_backward(const ScanBwdArgs& q, int io_dtype, cudaStream_t stream) {
    const Plan p = plan_of(q.B, q.T, q.H, q.N, q.G, io_dtype, q.seq_offsets, q.seq_offsets != nullptr);
    BwdDev d{};
    d.x = q.x, d.Bm = q.Bm, d.Cm = q.Cm, d.dy = q.dy;
    d.ldx = q.ldx, d.ldb = q.ldb, d.ldc = q.ldc, d.lddy = q.lddy;
    d.A = q.A, d.D = q.D, d.s0 = q.s0, d.dsT = q.dsT;
    d.dx = q.dx, d.ddt = q.ddt, d.dB = q.dB, d.dC = q.dC;
    d.lddx = q.lddx, d.ldddt = q.ldddt, d.lddb = q.lddb, d.lddc = q.lddc;
    d.dA = q.dA, d.dD = q.dD, d.dbias = q.ddt_bias, d.ds0 = q.ds0;
    d.H = q.H, d.G = q.G, d.softplus = q.softplus, d.dt_bf16 = q.dt_dtype == WKV7_BF16;
    d.seg = p.seg, d.chunk = p.chunk, d.seg_count = p.seg_count, d.chunk_count = p.chunk_count;
    uint8_t* ws = static_cast<uint8_t*>(q.ws);
    d.states = reinterpret_cast<__nv_bfloat16*>(ws);
    Decays* dec = reinterpret_cast<Decays*>(ws + p.off_dec);
    d.dec = dec;
    d.seg_state = reinterpret_cast<float*>(ws + p.off_seg);
    d.seg_decay = reinterpret_cast<float*>(ws + p.off_decay);
    d.part = reinterpret_cast<float*>(ws + p.off_part);
    d.scalars = reinterpret_cast<float*>(ws + p.off_scalars);
    d.shares = p.shares, d.rows = p.rows, d.status = q.status;
    const cudaError_t e = launch_decays(
        DecayArgs{q.dt, q.lddt, q.A, q.dt_bias, dec, q.H, q.softplus, d.dt_bf16, p.chunk, q.status}, stream);
    if (e != cudaSuccess) return e;
    if (io_dtype == WKV7_BF16) switch (q.N) {
            case 16: return bwd_typed<__nv_bfloat16, 16>(d, p, stream);
            case 32: return bwd_typed<__nv_bfloat16, 32>(d, p, stream);
            case 64: return bwd_typed<__nv_bfloat16, 64>(d, p, stream);
            default: return bwd_typed<__nv_bfloat16, 128>(d, p, stream);
        }
    switch (q.N) {
        case 16: return bwd_typed<float, 16>(d, p, stream);
        case 32: return bwd_typed<float, 32>(d, p, stream);
        case 64: return bwd_typed<float, 64>(d, p, stream);
        default: return bwd_typed<float, 128>(d, p, stream);
    }
}

}  // namespace wkv7
