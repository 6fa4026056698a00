// wkv7_conv.cu — short causal convolution over tokens, one filter per channel:
//
//   pre_t[c] = bias[c] + sum_{j<W} w[c][j] x_{t-W+1+j}[c],   y_t = act(pre_t)
//
// with the W - 1 rows before a sequence's first token taken from its state s0 (or
// zero), and the last W - 1 input rows as the state it leaves.
//
// Every element is read once and takes W multiply-adds, so the kernels are bound by
// memory: a thread keeps one vector of channels and walks down a strip of token
// rows with the last W rows in registers.  Neighbouring threads hold neighbouring
// channels.  Only the W - 1 rows above a strip are read twice (from L2).
//
// Measured: packed fp32 [16384][2307] W3 (a row stride that no vector divides, so accesses
// of one element) 61 us, 5.0 TB/s; bf16 B4 T1024 C2304 W4 12.6 us, 3.0 TB/s; a token of 256
// sequences (C2816 W4) 6.6 us, most of it the filters, which every thread fetches for one row;
// gradients of B4 T1024 C2304 W4 19.5 us and 3 for the sums and ds0: two blocks an SM of 128
// registers a thread, waiting for loads, with half of the issue slots used.
#include "seq_common.cuh"

namespace wkv7 {
namespace {

constexpr int kThreads = 256;
// Rows loaded before the first of them is used: enough bytes in flight for the memory's
// latency also where an access is a single element.
template <int VEC>
constexpr int kAheadOf = VEC == 1 ? 8 : 4;
// Channels per thread.  bf16: 4, not the 8 of a 16-byte access: with 8 the filter, the
// window and the rows in flight take 140 registers or more, one block per SM (B4 T1024
// C2304: 18.5 us against 13.0 with 4 and four blocks).
constexpr int kVecF = 4;

// Row `i` (0 .. W-2, oldest first) of the state of sequence n, or zeros.
template <typename IO, int VEC>
__device__ __forceinline__ void load_state(float (&f)[VEC], const IO* s0, long n, int i, int Wm1, int C, int c) {
    if (s0) {
        load_vec<VEC>(f, s0 + (n * Wm1 + i) * C + c);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = 0.f;
    }
}

template <int VEC, int W>
__device__ __forceinline__ void load_filter(float (&wr)[W][VEC], float (&br)[VEC], const float* w, const float* bias,
                                            int c) {
    // the VEC filters are VEC * W consecutive floats
    float f[VEC * W];
    const float* src = w + static_cast<long>(c) * W;
    if constexpr (VEC * W % 4 == 0 && VEC > 1) {
#pragma unroll
        for (int i = 0; i < VEC * W; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(src + i);
            f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC * W; ++i) f[i] = src[i];
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) wr[j][e] = f[e * W + j];
        br[e] = bias ? bias[c + e] : 0.f;
    }
}

// The sequences that rows of a strip belong to, one after the other.
struct Run {
    int n;
    long lo, hi;  // rows of sequence n
};
__device__ __forceinline__ Run run_start(const int32_t* offs, int B, int T, long row, int* status) {
    Run k;
    k.n = offs ? seq_of_row(offs, B, row) : static_cast<int>(row / T);
    seq_span(offs, k.n, T, k.lo, k.hi, status);
    return k;
}
// The next sequence with a row at or behind `row`; false when there is none.
__device__ __forceinline__ bool run_at(Run& k, const int32_t* offs, int B, int T, long row, int* status) {
    while (row >= k.hi) {
        if (k.n + 1 >= B) return false;
        ++k.n;
        seq_span(offs, k.n, T, k.lo, k.hi, status);
    }
    return true;
}
// Input row r of sequence k, or a row of its state where r lies before it.
template <typename IO, int VEC, int W>
__device__ __forceinline__ void load_before(float (&f)[VEC], const IO* x, long ldx, const IO* s0, const Run& k, long r,
                                            int C, int c) {
    if (r >= k.lo)
        load_vec<VEC>(f, x + r * ldx + c);
    else
        load_state<IO, VEC>(f, s0, k.n, static_cast<int>(r - k.lo) + W - 1, W - 1, C, c);
}

// The last W - 1 rows of [s0; x] of sequence n, channels c ..: all read before any
// is written, so that sT may be s0.
template <typename IO, int VEC, int W>
__device__ void write_state(const IO* x, long ldx, const IO* s0, IO* sT, const int32_t* offs, int T, int C, long n,
                            int c, int* status) {
    long lo, hi;
    seq_span(offs, static_cast<int>(n), T, lo, hi, status);
    const long len = hi - lo;
    float f[W - 1][VEC];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        if (len + i >= W - 1)
            load_vec<VEC>(f[i], x + (lo + len + i - (W - 1)) * ldx + c);
        else
            load_state<IO, VEC>(f[i], s0, n, static_cast<int>(len) + i, W - 1, C, c);
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) store_vec<VEC>(sT + (n * (W - 1) + i) * C + c, f[i]);
}

// Where no state is written: a thread per packed sequence looks at its offsets, some of
// which the rows' blocks pass over when a pair is bad.
__device__ __forceinline__ void look_at_spans(const int32_t* offs, long n, int B, int T, int* status) {
    long lo, hi;
    if (n < B) seq_span(offs, static_cast<int>(n), T, lo, hi, status);
}

// Blocks [0, blocks_rows): y, one thread per (strip, vector of channels).  Blocks
// after them: sT, one thread per (sequence, vector of channels).
template <typename IO, int VEC, int W>
__global__ void __launch_bounds__(kThreads, VEC == 1 ? 2 : 4)
    conv_fwd_kernel(const IO* __restrict__ x, long ldx, const float* __restrict__ w, const float* __restrict__ bias,
                    const IO* s0, IO* __restrict__ y, long ldy, IO* sT, const int32_t* __restrict__ offs, int B,
                    int T, long rows, int C, int act, int strip_rows, long strips, unsigned blocks_rows,
                    int* status) {
    constexpr int kAhead = kAheadOf<VEC>;
    // vectors of fp32 leave no registers for a vector's activation at once (B4 T4096 C2304 W4: 63 us
    // against 54 value by value; bf16 B4 T1024 C2304 9.7 us value by value, 9.5 at once)
    constexpr bool kActOne = sizeof(IO) == 4 && VEC > 1;
    const int Cv = C / VEC;
    if (blockIdx.x >= blocks_rows) {
        const long i = static_cast<long>(blockIdx.x - blocks_rows) * kThreads + threadIdx.x;
        if (!sT)
            look_at_spans(offs, i, B, T, status);
        else if (i < static_cast<long>(B) * Cv)
            write_state<IO, VEC, W>(x, ldx, s0, sT, offs, T, C, i / Cv, static_cast<int>(i % Cv) * VEC, status);
        return;
    }
    const long i = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= strips * Cv) return;
    const int c = static_cast<int>(i % Cv) * VEC;
    const long r0 = i / Cv * strip_rows, r1 = r0 + strip_rows < rows ? r0 + strip_rows : rows;

    float wr[W][VEC], br[VEC];
    load_filter<VEC, W>(wr, br, w, bias, c);
    Run k = run_start(offs, B, T, r0, status);
    for (long r = r0; r < r1 && run_at(k, offs, B, T, r, status);) {
        if (r < k.lo) r = k.lo;  // rows before the first sequence
        const long end = k.hi < r1 ? k.hi : r1;
        if (r >= end) break;
        float win[W - 1][VEC];  // the rows before the current one
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            load_before<IO, VEC, W>(win[j], x, ldx, s0, k, r - (W - 1) + j, C, c);
        const IO* src = x + r * ldx + c;
        IO* dst = y + r * ldy + c;
        auto row = [&](const Raw<IO, VEC>& in) {
            float out[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float p = br[e];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) p = fmaf(wr[j][e], win[j][e], p);
                const float v = in.get(e);
                out[e] = fmaf(wr[W - 1][e], v, p);
                if constexpr (kActOne) out[e] = act_one<IO>(out[e], act);
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
                win[W - 2][e] = v;
            }
            if constexpr (!kActOne) act_vec<IO, VEC>(out, act);
            store_vec<VEC>(dst, out);
            dst += ldy;
        };
        for (; r + kAhead <= end; r += kAhead) {  // no branch between the rows of a batch
            Raw<IO, VEC> nx[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) nx[u].load(src + u * ldx);
            src += kAhead * ldx;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) row(nx[u]);
        }
        for (; r < end; ++r) {
            Raw<IO, VEC> nx;
            nx.load(src);
            src += ldx;
            row(nx);
        }
    }
}

// One token per sequence: y and the state moved on by one row, one thread per
// (sequence, vector of channels).  s_out may be s_in.
template <typename IO, int VEC, int W>
__global__ void __launch_bounds__(kThreads)
    conv_step_kernel(const IO* __restrict__ x, long ldx, const float* __restrict__ w, const float* __restrict__ bias,
                     const IO* s_in, IO* __restrict__ y, long ldy, IO* s_out, int B, int C, int act) {
    const int Cv = C / VEC;
    const long i = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= static_cast<long>(B) * Cv) return;
    const long n = i / Cv;
    const int c = static_cast<int>(i % Cv) * VEC;
    float win[W][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_state<IO, VEC>(win[j], s_in, n, j, W - 1, C, c);
    load_vec<VEC>(win[W - 1], x + n * ldx + c);
    float wr[W][VEC], br[VEC];
    load_filter<VEC, W>(wr, br, w, bias, c);
    float out[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        float p = br[e];
#pragma unroll
        for (int j = 0; j < W; ++j) p = fmaf(wr[j][e], win[j][e], p);
        out[e] = p;
    }
    act_vec<IO, VEC>(out, act);
    store_vec<VEC>(y + n * ldy + c, out);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_vec<VEC>(s_out + (n * (W - 1) + j) * C + c, win[j + 1]);
}

// ---------------------------------------------------------------- backward
// With g_t = dy_t act'(pre_t) (pre recomputed from x):
//   dx_t = sum_j w[W-1-j] g_{t+j} over the rows t + j of the sequence, + dsT for its last W - 1 rows
//   dw[j] = sum_t g_t x_{t-W+1+j},   dbias = sum_t g_t
// and the rows of s0 get the same sum as dx at the positions before the sequence.
// A block covers 32 vectors of channels and 8 strips; its sums of dw and dbias over
// the strips go to the workspace, [block][(W + 1)][C], and conv_bwd_tail_kernel adds
// the blocks in their order, so the result does not depend on timing.  ds0 is made there too (as
// blocks of the first launch it lasted 2.4 us longer, behind a full wave of strips).
constexpr int kLanes = 32, kStrips = kThreads / kLanes;
constexpr int kAheadB = 4;
constexpr int kVecB = 4;  // channels per thread: x, g, w and dw windows of W rows stay in registers

template <typename IO, int VEC, int W>
__device__ void write_state_grad(const IO* x, long ldx, const IO* s0, const IO* dy, long lddy, const IO* dsT, IO* ds0,
                                 const float (&wr)[W][VEC], const float (&br)[VEC], const int32_t* offs, int T,
                                 int C, int act, long n, int c, int* status) {
    long lo, hi;
    seq_span(offs, static_cast<int>(n), T, lo, hi, status);
    const long len = hi - lo;
    float g[W - 1][VEC];  // of the first W - 1 tokens
    float row[2 * W - 2][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        load_state<IO, VEC>(row[j], s0, n, j, W - 1, C, c);
        if (j < len) {
            load_vec<VEC>(row[W - 1 + j], x + (lo + j) * ldx + c);
            load_vec<VEC>(g[j], dy + (lo + j) * lddy + c);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) row[W - 1 + j][e] = g[j][e] = 0.f;
        }
    }
#pragma unroll
    for (int t = 0; t < W - 1; ++t) {
        float p[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            p[e] = br[e];
#pragma unroll
            for (int j = 0; j < W; ++j) p[e] = fmaf(wr[j][e], row[t + j][e], p[e]);
        }
        act_grad_vec<IO, VEC>(g[t], p, act);
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[t][e] = t < len ? g[t][e] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        float d[VEC];
        if (dsT && i >= len)  // a sequence shorter than the filter passes rows of s0 on
            load_vec<VEC>(d, dsT + (n * (W - 1) + i - len) * C + c);
        else
#pragma unroll
            for (int e = 0; e < VEC; ++e) d[e] = 0.f;
#pragma unroll
        for (int t = 0; t <= i; ++t)
#pragma unroll
            for (int e = 0; e < VEC; ++e) d[e] = fmaf(wr[i - t][e], g[t][e], d[e]);
        store_vec<VEC>(ds0 + (n * (W - 1) + i) * C + c, d);
    }
}

template <typename IO, int VEC, int W>
__global__ void __launch_bounds__(kThreads, 2)
    conv_bwd_kernel(const IO* __restrict__ x, long ldx, const float* __restrict__ w, const float* __restrict__ bias,
                    const IO* __restrict__ s0, const IO* __restrict__ dy, long lddy, const IO* __restrict__ dsT,
                    IO* __restrict__ dx, long lddx, float* __restrict__ part, const int32_t* __restrict__ offs, int B,
                    int T, long rows, int C, int act, int strip_rows, int* status) {
    chain_next();
    const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
    const int c = (blockIdx.y * kLanes + lane) * VEC;
    const bool live = c < C;
    float wr[W][VEC], br[VEC];
    if (live) load_filter<VEC, W>(wr, br, w, bias, c);
    float acc[W + 1][VEC];  // dw, then dbias
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;

    const long r0 = (static_cast<long>(blockIdx.x) * kStrips + sub) * strip_rows;
    const long r1 = r0 + strip_rows < rows ? r0 + strip_rows : rows;
    if (live && r0 < rows) {
        Run k = run_start(offs, B, T, r0, status);
        for (long r = r0; r < r1 && run_at(k, offs, B, T, r, status);) {
            if (r < k.lo) r = k.lo;
            const long end = k.hi < r1 ? k.hi : r1;
            if (r >= end) break;
            // g of the rows [r, last): the W - 1 behind `end` are needed for dx alone
            const long last = end + W - 1 < k.hi ? end + W - 1 : k.hi;
            float xw[W][VEC], gq[W][VEC];  // rows u - W + 1 .. u
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if (j > 0) load_before<IO, VEC, W>(xw[j], x, ldx, s0, k, r - W + j, C, c);
#pragma unroll
                for (int e = 0; e < VEC; ++e) gq[j][e] = 0.f;
            }
            const IO *px = x + r * ldx + c, *pg = dy + r * lddy + c;
            IO* pd = dx + r * lddx + c;
            // row u comes in; with COUNT it belongs to the strip
            auto step = [&](const Raw<IO, VEC>& vx, const Raw<IO, VEC>& vg, bool count) {
                float p[VEC], g[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
#pragma unroll
                    for (int j = 0; j + 1 < W; ++j) {
                        xw[j][e] = xw[j + 1][e];
                        gq[j][e] = gq[j + 1][e];
                    }
                    xw[W - 1][e] = vx.get(e);
                    p[e] = br[e];
#pragma unroll
                    for (int j = 0; j < W; ++j) p[e] = fmaf(wr[j][e], xw[j][e], p[e]);
                    g[e] = vg.get(e);
                }
                act_grad_vec<IO, VEC>(g, p, act);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    gq[W - 1][e] = g[e];
                    if (count) {
#pragma unroll
                        for (int j = 0; j < W; ++j) acc[j][e] = fmaf(g[e], xw[j][e], acc[j][e]);
                        acc[W][e] += g[e];
                    }
                }
            };
            // dx of the oldest row in gq, + the gradient of the final state's row `extra`
            auto emit = [&](const IO* extra) {
                float d[VEC];
                if (extra)
                    load_vec<VEC>(d, extra);
                else
#pragma unroll
                    for (int e = 0; e < VEC; ++e) d[e] = 0.f;
#pragma unroll
                for (int j = 0; j < W; ++j)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) d[e] = fmaf(wr[W - 1 - j][e], gq[j][e], d[e]);
                store_vec<VEC>(pd, d);
                pd += lddx;
            };
            long u = r;
            auto one = [&]() {  // a row at the strip's head or tail
                Raw<IO, VEC> vx, vg;
                vx.load(px);
                vg.load(pg);
                px += ldx, pg += lddy;
                step(vx, vg, u < end);
                if (u - (W - 1) >= r) emit(nullptr);
                ++u;
            };
            const long head = r + W - 1 < last ? r + W - 1 : last;
            while (u < head) one();
            for (; u + kAheadB <= end; u += kAheadB) {  // no branch between the rows of a batch
                Raw<IO, VEC> nx[kAheadB], ng[kAheadB];
#pragma unroll
                for (int i = 0; i < kAheadB; ++i) {
                    nx[i].load(px + i * ldx);
                    ng[i].load(pg + i * lddy);
                }
                px += kAheadB * ldx, pg += kAheadB * lddy;
#pragma unroll
                for (int i = 0; i < kAheadB; ++i) {
                    step(nx[i], ng[i], true);
                    emit(nullptr);
                }
            }
            while (u < last) one();
            // The rows whose W - 1 followers are not all there: the sequence ends.  (Rows from
            // hi - (W - 1) on are rows of the final state, and all of those are among them.)
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                const long s = last - (W - 1) + j;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
#pragma unroll
                    for (int i = 0; i + 1 < W; ++i) gq[i][e] = gq[i + 1][e];
                    gq[W - 1][e] = 0.f;
                }
                if (s >= r && s < end) {
                    const long i = s - (k.hi - (W - 1));
                    emit(dsT && i >= 0 ? dsT + (static_cast<long>(k.n) * (W - 1) + i) * C + c : nullptr);
                }
            }
            r = end;
        }
    }
    // sums over the block's strips, in the order of the strips
    __shared__ float red[kStrips][kLanes * VEC];
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < VEC; ++e) red[sub][lane * VEC + e] = acc[j][e];
        __syncthreads();
        for (int q = threadIdx.x; q < kLanes * VEC; q += kThreads) {
            const int cc = blockIdx.y * kLanes * VEC + q;
            if (cc >= C) continue;
            float s = 0.f;
#pragma unroll
            for (int t = 0; t < kStrips; ++t) s += red[t][q];
            part[(static_cast<long>(blockIdx.x) * (W + 1) + j) * C + cc] = s;
        }
    }
}

// dw [C][W] and dbias [C] from the blocks' sums: 32 columns of [(W + 1)][C] per
// block, 8 threads each adding every eighth partial, then the eight in order.  The blocks from
// sum_blocks on: ds0, one thread per (sequence, vector of channels), from nothing that the
// kernel before writes.
template <typename IO, int VEC, int W>
__global__ void __launch_bounds__(kThreads)
    conv_bwd_tail_kernel(const float* __restrict__ part, float* __restrict__ dw, float* __restrict__ dbias, long nblk,
                         int C, unsigned sum_blocks, const IO* __restrict__ x, long ldx, const float* __restrict__ w,
                         const float* __restrict__ bias, const IO* __restrict__ s0, const IO* __restrict__ dy,
                         long lddy, const IO* __restrict__ dsT, IO* __restrict__ ds0,
                         const int32_t* __restrict__ offs, int B, int T, int act, int* status) {
    if (blockIdx.x >= sum_blocks) {
        const int Cv = C / VEC;
        const long i = static_cast<long>(blockIdx.x - sum_blocks) * kThreads + threadIdx.x;
        if (!ds0) return look_at_spans(offs, i, B, T, status);
        if (i >= static_cast<long>(B) * Cv) return;
        const int c = static_cast<int>(i % Cv) * VEC;
        float wr[W][VEC], br[VEC];
        load_filter<VEC, W>(wr, br, w, bias, c);
        write_state_grad<IO, VEC, W>(x, ldx, s0, dy, lddy, dsT, ds0, wr, br, offs, T, C, act, i / Cv, c, status);
        return;
    }
    chain_wait();
    __shared__ float red[kStrips][kLanes];
    const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
    const long cols = static_cast<long>(W + 1) * C, col = static_cast<long>(blockIdx.x) * kLanes + lane;
    float s = 0.f;
    if (col < cols)
        for (long b = sub; b < nblk; b += kStrips) s += part[b * cols + col];
    red[sub][lane] = s;
    __syncthreads();
    if (sub != 0 || col >= cols) return;
    s = 0.f;
#pragma unroll
    for (int t = 0; t < kStrips; ++t) s += red[t][lane];
    const int j = static_cast<int>(col / C), c = static_cast<int>(col % C);
    if (j < W)
        dw[static_cast<long>(c) * W + j] = s;
    else if (dbias)
        dbias[c] = s;
}

constexpr int kBwdStripRows = 32;  // the halo of W - 1 rows is read and worked on twice (16 rows: 27 us, 32: 24)
constexpr long kWant = 512;

// Blocks that take the sequences: a thread per vector of a state's channels, or per packed
// sequence where no state is wanted.
unsigned state_blocks(int B, int Cv, bool state, bool packed) {
    const long n = state ? static_cast<long>(B) * Cv : packed ? B : 0;
    return static_cast<unsigned>((n + kThreads - 1) / kThreads);
}

// True when VEC-element accesses at any row and at channel multiples of VEC are aligned.
bool vec_ok(int vec, int C, long ld0, long ld1) { return C % vec == 0 && ld0 % vec == 0 && ld1 % vec == 0; }

template <typename IO, int VEC, int W>
cudaError_t fwd_typed(const ConvArgs& p, cudaStream_t st) {
    const int Cv = p.C / VEC;
    const long rows = p.seq_offsets ? p.T : static_cast<long>(p.B) * p.T;
    // Rows per strip: the largest of 64, 32, 16 and 8 that still gives kWant threads for
    // every SM of the device (148 of them): fewer leave too few loads in flight, more and
    // shorter strips load filters and halos more often (1024 threads: 16 us against 13).
    int strip = 64;
    while (strip > 8 && (rows + strip - 1) / strip * Cv < 148L * kWant) strip >>= 1;
    const long strips = (rows + strip - 1) / strip;
    const unsigned nb = static_cast<unsigned>((strips * Cv + kThreads - 1) / kThreads);
    const unsigned ns = state_blocks(p.B, Cv, p.sT, p.seq_offsets);
    auto go = [&](unsigned blocks, unsigned blocks_rows) {
        if (blocks == 0) return;
        conv_fwd_kernel<IO, VEC, W><<<blocks, kThreads, 0, st>>>(
            static_cast<const IO*>(p.x), p.ldx, p.w, p.bias, static_cast<const IO*>(p.s0), static_cast<IO*>(p.y),
            p.ldy, static_cast<IO*>(p.sT), p.seq_offsets, p.B, p.T, rows, p.C, p.act, strip, strips, blocks_rows,
            p.status);
    };
    if (p.sT && p.sT == p.s0) {  // in place: every row has read its state before any is overwritten
        go(nb, nb);
        go(ns, 0);
    } else {
        go(nb + ns, nb);
    }
    return cudaGetLastError();
}

template <typename IO, int VEC, int W>
cudaError_t step_typed(const ConvArgs& p, cudaStream_t st) {
    const long n = static_cast<long>(p.B) * (p.C / VEC);
    conv_step_kernel<IO, VEC, W><<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(
        static_cast<const IO*>(p.x), p.ldx, p.w, p.bias, static_cast<const IO*>(p.s0), static_cast<IO*>(p.y), p.ldy,
        static_cast<IO*>(p.sT), p.B, p.C, p.act);
    return cudaGetLastError();
}

template <typename IO, int VEC, int W>
cudaError_t bwd_typed(const ConvBwdArgs& p, cudaStream_t st) {
    const long rows = p.seq_offsets ? p.T : static_cast<long>(p.B) * p.T;
    const long nblk = conv_bwd_blocks(rows);
    const IO *x = static_cast<const IO*>(p.x), *dy = static_cast<const IO*>(p.dy), *s0 = static_cast<const IO*>(p.s0),
             *dsT = static_cast<const IO*>(p.dsT);
    const int Cv = p.C / VEC;
    const unsigned sums = static_cast<unsigned>((static_cast<long>(W + 1) * p.C + kLanes - 1) / kLanes);
    const unsigned states = state_blocks(p.B, Cv, p.ds0, p.seq_offsets);
    auto* tail = conv_bwd_tail_kernel<IO, VEC, W>;
    if (nblk == 0) {  // the call's only kernel: not to start before what the stream holds has ended
        tail<<<sums + states, kThreads, 0, st>>>(p.ws, p.dw, p.dbias, nblk, p.C, sums, x, p.ldx, p.w, p.bias, s0, dy,
                                                 p.lddy, dsT, static_cast<IO*>(p.ds0), p.seq_offsets, p.B, p.T, p.act,
                                                 p.status);
        return cudaGetLastError();
    }
    const dim3 grid(static_cast<unsigned>(nblk), (Cv + kLanes - 1) / kLanes);
    conv_bwd_kernel<IO, VEC, W><<<grid, kThreads, 0, st>>>(x, p.ldx, p.w, p.bias, s0, dy, p.lddy, dsT,
                                                           static_cast<IO*>(p.dx), p.lddx, p.ws, p.seq_offsets, p.B,
                                                           p.T, rows, p.C, p.act, kBwdStripRows, p.status);
    launch_next(tail, sums + states, kThreads, 0, st, p.ws, p.dw, p.dbias, nblk, p.C, sums, x, p.ldx, p.w, p.bias, s0, dy,
                p.lddy, dsT, static_cast<IO*>(p.ds0), p.seq_offsets, p.B, p.T, p.act, p.status);
    return cudaGetLastError();
}

}  // namespace

long conv_bwd_blocks(long rows) { return (rows + kStrips * kBwdStripRows - 1) / (kStrips * kBwdStripRows); }

size_t conv_bwd_workspace_floats(long rows, int C, int W) {
    return static_cast<size_t>(conv_bwd_blocks(rows)) * (W + 1) * C;
}

#define WKV7_CONV_WIDTHS(FN, IO, VEC)                         \
    switch (p.W) {                                            \
        case 2: return FN<IO, VEC, 2>(p, stream);             \
        case 3: return FN<IO, VEC, 3>(p, stream);             \
        default: return FN<IO, VEC, 4>(p, stream);            \
    }

cudaError_t launch_conv(const ConvArgs& p, int io_dtype, cudaStream_t stream) {
    if (io_dtype == WKV7_BF16) {
        if (vec_ok(kVecF, p.C, p.ldx, p.ldy)) WKV7_CONV_WIDTHS(fwd_typed, __nv_bfloat16, kVecF)
        WKV7_CONV_WIDTHS(fwd_typed, __nv_bfloat16, 1)
    }
    if (vec_ok(kVecF, p.C, p.ldx, p.ldy)) WKV7_CONV_WIDTHS(fwd_typed, float, kVecF)
    WKV7_CONV_WIDTHS(fwd_typed, float, 1)
}

cudaError_t launch_conv_step(const ConvArgs& p, int io_dtype, cudaStream_t stream) {
    if (io_dtype == WKV7_BF16) {
        if (vec_ok(8, p.C, p.ldx, p.ldy)) WKV7_CONV_WIDTHS(step_typed, __nv_bfloat16, 8)
        WKV7_CONV_WIDTHS(step_typed, __nv_bfloat16, 1)
    }
    if (vec_ok(4, p.C, p.ldx, p.ldy)) WKV7_CONV_WIDTHS(step_typed, float, 4)
    WKV7_CONV_WIDTHS(step_typed, float, 1)
}

cudaError_t launch_conv_backward(const ConvBwdArgs& p, int io_dtype, cudaStream_t stream) {
    const bool v = vec_ok(kVecB, p.C, p.ldx, p.lddy) && p.lddx % kVecB == 0;
    if (io_dtype == WKV7_BF16) {
        if (v) WKV7_CONV_WIDTHS(bwd_typed, __nv_bfloat16, kVecB)
        WKV7_CONV_WIDTHS(bwd_typed, __nv_bfloat16, 1)
    }
    if (v) WKV7_CONV_WIDTHS(bwd_typed, float, kVecB)
    WKV7_CONV_WIDTHS(bwd_typed, float, 1)
}

}  // namespace wkv7
