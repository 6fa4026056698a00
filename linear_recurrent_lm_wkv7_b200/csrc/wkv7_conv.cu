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
#include "seq_common.cuh"

namespace wkv7 {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // rows loaded before the first of them is used

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
    if constexpr (VEC % 4 == 0) {
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

// The walk over rows: sequence n with rows [lo, hi).
struct Walk {
    int n;
    long lo, hi;
};
__device__ __forceinline__ Walk walk_start(const int32_t* offs, int B, int T, long row, int* status) {
    Walk k;
    k.n = offs ? seq_of_row(offs, B, row) : static_cast<int>(row / T);
    seq_span(offs, k.n, T, k.lo, k.hi, status);
    return k;
}
// Moves on to the sequence of `row`; true when `row` is its first.  Rows of no
// sequence lie outside [lo, hi).
__device__ __forceinline__ bool walk_to(Walk& k, const int32_t* offs, int B, int T, long row, int* status) {
    while (row >= k.hi && k.n + 1 < B) {
        ++k.n;
        seq_span(offs, k.n, T, k.lo, k.hi, status);
    }
    return row == k.lo;
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

// Blocks [0, blocks_rows): y, one thread per (strip, vector of channels).  Blocks
// after them: sT, one thread per (sequence, vector of channels).
template <typename IO, int VEC, int W>
__global__ void __launch_bounds__(kThreads)
    conv_fwd_kernel(const IO* __restrict__ x, long ldx, const float* __restrict__ w, const float* __restrict__ bias,
                    const IO* s0, IO* __restrict__ y, long ldy, IO* sT, const int32_t* __restrict__ offs, int B,
                    int T, long rows, int C, int act, int strip_rows, long strips, unsigned blocks_rows,
                    int* status) {
    const int Cv = C / VEC;
    if (blockIdx.x >= blocks_rows) {
        const long i = static_cast<long>(blockIdx.x - blocks_rows) * kThreads + threadIdx.x;
        if (i < static_cast<long>(B) * Cv)
            write_state<IO, VEC, W>(x, ldx, s0, sT, offs, T, C, i / Cv, static_cast<int>(i % Cv) * VEC, status);
        return;
    }
    const long i = static_cast<long>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= strips * Cv) return;
    const int c = static_cast<int>(i % Cv) * VEC;
    const long r0 = i / Cv * strip_rows, r1 = r0 + strip_rows < rows ? r0 + strip_rows : rows;

    float wr[W][VEC], br[VEC];
    load_filter<VEC, W>(wr, br, w, bias, c);
    Walk k = walk_start(offs, B, T, r0, status);
    float win[W - 1][VEC];  // the rows before the current one
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const long r = r0 - (W - 1) + j;
        if (r >= k.lo)
            load_vec<VEC>(win[j], x + r * ldx + c);
        else
#pragma unroll
            for (int e = 0; e < VEC; ++e) win[j][e] = 0.f;
        if (r < k.lo && r0 > k.lo)
            load_state<IO, VEC>(win[j], s0, k.n, static_cast<int>(r - k.lo) + W - 1, W - 1, C, c);
    }
    for (long r = r0; r < r1; r += kAhead) {
        float nx[kAhead][VEC];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (r + u < r1) load_vec<VEC>(nx[u], x + (r + u) * ldx + c);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (r + u >= r1) break;
            if (walk_to(k, offs, B, T, r + u, status)) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) load_state<IO, VEC>(win[j], s0, k.n, j, W - 1, C, c);
            }
            float out[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float p = br[e];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) p = fmaf(wr[j][e], win[j][e], p);
                out[e] = act_f32(fmaf(wr[W - 1][e], nx[u][e], p), act);
            }
            if (r + u >= k.lo && r + u < k.hi) store_vec<VEC>(y + (r + u) * ldy + c, out);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) win[j][e] = win[j + 1][e];
                win[W - 2][e] = nx[u][e];
            }
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
        out[e] = act_f32(p, act);
    }
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
// the strips go to the workspace, [block][(W + 1)][C], and conv_bwd_sum_kernel adds
// the blocks in their order, so the result does not depend on timing.
constexpr int kLanes = 32, kStrips = kThreads / kLanes;
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
    for (int t = 0; t < W - 1; ++t)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float p = br[e];
#pragma unroll
            for (int j = 0; j < W; ++j) p = fmaf(wr[j][e], row[t + j][e], p);
            g[t][e] = t < len ? g[t][e] * act_grad_f32(p, act) : 0.f;
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
__global__ void __launch_bounds__(kThreads)
    conv_bwd_kernel(const IO* __restrict__ x, long ldx, const float* __restrict__ w, const float* __restrict__ bias,
                    const IO* __restrict__ s0, const IO* __restrict__ dy, long lddy, const IO* __restrict__ dsT,
                    IO* __restrict__ dx, long lddx, IO* __restrict__ ds0, float* __restrict__ part,
                    const int32_t* __restrict__ offs, int B, int T, long rows, int C, int act, int strip_rows,
                    unsigned row_blocks, int* status) {
    const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
    const int c = (blockIdx.y * kLanes + lane) * VEC;
    const bool live = c < C;
    float wr[W][VEC], br[VEC];
    if (live) load_filter<VEC, W>(wr, br, w, bias, c);
    if (blockIdx.x >= row_blocks) {  // ds0: one sequence per strip slot
        const long n = static_cast<long>(blockIdx.x - row_blocks) * kStrips + sub;
        if (live && n < B)
            write_state_grad<IO, VEC, W>(x, ldx, s0, dy, lddy, dsT, ds0, wr, br, offs, T, C, act, n, c, status);
        return;
    }
    float acc[W + 1][VEC];  // dw, then dbias
#pragma unroll
    for (int j = 0; j <= W; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;

    const long r0 = (static_cast<long>(blockIdx.x) * kStrips + sub) * strip_rows;
    const long r1 = r0 + strip_rows < rows ? r0 + strip_rows : rows;
    if (live && r0 < rows) {
        Walk k = walk_start(offs, B, T, r0, status);
        float xw[W][VEC], gq[W][VEC];  // rows u-W+1 .. u
        long hq[W];                    // end row of the sequence of each of them, -1 without one
        int nq[W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            hq[j] = -1;
            nq[j] = 0;
            const long r = r0 - W + j;  // one row older than needed: the first shift drops it
            if (j > 0 && r >= k.lo) {
                load_vec<VEC>(xw[j], x + r * ldx + c);
            } else if (j > 0 && r0 > k.lo) {
                load_state<IO, VEC>(xw[j], s0, k.n, static_cast<int>(r - k.lo) + W - 1, W - 1, C, c);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) xw[j][e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) gq[j][e] = 0.f;
        }
        // rows [r0, r1) and the W - 1 after them, whose g the last dx need
        for (long u = r0; u < r1 + W - 1; ++u) {
            float xv[VEC], g[VEC];
            bool valid = false;
            if (u < rows) {
                load_vec<VEC>(xv, x + u * ldx + c);
                load_vec<VEC>(g, dy + u * lddy + c);
                if (walk_to(k, offs, B, T, u, status)) {
#pragma unroll
                    for (int j = 1; j < W; ++j) load_state<IO, VEC>(xw[j], s0, k.n, j - 1, W - 1, C, c);
                }
                valid = u >= k.lo && u < k.hi;
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) xv[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
#pragma unroll
                for (int j = 0; j + 1 < W; ++j) {
                    xw[j][e] = xw[j + 1][e];
                    gq[j][e] = gq[j + 1][e];
                }
                xw[W - 1][e] = xv[e];
                float p = br[e];
#pragma unroll
                for (int j = 0; j < W; ++j) p = fmaf(wr[j][e], xw[j][e], p);
                gq[W - 1][e] = valid ? g[e] * act_grad_f32(p, act) : 0.f;
                if (u < r1) {
#pragma unroll
                    for (int j = 0; j < W; ++j)
                        acc[j][e] = valid ? fmaf(gq[W - 1][e], xw[j][e], acc[j][e]) : acc[j][e];
                    acc[W][e] += gq[W - 1][e];
                }
            }
#pragma unroll
            for (int j = 0; j + 1 < W; ++j) {
                hq[j] = hq[j + 1];
                nq[j] = nq[j + 1];
            }
            hq[W - 1] = valid ? k.hi : -1;
            nq[W - 1] = k.n;
            const long s = u - (W - 1);
            if (s < r0 || hq[0] < 0) continue;
            float d[VEC];
            const long i = s - (hq[0] - (W - 1));  // row of the final state that x_s is
            if (dsT && i >= 0)
                load_vec<VEC>(d, dsT + (static_cast<long>(nq[0]) * (W - 1) + i) * C + c);
            else
#pragma unroll
                for (int e = 0; e < VEC; ++e) d[e] = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j)
                if (s + j < hq[0])
#pragma unroll
                    for (int e = 0; e < VEC; ++e) d[e] = fmaf(wr[W - 1 - j][e], gq[j][e], d[e]);
            store_vec<VEC>(dx + s * lddx + c, d);
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
// block, 8 threads each adding every eighth partial, then the eight in order.
__global__ void __launch_bounds__(kThreads)
    conv_bwd_sum_kernel(const float* __restrict__ part, float* __restrict__ dw, float* __restrict__ dbias, long nblk,
                        int C, int W) {
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

constexpr int kBwdStripRows = 16;

// True when VEC-element accesses at any row and at channel multiples of VEC are aligned.
bool vec_ok(int vec, int C, long ld0, long ld1) { return C % vec == 0 && ld0 % vec == 0 && ld1 % vec == 0; }

template <typename IO, int VEC, int W>
cudaError_t fwd_typed(const ConvArgs& p, cudaStream_t st) {
    const int Cv = p.C / VEC;
    const long rows = p.seq_offsets ? p.T : static_cast<long>(p.B) * p.T;
    // Rows per strip: the largest of 64, 32, 16 and 8 that still gives 1024 threads for
    // every SM of the device (148 of them), so that enough loads are in flight.
    int strip = 64;
    while (strip > 8 && (rows + strip - 1) / strip * Cv < 148L * 1024) strip >>= 1;
    const long strips = (rows + strip - 1) / strip;
    const unsigned nb = static_cast<unsigned>((strips * Cv + kThreads - 1) / kThreads);
    const unsigned ns = p.sT ? static_cast<unsigned>((static_cast<long>(p.B) * Cv + kThreads - 1) / kThreads) : 0;
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
    const unsigned ns = p.ds0 ? static_cast<unsigned>((p.B + kStrips - 1) / kStrips) : 0;
    const dim3 grid(static_cast<unsigned>(nblk) + ns, (p.C / VEC + kLanes - 1) / kLanes);
    if (grid.x)
        conv_bwd_kernel<IO, VEC, W><<<grid, kThreads, 0, st>>>(
            static_cast<const IO*>(p.x), p.ldx, p.w, p.bias, static_cast<const IO*>(p.s0),
            static_cast<const IO*>(p.dy), p.lddy, static_cast<const IO*>(p.dsT), static_cast<IO*>(p.dx), p.lddx,
            static_cast<IO*>(p.ds0), p.ws, p.seq_offsets, p.B, p.T, rows, p.C, p.act, kBwdStripRows,
            static_cast<unsigned>(nblk), p.status);
    const long cols = static_cast<long>(W + 1) * p.C;
    conv_bwd_sum_kernel<<<static_cast<unsigned>((cols + kLanes - 1) / kLanes), kThreads, 0, st>>>(p.ws, p.dw, p.dbias,
                                                                                                   nblk, p.C, W);
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
        if (vec_ok(8, p.C, p.ldx, p.ldy)) WKV7_CONV_WIDTHS(fwd_typed, __nv_bfloat16, 8)
        WKV7_CONV_WIDTHS(fwd_typed, __nv_bfloat16, 1)
    }
    if (vec_ok(4, p.C, p.ldx, p.ldy)) WKV7_CONV_WIDTHS(fwd_typed, float, 4)
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
