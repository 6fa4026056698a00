// wkv7_norm.cu — group norm over channels-last rows, with an activation:
//
//   x [N][L][C], G groups of Cg = C / G neighbouring channels; over the L Cg elements
//   of sample n and group g:  mean, var = mean((x - mean)^2), rstd = (var + eps)^-1/2
//   h = (x - mean) rstd,   y = act(h weight[c] + bias[c])
//
// and its gradient.  With q = dy act'(h weight + bias):
//   dbias = sum q,   dweight = sum q h   (over samples and rows)
//   dx = rstd (q w - m1 - h m2),   m1 = mean(q w),  m2 = mean(q w h)  over the group
//
// A few operations per element: memory is the bound, and what matters is to read x
// (and dy) once.  Two forms:
//   row form   (L = 1 and a group that fits a team's registers): a team of up to 32
//              lanes or a block holds the group, takes its mean, then the squares about
//              the mean, and writes; everything is read once.
//   split form (any other size): partial sums per (sample, split of the rows), joined
//              by a second pass that writes y.  x is read twice, the second time from
//              L2 where it fits.
// Measured: bf16 [4096][2048] in 32 groups 10.4 us (3.2 TB/s), its gradient 19.8 us + 3.2 for the
// sums; fp32 [3][2111][960] in 15 groups 28.7 us, two passes over 24 MB.
#include "seq_common.cuh"

namespace wkv7 {
namespace {

constexpr int kThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float rstd_of(float var, float eps) { return 1.f / sqrtf(var + eps); }

// Sum over the team of TEAM threads (32 lanes or fewer: shuffles; 256: the block).
// Every thread gets the same value.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* red) {
    constexpr int LN = TEAM < 32 ? TEAM : 32;
#pragma unroll
    for (int m = LN / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(kFull, v, m);
    if constexpr (TEAM > 32) {
        __syncthreads();  // the previous sum has been read
        if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TEAM / 32; ++i) v += red[i];
    }
    return v;
}

template <int VEC>
__device__ __forceinline__ void load_param(float (&f)[VEC], const float* p, int c, float none) {
    if (p) {
        load_vec<VEC>(f, p + c);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = none;
    }
}

// ---------------------------------------------------------------- row form
// A team stays on one group and walks rows, with the parameters in registers and the
// next row's vectors already on their way.  Block (bx, by): groups bx * gpb .., rows
// by * rpb + team row, in steps of gridDim.y * rpb; gpb * rpb teams in the block.  A
// team's lane holds vectors lane, lane + TEAM, .. of the group: K of them.
struct RowPlace {
    int lane, g, trow, rpb;
    bool member;
};
template <int TEAM>
__device__ __forceinline__ RowPlace row_place(int gpb, int G) {
    RowPlace p;
    p.lane = threadIdx.x % TEAM;
    const int team = threadIdx.x / TEAM;
    p.rpb = kThreads / TEAM / gpb;
    p.g = blockIdx.x * gpb + team % gpb;
    p.trow = team / gpb;
    p.member = p.trow < p.rpb && p.g < G;
    return p;
}

template <typename IO, int VEC, int TEAM, int K>
__global__ void __launch_bounds__(kThreads)
    norm_row_kernel(const IO* __restrict__ x, long ldx, const float* __restrict__ weight,
                    const float* __restrict__ bias, IO* __restrict__ y, long ldy, float* __restrict__ stats, long N,
                    int G, int Cg, int gpb, float eps, int act) {
    __shared__ float red[TEAM > 32 ? TEAM / 32 : 1];
    const RowPlace p = row_place<TEAM>(gpb, G);
    const int nv = Cg / VEC, c0 = p.g * Cg + p.lane * VEC;
    const float inv = 1.f / Cg;
    float wv[K][VEC], bv[K][VEC];
    Raw<IO, VEC> nx[K];
    const long step = static_cast<long>(gridDim.y) * p.rpb;
    long row = static_cast<long>(blockIdx.y) * p.rpb + p.trow;
    auto fetch = [&](long r) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (p.member && r < N && p.lane + k * TEAM < nv) nx[k].load(x + r * ldx + c0 + k * TEAM * VEC);
    };
    fetch(row);
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (p.member && p.lane + k * TEAM < nv) {
            load_param<VEC>(wv[k], weight, c0 + k * TEAM * VEC, 1.f);
            load_param<VEC>(bv[k], bias, c0 + k * TEAM * VEC, 0.f);
        }
    // every thread of the block takes the same number of turns: team_sum is collective
    for (long r0 = static_cast<long>(blockIdx.y) * p.rpb; r0 < N; r0 += step, row += step) {
        const bool live = p.member && row < N;
        float v[K][VEC], s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const bool mine = live && p.lane + k * TEAM < nv;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[k][e] = mine ? nx[k].get(e) : 0.f;
                s += v[k][e];
            }
        }
        fetch(row + step);
        const float mean = team_sum<TEAM>(s, red) * inv;
        s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (p.lane + k * TEAM < nv)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    v[k][e] -= mean;
                    s = fmaf(v[k][e], v[k][e], s);
                }
        const float rstd = rstd_of(team_sum<TEAM>(s, red) * inv, eps);
        if (!live) continue;
        if (stats && p.lane == 0)
            *reinterpret_cast<float2*>(stats + 2 * (row * G + p.g)) = make_float2(mean, rstd);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (p.lane + k * TEAM >= nv) continue;
            float out[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) out[e] = fmaf(v[k][e] * rstd, wv[k][e], bv[k][e]);
            act_vec<IO, VEC>(out, act);
            store_vec<VEC>(y + row * ldy + c0 + k * TEAM * VEC, out);
        }
    }
}

// The sums of dweight and dbias over a team's rows stay in registers; the block's go to
// part [by][2][C].
template <typename IO, int VEC, int TEAM, int K>
__global__ void __launch_bounds__(kThreads)
    norm_row_bwd_kernel(const IO* __restrict__ x, long ldx, const float* __restrict__ weight,
                        const float* __restrict__ bias, const float* __restrict__ stats, const IO* __restrict__ dy,
                        long lddy, IO* __restrict__ dx, long lddx, float* __restrict__ part, long N, int G, int Cg,
                        int gpb, int act) {
    chain_next();
    __shared__ float red[TEAM > 32 ? TEAM / 32 : 1];
    __shared__ float sums[kThreads * VEC];
    const RowPlace p = row_place<TEAM>(gpb, G);
    const int nv = Cg / VEC, c0 = p.g * Cg + p.lane * VEC;
    const float inv = 1.f / Cg;
    float wv[K][VEC], bv[K][VEC], aw[K][VEC], ab[K][VEC];
    Raw<IO, VEC> nx[K], ny[K];
    float2 ns = make_float2(0.f, 0.f);
    const long step = static_cast<long>(gridDim.y) * p.rpb;
    long row = static_cast<long>(blockIdx.y) * p.rpb + p.trow;
    auto fetch = [&](long r) {
        if (!p.member || r >= N) return;
        ns = *reinterpret_cast<const float2*>(stats + 2 * (r * G + p.g));
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (p.lane + k * TEAM < nv) {
                nx[k].load(x + r * ldx + c0 + k * TEAM * VEC);
                ny[k].load(dy + r * lddy + c0 + k * TEAM * VEC);
            }
    };
    fetch(row);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (p.member && p.lane + k * TEAM < nv) {
            load_param<VEC>(wv[k], weight, c0 + k * TEAM * VEC, 1.f);
            load_param<VEC>(bv[k], bias, c0 + k * TEAM * VEC, 0.f);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) aw[k][e] = ab[k][e] = 0.f;
    }
    for (long r0 = static_cast<long>(blockIdx.y) * p.rpb; r0 < N; r0 += step, row += step) {
        const bool live = p.member && row < N;
        const float mean = ns.x, rstd = ns.y;
        float h[K][VEC], q[K][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!live || p.lane + k * TEAM >= nv) continue;
            float pre[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                h[k][e] = (nx[k].get(e) - mean) * rstd;
                pre[e] = fmaf(h[k][e], wv[k][e], bv[k][e]);
                q[k][e] = ny[k].get(e);
            }
            act_grad_vec<IO, VEC>(q[k], pre, act);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                ab[k][e] += q[k][e];
                aw[k][e] = fmaf(q[k][e], h[k][e], aw[k][e]);
                q[k][e] *= wv[k][e];
                s1 += q[k][e];
                s2 = fmaf(q[k][e], h[k][e], s2);
            }
        }
        fetch(row + step);
        const float m1 = team_sum<TEAM>(s1, red) * inv;
        const float m2 = team_sum<TEAM>(s2, red) * inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!live || p.lane + k * TEAM >= nv) continue;
            float d[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) d[e] = rstd * (q[k][e] - m1 - h[k][e] * m2);
            store_vec<VEC>(dx + row * lddx + c0 + k * TEAM * VEC, d);
        }
    }
    // the block's sums: team rows in order
    const long C = static_cast<long>(G) * Cg;
    const int col = threadIdx.x / TEAM % gpb;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < VEC; ++e) sums[threadIdx.x * VEC + e] = which ? ab[k][e] : aw[k][e];
            __syncthreads();
            if (p.trow != 0 || !p.member || p.lane + k * TEAM >= nv) continue;
            float s[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[e] = 0.f;
            for (int t = 0; t < p.rpb; ++t)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[e] += sums[((t * gpb + col) * TEAM + p.lane) * VEC + e];
            store_vec<VEC>(part + (static_cast<long>(blockIdx.y) * 2 + which) * C + c0 + k * TEAM * VEC, s);
        }
}

// out [2][C] = dweight, dbias: the partials [nblk][2][C] added in a fixed order: 32
// columns a block, every 32nd partial a thread, then the 32 sums.
__global__ void __launch_bounds__(1024)
    norm_sum_kernel(const float* __restrict__ part, float* __restrict__ dw, float* __restrict__ db, long nblk,
                    long C) {
    chain_wait();
    __shared__ float red[32][33];
    const int lane = threadIdx.x % 32, sub = threadIdx.x / 32;
    const long col = static_cast<long>(blockIdx.x) * 32 + lane;
    float s = 0.f;
    if (col < 2 * C) {
#pragma unroll 8
        for (long b = sub; b < nblk; b += 32) s += part[b * 2 * C + col];
    }
    red[sub][lane] = s;
    __syncthreads();
    s = red[lane][sub];  // warp `sub` adds column `sub`
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(kFull, s, m);
    const long out = static_cast<long>(blockIdx.x) * 32 + sub;
    if (lane != 0 || out >= 2 * C) return;
    float* dst = out < C ? dw : db;
    if (dst) dst[out < C ? out : out - C] = s;
}

// ---------------------------------------------------------------- split form
// (count, mean, sum of squares about the mean) of a set of values
struct Moments {
    float n, mean, m2;
};
// Of the union of two sets.  No difference of large sums: safe for any mean.
__device__ __forceinline__ Moments merge(const Moments& a, const Moments& b) {
    const float n = a.n + b.n;
    if (n == 0.f) return a;
    const float d = b.mean - a.mean, f = b.n / n;
    return {n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * a.n * f};
}

// Block (sample and split, tile of 256 vectors of channels).  Thread: one vector, every
// `par`-th row of the split.
template <typename IO, int VEC>
__global__ void __launch_bounds__(kThreads)
    norm_stats_kernel(const IO* __restrict__ x, long ldx, float* __restrict__ part, long L, int C, int Cg, int lanes,
                      int splits, long split_rows) {
    chain_next();
    __shared__ Moments mom[kThreads];
    const int par = kThreads / lanes, lane = threadIdx.x % lanes, prow = threadIdx.x / lanes;
    const int c0 = blockIdx.y * lanes * VEC, c = c0 + lane * VEC;
    const bool member = prow < par && c < C;
    const long l0 = static_cast<long>(blockIdx.x % splits) * split_rows;
    const long l1 = l0 + split_rows < L ? l0 + split_rows : L;
    const IO* base = x + static_cast<long>(blockIdx.x / splits) * L * ldx + c;
    // sums about the first value of the thread: exact enough unless that value lies many
    // deviations off, and then it dominates the deviation itself
    float pivot = 0.f, s = 0.f, ss = 0.f;
    long cnt = 0;
    if (member && l0 + prow < l1) {
        float v[VEC];
        load_vec<VEC>(v, base + (l0 + prow) * ldx);
        pivot = v[0];
#pragma unroll 4
        for (long l = l0 + prow; l < l1; l += par) {
            load_vec<VEC>(v, base + l * ldx);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = v[e] - pivot;
                s += d;
                ss = fmaf(d, d, ss);
            }
            cnt += VEC;
        }
    }
    const float n = static_cast<float>(cnt);
    Moments mine{n, 0.f, 0.f};
    if (cnt) {
        const float md = s / n;
        mine.mean = pivot + md;
        mine.m2 = fmaxf(ss - s * md, 0.f);
    }
    mom[threadIdx.x] = mine;
    __syncthreads();
    // one warp per group of the tile: its members' moments, lane by lane, then across lanes
    const int cend = min(c0 + lanes * VEC, C);
    const int warp = threadIdx.x / 32, ln = threadIdx.x % 32;
    const int G = C / Cg;
    for (int g = c0 / Cg + warp; g * Cg < cend; g += kThreads / 32) {
        const int a = (max(g * Cg, c0) - c0) / VEC, b = (min((g + 1) * Cg, cend) - c0) / VEC;
        const int m = (b - a) * par;
        Moments t{0.f, 0.f, 0.f};
        for (int i = ln; i < m; i += 32) t = merge(t, mom[(i / (b - a)) * lanes + a + i % (b - a)]);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
            const Moments o{__shfl_down_sync(kFull, t.n, d), __shfl_down_sync(kFull, t.mean, d),
                            __shfl_down_sync(kFull, t.m2, d)};
            t = merge(t, o);
        }
        if (ln == 0) {
            // [sample][group][tile][split]: what one group is joined from lies together
            float* p = part + (((static_cast<long>(blockIdx.x / splits) * G + g) * gridDim.y + blockIdx.y) * splits + blockIdx.x % splits) * 3;
            p[0] = t.n, p[1] = t.mean, p[2] = t.m2;
        }
    }
}

// Mean and rstd of sample n's group g from the moments of its splits, in the tiles that
// hold it: a whole warp.
__device__ __forceinline__ float2 join_moments(const float* part, long n, int g, int G, int Cg, int splits, int tiles,
                                               int tile_c, float eps, int ln) {
    const int z0 = g * Cg / tile_c, z1 = ((g + 1) * Cg - 1) / tile_c, nz = z1 - z0 + 1;
    const float* base = part + (((n * G + g) * tiles + z0) * splits) * 3;
    // the mean, then the squares about it: no chain of merges, each with a division
    float cnt = 0.f, sum = 0.f, m2 = 0.f;
#pragma unroll 4
    for (int i = ln; i < splits * nz; i += 32) {
        cnt += base[3 * i];
        sum = fmaf(base[3 * i], base[3 * i + 1], sum);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        cnt += __shfl_xor_sync(kFull, cnt, d);
        sum += __shfl_xor_sync(kFull, sum, d);
    }
    const float mean = sum / cnt;
#pragma unroll 4
    for (int i = ln; i < splits * nz; i += 32) {
        const float d = base[3 * i + 1] - mean;
        m2 += fmaf(base[3 * i] * d, d, base[3 * i + 2]);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m2 += __shfl_xor_sync(kFull, m2, d);
    return make_float2(mean, rstd_of(m2 / cnt, eps));
}

// The statistics of every (sample, group), a warp each.
__global__ void __launch_bounds__(kThreads)
    norm_join_kernel(const float* __restrict__ part, float* __restrict__ stats, long units, int G, int Cg, int splits,
                     int tiles, int tile_c, float eps) {
    chain_wait();
    chain_next();
    const long u = static_cast<long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
    if (u >= units) return;
    const float2 s = join_moments(part, u / G, static_cast<int>(u % G), G, Cg, splits, tiles, tile_c, eps,
                                  threadIdx.x % 32);
    if (threadIdx.x % 32 == 0) *reinterpret_cast<float2*>(stats + 2 * u) = s;
}

// y from x and the statistics; thread: one vector of channels (all of one group: VEC
// divides Cg or is 1), rows prow, prow + par, .. of the split.  JOIN: every block joins the
// moments of its tile's groups itself, and the first split writes the statistics.
template <typename IO, int VEC, bool JOIN>
__global__ void __launch_bounds__(kThreads)
    norm_apply_kernel(const IO* __restrict__ x, long ldx, const float* __restrict__ weight,
                      const float* __restrict__ bias, float* __restrict__ stats, IO* __restrict__ y, long ldy, long L,
                      int C, int Cg, int lanes, int splits, long split_rows, int act, const float* __restrict__ part, float eps) {
    chain_wait();
    __shared__ float2 joined[JOIN ? kThreads * VEC : 1];
    const int par = kThreads / lanes, lane = threadIdx.x % lanes, prow = threadIdx.x / lanes;
    const int c0 = blockIdx.y * lanes * VEC, c = c0 + lane * VEC, G = C / Cg;
    const long n = blockIdx.x / splits;
    if constexpr (JOIN) {
        const int cend = min(c0 + lanes * VEC, C), g0 = c0 / Cg;
        for (int g = g0 + threadIdx.x / 32; g * Cg < cend; g += kThreads / 32) {
            const float2 s = join_moments(part, n, g, G, Cg, splits, gridDim.y, lanes * VEC, eps, threadIdx.x % 32);
            if (threadIdx.x % 32 == 0) {
                joined[g - g0] = s;
                if (stats && blockIdx.x % splits == 0) *reinterpret_cast<float2*>(stats + 2 * (n * G + g)) = s;
            }
        }
        __syncthreads();
    }
    if (prow >= par || c >= C) return;
    const long l0 = static_cast<long>(blockIdx.x % splits) * split_rows;
    const long l1 = l0 + split_rows < L ? l0 + split_rows : L;
    const float2 st = JOIN ? joined[c / Cg - c0 / Cg] : *reinterpret_cast<const float2*>(stats + 2 * (n * G + c / Cg));
    float wv[VEC], bv[VEC];
    load_param<VEC>(wv, weight, c, 1.f);
    load_param<VEC>(bv, bias, c, 0.f);
    const IO* src = x + n * L * ldx + c;
    IO* dst = y + n * L * ldy + c;
    auto row = [&](const Raw<IO, VEC>& in, long l) {
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = fmaf((in.get(e) - st.x) * st.y, wv[e], bv[e]);
        act_vec<IO, VEC>(v, act);
        store_vec<VEC>(dst + l * ldy, v);
    };
    long l = l0 + prow;
    Raw<IO, VEC> nx[4];
    for (; l + 3 * par < l1; l += 4 * par) {  // four rows' loads before the first is used
#pragma unroll
        for (int u = 0; u < 4; ++u) nx[u].load(src + (l + u * par) * ldx);
#pragma unroll
        for (int u = 0; u < 4; ++u) row(nx[u], l + u * par);
    }
    for (; l < l1; l += par) {
        nx[0].load(src + l * ldx);
        row(nx[0], l);
    }
}

// Per (sample, split, channel): sum of q h and sum of q, part [sample][split][2][C].
template <typename IO, int VEC>
__global__ void __launch_bounds__(kThreads)
    norm_bwd_sums_kernel(const IO* __restrict__ x, long ldx, const float* __restrict__ weight,
                         const float* __restrict__ bias, const float* __restrict__ stats, const IO* __restrict__ dy,
                         long lddy, float* __restrict__ part, long L, int C, int Cg, int lanes, int splits, long split_rows,
                         int act) {
    chain_next();
    __shared__ float sums[2][kThreads * VEC];
    const int par = kThreads / lanes, lane = threadIdx.x % lanes, prow = threadIdx.x / lanes;
    const int c = (blockIdx.y * lanes + lane) * VEC;
    const bool member = prow < par && c < C;
    const long l0 = static_cast<long>(blockIdx.x % splits) * split_rows;
    const long l1 = l0 + split_rows < L ? l0 + split_rows : L;
    const long n = blockIdx.x / splits;
    float aw[VEC], ab[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) aw[e] = ab[e] = 0.f;
    if (member) {
        const int g = c / Cg;
        const float mean = stats[2 * (n * (C / Cg) + g)], rstd = stats[2 * (n * (C / Cg) + g) + 1];
        float wv[VEC], bv[VEC];
        load_param<VEC>(wv, weight, c, 1.f);
        load_param<VEC>(bv, bias, c, 0.f);
#pragma unroll 4
        for (long l = l0 + prow; l < l1; l += par) {
            float h[VEC], q[VEC];
            load_vec<VEC>(h, x + (n * L + l) * ldx + c);
            load_vec<VEC>(q, dy + (n * L + l) * lddy + c);
            float pre[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                h[e] = (h[e] - mean) * rstd;
                pre[e] = fmaf(h[e], wv[e], bv[e]);
            }
            act_grad_vec<IO, VEC>(q, pre, act);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                ab[e] += q[e];
                aw[e] = fmaf(q[e], h[e], aw[e]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        sums[0][threadIdx.x * VEC + e] = aw[e];
        sums[1][threadIdx.x * VEC + e] = ab[e];
    }
    __syncthreads();
    if (prow != 0 || !member) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float s[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[e] = 0.f;
        for (int t = 0; t < par; ++t)
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[e] += sums[which][(t * lanes + lane) * VEC + e];
        store_vec<VEC>(part + ((n * splits + blockIdx.x % splits) * 2 + which) * C + c, s);
    }
}

// m1 and m2 of every (sample, group): mom [units][2], one block each.
__global__ void __launch_bounds__(kThreads)
    norm_bwd_join_kernel(const float* __restrict__ part, const float* __restrict__ weight, float* __restrict__ mom,
                         long L, int G, int Cg, int splits) {
    chain_wait();
    chain_next();
    __shared__ float red[kThreads / 32];
    const long u = blockIdx.x, n = u / G, C = static_cast<long>(G) * Cg;
    const int g = static_cast<int>(u % G);
    float s1 = 0.f, s2 = 0.f;
    for (long i = threadIdx.x; i < static_cast<long>(splits) * Cg; i += kThreads) {
        const long sp = i / Cg, c = static_cast<long>(g) * Cg + i % Cg;
        const float w = weight ? weight[c] : 1.f;
        const float* p = part + (n * splits + sp) * 2 * C + c;
        s2 = fmaf(w, p[0], s2);
        s1 = fmaf(w, p[C], s1);
    }
    s1 = team_sum<kThreads>(s1, red);
    s2 = team_sum<kThreads>(s2, red);
    if (threadIdx.x == 0) {
        const float cnt = static_cast<float>(L) * Cg;
        mom[2 * u] = s1 / cnt;
        mom[2 * u + 1] = s2 / cnt;
    }
}

template <typename IO, int VEC>
__global__ void __launch_bounds__(kThreads)
    norm_bwd_apply_kernel(const IO* __restrict__ x, long ldx, const float* __restrict__ weight,
                          const float* __restrict__ bias, const float* __restrict__ stats,
                          const float* __restrict__ mom, const IO* __restrict__ dy, long lddy, IO* __restrict__ dx,
                          long lddx, long L, int C, int Cg, int lanes, int splits, long split_rows, int act) {
    chain_wait();
    chain_next();
    const int par = kThreads / lanes, lane = threadIdx.x % lanes, prow = threadIdx.x / lanes;
    const int c = (blockIdx.y * lanes + lane) * VEC;
    if (prow >= par || c >= C) return;
    const long l0 = static_cast<long>(blockIdx.x % splits) * split_rows;
    const long l1 = l0 + split_rows < L ? l0 + split_rows : L;
    const long n = blockIdx.x / splits, u = n * (C / Cg) + c / Cg;
    const float mean = stats[2 * u], rstd = stats[2 * u + 1], m1 = mom[2 * u], m2 = mom[2 * u + 1];
    float wv[VEC], bv[VEC];
    load_param<VEC>(wv, weight, c, 1.f);
    load_param<VEC>(bv, bias, c, 0.f);
#pragma unroll 4
    for (long l = l0 + prow; l < l1; l += par) {
        float h[VEC], q[VEC];
        load_vec<VEC>(h, x + (n * L + l) * ldx + c);
        load_vec<VEC>(q, dy + (n * L + l) * lddy + c);
        float pre[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            h[e] = (h[e] - mean) * rstd;
            pre[e] = fmaf(h[e], wv[e], bv[e]);
        }
        act_grad_vec<IO, VEC>(q, pre, act);
#pragma unroll
        for (int e = 0; e < VEC; ++e) q[e] = rstd * (q[e] * wv[e] - m1 - h[e] * m2);
        store_vec<VEC>(dx + (n * L + l) * lddx + c, q);
    }
}

// ---------------------------------------------------------------- shapes
// VEC elements per access: a 16-byte vector where groups and row strides allow it.
template <typename IO>
bool vec_ok(int Cg, long a, long b, long c) {
    constexpr int v = kVec<IO>;
    return Cg % v == 0 && a % v == 0 && b % v == 0 && c % v == 0;
}

// How the split form cuts [N][L][C]: `lanes` vectors of channels per tile, and splits
// of the rows: some kSplitPerSm blocks for every SM, of 16 rows a thread at least.
constexpr int kSplitPerSm = 2;
struct Split {
    int lanes, tiles, splits;
    long split_rows;
};
Split split_of(long N, long L, int C, int vec) {
    Split s;
    const int nv = C / vec;
    s.lanes = nv < kThreads ? nv : kThreads;
    s.tiles = (nv + s.lanes - 1) / s.lanes;
    const int par = kThreads / s.lanes;
    const long want = (148L * kSplitPerSm + N * s.tiles - 1) / (N * s.tiles);
    const long most = (L + 16L * par - 1) / (16L * par);
    const long n = want < most ? want : most;
    s.split_rows = (L + n - 1) / n;
    s.splits = static_cast<int>((L + s.split_rows - 1) / s.split_rows);
    return s;
}

// Floats of the forward's partial moments, three to a (sample, group, tile, split).  The
// statistics that no caller wants lie behind them and are stored in pairs: rounded up, so
// that they begin on 16 bytes.
size_t moment_floats(const Split& s, long N, int G) {
    return (static_cast<size_t>(N) * s.splits * s.tiles * G * 3 + 3) / 4 * 4;
}

// The row form's team: the smallest that holds nv vectors, 0 when none does.
// Up to 32 lanes hold one vector each, one warp 2 or 4, a block 1 to 4.
int team_of(int nv) {
    for (int t = 1; t <= 32; t <<= 1)
        if (nv <= t) return t;
    if (nv <= 64) return 64;     // 32 lanes x 2
    if (nv <= 128) return 128;   // 32 lanes x 4
    if (nv <= 256) return 256;   // 256 threads x 1
    if (nv <= 1024) return 1024;  // 256 threads x 4
    return 0;
}
int team_threads(int team) { return team <= 32 ? team : team <= 128 ? 32 : 256; }

// The row form's grid: `per_sm` blocks for every SM share the rows, each with at least
// one turn.  Forward: what is resident at once.  Backward: fewer, as every block leaves
// two rows of partial sums.
struct RowGrid {
    int gpb, gx;
    long gy;
};
RowGrid row_grid_of(long N, int G, int team, int per_sm) {
    RowGrid r;
    const int teams = kThreads / team_threads(team);
    r.gpb = G < teams ? G : teams;
    r.gx = (G + r.gpb - 1) / r.gpb;
    const int rpb = teams / r.gpb;
    long gy = (148L * per_sm + r.gx - 1) / r.gx;
    const long most = (N + rpb - 1) / rpb;
    r.gy = gy < most ? gy : most;
    return r;
}

constexpr int kPerSmFwd = 4, kPerSmBwd = 2;
constexpr long kJoinMost = 8192;

#define WKV7_NORM_TEAMS(CALL)              \
    switch (team) {                        \
        case 1: CALL(1, 1); break;         \
        case 2: CALL(2, 1); break;         \
        case 4: CALL(4, 1); break;         \
        case 8: CALL(8, 1); break;         \
        case 16: CALL(16, 1); break;       \
        case 32: CALL(32, 1); break;       \
        case 64: CALL(32, 2); break;       \
        case 128: CALL(32, 4); break;      \
        case 256: CALL(256, 1); break;     \
        default: CALL(256, 4); break;      \
    }

template <typename IO, int VEC>
cudaError_t norm_typed(const NormArgs& p, cudaStream_t st) {
    const int Cg = p.C / p.G;
    const IO* x = static_cast<const IO*>(p.x);
    IO* y = static_cast<IO*>(p.y);
    const long units = static_cast<long>(p.N) * p.G;
    const int team = p.L == 1 ? team_of(Cg / VEC) : 0;
    if (team) {
        const RowGrid r = row_grid_of(p.N, p.G, team, kPerSmFwd);
        const dim3 grid(r.gx, static_cast<unsigned>(r.gy));
#define CALL(TEAM, K)                                                                                            \
    norm_row_kernel<IO, VEC, TEAM, K><<<grid, kThreads, 0, st>>>(x, p.ldx, p.weight, p.bias, y, p.ldy, p.stats,  \
                                                                 p.N, p.G, Cg, r.gpb, p.eps, p.act)
        WKV7_NORM_TEAMS(CALL)
#undef CALL
        return cudaGetLastError();
    }
    const Split s = split_of(p.N, p.L, p.C, VEC);
    float* part = p.ws;
    float* stats = p.stats ? p.stats : part + moment_floats(s, p.N, p.G);
    const dim3 grid(static_cast<unsigned>(p.N) * s.splits, s.tiles);
    norm_stats_kernel<IO, VEC><<<grid, kThreads, 0, st>>>(x, p.ldx, part, p.L, p.C, Cg, s.lanes, s.splits, s.split_rows);
    // A launch less where the blocks can join the moments on the side: up to kJoinMost of
    // them each (45 groups of 99 splits, fp32 [3][2111][960]: 21.4 us against 23 with a
    // launch for the join).
    const int tile_groups = (s.lanes * VEC + Cg - 1) / Cg + 1;
    if (static_cast<long>(tile_groups) * s.splits * ((Cg + s.lanes * VEC - 1) / (s.lanes * VEC) + 1) <= kJoinMost) {
        launch_next(norm_apply_kernel<IO, VEC, true>, grid, kThreads, 0, st, x, p.ldx, p.weight, p.bias, p.stats, y, p.ldy, p.L,
                    p.C, Cg, s.lanes, s.splits, s.split_rows, p.act, part,
                    p.eps);
    } else {
        launch_next(norm_join_kernel, static_cast<unsigned>((units + 7) / 8), kThreads, 0, st, part, stats, units, p.G, Cg, s.splits, s.tiles, s.lanes * VEC, p.eps);
        launch_next(norm_apply_kernel<IO, VEC, false>, grid, kThreads, 0, st, x, p.ldx, p.weight, p.bias, stats, y, p.ldy, p.L,
                    p.C, Cg, s.lanes, s.splits, s.split_rows, p.act, nullptr,
                    p.eps);
    }
    return cudaGetLastError();
}

template <typename IO, int VEC>
cudaError_t norm_bwd_typed(const NormBwdArgs& p, cudaStream_t st) {
    const int Cg = p.C / p.G;
    const IO *x = static_cast<const IO*>(p.x), *dy = static_cast<const IO*>(p.dy);
    IO* dx = static_cast<IO*>(p.dx);
    const int team = p.L == 1 ? team_of(Cg / VEC) : 0;
    long nblk;
    if (p.N == 0 || p.L == 0) {
        nblk = 0;  // no rows: dweight and dbias are zero
    } else if (team) {
        const RowGrid r = row_grid_of(p.N, p.G, team, kPerSmBwd);
        const dim3 grid(r.gx, static_cast<unsigned>(r.gy));
        nblk = r.gy;
#define CALL(TEAM, K)                                                                                             \
    norm_row_bwd_kernel<IO, VEC, TEAM, K><<<grid, kThreads, 0, st>>>(x, p.ldx, p.weight, p.bias, p.stats, dy,     \
                                                                     p.lddy, dx, p.lddx, p.ws, p.N, p.G, Cg,      \
                                                                     r.gpb, p.act)
        WKV7_NORM_TEAMS(CALL)
#undef CALL
    } else {
        const Split s = split_of(p.N, p.L, p.C, VEC);
        nblk = static_cast<long>(p.N) * s.splits;
        float* mom = p.ws + static_cast<size_t>(nblk) * 2 * p.C;
        const dim3 grid(static_cast<unsigned>(p.N) * s.splits, s.tiles);
        norm_bwd_sums_kernel<IO, VEC><<<grid, kThreads, 0, st>>>(x, p.ldx, p.weight, p.bias, p.stats, dy, p.lddy,
                                                                 p.ws, p.L, p.C, Cg, s.lanes, s.splits, s.split_rows, p.act);
        launch_next(norm_bwd_join_kernel, static_cast<unsigned>(static_cast<long>(p.N) * p.G), kThreads, 0, st, p.ws, p.weight, mom, p.L, p.G, Cg, s.splits);
        launch_next(norm_bwd_apply_kernel<IO, VEC>, grid, kThreads, 0, st, x, p.ldx, p.weight, p.bias, p.stats, mom, dy,
                    p.lddy, dx, p.lddx, p.L, p.C, Cg, s.lanes, s.splits, s.split_rows, p.act);
    }
    if (p.dw || p.db)
        launch_next(norm_sum_kernel, static_cast<unsigned>((2L * p.C + 31) / 32), 1024, 0, st, p.ws, p.dw, p.db, nblk,
                    p.C);
    return cudaGetLastError();
}

// Workspace of either vector width (the width depends on the row strides, which the
// size query does not know): the larger.
template <typename IO>
size_t ws_floats(int N, int L, int C, int G, bool backward) {
    size_t most = 0;
    const int Cg = C / G;
    for (int vec : {1, kVec<IO>}) {
        if (Cg % vec) continue;
        const int team = L == 1 ? team_of(Cg / vec) : 0;
        size_t n = 0;
        if (team) {
            if (backward) n = static_cast<size_t>(row_grid_of(N, G, team, kPerSmBwd).gy) * 2 * C;
        } else {
            const Split s = split_of(N, L, C, vec);
            n = backward ? static_cast<size_t>(N) * s.splits * 2 * C + static_cast<size_t>(N) * G * 2
                         : moment_floats(s, N, G) + static_cast<size_t>(N) * G * 2;
        }
        most = n > most ? n : most;
    }
    return most;
}

}  // namespace

size_t norm_workspace_floats(int N, int L, int C, int G, int io_dtype, bool backward) {
    if (N == 0 || L == 0) return 0;
    return io_dtype == WKV7_BF16 ? ws_floats<__nv_bfloat16>(N, L, C, G, backward)
                                 : ws_floats<float>(N, L, C, G, backward);
}

cudaError_t launch_norm(const NormArgs& p, int io_dtype, cudaStream_t stream) {
    const int Cg = p.C / p.G;
    if (io_dtype == WKV7_BF16)
        return vec_ok<__nv_bfloat16>(Cg, p.ldx, p.ldy, 0) ? norm_typed<__nv_bfloat16, 8>(p, stream)
                                                          : norm_typed<__nv_bfloat16, 1>(p, stream);
    return vec_ok<float>(Cg, p.ldx, p.ldy, 0) ? norm_typed<float, 4>(p, stream) : norm_typed<float, 1>(p, stream);
}

cudaError_t launch_norm_backward(const NormBwdArgs& p, int io_dtype, cudaStream_t stream) {
    const int Cg = p.C / p.G;
    if (io_dtype == WKV7_BF16)
        return vec_ok<__nv_bfloat16>(Cg, p.ldx, p.lddy, p.lddx) ? norm_bwd_typed<__nv_bfloat16, 8>(p, stream)
                                                                : norm_bwd_typed<__nv_bfloat16, 1>(p, stream);
    return vec_ok<float>(Cg, p.ldx, p.lddy, p.lddx) ? norm_bwd_typed<float, 4>(p, stream)
                                                    : norm_bwd_typed<float, 1>(p, stream);
}

}  // namespace wkv7
