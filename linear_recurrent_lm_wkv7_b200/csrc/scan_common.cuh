// scan_common.cuh — what the selective scan's forward and backward share: the cut
// into sequences, segments and chunks, the per-chunk decays, and the tile loads.
//
//   delta_t = softplus(dt_t + dt_bias) (or dt_t + dt_bias),   a_t = exp(A delta_t)
//   S_t = a_t S_{t-1} + delta_t x_t B_t^T  (64 x N per head),   y_t = S_t C_t + D x_t
//
// With l_t = sum_{i<=t} A delta_i from the start of a chunk of 64 tokens and S_0 the
// state there:
//   y_t = sum_{s<=t} exp(l_t - l_s) (C_t . B_s) delta_s x_s + exp(l_t) S_0 C_t + D x_t
//   S_64 = exp(l_64) S_0 + sum_s exp(l_64 - l_s) delta_s x_s B_s^T
// Only differences l_t - l_s with s <= t are exponentiated, so nothing overflows that
// the recurrence itself would not.  l is summed and kept as two floats:
// behind strong decays (|l| of thousands) the difference of two neighbours still
// has 32 bits.
#pragma once
#include "mma_common.cuh"
#include "seq_common.cuh"

namespace wkv7 {

constexpr int kChunk = 64;   // tokens per chunk
constexpr int kScanP = kHead;  // rows of the state
constexpr int kScanThreads = 256;

// Planes of an input; of fp32 values that only go into outputs of the io type (two
// leave an error of 2^-16, far below the rounding to bf16); of those that go into
// states and sums that stay fp32 (two left errors of 3e-6 in states, and of 2e-5 in dA
// where its terms cancel).
template <typename IO>
constexpr int kInPlanes = sizeof(IO) == 2 ? 1 : 3;
template <typename IO>
constexpr int kCalcPlanes = sizeof(IO) == 2 ? 2 : 3;
constexpr int kStatePlanes = 3;

// How sequences are cut into segments of `seg` tokens (a multiple of 64): dense ones
// into spb = ceil(T / seg) slots each; packed ones own the slots from
// offs[n] / seg + n on, which are at least as many as they need and end at
// T / seg + B at the latest.  Where seg covers T, slot n is packed sequence n, whatever the
// offsets hold: each is looked at, and those of a bad pair pass their states on.
struct SegMap {
    const int32_t* offs;
    int B, T;
    long seg;
    int spb;
};
// Whether slots are found through the offsets.
inline __host__ __device__ bool seg_cut(const SegMap& m) { return m.offs && m.seg < m.T; }
inline __host__ __device__ long seg_slots(const SegMap& m) {
    return seg_cut(m) ? m.T / m.seg + m.B : static_cast<long>(m.B) * m.spb;
}
// How a kernel that carries one head's state through chunks is best cut (wkv7_scan.cu).
struct CutCost {
    int chunk;       // tokens per chunk
    int per_sm;      // blocks that an SM runs at once
    double share;    // time of a chunk where it does, of a chunk's alone
    double states;   // time of a chunk in the pass that only makes states, of a chunk's otherwise
    double start;    // time before a block's first chunk, in chunks
    double join;     // of the join and the launches, in chunks
};
SegMap scan_segments(int B, int T, int H, const int32_t* offs, bool packed, const CutCost& cost);
__device__ __forceinline__ long seg_first(const SegMap& m, int n, long lo) {
    return seg_cut(m) ? lo / m.seg + n : static_cast<long>(n) * m.spb;
}
// Sequence n and rows [r0, r1) of a slot; false when the slot is not in use.
__device__ __forceinline__ bool seg_rows(const SegMap& m, long slot, int& n, long& r0, long& r1, long& lo, long& hi,
                                         int* status) {
    if (seg_cut(m)) {
        int a = 0, b = m.B - 1;  // the largest n whose first slot is not behind this one
        while (a < b) {
            const int c = (a + b + 1) >> 1;
            if (m.offs[c] / m.seg + c <= slot)
                a = c;
            else
                b = c - 1;
        }
        n = a;
    } else {
        n = static_cast<int>(slot / m.spb);
    }
    seq_span(m.offs, n, m.T, lo, hi, status);
    r0 = lo + (slot - seg_first(m, n, lo)) * m.seg;
    r1 = r0 + m.seg < hi ? r0 + m.seg : hi;
    return r0 >= lo && r0 < hi;
}

// ---------------------------------------------------------------- decays
// log(1 + e^x) = max(x, 0) + log1p(e^-|x|), to a few 2^-24 of the value: the exponent of 2
// as a sum of two floats, and log1p(t) = 2 artanh(t / (2 + t)) by its series (the argument
// is at most 1/3, so the term z^17 / 17 left out is below 2^-30).  -inf gives 0, NaN NaN.
__device__ __forceinline__ float softplus_f32(float x) {
    const float m = -fabsf(x), h = m * 1.44269504f;
    // -inf has no second part (its products would be NaN)
    const float l = m > -1e30f ? fmaf(m, 1.92596299e-8f, fmaf(m, 1.44269504f, -h)) : 0.f;
    const float t = ex2_ftz(h) * fmaf(l, 0.69314718f, 1.f);
    const float den = 2.f + t, r = rcp_ftz(den);
    const float q = t * r, z = fmaf(fmaf(-q, den, t), r, q), z2 = z * z;
    float p = fmaf(z2, 1.f / 15.f, 1.f / 13.f);
    p = fmaf(p, z2, 1.f / 11.f);
    p = fmaf(p, z2, 1.f / 9.f);
    p = fmaf(p, z2, 1.f / 7.f);
    p = fmaf(p, z2, 1.f / 5.f);
    p = fmaf(p, z2, 1.f / 3.f);
    const float lg = 2.f * fmaf(z * z2, p, z);
    return x > 0.f ? x + lg : x == x ? lg : x;
}

// A sum of two floats, the second below the first's last place.
struct Pair {
    float h, l;
};
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
    const float s = a.h + b.h, v = s - a.h;
    const float l = (a.h - (s - v)) + (b.h - v) + (a.l + b.l);  // what s lost, and the second parts
    const float r = s + l;
    return {r, l - (r - s)};
}
__device__ __forceinline__ Pair pair_mul(float x, Pair a) {
    const float p = x * a.h;
    return {p, fmaf(x, a.l, fmaf(x, a.h, -p))};
}
// A log2(e)
__device__ __forceinline__ Pair log2_rate(float A) {
    return {A * 1.44269504f, fmaf(A, 1.92596299e-8f, fmaf(A, 1.44269504f, -(A * 1.44269504f)))};
}
// Sums over this lane's value and those of the lanes before it.
__device__ __forceinline__ Pair pair_scan(Pair v, int lane) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const Pair o{__shfl_up_sync(0xffffffffu, v.h, m), __shfl_up_sync(0xffffffffu, v.l, m)};
        const Pair t = pair_add(o, v);
        if (lane >= m) v = t;
    }
    return v;
}

// 2^(h + l) for a small second part
__device__ __forceinline__ float exp2_pair(float h, float l) { return ex2_ftz(h) * fmaf(l, 0.69314718f, 1.f); }
// 2^(ah + al - bh - bl)
__device__ __forceinline__ float exp2_diff(float ah, float al, float bh, float bl) {
    const float s = ah - bh, v = s - ah;
    return exp2_pair(s, (ah - (s - v)) - (bh + v) + (al - bl));  // s and its rounding error
}

// Per token of a chunk, in shared memory.  hi + lo = l_t log2(e).
struct Decays {
    float delta[kChunk];  // 0 past the end
    float hi[kChunk], lo[kChunk];
    float from[kChunk];   // exp(l_t): from the chunk's start to t
    float to[kChunk];     // exp(l_64 - l_t): from t to the chunk's end
    float total;          // exp(l_64)
    float pad[3];
};
// exp(l_t - l_s)
__device__ __forceinline__ float decay_between(const Decays& d, int t, int s) {
    return ex2_ftz((d.hi[t] - d.hi[s]) + (d.lo[t] - d.lo[s]));
}

// One warp: the decays of the chunk whose raw dt values lane l holds for tokens 2 l
// and 2 l + 1 (`n` of them exist).
__device__ __forceinline__ void chunk_decays(Decays& d, float dt0, float dt1, int n, float A, float bias,
                                             bool softplus, int lane) {
    float e0 = dt0 + bias, e1 = dt1 + bias;
    if (softplus) {
        e0 = softplus_f32(e0);
        e1 = softplus_f32(e1);
    }
    if (2 * lane >= n) e0 = 0.f;
    if (2 * lane + 1 >= n) e1 = 0.f;
    const Pair rate = log2_rate(A), l0 = pair_mul(e0, rate), l1 = pair_add(l0, pair_mul(e1, rate));
    const Pair run = pair_scan(l1, lane);
    Pair before{__shfl_up_sync(0xffffffffu, run.h, 1), __shfl_up_sync(0xffffffffu, run.l, 1)};
    if (lane == 0) before = {0.f, 0.f};
    const Pair end{__shfl_sync(0xffffffffu, run.h, 31), __shfl_sync(0xffffffffu, run.l, 31)};
    const Pair c0 = pair_add(before, l0), c1 = run;
    *reinterpret_cast<float2*>(&d.delta[2 * lane]) = make_float2(e0, e1);
    *reinterpret_cast<float2*>(&d.hi[2 * lane]) = make_float2(c0.h, c1.h);
    *reinterpret_cast<float2*>(&d.lo[2 * lane]) = make_float2(c0.l, c1.l);
    *reinterpret_cast<float2*>(&d.from[2 * lane]) = make_float2(exp2_pair(c0.h, c0.l), exp2_pair(c1.h, c1.l));
    *reinterpret_cast<float2*>(&d.to[2 * lane]) =
        make_float2(exp2_diff(end.h, end.l, c0.h, c0.l), exp2_diff(end.h, end.l, c1.h, c1.l));
    if (lane == 31) d.total = exp2_pair(end.h, end.l);
}

// The decays of every (chunk slot, head) of `map` (segments of one chunk): out [slot][H].
// Made once, by a warp each: a chunk's take thousands of cycles of dependent steps
// (softplus, a scan in 64 bits), which in the kernels that walk chunks one after the
// other would stand in the way of every chunk (with each kernel making its own, states of
// the backward 117 us against 108 and gradients 170 against 165 at B4 T1024 H32 N128).
struct DecayArgs {
    const void* dt;
    long lddt;
    const float *A, *bias;
    Decays* out;
    int H, softplus, dt_bf16;
    SegMap map;
    int* status;
};
cudaError_t launch_decays(const DecayArgs& a, cudaStream_t stream);
// The cut at every chunk, and how many slots it has at most.
SegMap chunk_map(int B, int T, const int32_t* offs);
long chunk_slots(int B, int T, bool packed);
static_assert(sizeof(Decays) % 16 == 0, "copied in 16-byte pieces");
__device__ __forceinline__ void cp_decays(uint32_t dst, const Decays* src, int tid) {
    if (tid < static_cast<int>(sizeof(Decays) / 16))
        cp_async16(dst + tid * 16, reinterpret_cast<const uint8_t*>(src) + tid * 16, true);
}

// ---------------------------------------------------------------- tile loads
// Rows [0, 64) x COLS of a chunk into a tile: row r from src + r * ld while r < n,
// zeros behind.  bf16: asynchronous copies.  fp32: split into planes on the way.
template <typename TL, int COLS>
__device__ __forceinline__ void load_tile(uint32_t dst, const __nv_bfloat16* src, long ld, int n, int tid,
                                          int threads) {
    constexpr int per = COLS / 8;
    for (int i = tid; i < kChunk * per; i += threads) {
        const int r = i / per, c = i % per;
        cp_async16(dst + r * TL::pitch + c * 16, src + (r < n ? r * ld : 0) + c * 8, r < n);
    }
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t a) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(a) : "memory");
}
// fp32 rows on their way through registers: all of a tile's loads are in flight before
// the first is split (one latency a tile, not one an access).
template <int COLS, int THREADS>
struct TileRegs {
    static constexpr int per = COLS / 4, count = kChunk * per / THREADS;
    static_assert(kChunk * per % THREADS == 0, "whole turns");
    float4 v[count];
    __device__ __forceinline__ void fetch(const float* src, long ld, int n, int tid) {
#pragma unroll
        for (int k = 0; k < count; ++k) {
            const int i = tid + k * THREADS, r = i / per, c = i % per;
            v[k] = r < n ? *reinterpret_cast<const float4*>(src + r * ld + c * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    template <typename TL>
    __device__ __forceinline__ void put(uint32_t dst, int tid) const {
#pragma unroll
        for (int k = 0; k < count; ++k) {
            const int i = tid + k * THREADS, r = i / per, c = i % per;
            uint32_t a[TL::planes], b[TL::planes];
            split_pair<TL::planes, false>(a, v[k].x, v[k].y);
            split_pair<TL::planes, false>(b, v[k].z, v[k].w);
#pragma unroll
            for (int p = 0; p < TL::planes; ++p) sts64(dst + p * TL::plane + r * TL::pitch + c * 8, a[p], b[p]);
        }
    }
};
template <typename TL, int COLS>
__device__ __forceinline__ void load_tile(uint32_t dst, const float* src, long ld, int n, int tid, int) {
    TileRegs<COLS, kScanThreads> t;
    t.fetch(src, ld, n, tid);
    t.template put<TL>(dst, tid);
}

__device__ __forceinline__ float load_dt(const void* dt, long i, bool bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(dt)[i]) : static_cast<const float*>(dt)[i];
}

// The scaled transpose of x as planes: value pairs of an A fragment (tile stored
// [s][p]) times the two tokens' factors.
template <int PIN, int POUT>
__device__ __forceinline__ void scale_frag(uint32_t (&out)[POUT][4], const uint32_t (&in)[PIN][4], float f0, float f1,
                                           float f8, float f9) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float lo = 0.f, hi = 0.f;
#pragma unroll
        for (int p = PIN - 1; p >= 0; --p) {
            lo += bf_lo(in[p][r]);
            hi += bf_hi(in[p][r]);
        }
        uint32_t u[POUT];
        split_pair<POUT, PIN == 1>(u, lo * (r < 2 ? f0 : f8), hi * (r < 2 ? f1 : f9));
#pragma unroll
        for (int p = 0; p < POUT; ++p) out[p][r] = u[p];
    }
}

}  // namespace wkv7
