// seq_common.cuh — what the causal convolution, the selective scan and the group
// norm share: 16-byte vectors of either storage type, the activation and its
// derivative, and the walk over packed sequences.
#pragma once
#include "packed_f32.cuh"
#include "sm100_ptx.cuh"
#include "wkv7_internal.cuh"

namespace wkv7 {

// ---------------------------------------------------------------- vectors
// VEC consecutive elements as floats, in accesses of 8 or 16 bytes (VEC = 4 or 8,
// the address aligned to VEC elements) or element by element (VEC = 1).
template <int VEC>
__device__ __forceinline__ void load_vec(float (&f)[VEC], const __nv_bfloat16* p) {
    if constexpr (VEC == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else if constexpr (VEC == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        f[0] = __uint_as_float(u.x << 16), f[1] = __uint_as_float(u.x & 0xffff0000u);
        f[2] = __uint_as_float(u.y << 16), f[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
        static_assert(VEC == 1, "8, 4 or 1 bf16");
        f[0] = __bfloat162float(*p);
    }
}
template <int VEC>
__device__ __forceinline__ void load_vec(float (&f)[VEC], const float* p) {
    if constexpr (VEC == 8) {
        const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 4);
        f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w, f[4] = v.x, f[5] = v.y, f[6] = v.z, f[7] = v.w;
    } else if constexpr (VEC == 4) {
        const float4 u = *reinterpret_cast<const float4*>(p);
        f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
    } else {
        static_assert(VEC == 1, "8, 4 or 1 fp32");
        f[0] = *p;
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&f)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                  pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
    } else {
        static_assert(VEC == 1, "8, 4 or 1 bf16");
        *p = __float2bfloat16_rn(f[0]);
    }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&f)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        static_assert(VEC == 1, "8, 4 or 1 fp32");
        *p = f[0];
    }
}
// A vector as it lies in memory: what waits for its turn in registers takes half of them
// in bf16.
template <typename IO, int VEC>
struct alignas(sizeof(IO) * VEC) Raw {
    IO v[VEC];
    __device__ __forceinline__ void load(const IO* p) { *this = *reinterpret_cast<const Raw*>(p); }
    __device__ __forceinline__ float get(int e) const { return to_f32(v[e]); }
};
// elements of a 16-byte vector
template <typename IO>
constexpr int kVec = 16 / static_cast<int>(sizeof(IO));

// ---------------------------------------------------------------- activation
// 1 / (1 + exp(-x)).  exp(-x) overflows to +inf below x = -88, where the quotient is 0, its
// limit; a subnormal exp(-x) counts as 0 beside the 1.
// The rounding of -x log2(e) to a float is a relative error of 2^-24 |x| in the exponential
// (2^-18 at x = -40): far below a bf16 result's rounding, 2^-9.  For fp32 results that rounding
// error goes in behind the exponential (2^-21 for every x), two values an instruction where
// registers allow it.  (Warm, in a graph: norm of fp32 [3][2111][960] 19.1 us, 18.3 without the
// second part; convolution of fp32 B4 T4096 C2304 54.1 and 53.4, with expf 14 % longer.)
template <typename IO>
__device__ __forceinline__ float sigmoid_one(float x) {
    if constexpr (sizeof(IO) == 2) return rcp_ftz(1.f + ex2_ftz(-1.44269504f * x));
    const float u = fmaxf(-x, -200.f);  // of +inf there would be no second part; SiLU of -inf is NaN
    const float h = u * 1.44269504f, l = fmaf(u, 1.92596299e-8f, fmaf(u, 1.44269504f, -h));
    return rcp_ftz(fmaf(ex2_ftz(h), fmaf(l, 0.69314718f, 1.f), 1.f));
}
__device__ __forceinline__ float2 sigmoid_pair(float2 x) {  // of fp32, the same bits
    const float2 u = make_float2(fmaxf(-x.x, -200.f), fmaxf(-x.y, -200.f));
    const float2 h = mul2(u, make_float2(1.44269504f, 1.44269504f));
    const float2 r = fma2(u, make_float2(1.44269504f, 1.44269504f), make_float2(-h.x, -h.y));
    const float2 l = fma2(u, make_float2(1.92596299e-8f, 1.92596299e-8f), r);
    const float2 c = fma2(l, make_float2(0.69314718f, 0.69314718f), make_float2(1.f, 1.f));
    const float2 n = fma2(make_float2(ex2_ftz(h.x), ex2_ftz(h.y)), c, make_float2(1.f, 1.f));
    return make_float2(rcp_ftz(n.x), rcp_ftz(n.y));
}
template <typename IO, int VEC>
__device__ __forceinline__ void sigmoid_vec(float (&s)[VEC], const float (&x)[VEC]) {
    if constexpr (sizeof(IO) == 2 || VEC == 1) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[e] = sigmoid_one<IO>(x[e]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
            const float2 v = sigmoid_pair(make_float2(x[e], x[e + 1]));
            s[e] = v.x, s[e + 1] = v.y;
        }
    }
}
template <typename IO>
__device__ __forceinline__ float act_one(float x, int act) {
    return act == WKV7_ACT_SILU ? x * sigmoid_one<IO>(x) : x;
}
template <typename IO, int VEC>
__device__ __forceinline__ void act_vec(float (&x)[VEC], int act) {
    if (act != WKV7_ACT_SILU) return;
    float s[VEC];
    sigmoid_vec<IO, VEC>(s, x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) x[e] *= s[e];
}
// g *= d act(x) / dx
template <typename IO, int VEC>
__device__ __forceinline__ void act_grad_vec(float (&g)[VEC], const float (&x)[VEC], int act) {
    if (act != WKV7_ACT_SILU) return;
    float s[VEC];
    sigmoid_vec<IO, VEC>(s, x);
#pragma unroll
    for (int e = 0; e < VEC; ++e) g[e] *= s[e] * (1.f + x[e] * (1.f - s[e]));
}

// ---------------------------------------------------------------- launches of one call
// A call's second and later kernels are launched while the one before still runs, so that
// the way to their start is over when it ends.  Each begins with chain_wait, for every
// thread of every block that reads or overwrites what came before: it returns when the
// kernel before has completed (and with it all before that one).  chain_next, in the kernel
// before, lets the next one come.  A call's first kernel is launched plainly, and so starts
// when all that the stream holds has ended.
// (Four kernels of a packed fp32 scan, 5003 rows of H12 N64: 88 us in plain launches, 82 so.)
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void chain_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_next(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                        const A&... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid, c.blockDim = dim3(threads), c.dynamicSmemBytes = smem, c.stream = stream;
    c.attrs = &attr, c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kern, static_cast<P>(args)...);
}

// ---------------------------------------------------------------- packed sequences
// Start and end row of sequence n of B.  `offs` null: dense sequences of T rows.
// Packed offsets that are not monotone or leave [0, T] give an empty sequence and
// set WKV7_ERR_DEVICE_BOUNDS, so that no row outside the tensors is ever addressed.
__device__ __forceinline__ void seq_span(const int32_t* offs, int n, int T, long& lo, long& hi, int* status) {
    if (!offs) {
        lo = static_cast<long>(n) * T;
        hi = lo + T;
        return;
    }
    lo = offs[n];
    hi = offs[n + 1];
    if (lo < 0 || hi < lo || hi > T) {
        report_status(status, WKV7_ERR_DEVICE_BOUNDS);
        hi = lo = 0;
    }
}

// The sequence that owns packed row `row`: the largest n in [0, B) with
// offs[n] <= row (sequences of no tokens share their offset with the next one and
// are passed over).  The caller checks that row < offs[n + 1].
__device__ __forceinline__ int seq_of_row(const int32_t* offs, int B, long row) {
    int a = 0, b = B - 1;
    while (a < b) {
        const int m = (a + b + 1) >> 1;
        if (offs[m] <= row)
            a = m;
        else
            b = m - 1;
    }
    return a;
}

}  // namespace wkv7
