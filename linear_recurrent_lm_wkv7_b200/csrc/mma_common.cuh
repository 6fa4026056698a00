// mma_common.cuh — warp-level bf16 products of the selective scan: fragments of
// m16n8k16 with fp32 accumulation, fed by ldmatrix from padded shared-memory tiles.
//
// Values of more bits than bf16 are carried as a sum of bf16 planes, each holding the
// leading bits of what the planes before it left over: two planes hold 16 bits of
// mantissa (relative error 2^-16), three hold all 24.  A product of a P-plane by a
// Q-plane value sums the plane products (i, j) with i + j < max(P, Q); what is left
// out is below the last plane's rounding.
//
// Tiles: rows of `cols` bf16 at a pitch of cols + 8 elements.  The pitch is an odd
// number of 16-byte chunks for cols a multiple of 16, so the eight rows that one
// ldmatrix phase reads fall into different banks.
#pragma once
#include <cstdint>

#include "packed_f32.cuh"
#include "sm100_ptx.cuh"

namespace wkv7 {

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm4(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ void stsm2t(uint32_t addr, uint32_t r0, uint32_t r1) {
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(addr), "r"(r0), "r"(r1)
                 : "memory");
}
// 16-byte asynchronous copy, zero-filled when `full` is false (nothing is read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
    const uint32_t n = full ? 16u : 0u;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two floats as bf16 planes, `lo` in the low half of a pair.  All planes but the last of
// two are cut, not rounded (three planes hold 8 + 8 + 8 bits, a whole fp32): cutting is a
// byte permutation, while the rounding conversion runs on the same quarter-rate unit as
// the exponentials.
// CUT = false rounds every plane: for products of two values in planes each, where the
// products left out would add up with one sign.
template <int P, bool CUT = true>
__device__ __forceinline__ void split_pair(uint32_t (&r)[P], float lo, float hi) {
#pragma unroll
    for (int k = 0; k < P; ++k) {
        if (!CUT) {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[k]) : "f"(hi), "f"(lo));
            if (k + 1 < P) {
                lo -= __uint_as_float(r[k] << 16);
                hi -= __uint_as_float(r[k] & 0xffff0000u);
            }
        } else if (P < 3 && k + 1 == P) {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[k]) : "f"(hi), "f"(lo));
        } else {
            const uint32_t a = __float_as_uint(lo), b = __float_as_uint(hi);
            r[k] = __byte_perm(a, b, 0x7632);
            if (k + 1 < P) {  // x + (-cut(x)): the sign bit is cut(x)'s top bit
                const float2 v = add2(make_float2(lo, hi), make_float2(__uint_as_float((a & 0xffff0000u) ^ 0x80000000u),
                                                                       __uint_as_float((b & 0xffff0000u) ^ 0x80000000u)));
                lo = v.x, hi = v.y;
            }
        }
    }
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// d += a b over the planes of both.  The tensor cores cut their sums, so each product added to a
// running sum costs up to 2^-23 of it, always towards zero.  With three planes of both, for fp32
// inputs, a step's six products are therefore summed from zero, the smallest first, and added
// in fp32: a cut of the step's own sum instead of six of d.  (Errors against 64 bits of y 1.1e-7
// where they were 4.8e-7, of ddt 2.1e-7 and 1.5e-6, like those of plain fp32 sums; B4 T1024
// H32 N64 211 us and 198, gradients 330 and 323.)
template <int PA, int PB>
__device__ __forceinline__ void mma_planes(float (&d)[4], const uint32_t (&a)[PA][4], const uint32_t (&b)[PB][2]) {
    constexpr int top = PA > PB ? PA : PB;
    if constexpr (PA < 3 || PB < 3) {
#pragma unroll
        for (int i = 0; i < PA; ++i)
#pragma unroll
            for (int j = 0; j < PB; ++j)
                if (i + j < top) mma16816(d, a[i], b[j][0], b[j][1]);
    } else {
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = top - 1; k >= 0; --k)
#pragma unroll
            for (int i = 0; i < PA; ++i)
                if (k - i >= 0 && k - i < PB) mma16816(t, a[i], b[k - i][0], b[k - i][1]);
        const float2 u = add2(make_float2(d[0], d[1]), make_float2(t[0], t[1]));
        const float2 v = add2(make_float2(d[2], d[3]), make_float2(t[2], t[3]));
        d[0] = u.x, d[1] = u.y, d[2] = v.x, d[3] = v.y;
    }
}

// A tile in shared memory: PLANES x ROWS x COLS.
template <int PLANES, int ROWS, int COLS>
struct Tile {
    static constexpr int pitch = (COLS + 8) * 2;  // bytes
    static constexpr int plane = ROWS * pitch;
    static constexpr int bytes = PLANES * plane;
    static constexpr int planes = PLANES;
    __device__ static __forceinline__ uint32_t at(int row, int col) { return row * pitch + col * 2; }
};
// The same without padding, as one contiguous copy brings it: row r holds its 16-byte pieces
// at their index xor a number that differs between rows of the same banks.
template <int PLANES, int ROWS, int COLS>
struct SwizzledTile {
    static constexpr int pitch = COLS * 2;
    static constexpr int plane = ROWS * pitch;
    static constexpr int bytes = PLANES * plane;
    static constexpr int planes = PLANES;
    static constexpr int pieces = COLS / 8, per_line = pitch < 128 ? 128 / pitch : 1;
    __host__ __device__ static constexpr int swizzle(int row) { return row / per_line & (pieces < 8 ? pieces - 1 : 7); }
    __device__ static __forceinline__ uint32_t at(int row, int col) {
        return row * pitch + (col * 2 ^ swizzle(row) * 16);
    }
};

// Lane addresses of the four 8x8 blocks of a 16 x 16 piece at (row, col) of a tile:
// blocks in the order (0,0) (8,0) (0,8) (8,8) of (row, col): the A fragment of a
// row-major A, or with `t` (transposing load) of an A stored [k][m], where row is k.
template <typename TL>
__device__ __forceinline__ uint32_t addr_a(uint32_t base, int row, int col, int lane) {
    return base + TL::at(row + (lane & 15), col + (lane >> 4) * 8);
}
// Order (0,0) (0,8) (8,0) (8,8): two n-tiles' B fragments (k 0-7 and 8-15 of rows
// n 0-7, then of rows n 8-15) from a B stored [n][k].
template <typename TL>
__device__ __forceinline__ uint32_t addr_b(uint32_t base, int row, int col, int lane) {
    return base + TL::at(row + (lane & 7) + (lane >> 4) * 8, col + ((lane >> 3) & 1) * 8);
}

// A fragments [m 16][k 16] of a tile stored [m][k].
template <typename TL>
__device__ __forceinline__ void frag_a(uint32_t (&f)[TL::planes][4], uint32_t base, int m, int k, int lane) {
#pragma unroll
    for (int p = 0; p < TL::planes; ++p) ldsm4(f[p], addr_a<TL>(base + p * TL::plane, m, k, lane));
}
// The same of a tile stored [k][m].
template <typename TL>
__device__ __forceinline__ void frag_a_t(uint32_t (&f)[TL::planes][4], uint32_t base, int m, int k, int lane) {
#pragma unroll
    for (int p = 0; p < TL::planes; ++p) {
        uint32_t r[4];  // (k 0-7, m 0-7), (k 8-15, m 0-7), (k 0-7, m 8-15), (k 8-15, m 8-15)
        ldsm4t(r, addr_a<TL>(base + p * TL::plane, k, m, lane));
        f[p][0] = r[0], f[p][1] = r[2], f[p][2] = r[1], f[p][3] = r[3];
    }
}
// B fragments of two n-tiles [n 16][k 16] of a tile stored [n][k]: f[tile][plane][2].
template <typename TL>
__device__ __forceinline__ void frag_b(uint32_t (&f)[2][TL::planes][2], uint32_t base, int n, int k, int lane) {
#pragma unroll
    for (int p = 0; p < TL::planes; ++p) {
        uint32_t r[4];
        ldsm4(r, addr_b<TL>(base + p * TL::plane, n, k, lane));
        f[0][p][0] = r[0], f[0][p][1] = r[1], f[1][p][0] = r[2], f[1][p][1] = r[3];
    }
}
// The same of a tile stored [k][n].
template <typename TL>
__device__ __forceinline__ void frag_b_t(uint32_t (&f)[2][TL::planes][2], uint32_t base, int n, int k, int lane) {
#pragma unroll
    for (int p = 0; p < TL::planes; ++p) {
        uint32_t r[4];  // (k 0-7, n 0-7), (k 8-15, n 0-7), (k 0-7, n 8-15), (k 8-15, n 8-15)
        ldsm4t(r, addr_a<TL>(base + p * TL::plane, k, n, lane));
        f[0][p][0] = r[0], f[0][p][1] = r[1], f[1][p][0] = r[2], f[1][p][1] = r[3];
    }
}

}  // namespace wkv7
