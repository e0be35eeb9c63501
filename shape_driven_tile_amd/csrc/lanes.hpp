// What the MX4, 8-bit and feed-forward kernels share: loads at any alignment,
// packing, the stores of a wave's outputs from registers.
#pragma once

#include "gemm_kernel.hpp"

namespace sdt {

typedef int int8v_t __attribute__((ext_vector_type(8)));
typedef int int2_t __attribute__((ext_vector_type(2)));
typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));
typedef float floatx2_t __attribute__((ext_vector_type(2)));

// Sixteen-byte accesses at any alignment of the element: the memory system takes
// them, and a row that starts off 16 bytes costs no more than the lines it
// straddles.
typedef uint4_t __attribute__((aligned(2))) uint4_any_t;

// Eight elements from x, of which `valid` lie below K: none past K is read.
template <bool ONCE = false>
__device__ __forceinline__ uint4_t load8(const uint16_t* x, int valid) {
    if (valid >= 8) {
        if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const uint4_any_t*>(x));
        return *reinterpret_cast<const uint4_any_t*>(x);
    }
    uint4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t lo = 2 * d < valid ? x[2 * d] : 0u;
        const uint32_t hi = 2 * d + 1 < valid ? x[2 * d + 1] : 0u;
        v[d] = lo | (hi << 16);
    }
    return v;
}

// A value that no work of this kernel writes, from a uniform address, by a scalar load.
__device__ __forceinline__ int uniform_load(const int32_t* p) {
    return *reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(
        reinterpret_cast<uint64_t>(p));
}

// Two values rounded to the type, packed (one instruction).
template <typename Elt>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const floatx2_t v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, typename Elt::vec2));
}

// silu(g) * u = g / (1 + exp(-g)) * u of the gated product, in fp32: 2^t by the
// hardware instruction (one step off), t = -g log2(e) in two parts so that the
// rounding of t does not grow with g, and the hardware reciprocal (one step off).
// Limited to +-88, where 2^t is still finite and 1 / (1 + 2^t) already below the
// normal numbers.  The library's expf and division took 3 us of a
// 128 x 64 tile's 11.  The empty asm keeps the product an fp32 value: left to
// itself the compiler rounds s * u straight to fp16 in some kernels and not in
// others, and the layer's results would depend on which ran.
__device__ __forceinline__ float silu_mul(float g, float u) {
    constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147182f;
    const float x = -__builtin_amdgcn_fmed3f(g, -88.0f, 88.0f);
    const float t = x * kLog2e;
    const float low = __builtin_fmaf(x, kLog2e, -t) + x * kLog2eLow;
    const float z = __builtin_amdgcn_exp2f(t);
    const float ez = __builtin_fmaf(z * kLn2, low, z);
    const float s = g * __builtin_amdgcn_rcpf(1.0f + ez);
    float r = s * u;
    asm("" : "+v"(r));
    return r;
}

// ---- epilogues in registers ------------------------------------------------------------
// Lane l holds, of the 16 x 16 part (i, j) of a wave's outputs, row l % 16 and
// columns 4 (l / 16) .. + 3.  Lanes of different quarters swap registers
// (v_permlane16_swap: rows 1, 3 of the first operand against rows 0, 2 of the
// second; v_permlane32_swap: its upper half against the lower) until each holds
// 16 bytes of one row, so that no LDS is needed beside the stages in flight.

__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// A wave's FN x FM parts, `left` rows from mb, columns nb .. (of N): 16-byte
// stores, 64 bytes of 16 rows at a time.  Whole in columns they go through a
// descriptor that drops the rows past the last.
template <typename Elt, int FN, int FM>
__device__ __forceinline__ void store_parts(uint16_t* C, int64_t ldc, const floatx4_t (&acc)[FN][FM],
                                            uint32_t mb, int left, uint32_t nb, int N, int lane) {
    const int fr = lane & 15, fq = lane >> 4;
    if (left <= 0) return;
    const int rows = min(left, FM * 16);
    const int columns = N - (int)nb;              // to the right of nb (none where nb is past N)
    const bool whole = columns >= FN * 16 && ldc < (1 << 30) / (FM * 16);   // 32-bit offsets
    C += (int64_t)mb * ldc + nb;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(C, (uint32_t)((rows - 1) * ldc + FN * 16) * 2);
    const int n = (fq & 1) * 16 + (fq >> 1) * 8;
    const uint32_t off = (uint32_t)(fr * (int)ldc + n) * 2;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
#pragma unroll
        for (int i = 0; i < FN; i += 2) {
            uint32_t a0 = pack2<Elt>(acc[i][j][0], acc[i][j][1]);
            uint32_t a1 = pack2<Elt>(acc[i][j][2], acc[i][j][3]);
            uint32_t b0 = pack2<Elt>(acc[i + 1][j][0], acc[i + 1][j][1]);
            uint32_t b1 = pack2<Elt>(acc[i + 1][j][2], acc[i + 1][j][3]);
            swap16(a0, b0);                           // quarters 0, 2: part i; 1, 3: part i + 1
            swap16(a1, b1);
            const uint4_t v = {a0, a1, b0, b1};
            if (whole) {
                __builtin_amdgcn_raw_buffer_store_b128(v, r, off + (uint32_t)(j * 32 * (int)ldc) + i * 32,
                                                       0, 0);
            } else if (j * 16 + fr < rows) {
                uint16_t* c = C + (j * 16 + fr) * ldc + n + i * 16;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    const uint32_t w = v[d >> 1];
                    if (i * 16 + n + d < columns) c[d] = (uint16_t)(w >> (16 * (d & 1)));
                }
            }
        }
    }
}

}  // namespace sdt
