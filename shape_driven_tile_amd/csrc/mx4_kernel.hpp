// MX4 (microscaled 4-bit) kernels for gfx950: quantisation, the values back,
// and products on the scaled MFMAs.
//
// The format (sdt.h): blocks of 32 k share a scale 2^(e - 127); values are
// e2m1 codes.  v_mfma_scale_f32_16x16x128_f8f6f4 takes, per lane, one operand
// row's block of 32 codes (16 bytes) and that block's scale byte: lane l holds
// row l % 16 and the block of quarter l / 16.  It adds over k in a fixed tree
// whatever block a quarter holds, so a k-tile of 256 (8 blocks, 128 bytes a
// row) runs as two MFMAs, s = 0 and 1, in which quarter g holds block 2 g + s.
// A lane's two scale bytes of a row are then neighbours, and with four 16-row
// parts to a 64-row scale tile its eight bytes are one 8-byte load, picked
// apart by the instruction's byte selects: no instruction is spent on scales
// in the loop.  Blocks past K have scale bytes of zero on both sides: their
// products are below 36 * 2^-254, so the loop needs no partial k-tile: nothing
// is masked in it.
#pragma once

#include "gemm_kernel.hpp"

namespace sdt {

typedef int int8v_t __attribute__((ext_vector_type(8)));
typedef int int2_t __attribute__((ext_vector_type(2)));
typedef unsigned short ushort2_t __attribute__((ext_vector_type(2)));
typedef float floatx2_t __attribute__((ext_vector_type(2)));

constexpr int kMx4Tile = 512;      // bytes of a scale tile: 64 rows x 8 blocks

// The float 2^(e - 127) of a scale byte (255: NaN).
__device__ __forceinline__ float mx4_scale_value(int e) {
    const uint32_t bits = e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : (uint32_t)e << 23;
    return __builtin_bit_cast(float, bits);
}

// Offset in its tile of the scale byte of row r % 64, block b % 8.
__device__ __forceinline__ int mx4_scale_offset(int r, int b) {
    return (((b >> 1) & 3) * 16 + (r & 15)) * 8 + ((r >> 4) & 3) * 2 + (b & 1);
}

// Element types of the conversions.  `quad` is two packed 16-bit elements.
struct Mx4F16 : F16 {
    static constexpr uint32_t kInf = 0x7c00;
    static __device__ __forceinline__ uint32_t to_codes(uint32_t old, uint32_t two, float scale,
                                                        int sel) {
        const half2_t v = __builtin_bit_cast(half2_t, two);
        switch (sel) {   // an immediate of the instruction
            case 0: return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, v, scale, 0);
            case 1: return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, v, scale, 1);
            case 2: return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, v, scale, 2);
            default: return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, v, scale, 3);
        }
    }
    // The codes of byte `sel` as two packed elements, unscaled (exact).
    static __device__ __forceinline__ vec2 codes(uint32_t w, int sel) {
        switch (sel) {
            case 0: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0);
            case 1: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1);
            case 2: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2);
            default: return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3);
        }
    }
    static __device__ __forceinline__ float widen(uint32_t bits16) {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
    }
};
struct Mx4BF16 : BF16 {
    static constexpr uint32_t kInf = 0x7f80;
    static __device__ __forceinline__ uint32_t to_codes(uint32_t old, uint32_t two, float scale,
                                                        int sel) {
        const bf16x2_t v = __builtin_bit_cast(bf16x2_t, two);
        switch (sel) {
            case 0: return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, v, scale, 0);
            case 1: return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, v, scale, 1);
            case 2: return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, v, scale, 2);
            default: return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, v, scale, 3);
        }
    }
    static __device__ __forceinline__ vec2 codes(uint32_t w, int sel) {
        switch (sel) {
            case 0: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0);
            case 1: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1);
            case 2: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2);
            default: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3);
        }
    }
    static __device__ __forceinline__ float widen(uint32_t bits16) {
        return __builtin_bit_cast(float, bits16 << 16);
    }
};

// ---- quantisation ---------------------------------------------------------------

struct Mx4Quant {
    const uint16_t* X;
    int64_t ldx;           // elements
    const int32_t* index;  // rows named by a list (nullptr: row p itself)
    int divisor;           // with a list: source row index[p] / divisor (0: p)
    int64_t xrows;
    uint8_t* Q;
    int64_t ldq;           // bytes
    uint8_t* S;
    int64_t rows;
    int K, nkt;
};

// Sixteen-byte accesses at any alignment of the element: the memory system takes
// them, and a row that starts off 16 bytes costs no more than the lines it
// straddles.
typedef uint4_t __attribute__((aligned(2))) uint4_any_t;

// Eight elements from x, of which `valid` lie below K: none past K is read.
__device__ __forceinline__ uint4_t mx4_load8(const uint16_t* x, int valid) {
    if (valid >= 8) return *reinterpret_cast<const uint4_any_t*>(x);
    uint4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t lo = 2 * d < valid ? x[2 * d] : 0u;
        const uint32_t hi = 2 * d + 1 < valid ? x[2 * d + 1] : 0u;
        v[d] = lo | (hi << 16);
    }
    return v;
}

// The largest magnitude of packed elements, as a 16-bit pattern without its
// sign: the patterns' order is the magnitudes' (an infinity or a NaN lies at or
// above the infinity's).
__device__ __forceinline__ uint32_t mx4_top(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t w[4] = {a & 0x7fff7fffu, b & 0x7fff7fffu, c & 0x7fff7fffu, d & 0x7fff7fffu};
    ushort2_t m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(ushort2_t, w[i]));
    return m[0] > m[1] ? m[0] : m[1];
}

// Scale byte of a block whose largest magnitude is `top`, and the codes of eight
// of its elements (zeros in a block that holds an infinity or a NaN).
template <typename Elt>
__device__ __forceinline__ int mx4_encode(uint32_t top, uint32_t a, uint32_t b, uint32_t c,
                                          uint32_t d, uint32_t& q) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, Elt::widen(top));
    const int e = top >= Elt::kInf ? 255 : max((int)(bits >> 23) - 2, 0);
    q = 0;
    if (e != 255) {
        const float scale = mx4_scale_value(e);
        q = Elt::to_codes(q, a, scale, 0);
        q = Elt::to_codes(q, b, scale, 1);
        q = Elt::to_codes(q, c, scale, 2);
        q = Elt::to_codes(q, d, scale, 3);
    }
    return e;
}

// One workgroup per 64 x 256 tile (one scale tile).  32 lanes take a row's 256
// elements, 8 each (16 bytes); 4 lanes share a block and agree on its maximum
// by two lane exchanges.  All eight rows of a lane are loaded before the first
// is used.
template <typename Elt>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(Mx4Quant p) {
    __shared__ uint8_t sm[kMx4Tile];
    const int t = threadIdx.x;
    const int64_t rt = blockIdx.x / p.nkt;
    const int kt = blockIdx.x - (int)(rt * p.nkt);
    const int l32 = t & 31;
    const int k = kt * 256 + l32 * 8;
    const int nb = (p.K + 31) / 32;
    const int valid = p.K - k;             // elements of this lane's eight below K

    uint4_t v[8];
    bool have[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = rt * 64 + (t >> 5) + 8 * i;
        int64_t src = row;
        bool ok = row < p.rows;
        if (p.index != nullptr && ok) {
            const int idx = p.index[row];
            ok = idx >= 0;
            if (p.divisor > 0) src = idx / p.divisor;
            ok = ok && src < p.xrows;
        }
        have[i] = ok;
        v[i] = uint4_t{0, 0, 0, 0};
        if (ok) v[i] = mx4_load8(p.X + src * p.ldx + k, valid);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = (t >> 5) + 8 * i;
        uint32_t top = mx4_top(v[i][0], v[i][1], v[i][2], v[i][3]);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        uint32_t q;
        const int e = mx4_encode<Elt>(top, v[i][0], v[i][1], v[i][2], v[i][3], q);
        const int b = l32 >> 2;
        const int64_t row = rt * 64 + r;
        const bool in = kt * 8 + b < nb;
        if (in && have[i])
            *reinterpret_cast<uint32_t*>(p.Q + row * p.ldq + kt * 128 + l32 * 4) = q;
        if ((l32 & 3) == 0) sm[mx4_scale_offset(r, b)] = in && have[i] ? (uint8_t)e : 0;
    }
    __syncthreads();
    if (t < kMx4Tile / 4)
        reinterpret_cast<uint32_t*>(p.S + (int64_t)blockIdx.x * kMx4Tile)[t] =
            reinterpret_cast<const uint32_t*>(sm)[t];
}

struct Mx4QuantTokens {
    const uint16_t* X;
    int64_t ldx;           // elements
    const int32_t* pos;    // plan row of each slot (token * topk + j), -1: none
    uint8_t* Q;
    int64_t ldq;           // bytes
    uint8_t* S;
    int64_t tokens;
    int topk, K, nkt;
};

// The layer's tokens, each quantised once: codes by token (the products gather
// their rows), scales to the tiles of every plan row of the token, two bytes per
// pair of blocks.  Rounded once per token instead of topk times: 4096 tokens of
// 2048, 6 experts each, 22 -> 9 us against quantising the plan's rows.
template <typename Elt>
__global__ __launch_bounds__(256) void mx4_quantize_tokens_kernel(Mx4QuantTokens p) {
    __shared__ uint16_t sm[64 * 4];        // scale bytes of 64 tokens, by pairs of blocks
    const int t = threadIdx.x;
    const int64_t rt = blockIdx.x / p.nkt;
    const int kt = blockIdx.x - (int)(rt * p.nkt);
    const int l32 = t & 31;
    const int k = kt * 256 + l32 * 8;
    const int nb = (p.K + 31) / 32;
    const int valid = p.K - k;
    uint4_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = rt * 64 + (t >> 5) + 8 * i;
        v[i] = uint4_t{0, 0, 0, 0};
        if (row < p.tokens) v[i] = mx4_load8(p.X + row * p.ldx + k, valid);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = (t >> 5) + 8 * i;
        uint32_t top = mx4_top(v[i][0], v[i][1], v[i][2], v[i][3]);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        uint32_t q;
        const int e = mx4_encode<Elt>(top, v[i][0], v[i][1], v[i][2], v[i][3], q);
        const int b = l32 >> 2;
        const int64_t row = rt * 64 + r;
        const bool in = kt * 8 + b < nb;
        if (in && row < p.tokens)
            *reinterpret_cast<uint32_t*>(p.Q + row * p.ldq + kt * 128 + l32 * 4) = q;
        if ((l32 & 3) == 0) reinterpret_cast<uint8_t*>(sm)[r * 8 + b] = in ? (uint8_t)e : 0;
    }
    __syncthreads();
    const int slots = (int)min((int64_t)64, p.tokens - rt * 64) * p.topk;
    for (int i = t; i < slots * 4; i += 256) {
        const int slot = i >> 2, g = i & 3;
        const int row = p.pos[rt * 64 * p.topk + slot];
        if (row < 0) continue;
        uint8_t* tile = p.S + ((int64_t)(row >> 6) * p.nkt + kt) * kMx4Tile;
        *reinterpret_cast<uint16_t*>(tile + mx4_scale_offset(row & 63, 2 * g)) =
            sm[slot / p.topk * 4 + g];
    }
}

struct Mx4Dequant {
    const uint8_t* Q;
    int64_t ldq;
    const uint8_t* S;
    void* Y;
    int64_t ldy;     // elements
    int64_t rows;
    int K, nkt;
};

// The values back: the tile split of the quantiser, eight values a lane.
// OUT: 0 fp16, 1 bf16, 2 fp32.  A code's value and its scale are exact in
// fp32; 16-bit outputs are rounded from there.
template <int OUT>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(Mx4Dequant p) {
    __shared__ uint32_t sm[kMx4Tile / 4];
    const int t = threadIdx.x;
    const int64_t rt = blockIdx.x / p.nkt;
    const int kt = blockIdx.x - (int)(rt * p.nkt);
    if (t < kMx4Tile / 4)
        sm[t] = reinterpret_cast<const uint32_t*>(p.S + (int64_t)blockIdx.x * kMx4Tile)[t];
    const int l32 = t & 31;
    const int k = kt * 256 + l32 * 8;
    const int valid = p.K - k;
    uint32_t q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = rt * 64 + (t >> 5) + 8 * i;
        q[i] = row < p.rows && valid > 0
                   ? *reinterpret_cast<const uint32_t*>(p.Q + row * p.ldq + kt * 128 + l32 * 4)
                   : 0u;
    }
    __syncthreads();
    const uint8_t* sc = reinterpret_cast<const uint8_t*>(sm);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = (t >> 5) + 8 * i;
        const int64_t row = rt * 64 + r;
        if (row >= p.rows || valid <= 0) continue;
        const float scale = mx4_scale_value(sc[mx4_scale_offset(r, l32 >> 2)]);
        float f[8];
        {
            const floatx2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 0);
            const floatx2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 1);
            const floatx2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 2);
            const floatx2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.0f, 3);
            f[0] = a[0] * scale; f[1] = a[1] * scale;
            f[2] = b[0] * scale; f[3] = b[1] * scale;
            f[4] = c[0] * scale; f[5] = c[1] * scale;
            f[6] = d[0] * scale; f[7] = d[1] * scale;
        }
        if constexpr (OUT == 2) {
            float* y = static_cast<float*>(p.Y) + row * p.ldy + k;
            typedef floatx4_t __attribute__((aligned(4))) floatx4_any_t;
            if (valid >= 8) {
                *reinterpret_cast<floatx4_any_t*>(y) = floatx4_t{f[0], f[1], f[2], f[3]};
                *reinterpret_cast<floatx4_any_t*>(y + 4) = floatx4_t{f[4], f[5], f[6], f[7]};
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < valid) y[j] = f[j];
            }
        } else {
            typedef std::conditional_t<OUT == 0, _Float16, __bf16> scalar;
            uint16_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const scalar s = (scalar)f[j];
                h[j] = __builtin_bit_cast(uint16_t, s);
            }
            uint16_t* y = static_cast<uint16_t*>(p.Y) + row * p.ldy + k;
            if (valid >= 8) {
                *reinterpret_cast<uint4_any_t*>(y) = __builtin_bit_cast(uint4_t, h);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < valid) y[j] = h[j];
            }
        }
    }
}

// Row-major scale bytes into tiles: one workgroup of 256 per 64 x 8 tile.
__global__ __launch_bounds__(256) void mx4_pack_scales_kernel(const uint8_t* R, int64_t ldr,
                                                                     int64_t rows, int nb, int nkt,
                                                                     uint8_t* S) {
    const int64_t rt = blockIdx.x / nkt;
    const int kt = blockIdx.x - (int)(rt * nkt);
    for (int i = threadIdx.x; i < kMx4Tile; i += 256) {
        const int r = i >> 3, b = i & 7;
        const int64_t row = rt * 64 + r;
        const int blk = kt * 8 + b;
        const uint8_t v = row < rows && blk < nb ? R[row * ldr + blk] : 0;
        S[(int64_t)blockIdx.x * kMx4Tile + mx4_scale_offset(r, b)] = v;
    }
}

// ---- products ----------------------------------------------------------------------

struct Mx4Gemm {
    const uint8_t *A, *B, *B2;     // codes (B2: the gated product's second matrix)
    const uint8_t *SA, *SB, *SB2;  // tiled scales
    uint16_t* C;
    int64_t lda, ldb, ldb2, ldc;   // bytes; ldc elements
    int M, N;
    int rowbytes, nkt;             // codes of one row; k-tiles
    int gm, gn, nxcd;              // output tiles (grouped: gm 64-row tiles of the plan)
    // grouped products: the plan, and the experts' strides in bytes
    const int32_t *tiles, *offsets, *counts;
    int64_t eqb, esb, eqb2, esb2;
    // rows of A by token: row p of the plan is A's row slots[p] / topk (nullptr: p)
    const int32_t* slots;
    int topk;
    uint32_t abytes;               // of all of A's rows, at most kNoRow
    // gated product quantised (QOUT): codes, scales and their k-tiles
    uint8_t *QO, *SO;
    int64_t ldqo;
    int nkto;
};

// A row offset that lies past every descriptor, with any k offset added.
constexpr uint32_t kNoRow = 0x40000000u;

// Byte offset of row `row` (of `rows`) of a workgroup whose first is m0.
__device__ __forceinline__ uint32_t mx4_row_offset(const Mx4Gemm& p, int64_t m0, int row, int rows) {
    if (p.slots == nullptr) return (uint32_t)(row * p.lda);
    if (row >= rows) return kNoRow;
    return (uint32_t)(p.slots[m0 + row] / p.topk) * (uint32_t)p.lda;
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx4_rows_rsrc(const Mx4Gemm& p, int64_t m0,
                                                                int rows) {
    return p.slots == nullptr
               ? make_rsrc(p.A + m0 * p.lda, (uint32_t)((rows - 1) * p.lda + p.rowbytes))
               : make_rsrc(p.A, p.abytes);
}

// acc += B_frag . A_frag^T over one 128-deep half; BYTE_A, BYTE_B pick the
// lane's scale bytes.
template <int BYTE_B, int BYTE_A>
__device__ __forceinline__ floatx4_t mx4_mfma(int4_t b, int4_t a, floatx4_t c, int sb, int sa) {
    const int8v_t b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    const int8v_t a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b8, a8, c, 4, 4, BYTE_B, sb, BYTE_A, sa);
}

// One 16-row part of a 64-row scale tile: byte 2 (part % 2) + s of dword
// part / 2 of the lane's eight.
template <int S, int PB, int PA>
__device__ __forceinline__ floatx4_t mx4_mfma_part(int4_t b, int4_t a, floatx4_t c, int sb, int sa) {
    return mx4_mfma<2 * (PB & 1) + S, 2 * (PA & 1) + S>(b, a, c, sb, sa);
}

// silu(g) * u of the gated product, in fp32.  The empty asm keeps the product an
// fp32 value: left to itself the compiler rounds s * u straight to fp16 in some
// kernels and not in others, and the layer's results would depend on which ran.
__device__ __forceinline__ float silu_mul(float g, float u) {
    const float s = g / (1.0f + expf(-g));
    float r = s * u;
    asm("" : "+v"(r));
    return r;
}

// Rows and expert of 64-row tile `g` of a plan for tiles of BM rows: false
// where a tile of BM rows does not start there.
__device__ __forceinline__ bool mx4_group(const Mx4Gemm& p, int g, int bm64, int& e, int64_t& m0,
                                          int& rows) {
    e = __builtin_amdgcn_readfirstlane(p.tiles[g]);
    if (e < 0) return false;
    const int first = p.offsets[e];
    if (((g - first / 64) % bm64) != 0) return false;
    m0 = (int64_t)g * 64;
    rows = __builtin_amdgcn_readfirstlane(first + p.counts[e] - g * 64);
    return rows > 0;
}

// The few-row product: 16 columns of C per workgroup, whose NW waves split the
// k-tiles (w, w + NW, ...) and read B straight from memory, each code once;
// up to 64 rows of A (four 16-row parts, skipped where there are no rows).
// The waves' partial sums are added in wave order through LDS.  Bound by the
// stream of B: 16 loads of 1 KB are in flight per wave pair, and the many small
// workgroups keep every CU loading.
template <typename Elt, bool GROUPED, bool GATED, int NW>
__global__ __launch_bounds__(NW * 64) void mx4_skinny_kernel(Mx4Gemm p) {
    typedef typename Elt::scalar scalar;
    constexpr int U = 2;                     // k-tiles loaded together
    __shared__ floatx4_t red[(GATED ? 2 : 1) * NW * 4 * 64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l = xcd_remap(blockIdx.x, gridDim.x, p.nxcd);
    const int g = l / p.gn, nt = l - g * p.gn;
    int e = 0, rows;
    int64_t m0;
    if constexpr (GROUPED) {
        if (!mx4_group(p, g, 1, e, m0, rows)) return;
        rows = min(rows, 64);
    } else {
        m0 = (int64_t)g * 64;
        rows = (int)min((int64_t)64, p.M - m0);
    }
    const int nmb = (rows + 15) >> 4;
    const int n0 = nt * 16;
    const int fr = lane & 15, fq = lane >> 4;

    const int rows_b = min(16, p.N - n0);
    const uint32_t sbytes_b = (uint32_t)p.nkt * kMx4Tile;
    const __amdgpu_buffer_rsrc_t ra = mx4_rows_rsrc(p, m0, rows);
    const __amdgpu_buffer_rsrc_t rsa = make_rsrc(p.SA + (m0 / 64) * sbytes_b, sbytes_b);
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc(p.B + e * p.eqb + (int64_t)n0 * p.ldb, (uint32_t)((rows_b - 1) * p.ldb + p.rowbytes));
    const __amdgpu_buffer_rsrc_t rsb =
        make_rsrc(p.SB + e * p.esb + (int64_t)(n0 / 64) * sbytes_b, sbytes_b);
    const __amdgpu_buffer_rsrc_t rb2 = make_rsrc(
        GATED ? p.B2 + e * p.eqb2 + (int64_t)n0 * p.ldb2 : p.B,
        GATED ? (uint32_t)((rows_b - 1) * p.ldb2 + p.rowbytes) : 0u);
    const __amdgpu_buffer_rsrc_t rsb2 = make_rsrc(
        GATED ? p.SB2 + e * p.esb2 + (int64_t)(n0 / 64) * sbytes_b : p.SB, GATED ? sbytes_b : 0u);

    uint32_t voff_a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) voff_a[j] = mx4_row_offset(p, m0, j * 16 + fr, rows) + fq * 32;
    const uint32_t voff_b = (uint32_t)(fr * p.ldb) + fq * 32;
    const uint32_t voff_b2 = GATED ? (uint32_t)(fr * p.ldb2) + fq * 32 : 0u;
    const uint32_t voff_sb = lane * 8 + ((n0 >> 4) & 3) * 2;

    floatx4_t acc[4], acc2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        acc[j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
        acc2[j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    }
    // The k offset goes into the lane offset, which the descriptor's range check
    // covers: the last row's bytes past its blocks are not read.
    auto load16 = [](__amdgpu_buffer_rsrc_t r, uint32_t off) {
        return __builtin_bit_cast(int4_t, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
    };
    for (int kt0 = wave; kt0 < p.nkt; kt0 += NW * U) {
        int4_t fb[U][2], fb2[U][2], fa[U][2];
        int sb[U], sb2[U];
        int2_t sa[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kt = kt0 + u * NW;
            // past the last k-tile: an offset past every descriptor, read as zero
            const bool in = kt < p.nkt;
            const uint32_t so = in ? (uint32_t)kt * 128 : 0x40000000u;
            const uint32_t ss = in ? (uint32_t)kt * kMx4Tile : 0x40000000u;
            fb[u][0] = load16(rb, voff_b + so);
            fb[u][1] = load16(rb, voff_b + 16 + so);
            sb[u] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rsb, voff_sb + ss, 0, 0);
            if constexpr (GATED) {
                fb2[u][0] = load16(rb2, voff_b2 + so);
                fb2[u][1] = load16(rb2, voff_b2 + 16 + so);
                sb2[u] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rsb2, voff_sb + ss, 0, 0);
            }
            fa[u][0] = load16(ra, voff_a[0] + so);
            fa[u][1] = load16(ra, voff_a[0] + 16 + so);
            sa[u] = __builtin_bit_cast(
                int2_t, __builtin_amdgcn_raw_buffer_load_b64(rsa, lane * 8 + ss, 0, 0));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kt = kt0 + u * NW;
            const uint32_t so = kt < p.nkt ? (uint32_t)kt * 128 : 0x40000000u;
            acc[0] = mx4_mfma<0, 0>(fb[u][0], fa[u][0], acc[0], sb[u], sa[u][0]);
            acc[0] = mx4_mfma<1, 1>(fb[u][1], fa[u][1], acc[0], sb[u], sa[u][0]);
            if constexpr (GATED) {
                acc2[0] = mx4_mfma<0, 0>(fb2[u][0], fa[u][0], acc2[0], sb2[u], sa[u][0]);
                acc2[0] = mx4_mfma<1, 1>(fb2[u][1], fa[u][1], acc2[0], sb2[u], sa[u][0]);
            }
#pragma unroll
            for (int j = 1; j < 4; ++j) {
                if (j < nmb) {
                    const uint32_t va = voff_a[j] + so;
                    const int4_t a0 = load16(ra, va), a1 = load16(ra, va + 16);
                    const int s = sa[u][j >> 1];
                    if (j & 1) {
                        acc[j] = mx4_mfma<0, 2>(fb[u][0], a0, acc[j], sb[u], s);
                        acc[j] = mx4_mfma<1, 3>(fb[u][1], a1, acc[j], sb[u], s);
                        if constexpr (GATED) {
                            acc2[j] = mx4_mfma<0, 2>(fb2[u][0], a0, acc2[j], sb2[u], s);
                            acc2[j] = mx4_mfma<1, 3>(fb2[u][1], a1, acc2[j], sb2[u], s);
                        }
                    } else {
                        acc[j] = mx4_mfma<0, 0>(fb[u][0], a0, acc[j], sb[u], s);
                        acc[j] = mx4_mfma<1, 1>(fb[u][1], a1, acc[j], sb[u], s);
                        if constexpr (GATED) {
                            acc2[j] = mx4_mfma<0, 0>(fb2[u][0], a0, acc2[j], sb2[u], s);
                            acc2[j] = mx4_mfma<1, 1>(fb2[u][1], a1, acc2[j], sb2[u], s);
                        }
                    }
                }
            }
        }
    }
    // Part j of every wave to LDS, then wave j adds part j in wave order.
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (j < nmb) {
            red[(wave * 4 + j) * 64 + lane] = acc[j];
            if constexpr (GATED) red[((NW + wave) * 4 + j) * 64 + lane] = acc2[j];
        }
    }
    __syncthreads();
    for (int j = wave; j < nmb; j += NW) {
        floatx4_t s = red[j * 64 + lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += red[(w * 4 + j) * 64 + lane];
        if constexpr (GATED) {
            floatx4_t s2 = red[(NW * 4 + j) * 64 + lane];
#pragma unroll
            for (int w = 1; w < NW; ++w) s2 += red[((NW + w) * 4 + j) * 64 + lane];
#pragma unroll
            for (int d = 0; d < 4; ++d) s[d] = silu_mul(s[d], s2[d]);
        }
        // lane l: row l % 16 of the part, columns 4 (l / 16) .. + 3
        const int m = j * 16 + fr;
        if (m >= rows) continue;
        const int n = n0 + fq * 4;
        uint16_t h[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const scalar v = (scalar)s[d];
            h[d] = __builtin_bit_cast(uint16_t, v);
        }
        uint16_t* c = p.C + (m0 + m) * p.ldc + n;
        if (n + 3 < p.N) {
            *reinterpret_cast<uint2_t*>(c) = __builtin_bit_cast(uint2_t, h);
        } else {
#pragma unroll
            for (int d = 0; d < 4; ++d)
                if (n + d < p.N) c[d] = h[d];
        }
    }
}

// The gated product of a workgroup (64 columns: a wave has 32, one block, of its
// 16 FM rows) rounded to the type, quantised and stored: what mx4_quantize makes
// of it, without its way through memory.  Lane l holds columns 16 i + 4 (l / 16)
// .. + 3 of row l % 16 of part j in out[i][j]; a row's block is in four lanes.
template <typename Elt, int BM, int FM>
__device__ __forceinline__ void mx4_store_quantized(const Mx4Gemm& p, const floatx4_t (&out)[2][FM],
                                                    int64_t m0, int64_t n0, int rows, int wave_m,
                                                    int wave_n, int lane, int4_t* smem) {
    typedef typename Elt::scalar scalar;
    constexpr int WTM = FM * 16;
    // codes: 16 bytes per row of the wave; scales: two bytes (the waves' blocks) per
    // row in the order of the scale tile, whose quarter they are
    uint16_t* codes = reinterpret_cast<uint16_t*>(smem) + (wave_n * BM + wave_m * WTM) * 8;
    uint8_t* scales = reinterpret_cast<uint8_t*>(smem) + 2 * BM * 16;
    const int fr = lane & 15, fq = lane >> 4;
    const int64_t block = n0 / 32 + wave_n;
    const int nb = (p.N + 31) / 32;
    const bool in = block < nb;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const scalar lo = (scalar)out[c >> 1][j][2 * (c & 1)];
            const scalar hi = (scalar)out[c >> 1][j][2 * (c & 1) + 1];
            w[c] = __builtin_bit_cast(uint16_t, lo) |
                   ((uint32_t)__builtin_bit_cast(uint16_t, hi) << 16);
        }
        uint32_t top = mx4_top(w[0], w[1], w[2], w[3]);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        uint32_t q;
        const int e = mx4_encode<Elt>(top, w[0], w[1], w[2], w[3], q);
        codes[(j * 16 + fr) * 8 + fq] = (uint16_t)q;
        codes[(j * 16 + fr) * 8 + 4 + fq] = (uint16_t)(q >> 16);
        const int r = wave_m * WTM + j * 16 + fr;
        if (fq == 0)
            scales[(r >> 6) * 128 + fr * 8 + ((r >> 4) & 3) * 2 + wave_n] =
                in && r < rows ? (uint8_t)e : 0;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (lane < WTM && wave_m * WTM + lane < rows && in)
        *reinterpret_cast<int4_t*>(p.QO + (m0 + wave_m * WTM + lane) * p.ldqo + block * 16) =
            reinterpret_cast<const int4_t*>(codes)[lane];
    __syncthreads();
    // 128 bytes a quarter; the last columns' workgroup also clears the quarters
    // past them, whose blocks hold nothing
    const int t = threadIdx.x;
    const int g0 = (int)(n0 / 64) & 3;
    const int quarters = n0 + 64 >= p.N ? 4 - g0 : 1;
    const int st = t >> 7, g = (t >> 5) & 3;      // 64-row tile, quarter past g0
    const uint32_t* from = reinterpret_cast<const uint32_t*>(scales) + st * 32 + (t & 31);
    if (st * 64 < min(rows, BM) && g < quarters) {
        uint8_t* tile = p.SO + ((m0 / 64 + st) * p.nkto + n0 / 256) * kMx4Tile + (g0 + g) * 128;
        reinterpret_cast<uint32_t*>(tile)[t & 31] = g == 0 ? *from : 0u;
    }
}

// The tiled product: BM x BN outputs per workgroup, WM x WN waves of 16x16x128
// MFMAs.  A stage holds the codes of BM + BN rows x 128 bytes and their scale
// tiles, loaded straight into LDS; NS stages.  16-byte chunk 2 g + s of row r
// (block 2 g + s of the k-tile) is kept at position (4 s + g) ^ swz_pp(r), so a
// fragment read of half s has the conflict-free pattern of the 16-bit kernels.
// One barrier per k-tile: after it the loads of k-tile i + NS go into the stage
// that k-tile i has left, the fragments of i + 1 are read into a second set of
// registers, and the MFMAs of i run.  The LDS of two workgroups fits a CU: one's
// prologue, waits and epilogue run under the other's MFMAs.
// GATED: the B rows of a wave are 32 of the first matrix and the same 32 of the
// second, so a lane holds both factors of its outputs; BN / 2 columns per
// workgroup.  GROUPED: rows are a plan's, the expert's matrices are found from
// the row tile.
template <typename Elt, int BM, int BN, int WM, int WN, int NS, bool GROUPED, bool GATED,
          bool QOUT = false>
__global__ __launch_bounds__(WM * WN * 64, 2) void mx4_gemm_kernel(Mx4Gemm p) {
    constexpr int NW = WM * WN;
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int FM = WTM / 16, FN = WTN / 16;
    constexpr int A_UNITS = BM * 8, B_UNITS = BN * 8;
    constexpr int SA_UNITS = BM / 64 * 32, SB_UNITS = BN / 64 * 32;
    constexpr int S_BASE = A_UNITS + B_UNITS;
    constexpr int STAGE = S_BASE + SA_UNITS + SB_UNITS;
    constexpr int A_DMA = A_UNITS / (64 * NW), B_DMA = B_UNITS / (64 * NW);
    constexpr int ST = (BM + BN) / 64;            // scale tiles of a stage
    constexpr int S_DMA = (ST + NW - 1) / NW;     // per wave (spare waves repeat a tile)
    constexpr int L = A_DMA + B_DMA + S_DMA;
    static_assert(A_UNITS % (64 * NW) == 0 && B_UNITS % (64 * NW) == 0, "whole 8-row slabs");
    static_assert(BM % 64 == 0 && BN % 64 == 0, "whole scale tiles");
    static_assert(!GATED || (WTN == 64 && BN == 128), "gated: 32 + 32 columns per wave");
    static_assert(WTM == 32 || WTM % 64 == 0, "a wave's rows: halves of or whole scale tiles");
    static_assert(WTN == 32 || WTN == 64, "a wave's columns: half of or a whole scale tile");
    static_assert(2 * NS * STAGE * 16 <= 160 * 1024, "the stages of two workgroups fit the LDS");
    static_assert(NW * 256 <= NS * STAGE, "epilogue stage");
    __shared__ int4_t smem[NS * STAGE];

    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wave_m = wave % WM, wave_n = wave / WM;

    const int BNO = GATED ? BN / 2 : BN;          // output columns
    const int logical = xcd_remap(blockIdx.x, p.gm * p.gn, p.nxcd);
    int64_t m0, n0;
    int e = 0, limit;                             // limit: rows of C past m0 that exist
    if constexpr (GROUPED) {
        const int g = logical / p.gn;
        if (!mx4_group(p, g, BM / 64, e, m0, limit)) return;
        n0 = (int64_t)(logical - g * p.gn) * BNO;
    } else {
        GemmParams gp;
        gp.gm = p.gm;
        gp.gn = p.gn;
        grouped_origin(gp, logical, BM, BNO, m0, n0);
        limit = (int)min((int64_t)p.M - m0, (int64_t)BM);
    }
    const int rows_a = min(limit, BM);
    const int rows_b = (int)min((int64_t)BNO, (int64_t)p.N - n0);
    const uint32_t srow = (uint32_t)p.nkt * kMx4Tile;   // scale bytes of 64 rows

    const __amdgpu_buffer_rsrc_t ra = mx4_rows_rsrc(p, m0, rows_a);
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc(p.B + e * p.eqb + n0 * p.ldb, (uint32_t)((rows_b - 1) * p.ldb + p.rowbytes));
    const __amdgpu_buffer_rsrc_t rb2 =
        make_rsrc(GATED ? p.B2 + e * p.eqb2 + n0 * p.ldb2 : p.B,
                  GATED ? (uint32_t)((rows_b - 1) * p.ldb2 + p.rowbytes) : 0u);
    const __amdgpu_buffer_rsrc_t rsa =
        make_rsrc(p.SA + (m0 / 64) * srow, (uint32_t)((rows_a + 63) / 64) * srow);
    const __amdgpu_buffer_rsrc_t rsb = make_rsrc(p.SB + e * p.esb + (n0 / 64) * srow,
                                                 (uint32_t)((rows_b + 63) / 64) * srow);
    const __amdgpu_buffer_rsrc_t rsb2 =
        make_rsrc(GATED ? p.SB2 + e * p.esb2 + (n0 / 64) * srow : p.SB,
                  GATED ? (uint32_t)((rows_b + 63) / 64) * srow : 0u);
    uint32_t voff_a[A_DMA], voff_b[B_DMA];
#pragma unroll
    for (int j = 0; j < A_DMA; ++j) {
        const int row = (wave * A_DMA + j) * 8 + (lane >> 3);
        const int pos = (lane & 7) ^ swz_pp(row);
        voff_a[j] = mx4_row_offset(p, m0, row, rows_a) + ((pos & 3) * 2 + (pos >> 2)) * 16;
    }
#pragma unroll
    for (int j = 0; j < B_DMA; ++j) {
        const int row = (wave * B_DMA + j) * 8 + (lane >> 3);
        const int pos = (lane & 7) ^ swz_pp(row);
        // gated: LDS rows 64 w + 32 h + i are row 32 w + i of matrix h
        const int src = GATED ? (row >> 6) * 32 + (row & 31) : row;
        voff_b[j] = (uint32_t)(src * (GATED && (row & 32) ? p.ldb2 : p.ldb)) +
                    ((pos & 3) * 2 + (pos >> 2)) * 16;
    }
    auto load_tile = [&](int kt, int stage) {
        int4_t* base = smem + stage * STAGE;
        // in the lane offset, which the descriptor's range check covers: the
        // last row's bytes past its blocks are not read
        const uint32_t koff = (uint32_t)kt * 128;
#pragma unroll
        for (int j = 0; j < A_DMA; ++j)
            dma16(ra, base + (wave * A_DMA + j) * 64, voff_a[j] + koff, 0);
#pragma unroll
        for (int j = 0; j < B_DMA; ++j) {
            const bool second = GATED && (((wave * B_DMA + j) * 8) & 32) != 0;
            dma16(second ? rb2 : rb, base + A_UNITS + (wave * B_DMA + j) * 64, voff_b[j] + koff, 0);
        }
#pragma unroll
        for (int j = 0; j < S_DMA; ++j) {
            const int st = (wave * S_DMA + j) % ST;
            int4_t* dst = base + S_BASE + st * 32;
            if (lane < 32) {
                if (st < BM / 64)
                    dma16(rsa, dst, st * srow + lane * 16, kt * kMx4Tile);
                else if (GATED && st > BM / 64)
                    dma16(rsb2, dst, lane * 16, kt * kMx4Tile);
                else
                    dma16(rsb, dst, (st - BM / 64) * srow + lane * 16, kt * kMx4Tile);
            }
        }
    };

    floatx4_t acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    const int frow = lane & 15, fq = lane >> 4;
    const int fsw = swz_pp(frow);
    const int a_row0 = wave_m * WTM + frow;
    const int b_row0 = A_UNITS / 8 + wave_n * WTN + frow;
    constexpr int SAW = FM / 2, SBW = FN / 2;     // scale dwords per lane (two parts each)
    struct Frags {
        int4_t a[2][FM], b[2][FN];
        int sa[SAW], sb[SBW];
    };
    auto read_tile = [&](int stage, Frags& f) {
        const int4_t* base = smem + stage * STAGE;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int chunk = (4 * s + fq) ^ fsw;
#pragma unroll
            for (int j = 0; j < FM; ++j) f.a[s][j] = base[(a_row0 + j * 16) * 8 + chunk];
#pragma unroll
            for (int i = 0; i < FN; ++i) f.b[s][i] = base[(b_row0 + i * 16) * 8 + chunk];
        }
        const int* sbase = reinterpret_cast<const int*>(base + S_BASE);
#pragma unroll
        for (int d = 0; d < SAW; ++d) {
            const int part = wave_m * FM + 2 * d;      // 16-row part of the tile's BM rows
            f.sa[d] = sbase[(part >> 2) * 128 + lane * 2 + ((part >> 1) & 1)];
        }
#pragma unroll
        for (int d = 0; d < SBW; ++d) {
            if constexpr (GATED) {
                // dword d: matrix d's columns 32 wave_n .. + 31 of its one tile
                f.sb[d] = sbase[(BM / 64 + d) * 128 + lane * 2 + (wave_n & 1)];
            } else {
                const int part = wave_n * FN + 2 * d;
                f.sb[d] = sbase[(BM / 64 + (part >> 2)) * 128 + lane * 2 + ((part >> 1) & 1)];
            }
        }
    };
    auto mfma_half = [&](auto half, const Frags& f) {
        constexpr int S = decltype(half)::value;
#pragma unroll
        for (int i = 0; i < FN; i += 2)
#pragma unroll
            for (int j = 0; j < FM; j += 2) {
                const int b = f.sb[i / 2], a = f.sa[j / 2];
                acc[i][j] = mx4_mfma_part<S, 0, 0>(f.b[S][i], f.a[S][j], acc[i][j], b, a);
                acc[i][j + 1] = mx4_mfma_part<S, 0, 1>(f.b[S][i], f.a[S][j + 1], acc[i][j + 1], b, a);
                acc[i + 1][j] = mx4_mfma_part<S, 1, 0>(f.b[S][i + 1], f.a[S][j], acc[i + 1][j], b, a);
                acc[i + 1][j + 1] =
                    mx4_mfma_part<S, 1, 1>(f.b[S][i + 1], f.a[S][j + 1], acc[i + 1][j + 1], b, a);
            }
    };
    auto barrier = [&]() {
        // not __syncthreads: its release would wait for every load in flight
        wait_lds();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    };

    const int nkt = p.nkt;
    Frags f[2];
    int i = 0, s = 0;                             // k-tile, its stage
    auto step = [&](auto waits, Frags& cur, Frags& next) {
        wait_global_loads<decltype(waits)::value>();   // k-tile i + 1 has landed
        barrier();
        const int sn = (s + 1 == NS) ? 0 : s + 1;
        if (i + NS < nkt) load_tile(i + NS, s);
        if (i + 1 < nkt) read_tile(sn, next);
        mfma_half(std::integral_constant<int, 0>{}, cur);
        mfma_half(std::integral_constant<int, 1>{}, cur);
        // keeps the MFMAs, values to the compiler, before the waits that follow
#pragma unroll
        for (int n = 0; n < FN; ++n)
#pragma unroll
            for (int m = 0; m < FM; ++m) asm volatile("" : "+v"(acc[n][m]));
        s = sn;
        ++i;
    };
    using Steady = std::integral_constant<int, (NS - 2) * L>;
    using Last = std::integral_constant<int, 0>;

    for (int j = 0; j < min(nkt, NS); ++j) load_tile(j, j);
    if (nkt >= NS)
        wait_global_loads<(NS - 1) * L>();
    else
        wait_global_loads<0>();
    barrier();
    if (nkt > 0) read_tile(0, f[0]);
    while (i + NS < nkt) {                        // k-tiles i + 1 .. i + NS - 1, and i + NS for the second
        step(Steady{}, f[0], f[1]);
        step(Steady{}, f[1], f[0]);
    }
    while (i < nkt) {
        step(Last{}, f[0], f[1]);
        if (i < nkt) step(Last{}, f[1], f[0]);
    }

    // The stages are not read any more after the last k-tile's barrier (with no
    // k-tile nothing was): 4 KB of them per wave stage its output.
    GemmParams gp;
    gp.C = p.C;
    gp.ldc = p.ldc;
    gp.M = (int)(m0 + rows_a);
    gp.N = p.N;
    int4_t* stage = smem + wave * 256;
    const int64_t mb = m0 + wave_m * WTM;
    if constexpr (GATED) {
        floatx4_t out[FN / 2][FM];
#pragma unroll
        for (int i = 0; i < FN / 2; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    out[i][j][d] = silu_mul(acc[i][j][d], acc[i + FN / 2][j][d]);
        if constexpr (QOUT) {
            mx4_store_quantized<Elt, BM, FM>(p, out, m0, n0, rows_a, wave_m, wave_n, lane, smem);
            return;
        }
        gemm_epilogue<Elt, 16>(gp, out, mb, n0 + wave_n * (WTN / 2), lane, stage);
    } else {
        gemm_epilogue<Elt, 16>(gp, acc, mb, n0 + wave_n * WTN, lane, stage);
    }
}

// ---- 16-bit activations, MX4 weights, one token -------------------------------------

struct Mx4Gemv {
    const uint16_t* x;
    const uint8_t* B;
    int64_t ldb;
    const uint8_t* SB;
    uint16_t* y;
    int N, K, rowbytes, nkt;
};

// y of 16 rows of B per workgroup, whose NW waves split the k-tiles.  Lane l
// takes row l % 16, blocks 2 (l / 16) and + 1 of a k-tile: 32 bytes of codes,
// converted two at a time to the activations' type (exact) and multiplied by
// pairs into an fp32 sum per block, which the block's scale then multiplies
// once.  The four quarters' sums are added by lane exchanges, the waves' in
// wave order through LDS.
template <typename Elt, int NW>
__global__ __launch_bounds__(NW * 64) void mx4_gemv_kernel(Mx4Gemv p) {
    typedef typename Elt::scalar scalar;
    typedef typename Elt::vec2 vec2;
    __shared__ float red[NW * 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n0 = blockIdx.x * 16;
    const int fr = lane & 15, fq = lane >> 4;
    const int rows_b = min(16, p.N - n0);
    const uint32_t srow = (uint32_t)p.nkt * kMx4Tile;
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc(p.B + (int64_t)n0 * p.ldb, (uint32_t)((rows_b - 1) * p.ldb + p.rowbytes));
    const __amdgpu_buffer_rsrc_t rsb = make_rsrc(p.SB + (int64_t)(n0 / 64) * srow, srow);
    const uint32_t voff_b = (uint32_t)(fr * p.ldb) + fq * 32;
    const uint32_t voff_s = lane * 8 + ((n0 >> 4) & 3) * 2;
    const bool aligned = (reinterpret_cast<uintptr_t>(p.x) & 15) == 0;
    float sum = 0.0f;
    for (int kt = wave; kt < p.nkt; kt += NW) {
        int4_t w[2];
        w[0] = __builtin_bit_cast(int4_t,
                                  __builtin_amdgcn_raw_buffer_load_b128(rb, voff_b + kt * 128, 0, 0));
        w[1] = __builtin_bit_cast(
            int4_t, __builtin_amdgcn_raw_buffer_load_b128(rb, voff_b + 16 + kt * 128, 0, 0));
        const int sc =
            (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rsb, voff_s, kt * kMx4Tile, 0);
        const int k0 = kt * 256 + fq * 64;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int kb = k0 + s * 32;
            const int valid = p.K - kb;
            if (valid <= 0) continue;
            uint4_t xv[4];
            if (aligned && valid >= 32) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    xv[c] = *reinterpret_cast<const uint4_t*>(p.x + kb + 8 * c);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int k = 8 * c + 2 * d;
                        const uint32_t lo = k < valid ? p.x[kb + k] : 0u;
                        const uint32_t hi = k + 1 < valid ? p.x[kb + k + 1] : 0u;
                        xv[c][d] = lo | (hi << 16);
                    }
            }
            float part = 0.0f;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const uint32_t xw = xv[c][d];
                    part = Elt::dot2(Elt::codes((uint32_t)w[s][c], d), __builtin_bit_cast(vec2, xw), part);
                }
            sum += part * mx4_scale_value((sc >> (8 * s)) & 255);
        }
    }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (lane < 16) red[wave * 16 + lane] = sum;
    __syncthreads();
    if (threadIdx.x < rows_b) {
        float s = red[threadIdx.x];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += red[w * 16 + threadIdx.x];
        const scalar v = (scalar)s;
        p.y[n0 + threadIdx.x] = __builtin_bit_cast(uint16_t, v);
    }
}

}  // namespace sdt
