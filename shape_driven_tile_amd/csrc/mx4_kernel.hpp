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
#include "moe_kernel.hpp"

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
    int nxcd;              // 1: tiles in launch order
};

// Sixteen-byte accesses at any alignment of the element: the memory system takes
// them, and a row that starts off 16 bytes costs no more than the lines it
// straddles.
typedef uint4_t __attribute__((aligned(2))) uint4_any_t;

// Eight elements from x, of which `valid` lie below K: none past K is read.
template <bool ONCE = false>
__device__ __forceinline__ uint4_t mx4_load8(const uint16_t* x, int valid) {
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
// is used.  LARGE (matrices past the caches): neighbouring tiles, which share the
// lines that rows off them straddle, on one XCD, and loads that do not stay
// (8191 x 8170 bf16: 42.9 -> 33.7 us; 4096 x 2048, from the caches, 7.0 -> 7.7).
template <typename Elt, bool LARGE>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(Mx4Quant p) {
    __shared__ uint8_t sm[kMx4Tile];
    const int t = threadIdx.x;
    const int tile = xcd_remap(blockIdx.x, gridDim.x, p.nxcd);
    const int64_t rt = tile / p.nkt;
    const int kt = tile - (int)(rt * p.nkt);
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
        if (ok) v[i] = mx4_load8<LARGE>(p.X + src * p.ldx + k, valid);
    }
    if (t < kMx4Tile / 4) reinterpret_cast<uint32_t*>(sm)[t] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (rt * 64 + 8 * i >= p.rows) break;
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
        reinterpret_cast<uint32_t*>(p.S + (int64_t)tile * kMx4Tile)[t] =
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

// 16 tokens x 256 of the layer's input, read and quantised once; codes and scales
// go to every plan row of the token: `to` holds those of the tokens' slots, ready
// after `prepare`, which runs while the loads are on their way.
template <typename Elt, typename F>
__device__ __forceinline__ void mx4_quantize_token_tile(const Mx4QuantTokens& p, int64_t first, int kt,
                                                        uint16_t* sm, const int32_t* to, F prepare) {
    const int t = threadIdx.x;
    const int l32 = t & 31;
    const int k = kt * 256 + l32 * 8;
    const int nb = (p.K + 31) / 32;
    const int valid = p.K - k;
    uint4_t v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t row = first + (t >> 5) + 8 * i;
        v[i] = uint4_t{0, 0, 0, 0};
        if (row < p.tokens) v[i] = mx4_load8(p.X + row * p.ldx + k, valid);
    }
    const int slots = (int)min((int64_t)16, p.tokens - first) * p.topk;
    prepare(slots);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = (t >> 5) + 8 * i;
        uint32_t top = mx4_top(v[i][0], v[i][1], v[i][2], v[i][3]);
        top = max(top, (uint32_t)__shfl_xor((int)top, 1));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2));
        uint32_t q;
        const int e = mx4_encode<Elt>(top, v[i][0], v[i][1], v[i][2], v[i][3], q);
        const int b = l32 >> 2;
        const bool in = kt * 8 + b < nb;
        // scale bytes of the 16 tokens, by pairs of blocks
        if ((l32 & 3) == 0) reinterpret_cast<uint8_t*>(sm)[r * 8 + b] = in ? (uint8_t)e : 0;
        if (in && first + r < p.tokens) {
            uint8_t* q0 = p.Q + kt * 128 + l32 * 4;
            for (int j = 0; j < p.topk; ++j) {
                const int64_t at = to[r * p.topk + j];
                if (at >= 0) *reinterpret_cast<uint32_t*>(q0 + at * p.ldq) = q;
            }
        }
    }
    __syncthreads();
    for (int i = t; i < slots * 4; i += 256) {
        const int slot = i >> 2, g = i & 3;
        const int row = to[slot];
        if (row < 0) continue;
        uint8_t* tile = p.S + ((int64_t)(row >> 6) * p.nkt + kt) * kMx4Tile;
        *reinterpret_cast<uint16_t*>(tile + mx4_scale_offset(row & 63, 2 * g)) =
            sm[slot / p.topk * 4 + g];
    }
}

// Bound by the writes of the rows' codes (4096 tokens of 2048, 6 experts each: 13 us;
// quantising the plan's rows one by one took 22); 16 tokens a workgroup, so that a
// decode batch also fills the CUs.
template <typename Elt>
__global__ __launch_bounds__(256) void mx4_quantize_tokens_kernel(Mx4QuantTokens p) {
    __shared__ uint16_t sm[16 * 4];
    __shared__ int32_t to[16 * kMaxTopk];
    const int64_t first = (int64_t)(blockIdx.x / p.nkt) * 16;
    mx4_quantize_token_tile<Elt>(p, first, blockIdx.x % p.nkt, sm, to, [&](int slots) {
        for (int i = threadIdx.x; i < slots; i += 256) to[i] = p.pos[first * p.topk + i];
    });
}

// Few slots: the plan and the tokens' quantisation in one launch.  Every workgroup
// makes the plan for itself, a slot a thread, and the first writes its arrays
// (moe_plan's).  One token of 8 experts: 5.0 us, in two launches 4.2 + 3.7; 256
// slots: 11.9 and 4.8 + 4.3, for every slot is compared with all before it.
constexpr int kPlanQuantizeSlots = 64;

template <typename Elt>
__global__ __launch_bounds__(256) void moe_plan_quantize_kernel(PlanParams q, Mx4QuantTokens p) {
    __shared__ uint16_t sm[16 * 4];
    __shared__ alignas(16) int32_t slot[256];
    __shared__ int32_t place[256];
    __shared__ int hist[kMaxExperts];           // an expert's slots, then its first row
    __shared__ int stop[kMaxExperts];           // the row after its last
    __shared__ int owner[256];                  // expert of 64 rows
    __shared__ int wsum[4];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t first = (int64_t)(blockIdx.x / p.nkt) * 16;
    mx4_quantize_token_tile<Elt>(p, first, blockIdx.x % p.nkt, sm, place + first * p.topk, [&](int) {
        const int x = t < q.R ? q.idx[t] : -1;
        const bool valid = x >= 0 && x < q.E;
        slot[t] = valid ? x : -1;
        for (int i = t; i < kMaxExperts; i += 256) hist[i] = 0;
        __syncthreads();
        if (valid) atomicAdd(&hist[x], 1);
        // rank among the slots before it that chose the same expert
        int rank = 0;
        for (int j = 0; j < q.R; j += 4) {
            const int4_t o = *reinterpret_cast<const int4_t*>(slot + j);
#pragma unroll
            for (int c = 0; c < 4; ++c) rank += j + c < t && o[c] == x ? 1 : 0;
        }
        __syncthreads();
        // four experts a thread: where their rows start
        int count[4], start[4], sum = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            count[c] = hist[4 * t + c];
            start[c] = sum;
            sum += (count[c] + 63) & ~63;
        }
        int scan = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(scan, d);
            if (lane >= d) scan += o;
        }
        if (lane == 63) wsum[wave] = scan;
        __syncthreads();
        int before = scan - sum, end = 0;
        for (int w = 0; w < 4; ++w) {
            before += w < wave ? wsum[w] : 0;
            end += wsum[w];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int e = 4 * t + c, at = start[c] + before;
            hist[e] = at;
            stop[e] = at + count[c];
            for (int r = at / 64; r < (at + count[c] + 63) / 64; ++r) owner[r] = e;
            if (blockIdx.x == 0 && e < q.E) {
                q.counts[e] = count[c];
                q.offsets[e] = at;
                if (e == q.E - 1) q.offsets[q.E] = end;
            }
        }
        __syncthreads();
        place[t] = valid ? hist[x] + rank : -1;
        if (blockIdx.x != 0) return;
        if (t < q.R) {
            q.pos[t] = place[t];
            if (valid) q.rows[place[t]] = t;
        }
        for (int r = t; r < q.cap; r += 256)
            if (r >= end || r >= stop[owner[r / 64]]) q.rows[r] = -1;
        for (int r = t; r < q.cap / 64; r += 256) q.tiles[r] = r < end / 64 ? owner[r] : -1;
    });
}

struct Mx4Dequant {
    const uint8_t* Q;
    int64_t ldq;
    const uint8_t* S;
    void* Y;
    int64_t ldy;     // elements
    int64_t rows;
    int K, nkt;
    int nxcd;        // 1: tiles in launch order
};

// The values back: the tile split of the quantiser (8191 x 8170 to bf16 with the
// tiles' order by XCD 30.6 -> 27.7 us), eight values a lane.
// OUT: 0 fp16, 1 bf16, 2 fp32.  A code's value and its scale are exact in
// fp32; 16-bit outputs are rounded from there.
template <int OUT>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(Mx4Dequant p) {
    __shared__ uint32_t sm[kMx4Tile / 4];
    const int t = threadIdx.x;
    const int tile = xcd_remap(blockIdx.x, gridDim.x, p.nxcd);
    const int64_t rt = tile / p.nkt;
    const int kt = tile - (int)(rt * p.nkt);
    if (t < kMx4Tile / 4)
        sm[t] = reinterpret_cast<const uint32_t*>(p.S + (int64_t)tile * kMx4Tile)[t];
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
    uint32_t lda, ldb, ldb2;       // bytes
    int64_t ldc;                   // elements
    int M, N;
    int rowbytes, nkt;             // codes of one row; k-tiles
    int gm, gn, nxcd;              // output tiles (grouped: gm 64-row tiles of the plan)
    // grouped products: the plan, and the experts' strides in bytes
    const int32_t *tiles, *offsets, *counts;
    int experts;
    int64_t eqb, esb, eqb2, esb2;
    // gated product quantised (QOUT): codes, scales and their k-tiles
    uint8_t *QO, *SO;
    int64_t ldqo;
    int nkto;
};

// A value that no work of this kernel writes, from a uniform address, by a scalar load.
__device__ __forceinline__ int uniform_load(const int32_t* p) {
    return *reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(
        reinterpret_cast<uint64_t>(p));
}

// LDS place of a row's 16-byte chunks: chunk c (block c of the k-tile) of row r is
// kept at c ^ mx4_swz(r).  A fragment read of half s takes chunk 2 g + s in quarter
// g; its bank pattern is that of the 16-bit kernels (chunk 4 s + g at 4 s + g ^
// swz_pp(r)) with the places' three bits turned round, so it is as free of
// conflicts.  Chunks in order keep an aligned 64 bytes to four neighbouring lanes
// of a load (halves first: 0-8% slower on most tiles, 3% faster on some).
__device__ __forceinline__ int mx4_swz(int row) {
    return ((row & 1) ? 1 : 0) ^ ((row & 2) ? 3 : 0) ^ ((row & 4) ? 6 : 0);
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

// Expert, first row and rows of 64-row tile `g` of a plan; false where it has none.
__device__ __forceinline__ bool mx4_group(const Mx4Gemm& p, int g, int& e, int64_t& m0, int& rows) {
    e = uniform_load(p.tiles + g);
    if (e < 0) return false;
    m0 = (int64_t)g * 64;
    rows = min(uniform_load(p.offsets + e) + uniform_load(p.counts + e) - g * 64, 64);
    return rows > 0;
}

// Two values rounded to the type, packed (one instruction).
template <typename Elt>
__device__ __forceinline__ uint32_t mx4_pack2(float a, float b) {
    const floatx2_t v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, typename Elt::vec2));
}

// The few-row product: BN columns of C (gated: of each matrix) and up to 64 rows
// per workgroup, whose NW waves split the k-tiles (w, w + NW, ...) and stream B
// once.  Bound by that stream.  Every wave has LDS of its own, so the loop has no
// barrier: rows come straight into it, eight lanes to a row's 128 bytes, several
// k-tiles in flight, and are read from there as fragments.  (Loaded as fragments,
// a lane to a row, each instruction touches 64 lines: 5.8 bytes a clock and CU,
// a third of what memory gives.)  Few rows (NMB = 1: 16) leave the LDS to more
// stages.  The waves' partial sums are added in wave order.  16 x 12288 x 4096: 7.0
// us (3.8 TB/s of weights, 9.9 without the LDS); experts' products of 64 tokens:
// 41 and 25 us (5.2 and 4.3 TB/s).
// A wave's LDS: grouped products have many short tiles, and three workgroups a CU
// with two stages pass them faster than two with three (64 tokens of 32 experts:
// 44.2 -> 41.8 and 27.6 -> 24.6 us; 8 tokens of 64: 21.3 -> 19.7 and 13.5 -> 11.8).
constexpr int skinny_wave_lds(bool grouped) { return (grouped ? 23 : 35) * 1024; }

template <typename Elt, bool GROUPED, bool GATED, bool QOUT, int NW, int NMB>
__device__ __forceinline__ void mx4_skinny_body(const Mx4Gemm& p, char* smem, int e, int64_t m0,
                                                int n0, int rows) {
    typedef typename Elt::scalar scalar;
    constexpr int MATS = GATED ? 2 : 1;
    constexpr int BN = 64 / MATS;
    constexpr int PB = BN / 16;                   // 16-column parts of a matrix
    constexpr int B_BYTES = BN * 128, A_BYTES = NMB * 16 * 128;
    constexpr int STAGE = MATS * (B_BYTES + kMx4Tile) + A_BYTES + kMx4Tile;
    constexpr int kWaveLds = skinny_wave_lds(GROUPED);
    constexpr int NS = kWaveLds / STAGE >= 3 ? 3 : kWaveLds / STAGE;
    constexpr int L = MATS * (B_BYTES / 1024 + 1) + A_BYTES / 1024 + 1;
    static_assert(NS >= 1 && NS * STAGE <= kWaveLds, "a wave's stages");
    static_assert(MATS * PB * NMB * 1024 <= kWaveLds, "a wave's sums");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fq = lane >> 4;
    const int rows_b = min(BN, p.N - n0);
    const uint32_t srow = (uint32_t)p.nkt * kMx4Tile;

    __amdgpu_buffer_rsrc_t rb[MATS], rsb[MATS];
    uint32_t voff_b[MATS][B_BYTES / 1024], voff_a[A_BYTES / 1024];
    const int pos = (lane & 7) ^ mx4_swz(lane >> 3);   // chunk of the k-tile at this place
    const uint32_t chunk = pos * 16;
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
        const uint8_t* q = m == 0 ? p.B + e * p.eqb : p.B2 + e * p.eqb2;
        const uint8_t* sc = m == 0 ? p.SB + e * p.esb : p.SB2 + e * p.esb2;
        const uint32_t ld = m == 0 ? p.ldb : p.ldb2;
        rb[m] = make_rsrc(q + (uint64_t)(uint32_t)n0 * ld, (uint32_t)((rows_b - 1) * ld + p.rowbytes));
        rsb[m] = make_rsrc(sc + (int64_t)(n0 / 64) * srow, srow);
#pragma unroll
        for (int j = 0; j < B_BYTES / 1024; ++j)
            voff_b[m][j] = (uint32_t)((j * 8 + (lane >> 3)) * ld) + chunk;
    }
    const __amdgpu_buffer_rsrc_t ra =
        make_rsrc(p.A + m0 * p.lda, (uint32_t)((rows - 1) * p.lda + p.rowbytes));
    const __amdgpu_buffer_rsrc_t rsa = make_rsrc(p.SA + (m0 / 64) * srow, srow);
#pragma unroll
    for (int j = 0; j < A_BYTES / 1024; ++j)
        voff_a[j] = (uint32_t)((j * 8 + (lane >> 3)) * p.lda) + chunk;

    char* const mine = smem + wave * kWaveLds;
    auto load = [&](int kt, int stage) {
        int4_t* at = reinterpret_cast<int4_t*>(mine + stage * STAGE);
        // in the lane offset, which the descriptor's range check covers
        const uint32_t koff = (uint32_t)kt * 128;
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
#pragma unroll
            for (int j = 0; j < B_BYTES / 1024; ++j) dma16(rb[m], at + j * 64, voff_b[m][j] + koff, 0);
            at += B_BYTES / 16;
        }
#pragma unroll
        for (int j = 0; j < A_BYTES / 1024; ++j) dma16(ra, at + j * 64, voff_a[j] + koff, 0);
        at += A_BYTES / 16;
        if (lane < 32) {
#pragma unroll
            for (int m = 0; m < MATS; ++m) dma16(rsb[m], at + m * 32, lane * 16, kt * kMx4Tile);
            dma16(rsa, at + MATS * 32, lane * 16, kt * kMx4Tile);
        }
    };

    floatx4_t acc[MATS][PB][NMB];
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int i = 0; i < PB; ++i)
#pragma unroll
            for (int j = 0; j < NMB; ++j) acc[m][i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    const int n = (p.nkt - wave + NW - 1) / NW;   // this wave's k-tiles (0 or less: none)
    const int fsw = mx4_swz(fr);
    for (int j = 0; j < min(n, NS); ++j) load(wave + j * NW, j);
    int stage = 0;
    for (int j = 0; j < n; ++j) {
        const int younger = min(n - 1 - j, NS - 1);   // k-tiles that may stay in flight
        if (NS > 2 && younger == 2)
            wait_global_loads<NS == 3 ? 2 * L : 0>();
        else if (NS > 1 && younger == 1)
            wait_global_loads<L>();
        else
            wait_global_loads<0>();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        const int4_t* at = reinterpret_cast<const int4_t*>(mine + stage * STAGE);
        int4_t fb[MATS][2][PB], fa[2][NMB];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int c = (2 * fq + s) ^ fsw;
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int i = 0; i < PB; ++i)
                    fb[m][s][i] = at[m * (B_BYTES / 16) + (i * 16 + fr) * 8 + c];
#pragma unroll
            for (int i = 0; i < NMB; ++i)
                fa[s][i] = at[MATS * (B_BYTES / 16) + (i * 16 + fr) * 8 + c];
        }
        const int2_t* sc = reinterpret_cast<const int2_t*>(at + (MATS * B_BYTES + A_BYTES) / 16);
        int2_t sb[MATS];
#pragma unroll
        for (int m = 0; m < MATS; ++m) sb[m] = sc[m * 64 + lane];
        const int2_t sa = sc[MATS * 64 + lane];
        // BN = 32: the columns are one half of the scale tile, a dword of the lane's two
        if constexpr (BN == 32) {
#pragma unroll
            for (int m = 0; m < MATS; ++m) sb[m][0] = (n0 & 32) ? sb[m][1] : sb[m][0];
        }
        wait_lds();
        __builtin_amdgcn_sched_barrier(0);
        if (j + NS < n) load(wave + (j + NS) * NW, stage);
        auto half = [&](auto which) {
            constexpr int S = decltype(which)::value;
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int i = 0; i < PB; i += 2) {
                    const int b = sb[m][i >> 1];
                    acc[m][i][0] = mx4_mfma_part<S, 0, 0>(fb[m][S][i], fa[S][0], acc[m][i][0], b, sa[0]);
                    acc[m][i + 1][0] =
                        mx4_mfma_part<S, 1, 0>(fb[m][S][i + 1], fa[S][0], acc[m][i + 1][0], b, sa[0]);
                    if constexpr (NMB == 4) {
                        acc[m][i][1] =
                            mx4_mfma_part<S, 0, 1>(fb[m][S][i], fa[S][1], acc[m][i][1], b, sa[0]);
                        acc[m][i + 1][1] = mx4_mfma_part<S, 1, 1>(fb[m][S][i + 1], fa[S][1],
                                                                  acc[m][i + 1][1], b, sa[0]);
                        acc[m][i][2] =
                            mx4_mfma_part<S, 0, 0>(fb[m][S][i], fa[S][2], acc[m][i][2], b, sa[1]);
                        acc[m][i + 1][2] = mx4_mfma_part<S, 1, 0>(fb[m][S][i + 1], fa[S][2],
                                                                  acc[m][i + 1][2], b, sa[1]);
                        acc[m][i][3] =
                            mx4_mfma_part<S, 0, 1>(fb[m][S][i], fa[S][3], acc[m][i][3], b, sa[1]);
                        acc[m][i + 1][3] = mx4_mfma_part<S, 1, 1>(fb[m][S][i + 1], fa[S][3],
                                                                  acc[m][i + 1][3], b, sa[1]);
                    }
                }
        };
        half(std::integral_constant<int, 0>{});
        half(std::integral_constant<int, 1>{});
        stage = stage + 1 == NS ? 0 : stage + 1;
    }

    // Every wave's sums to its own LDS, then wave j adds row part j (and its columns'
    // parts) in wave order.
    floatx4_t* red = reinterpret_cast<floatx4_t*>(mine);
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int i = 0; i < PB; ++i)
#pragma unroll
            for (int j = 0; j < NMB; ++j) red[((m * PB + i) * NMB + j) * 64 + lane] = acc[m][i][j];
    __syncthreads();
    auto total = [&](int m, int i, int j) {
        const char* at = smem + (((m * PB + i) * NMB + j) * 64 + lane) * 16;
        floatx4_t s = *reinterpret_cast<const floatx4_t*>(at);
#pragma unroll
        for (int w = 1; w < NW; ++w)
            s += *reinterpret_cast<const floatx4_t*>(at + w * kWaveLds);
        return s;
    };
    auto output = [&](int i, int j) {             // part (i, j): row fr, columns 4 fq .. + 3
        floatx4_t s = total(0, i, j);
        if constexpr (GATED) {
            const floatx4_t u = total(1, i, j);
#pragma unroll
            for (int d = 0; d < 4; ++d) s[d] = silu_mul(s[d], u[d]);
        }
        return s;
    };
    if constexpr (QOUT) {
        for (int j = wave; j < NMB; j += NW) {
            const int r = j * 16 + fr;
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const floatx4_t s = output(i, j);
                w[2 * i] = mx4_pack2<Elt>(s[0], s[1]);
                w[2 * i + 1] = mx4_pack2<Elt>(s[2], s[3]);
            }
            uint32_t top = mx4_top(w[0], w[1], w[2], w[3]);
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            uint32_t q;
            const int ex = mx4_encode<Elt>(top, w[0], w[1], w[2], w[3], q);
            if (r >= rows) continue;
            const int block = n0 / 32, nb = (p.N + 31) / 32;
            uint16_t* to = reinterpret_cast<uint16_t*>(p.QO + (m0 + r) * p.ldqo + block * 16);
            to[fq] = (uint16_t)q;
            to[4 + fq] = (uint16_t)(q >> 16);
            uint8_t* tile = p.SO + (m0 / 64 * p.nkto + block / 8) * kMx4Tile;
            if (fq == 0) tile[mx4_scale_offset(r, block & 7)] = (uint8_t)ex;
            // the last block's workgroup clears those past it, which hold nothing
            if (fq == 1 && block == nb - 1)
                for (int x = block + 1; x & 7; ++x) tile[mx4_scale_offset(r, x & 7)] = 0;
        }
    } else {
        for (int u = wave; u < PB * NMB; u += NW) {
            const int i = u / NMB, j = u - i * NMB;
            const floatx4_t s = output(i, j);
            const int m = j * 16 + fr;
            if (m >= rows) continue;
            const int c0 = n0 + i * 16 + fq * 4;
            uint16_t* c = p.C + (m0 + m) * p.ldc + c0;
            if (c0 + 3 < p.N) {
                *reinterpret_cast<uint2_t*>(c) =
                    uint2_t{mx4_pack2<Elt>(s[0], s[1]), mx4_pack2<Elt>(s[2], s[3])};
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const scalar v = (scalar)s[d];
                    if (c0 + d < p.N) c[d] = __builtin_bit_cast(uint16_t, v);
                }
            }
        }
    }
}

template <typename Elt, bool GROUPED, bool GATED, bool QOUT, int NW>
__global__ __launch_bounds__(NW * 64) void mx4_skinny_kernel(Mx4Gemm p) {
    __shared__ int4_t smem[NW * skinny_wave_lds(GROUPED) / 16];
    const int l = xcd_remap(blockIdx.x, gridDim.x, p.nxcd);
    const int g = l / p.gn, nt = l - g * p.gn;
    const int n0 = nt * (GATED ? 32 : 64);
    int e = 0, rows;
    int64_t m0;
    if constexpr (GROUPED) {
        if (!mx4_group(p, g, e, m0, rows)) return;
    } else {
        m0 = (int64_t)g * 64;
        rows = (int)min((int64_t)64, p.M - m0);
    }
    char* const lds = reinterpret_cast<char*>(smem);
    if (rows <= 16)
        mx4_skinny_body<Elt, GROUPED, GATED, QOUT, NW, 1>(p, lds, e, m0, n0, rows);
    else
        mx4_skinny_body<Elt, GROUPED, GATED, QOUT, NW, 4>(p, lds, e, m0, n0, rows);
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
__device__ __forceinline__ void mx4_store(uint16_t* C, int64_t ldc, const floatx4_t (&acc)[FN][FM],
                                          uint32_t mb, int left, uint32_t nb, int N, int lane) {
    const int fr = lane & 15, fq = lane >> 4;
    if (left <= 0) return;
    const int rows = min(left, FM * 16);
    const int columns = N - (int)nb;              // to the right of nb (none where nb is past N)
    const bool whole = columns >= FN * 16 && ldc < (1 << 24);
    C += (int64_t)mb * ldc + nb;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(C, (uint32_t)((rows - 1) * ldc + FN * 16) * 2);
    const int n = (fq & 1) * 16 + (fq >> 1) * 8;
    const uint32_t off = (uint32_t)(fr * (int)ldc + n) * 2;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
#pragma unroll
        for (int i = 0; i < FN; i += 2) {
            uint32_t a0 = mx4_pack2<Elt>(acc[i][j][0], acc[i][j][1]);
            uint32_t a1 = mx4_pack2<Elt>(acc[i][j][2], acc[i][j][3]);
            uint32_t b0 = mx4_pack2<Elt>(acc[i + 1][j][0], acc[i + 1][j][1]);
            uint32_t b1 = mx4_pack2<Elt>(acc[i + 1][j][2], acc[i + 1][j][3]);
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

// A wave's 32 columns of the gated product (block n0 / 32 + wave_n) rounded to the
// type, quantised and stored: what mx4_quantize makes of it, without its way
// through memory.  `rows`: rows of the tile that exist.
template <typename Elt, int FM>
__device__ __forceinline__ void mx4_store_quantized(const Mx4Gemm& p, const floatx4_t (&out)[2][FM],
                                                    uint32_t m0, uint32_t n0, int rows, int wave_m,
                                                    int wave_n, int lane) {
    static_assert(FM == 2 || FM == 4, "a wave's rows: half of or a whole scale tile");
    const int fr = lane & 15, fq = lane >> 4;
    const uint32_t block = n0 / 32 + wave_n;
    const bool in = block < (uint32_t)(p.N + 31) / 32;
    uint32_t q[4] = {0, 0, 0, 0};
    int e = 0;                                        // of row 16 fq + fr of the wave's
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
            w[c] = mx4_pack2<Elt>(out[c >> 1][j][2 * (c & 1)], out[c >> 1][j][2 * (c & 1) + 1]);
        uint32_t top = mx4_top(w[0], w[1], w[2], w[3]);
        top = max(top, (uint32_t)__shfl_xor((int)top, 16));
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        const int ej = mx4_encode<Elt>(top, w[0], w[1], w[2], w[3], q[j]);
        e = fq == j ? ej : e;
    }
    // transposed: lane (fr, fq) has the codes of row 16 fq + fr, quarter c's in q[c]:
    // low half of columns 4 c .., high half of columns 16 + 4 c ..
    swap16(q[0], q[1]);
    swap16(q[2], q[3]);
    swap32(q[0], q[2]);
    swap32(q[1], q[3]);
    const int r = wave_m * FM * 16 + fq * 16 + fr;
    if (fq >= FM || (r & ~63) >= rows) return;
    if (in && r < rows) {
        const uint4_t v = {(q[0] & 0xffffu) | (q[1] << 16), (q[2] & 0xffffu) | (q[3] << 16),
                           (q[0] >> 16) | (q[1] & 0xffff0000u), (q[2] >> 16) | (q[3] & 0xffff0000u)};
        *reinterpret_cast<uint4_t*>(p.QO + (int64_t)(m0 + r) * p.ldqo + block * 16) = v;
    }
    // a byte per row and block; the last columns' workgroup also clears the quarters
    // past them, whose blocks hold nothing
    const int g0 = (int)(n0 / 64) & 3;
    uint8_t* tile = p.SO + ((int64_t)((m0 + r) / 64) * p.nkto + n0 / 256) * kMx4Tile;
    tile[mx4_scale_offset(r & 63, 2 * g0 + wave_n)] = in && r < rows ? (uint8_t)e : 0;
    if (n0 + 64 >= (uint32_t)p.N)
        for (int g = g0 + 1; g < 4; ++g) tile[mx4_scale_offset(r & 63, 2 * g + wave_n)] = 0;
}

// The tiled product: output tiles of BM x BN, WM x WN waves of 16x16x128 MFMAs.
// A stage holds the codes of BM + BN rows x 128 bytes and their scale tiles,
// loaded straight into LDS; NS stages.  A row's chunks lie as mx4_swz says.
//
// A workgroup takes tiles in turn, its k-tiles one stream: once the fragments of a
// k-tile are in registers the loads of the one NS further on go into its stage,
// under the second half of its MFMAs.  Past a tile's last k-tile the loads are
// the next tile's, so neither its first loads nor the epilogue (in registers)
// leaves the memory idle.  Two workgroups share a CU: one's LDS reads and waits
// run under the other's MFMAs.
//
// GATED: the B rows of a wave are 32 of the first matrix and the same 32 of the
// second, so a lane holds both factors of its outputs; BN / 2 columns per tile.
// GROUPED: a tile's rows are one expert's of a plan; the tiles are counted from
// the plan's counts, so the grid holds no empty ones.
//
// Bound by the loads into LDS (53 bytes a clock and CU from rows on 128-byte lines,
// 650 of a 128 x 128 k-tile's 1050 clocks; 30 from others) and, on short k-loops,
// by the epilogue.  1024 x 8192 x 8192: 40 us (3.4 PFLOP/s); 4096 tokens of 64
// experts, 2048 -> 1024: gated 114-118 us, down 66 (1.8 and 1.6 PFLOP/s), of which the
// epilogues and the stores are 20 and 18 (left out, for timing alone: 94 and 49).
// With loader waves and one workgroup a CU those took 167 and 106.
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
    constexpr int BNO = GATED ? BN / 2 : BN;      // output columns
    constexpr int PRE = GROUPED ? 512 : 1;        // pairs of experts (kMaxExperts / 2)
    static_assert(A_UNITS % (64 * NW) == 0 && B_UNITS % (64 * NW) == 0, "whole 8-row slabs");
    static_assert(BM % 64 == 0 && BN % 64 == 0, "whole scale tiles");
    static_assert(!GATED || (WTN == 64 && BN == 128), "gated: 32 + 32 columns per wave");
    static_assert(WTM == 32 || WTM % 64 == 0, "a wave's rows: halves of or whole scale tiles");
    static_assert(WTN == 32 || WTN == 64, "a wave's columns: half of or a whole scale tile");
    static_assert(2 * (NS * STAGE * 16 + PRE * 4 + 64) <= 160 * 1024, "two workgroups fit the LDS");
    __shared__ int4_t smem[NS * STAGE];
    __shared__ int upto[PRE];                     // row tiles of the pairs of experts up to each
    __shared__ int wsum[NW];

    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wave_m = wave % WM, wave_n = wave / WM;
    const int nkt = p.nkt;

    int row_tiles = p.gm;
    if constexpr (GROUPED) {
        constexpr int EPT = PRE / (NW * 64);
        int c[EPT], sum = 0;
#pragma unroll
        for (int u = 0; u < EPT; ++u) {
            const int x = (t * EPT + u) * 2;
            sum += x < p.experts ? (int)((uint32_t)(p.counts[x] + BM - 1) / BM) : 0;
            sum += x + 1 < p.experts ? (int)((uint32_t)(p.counts[x + 1] + BM - 1) / BM) : 0;
            c[u] = sum;
        }
        int scan = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(scan, d);
            if (lane >= d) scan += o;
        }
        if (lane == 63) wsum[wave] = scan;
        __syncthreads();
        int before = scan - sum;
        row_tiles = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            before += w < wave ? wsum[w] : 0;
            row_tiles += wsum[w];
        }
#pragma unroll
        for (int u = 0; u < EPT; ++u) upto[t * EPT + u] = before + c[u];
        __syncthreads();
        row_tiles = __builtin_amdgcn_readfirstlane(row_tiles);
    }
    // This workgroup's tiles: every XCD has a contiguous range, its workgroups
    // take it in turn.
    const int total = row_tiles * p.gn;
    const int xcd = blockIdx.x % p.nxcd;
    const int turn = ((int)gridDim.x - xcd + p.nxcd - 1) / p.nxcd;
    const int last = (xcd + 1) * (total / p.nxcd) + min(xcd + 1, total % p.nxcd);
    int tile = xcd * (total / p.nxcd) + min(xcd, total % p.nxcd) + blockIdx.x / p.nxcd;
    if (tile >= last) return;
    // grouped: row and column tile, and how far a turn moves them
    int tm = tile / p.gn, tn = tile - tm * p.gn;
    const int turn_m = turn / p.gn, turn_n = turn - turn_m * p.gn;

    struct Place {
        uint32_t m0, n0;
        int rows;                                 // of the tile that exist
        int e;
    };
    auto locate = [&]() {
        Place x;
        x.e = 0;
        if constexpr (GROUPED) {
            x.n0 = (uint32_t)tn * BNO;
            int before = 0;                       // the pairs whose tiles all lie before tm
            for (int c = 0; 2 * c < p.experts; c += 64) {
                const bool in = 2 * (c + lane) < p.experts && upto[c + lane] <= tm;
                before += __popcll(__ballot(in));
            }
            before = __builtin_amdgcn_readfirstlane(before);
            int t0 = before == 0 ? 0 : __builtin_amdgcn_readfirstlane(upto[before - 1]);
            x.e = 2 * before;
            // scalar loads: a vector load's wait would be for every load in flight
            const int odd = x.e + 1 < p.experts ? 1 : 0;
            const int c0 = uniform_load(p.counts + x.e), c1 = uniform_load(p.counts + x.e + odd);
            const int o0 = uniform_load(p.offsets + x.e), o1 = uniform_load(p.offsets + x.e + odd);
            const int first = (int)((uint32_t)(c0 + BM - 1) / BM);
            const bool second = tm - t0 >= first;
            t0 += second ? first : 0;
            x.e += second ? 1 : 0;
            x.m0 = (uint32_t)(second ? o1 : o0) + (uint32_t)(tm - t0) * BM;
            x.rows = min((second ? c1 : c0) - (tm - t0) * BM, BM);
        } else {
            GemmParams gp;
            gp.gm = p.gm;
            gp.gn = p.gn;
            int64_t m0, n0;
            grouped_origin(gp, tile, BM, BNO, m0, n0);
            x.m0 = (uint32_t)m0;
            x.n0 = (uint32_t)n0;
            x.rows = min(p.M - (int)x.m0, BM);
        }
        return x;
    };
    auto next_tile = [&]() {
        tile += turn;
        tm += turn_m;
        tn += turn_n;
        if (tn >= p.gn) {
            tn -= p.gn;
            ++tm;
        }
    };

    // ---- the stream of k-tiles: the loads' position ------------------------------------
    const uint32_t srow = (uint32_t)nkt * kMx4Tile;   // scale bytes of 64 rows
    uint32_t voff_a[A_DMA], voff_b[B_DMA];
#pragma unroll
    for (int j = 0; j < A_DMA; ++j) {
        const int row = (wave * A_DMA + j) * 8 + (lane >> 3);
        const int pos = (lane & 7) ^ mx4_swz(row);
        voff_a[j] = (uint32_t)(row * p.lda) + pos * 16;
    }
#pragma unroll
    for (int j = 0; j < B_DMA; ++j) {
        const int row = (wave * B_DMA + j) * 8 + (lane >> 3);
        const int pos = (lane & 7) ^ mx4_swz(row);
        // gated: LDS rows 64 w + 32 h + i are row 32 w + i of matrix h
        const int src = GATED ? (row >> 6) * 32 + (row & 31) : row;
        voff_b[j] = (uint32_t)(src * (GATED && (row & 32) ? p.ldb2 : p.ldb)) +
                    pos * 16;
    }
    Place at = locate(), next_at = at;        // the tile that is multiplied, that is loaded
    int load_kt = 0;
    bool loads = nkt > 0;                         // loads are left
    __amdgpu_buffer_rsrc_t ra, rb, rb2, rsa, rsb, rsb2;
    auto describe = [&](const Place& x) {
        const int rows_b = min(BNO, p.N - (int)x.n0);
        const uint32_t sa = (uint32_t)((x.rows + 63) / 64) * srow;
        const uint32_t sb = (uint32_t)((rows_b + 63) / 64) * srow;
        const uint32_t last_b = (uint32_t)(rows_b - 1);
        ra = make_rsrc(p.A + (uint64_t)x.m0 * p.lda, (uint32_t)(x.rows - 1) * p.lda + p.rowbytes);
        rb = make_rsrc(p.B + x.e * p.eqb + (uint64_t)x.n0 * p.ldb, last_b * p.ldb + p.rowbytes);
        rsa = make_rsrc(p.SA + (uint64_t)(x.m0 / 64) * srow, sa);
        const uint64_t s0 = (uint64_t)(x.n0 / 64) * srow;
        rsb = make_rsrc(p.SB + x.e * p.esb + s0, sb);
        if constexpr (GATED) {
            rb2 = make_rsrc(p.B2 + x.e * p.eqb2 + (uint64_t)x.n0 * p.ldb2, last_b * p.ldb2 + p.rowbytes);
            rsb2 = make_rsrc(p.SB2 + x.e * p.esb2 + s0, sb);
        }
    };
    auto load_codes = [&](int stage) {
        int4_t* base = smem + stage * STAGE;
        // in the lane offset, which the descriptor's range check covers: the
        // last row's bytes past its blocks are not read
        const uint32_t koff = (uint32_t)load_kt * 128;
#pragma unroll
        for (int j = 0; j < A_DMA; ++j)
            dma16(ra, base + (wave * A_DMA + j) * 64, voff_a[j] + koff, 0);
#pragma unroll
        for (int j = 0; j < B_DMA; ++j) {
            const bool second = GATED && (((wave * B_DMA + j) * 8) & 32) != 0;
            dma16(second ? rb2 : rb, base + A_UNITS + (wave * B_DMA + j) * 64, voff_b[j] + koff, 0);
        }
    };
    auto load_scales = [&](int stage) {
#pragma unroll
        for (int j = 0; j < S_DMA; ++j) {
            const int st = (wave * S_DMA + j) % ST;
            int4_t* dst = smem + stage * STAGE + S_BASE + st * 32;
            if (lane < 32) {
                if (st < BM / 64)
                    dma16(rsa, dst, st * srow + lane * 16, load_kt * kMx4Tile);
                else if (GATED && st > BM / 64)
                    dma16(rsb2, dst, lane * 16, load_kt * kMx4Tile);
                else
                    dma16(rsb, dst, (st - BM / 64) * srow + lane * 16, load_kt * kMx4Tile);
            }
        }
    };
    auto advance = [&]() {
        if (++load_kt < nkt) return;
        load_kt = 0;
        if (!loads) return;
        next_tile();
        loads = tile < last;
        if (loads) {
            next_at = locate();
            describe(next_at);
        } else {
            // Nothing is left: the loads go on, so that the loop has no branch for
            // them, from empty descriptors (zeros, to stages that are not read).
            ra = make_rsrc(p.A, 0);
            rb = make_rsrc(p.B, 0);
            rsa = make_rsrc(p.SA, 0);
            rsb = make_rsrc(p.SB, 0);
            if constexpr (GATED) {
                rb2 = make_rsrc(p.B, 0);
                rsb2 = make_rsrc(p.SB, 0);
            }
        }
    };

    floatx4_t acc[FN][FM];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};
    };

    const int frow = lane & 15, fq = lane >> 4;
    const int fsw = mx4_swz(frow);
    const int a_row0 = wave_m * WTM + frow;
    const int b_row0 = A_UNITS / 8 + wave_n * WTN + frow;
    constexpr int SAW = FM / 2, SBW = FN / 2;     // scale dwords per lane (two parts each)
    struct Frags {
        int4_t a[2][FM], b[2][FN];
        int sa[SAW], sb[SBW];
    };
    auto read_half = [&](int stage, int s, Frags& f) {
        const int4_t* base = smem + stage * STAGE;
        const int chunk = (2 * fq + s) ^ fsw;
#pragma unroll
        for (int j = 0; j < FM; ++j) f.a[s][j] = base[(a_row0 + j * 16) * 8 + chunk];
#pragma unroll
        for (int i = 0; i < FN; ++i) f.b[s][i] = base[(b_row0 + i * 16) * 8 + chunk];
    };
    auto read_scales = [&](int stage, Frags& f) {
        const int4_t* base = smem + stage * STAGE;
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
    // The MFMAs are values to the compiler: an empty asm that reads them keeps it
    // from moving them past the waits and barriers that follow.
    auto pin = [&]() {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) asm volatile("" : "+v"(acc[i][j]));
    };
    auto barrier = [&]() {
        // not __syncthreads: its release would wait for every load in flight
        wait_lds();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    };
    auto store = [&]() {
        const uint32_t mb = at.m0 + wave_m * WTM;
        const int left = at.rows - wave_m * WTM;
        if constexpr (GATED) {
            floatx4_t out[FN / 2][FM];
#pragma unroll
            for (int i = 0; i < FN / 2; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
#pragma unroll
                    for (int d = 0; d < 4; ++d)
                        out[i][j][d] = silu_mul(acc[i][j][d], acc[i + FN / 2][j][d]);
            if constexpr (QOUT)
                mx4_store_quantized<Elt, FM>(p, out, at.m0, at.n0, at.rows, wave_m, wave_n, lane);
            else
                mx4_store<Elt, FN / 2, FM>(p.C, p.ldc, out, mb, left, at.n0 + wave_n * (WTN / 2), p.N,
                                           lane);
        } else {
            mx4_store<Elt, FN, FM>(p.C, p.ldc, acc, mb, left, at.n0 + wave_n * WTN, p.N, lane);
        }
    };

    clear();
    if (nkt == 0) {                               // every sum is empty
        for (; tile < last; next_tile()) {
            at = locate();
            store();
        }
        return;
    }
    describe(at);
#pragma unroll
    for (int j = 0; j < NS; ++j) {
        load_codes(j);
        load_scales(j);
        advance();
    }
    wait_global_loads<(NS - 1) * L>();            // k-tile 0 has landed
    barrier();
    // One k-tile a turn: `kt` of tile `at`, landed in stage s.
    int kt = 0, s = 0;
    for (;;) {
        // The loads stand in this tile or the next (the host sees to nkt > NS where
        // a workgroup has more than one): is there a next?
        const bool more = loads || next_at.m0 != at.m0 || next_at.n0 != at.n0;
        Frags f;
        read_half(s, 0, f);
        read_scales(s, f);
        read_half(s, 1, f);
        mfma_half(std::integral_constant<int, 0>{}, f);
        pin();
        barrier();                                // every wave has read stage s
        load_codes(s);
        mfma_half(std::integral_constant<int, 1>{}, f);
        // a load between every two MFMAs (masks: 0x020 global read, 0x008 MFMA)
#pragma unroll
        for (int m = 0; m < A_DMA + B_DMA; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, FM * FN / (A_DMA + B_DMA), 0);
        }
        pin();
        load_scales(s);
        advance();
        s = (s + 1 == NS) ? 0 : s + 1;
        if (++kt == nkt) {
            store();
            if (!more) break;
            kt = 0;
            at = next_at;
            clear();
        }
        // the next k-tile has landed: at most the NS - 1 after it are on their way
        // (after a tile's stores, which are younger and counted too, the wait is also
        // for loads of those)
        wait_global_loads<(NS - 1) * L>();
        barrier();
    }
    wait_global_loads<0>();
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

// y of 16 rows of B per workgroup, whose NW waves split the k-tiles.  Bound by the
// stream of B, which comes as in mx4_skinny_body: straight into LDS of each wave,
// eight lanes to a row's 128 bytes, NS k-tiles in flight.  The activations are in
// LDS, XK of them at a time, zeros past K.  Lane l takes row l % 16, blocks
// 2 (l / 16) and + 1 of a k-tile: the codes are converted two at a time to
// the activations' type (exact) and multiplied by pairs into an fp32 sum per
// block, which the block's scale then multiplies once.  The four quarters' sums
// are added by lane exchanges, the waves' in wave order through LDS.  12288 x 4096:
// 8.0 us with NS = 2 and XK = 4096, which lets three workgroups share a CU, and 9.0
// with NS = 3 and XK = 8192; 4096 x 12288: 9.8 and 9.4 (32 rows a workgroup: 9.2 with
// four waves, 11.0 with eight; the conversions left out, the time is the same).
template <typename Elt, int NW, int NS, int XK>
__global__ __launch_bounds__(NW * 64) void mx4_gemv_kernel(Mx4Gemv p) {
    typedef typename Elt::scalar scalar;
    typedef typename Elt::vec2 vec2;
    constexpr int BN = 16;
    constexpr int CODES = BN * 128, STAGE = CODES + kMx4Tile;
    constexpr int L = CODES / 1024 + 1;            // loads of a k-tile
    __shared__ int4_t stages[NW * NS * STAGE / 16];
    __shared__ uint4_t xs[XK / 8];
    __shared__ float red[NW * BN];
    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int n0 = blockIdx.x * BN;
    const int fr = lane & 15, fq = lane >> 4;
    const int fsw = mx4_swz(fr);
    const int rows_b = min(BN, p.N - n0);
    const uint32_t srow = (uint32_t)p.nkt * kMx4Tile;
    const __amdgpu_buffer_rsrc_t rb =
        make_rsrc(p.B + (int64_t)n0 * p.ldb, (uint32_t)((rows_b - 1) * p.ldb + p.rowbytes));
    const __amdgpu_buffer_rsrc_t rsb = make_rsrc(p.SB + (int64_t)(n0 / 64) * srow, srow);
    uint32_t voff[CODES / 1024];
    const int pos = (lane & 7) ^ mx4_swz(lane >> 3);    // chunk of the k-tile at this place
#pragma unroll
    for (int j = 0; j < CODES / 1024; ++j)
        voff[j] = (uint32_t)((j * 8 + (lane >> 3)) * p.ldb) + pos * 16;
    int4_t* const mine = stages + wave * (NS * STAGE / 16);
    auto load = [&](int kt, int stage) {
        int4_t* at = mine + stage * (STAGE / 16);
#pragma unroll
        for (int j = 0; j < CODES / 1024; ++j) dma16(rb, at + j * 64, voff[j] + (uint32_t)kt * 128, 0);
        if (lane < 32) dma16(rsb, at + CODES / 16, lane * 16, kt * kMx4Tile);
    };

    float sum = 0.0f;
    for (int k0 = 0; k0 < p.nkt; k0 += XK / 256) {
        const int n1 = min(p.nkt - k0, XK / 256);   // k-tiles of this turn
        const int n = (n1 - wave + NW - 1) / NW;        // this wave's
        for (int j = 0; j < min(n, NS); ++j) load(k0 + wave + j * NW, j);
        if (k0 > 0) __syncthreads();                    // xs has been read
        for (int i = t; i < n1 * 32; i += NW * 64)
            xs[i] = mx4_load8(p.x + (int64_t)k0 * 256 + i * 8, p.K - k0 * 256 - i * 8);
        wait_lds();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
        int stage = 0;
        for (int j = 0; j < n; ++j) {
            const int younger = min(n - 1 - j, NS - 1);
            if (NS > 2 && younger == 2)
                wait_global_loads<2 * L>();
            else if (younger == 1)
                wait_global_loads<L>();
            else
                wait_global_loads<0>();
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("" ::: "memory");
            const int4_t* at = mine + stage * (STAGE / 16);
            int4_t w[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) w[s] = at[fr * 8 + ((2 * fq + s) ^ fsw)];
            const uint32_t sc =
                reinterpret_cast<const uint16_t*>(at + CODES / 16)[lane * 4 + ((n0 >> 4) & 3)];
            wait_lds();
            __builtin_amdgcn_sched_barrier(0);
            if (j + NS < n) load(k0 + wave + (j + NS) * NW, stage);
            const uint4_t* xk = xs + (wave + j * NW) * 32 + fq * 8;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                float part = 0.0f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4_t xv = xk[s * 4 + c];
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const uint32_t xw = xv[d];
                        part = Elt::dot2(Elt::codes((uint32_t)w[s][c], d),
                                         __builtin_bit_cast(vec2, xw), part);
                    }
                }
                sum += part * mx4_scale_value((sc >> (8 * s)) & 255);
            }
            stage = stage + 1 == NS ? 0 : stage + 1;
        }
    }
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (lane < 16) red[wave * BN + lane] = sum;
    __syncthreads();
    if (t < rows_b) {
        float s = red[t];
#pragma unroll
        for (int w = 1; w < NW; ++w) s += red[w * BN + t];
        const scalar v = (scalar)s;
        p.y[n0 + t] = __builtin_bit_cast(uint16_t, v);
    }
}

}  // namespace sdt
