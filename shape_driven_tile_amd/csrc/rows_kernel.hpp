// Row-wise kernels for gfx950: 8-bit codes with a scale for each block of 128
// and back, and the root-mean-square norm with its gradients.  All are bound by
// memory: every element is read once, in 16-byte accesses, and kept in registers
// between the passes over a row.
//
// Codes (e4m3, largest 448): a block's scale is s = max |x| / 448 in fp32, at
// least 2^-126; a code is the fp32 quotient x / s rounded to nearest even.  A
// block that holds an infinity or a NaN has a NaN scale and zero codes.
#pragma once

#include "lanes.hpp"

namespace sdt {

constexpr float kFp8Max = 448.0f;

__device__ __forceinline__ float widen(F16, uint32_t bits16) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits16);
}
__device__ __forceinline__ float widen(BF16, uint32_t bits16) {
    return __builtin_bit_cast(float, bits16 << 16);
}

// Eight elements of a row of K >= 8 from column k on, zeros past K: a partial chunk is
// loaded as the row's last eight elements and moved down, and one past the row is that
// load cleared, so that no load depends on a branch (with one around each, the eight of
// a lane's rows wait for each other: 78 us for 8192 x 8192 fp16 codes by eight rows).
__device__ __forceinline__ uint4_t load_wide(const uint16_t* row, int k, int K) {
    return *reinterpret_cast<const uint4_any_t*>(row + min(k, K - 8));
}
__device__ __forceinline__ uint4_t move_down(uint4_t v, int k, int K) {
    const int s = k - (K - 8);                   // elements to move by (8 and more: none left)
    if (s <= 0) return v;
    if (s & 4) v = uint4_t{v[2], v[3], 0, 0};
    if (s & 2) v = uint4_t{v[1], v[2], v[3], 0};
    if (s & 1)
        v = uint4_t{(v[0] >> 16) | (v[1] << 16), (v[1] >> 16) | (v[2] << 16), (v[2] >> 16) | (v[3] << 16),
                    v[3] >> 16};
    return s >= 8 ? uint4_t{0, 0, 0, 0} : v;
}

// Eight packed elements as fp32.
template <typename Elt>
__device__ __forceinline__ void unpack8(uint4_t v, float (&x)[8]) {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t w = v[d];
        x[2 * d] = widen(Elt{}, w & 0xffffu);
        x[2 * d + 1] = widen(Elt{}, w >> 16);
    }
}
template <typename Elt>
__device__ __forceinline__ uint4_t pack8(const float (&x)[8]) {
    return uint4_t{pack2<Elt>(x[0], x[1]), pack2<Elt>(x[2], x[3]), pack2<Elt>(x[4], x[5]),
                   pack2<Elt>(x[6], x[7])};
}

// Eight elements to y, of which `valid` lie below K: none past K is written.
__device__ __forceinline__ void store8(uint16_t* y, uint4_t v, int valid) {
    if (valid >= 8) {
        *reinterpret_cast<uint4_any_t*>(y) = v;
        return;
    }
#pragma unroll
    for (int d = 0; d < 8; ++d) {
        const uint32_t w = v[d >> 1];
        if (d < valid) y[d] = (uint16_t)(w >> (16 * (d & 1)));
    }
}

// The same value from the lane n places further round in the row of 16.
template <int N>
__device__ __forceinline__ uint32_t turn16(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, false);
}
// The largest of 16 neighbouring lanes, in each of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max(v, turn16<8>(v));
    v = max(v, turn16<4>(v));
    v = max(v, turn16<2>(v));
    return max(v, turn16<1>(v));
}

// The largest magnitude of eight packed elements, as an fp32 bit pattern: found among
// the 16-bit patterns without their signs, whose order is the magnitudes' (infinities
// and NaN above all).
template <typename Elt>
__device__ __forceinline__ uint32_t top8(uint4_t v) {
    ushort2_t m = {0, 0};
#pragma unroll
    for (int d = 0; d < 4; ++d)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(ushort2_t, v[d] & 0x7fff7fffu));
    const float x = widen(Elt{}, max(m[0], m[1]));
    return __builtin_bit_cast(uint32_t, x);
}

// The largest magnitude of eight values as a bit pattern.
__device__ __forceinline__ uint32_t top8(const float (&x)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int d = 0; d < 8; ++d) m = max(m, __builtin_bit_cast(uint32_t, x[d]) & 0x7fffffffu);
    return m;
}

// A block's scale from the bit pattern of its largest magnitude.
__device__ __forceinline__ float fp8_scale(uint32_t top) {
    if (top >= 0x7f800000u) return __builtin_bit_cast(float, 0x7fc00000u);
    return fmaxf(__builtin_bit_cast(float, top) / kFp8Max, 0x1p-126f);
}

// Eight codes.  The quotients are correctly rounded by one correction of x * (1 /
// s) (Markstein's): its residual is exact, and what is left of the reciprocal's
// error is 2^-47 of the quotient.  Small scales are brought up first, so that the
// residual does not underflow; both factors are powers of two.  The residual is taken as
// -(t s - v): where v is a zero, v - t s would be +0 whatever its sign, and the code's
// with it.
__device__ __forceinline__ uint2_t fp8_codes(const float (&x)[8], float scale) {
    if (scale != scale) return uint2_t{0, 0};
    const float lift = scale < 0x1p-60f ? 0x1p64f : 1.0f;
    const float s = scale * lift, inv = 1.0f / s;
    float q[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) {
        const float v = x[d] * lift, t = v * inv;
        q[d] = __builtin_fmaf(-__builtin_fmaf(t, s, -v), inv, t);
    }
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    return uint2_t{(uint32_t)lo, (uint32_t)hi};
}

// Eight codes to q, 8-byte aligned, of which `valid` lie below K; none past it.
__device__ __forceinline__ void store_codes(uint8_t* q, uint2_t c, int valid) {
    if (valid >= 8) {
        *reinterpret_cast<uint2_t*>(q) = c;
        return;
    }
#pragma unroll
    for (int d = 0; d < 8; ++d) {
        const uint32_t w = c[d >> 2];
        if (d < valid) q[d] = (uint8_t)(w >> (8 * (d & 3)));
    }
}

struct Fp8Quant {
    const uint16_t* X;
    int64_t ldx;           // elements
    uint8_t* Q;
    int64_t ldq;           // bytes
    float* S;
    int64_t lds;           // floats: between blocks of k (rows' scales), between rows of blocks
    int64_t rows;
    int K, nct;            // column tiles of 2048 (rows' scales) or 128
};

// Scales for each row: RPT rows x 2048 columns a workgroup (one, or eight short ones), 16
// lanes a block.  All rows of a lane are loaded before the first is used.  Bound by memory:
// 8192 x 8192 fp16 36-41 us (5.0-5.5 TB/s; a copy 5.1), 4096 x 4096 13.3 us (3.8).
template <typename Elt, int RPT>
__global__ __launch_bounds__(256) void fp8_quantize_rows_kernel(Fp8Quant p) {
    const int t = threadIdx.x;
    const int64_t r0 = (int64_t)(blockIdx.x / p.nct) * RPT;
    const int k = (int)(blockIdx.x % p.nct) * 2048 + t * 8;
    const int valid = p.K - k;
    uint4_t v[RPT];
    if constexpr (RPT == 1) {                    // any K
        v[0] = uint4_t{0, 0, 0, 0};
        if (valid > 0) v[0] = load8(p.X + r0 * p.ldx + k, valid);
    } else {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            v[i] = load_wide(p.X + min(r0 + i, p.rows - 1) * p.ldx, k, p.K);
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        if (r0 + i >= p.rows) break;
        if constexpr (RPT > 1) v[i] = move_down(v[i], k, p.K);
        const float scale = fp8_scale(max16(top8<Elt>(v[i])));
        if (valid > 0) {
            float x[8];
            unpack8<Elt>(v[i], x);
            store_codes(p.Q + (r0 + i) * p.ldq + k, fp8_codes(x, scale), valid);
            if ((t & 15) == 0) p.S[(int64_t)(k >> 7) * p.lds + r0 + i] = scale;
        }
    }
}

// Scales for each block of 128 rows x 128 columns: one workgroup a block (8192 x 8192 fp16
// 36.6 us, 5.5 TB/s).
// WIDE: rows of 8 elements and more.
template <typename Elt, bool WIDE>
__global__ __launch_bounds__(256) void fp8_quantize_blocks_kernel(Fp8Quant p) {
    __shared__ uint32_t tops[4];
    const int t = threadIdx.x;
    const int64_t rb = blockIdx.x / p.nct;
    const int kb = (int)(blockIdx.x % p.nct);
    const int k = kb * 128 + (t & 15) * 8;
    const int valid = p.K - k;
    uint4_t v[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        // rows past the last repeat it
        const uint16_t* row = p.X + min(rb * 128 + i * 16 + (t >> 4), p.rows - 1) * p.ldx;
        if constexpr (WIDE) {
            v[i] = load_wide(row, k, p.K);
        } else {
            v[i] = uint4_t{0, 0, 0, 0};
            if (valid > 0) v[i] = load8(row + k, valid);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (WIDE) v[i] = move_down(v[i], k, p.K);
        top = max(top, top8<Elt>(v[i]));
    }
    top = max16(top);
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    if ((t & 63) == 0) tops[t >> 6] = top;
    __syncthreads();
    const float scale = fp8_scale(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
    if (t == 0) p.S[rb * p.lds + kb] = scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t row = rb * 128 + i * 16 + (t >> 4);
        if (row >= p.rows) break;
        float x[8];
        unpack8<Elt>(v[i], x);
        store_codes(p.Q + row * p.ldq + k, fp8_codes(x, scale), valid);
    }
}

struct Fp8Dequant {
    const uint8_t* Q;
    int64_t ldq;
    const float* S;
    int64_t lds;
    int block;             // 1: scales for each row; 128: for each 128 rows
    void* Y;
    int64_t ldy;           // elements
    int64_t rows;
    int K, nct;            // column tiles of 2048
};

// RPT rows x 2048 columns a workgroup, eight codes a lane and row (8192 x 8192 39.5 us, 5.1
// TB/s).
template <typename Out, int RPT>
__global__ __launch_bounds__(256) void fp8_dequantize_kernel(Fp8Dequant p) {
    const int64_t r0 = (int64_t)(blockIdx.x / p.nct) * RPT;
    const int k = (int)(blockIdx.x % p.nct) * 2048 + threadIdx.x * 8;
    const int valid = p.K - k;
    if (valid <= 0) return;
    uint2_t c[RPT];
    float s[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int64_t row = min(r0 + i, p.rows - 1);
        const uint8_t* q = p.Q + row * p.ldq;
        if constexpr (RPT > 1) {                 // K >= 8: as load_wide
            typedef uint2_t __attribute__((aligned(1))) uint2_any_t;
            c[i] = *reinterpret_cast<const uint2_any_t*>(q + min(k, p.K - 8));
        } else {
            c[i] = uint2_t{0, 0};
            if (valid >= 8) {
                c[i] = *reinterpret_cast<const uint2_t*>(q + k);
            } else {
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    if (d < valid) c[i][d >> 2] |= (uint32_t)q[k + d] << (8 * (d & 3));
            }
        }
        s[i] = p.block == 1 ? p.S[(int64_t)(k >> 7) * p.lds + row]
                            : p.S[(row >> 7) * p.lds + (k >> 7)];
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        if (r0 + i >= p.rows) break;
        if (RPT > 1 && valid < 8)
            c[i] = __builtin_bit_cast(uint2_t, __builtin_bit_cast(uint64_t, c[i]) >> (8 * (8 - valid)));
        float x[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int w = (int)c[i][h];
            const floatx2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
            const floatx2_t b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
            x[4 * h] = a[0] * s[i];
            x[4 * h + 1] = a[1] * s[i];
            x[4 * h + 2] = b[0] * s[i];
            x[4 * h + 3] = b[1] * s[i];
        }
        if constexpr (std::is_same_v<Out, float>) {
            float* y = static_cast<float*>(p.Y) + (r0 + i) * p.ldy + k;
#pragma unroll
            for (int d = 0; d < 8; ++d)
                if (d < valid) y[d] = x[d];
        } else {
            store8(static_cast<uint16_t*>(p.Y) + (r0 + i) * p.ldy + k, pack8<Out>(x), valid);
        }
    }
}

// ---- the norm ------------------------------------------------------------------------

struct Norm {
    const uint16_t *X, *R, *W;     // R (residual) and W (weight, K values) may be null
    int64_t ldx, ldr;
    uint16_t *T, *Y;               // x + r, the normed rows; either may be null
    int64_t ldt, ldy;
    uint8_t* Q;                    // the normed rows in 8 bits, or null
    int64_t ldq;
    float* S;
    int64_t lds;
    float* rstd;                   // or null
    int64_t rows;
    int K;
    float eps;
    // the gradient
    const uint16_t *DY, *DT;       // of y, of x + r (or null)
    int64_t lddy, lddt;
    const float* rstd_in;
    uint16_t* DX;
    int64_t lddx;
    float* dw_part;                // a row of K sums for each workgroup, or null
};

// The sum of a value over the T threads of a row's workgroup (T = 64: a wave of a
// workgroup of four), in the same order on every thread.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* sm) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    if constexpr (T > 64) {
        __syncthreads();           // the last use of sm is over
        if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = v;
        __syncthreads();
        v = sm[0];
#pragma unroll
        for (int w = 1; w < T / 64; ++w) v += sm[w];
    }
    return v;
}

// A row by T threads, CH chunks of eight elements each (K <= 8 T CH).  T = 64:
// four rows a workgroup.  The row stays in registers between its two passes, so memory
// is read once: with residual and total 8192 x 4096 bf16 48 us (5.6 TB/s), in 8 bits 48.3
// (4.9), 4097 x 8170 52 (4.5).
template <typename Elt, int T, int CH>
__global__ __launch_bounds__(T == 64 ? 256 : T) void rms_norm_kernel(Norm p) {
    __shared__ float sm[T / 64];
    const int t = T == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int64_t row = T == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
    if (row >= p.rows) return;     // whole waves, and with T = 64 no barrier follows
    float v[CH][8];
    uint4_t a[CH], b[CH], w[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = (i * T + t) * 8;
        a[i] = b[i] = w[i] = uint4_t{0, 0, 0, 0};
        if constexpr (T == 64) {                 // any K
            if (k < p.K) {
                a[i] = load8(p.X + row * p.ldx + k, p.K - k);
                if (p.R) b[i] = load8(p.R + row * p.ldr + k, p.K - k);
                if (p.W) w[i] = load8(p.W + k, p.K - k);
            }
        } else {
            a[i] = load_wide(p.X + row * p.ldx, k, p.K);
            if (p.R) b[i] = load_wide(p.R + row * p.ldr, k, p.K);
            if (p.W) w[i] = load_wide(p.W, k, p.K);
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = (i * T + t) * 8;
        if constexpr (T > 64) {
            a[i] = move_down(a[i], k, p.K);
            b[i] = move_down(b[i], k, p.K);
            w[i] = move_down(w[i], k, p.K);
        }
        unpack8<Elt>(a[i], v[i]);
        if (p.R) {
            // the sum as it is kept, rounded to the type, is what is normed
            float r[8];
            unpack8<Elt>(b[i], r);
#pragma unroll
            for (int d = 0; d < 8; ++d) v[i][d] += r[d];
            a[i] = pack8<Elt>(v[i]);
            unpack8<Elt>(a[i], v[i]);
        }
        if (p.T && k < p.K) store8(p.T + row * p.ldt + k, a[i], p.K - k);
#pragma unroll
        for (int d = 0; d < 8; ++d) sum = __builtin_fmaf(v[i][d], v[i][d], sum);
    }
    sum = row_sum<T>(sum, sm);
    const float rstd = 1.0f / sqrtf(sum / (float)p.K + p.eps);
    if (p.rstd && t == 0) p.rstd[row] = rstd;
    if (!p.Y && !p.Q) return;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = (i * T + t) * 8;
        if (p.W) {
            float g[8];
            unpack8<Elt>(w[i], g);
#pragma unroll
            for (int d = 0; d < 8; ++d) v[i][d] = v[i][d] * rstd * g[d];
        } else {
#pragma unroll
            for (int d = 0; d < 8; ++d) v[i][d] *= rstd;
        }
        if (p.Y && k < p.K) store8(p.Y + row * p.ldy + k, pack8<Elt>(v[i]), p.K - k);
        if (p.Q) {
            // 8 bits from the fp32 values, not from their rounding to 16
            if (k >= p.K) {
#pragma unroll
                for (int d = 0; d < 8; ++d) v[i][d] = 0.0f;
            } else if (p.K - k < 8) {
#pragma unroll
                for (int d = 0; d < 8; ++d) v[i][d] = d < p.K - k ? v[i][d] : 0.0f;
            }
            const float scale = fp8_scale(max16(top8(v[i])));
            if (k < p.K) {
                store_codes(p.Q + row * p.ldq + k, fp8_codes(v[i], scale), p.K - k);
                if ((t & 15) == 0) p.S[(int64_t)(k >> 7) * p.lds + row] = scale;
            }
        }
    }
}

// dx = rstd (dn - n mean(dn n)) + dt with n = t rstd, dn = dy w, and each
// workgroup's sums of dy n over its rows (row, row + grid, ...).  T = 64: the
// workgroup's four waves take rows in turn and add up in LDS.  Bound by memory where rows
// fit the registers, 8192 x 4096 bf16 with the columns' sums 51-57 us (4.7-5.3 TB/s), and by
// them and the second reading where not (1024 x 32768 142 us, 1.9; without dtotal 122,
// 1.65).
template <typename Elt, int T, int CH>
__global__ __launch_bounds__(T == 64 ? 256 : T) void rms_norm_backward_kernel(Norm p) {
    constexpr int WG = T == 64 ? 256 : T;
    constexpr int PER = WG / T;                  // rows at a time
    __shared__ float sm[T / 64];
    __shared__ float dws[PER > 1 ? PER * CH * 64 * 8 : 1];
    const int t = T == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int sub = T == 64 ? threadIdx.x >> 6 : 0;
    float dw[CH][8];
    uint4_t w[CH];                               // packed: half the registers
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = (i * T + t) * 8;
        const uint32_t one = pack2<Elt>(1.0f, 1.0f);
        w[i] = uint4_t{one, one, one, one};
        if (p.W && k < p.K) w[i] = load8(p.W + k, p.K - k);
#pragma unroll
        for (int d = 0; d < 8; ++d) dw[i][d] = 0.0f;
    }
    const int64_t step = (int64_t)gridDim.x * PER;
    auto load = [&](int64_t row, int i, uint4_t& a, uint4_t& b, uint4_t& c) {
        const int k = (i * T + t) * 8;
        a = b = c = uint4_t{0, 0, 0, 0};
        if constexpr (T == 64) {                 // any K
            if (k < p.K) {
                a = load8(p.X + row * p.ldx + k, p.K - k);
                b = load8(p.DY + row * p.lddy + k, p.K - k);
                if (p.DT) c = load8(p.DT + row * p.lddt + k, p.K - k);
            }
        } else {
            a = load_wide(p.X + row * p.ldx, k, p.K);
            b = load_wide(p.DY + row * p.lddy, k, p.K);
            if (p.DT) c = load_wide(p.DT + row * p.lddt, k, p.K);
        }
    };
    // A chunk's n, dn and dy.
    auto values = [&](int i, uint4_t a, uint4_t b, float rstd, float (&n)[8], float (&dn)[8], float (&dy)[8]) {
        const int k = (i * T + t) * 8;
        float g[8];
        asm volatile("" : "+v"(w[i]));           // unpacked here each time
        unpack8<Elt>(w[i], g);
        unpack8<Elt>(T > 64 ? move_down(a, k, p.K) : a, n);
        unpack8<Elt>(T > 64 ? move_down(b, k, p.K) : b, dy);
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            n[d] *= rstd;
            dn[d] = dy[d] * g[d];
        }
    };
    auto store = [&](int64_t row, int i, uint4_t c, float rstd, float inner, const float (&n)[8],
                     const float (&dn)[8]) {
        const int k = (i * T + t) * 8;
        if (k >= p.K) return;
        float dt[8];
        unpack8<Elt>(T > 64 ? move_down(c, k, p.K) : c, dt);
#pragma unroll
        for (int d = 0; d < 8; ++d)
            dt[d] = __builtin_fmaf(rstd, __builtin_fmaf(-n[d], inner, dn[d]), dt[d]);
        store8(p.DX + row * p.lddx + k, pack8<Elt>(dt), p.K - k);
    };
    int64_t row = (int64_t)blockIdx.x * PER + sub;
    if constexpr (CH > 2) {
        // Long rows, whose values do not fit the registers beside the sums: read again
        // from the caches for the second pass.
        for (; row < p.rows; row += step) {
            const float rstd = p.rstd_in[row];
            float inner = 0.0f;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                uint4_t a, b, c;
                float n[8], dn[8], dy[8];
                load(row, i, a, b, c);
                values(i, a, b, rstd, n, dn, dy);
#pragma unroll
                for (int d = 0; d < 8; ++d) inner = __builtin_fmaf(dn[d], n[d], inner);
            }
            inner = row_sum<T>(inner, sm) / (float)p.K;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                uint4_t a, b, c;
                float n[8], dn[8], dy[8];
                load(row, i, a, b, c);
                values(i, a, b, rstd, n, dn, dy);
#pragma unroll
                for (int d = 0; d < 8; ++d) dw[i][d] = __builtin_fmaf(dy[d], n[d], dw[i][d]);
                store(row, i, c, rstd, inner, n, dn);
            }
        }
    } else if (row < p.rows) {
        // The next row is on its way while this one is worked on, where a wave may have
        // the registers (8192 x 2048: 35.6 -> 32.1 us; 2048 x 16384 by 1024 threads, which
        // spill: 77 -> 91).
        constexpr bool AHEAD = T <= 256;
        uint4_t a[CH], b[CH], c[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) load(row, i, a[i], b[i], c[i]);
        float rstd = p.rstd_in[row];
        while (true) {
            float n[CH][8], dn[CH][8], inner = 0.0f;
            uint4_t dt[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) {
                float dy[8];
                values(i, a[i], b[i], rstd, n[i], dn[i], dy);
                dt[i] = c[i];
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    dw[i][d] = __builtin_fmaf(dy[d], n[i][d], dw[i][d]);
                    inner = __builtin_fmaf(dn[i][d], n[i][d], inner);
                }
            }
            const float now = rstd;
            const int64_t next = row + step;
            const bool more = next < p.rows;
            auto fetch = [&]() {
#pragma unroll
                for (int i = 0; i < CH; ++i) load(next, i, a[i], b[i], c[i]);
                rstd = p.rstd_in[next];
            };
            if (AHEAD && more) fetch();
            inner = row_sum<T>(inner, sm) / (float)p.K;
#pragma unroll
            for (int i = 0; i < CH; ++i) store(row, i, dt[i], now, inner, n[i], dn[i]);
            if (!more) break;
            if (!AHEAD) fetch();
            row = next;
        }
    }
    if (!p.dw_part) return;
    float* out = p.dw_part + (int64_t)blockIdx.x * p.K;
    if constexpr (PER > 1) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int d = 0; d < 8; ++d) dws[(sub * CH + i) * 512 + t * 8 + d] = dw[i][d];
        __syncthreads();
        for (int k = threadIdx.x; k < p.K; k += WG) {
            float s = dws[k];
#pragma unroll
            for (int w = 1; w < PER; ++w) s += dws[w * CH * 512 + k];
            out[k] = s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = (i * T + t) * 8;
#pragma unroll
            for (int d = 0; d < 8; ++d)
                if (k + d < p.K) out[k + d] = dw[i][d];
        }
    }
}

struct ColumnSum {
    const float* part;
    float* out;
    int parts, K;
};

// out[k] = sum over the parts, 64 columns a workgroup; 16 waves take every
// sixteenth part, and their sums are added in wave order.
__global__ __launch_bounds__(1024) void column_sum_kernel(ColumnSum p) {
    __shared__ float sm[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int k = blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (k < p.K) {
        int i = wave;
        for (; i + 48 < p.parts; i += 64) {      // four loads in flight
            const float a = p.part[(int64_t)i * p.K + k];
            const float b = p.part[(int64_t)(i + 16) * p.K + k];
            const float c = p.part[(int64_t)(i + 32) * p.K + k];
            const float d = p.part[(int64_t)(i + 48) * p.K + k];
            s += (a + b) + (c + d);
        }
        for (; i < p.parts; i += 16) s += p.part[(int64_t)i * p.K + k];
    }
    sm[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && k < p.K) {
#pragma unroll
        for (int w = 1; w < 16; ++w) s += sm[w][lane];
        p.out[k] = s;
    }
}

}  // namespace sdt
