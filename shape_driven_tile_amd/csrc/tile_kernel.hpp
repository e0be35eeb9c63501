// Products for gfx950 whose operands or epilogue the plain 16-bit kernels do not
// take: 8-bit codes with a scale for each block of 128, operands that are stored
// along the other dimension, two weight matrices with a gated epilogue.
//
// A k-tile is 128 bytes of a row: 64 16-bit values or 128 codes (one block of
// scales), in two halves of four 16-byte chunks; lane l of an MFMA operand holds
// row l % 16 and, in half h, chunk 4 h + l / 16.  For 16 bits a half is one
// v_mfma_f32_16x16x32; for 8 bits the halves together are one
// v_mfma_f32_16x16x128 (it adds over k whatever order both operands share).
//
// An operand whose rows run along k (K-major) lies in LDS as 8 chunks a row, chunk
// c of row r at c ^ swz_pp(r).  One whose rows run along its other dimension lies
// as it comes, 64 rows of k, and is turned by ds_read_b64_tr_b16: 16 lanes read
// four rows x 16 values and each gets the four k of one column; two reads make a
// half's eight.  Its 32-byte units are kept at unit ^ turned_swz(k), so that the
// eight rows that 32 lanes read at a time fall on distinct banks.
#pragma once

#include "rows_kernel.hpp"

namespace sdt {

typedef short short4_t __attribute__((ext_vector_type(4)));

struct TileGemm {
    const uint8_t *A[2], *B[2];    // two pairs: of products that are added, of a
                                   // batch, or (B) the gated product's matrices
    const float *SA, *SB;          // 8 bits: scales of A's rows and of B's blocks
    uint16_t* C[2];
    int64_t lda[2], ldb[2];        // bytes
    int64_t ldsa, ldsb;            // floats: between blocks of k, between blocks of rows
    int64_t ldc[2];                // elements
    int M, N, L;                   // output, and the contraction of one product
    int nkt;                       // k-tiles of one product
    int products, batch;           // products added up (1, 2); outputs (1, 2)
    int gm, gn, nxcd;
    int splits;                    // workgroups along the k-tiles of a tile
    float* ws;                     // splits > 1: their sums
    // gated: both factors, kept where g is not null
    void *G, *U;
    int64_t ldg, ldu;              // elements
    int wide;                      // they are fp32 (else of the output's type)
    int act;                       // 0: silu, 1: gelu (tanh)
};

// ---- activations ---------------------------------------------------------------------
// Both are g * sigmoid(t): t = g for silu; gelu's tanh form is g (1 + tanh z) / 2 = g
// sigmoid(2 z), z = sqrt(2 / pi) (g + 0.044715 g^3).

// sigmoid(t) and 1 - sigmoid(t), each to a few steps of its own size: e = exp(-t)
// as in silu_mul, s = 1 / (1 + e), 1 - s = e s; past +-88 the smaller one is 0.
__device__ __forceinline__ void sigmoid2(float t, float& s, float& r) {
    constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596303e-8f, kLn2 = 0.693147182f;
    const float x = -__builtin_amdgcn_fmed3f(t, -88.0f, 88.0f);
    const float y = x * kLog2e;
    const float low = __builtin_fmaf(x, kLog2e, -y) + x * kLog2eLow;
    const float z = __builtin_amdgcn_exp2f(y);
    const float e = __builtin_fmaf(z * kLn2, low, z);
    s = __builtin_amdgcn_rcpf(1.0f + e);
    r = t >= 88.0f ? 0.0f : e * s;
    s = t <= -88.0f ? 0.0f : s;
}
constexpr float kGelu1 = 1.59576912f;              // 2 sqrt(2 / pi)
constexpr float kGelu3 = 0.0713548163f;            // and times 0.044715

__device__ __forceinline__ float act_argument(float g, int act) {
    return act == 0 ? g : g * __builtin_fmaf(kGelu3 * g, g, kGelu1);
}
// a(g) u
__device__ __forceinline__ float act_mul(float g, float u, int act) {
    float s, r;
    sigmoid2(act_argument(g, act), s, r);
    return g * s * u;
}
// a(g) and its derivative
__device__ __forceinline__ void act_and_slope(float g, int act, float& a, float& da) {
    float s, r;
    sigmoid2(act_argument(g, act), s, r);
    a = g * s;
    const float c = __builtin_amdgcn_fmed3f(g, -100.0f, 100.0f);     // r is 0 beyond
    const float dt = act == 0 ? 1.0f : __builtin_fmaf(3.0f * kGelu3 * c, c, kGelu1);
    da = __builtin_fmaf(a * r, dt, s);
}

// ---- operands ------------------------------------------------------------------------

// Where a 32-byte pair of chunks of k-row `k` lies in a turned operand of UPR
// chunks a row (see the head of this file): the XOR of the chunk's place.
template <int UPR>
__device__ __forceinline__ int turned_swz(int k) {
    if constexpr (UPR >= 16) return 2 * ((k & 3) | ((k >> 1) & 4));
    return 2 * (((k >> 1) & 1) | ((k >> 2) & 2));
}

// One operand of a workgroup's tile: R of its rows (columns of a turned operand),
// by NW waves, `DMA` 1 KB loads a wave and k-tile.
template <bool TURNED, int R, int NW>
struct Operand {
    static constexpr int UPR = TURNED ? R / 8 : 8;       // chunks of an LDS row
    static constexpr int UNITS = R * 8;                  // chunks of a stage
    static constexpr int DMA = UNITS / (64 * NW);
    static_assert(UNITS % (64 * NW) == 0, "whole loads");

    // The lane's byte offset of load j from the tile's first row (or k-row) and
    // chunk; `src` maps an LDS row to the matrix's (the gated product's pairs).
    template <typename F>
    static __device__ __forceinline__ uint32_t offset(int wave, int lane, int j, int64_t ld, F src) {
        const int u = (wave * DMA + j) * 64 + lane;
        if constexpr (TURNED) {
            const int k = u / UPR, c = (u % UPR) ^ turned_swz<UPR>(k);
            return (uint32_t)(k * ld) + c * 16;
        }
        const int row = u >> 3;
        return (uint32_t)(src(row) * ld) + ((u & 7) ^ swz_pp(row)) * 16;
    }
    // The k-tiles of the operand in turn, by scalar arithmetic alone (a load of the
    // pointers in the loop would hold up the loads that follow it).  `rows` of the
    // operand's rows exist from its first one (or column) at `base` on.  Bytes past the
    // last row's end read as zero; the end is rounded up to the 4 bytes that its last
    // value lies in.
    struct Stream {
        const uint8_t* at;
        int64_t ld;
        int end;                                         // bytes of the last row
        int left;                                        // TURNED: k-rows left
        uint32_t bytes;
        __device__ __forceinline__ void start(const uint8_t* base, int64_t stride, int rows, int k, int L,
                                              int z) {
            ld = stride;
            if constexpr (TURNED) {
                at = base + (int64_t)k * 64 * ld;
                left = L - k * 64;
                end = (rows * 2 + 3) & ~3;
            } else {
                at = base + (int64_t)k * 128;
                bytes = (uint32_t)((rows - 1) * ld + ((L * z + 3) & ~3) - k * 128);
            }
        }
        // `some` false: a descriptor of nothing, which the loads go through without a
        // branch around them.
        __device__ __forceinline__ __amdgpu_buffer_rsrc_t next(bool some = true) {
            if constexpr (TURNED) {
                const uint32_t n = (uint32_t)((min(64, left) - 1) * (int)ld + end);
                const __amdgpu_buffer_rsrc_t r = make_rsrc(at, some ? n : 0u);
                at += 64 * ld;
                left -= 64;
                return r;
            }
            const __amdgpu_buffer_rsrc_t r = make_rsrc(at, some ? bytes : 0u);
            at += 128;
            bytes -= 128;
            return r;
        }
    };
    // Where the lane reads half 0 of the fragment of part P (16 rows), in bytes of a
    // stage; part P + j (P a multiple of the parts j runs over) and half h from it.
    static __device__ __forceinline__ int place(int P, int lane) {
        const int fr = lane & 15, fq = lane >> 4;
        if constexpr (TURNED) {
            const int k = 8 * fq + (fr >> 2), c = fr & 3;    // + 32 h + 4 t: the same swizzle
            return k * (UPR * 16) + ((P * 32) ^ (turned_swz<UPR>(k) * 16)) + c * 8;
        }
        return (P * 16 + fr) * 128 + (fq ^ swz_pp(fr)) * 16;
    }
    // Eight values, or 16 codes.  (Turned fragments by the compiler's own read: it holds
    // one back until every load into LDS issued before it has landed.)
    static __device__ __forceinline__ int4_t fragment(const int4_t* stage, int at, int j, int h) {
        const char* base = reinterpret_cast<const char*>(stage);
        if constexpr (TURNED) {
            typedef __attribute__((address_space(3))) short4_t* lds4;
            const char* from = base + (at ^ (j * 32)) + h * 32 * (UPR * 16);
            const int2_t lo = __builtin_bit_cast(int2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)from));
            const int2_t hi = __builtin_bit_cast(
                int2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(from + 4 * (UPR * 16))));
            return int4_t{lo[0], lo[1], hi[0], hi[1]};
        }
        return *reinterpret_cast<const int4_t*>(base + (at ^ (h * 64)) + j * 2048);
    }
    // Both halves of parts 0 .. F - 1.  Turned ones two parts at a time, each in one
    // block with its wait, so that loads for later k-tiles stay in flight.
    template <int F>
    static __device__ __forceinline__ void fragments(const int4_t* stage, int at, int4_t (&f)[F][2]) {
        if constexpr (TURNED) {
            static_assert(F % 2 == 0, "parts in pairs");
            const uint32_t base =
                (uint32_t) reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)stage);
#pragma unroll
            for (int j = 0; j < F; j += 2) {
                int2_t v[8];
                asm volatile(
                    "ds_read_b64_tr_b16 %0, %8\n\t"
                    "ds_read_b64_tr_b16 %1, %8 offset:%10\n\t"
                    "ds_read_b64_tr_b16 %2, %8 offset:%11\n\t"
                    "ds_read_b64_tr_b16 %3, %8 offset:%12\n\t"
                    "ds_read_b64_tr_b16 %4, %9\n\t"
                    "ds_read_b64_tr_b16 %5, %9 offset:%10\n\t"
                    "ds_read_b64_tr_b16 %6, %9 offset:%11\n\t"
                    "ds_read_b64_tr_b16 %7, %9 offset:%12\n\t"
                    "s_waitcnt lgkmcnt(0)"
                    : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]), "=&v"(v[4]), "=&v"(v[5]),
                      "=&v"(v[6]), "=&v"(v[7])
                    : "v"(base + (uint32_t)(at ^ (j * 32))), "v"(base + (uint32_t)(at ^ (j * 32 + 32))),
                      "i"(4 * UPR * 16), "i"(32 * UPR * 16), "i"(36 * UPR * 16)
                    : "memory");
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    f[j + q / 2][q % 2] =
                        int4_t{v[2 * q][0], v[2 * q][1], v[2 * q + 1][0], v[2 * q + 1][1]};
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < F; ++j) f[j][h] = fragment(stage, at, j, h);
        }
    }
};

// Bytes past a row's end (`valid` of a chunk's 16 lie below it) cleared.
__device__ __forceinline__ int4_t tail_mask(int valid) {
    int4_t m;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const int n = valid - 4 * d;
        m[d] = n >= 4 ? -1 : n <= 0 ? 0 : (1 << (8 * n)) - 1;
    }
    return m;
}

// The sums of a block of 128 codes (lane l: row l % 16 of A, four columns of B).
__device__ __forceinline__ floatx4_t fp8_block(const int4_t (&b)[2], const int4_t (&a)[2]) {
    const int8v_t b8 = {b[0][0], b[0][1], b[0][2], b[0][3], b[1][0], b[1][1], b[1][2], b[1][3]};
    const int8v_t a8 = {a[0][0], a[0][1], a[0][2], a[0][3], a[1][0], a[1][1], a[1][2], a[1][3]};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b8, a8, floatx4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0,
                                                           0, 0);
}

// acc += B . A^T over a k-tile (lane l: row l % 16 of A, four columns of B); 8 bits:
// times the blocks' scales.  The MFMA of a block starts from zero and its sums are
// scaled and added in fp32.  Inside the MFMA the products of eight neighbouring codes
// are aligned to the largest one's exponents and cut below 2^-13 of it before they are
// added to the others in fp32 (measured lane by lane; v_mfma_f32_16x16x32_fp8_fp8, at
// half the rate, does the same): on normal values 1.5e-5 of a sum, an eighth of fp16's
// rounding.
template <typename Elt, bool FP8>
__device__ __forceinline__ void tile_mma(floatx4_t& acc, const int4_t (&b)[2], const int4_t (&a)[2],
                                         float scale) {
    if constexpr (FP8) {
        const floatx4_t v = fp8_block(b, a);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(v[e], scale, acc[e]);
    } else {
        typedef typename Elt::frag8 frag8;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            acc = Elt::mfma16(__builtin_bit_cast(frag8, b[h]), __builtin_bit_cast(frag8, a[h]), acc);
    }
}

// Four bytes a lane from memory into LDS at base + 4 * lane.
__device__ __forceinline__ void dma4(const float* from, float* lds_wave_base) {
    typedef const __attribute__((address_space(1))) uint32_t* global_ptr;
    __builtin_amdgcn_global_load_lds((global_ptr) reinterpret_cast<uint64_t>(from),
                                     (__attribute__((address_space(3))) uint32_t*)lds_wave_base, 4, 0, 0);
}

// A wave's parts of both factors, in fp32, `left` rows from mb and columns nb .. of N.
template <int FN, int FM>
__device__ __forceinline__ void store_wide(float* C, int64_t ldc, const floatx4_t (&acc)[FN][FM], int64_t mb,
                                           int left, int nb, int N, int lane) {
    const int fr = lane & 15, fq = lane >> 4;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        if (j * 16 + fr >= left) continue;
        float* row = C + (mb + j * 16 + fr) * ldc;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const int n = nb + i * 16 + fq * 4;
            if (n + 3 < N) {
                *reinterpret_cast<floatx4_t*>(row + n) = acc[i][j];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < N) row[n + e] = acc[i][j][e];
            }
        }
    }
}

// What a wave does with its sums: FN x FM parts, rows from mb (`left` of them),
// columns from nb.  GATED: the parts' first half is the gate's, the second the other
// factor's.
template <typename Elt, bool GATED, int FN, int FM>
__device__ __forceinline__ void tile_store(const TileGemm& p, int batch, const floatx4_t (&acc)[FN][FM],
                                           uint32_t mb, int left, uint32_t nb, int lane) {
    if constexpr (GATED) {
        constexpr int H = FN / 2;
        // references to the two halves
        const floatx4_t(&g)[H][FM] = *reinterpret_cast<const floatx4_t(*)[H][FM]>(&acc[0]);
        const floatx4_t(&u)[H][FM] = *reinterpret_cast<const floatx4_t(*)[H][FM]>(&acc[H]);
        if (p.G) {
            if (p.wide) {
                store_wide<H, FM>(static_cast<float*>(p.G), p.ldg, g, mb, left, nb, p.N, lane);
                store_wide<H, FM>(static_cast<float*>(p.U), p.ldu, u, mb, left, nb, p.N, lane);
            } else {
                store_parts<Elt, H, FM>(static_cast<uint16_t*>(p.G), p.ldg, g, mb, left, nb, p.N, lane);
                store_parts<Elt, H, FM>(static_cast<uint16_t*>(p.U), p.ldu, u, mb, left, nb, p.N, lane);
            }
        }
        floatx4_t out[H][FM];
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) out[i][j][e] = act_mul(g[i][j][e], u[i][j][e], p.act);
        store_parts<Elt, H, FM>(p.C[0], p.ldc[0], out, mb, left, nb, p.N, lane);
    } else {
        store_parts<Elt, FN, FM>(p.C[batch], p.ldc[batch], acc, mb, left, nb, p.N, lane);
    }
}

// A wave's sums of a split, as they lie in the registers.
template <int FN, int FM>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t split_slot(const TileGemm& p, int64_t tile, int split,
                                                             int wave, int waves) {
    constexpr int FLOATS = FN * FM * 256;
    return make_rsrc(p.ws + ((tile * p.splits + split) * waves + wave) * FLOATS, FLOATS * 4);
}

// Waits until at most the youngest n (<= MOST) of the k-tiles on their way, of L loads
// each, have not landed.
template <int MOST, int L>
__device__ __forceinline__ void wait_tiles(int n) {
    if constexpr (MOST > 0) {
        if (n < MOST) return wait_tiles<MOST - 1, L>(n);
    }
    wait_global_loads<MOST * L>();
}

// ---- the tiled product -----------------------------------------------------------------
// Output tiles of BM x BN by WM x WN waves, NS stages; two workgroups a CU, one's
// reads and waits under the other's MFMAs.  The loads of the k-tile NS further on go
// into a stage once its fragments are in registers, between the MFMAs.  GATED: B's
// LDS rows alternate between the two matrices, so that a lane holds both factors of
// its outputs; BN / 2 columns a tile.  A k-tile of 128 x 128 costs a CU 0.92 us with two
// tiles at a time (0.46 a tile), 0.72 with one: bound by a workgroup's own chain of waits,
// which the other fills.  Deeper stages instead of the second workgroup do not (2048 x 3000 x 2048
// turned, 384 tiles: 53 us against 32).  2048^3: nn 28.9 us, tn 27.8, 8 bits 14.7; gated 500
// x 1400 x 1000 13.1.
template <typename Elt, bool FP8, int BM, int BN, int WM, int WN, int NS, bool TA, bool TB, bool GATED>
__global__ __launch_bounds__(WM * WN * 64, 2) void tile_gemm_kernel(TileGemm p) {
    constexpr int NW = WM * WN;
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int FM = WTM / 16, FN = WTN / 16;
    constexpr int BNO = GATED ? BN / 2 : BN;
    constexpr int Z = FP8 ? 1 : 2;
    constexpr int RW = BM / NW;                   // rows whose scales a wave loads
    typedef Operand<TA, BM, NW> OpA;
    typedef Operand<TB, BN, NW> OpB;
    constexpr int S_UNITS = FP8 ? NW * 16 : 0;    // 64 floats a wave: 32 of rows, 32 of columns
    constexpr int STAGE = OpA::UNITS + OpB::UNITS + S_UNITS;
    constexpr int L = OpA::DMA + OpB::DMA + (FP8 ? 1 : 0);
    static_assert(!FP8 || (!TA && !TB && !GATED && RW <= 32 && BN <= 128), "8 bits: K-major operands");
    static_assert(!GATED || (!TB && FN % 4 == 0), "a wave's parts of both matrices, in pairs");
    static_assert(GATED || FN % 2 == 0, "parts in pairs");
    static_assert(NS * STAGE * 16 <= 160 * 1024, "the stages fit the LDS");
    __shared__ int4_t smem[NS * STAGE];

    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wave_m = wave % WM, wave_n = wave / WM;

    // ---- workgroup -> tile, batch and range of k-tiles ------------------------------
    const int tiles = p.gm * p.gn;
    const int w = xcd_remap(blockIdx.x, gridDim.x, p.nxcd);
    const int outer = w / tiles, tile = w - outer * tiles;
    const int batch = outer / p.splits, split = outer - batch * p.splits;
    GemmParams gp;
    gp.gm = p.gm;
    gp.gn = p.gn;
    int64_t m0, n0;
    grouped_origin(gp, tile, BM, BNO, m0, n0);
    const int rows_a = (int)min((int64_t)BM, p.M - m0);
    const int rows_b = (int)min((int64_t)BNO, p.N - n0);
    const int all = p.products * p.nkt;
    const int first = (int)((int64_t)all * split / p.splits);
    const int end = (int)((int64_t)all * (split + 1) / p.splits);

    uint32_t voff_a[OpA::DMA], voff_b[OpB::DMA];
    auto offsets = [&](int pair) {
#pragma unroll
        for (int j = 0; j < OpA::DMA; ++j)
            voff_a[j] = OpA::offset(wave, lane, j, p.lda[pair], [](int r) { return r; });
#pragma unroll
        for (int j = 0; j < OpB::DMA; ++j) {
            if constexpr (GATED) {
                const bool second = ((wave * OpB::DMA + j) * 8) % WTN >= WTN / 2;
                voff_b[j] = OpB::offset(wave, lane, j, second ? p.ldb[1] : p.ldb[0], [](int r) {
                    return r / WTN * (WTN / 2) + r % (WTN / 2);
                });
            } else {
                voff_b[j] = OpB::offset(wave, lane, j, p.ldb[pair], [](int r) { return r; });
            }
        }
    };
    // The k-tile that the next load takes.  The pointers of both pairs stay at hand.
    typename OpA::Stream sa;
    typename OpB::Stream sb, sb2;
    const uint8_t* const a1 = p.A[1];
    const uint8_t* const b1 = p.B[1];
    const int64_t lda1 = p.lda[1], ldb1 = p.ldb[1];
    int load_k = first >= p.nkt ? first - p.nkt : first;
    auto start = [&](bool second) {
        const int64_t lda = second ? lda1 : p.lda[0], ldb = second ? ldb1 : p.ldb[0];
        sa.start((second ? a1 : p.A[0]) + (TA ? m0 * 2 : m0 * lda), lda, TA ? (int)(p.M - m0) : rows_a, load_k,
                 p.L, Z);
        const int columns = TB ? (int)(p.N - n0) : rows_b;
        sb.start((second ? b1 : p.B[0]) + (TB ? n0 * 2 : n0 * ldb), ldb, columns, load_k, p.L, Z);
        if constexpr (GATED) sb2.start(b1 + n0 * ldb1, ldb1, columns, load_k, p.L, Z);
        offsets(second ? 1 : 0);
    };
    start(batch == 1 || first >= p.nkt);
    // the scales this lane loads: a row's (lanes 0-31) or the columns' block's
    const float* scale_at = nullptr;
    int64_t scale_step = 0;
    if constexpr (FP8) {
        const int64_t row = min(m0 + wave * RW + min(lane & 31, RW - 1), (int64_t)p.M - 1);
        scale_at = lane < 32 ? p.SA + row : p.SB + (n0 >> 7) * p.ldsb;
        scale_step = lane < 32 ? p.ldsa : 1;
    }

    int coming = first;                           // the k-tile that the next load takes
    // The loads of a k-tile, one by one: 0 (8 bits) scales, then A's, then B's.
    struct Target {
        int4_t* base;
        __amdgpu_buffer_rsrc_t ra, rb, r2;
    };
    auto begin = [&](int stage) {
        const bool some = coming < end;
        Target x{smem + stage * STAGE, sa.next(some), sb.next(some)};
        if constexpr (GATED) x.r2 = sb2.next(some);
        return x;
    };
    auto issue = [&](const Target& x, int n) {
        constexpr int S = FP8 ? 1 : 0;
        if (FP8 && n == 0) {
            if constexpr (FP8)
                dma4(scale_at + min(load_k, p.nkt - 1) * scale_step,
                     reinterpret_cast<float*>(x.base + OpA::UNITS + OpB::UNITS + wave * 16));
        } else if (n < S + OpA::DMA) {
            const int j = n - S;
            dma16(x.ra, x.base + (wave * OpA::DMA + j) * 64, voff_a[j], 0);
        } else {
            const int j = n - S - OpA::DMA;
            const bool second = GATED && ((wave * OpB::DMA + j) * 8) % WTN >= WTN / 2;
            dma16(second ? x.r2 : x.rb, x.base + OpA::UNITS + (wave * OpB::DMA + j) * 64, voff_b[j], 0);
        }
    };
    auto done = [&]() {
        ++coming;
        ++load_k;
    };
    auto load = [&](int stage) {
        const Target x = begin(stage);
#pragma unroll
        for (int n = 0; n < L; ++n) issue(x, n);
        done();
    };
    // The loads have come to the end of a product that another is added to.
    auto second_product = [&]() {
        if (load_k == p.nkt && p.products == 2) {
            load_k = 0;
            start(true);
        }
    };

    floatx4_t acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    const int at_a = OpA::place(wave_m * FM, lane), at_b = OpB::place(wave_n * FN, lane);
    struct Frags {
        int4_t a[FM][2], b[FN][2];
        float sa[FM], sb;                         // scales
    };
    auto read_scales = [&](int stage, Frags& f) {
        const float* sc = reinterpret_cast<const float*>(smem + stage * STAGE + OpA::UNITS + OpB::UNITS);
        f.sb = sc[32];
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int r = (wave_m * FM + j) * 16 + (lane & 15);
            f.sa[j] = sc[(r / RW) * 64 + r % RW];
        }
    };
    auto read_a = [&](int stage, Frags& f) {
        OpA::template fragments<FM>(smem + stage * STAGE, at_a, f.a);
        if constexpr (FP8) read_scales(stage, f);
    };
    auto read_b = [&](int stage, Frags& f) {
        OpB::template fragments<FN>(smem + stage * STAGE + OpA::UNITS, at_b, f.b);
    };
    // The last k-tile of a product: what its K-major rows hold past their end is
    // not zero.
    auto clear_tail = [&](Frags& f) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int4_t m = tail_mask(p.L * Z - (p.nkt - 1) * 128 - (4 * h + (lane >> 4)) * 16);
            if constexpr (!TA) {
#pragma unroll
                for (int j = 0; j < FM; ++j) f.a[j][h] &= m;
            }
            if constexpr (!TB) {
#pragma unroll
                for (int i = 0; i < FN; ++i) f.b[i][h] &= m;
            }
        }
    };
    auto mma = [&](const Frags& f, int i0, int i1) {
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const float scale = FP8 ? f.sa[j] * f.sb : 0.0f;
#pragma unroll
            for (int i = i0; i < i1; ++i) tile_mma<Elt, FP8>(acc[i][j], f.b[i], f.a[j], scale);
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

    // All but the youngest N k-tiles on their way have landed, for every wave.
    auto landed = [&](auto n) {
        wait_global_loads<decltype(n)::value * L>();
        barrier();
    };
    typedef std::integral_constant<int, NS - 1> Others;
    typedef std::integral_constant<int, NS - 2> Later;
    const bool ragged = (!TA || !TB) && (p.L * Z) % 128 != 0;
    Frags f[2];
    int s = 0, kt = first;
    // One k-tile, not the last: its fragments are in registers (f[P]); the next k-tile's
    // are read while it is multiplied.  The loads into the stage that it has left go out
    // between the MFMAs: a CU takes in 64 bytes a clock, and a wave that issues them in
    // one go waits out the others' too (1024^2, a 64 x 64 tile's k-tile: 640 clocks).
    auto step = [&](auto which) {
        constexpr int P = decltype(which)::value;
        const int sn = (s + 1 == NS) ? 0 : s + 1;
        landed(Later{});                          // and every wave has read stage s
        Frags& next = f[P ^ 1];
        if constexpr (FP8) {
            // An MFMA's sums are scaled and added four MFMAs later: sooner the wave would
            // have to wait for them (2048^3 17.5 us, so 16.4).  Two fragments are read after
            // each MFMA until all are (before the first: 16.4 us, so 15.3).
            constexpr int ALL = FM * FN, GAP = ALL > L ? ALL / L : 1;
            static_assert(ALL >= FM + FN, "every fragment has its MFMA");
            const Target x = begin(s);
            const int4_t* const from = smem + sn * STAGE;
            auto read = [&](int part) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (part < FN)
                        next.b[part][h] = OpB::fragment(from + OpA::UNITS, at_b, part, h);
                    else if (part < FN + FM)
                        next.a[part - FN][h] = OpA::fragment(from, at_a, part - FN, h);
                }
            };
            floatx4_t v[4];
            float scale[4];
            auto add = [&](int n) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[n % FN][n / FN][e] = __builtin_fmaf(v[n % 4][e], scale[n % 4], acc[n % FN][n / FN][e]);
            };
            read_scales(sn, next);
#pragma unroll
            for (int n = 0; n < ALL; ++n) {
                if (n >= 4) add(n - 4);
                __builtin_amdgcn_sched_barrier(0);
                scale[n % 4] = f[P].sa[n / FN] * f[P].sb;
                v[n % 4] = fp8_block(f[P].b[n % FN], f[P].a[n / FN]);
                read(n);
                if (n % GAP == 0 && n / GAP < L) issue(x, n / GAP);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int l = ALL / GAP; l < L; ++l) issue(x, l);
#pragma unroll
            for (int n = ALL - 4; n < ALL; ++n) add(n);
            done();
        } else {
            if constexpr (!TA) read_a(sn, next);
            if constexpr (!TB) read_b(sn, next);
            __builtin_amdgcn_sched_barrier(0);
            load(s);
            mma(f[P], 0, FN / 2);
#pragma unroll
            for (int m = 0; m < L; ++m) {             // masks: 0x008 MFMA, 0x020 global read
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, FM * FN * 2 / ((TA || TB ? 2 : 1) * L), 0);
            }
            // turned fragments come with their wait: under the MFMAs issued before them
            if constexpr (TA) read_a(sn, next);
            mma(f[P], FN / 2, FN);
            if constexpr (TB) read_b(sn, next);
        }
        pin();
        s = sn;
        ++kt;
    };
    if (first < end) {
#pragma unroll
        for (int j = 0; j < NS; ++j) {
            load(j);
            second_product();
        }
        landed(Others{});
        read_a(0, f[0]);
        read_b(0, f[0]);
        while (kt < end) {
            // the next k-tile that is partial, the last, or whose load ends a product
            const int product = kt < p.nkt ? p.nkt : 2 * p.nkt;
            int special = (ragged ? min(product, end) : end) - 1;
            if (p.products == 2 && coming <= p.nkt) special = min(special, p.nkt - 1 - NS);
            while (kt + 2 <= special) {
                step(std::integral_constant<int, 0>{});
                step(std::integral_constant<int, 1>{});
            }
            // one k-tile by itself
            if (ragged && kt == product - 1) clear_tail(f[0]);
            mma(f[0], 0, FN);
            pin();
            if (kt + 1 == end) break;
            landed(Later{});
            load(s);
            second_product();
            s = (s + 1 == NS) ? 0 : s + 1;
            ++kt;
            read_a(s, f[0]);
            read_b(s, f[0]);
        }
        wait_global_loads<0>();                   // none is left when the workgroup ends
    }

    if (p.splits > 1) {
        store_partial<0>(acc, split_slot<FN, FM>(p, (int64_t)batch * tiles + tile, split, wave, NW), lane);
        return;
    }
    tile_store<Elt, GATED, FN, FM>(p, batch, acc, (uint32_t)m0 + wave_m * WTM, rows_a - wave_m * WTM,
                                   (uint32_t)n0 + wave_n * (WTN * BNO / BN), lane);
}

// Adds the splits of a tile in their order and stores it.
template <typename Elt, int BM, int BN, int WM, int WN, bool GATED>
__global__ __launch_bounds__(WM * WN * 64) void tile_reduce_kernel(TileGemm p) {
    constexpr int NW = WM * WN;
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int FM = WTM / 16, FN = WTN / 16;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wave_m = wave % WM, wave_n = wave / WM;
    const int tiles = p.gm * p.gn;
    const int batch = blockIdx.x / tiles, tile = blockIdx.x - batch * tiles;
    GemmParams gp;
    gp.gm = p.gm;
    gp.gn = p.gn;
    int64_t m0, n0;
    constexpr int BNO = GATED ? BN / 2 : BN;
    grouped_origin(gp, tile, BM, BNO, m0, n0);
    floatx4_t acc[FN][FM];
    load_partial<0, false>(acc, split_slot<FN, FM>(p, blockIdx.x, 0, wave, NW), lane);
    for (int s = 1; s < p.splits; ++s)
        load_partial<0, true>(acc, split_slot<FN, FM>(p, blockIdx.x, s, wave, NW), lane);
    const int rows = (int)min((int64_t)BM, p.M - m0);
    tile_store<Elt, GATED, FN, FM>(p, batch, acc, (uint32_t)m0 + wave_m * WTM, rows - wave_m * WTM,
                                   (uint32_t)n0 + wave_n * (WTN * BNO / BN), lane);
}

// ---- few rows ------------------------------------------------------------------------
// PB * 16 columns of C (gated: of each matrix) and up to NMB * 16 rows a workgroup, whose
// NW waves take every NW-th k-tile and stream B once.  Every wave has LDS of its
// own, so the loop has no barrier: rows come straight into it in whole 128-byte
// lines, NS k-tiles in flight, and are read from there as fragments.  The waves'
// sums are added in wave order.  Bound by B's stream: one row of 12288 x 4096, 8 bits
// 10.2 us (50 MB, 4.9 TB/s), gated of 16 bits 38.0 (201 MB, 5.3 TB/s).
template <typename Elt, bool FP8, bool GATED, int NW, int PB, int NMB, int NS>
__global__ __launch_bounds__(NW * 64) void rows_gemm_kernel(TileGemm p) {
    constexpr int MATS = GATED ? 2 : 1;
    constexpr int BN = PB * 16;
    constexpr int Z = FP8 ? 1 : 2;
    constexpr int A_UNITS = NMB * 128, B_UNITS = BN * 8;       // of one matrix
    constexpr int S_UNITS = FP8 ? 32 : 0;                      // 64 floats of rows, 64 of columns
    constexpr int STAGE = A_UNITS + MATS * B_UNITS + S_UNITS;
    constexpr int A_DMA = A_UNITS / 64, B_DMA = B_UNITS / 64;
    constexpr int L = A_DMA + MATS * B_DMA + (FP8 ? 2 : 0);
    constexpr int SUMS = MATS * PB * NMB * 64;                 // 16-byte units
    constexpr int MINE = NS * STAGE > SUMS ? NS * STAGE : SUMS;
    static_assert(!FP8 || !GATED, "one matrix of scales");
    static_assert(NW * MINE * 16 <= 160 * 1024, "LDS");
    __shared__ int4_t smem[NW * MINE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int fr = lane & 15, fq = lane >> 4;
    const int w = xcd_remap(blockIdx.x, gridDim.x, p.nxcd);
    const int64_t n0 = (int64_t)w * BN;
    const int rows_a = p.M;
    const int rows_b = (int)min((int64_t)BN, p.N - n0);

    const int chunk = ((lane & 7) ^ swz_pp(lane >> 3)) * 16;
    uint32_t voff_a[A_DMA], voff_b[MATS][B_DMA];
#pragma unroll
    for (int j = 0; j < A_DMA; ++j) voff_a[j] = (uint32_t)((j * 8 + (lane >> 3)) * p.lda[0]) + chunk;
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int j = 0; j < B_DMA; ++j)
            voff_b[m][j] = (uint32_t)((j * 8 + (lane >> 3)) * p.ldb[m]) + chunk;
    const float *sa_at = nullptr, *sb_at = nullptr;
    if constexpr (FP8) {
        sa_at = p.SA + min(lane, p.M - 1);
        sb_at = p.SB + (n0 >> 7) * p.ldsb;
    }
    int4_t* const mine = smem + wave * MINE;
    typedef Operand<false, NMB * 16, 1> OpA;
    typedef Operand<false, BN, 1> OpB;
    const uint8_t* const a0 = p.A[0];
    const uint8_t* const b0[2] = {p.B[0] + n0 * p.ldb[0], GATED ? p.B[1] + n0 * p.ldb[1] : nullptr};
    // bytes up to the last row's end, which is rounded up to 4
    const int row_end = (p.L * Z + 3) & ~3;
    const uint32_t a_end = (uint32_t)((rows_a - 1) * p.lda[0] + row_end);
    const uint32_t b_end[2] = {(uint32_t)((rows_b - 1) * p.ldb[0] + row_end),
                               (uint32_t)((rows_b - 1) * p.ldb[1] + row_end)};
    auto load = [&](int kt, int stage) {
        int4_t* at = mine + stage * STAGE;
        const __amdgpu_buffer_rsrc_t ra = make_rsrc(a0 + kt * 128, a_end - kt * 128);
#pragma unroll
        for (int j = 0; j < A_DMA; ++j) dma16(ra, at + j * 64, voff_a[j], 0);
        at += A_UNITS;
#pragma unroll
        for (int m = 0; m < MATS; ++m) {
            const __amdgpu_buffer_rsrc_t rb = make_rsrc(b0[m] + kt * 128, b_end[m] - kt * 128);
#pragma unroll
            for (int j = 0; j < B_DMA; ++j) dma16(rb, at + j * 64, voff_b[m][j], 0);
            at += B_UNITS;
        }
        if constexpr (FP8) {
            dma4(sa_at + kt * p.ldsa, reinterpret_cast<float*>(at));
            dma4(sb_at + kt, reinterpret_cast<float*>(at) + 64);
        }
    };

    floatx4_t acc[MATS][PB][NMB];
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int i = 0; i < PB; ++i)
#pragma unroll
            for (int j = 0; j < NMB; ++j) acc[m][i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    const int place = OpA::place(0, lane);        // the same in B's rows
    const int n = (p.nkt - wave + NW - 1) / NW;   // this wave's k-tiles (0 or less: none)
    for (int j = 0; j < min(n, NS); ++j) load(wave + j * NW, j);
    int stage = 0;
    for (int j = 0; j < n; ++j) {
        wait_tiles<NS - 1, L>(min(n - 1 - j, NS - 1));
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        const int4_t* at = mine + stage * STAGE;
        int4_t fa[NMB][2], fb[MATS][PB][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < NMB; ++j) fa[j][h] = OpA::fragment(at, place, j, h);
#pragma unroll
            for (int m = 0; m < MATS; ++m)
#pragma unroll
                for (int i = 0; i < PB; ++i)
                    fb[m][i][h] = OpB::fragment(at + A_UNITS + m * B_UNITS, place, i, h);
        }
        float scale[NMB] = {};
        if constexpr (FP8) {
            const float* sc = reinterpret_cast<const float*>(at + A_UNITS + MATS * B_UNITS);
#pragma unroll
            for (int j = 0; j < NMB; ++j) scale[j] = sc[j * 16 + fr] * sc[64];
        }
        wait_lds();
        __builtin_amdgcn_sched_barrier(0);
        const int kt = wave + j * NW;
        if (j + NS < n) load(kt + NS * NW, stage);
        if (kt == p.nkt - 1 && (p.L * Z) % 128 != 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int4_t mask = tail_mask(p.L * Z - kt * 128 - (4 * h + fq) * 16);
#pragma unroll
                for (int j = 0; j < NMB; ++j) fa[j][h] &= mask;
#pragma unroll
                for (int m = 0; m < MATS; ++m)
#pragma unroll
                    for (int i = 0; i < PB; ++i) fb[m][i][h] &= mask;
            }
        }
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int i = 0; i < PB; ++i)
#pragma unroll
                for (int j = 0; j < NMB; ++j) tile_mma<Elt, FP8>(acc[m][i][j], fb[m][i], fa[j], scale[j]);
        stage = stage + 1 == NS ? 0 : stage + 1;
    }

    floatx4_t* red = reinterpret_cast<floatx4_t*>(mine);
#pragma unroll
    for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int i = 0; i < PB; ++i)
#pragma unroll
            for (int j = 0; j < NMB; ++j) red[((m * PB + i) * NMB + j) * 64 + lane] = acc[m][i][j];
    __syncthreads();
    auto total = [&](int m, int i, int j) {
        const floatx4_t* at = reinterpret_cast<const floatx4_t*>(smem) + ((m * PB + i) * NMB + j) * 64 + lane;
        floatx4_t s = at[0];
#pragma unroll
        for (int v = 1; v < NW; ++v) s += at[v * MINE];
        return s;
    };
    for (int u = wave; u < PB * NMB; u += NW) {
        const int i = u / NMB, j = u - i * NMB;
        const int r = j * 16 + fr;
        const int c0 = (int)n0 + i * 16 + fq * 4;
        floatx4_t v[3];
        v[0] = total(0, i, j);
        int outs = 1;
        if constexpr (GATED) {
            v[1] = v[0];
            v[2] = total(1, i, j);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[0][e] = act_mul(v[1][e], v[2][e], p.act);
            if (p.G) outs = 3;
        }
        if (r >= rows_a) continue;
#pragma unroll
        for (int o = 0; o < (GATED ? 3 : 1); ++o) {
            if (o >= outs) break;
            const int64_t ld = o == 0 ? p.ldc[0] : o == 1 ? p.ldg : p.ldu;
            void* to = o == 0 ? static_cast<void*>(p.C[0]) : o == 1 ? p.G : p.U;
            if (GATED && o > 0 && p.wide) {
                float* c = static_cast<float*>(to) + r * ld + c0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c0 + e < p.N) c[e] = v[o][e];
                continue;
            }
            uint16_t* c = static_cast<uint16_t*>(to) + r * ld + c0;
            const uint32_t lo = pack2<Elt>(v[o][0], v[o][1]), hi = pack2<Elt>(v[o][2], v[o][3]);
            if (c0 + 3 < p.N) {
                *reinterpret_cast<uint2_t*>(c) = uint2_t{lo, hi};
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t word = e < 2 ? lo : hi;
                    if (c0 + e < p.N) c[e] = (uint16_t)(word >> (16 * (e & 1)));
                }
            }
        }
    }
}

// ---- gradients of the gated product, element by element -----------------------------------

struct GatedGrad {
    const void *G, *U;             // fp32 (wide) or the type
    int64_t ldg, ldu;
    const uint16_t* DH;
    int64_t lddh;
    uint16_t *DG, *DU;
    int64_t ldd;
    int64_t M;
    int N, nct;                    // column tiles of 2048
    int wide, act;
};

// dg = dh u a'(g), du = dh a(g), eight columns of a row a lane.  Both are rounded to
// the type, which the MFMAs of the three products that read them take.  Bound by memory:
// 4096 x 12288 from fp32 factors 138 us (704 MB, 5.1 TB/s).
template <typename Elt, int RPT>
__global__ __launch_bounds__(256) void gated_grad_kernel(GatedGrad p) {
    const int64_t r0 = (int64_t)(blockIdx.x / p.nct) * RPT;
    const int n = (int)(blockIdx.x % p.nct) * 2048 + threadIdx.x * 8;
    const int valid = p.N - n;
    if (valid <= 0) return;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int64_t row = r0 + i;
        if (row >= p.M) break;
        float g[8], u[8], dh[8], dg[8], du[8];
        if (p.wide) {
            const float* gr = static_cast<const float*>(p.G) + row * p.ldg + n;
            const float* ur = static_cast<const float*>(p.U) + row * p.ldu + n;
            if (valid >= 8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const floatx4_t a = *reinterpret_cast<const floatx4_t*>(gr + 4 * h);
                    const floatx4_t b = *reinterpret_cast<const floatx4_t*>(ur + 4 * h);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        g[4 * h + e] = a[e];
                        u[4 * h + e] = b[e];
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    g[e] = e < valid ? gr[e] : 0.0f;
                    u[e] = e < valid ? ur[e] : 0.0f;
                }
            }
        } else {
            unpack8<Elt>(load8(static_cast<const uint16_t*>(p.G) + row * p.ldg + n, valid), g);
            unpack8<Elt>(load8(static_cast<const uint16_t*>(p.U) + row * p.ldu + n, valid), u);
        }
        unpack8<Elt>(load8(p.DH + row * p.lddh + n, valid), dh);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float a, da;
            act_and_slope(g[e], p.act, a, da);
            dg[e] = dh[e] * u[e] * da;
            du[e] = dh[e] * a;
        }
        store8(p.DG + row * p.ldd + n, pack8<Elt>(dg), valid);
        store8(p.DU + row * p.ldd + n, pack8<Elt>(du), valid);
    }
}

}  // namespace sdt
