// The 16-bit products of tile_kernel.hpp on 256 x 256 tiles with the ping-pong
// schedule (8 waves, 2 per SIMD).
//
// Waves 0-3 (group 0, columns 0-127 of the tile) and 4-7 (group 1) run one barrier
// interval apart: in each interval one group issues the 64 MFMAs of a 64-deep k-tile
// from registers while the other reads its next 24 fragments from LDS and issues
// global -> LDS loads, group 0 those of A (two 32 KB stages), group 1 those of B
// (three); the 160 KB are full.  A turned operand's fragments take two
// ds_read_b64_tr_b16 where a K-major one's take one ds_read_b128: as many bytes and,
// on distinct banks, as many LDS clocks.  Two products that are added have the same
// strides here: other offsets for the second would not fit the registers.  Bound by the
// part's power: 8192 x 4096 x 4096 nn 190-203 us, tn 192-222 (1240-1450 TFLOP/s; the library's
// product of K-major operands 1460); gated 4096 x 12288 x 4096 604-647 (1270-1365).
#pragma once

#include "tile_kernel.hpp"

namespace sdt {

constexpr int kTilePpLdsUnits = 2 * 256 * 8 + 3 * 256 * 8;   // 160 KB of 16-byte units

template <typename Elt, bool TA, bool TB, bool GATED>
__global__ __launch_bounds__(512) void tile_pp_kernel(TileGemm p) {
    typedef typename Elt::frag8 frag8;
    constexpr int BM = 256, BN = 256, BNO = GATED ? 128 : 256;
    constexpr int WTM = 128, WTN = 64;            // per wave: 2 x 4 waves
    constexpr int FM = WTM / 16, FN = WTN / 16;
    typedef Operand<TA, BM, 4> OpA;               // loaded by one group's four waves
    typedef Operand<TB, BN, 4> OpB;
    constexpr int UNITS = OpA::UNITS;
    constexpr int B_BASE = 2 * UNITS;
    constexpr int DMA = OpA::DMA;                 // loads per k-tile per wave
    static_assert(OpB::UNITS == UNITS && OpB::DMA == DMA, "square tiles");
    __shared__ int4_t smem[kTilePpLdsUnits];

    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int grp = wave >> 2;
    const int wave_m = wave & 1;
    const int wave_n = wave >> 1;
    const int lw = wave & 3;                      // loader index within the group

    // A batch's tiles lie one under the other.  Where the grid is made of 16 x 16
    // blocks of tiles, the 256 workgroups in flight cover one block and each of 8 XCDs
    // a 4 x 8 part of it.
    const int w = blockIdx.x;
    const int gm = p.gm * p.batch;
    int64_t m0, n0;
    if (p.nxcd == 8 && (gm & 15) == 0 && (p.gn & 15) == 0) {
        const int x = w & 7, idx = w >> 3;
        const int blk = idx >> 5, k = idx & 31;
        const int bn = p.gn >> 4;
        const int bm_ = blk / bn, bn_ = blk - bm_ * bn;
        m0 = (int64_t)(bm_ * 16 + (x & 3) * 4 + (k & 3)) * BM;
        n0 = (int64_t)(bn_ * 16 + (x >> 2) * 8 + (k >> 2)) * BNO;
    } else {
        GemmParams gp;
        gp.gm = gm;
        gp.gn = p.gn;
        grouped_origin(gp, xcd_remap(w, gm * p.gn, p.nxcd), BM, BNO, m0, n0);
    }
    const int batch = (int)(m0 / BM) >= p.gm ? 1 : 0;
    m0 -= (int64_t)batch * p.gm * BM;
    const int rows_a = (int)min((int64_t)BM, p.M - m0);
    const int rows_b = (int)min((int64_t)BNO, p.N - n0);
    const int all = p.products * p.nkt;

    // This group's operand: group 0 loads A, group 1 B.  The k-tile that the next load
    // takes; the pointers of both pairs stay at hand.
    uint32_t voff[DMA];
#pragma unroll
    for (int j = 0; j < DMA; ++j) {
        if (grp == 0) {
            voff[j] = OpA::offset(lw, lane, j, p.lda[0], [](int r) { return r; });
        } else if constexpr (GATED) {
            const bool second = ((lw * DMA + j) * 8) % WTN >= WTN / 2;
            voff[j] = OpB::offset(lw, lane, j, second ? p.ldb[1] : p.ldb[0], [](int r) {
                return r / WTN * (WTN / 2) + r % (WTN / 2);
            });
        } else {
            voff[j] = OpB::offset(lw, lane, j, p.ldb[0], [](int r) { return r; });
        }
    }
    typename OpA::Stream stream_a;
    typename OpB::Stream stream_b, stream_u;
    const int64_t a_at = TA ? m0 * 2 : m0 * p.lda[0], b_at = TB ? n0 * 2 : n0 * p.ldb[0];
    const uint8_t* const a1 = p.A[1] + a_at;
    const uint8_t* const b1 = GATED ? p.B[1] + n0 * p.ldb[1] : p.B[1] + b_at;
    const int columns_a = TA ? (int)(p.M - m0) : rows_a, columns_b = TB ? (int)(p.N - n0) : rows_b;
    stream_a.start(batch ? a1 : p.A[0] + a_at, p.lda[0], columns_a, 0, p.L, 2);
    stream_b.start(batch ? b1 : p.B[0] + b_at, p.ldb[0], columns_b, 0, p.L, 2);
    if constexpr (GATED) stream_u.start(b1, p.ldb[1], columns_b, 0, p.L, 2);
    int load_k = 0;
    auto dma_a = [&](int stage) {
        const __amdgpu_buffer_rsrc_t r = stream_a.next();
        int4_t* const dst = smem + stage * UNITS + lw * DMA * 64;
#pragma unroll
        for (int j = 0; j < DMA; ++j) dma16(r, dst + j * 64, voff[j], 0);
        if (++load_k == p.nkt && p.products == 2) stream_a.start(a1, p.lda[0], columns_a, 0, p.L, 2);
    };
    auto dma_b = [&](int stage) {
        const __amdgpu_buffer_rsrc_t r = stream_b.next();
        int4_t* const dst = smem + B_BASE + stage * UNITS + lw * DMA * 64;
        if constexpr (GATED) {
            const __amdgpu_buffer_rsrc_t r2 = stream_u.next();
#pragma unroll
            for (int j = 0; j < DMA; ++j) {
                const bool second = ((lw * DMA + j) * 8) % WTN >= WTN / 2;
                dma16(second ? r2 : r, dst + j * 64, voff[j], 0);
            }
        } else {
#pragma unroll
            for (int j = 0; j < DMA; ++j) dma16(r, dst + j * 64, voff[j], 0);
            if (++load_k == p.nkt && p.products == 2) stream_b.start(b1, p.ldb[0], columns_b, 0, p.L, 2);
        }
    };

    floatx4_t acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    int at_a = OpA::place(wave_m * FM, lane), at_b = OpB::place(wave_n * FN, lane);
    int4_t fa[2][FM], fb[2][FN];
    auto read_a = [&](int sa) {
        // the parts' places are made from this each time: kept, they would not fit
        // the registers
        asm volatile("" : "+v"(at_a));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < FM; ++j) fa[h][j] = OpA::fragment(smem + sa * UNITS, at_a, j, h);
    };
    auto read_b = [&](int sb) {
        asm volatile("" : "+v"(at_b));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < FN; ++i) fb[h][i] = OpB::fragment(smem + B_BASE + sb * UNITS, at_b, i, h);
    };
    // The last k-tile of a product: what its K-major rows hold past their end is
    // not zero.
    auto clear_tail = [&](int k) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int4_t m = tail_mask(p.L * 2 - k * 128 - (4 * h + (lane >> 4)) * 16);
            if constexpr (!TA) {
#pragma unroll
                for (int j = 0; j < FM; ++j) fa[h][j] &= m;
            }
            if constexpr (!TB) {
#pragma unroll
                for (int i = 0; i < FN; ++i) fb[h][i] &= m;
            }
        }
    };
    const bool ragged = (!TA || !TB) && (p.L & 63) != 0;
    auto mfma_tile = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j)
                    acc[i][j] = Elt::mfma16(__builtin_bit_cast(frag8, fb[h][i]),
                                            __builtin_bit_cast(frag8, fa[h][j]), acc[i][j]);
        // The MFMAs are values to the compiler: an empty asm that reads them
        // keeps it from moving them past the wait and the barrier that follow.
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) asm volatile("" : "+v"(acc[i][j]));
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };

    // ---- prologue: A(0), B(0), B(1) -------------------------------------------------
    if (all > 0) {
        if (grp == 0) {
            dma_a(0);
        } else {
            dma_b(0);
            if (all > 1) dma_b(1);
        }
    }
    wait_global_loads<0>();
    __syncthreads();

    // ---- one k-tile: read phase, then MFMA phase --------------------------------------
    // The last two k-tiles have a copy of the step of their own, so that every wait is
    // a constant on one path.
    int i = 0, sb = 0;                        // k-tile; its B stage (i % 3)
    auto step = [&](auto group, auto left) {
        constexpr int G = decltype(group)::value;
        constexpr int LEFT = decltype(left)::value;       // k-tiles after this one (2: or more)
        const int sa = i & 1;
        const int sb2 = (sb == 0) ? 2 : sb - 1;   // (i + 2) % 3
        // Turned fragments first: the compiler holds back a ds_read_tr until every load
        // into LDS that was issued before it has landed.  Those of the last read phase
        // have; this one's would take it the phase (8192 x 4096 x 4096: nn 243 -> 194 us, tn 231 -> 202).
        if constexpr (TB) read_b(sb);
        if constexpr (TA) read_a(sa);
        if constexpr (TA || TB) __builtin_amdgcn_sched_barrier(0);
        if constexpr (G == 0 && LEFT >= 1) dma_a(sa ^ 1);
        if constexpr (G == 1 && LEFT >= 2) dma_b(sb2);
        if constexpr (!TB) read_b(sb);
        if constexpr (!TA) read_a(sa);
        // The loads among the other reads (masks: 0x020 global read, 0x100 LDS read).
        constexpr int READS = 2 * ((TA ? 0 : FM) + (TB ? 0 : FN)) / DMA;
        if constexpr (READS > 0) {
#pragma unroll
            for (int m = 0; m < DMA; ++m) {
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
            }
        }
        if constexpr (G == 1) {
            // B(i+1) must be in LDS before group 0 reads k-tile i + 1 in the next
            // phase; B(i+2) may stay in flight.
            wait_global_loads<LEFT >= 2 ? DMA : 0>();
        }
        wait_lds();
        __builtin_amdgcn_sched_barrier(0);
        // (a first product that another is added to ends before the last k-tile)
        if (ragged && (LEFT == 0 || (!GATED && i == p.nkt - 1))) clear_tail(p.nkt - 1);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
        mfma_tile();
        if constexpr (G == 0) wait_global_loads<0>();  // A(i+1), read by both groups next
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
        sb = (sb == 2) ? 0 : sb + 1;
        ++i;
    };
    auto loop = [&](auto group) {
        while (i + 2 < all) step(group, std::integral_constant<int, 2>{});
        if (i + 1 < all) step(group, std::integral_constant<int, 1>{});
        if (i < all) step(group, std::integral_constant<int, 0>{});
    };
    if (grp == 0) {
        loop(std::integral_constant<int, 0>{});
    } else {
        __syncthreads();                      // one phase behind group 0
        loop(std::integral_constant<int, 1>{});
    }

    // Group 0 stores while group 1 runs its last MFMA phase, and takes the barrier
    // that matches group 1's extra one at the very end.  Every LDS read is done: the
    // plain store's stages are 4 KB a wave of A's second.
    if constexpr (GATED) {
        tile_store<Elt, true, FN, FM>(p, 0, acc, (uint32_t)m0 + wave_m * WTM, rows_a - wave_m * WTM,
                                      (uint32_t)n0 + wave_n * (WTN / 2), lane);
    } else {
        GemmParams gp;
        gp.C = p.C[batch];
        gp.ldc = p.ldc[batch];
        gp.M = p.M;
        gp.N = p.N;
        store_block_staged<Elt>(gp, acc, m0 + wave_m * WTM, n0 + wave_n * WTN, lane,
                                smem + UNITS + wave * 256);
    }
    if (grp == 0) __syncthreads();
}

}  // namespace sdt
