// The 256 x 256 MX4 product with the ping-pong schedule (8 waves, 2 per SIMD).
//
// An MX4 k-tile of 256 is 128 bytes a row and 64 MFMAs a wave, as a 64-deep
// k-tile of the 16-bit ping-pong kernel is, and each MFMA takes as many cycles:
// the same schedule carries it at four times the rate.  Waves 0-3 (group 0,
// columns 0-127 of the tile) and 4-7 (group 1) run one barrier interval apart:
// in each interval one group issues the 64 MFMAs of a k-tile from registers
// while the other reads its next 24 fragments from LDS and issues global -> LDS
// loads, group 0 those of A (two 32 KB stages), group 1 those of B (three).
// The 160 KB are full, so scales go from memory into registers, one k-tile
// ahead: 8 bytes a lane per 64 rows, three coalesced 512-byte loads a wave.
// 8192^3: 228-250 us (4.4-4.8 PFLOP/s), MFMAs busy 58% of the clocks; bound by the
// power limit (a register-only loop of these MFMAs on random codes: 6.15-7.15
// PFLOP/s) and by the stage loads (197 us with them left out).  128 x 128 tiles,
// two workgroups a CU, take 301 us there.  The accumulators and fragments fill the
// 256 registers; four more spill to 16 bytes of scratch a lane.
#pragma once

#include "mx4_kernel.hpp"

namespace sdt {

constexpr int kMx4PpLdsUnits = 2 * 256 * 8 + 3 * 256 * 8;   // 160 KB of 16-byte units

template <typename Elt>
__global__ __launch_bounds__(512) void mx4_pp_kernel(Mx4Gemm p) {
    constexpr int BM = 256, BN = 256;
    constexpr int WTM = 128, WTN = 64;            // per wave: 2 x 4 waves
    constexpr int FM = WTM / 16, FN = WTN / 16;
    constexpr int UNITS = 256 * 8;                // 16-byte LDS units of a stage
    constexpr int B_BASE = 2 * UNITS;
    constexpr int DMA = 8;                        // loads per k-tile per wave: 64 rows
    __shared__ int4_t smem[kMx4PpLdsUnits];

    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int grp = wave >> 2;
    const int wave_m = wave & 1;
    const int wave_n = wave >> 1;
    const int lw = wave & 3;                      // loader index within the group

    // Where the grid is made of 16 x 16 blocks of tiles, the 256 workgroups in
    // flight cover one block and each of 8 XCDs a 4 x 8 part of it.
    const int w = blockIdx.x;
    int64_t m0, n0;
    if (p.nxcd == 8 && (p.gm & 15) == 0 && (p.gn & 15) == 0) {
        const int x = w & 7, idx = w >> 3;
        const int blk = idx >> 5, k = idx & 31;
        const int bn = p.gn >> 4;
        const int bm_ = blk / bn, bn_ = blk - bm_ * bn;
        m0 = (int64_t)(bm_ * 16 + (x & 3) * 4 + (k & 3)) * BM;
        n0 = (int64_t)(bn_ * 16 + (x >> 2) * 8 + (k >> 2)) * BN;
    } else {
        GemmParams gp;
        gp.gm = p.gm;
        gp.gn = p.gn;
        grouped_origin(gp, xcd_remap(w, p.gm * p.gn, p.nxcd), BM, BN, m0, n0);
    }
    const int rows_a = (int)min((int64_t)BM, (int64_t)p.M - m0);
    const int rows_b = (int)min((int64_t)BN, (int64_t)p.N - n0);
    const uint32_t srow = (uint32_t)p.nkt * kMx4Tile;   // scale bytes of 64 rows

    // This group's operand: group 0 loads A, group 1 B.
    const uint8_t* src = grp == 0 ? p.A + m0 * p.lda : p.B + n0 * p.ldb;
    const int64_t ld = grp == 0 ? p.lda : p.ldb;
    const uint32_t src_bytes =
        (uint32_t)(((grp == 0 ? rows_a : rows_b) - 1) * ld + p.rowbytes);
    uint32_t voff[DMA];
#pragma unroll
    for (int j = 0; j < DMA; ++j) {
        const int row = lw * 64 + j * 8 + (lane >> 3);
        const int pos = (lane & 7) ^ mx4_swz(row);
        voff[j] = (uint32_t)(row * ld) + pos * 16;
    }
    // The k offset moves the descriptor: rows past M or N and the last row's
    // bytes past its blocks lie past its end and read as zero.
    int4_t* const dst = smem + (grp == 0 ? 0 : B_BASE) + lw * DMA * 64;
    auto dma = [&](int kt, int stage) {
        const __amdgpu_buffer_rsrc_t r = make_rsrc(src + kt * 128, src_bytes - kt * 128);
#pragma unroll
        for (int j = 0; j < DMA; ++j) dma16(r, dst + stage * UNITS + j * 64, voff[j], 0);
    };

    // Scale tiles of this wave: two of A, one of B (none past the matrix: the
    // descriptor is empty and zeros are read).
    auto tile_rsrc = [&](const uint8_t* s, int64_t tile, bool in) {
        return make_rsrc(in ? s + tile * srow : s, in ? srow : 0u);
    };
    const __amdgpu_buffer_rsrc_t rs0 =
        tile_rsrc(p.SA, m0 / 64 + wave_m * 2, wave_m * 128 < rows_a);
    const __amdgpu_buffer_rsrc_t rs1 =
        tile_rsrc(p.SA, m0 / 64 + wave_m * 2 + 1, wave_m * 128 + 64 < rows_a);
    const __amdgpu_buffer_rsrc_t rs2 = tile_rsrc(p.SB, n0 / 64 + wave_n, wave_n * 64 < rows_b);
    int2_t sc[3], next[3];
    auto load_scales = [&](int kt, int2_t (&s)[3]) {
        const int so = kt * kMx4Tile;
        s[0] = __builtin_bit_cast(int2_t, __builtin_amdgcn_raw_buffer_load_b64(rs0, lane * 8, so, 0));
        s[1] = __builtin_bit_cast(int2_t, __builtin_amdgcn_raw_buffer_load_b64(rs1, lane * 8, so, 0));
        s[2] = __builtin_bit_cast(int2_t, __builtin_amdgcn_raw_buffer_load_b64(rs2, lane * 8, so, 0));
    };

    floatx4_t acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    const int frow = lane & 15, fq = lane >> 4;
    const int fsw = mx4_swz(frow);
    const int a_row0 = wave_m * WTM + frow;
    const int b_row0 = wave_n * WTN + frow;
    int4_t fa[2][FM], fb[2][FN];
    auto read_tile = [&](int sa, int sb) {
        const int4_t* abase = smem + sa * UNITS;
        const int4_t* bbase = smem + B_BASE + sb * UNITS;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int chunk = (2 * fq + h) ^ fsw;
#pragma unroll
            for (int j = 0; j < FM; ++j) fa[h][j] = abase[(a_row0 + j * 16) * 8 + chunk];
#pragma unroll
            for (int i = 0; i < FN; ++i) fb[h][i] = bbase[(b_row0 + i * 16) * 8 + chunk];
        }
    };
    auto mfma_half = [&](auto half) {
        constexpr int S = decltype(half)::value;
#pragma unroll
        for (int i = 0; i < FN; i += 2) {
            const int b = sc[2][i >> 1];
#pragma unroll
            for (int j = 0; j < FM; j += 2) {
                const int a = sc[j >> 2][(j >> 1) & 1];
                acc[i][j] = mx4_mfma_part<S, 0, 0>(fb[S][i], fa[S][j], acc[i][j], b, a);
                acc[i][j + 1] = mx4_mfma_part<S, 0, 1>(fb[S][i], fa[S][j + 1], acc[i][j + 1], b, a);
                acc[i + 1][j] = mx4_mfma_part<S, 1, 0>(fb[S][i + 1], fa[S][j], acc[i + 1][j], b, a);
                acc[i + 1][j + 1] =
                    mx4_mfma_part<S, 1, 1>(fb[S][i + 1], fa[S][j + 1], acc[i + 1][j + 1], b, a);
            }
        }
    };
    auto mfma_tile = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        mfma_half(std::integral_constant<int, 0>{});
        mfma_half(std::integral_constant<int, 1>{});
        // The MFMAs are values to the compiler: an empty asm that reads them
        // keeps it from moving them past the wait and the barrier that follow.
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) asm volatile("" : "+v"(acc[i][j]));
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };

    // ---- prologue: A(0), B(0), B(1), the first scales -------------------------------
    const int nkt = p.nkt;
    if (nkt > 0) {
        load_scales(0, next);
        dma(0, 0);
        if (grp == 1 && nkt > 1) dma(1, 1);
    }
    wait_global_loads<0>();
    __syncthreads();

    // ---- one k-tile: read phase, then MFMA phase --------------------------------------
    // Each group has its own copy of the loop and the last two k-tiles theirs, so
    // that every wait is a constant on one path: the compiler then sees that the
    // scales have arrived and adds no wait of its own.
    int i = 0, sb = 0;                        // k-tile; its B stage (i % 3)
    auto step = [&](auto group, auto left) {
        constexpr int G = decltype(group)::value;
        constexpr int LEFT = decltype(left)::value;       // k-tiles after this one (2: or more)
        const int sa = i & 1;
        const int sb2 = (sb == 0) ? 2 : sb - 1;   // (i + 2) % 3
        // The scales of this k-tile, which have arrived, leave the registers that
        // those of the next are loaded into.
        auto scales = [&]() {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int d = 0; d < 3; ++d) {
                sc[d] = next[d];
                asm volatile("" : "+v"(sc[d]));   // copied here, not before a wait above
            }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (LEFT >= 1) load_scales(i + 1, next);
            __builtin_amdgcn_sched_barrier(0);
        };
        if constexpr (G == 0) scales();
        if constexpr (G == 0 && LEFT >= 1) dma(i + 1, sa ^ 1);
        if constexpr (G == 1 && LEFT >= 2) dma(i + 2, sb2);
        read_tile(sa, sb);
        // 8 loads and 24 fragment reads per wave, interleaved (masks: 0x020
        // global read, 0x100 LDS read).
#pragma unroll
        for (int m = 0; m < DMA; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
        }
        if constexpr (G == 1) {
            // B(i+1) must be in LDS before group 0 reads k-tile i + 1 in the next
            // phase; the scales of k-tile i were issued after it and before B(i+2).
            __builtin_amdgcn_sched_barrier(0);
            wait_global_loads<LEFT >= 2 ? DMA : 0>();
            scales();
        }
        wait_lds();
        __builtin_amdgcn_sched_barrier(0);
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
        while (i + 2 < nkt) step(group, std::integral_constant<int, 2>{});
        if (i + 1 < nkt) step(group, std::integral_constant<int, 1>{});
        if (i < nkt) step(group, std::integral_constant<int, 0>{});
    };
    if (grp == 0) {
        loop(std::integral_constant<int, 0>{});
    } else {
        __syncthreads();                      // one phase behind group 0
        loop(std::integral_constant<int, 1>{});
    }

    // Group 0 stores while group 1 runs its last MFMA phase, and takes the
    // barrier that matches group 1's extra one at the very end.  The stage is
    // A's second, 4 KB a wave: its last reads have completed.
    GemmParams gp;
    gp.C = p.C;
    gp.ldc = p.ldc;
    gp.M = p.M;
    gp.N = p.N;
    store_block_staged<Elt>(gp, acc, m0 + wave_m * WTM, n0 + wave_n * WTN, lane,
                            smem + UNITS + wave * 256);
    if (grp == 0) __syncthreads();
}

}  // namespace sdt
