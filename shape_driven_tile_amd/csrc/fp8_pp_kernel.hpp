// The 8-bit product on 256 x 256 tiles with the ping-pong schedule (8 waves, 2 per
// SIMD).
//
// A k-tile is one block of scales: 128 codes a row, 32 v_mfma_f32_16x16x128 a wave
// and, since their sums are scaled before they are added, 128 v_fma_f32 beside them:
// half the MFMAs' clocks, issued between them.  8192^3: 408-410 us launch after launch (2.7
// PFLOP/s), 430-515 launched by itself or under the profiler, the MFMAs busy 67% of the
// clocks at some 1.53 GHz, the part's power limit; 4096^3 56 us.
//
// Waves 0-3 (group 0, columns 0-127 of the tile) and 4-7 (group 1) run one barrier
// interval apart, one multiplying from registers while the other reads its next 24
// fragments and issues global -> LDS loads.  A group reads only its half of B, so two
// stages of everything do (128 KB), which leaves room for the scales (P = interval,
// tile t in stage t % 2):
//   group 0: P 2t   loads A(t+1), reads tile t              | P 2t+1 MFMAs of tile t
//   group 1: P 2t+1 loads B1(t+1), B0(t+2), reads tile t    | P 2t+2 MFMAs of tile t
// A(t+1) goes where A(t-1) was (last read in P 2t-1) and is read from P 2t+2 on; B0(t+2)
// where B0(t) was (P 2t), read in P 2t+4; B1(t+1) where B1(t-1) was (P 2t-1), read in
// P 2t+3.
#pragma once

#include "tile_kernel.hpp"

namespace sdt {

template <typename Elt>
__global__ __launch_bounds__(512) void fp8_pp_kernel(TileGemm p) {
    constexpr int BM = 256, BN = 256;
    constexpr int WTM = 128, WTN = 64;            // per wave: 2 x 4 waves
    constexpr int FM = WTM / 16, FN = WTN / 16;
    constexpr int UNITS = 256 * 8;                // 16-byte LDS units of a stage
    constexpr int HALF = UNITS / 2;
    constexpr int B_BASE = 2 * UNITS;             // two stages of A, then of B
    constexpr int S_BASE = 4 * UNITS;             // scales: of A's rows, of B's halves
    constexpr int S_A = 64, S_B = 16;             // units: 256 floats; 64 copies of one
    constexpr int S_STAGE = S_A + 2 * S_B;        // four: a k-tile's are read while it is multiplied
    __shared__ int4_t smem[S_BASE + 4 * S_STAGE];

    const int t = threadIdx.x;
    const int lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int grp = wave >> 2;
    const int wave_m = wave & 1;
    const int wave_n = wave >> 1;
    const int lw = wave & 3;                      // loader index within the group

    // Where the grid is made of 16 x 16 blocks of tiles, the 256 workgroups in flight
    // cover one block and each of 8 XCDs a 4 x 8 part of it.
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
    const int rows_a = (int)min((int64_t)BM, p.M - m0);
    const int rows_b = (int)min((int64_t)BN, p.N - n0);
    const int nkt = p.nkt;

    // A load is 8 rows x 128 bytes: lane's row and chunk of load 0 of wave 0, the
    // others by adding rows (their swizzle is the same).  `voff` is made anew each
    // time: eight offsets kept would not fit the registers.
    const int64_t ld = grp == 0 ? p.lda[0] : p.ldb[0];
    const uint32_t voff0 = (uint32_t)((lane >> 3) * ld) + ((lane & 7) ^ swz_pp(lane >> 3)) * 16;
    const uint32_t step8 = (uint32_t)(8 * ld);    // bytes of 8 rows
    const uint8_t* const src = grp == 0 ? p.A[0] + m0 * ld : p.B[0] + n0 * ld;
    const uint32_t src_bytes = (uint32_t)(((grp == 0 ? rows_a : rows_b) - 1) * ld + ((p.L + 3) & ~3));
    // `n` loads of this wave: rows (first + j) * 8 .. of k-tile kt into LDS at dst
    auto dma = [&](auto count, int kt, int first, int4_t* dst) {
        constexpr int N = decltype(count)::value;
        const __amdgpu_buffer_rsrc_t r = make_rsrc(src + (int64_t)kt * 128, src_bytes - (uint32_t)kt * 128);
        uint32_t v = voff0 + (uint32_t)first * step8;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            dma16(r, dst + j * 64, v, 0);
            v += step8;
        }
    };
    typedef std::integral_constant<int, 8> Eight;
    typedef std::integral_constant<int, 4> Four;
    int4_t* const scales = smem + S_BASE;
    const float* const sa_at = p.SA + m0;
    const int blocks = (p.N + 127) / 128;
    const float* const sb0_at = p.SB + (n0 >> 7) * p.ldsb;
    const float* const sb1_at = p.SB + min((n0 >> 7) + 1, (int64_t)blocks - 1) * p.ldsb;
    // loads of each kind: 9 (A and its rows' scales), 5 (half of B and its scale)
    auto load_a = [&](int kt) {
        const int s = kt & 1;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            make_rsrc(sa_at + kt * p.ldsa, (uint32_t)rows_a * 4),
            (lds_void_ptr)(scales + (kt & 3) * S_STAGE + lw * 16), 4, lw * 256 + lane * 4, 0, 0, 0);
        dma(Eight{}, kt, lw * 8, smem + s * UNITS + lw * 8 * 64);
    };
    auto load_b = [&](int kt, int half) {
        const int s = kt & 1;
        // the four waves write the same 64 copies of the one scale
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            make_rsrc((half ? sb1_at : sb0_at) + kt, 4),
            (lds_void_ptr)(scales + (kt & 3) * S_STAGE + S_A + half * S_B), 4, 0, 0, 0, 0);
        dma(Four{}, kt, half * 16 + lw * 4, smem + B_BASE + s * UNITS + half * HALF + lw * 4 * 64);
    };
    constexpr int LB = 5;

    floatx4_t acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = floatx4_t{0.f, 0.f, 0.f, 0.f};

    typedef Operand<false, 256, 4> Op;
    const int at_a = Op::place(wave_m * FM, lane), at_b = Op::place(wave_n * FN, lane);
    int4_t fa[FM][2], fb[FN][2];
    auto read_tile = [&](int s) {
        const int4_t* abase = smem + s * UNITS;
        const int4_t* bbase = smem + B_BASE + s * UNITS;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < FM; ++j) fa[j][h] = Op::fragment(abase, at_a, j, h);
#pragma unroll
            for (int i = 0; i < FN; ++i) fb[i][h] = Op::fragment(bbase, at_b, i, h);
        }
    };
    auto clear_tail = [&]() {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int4_t m = tail_mask(p.L - (nkt - 1) * 128 - (4 * h + (lane >> 4)) * 16);
#pragma unroll
            for (int j = 0; j < FM; ++j) fa[j][h] &= m;
#pragma unroll
            for (int i = 0; i < FN; ++i) fb[i][h] &= m;
        }
    };
    auto mfma_tile = [&](int kt) {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        const float* sc = reinterpret_cast<const float*>(scales + (kt & 3) * S_STAGE);
        const float sb = sc[S_A * 4 + grp * S_B * 4];
        sc += wave_m * WTM + (lane & 15);
        // The sums of an MFMA are scaled and added while the next four run: sooner the
        // wave would have to wait for them.
        floatx4_t v[4];                           // of MFMAs n % 4
        float scale, ahead[3];                    // of part j - 1; of the next ones, as they come
        ahead[0] = sc[0];
        ahead[1] = sc[16];
        auto add = [&](int i, int j) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][j][e] = __builtin_fmaf(v[i][e], scale, acc[i][j][e]);
        };
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            if (j > 0) scale = ahead[(j - 1) % 3] * sb;
            if (j + 2 < FM) ahead[(j + 2) % 3] = sc[(j + 2) * 16];
            const int8v_t a8 = {fa[j][0][0], fa[j][0][1], fa[j][0][2], fa[j][0][3],
                                fa[j][1][0], fa[j][1][1], fa[j][1][2], fa[j][1][3]};
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                const int8v_t b8 = {fb[i][0][0], fb[i][0][1], fb[i][0][2], fb[i][0][3],
                                    fb[i][1][0], fb[i][1][1], fb[i][1][2], fb[i][1][3]};
                if (j > 0) add(i, j - 1);
                __builtin_amdgcn_sched_barrier(0);
                v[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    b8, a8, floatx4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        scale = ahead[(FM - 1) % 3] * sb;
#pragma unroll
        for (int i = 0; i < FN; ++i) add(i, FM - 1);
        // The sums are values to the compiler: an empty asm that reads them keeps
        // them from moving past the wait and the barrier that follow.
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) asm volatile("" : "+v"(acc[i][j]));
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
    };

    // ---- prologue: A(0), B(0), B0(1) -------------------------------------------------
    if (nkt > 0) {
        if (grp == 0) {
            load_a(0);
        } else {
            load_b(0, 0);
            load_b(0, 1);
            if (nkt > 1) load_b(1, 0);
        }
    }
    wait_global_loads<0>();
    __syncthreads();

    // ---- one k-tile: read phase, then MFMA phase --------------------------------------
    // The last two k-tiles have a copy of the step of their own, so that every wait is
    // a constant on one path.
    const bool ragged = (p.L & 127) != 0;
    int i = 0;                                // k-tile
    auto step = [&](auto group, auto left) {
        constexpr int G = decltype(group)::value;
        constexpr int LEFT = decltype(left)::value;       // k-tiles after this one (2: or more)
        if constexpr (G == 0 && LEFT >= 1) load_a(i + 1);
        if constexpr (G == 1 && LEFT >= 1) load_b(i + 1, 1);
        if constexpr (G == 1 && LEFT >= 2) load_b(i + 2, 0);
        read_tile(i & 1);
        // The loads among the fragment reads (masks: 0x020 global read, 0x100 LDS read).
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
        }
        if constexpr (G == 1) {
            // B0(i+1), loaded in the last read phase, is read by group 0 in the next
            __builtin_amdgcn_sched_barrier(0);
            wait_global_loads<LEFT >= 2 ? 2 * LB : LEFT == 1 ? LB : 0>();
        }
        wait_lds();
        __builtin_amdgcn_sched_barrier(0);
        if (LEFT == 0 && ragged) clear_tail();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
        mfma_tile(i);
        if constexpr (G == 0) wait_global_loads<0>();              // A(i+1)
        if constexpr (G == 1) wait_global_loads<LEFT >= 2 ? LB : 0>();   // B1(i+1); B0(i+2) may stay
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
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

    // Group 0 stores while group 1 runs its last MFMA phase, and takes the barrier
    // that matches group 1's extra one at the very end.  Every LDS read is done.
    GemmParams gp;
    gp.C = p.C[0];
    gp.ldc = p.ldc[0];
    gp.M = p.M;
    gp.N = p.N;
    store_block_staged<Elt>(gp, acc, m0 + wave_m * WTM, n0 + wave_n * WTN, lane, smem + wave * 256);
    if (grp == 0) __syncthreads();
}

}  // namespace sdt
