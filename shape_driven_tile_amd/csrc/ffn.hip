// C ABI of the feed-forward entry points (declared in sdt.h): 8-bit matrices and
// their products, the norm, the gated block, products of operands stored along
// the other dimension.  Argument checks on the host, the choice of a kernel, the
// launch.  Allocates nothing.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "fp8_pp_kernel.hpp"
#include "launcher.hpp"
#include "runtime.hpp"
#include "sdt.h"
#include "tile_kernel.hpp"
#include "tile_pp_kernel.hpp"

namespace sdt {
namespace {

constexpr int64_t kMaxK = int64_t(1) << 23;
constexpr int64_t kMaxStride = int64_t(1) << 22;          // elements, exclusive (gemm_f16's)
constexpr int64_t kMaxRows = INT_MAX - 255;           // the last tile's end fits 32 bits
constexpr int64_t kMaxNorm = 32768;                   // elements of a normed row
constexpr int kSplitTarget = 256;                     // workgroups that a split aims at

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int launched(hipError_t e) { return e == hipSuccess ? SDT_OK : fail_hip(e); }

template <typename P>
int launch(const void* kernel, int64_t grid, int threads, P& params, void* stream) {
    if (grid * threads > UINT32_MAX) return SDT_ERR_UNSUPPORTED;      // a launch's threads
    if (grid == 0) return SDT_OK;
    void* args[] = {&params};
    return launched(hipLaunchKernel(kernel, dim3((unsigned)grid), dim3((unsigned)threads), args, 0,
                                    static_cast<hipStream_t>(stream)));
}

// ---- 8-bit matrices -------------------------------------------------------------------

bool known_block(const sdt_fp8* m) { return m && (m->block == 1 || m->block == 128); }

// Codes and scales of a rows x K matrix (both > 0).
int check_fp8(int64_t rows, int64_t K, const sdt_fp8& m) {
    if (!m.q || !m.s) return SDT_ERR_INVALID_ARG;
    if (m.ldq < K || m.lds < (m.block == 1 ? rows : ceil_div(K, 128))) return SDT_ERR_INVALID_ARG;
    if (K > kMaxK || rows > kMaxRows || m.ldq >= 2 * kMaxStride || m.lds > INT_MAX) return SDT_ERR_UNSUPPORTED;
    if (misaligned(m.q, 16) || misaligned(m.s, 4) || (rows > 1 && m.ldq % 16 != 0))
        return SDT_ERR_UNSUPPORTED;
    return SDT_OK;
}

// Rows a workgroup of 256 lanes, eight elements each, takes.  One, as a rule: codes of
// 4096 x 4096 13.3 us and 15.7 by eight rows together, 8192 x 8192 39.1 and 42.1, dg and du of
// 8192 x 4096 110 and 116.  Short rows leave lanes idle: from 128 of them a CU on, codes of up
// to 1024 elements by eight together (65536 x 512 32.9 us and 29.7, 262144 x 128 112 and 101;
// 16384 x 512 11.1 and 11.7, 32768 x 1500 30.7 and 29.9), dg and du of up to 256 by four
// (131072 x 256 118 and 112, 262144 x 128 193 and 166; 65536 x 512 103 and 108).  Besides,
// where one by one would be more threads than a launch has.
bool many_short(int64_t rows, int64_t K, int64_t most, int num_cu) {
    return (K <= most && rows >= int64_t(128) * num_cu) || rows * ceil_div(K, 2048) * 256 > UINT32_MAX;
}
// Values back, which are less work a row: eight rows together from 32 row tiles a CU on
// (8192 x 2048 10.8 us and 8.9, 32768 x 512 17.5 and 13.2, 8192 x 8192 39.0 and 39.7; 4096 x
// 2048 5.4 and 5.8).
bool many_tiles(int64_t rows, int64_t nct, int num_cu) { return rows * nct >= int64_t(32) * num_cu; }

template <typename Elt>
int quantize8(int64_t rows, int64_t K, const void* X, int64_t ldx, const sdt_fp8* out, void* stream) {
    if (rows < 0 || K < 0 || !known_block(out)) return SDT_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return SDT_OK;
    if (!X || ldx < K) return SDT_ERR_INVALID_ARG;
    int rc = check_fp8(rows, K, *out);
    if (rc != SDT_OK) return rc;
    if (misaligned(X, 2)) return SDT_ERR_UNSUPPORTED;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != SDT_OK) return rc;
    Fp8Quant p;
    p.X = static_cast<const uint16_t*>(X);
    p.ldx = ldx;
    p.Q = static_cast<uint8_t*>(out->q);
    p.ldq = out->ldq;
    p.S = out->s;
    p.lds = out->lds;
    p.rows = rows;
    p.K = (int)K;
    if (out->block == 128) {
        p.nct = (int)ceil_div(K, 128);
        return launch(K >= 8 ? reinterpret_cast<const void*>(&fp8_quantize_blocks_kernel<Elt, true>)
                             : reinterpret_cast<const void*>(&fp8_quantize_blocks_kernel<Elt, false>),
                      ceil_div(rows, 128) * p.nct, 256, p, stream);
    }
    p.nct = (int)ceil_div(K, 2048);
    if (K >= 8 && many_short(rows, K, 1024, dev.num_cu))
        return launch(reinterpret_cast<const void*>(&fp8_quantize_rows_kernel<Elt, 8>),
                      ceil_div(rows, 8) * p.nct, 256, p, stream);
    return launch(reinterpret_cast<const void*>(&fp8_quantize_rows_kernel<Elt, 1>), rows * p.nct, 256, p,
                  stream);
}

template <typename Out>
int dequantize8(int64_t rows, int64_t K, const sdt_fp8* m, void* Y, int64_t ldy, void* stream) {
    if (rows < 0 || K < 0 || !known_block(m)) return SDT_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return SDT_OK;
    if (!Y || ldy < K) return SDT_ERR_INVALID_ARG;
    int rc = check_fp8(rows, K, *m);
    if (rc != SDT_OK) return rc;
    if (misaligned(Y, std::is_same_v<Out, float> ? 4 : 2)) return SDT_ERR_UNSUPPORTED;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != SDT_OK) return rc;
    Fp8Dequant p;
    p.Q = static_cast<const uint8_t*>(m->q);
    p.ldq = m->ldq;
    p.S = m->s;
    p.lds = m->lds;
    p.block = m->block;
    p.Y = Y;
    p.ldy = ldy;
    p.rows = rows;
    p.K = (int)K;
    p.nct = (int)ceil_div(K, 2048);
    if (K >= 8 && many_tiles(rows, p.nct, dev.num_cu))
        return launch(reinterpret_cast<const void*>(&fp8_dequantize_kernel<Out, 8>), ceil_div(rows, 8) * p.nct,
                      256, p, stream);
    return launch(reinterpret_cast<const void*>(&fp8_dequantize_kernel<Out, 1>), rows * p.nct, 256, p, stream);
}

// ---- products ---------------------------------------------------------------------------

int check_out(int64_t rows, int64_t N, const void* C, int64_t ldc) {
    if (!C || ldc < N) return SDT_ERR_INVALID_ARG;
    if (misaligned(C, 16) || (rows > 1 && ldc % 8 != 0)) return SDT_ERR_UNSUPPORTED;
    return SDT_OK;
}

// A 16-bit operand of `rows` rows of K (> 0) elements, as gemm_f16's.
int check_in(int64_t rows, int64_t K, const void* A, int64_t lda) {
    if (!A || lda < K) return SDT_ERR_INVALID_ARG;
    if (lda >= kMaxStride) return SDT_ERR_UNSUPPORTED;
    if (misaligned(A, 16) || (rows > 1 && lda % 8 != 0)) return SDT_ERR_UNSUPPORTED;
    return SDT_OK;
}

// Bytes from row to row of an operand of `rows` rows, `size` bytes an element, whose caller
// gave a stride of `ld` elements.  A single row's may be any, but the kernels address the
// rows after it too and find them past its end: at whole 16 bytes they are.  (A row of five
// 16-bit values, turned: it ends in the 4 bytes 8 .. 11, and at a stride of 10 bytes the next
// row would begin in them.)
int64_t row_bytes(int64_t rows, int64_t ld, int size) {
    return rows > 1 ? ld * size : ceil_div(ld * size, 16) * 16;
}

TileGemm product(int64_t M, int64_t N, int64_t L, int z, int nxcd) {
    TileGemm p = {};
    p.M = (int)M;
    p.N = (int)N;
    p.L = (int)L;
    p.nkt = (int)ceil_div(L * z, 128);
    p.products = p.batch = p.splits = 1;
    p.nxcd = nxcd;
    return p;
}

template <typename Elt, bool FP8, int BM, int BN, int WM, int WN, int NS, bool TA, bool TB, bool GATED>
int launch_tile(TileGemm& p, void* stream) {
    p.gm = (int)ceil_div(p.M, BM);
    p.gn = (int)ceil_div(p.N, GATED ? BN / 2 : BN);
    const int64_t grid = (int64_t)p.gm * p.gn * p.batch * p.splits;
    const int rc = launch(
        reinterpret_cast<const void*>(&tile_gemm_kernel<Elt, FP8, BM, BN, WM, WN, NS, TA, TB, GATED>), grid,
        WM * WN * 64, p, stream);
    // only 64-row tiles are split: where 128-row ones are taken they fill the CUs
    if constexpr (BM == 64) {
        if (rc == SDT_OK && p.splits > 1)
            return launch(reinterpret_cast<const void*>(&tile_reduce_kernel<Elt, BM, BN, WM, WN, GATED>),
                          (int64_t)p.gm * p.gn * p.batch, WM * WN * 64, p, stream);
    }
    return rc;
}

template <typename Elt, bool TA, bool TB, bool GATED>
int launch_pp(TileGemm& p, void* stream) {
    p.gm = (int)ceil_div(p.M, 256);
    p.gn = (int)ceil_div(p.N, GATED ? 128 : 256);
    return launch(reinterpret_cast<const void*>(&tile_pp_kernel<Elt, TA, TB, GATED>),
                  (int64_t)p.gm * p.gn * p.batch, 512, p, stream);
}

// Whether t256 tiles of 256 x 256, a workgroup a CU, beat t128 of 128 x 128, two: by a
// CU's time in us, `kt` k-tiles of 128 bytes a tile (16 bits, gated and turned, and 8
// bits; fitted to both sides at 81 sizes of 64 to 1024 large tiles, 8 to 64 k-tiles, half of
// them with rows off 128 bytes).  A round of 256 x 256 tiles takes 1.4 a k-tile (8 bits 1.55)
// and 10.5 (9.5) besides, a partial one down to 0.7 of the 1.4 as its tiles get fewer.  One
// of 128 x 128 tiles takes 0.95 and 6 (1.05 and 5.5), a partial one its share and a tenth,
// since CUs go on to it as they come free; right after the first round, whose tiles end
// together, 0.65 at least.  256 against 128, nn and 8 bits: 128 large tiles, 2048 x 4096 x
// 4096 73 and 62, 46 and 38; 144 (3000^3) 62 and 92, 39 and 50; 160 (2560 x 4096 x 2048) 42
// and 54, 27 and 33; 256 (4096^3) 95 and 125, 55 and 68; 288 (2304 x 8192 x 8192) 311 and 295,
// 179 and 165; 512 (8192 x 4096 x 1024) 57 and 77, 36 and 48; 576 (6000 x 6000 x 512) 63 and
// 52, 49 and 35.  What it takes is 0.4% slower than the better side in the mean, 13% (8 bits
// 22%: 7064 x 4008 x 472, 40 and 33) at most.
bool large_tiles(int64_t t256, int64_t t128, int64_t kt, int64_t cu, bool fp8) {
    const double k = (double)kt;
    const double slope = fp8 ? 1.55 : 1.4, besides = fp8 ? 9.5 : 10.5;
    const int64_t rest256 = t256 % cu;
    double large = (double)(t256 / cu) * (slope * k + besides);
    if (rest256 > 0) large += slope * (0.7 + 0.3 * (double)rest256 / (double)cu) * k + besides;
    const int64_t whole = t128 / (2 * cu), rest = t128 % (2 * cu);
    double part = rest > 0 ? 0.1 + 0.9 * (double)rest / (2.0 * (double)cu) : 0.0;
    if (rest > 0 && whole == 1) part = std::max(part, 0.65);
    const double full = fp8 ? 1.05 * k + 5.5 : 0.95 * k + 6.0;
    return large < full * ((double)whole + part);
}

// Few rows: the weights are streamed.
template <typename Elt, bool FP8, bool GATED, int NW, int PB, int NMB, int NS>
int launch_rows(TileGemm& p, void* stream) {
    p.gm = 1;
    p.gn = (int)ceil_div(p.N, PB * 16);
    return launch(reinterpret_cast<const void*>(&rows_gemm_kernel<Elt, FP8, GATED, NW, PB, NMB, NS>), p.gn,
                  NW * 64, p, stream);
}
constexpr int kFewRows = 16;

// 8 bits, up to 16 rows, or up to 64 of weights that are soon read: 64 rows, weights from
// memory, streamed against split tiles: 4096 x 4096 (16 MB) 9.3 us and 12.2, 3000 x 8192 (23
// MB) 14.3 and 14.6, 4096 x 8192 (32 MB) 14.5 and 15.0, 8192 x 4096 (32 MB) 16.4 and 14.6, 10240
// x 4096 (40 MB) 22.9 and 18.1, 4096 x 12288 (48 MB) 22.1 and 20.1; 17 rows of the last 16.3 and
// 18.1.  16 columns a workgroup where 32 would leave CUs idle.
bool few_rows8(int64_t M, int64_t N, int64_t K) {
    return M <= kFewRows || (M <= 64 && N * K <= int64_t(1) << 25);
}
template <typename Elt>
int launch_rows8(TileGemm& p, int num_cu, void* stream) {
    if (p.M > kFewRows) return launch_rows<Elt, true, false, 4, 1, 4, 3>(p, stream);
    return ceil_div(p.N, 32) < num_cu ? launch_rows<Elt, true, false, 8, 1, 1, 4>(p, stream)
                                      : launch_rows<Elt, true, false, 4, 2, 1, 3>(p, stream);
}

// How a product with a workspace is laid out: its tiles' side and the workgroups
// along each tile's k-tiles.  `from`: 128 x 128 tiles that are worth more than 64 x 64
// ones (256 x 12288 x 4096, 192 of them: turned 45-51 us against 49, 8 bits 30 against
// 28).  Fewer are where the 64 x 64 ones are more than the two a CU that run at once and
// K is at most 1024 (`brief` k-tiles): 1408 x 2048, 176 of them, turned 9.3 us against 10.7
// at K = 512, 13.7 against 14.8 at 1024 and 24.8 against 24.7 at 2048; 8 bits 7.3 against
// 9.1, 9.1 against 11.0 and 16.0 against 15.7.  Where tiles leave CUs idle, each split
// keeps eight k-tiles at least.
struct Split {
    int side, splits;
    int64_t bytes;
};
Split plan_split(int64_t M, int64_t N, int64_t kt, int batch, int64_t from, int64_t brief) {
    Split s;
    const int64_t t128 = ceil_div(M, 128) * ceil_div(N, 128) * batch;
    const int64_t t64 = ceil_div(M, 64) * ceil_div(N, 64) * batch;
    s.side = t128 >= from || (t64 > 2 * kSplitTarget && kt <= brief) ? 128 : 64;
    const int64_t tiles = ceil_div(M, s.side) * ceil_div(N, s.side) * batch;
    int64_t n = tiles > 0 ? kSplitTarget / tiles : 1;
    n = std::min(n, kt / 8);
    s.splits = s.side == 128 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(n, 16));
    s.bytes = s.splits > 1 ? tiles * s.splits * 64 * 64 * 4 : 0;
    return s;
}
Split plan_turned(int64_t M, int64_t N, int64_t kt, int batch) {
    return plan_split(M, N, kt, batch, kSplitTarget * 3 / 4, 16);
}
Split plan_split8(int64_t M, int64_t N, int64_t K) {
    return plan_split(M, N, ceil_div(K, 128), 1, kSplitTarget, 8);
}
// Gated: 64 columns of both matrices a tile.  128 rows only where there are tiles for
// more than one a CU (512 x 4096 x 4096, 256 of them: 51 us against 36; 1024 x 4096 x
// 4096, 512: 60 against 70).
Split plan_gated(int64_t M, int64_t N, int64_t K) {
    Split s;
    s.side = ceil_div(M, 128) * ceil_div(N, 64) >= kSplitTarget * 3 / 2 ? 128 : 64;
    const int64_t tiles = ceil_div(M, s.side) * ceil_div(N, 64), kt = ceil_div(K, 64);
    const int64_t n = std::min(tiles > 0 ? kSplitTarget / tiles : 1, kt / 8);
    s.splits = s.side == 128 ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(n, 16));
    s.bytes = s.splits > 1 ? tiles * s.splits * 64 * 128 * 4 : 0;
    return s;
}
void take_split(TileGemm& p, const Split& s, void* ws, int64_t ws_bytes) {
    if (s.splits > 1 && ws_bytes >= s.bytes) {
        p.splits = s.splits;
        p.ws = static_cast<float*>(ws);
    }
}

template <typename Elt>
int gemm8(int64_t M, int64_t N, int64_t K, const sdt_fp8* A, const sdt_fp8* B, void* C, int64_t ldc, void* ws,
          int64_t ws_bytes, void* stream) {
    if (M < 0 || N < 0 || K < 0 || ws_bytes < 0 || (ws_bytes > 0 && !ws)) return SDT_ERR_INVALID_ARG;
    if (!known_block(A) || !known_block(B) || A->block != 1 || B->block != 128) return SDT_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SDT_OK;
    int rc = check_out(M, N, C, ldc);
    if (rc == SDT_OK && K > 0) rc = check_fp8(M, K, *A);
    if (rc == SDT_OK && K > 0) rc = check_fp8(N, K, *B);
    if (rc != SDT_OK) return rc;
    if (M > kMaxRows || N > kMaxRows || misaligned(ws, 16)) return SDT_ERR_UNSUPPORTED;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != SDT_OK) return rc;
    TileGemm p = product(M, N, K, 1, dev.nxcd);
    p.A[0] = static_cast<const uint8_t*>(A->q);
    p.B[0] = static_cast<const uint8_t*>(B->q);
    p.SA = A->s;
    p.SB = B->s;
    p.C[0] = static_cast<uint16_t*>(C);
    p.lda[0] = row_bytes(M, A->ldq, 1);
    p.ldb[0] = row_bytes(N, B->ldq, 1);
    p.ldsa = A->lds;
    p.ldsb = B->lds;
    p.ldc[0] = ldc;
    if (few_rows8(M, N, K)) return launch_rows8<Elt>(p, dev.num_cu, stream);
    if (large_tiles(ceil_div(M, 256) * ceil_div(N, 256), ceil_div(M, 128) * ceil_div(N, 128), p.nkt, dev.num_cu,
                    true)) {
        p.gm = (int)ceil_div(M, 256);
        p.gn = (int)ceil_div(N, 256);
        return launch(reinterpret_cast<const void*>(&fp8_pp_kernel<Elt>), (int64_t)p.gm * p.gn, 512, p, stream);
    }
    const Split s = plan_split8(M, N, K);
    take_split(p, s, ws, ws_bytes);
    return s.side == 128 ? launch_tile<Elt, true, 128, 128, 2, 2, 2, false, false, false>(p, stream)
                         : launch_tile<Elt, true, 64, 64, 2, 2, 4, false, false, false>(p, stream);
}

template <typename Elt, bool TA, bool TB>
int launch_split(TileGemm& p, void* ws, int64_t ws_bytes, int num_cu, void* stream) {
    const int64_t kt = (int64_t)p.nkt * p.products;
    const Split s = plan_turned(p.M, p.N, kt, p.batch);
    const bool strides = p.products == 1 || (p.lda[0] == p.lda[1] && p.ldb[0] == p.ldb[1]);
    if (strides && large_tiles(ceil_div(p.M, 256) * ceil_div(p.N, 256) * p.batch,
                               ceil_div(p.M, 128) * ceil_div(p.N, 128) * p.batch, kt, num_cu, false))
        return launch_pp<Elt, TA, TB, false>(p, stream);
    take_split(p, s, ws, ws_bytes);
    return s.side == 128 ? launch_tile<Elt, false, 128, 128, 2, 2, 2, TA, TB, false>(p, stream)
                         : launch_tile<Elt, false, 64, 64, 2, 2, 4, TA, TB, false>(p, stream);
}

// C (M x N) = A . B, A (M x L) or, TA, A^T with A (L x M); B (L x N).
template <typename Elt, bool TA>
int gemm_turned(int64_t M, int64_t N, int64_t L, const void* A, int64_t lda, const void* B, int64_t ldb,
                void* C, int64_t ldc, void* ws, int64_t ws_bytes, void* stream) {
    if (M < 0 || N < 0 || L < 0 || ws_bytes < 0 || (ws_bytes > 0 && !ws)) return SDT_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SDT_OK;
    int rc = check_out(M, N, C, ldc);
    if (rc == SDT_OK && L > 0) rc = TA ? check_in(L, M, A, lda) : check_in(M, L, A, lda);
    if (rc == SDT_OK && L > 0) rc = check_in(L, N, B, ldb);
    if (rc != SDT_OK) return rc;
    if (M > kMaxRows || N > kMaxRows || L > kMaxRows || misaligned(ws, 16)) return SDT_ERR_UNSUPPORTED;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != SDT_OK) return rc;
    TileGemm p = product(M, N, L, 2, dev.nxcd);
    p.A[0] = static_cast<const uint8_t*>(A);
    p.B[0] = static_cast<const uint8_t*>(B);
    p.C[0] = static_cast<uint16_t*>(C);
    p.lda[0] = row_bytes(TA ? L : M, lda, 2);
    p.ldb[0] = row_bytes(L, ldb, 2);
    p.ldc[0] = ldc;
    return launch_split<Elt, TA, true>(p, ws, ws_bytes, dev.num_cu, stream);
}

// ---- the norm ---------------------------------------------------------------------------

// Threads and chunks of a row of K: one wave up to 512 elements.
template <template <typename, int, int> class K, typename Elt>
const void* norm_kernel(int64_t n, int* threads) {
    if (n <= 512) return *threads = 64, K<Elt, 64, 1>::get();
    if (n <= 1024) return *threads = 128, K<Elt, 128, 1>::get();
    if (n <= 2048) return *threads = 256, K<Elt, 256, 1>::get();
    if (n <= 4096) return *threads = 256, K<Elt, 256, 2>::get();
    if (n <= 8192) return *threads = 512, K<Elt, 512, 2>::get();
    if (n <= 16384) return *threads = 1024, K<Elt, 1024, 2>::get();
    return *threads = 1024, K<Elt, 1024, 4>::get();
}
template <typename Elt, int T, int CH>
struct Forward {
    static const void* get() { return reinterpret_cast<const void*>(&rms_norm_kernel<Elt, T, CH>); }
};
template <typename Elt, int T, int CH>
struct Backward {
    static const void* get() { return reinterpret_cast<const void*>(&rms_norm_backward_kernel<Elt, T, CH>); }
};

// A 16-bit matrix of the norm: any alignment of its elements.
int check_rows(int64_t K, const void* X, int64_t ld, bool needed) {
    if (!X) return needed ? SDT_ERR_INVALID_ARG : SDT_OK;
    if (ld < K) return SDT_ERR_INVALID_ARG;
    return misaligned(X, 2) ? SDT_ERR_UNSUPPORTED : SDT_OK;
}

template <typename Elt>
int norm(const sdt_norm* a, void* stream) {
    if (!a || a->rows < 0 || a->K < 0 || !std::isfinite(a->eps) || a->eps < 0.0f) return SDT_ERR_INVALID_ARG;
    if (a->rows == 0 || a->K == 0) return SDT_OK;
    if (!a->total && !a->y && !a->q && !a->rstd) return SDT_ERR_INVALID_ARG;
    int rc = check_rows(a->K, a->x, a->ldx, true);
    if (rc == SDT_OK) rc = check_rows(a->K, a->residual, a->ldr, false);
    if (rc == SDT_OK) rc = check_rows(a->K, a->weight, a->K, false);
    if (rc == SDT_OK) rc = check_rows(a->K, a->total, a->ldt, false);
    if (rc == SDT_OK) rc = check_rows(a->K, a->y, a->ldy, false);
    if (rc == SDT_OK && a->q) rc = check_fp8(a->rows, a->K, sdt_fp8{a->q, a->ldq, a->s, a->lds, 1});
    if (rc != SDT_OK) return rc;
    if (misaligned(a->rstd, 4) || a->K > kMaxNorm || a->rows > kMaxRows) return SDT_ERR_UNSUPPORTED;
    Norm p = {};
    p.X = static_cast<const uint16_t*>(a->x);
    p.ldx = a->ldx;
    p.R = static_cast<const uint16_t*>(a->residual);
    p.ldr = a->ldr;
    p.W = static_cast<const uint16_t*>(a->weight);
    p.T = static_cast<uint16_t*>(a->total);
    p.ldt = a->ldt;
    p.Y = static_cast<uint16_t*>(a->y);
    p.ldy = a->ldy;
    p.Q = static_cast<uint8_t*>(a->q);
    p.ldq = a->ldq;
    p.S = a->s;
    p.lds = a->lds;
    p.rstd = a->rstd;
    p.rows = a->rows;
    p.K = (int)a->K;
    p.eps = a->eps;
    int threads;
    const void* k = norm_kernel<Forward, Elt>(a->K, &threads);
    return threads == 64 ? launch(k, ceil_div(a->rows, 4), 256, p, stream)
                         : launch(k, a->rows, threads, p, stream);
}

// Workgroups of the gradient, each of which keeps the weight's gradient of its rows:
// two of 256 threads a CU.  (1024 of them: 16384 x 1024 36.5 us against 39.4, 8192 x 2048
// 37.5 against 32.1.)
int64_t norm_parts(int64_t rows, int64_t K) {
    return std::min<int64_t>(K <= 512 ? ceil_div(rows, 4) : rows, 512);
}

template <typename Elt>
int norm_backward(const sdt_norm_grad* a, void* stream) {
    if (!a || a->rows < 0 || a->K < 0) return SDT_ERR_INVALID_ARG;
    if (a->K == 0) return SDT_OK;
    if (a->rows == 0 && !a->dweight) return SDT_OK;
    if (misaligned(a->dweight, 4) || a->K > kMaxNorm || a->rows > kMaxRows) return SDT_ERR_UNSUPPORTED;
    Norm p = {};
    p.rows = a->rows;
    p.K = (int)a->K;
    const int64_t parts = norm_parts(a->rows, a->K);
    if (a->rows > 0) {
        int rc = check_rows(a->K, a->total, a->ldt, true);
        if (rc == SDT_OK) rc = check_rows(a->K, a->weight, a->K, false);
        if (rc == SDT_OK) rc = check_rows(a->K, a->dy, a->lddy, true);
        if (rc == SDT_OK) rc = check_rows(a->K, a->dtotal, a->lddt, false);
        if (rc == SDT_OK) rc = check_rows(a->K, a->dx, a->lddx, true);
        if (rc != SDT_OK) return rc;
        if (!a->rstd) return SDT_ERR_INVALID_ARG;
        if (a->dweight && (!a->workspace || a->workspace_bytes < parts * a->K * 4)) return SDT_ERR_INVALID_ARG;
        if (misaligned(a->rstd, 4) || (a->dweight && misaligned(a->workspace, 16))) return SDT_ERR_UNSUPPORTED;
        p.X = static_cast<const uint16_t*>(a->total);
        p.ldx = a->ldt;
        p.W = static_cast<const uint16_t*>(a->weight);
        p.rstd_in = a->rstd;
        p.DY = static_cast<const uint16_t*>(a->dy);
        p.lddy = a->lddy;
        p.DT = static_cast<const uint16_t*>(a->dtotal);
        p.lddt = a->lddt;
        p.DX = static_cast<uint16_t*>(a->dx);
        p.lddx = a->lddx;
        p.dw_part = a->dweight ? static_cast<float*>(a->workspace) : nullptr;
        int threads;
        const void* k = norm_kernel<Backward, Elt>(a->K, &threads);
        rc = launch(k, parts, threads == 64 ? 256 : threads, p, stream);
        if (rc != SDT_OK) return rc;
    }
    if (!a->dweight) return SDT_OK;
    ColumnSum c;                                  // no rows: no parts, zeros
    c.part = static_cast<const float*>(a->workspace);
    c.out = a->dweight;
    c.parts = (int)parts;
    c.K = (int)a->K;
    return launch(reinterpret_cast<const void*>(&column_sum_kernel), ceil_div(a->K, 64), 1024, c, stream);
}

// ---- the gated block ----------------------------------------------------------------------

// Both factors, kept for the gradients: fp32 or 16 bits.
int check_factors(int64_t M, int64_t N, const void* g, int64_t ldg, const void* u, int64_t ldu, int wide) {
    if ((wide | 1) != 1) return SDT_ERR_INVALID_ARG;
    if (!g || !u || ldg < N || ldu < N) return SDT_ERR_INVALID_ARG;
    const int unit = wide ? 4 : 8;
    if (misaligned(g, 16) || misaligned(u, 16)) return SDT_ERR_UNSUPPORTED;
    return M > 1 && (ldg % unit != 0 || ldu % unit != 0) ? SDT_ERR_UNSUPPORTED : SDT_OK;
}

template <typename Elt>
int gated(const sdt_gated_ff* a, void* stream) {
    if (!a || a->M < 0 || a->N < 0 || a->K < 0 || (a->act | 1) != 1) return SDT_ERR_INVALID_ARG;
    if (a->M == 0 || a->N == 0) return SDT_OK;
    const int64_t M = a->M, N = a->N, K = a->K;
    int rc = check_out(M, N, a->h, a->ldh);
    if (rc == SDT_OK && K > 0) rc = check_in(M, K, a->x, a->ldx);
    if (rc == SDT_OK && K > 0) rc = check_in(N, K, a->gate, a->ldgate);
    if (rc == SDT_OK && K > 0) rc = check_in(N, K, a->up, a->ldup);
    if (rc == SDT_OK && (a->g || a->u)) rc = check_factors(M, N, a->g, a->ldg, a->u, a->ldu, a->wide);
    if (rc != SDT_OK) return rc;
    if (a->workspace_bytes < 0 || (a->workspace_bytes > 0 && !a->workspace)) return SDT_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxRows || K > kMaxK || misaligned(a->workspace, 16)) return SDT_ERR_UNSUPPORTED;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != SDT_OK) return rc;
    TileGemm p = product(M, N, K, 2, dev.nxcd);
    p.A[0] = static_cast<const uint8_t*>(a->x);
    p.B[0] = static_cast<const uint8_t*>(a->gate);
    p.B[1] = static_cast<const uint8_t*>(a->up);
    p.C[0] = static_cast<uint16_t*>(a->h);
    p.lda[0] = row_bytes(M, a->ldx, 2);
    p.ldb[0] = row_bytes(N, a->ldgate, 2);
    p.ldb[1] = row_bytes(N, a->ldup, 2);
    p.ldc[0] = a->ldh;
    p.G = a->g;
    p.U = a->u;
    p.ldg = a->ldg;
    p.ldu = a->ldu;
    p.wide = a->wide;
    p.act = a->act;
    if (M <= kFewRows) return launch_rows<Elt, false, true, 4, 1, 1, 4>(p, stream);
    if (large_tiles(ceil_div(M, 256) * ceil_div(N, 128), ceil_div(M, 128) * ceil_div(N, 64), p.nkt, dev.num_cu,
                    false))
        return launch_pp<Elt, false, false, true>(p, stream);
    const Split s = plan_gated(M, N, K);
    take_split(p, s, a->workspace, a->workspace_bytes);
    return s.side == 128 ? launch_tile<Elt, false, 128, 128, 2, 2, 2, false, false, true>(p, stream)
                         : launch_tile<Elt, false, 64, 128, 2, 2, 3, false, false, true>(p, stream);
}

// The backward's buffer: dg and du side by side (rows of 2 N' elements), then the
// splits' sums of the product that needs most.
struct GatedLayout {
    int64_t ld, at, bytes;                        // elements of a row; the sums' offset; -1: more
                                                  // than operands may have
};
GatedLayout gated_layout(int64_t M, int64_t N, int64_t K) {
    GatedLayout l;
    const int64_t np = ceil_div(N, 8) * 8;
    l.ld = 2 * np;
    l.at = l.bytes = 0;
    if (M == 0 || N == 0 || K == 0) return l;     // no buffer is used
    if (M > kMaxRows || l.ld >= kMaxStride || K >= kMaxStride) {
        l.bytes = -1;
        return l;
    }
    l.at = ceil_div(M * l.ld * 2, 256) * 256;
    l.bytes = l.at + std::max(plan_turned(M, K, 2 * ceil_div(N, 64), 1).bytes,
                              plan_turned(N, K, ceil_div(M, 64), 2).bytes);
    return l;
}

template <typename Elt>
int gated_backward(const sdt_gated_ff_grad* a, void* stream) {
    if (!a || a->M < 0 || a->N < 0 || a->K < 0 || (a->act | 1) != 1) return SDT_ERR_INVALID_ARG;
    const int64_t M = a->M, N = a->N, K = a->K;
    if (!a->dx && !a->dgate && !a->dup) return SDT_ERR_INVALID_ARG;
    if ((a->dgate == nullptr) != (a->dup == nullptr)) return SDT_ERR_INVALID_ARG;
    if (K == 0 || (M == 0 && N == 0)) return SDT_OK;
    int rc = SDT_OK;
    const bool input = a->dx && M > 0, weights = a->dgate && N > 0;
    if (input) rc = check_out(M, K, a->dx, a->lddx);
    if (rc == SDT_OK && weights) rc = check_out(N, K, a->dgate, a->lddgate);
    if (rc == SDT_OK && weights) rc = check_out(N, K, a->dup, a->lddup);
    if (rc != SDT_OK) return rc;
    const GatedLayout l = gated_layout(M, N, K);
    if (M > 0 && N > 0) {
        if (weights) rc = check_in(M, K, a->x, a->ldx);
        if (rc == SDT_OK && input) rc = check_in(N, K, a->gate, a->ldgate);
        if (rc == SDT_OK && input) rc = check_in(N, K, a->up, a->ldup);
        if (rc == SDT_OK) rc = check_factors(M, N, a->g, a->ldg, a->u, a->ldu, a->wide);
        if (rc == SDT_OK) rc = check_rows(N, a->dh, a->lddh, true);
        if (rc != SDT_OK) return rc;
        if (l.bytes < 0) return SDT_ERR_UNSUPPORTED;
        if (!a->workspace || a->workspace_bytes < l.bytes) return SDT_ERR_INVALID_ARG;
        if (misaligned(a->workspace, 16)) return SDT_ERR_UNSUPPORTED;
    }
    if (M > kMaxRows || N > kMaxRows || K > kMaxRows) return SDT_ERR_UNSUPPORTED;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != SDT_OK) return rc;
    uint16_t* const dg = static_cast<uint16_t*>(a->workspace);
    uint16_t* const du = dg ? dg + l.ld / 2 : nullptr;
    char* const ws = dg ? static_cast<char*>(a->workspace) + l.at : nullptr;
    if (M > 0 && N > 0) {
        GatedGrad p;
        p.G = a->g;
        p.U = a->u;
        p.ldg = a->ldg;
        p.ldu = a->ldu;
        p.DH = static_cast<const uint16_t*>(a->dh);
        p.lddh = a->lddh;
        p.DG = dg;
        p.DU = du;
        p.ldd = l.ld;
        p.M = M;
        p.N = (int)N;
        p.nct = (int)ceil_div(N, 2048);
        p.wide = a->wide;
        p.act = a->act;
        rc = many_short(M, N, 256, dev.num_cu)
                 ? launch(reinterpret_cast<const void*>(&gated_grad_kernel<Elt, 4>), ceil_div(M, 4) * p.nct, 256,
                          p, stream)
                 : launch(reinterpret_cast<const void*>(&gated_grad_kernel<Elt, 1>), M * p.nct, 256, p, stream);
        if (rc != SDT_OK) return rc;
    }
    if (input) {                                  // dx = dg . gate + du . up
        TileGemm p = product(M, K, N, 2, dev.nxcd);
        p.A[0] = reinterpret_cast<const uint8_t*>(dg);
        p.A[1] = reinterpret_cast<const uint8_t*>(du);
        p.B[0] = static_cast<const uint8_t*>(a->gate);
        p.B[1] = static_cast<const uint8_t*>(a->up);
        p.C[0] = static_cast<uint16_t*>(a->dx);
        p.lda[0] = p.lda[1] = l.ld * 2;
        p.ldb[0] = row_bytes(N, a->ldgate, 2);
        p.ldb[1] = row_bytes(N, a->ldup, 2);
        p.ldc[0] = a->lddx;
        p.products = 2;
        rc = launch_split<Elt, false, true>(p, ws, l.bytes - l.at, dev.num_cu, stream);
        if (rc != SDT_OK) return rc;
    }
    if (weights) {                                // dgate = dg^T . x, dup = du^T . x
        TileGemm p = product(N, K, M, 2, dev.nxcd);
        p.A[0] = reinterpret_cast<const uint8_t*>(dg);
        p.A[1] = reinterpret_cast<const uint8_t*>(du);
        p.B[0] = p.B[1] = static_cast<const uint8_t*>(a->x);
        p.C[0] = static_cast<uint16_t*>(a->dgate);
        p.C[1] = static_cast<uint16_t*>(a->dup);
        p.lda[0] = p.lda[1] = l.ld * 2;
        p.ldb[0] = p.ldb[1] = row_bytes(M, a->ldx, 2);
        p.ldc[0] = a->lddgate;
        p.ldc[1] = a->lddup;
        p.batch = 2;
        rc = launch_split<Elt, true, true>(p, ws, l.bytes - l.at, dev.num_cu, stream);
    }
    return rc;
}

}  // namespace
}  // namespace sdt

using sdt::BF16;
using sdt::F16;

extern "C" {

int fp8_quantize_f16(int64_t rows, int64_t K, const void* X, int64_t ldx, const sdt_fp8* out, void* stream) {
    return sdt::quantize8<F16>(rows, K, X, ldx, out, stream);
}
int fp8_quantize_bf16(int64_t rows, int64_t K, const void* X, int64_t ldx, const sdt_fp8* out, void* stream) {
    return sdt::quantize8<BF16>(rows, K, X, ldx, out, stream);
}
int fp8_dequantize_f16(int64_t rows, int64_t K, const sdt_fp8* m, void* Y, int64_t ldy, void* stream) {
    return sdt::dequantize8<F16>(rows, K, m, Y, ldy, stream);
}
int fp8_dequantize_bf16(int64_t rows, int64_t K, const sdt_fp8* m, void* Y, int64_t ldy, void* stream) {
    return sdt::dequantize8<BF16>(rows, K, m, Y, ldy, stream);
}
int fp8_dequantize_f32(int64_t rows, int64_t K, const sdt_fp8* m, void* Y, int64_t ldy, void* stream) {
    return sdt::dequantize8<float>(rows, K, m, Y, ldy, stream);
}
int gemm_fp8_f16(int64_t M, int64_t N, int64_t K, const sdt_fp8* A, const sdt_fp8* B, void* C, int64_t ldc,
                 void* workspace, int64_t workspace_bytes, void* stream) {
    return sdt::gemm8<F16>(M, N, K, A, B, C, ldc, workspace, workspace_bytes, stream);
}
int gemm_fp8_bf16(int64_t M, int64_t N, int64_t K, const sdt_fp8* A, const sdt_fp8* B, void* C, int64_t ldc,
                 void* workspace, int64_t workspace_bytes, void* stream) {
    return sdt::gemm8<BF16>(M, N, K, A, B, C, ldc, workspace, workspace_bytes, stream);
}
int64_t sdt_gemm_fp8_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || M > sdt::kMaxRows || N > sdt::kMaxRows || K > sdt::kMaxK) return -1;
    if (M > 0 && N > 0 && K >= 2 * sdt::kMaxStride) return -1;
    return sdt::few_rows8(M, N, K) ? 0 : sdt::plan_split8(M, N, K).bytes;
}

int rms_norm_f16(const sdt_norm* args, void* stream) { return sdt::norm<F16>(args, stream); }
int rms_norm_bf16(const sdt_norm* args, void* stream) { return sdt::norm<BF16>(args, stream); }
int rms_norm_backward_f16(const sdt_norm_grad* args, void* stream) {
    return sdt::norm_backward<F16>(args, stream);
}
int rms_norm_backward_bf16(const sdt_norm_grad* args, void* stream) {
    return sdt::norm_backward<BF16>(args, stream);
}
int64_t sdt_rms_norm_workspace_size(int64_t rows, int64_t K) {
    if (rows < 0 || K < 0 || rows > sdt::kMaxRows || K > sdt::kMaxNorm) return -1;
    return sdt::norm_parts(rows, K) * K * 4;
}

int gated_ff_f16(const sdt_gated_ff* args, void* stream) { return sdt::gated<F16>(args, stream); }
int gated_ff_bf16(const sdt_gated_ff* args, void* stream) { return sdt::gated<BF16>(args, stream); }
int64_t sdt_gated_ff_split_size(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || M > sdt::kMaxRows || N > sdt::kMaxRows || K > sdt::kMaxK) return -1;
    if (M > 0 && N > 0 && K >= sdt::kMaxStride) return -1;
    return M <= sdt::kFewRows ? 0 : sdt::plan_gated(M, N, K).bytes;
}
int gated_ff_backward_f16(const sdt_gated_ff_grad* args, void* stream) {
    return sdt::gated_backward<F16>(args, stream);
}
int gated_ff_backward_bf16(const sdt_gated_ff_grad* args, void* stream) {
    return sdt::gated_backward<BF16>(args, stream);
}
int64_t sdt_gated_ff_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || M > sdt::kMaxRows || N > sdt::kMaxRows || K > sdt::kMaxRows) return -1;
    return sdt::gated_layout(M, N, K).bytes;
}

int gemm_f16_nn(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb,
                void* C, int64_t ldc, void* workspace, int64_t workspace_bytes, void* stream) {
    return sdt::gemm_turned<F16, false>(M, N, K, A, lda, B, ldb, C, ldc, workspace, workspace_bytes, stream);
}
int gemm_bf16_nn(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb,
                 void* C, int64_t ldc, void* workspace, int64_t workspace_bytes, void* stream) {
    return sdt::gemm_turned<BF16, false>(M, N, K, A, lda, B, ldb, C, ldc, workspace, workspace_bytes, stream);
}
int gemm_f16_tn(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb,
                void* C, int64_t ldc, void* workspace, int64_t workspace_bytes, void* stream) {
    return sdt::gemm_turned<F16, true>(M, N, K, A, lda, B, ldb, C, ldc, workspace, workspace_bytes, stream);
}
int gemm_bf16_tn(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* B, int64_t ldb,
                 void* C, int64_t ldc, void* workspace, int64_t workspace_bytes, void* stream) {
    return sdt::gemm_turned<BF16, true>(M, N, K, A, lda, B, ldb, C, ldc, workspace, workspace_bytes, stream);
}
int64_t sdt_gemm_turned_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || M > sdt::kMaxRows || N > sdt::kMaxRows || K > sdt::kMaxRows) return -1;
    // one layout's operands at least have to be such: B's rows are N long, A's K or M
    if (M > 0 && K > 0 && (N >= sdt::kMaxStride || (M >= sdt::kMaxStride && K >= sdt::kMaxStride))) return -1;
    return sdt::plan_turned(M, N, sdt::ceil_div(K, 64), 1).bytes;
}

}  // extern "C"
