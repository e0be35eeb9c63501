// C ABI of the MX4 and expert entry points (declared in sdt.h): argument
// checks on the host, the choice of a kernel, the launch.  Allocates nothing.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "launcher.hpp"
#include "moe_kernel.hpp"
#include "mx4_kernel.hpp"
#include "mx4_pp_kernel.hpp"
#include "runtime.hpp"
#include "sdt.h"

namespace sdt {
namespace {

constexpr int64_t kMaxK = int64_t(1) << 23;
constexpr int64_t kMaxLd = (int64_t(1) << 22) + 16;   // bytes, exclusive
constexpr int64_t kMaxRows = INT_MAX - 255;           // the last tile's end fits 32 bits

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int64_t row_bytes(int64_t K) { return ceil_div(K, 32) * 16; }
int64_t k_tiles(int64_t K) { return ceil_div(K, 256); }

int launched(hipError_t e) { return e == hipSuccess ? SDT_OK : fail_hip(e); }

template <typename P>
int launch(const void* kernel, int64_t grid, int threads, P& params, void* stream) {
    if (grid > INT_MAX) return SDT_ERR_UNSUPPORTED;
    void* args[] = {&params};
    return launched(hipLaunchKernel(kernel, dim3((unsigned)grid), dim3((unsigned)threads), args, 0,
                                    static_cast<hipStream_t>(stream)));
}

// An MX4 matrix's arguments (rows, K >= 0 checked by the caller).
int check_mx4(int64_t rows, int64_t K, const void* Q, int64_t ldq, const void* S) {
    if (rows == 0 || K == 0) return SDT_OK;
    if (!Q || !S) return SDT_ERR_INVALID_ARG;
    if (ldq < row_bytes(K)) return SDT_ERR_INVALID_ARG;
    if (K > kMaxK || rows > kMaxRows || ldq >= kMaxLd) return SDT_ERR_UNSUPPORTED;
    if (misaligned(Q, 16) || misaligned(S, 16) || ldq % 16 != 0) return SDT_ERR_UNSUPPORTED;
    return SDT_OK;
}

int check_out(int64_t rows, int64_t N, const void* C, int64_t ldc) {
    if (!C || ldc < N) return SDT_ERR_INVALID_ARG;
    if (misaligned(C, 16) || (rows > 1 && ldc % 8 != 0)) return SDT_ERR_UNSUPPORTED;
    return SDT_OK;
}

// 16-bit rows x K of 64 MB or more: twice the L2 caches' 32.
bool past_caches(int64_t rows, int64_t K) { return rows * K >= int64_t(1) << 25; }

template <typename Elt>
int quantize(int64_t rows, int64_t K, const void* X, int64_t xrows, int64_t ldx,
             const int32_t* index, int divisor, void* Q, int64_t ldq, void* S, void* stream) {
    if (rows < 0 || K < 0 || xrows < 0 || divisor < 0) return SDT_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return SDT_OK;
    if (ldx < K || (!X && xrows > 0)) return SDT_ERR_INVALID_ARG;
    int rc = check_mx4(rows, K, Q, ldq, S);
    if (rc != SDT_OK) return rc;
    if (misaligned(X, 2) || misaligned(index, 4)) return SDT_ERR_UNSUPPORTED;
    Mx4Quant p;
    p.X = static_cast<const uint16_t*>(X);
    p.ldx = ldx;
    p.index = index;
    p.divisor = divisor;
    p.xrows = xrows;
    p.Q = static_cast<uint8_t*>(Q);
    p.ldq = ldq;
    p.S = static_cast<uint8_t*>(S);
    p.rows = rows;
    p.K = (int)K;
    p.nkt = (int)k_tiles(K);
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != SDT_OK) return rc;
    const bool large = past_caches(rows, K);
    p.nxcd = large ? dev.nxcd : 1;
    return launch(large ? reinterpret_cast<const void*>(&mx4_quantize_kernel<Elt, true>)
                        : reinterpret_cast<const void*>(&mx4_quantize_kernel<Elt, false>),
                  ceil_div(rows, 64) * p.nkt, 256, p, stream);
}

template <int OUT>
int dequantize(int64_t rows, int64_t K, const void* Q, int64_t ldq, const void* S, void* Y,
               int64_t ldy, void* stream) {
    if (rows < 0 || K < 0) return SDT_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return SDT_OK;
    if (!Y || ldy < K) return SDT_ERR_INVALID_ARG;
    int rc = check_mx4(rows, K, Q, ldq, S);
    if (rc != SDT_OK) return rc;
    constexpr int z = OUT == 2 ? 4 : 2;
    if (misaligned(Y, z)) return SDT_ERR_UNSUPPORTED;
    Mx4Dequant p;
    p.Q = static_cast<const uint8_t*>(Q);
    p.ldq = ldq;
    p.S = static_cast<const uint8_t*>(S);
    p.Y = Y;
    p.ldy = ldy;
    p.rows = rows;
    p.K = (int)K;
    p.nkt = (int)k_tiles(K);
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != SDT_OK) return rc;
    p.nxcd = past_caches(rows, K) ? dev.nxcd : 1;
    return launch(reinterpret_cast<const void*>(&mx4_dequantize_kernel<OUT>),
                  ceil_div(rows, 64) * p.nkt, 256, p, stream);
}

// ---- products -----------------------------------------------------------------------

// Two workgroups a CU take the tiles in turn; one per tile on k-loops too short
// for that (the loads would run more than a tile ahead).  row_tiles: of a plan,
// as many as any choice of experts can give.
template <typename Elt, int BM, int BN, int WM, int WN, int NS, bool GROUPED, bool GATED,
          bool QOUT = false>
int launch_tile(Mx4Gemm p, int64_t row_tiles, int num_cu, void* stream) {
    p.gm = (int)row_tiles;
    p.gn = (int)ceil_div(p.N, GATED ? BN / 2 : BN);
    const int64_t tiles = row_tiles * p.gn;
    if (tiles > INT_MAX) return SDT_ERR_UNSUPPORTED;
    const int64_t grid = p.nkt > NS || p.nkt == 0 ? std::min<int64_t>(tiles, 2 * num_cu) : tiles;
    return launch(
        reinterpret_cast<const void*>(&mx4_gemm_kernel<Elt, BM, BN, WM, WN, NS, GROUPED, GATED, QOUT>),
        grid, WM * WN * 64, p, stream);
}

// Waves that split the k-tiles: two where the workgroups outnumber the CUs (two of
// them share one: 64 tokens of 32 experts, 50 -> 45 and 35 -> 28 us against four),
// four where not (64 x 4096 x 4096, 64 workgroups: 7.5 us against 9.0 with two).  64
// columns a workgroup at any N: 12288 gives 192 workgroups and leaves 64 CUs idle.
template <typename Elt, bool GROUPED, bool GATED, bool QOUT = false>
int launch_skinny(Mx4Gemm p, int64_t groups, int num_cu, void* stream) {
    p.gm = (int)groups;
    p.gn = (int)ceil_div(p.N, GATED ? 32 : 64);
    const int64_t grid = (int64_t)p.gm * p.gn;
    if (grid > num_cu)
        return launch(reinterpret_cast<const void*>(&mx4_skinny_kernel<Elt, GROUPED, GATED, QOUT, 2>),
                      grid, 2 * 64, p, stream);
    return launch(reinterpret_cast<const void*>(&mx4_skinny_kernel<Elt, GROUPED, GATED, QOUT, 4>), grid,
                  4 * 64, p, stream);
}

// Which kernel a product runs, from the number of output tiles of each against
// the CUs (us measured on MI355X, K = 4096 where not named):
//   few rows (M <= 64, or <= 128 with at most one 64 x 64 tile a CU): the weights
//   are streamed (100x4096: 8.3 against 9.8 with 64 x 64 tiles; 256x4096: 10.4
//   against 9.4);
//   at most one 64 x 64 tile a CU: those (1024^3: 4.9, with 128 x 128 6.3);
//   at most one 64 x 128 tile a CU: those (512x4096: 11.6, with 64 x 64 12.1, with
//   128 x 128 14.1; just past it, 256x12288: 15.6 against 14.6);
//   else 128 x 128, two workgroups a CU in turn, or 256 x 256, one, by the estimate
//   below.
// A CU's time: a round of 256 x 256 tiles that fills the chip takes 1.7 us a
// k-tile and 7.5 besides, one that does not 1.25 a k-tile; a 128 x 128 tile 0.58
// and 1.6, and 3 once.  2560x4096: 27.9 (256) against 32.5 (128); 4096x5120: 57.9
// against 51.7; 1024x8192x8192: 46.3 against 40.0; 6000x6000x500: 44.5 against
// 27.9; 4096x4096x1024: 15.9 against 18.3; 8192^3: 246 against 301.
bool large_tiles_win(int64_t M, int64_t N, int64_t nkt, int64_t cu) {
    const int64_t t256 = ceil_div(M, 256) * ceil_div(N, 256);
    const int64_t t128 = ceil_div(M, 128) * ceil_div(N, 128);
    const double k = (double)nkt;
    const double large = (double)(t256 / cu) * (1.7 * k + 7.5) + (t256 % cu ? 1.25 * k + 7.5 : 0.0);
    const double small = (double)t128 / (double)cu * (0.58 * k + 1.6) + 3.0;
    return t128 > cu && large < small;
}

template <typename Elt>
int gemm(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, const void* SA, const void* B,
         int64_t ldb, const void* SB, void* C, int64_t ldc, void* stream) {
    if (M < 0 || N < 0 || K < 0) return SDT_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return SDT_OK;
    int rc = check_out(M, N, C, ldc);
    if (rc == SDT_OK) rc = check_mx4(M, K, A, lda, SA);
    if (rc == SDT_OK) rc = check_mx4(N, K, B, ldb, SB);
    if (rc != SDT_OK) return rc;
    if (M > kMaxRows || N > kMaxRows) return SDT_ERR_UNSUPPORTED;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != SDT_OK) return rc;
    Mx4Gemm p = {};
    p.A = static_cast<const uint8_t*>(A);
    p.SA = static_cast<const uint8_t*>(SA);
    p.B = static_cast<const uint8_t*>(B);
    p.SB = static_cast<const uint8_t*>(SB);
    p.C = static_cast<uint16_t*>(C);
    p.lda = (uint32_t)lda;
    p.ldb = (uint32_t)ldb;
    p.ldc = ldc;
    p.M = (int)M;
    p.N = (int)N;
    p.rowbytes = (int)row_bytes(K);
    p.nkt = (int)k_tiles(K);
    p.nxcd = dev.nxcd;
    const int64_t cu = dev.num_cu;
    const int64_t t64 = ceil_div(M, 64) * ceil_div(N, 64);
    if (M <= 64 || (M <= 128 && t64 <= cu))
        return launch_skinny<Elt, false, false>(p, ceil_div(M, 64), dev.num_cu, stream);
    if (large_tiles_win(M, N, p.nkt, cu)) {
        p.gm = (int)ceil_div(M, 256);
        p.gn = (int)ceil_div(N, 256);
        return launch(reinterpret_cast<const void*>(&mx4_pp_kernel<Elt>), (int64_t)p.gm * p.gn, 512,
                      p, stream);
    }
    if (t64 <= cu)
        return launch_tile<Elt, 64, 64, 2, 2, 4, false, false>(p, ceil_div(M, 64), dev.num_cu, stream);
    if (ceil_div(M, 64) * ceil_div(N, 128) <= cu)
        return launch_tile<Elt, 64, 128, 2, 2, 3, false, false>(p, ceil_div(M, 64), dev.num_cu, stream);
    return launch_tile<Elt, 128, 128, 2, 2, 2, false, false>(p, ceil_div(M, 128), dev.num_cu, stream);
}

template <typename Elt>
int gemv(int64_t N, int64_t K, const void* x, const void* B, int64_t ldb, const void* SB, void* y,
         void* stream) {
    if (N < 0 || K < 0) return SDT_ERR_INVALID_ARG;
    if (N == 0) return SDT_OK;
    if (!y || (!x && K > 0)) return SDT_ERR_INVALID_ARG;
    int rc = check_mx4(N, K, B, ldb, SB);
    if (rc != SDT_OK) return rc;
    if (N > kMaxRows || misaligned(x, 2) || misaligned(y, 2)) return SDT_ERR_UNSUPPORTED;
    Mx4Gemv p;
    p.x = static_cast<const uint16_t*>(x);
    p.B = static_cast<const uint8_t*>(B);
    p.ldb = ldb;
    p.SB = static_cast<const uint8_t*>(SB);
    p.y = static_cast<uint16_t*>(y);
    p.N = (int)N;
    p.K = (int)K;
    p.rowbytes = (int)row_bytes(K);
    p.nkt = (int)k_tiles(K);
    const void* k = K <= 4096 ? reinterpret_cast<const void*>(&mx4_gemv_kernel<Elt, 8, 2, 4096>)
                              : reinterpret_cast<const void*>(&mx4_gemv_kernel<Elt, 8, 3, 8192>);
    return launch(k, ceil_div(N, 16), 8 * 64, p, stream);
}

// ---- experts ---------------------------------------------------------------------------

int check_route(int64_t T, int64_t E, const void* logits, int64_t ld, const sdt_route* c,
                const void* idx, const void* w, int z) {
    if (!c || T < 0 || E < 1 || ld < E) return SDT_ERR_INVALID_ARG;
    if (c->groups < 1 || E % c->groups != 0 || c->groups_kept < 1 || c->groups_kept > c->groups)
        return SDT_ERR_INVALID_ARG;
    const int64_t per = E / c->groups;
    if (c->topk < 1 || c->topk > std::min<int64_t>(kMaxTopk, c->groups_kept * per))
        return SDT_ERR_INVALID_ARG;
    if ((c->group_top != 1 && c->group_top != 2) || c->group_top > per) return SDT_ERR_INVALID_ARG;
    if ((c->score | 1) != 1 || (c->renormalize | 1) != 1 || !std::isfinite(c->scale))
        return SDT_ERR_INVALID_ARG;
    if (E > kMaxExperts || c->groups > kMaxGroups || T > INT_MAX) return SDT_ERR_UNSUPPORTED;
    if (T == 0) return SDT_OK;
    if (!logits || !idx || !w) return SDT_ERR_INVALID_ARG;
    if (misaligned(logits, z) || misaligned(idx, 4) || misaligned(w, 4)) return SDT_ERR_UNSUPPORTED;
    return SDT_OK;
}

RouteParams route_params(int64_t T, int64_t E, const void* logits, int64_t ld, const sdt_route* c) {
    RouteParams p = {};
    p.logits = logits;
    p.ld = ld;
    p.T = T;
    p.E = (int)E;
    p.topk = c->topk;
    p.score = c->score;
    p.groups = c->groups;
    p.kept = c->groups_kept;
    p.group_top = c->groups > 1 ? c->group_top : 1;
    p.renormalize = c->renormalize;
    p.scale = c->scale;
    return p;
}

template <typename T, int EPL>
const void* route_kernel(const RouteParams& p, bool backward) {
    if (backward) return reinterpret_cast<const void*>(&moe_route_backward_kernel<T, EPL>);
    return p.bias != nullptr || p.group_top == 2
               ? reinterpret_cast<const void*>(&moe_route_kernel<T, EPL, true>)
               : reinterpret_cast<const void*>(&moe_route_kernel<T, EPL, false>);
}

template <typename T>
int launch_route(RouteParams& p, bool backward, void* stream) {
    const void* k = p.E <= 64    ? route_kernel<T, 1>(p, backward)
                    : p.E <= 128 ? route_kernel<T, 2>(p, backward)
                    : p.E <= 256 ? route_kernel<T, 4>(p, backward)
                    : p.E <= 512 ? route_kernel<T, 8>(p, backward)
                                 : route_kernel<T, 16>(p, backward);
    return launch(k, ceil_div(p.T, 4), 256, p, stream);
}

template <typename T>
int route(int64_t n, int64_t E, const void* logits, int64_t ld, const float* bias,
          const sdt_route* cfg, int32_t* idx, float* weights, void* stream) {
    int rc = check_route(n, E, logits, ld, cfg, idx, weights, sizeof(T));
    if (rc != SDT_OK || n == 0) return rc;
    if (misaligned(bias, 4)) return SDT_ERR_UNSUPPORTED;
    RouteParams p = route_params(n, E, logits, ld, cfg);
    p.bias = bias;
    p.idx = idx;
    p.weights = weights;
    return launch_route<T>(p, false, stream);
}

template <typename T>
int route_backward(int64_t n, int64_t E, const void* logits, int64_t ld, const sdt_route* cfg,
                   const int32_t* idx, const float* dweights, void* dlogits, int64_t ldd,
                   void* stream) {
    int rc = check_route(n, E, logits, ld, cfg, idx, dweights, sizeof(T));
    if (rc == SDT_OK && ldd < E) rc = SDT_ERR_INVALID_ARG;
    if (rc != SDT_OK || n == 0) return rc;
    if (!dlogits) return SDT_ERR_INVALID_ARG;
    if (misaligned(dlogits, sizeof(T))) return SDT_ERR_UNSUPPORTED;
    RouteParams p = route_params(n, E, logits, ld, cfg);
    p.idx = const_cast<int32_t*>(idx);
    p.dweights = dweights;
    p.dlogits = dlogits;
    p.ldd = ldd;
    return launch_route<T>(p, true, stream);
}

// The plan's sizes and arrays; *rows its row count.
int check_plan(const sdt_moe_plan* q, int64_t* rows) {
    if (!q) return SDT_ERR_INVALID_ARG;
    *rows = sdt_moe_plan_rows(q->tokens, q->topk, q->experts);
    if (*rows < 0) return SDT_ERR_INVALID_ARG;
    if (q->experts > kMaxExperts) return SDT_ERR_UNSUPPORTED;
    if (!q->counts || !q->offsets) return SDT_ERR_INVALID_ARG;
    if (q->tokens > 0 && (!q->rows || !q->pos || !q->tiles)) return SDT_ERR_INVALID_ARG;
    if (misaligned(q->counts, 4) || misaligned(q->offsets, 4) || misaligned(q->rows, 4) ||
        misaligned(q->pos, 4) || misaligned(q->tiles, 4))
        return SDT_ERR_UNSUPPORTED;
    return SDT_OK;
}

int check_experts(int64_t N, int64_t K, const sdt_mx4_experts* B) {
    if (!B) return SDT_ERR_INVALID_ARG;
    int rc = check_mx4(N, K, B->q, B->ldq, B->s);
    if (rc != SDT_OK || K == 0) return rc;
    if (B->q_expert < 0 || B->s_expert < 0) return SDT_ERR_INVALID_ARG;
    if (B->q_expert % 16 != 0 || B->s_expert % 16 != 0) return SDT_ERR_UNSUPPORTED;
    return SDT_OK;
}

// Rows an expert where the tokens choose evenly: picks the grouped kernel.
int64_t rows_per_expert(const sdt_moe_plan* plan) {
    return plan->tokens * plan->topk / plan->experts;
}
// Up to these the weights are streamed, up to 64 they meet 64 x 128 tiles, above
// 128 x 128 (layers of 16 experts, 2048 x 1024, us: 8 rows 32.9 streamed and 34.4
// in 64 x 128 tiles, 16 rows 37.2 and 35.0; 64 rows 39.8 and in 128 x 128 40.8, 128
// rows 49.0 and 45.2).  The host does not know the choice: where the tokens reach few
// of many experts this streams weights that tiles would share (256 experts, 256
// tokens of 8: all on eight experts 148 us and 40 in tiles, spread evenly 176 and 191).
constexpr int64_t kSkinnyRows = 12;

template <typename Elt, int BM, int BN, int NS>
int launch_grouped_tile(const Mx4Gemm& p, const sdt_moe_plan* plan, bool gated, int num_cu,
                        void* stream) {
    // every expert's rows end inside a tile at most once
    const int64_t R = plan->tokens * plan->topk;
    const int64_t row_tiles = (R + (BM - 1) * std::min<int64_t>(plan->experts, R)) / BM;
    if (p.QO) return launch_tile<Elt, BM, BN, 2, 2, NS, true, true, true>(p, row_tiles, num_cu, stream);
    if (gated) return launch_tile<Elt, BM, BN, 2, 2, NS, true, true>(p, row_tiles, num_cu, stream);
    return launch_tile<Elt, BM, BN, 2, 2, NS, true, false>(p, row_tiles, num_cu, stream);
}

// The gated product's quantised form, where its codes and scales are wanted.
struct Mx4Out {
    uint8_t* q;
    uint8_t* s;
    int64_t ldq;
};

template <typename Elt>
int moe_gemm(const sdt_moe_plan* plan, int64_t N, int64_t K, const void* A, int64_t lda,
             const void* SA, const sdt_mx4_experts* B, const sdt_mx4_experts* up, void* C,
             int64_t ldc, void* stream, const Mx4Out& out = {}) {
    int64_t rows;
    int rc = check_plan(plan, &rows);
    if (rc != SDT_OK) return rc;
    if (N < 0 || K < 0) return SDT_ERR_INVALID_ARG;
    rc = check_experts(N, K, B);
    if (rc == SDT_OK && up) rc = check_experts(N, K, up);
    if (rc != SDT_OK || rows == 0 || N == 0) return rc;
    if (!out.q) rc = check_out(rows, N, C, ldc);
    if (rc == SDT_OK) rc = check_mx4(rows, K, A, lda, SA);
    if (rc != SDT_OK) return rc;
    if (N > kMaxRows) return SDT_ERR_UNSUPPORTED;
    DeviceInfo dev;
    rc = device_info(&dev);
    if (rc != SDT_OK) return rc;
    Mx4Gemm p = {};
    p.A = static_cast<const uint8_t*>(A);
    p.SA = static_cast<const uint8_t*>(SA);
    p.B = static_cast<const uint8_t*>(B->q);
    p.SB = static_cast<const uint8_t*>(B->s);
    p.C = static_cast<uint16_t*>(C);
    p.lda = (uint32_t)lda;
    p.ldb = (uint32_t)B->ldq;
    p.ldc = ldc;
    p.M = (int)rows;
    p.N = (int)N;
    p.rowbytes = (int)row_bytes(K);
    p.nkt = (int)k_tiles(K);
    p.nxcd = dev.nxcd;
    p.tiles = plan->tiles;
    p.offsets = plan->offsets;
    p.counts = plan->counts;
    p.eqb = B->q_expert;
    p.esb = B->s_expert;
    if (up) {
        p.B2 = static_cast<const uint8_t*>(up->q);
        p.SB2 = static_cast<const uint8_t*>(up->s);
        p.ldb2 = (uint32_t)up->ldq;
        p.eqb2 = up->q_expert;
        p.esb2 = up->s_expert;
    }
    p.experts = plan->experts;
    p.QO = out.q;
    p.SO = out.s;
    p.ldqo = out.ldq;
    p.nkto = (int)k_tiles(N);
    const int64_t per = rows_per_expert(plan);
    if (per <= kSkinnyRows)
        return p.QO ? launch_skinny<Elt, true, true, true>(p, rows / 64, dev.num_cu, stream)
               : up ? launch_skinny<Elt, true, true>(p, rows / 64, dev.num_cu, stream)
                    : launch_skinny<Elt, true, false>(p, rows / 64, dev.num_cu, stream);
    return per <= 64 ? launch_grouped_tile<Elt, 64, 128, 3>(p, plan, up, dev.num_cu, stream)
                     : launch_grouped_tile<Elt, 128, 128, 2>(p, plan, up, dev.num_cu, stream);
}

PlanParams plan_params(const int32_t* idx, const sdt_moe_plan* plan, int64_t rows) {
    PlanParams p;
    p.idx = idx;
    p.counts = plan->counts;
    p.offsets = plan->offsets;
    p.rows = plan->rows;
    p.pos = plan->pos;
    p.tiles = plan->tiles;
    p.R = (int)(plan->tokens * plan->topk);
    p.E = plan->experts;
    p.cap = (int)rows;
    return p;
}

// The plan and its rows of X, quantised.
template <typename Elt>
int plan_and_quantize(const int32_t* idx, const sdt_moe_plan* plan, int64_t rows, int64_t K,
                      const void* X, int64_t ldx, void* Q, int64_t ldq, void* S, void* stream) {
    Mx4QuantTokens p;
    p.X = static_cast<const uint16_t*>(X);
    p.ldx = ldx;
    p.pos = plan->pos;
    p.Q = static_cast<uint8_t*>(Q);
    p.ldq = ldq;
    p.S = static_cast<uint8_t*>(S);
    p.tokens = plan->tokens;
    p.topk = plan->topk;
    p.K = (int)K;
    p.nkt = (int)k_tiles(K);
    const int64_t grid = ceil_div(p.tokens, 16) * p.nkt;
    if (plan->tokens * plan->topk <= kPlanQuantizeSlots) {
        PlanParams q = plan_params(idx, plan, rows);
        void* args[] = {&q, &p};
        return launched(hipLaunchKernel(reinterpret_cast<const void*>(&moe_plan_quantize_kernel<Elt>),
                                        dim3((unsigned)grid), dim3(256), args, 0,
                                        static_cast<hipStream_t>(stream)));
    }
    const int rc = moe_plan(idx, plan, stream);
    if (rc != SDT_OK) return rc;
    if (plan->topk > kMaxTopk)
        return quantize<Elt>(rows, K, X, plan->tokens, ldx, plan->rows, plan->topk, Q, ldq, S, stream);
    return launch(reinterpret_cast<const void*>(&mx4_quantize_tokens_kernel<Elt>), grid, 256, p, stream);
}

template <typename S>
int combine(const sdt_moe_plan* plan, int64_t N, const void* D, int64_t ldd, const float* weights,
            void* Y, int64_t ldy, void* stream) {
    int64_t rows;
    int rc = check_plan(plan, &rows);
    if (rc != SDT_OK) return rc;
    if (N < 0) return SDT_ERR_INVALID_ARG;
    if (plan->tokens == 0 || N == 0) return SDT_OK;
    if (!weights) return SDT_ERR_INVALID_ARG;
    rc = check_out(2, N, D, ldd);
    if (rc == SDT_OK) rc = check_out(plan->tokens, N, Y, ldy);
    if (rc != SDT_OK) return rc;
    if (misaligned(weights, 4) || N > INT_MAX - 8) return SDT_ERR_UNSUPPORTED;
    CombineParams p;
    p.D = static_cast<const uint16_t*>(D);
    p.ldd = ldd;
    p.pos = plan->pos;
    p.weights = weights;
    p.Y = static_cast<uint16_t*>(Y);
    p.ldy = ldy;
    p.T = plan->tokens;
    p.topk = plan->topk;
    p.N = (int)N;
    p.nch = (int)ceil_div(N, 8);
    return launch(reinterpret_cast<const void*>(&moe_combine_kernel<S>),
                  ceil_div(plan->tokens * p.nch, 256), 256, p, stream);
}

// The layer's buffers, one after another, each from a multiple of 256 bytes.
struct LayerLayout {
    int64_t xq, xs, hq, hs, d, bytes;
    int64_t ldx, ldhq, ldd;   // bytes, bytes, elements
};
LayerLayout layer_layout(int64_t rows, int64_t N, int64_t K) {
    LayerLayout l;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += ceil_div(bytes, 256) * 256;
        return here;
    };
    l.ldx = row_bytes(K);
    l.ldhq = row_bytes(N);
    l.ldd = ceil_div(K, 8) * 8;
    l.xq = take(rows * l.ldx);
    l.xs = take(sdt_mx4_scale_bytes(rows, K));
    l.hq = take(rows * l.ldhq);
    l.hs = take(sdt_mx4_scale_bytes(rows, N));
    l.d = take(rows * l.ldd * 2);
    l.bytes = at;
    return l;
}

template <typename Elt>
int moe_layer(const sdt_moe_layer* layer, const int32_t* idx, const float* weights,
              const sdt_moe_plan* plan, const void* X, int64_t ldx, void* Y, int64_t ldy,
              void* workspace, int64_t workspace_bytes, void* stream) {
    typedef std::conditional_t<std::is_same_v<Elt, Mx4F16>, _Float16, __bf16> S;
    int64_t rows;
    int rc = check_plan(plan, &rows);
    if (rc != SDT_OK) return rc;
    if (!layer || layer->N < 0 || layer->K < 0) return SDT_ERR_INVALID_ARG;
    const int64_t N = layer->N, K = layer->K, T = plan->tokens;
    // everything is checked before the first launch
    rc = check_experts(N, K, &layer->gate);
    if (rc == SDT_OK) rc = check_experts(N, K, &layer->up);
    if (rc == SDT_OK) rc = check_experts(K, N, &layer->down);
    if (rc != SDT_OK) return rc;
    if (T == 0) return moe_plan(idx, plan, stream);
    if (!idx || !weights) return SDT_ERR_INVALID_ARG;
    const LayerLayout l = layer_layout(rows, N, K);
    if (K > 0) {
        if (!X || ldx < K) return SDT_ERR_INVALID_ARG;
        rc = check_out(T, K, Y, ldy);
        if (rc != SDT_OK) return rc;
        if (!workspace || workspace_bytes < l.bytes) return SDT_ERR_INVALID_ARG;
        if (misaligned(workspace, 16) || misaligned(X, 2)) return SDT_ERR_UNSUPPORTED;
        if (K > kMaxK || N > kMaxK || l.ldx >= kMaxLd || l.ldhq >= kMaxLd) return SDT_ERR_UNSUPPORTED;
    }
    if (misaligned(idx, 4) || misaligned(weights, 4)) return SDT_ERR_UNSUPPORTED;
    uint8_t* w = static_cast<uint8_t*>(workspace);
    if (K == 0) return moe_plan(idx, plan, stream);
    // Every token is read and quantised once; the gated product comes out quantised.
    rc = plan_and_quantize<Elt>(idx, plan, rows, K, X, ldx, w + l.xq, l.ldx, w + l.xs, stream);
    const Mx4Out hq = {w + l.hq, w + l.hs, l.ldhq};
    if (rc == SDT_OK)
        rc = moe_gemm<Elt>(plan, N, K, w + l.xq, l.ldx, w + l.xs, &layer->gate, &layer->up, nullptr, 0,
                           stream, hq);
    if (rc == SDT_OK)
        rc = moe_gemm<Elt>(plan, K, N, w + l.hq, l.ldhq, w + l.hs, &layer->down, nullptr, w + l.d,
                           l.ldd, stream);
    if (rc == SDT_OK) rc = combine<S>(plan, K, w + l.d, l.ldd, weights, Y, ldy, stream);
    return rc;
}

}  // namespace
}  // namespace sdt

using namespace sdt;

extern "C" int64_t sdt_mx4_row_bytes(int64_t K) { return K < 0 ? -1 : row_bytes(K); }

extern "C" int64_t sdt_mx4_scale_bytes(int64_t rows, int64_t K) {
    if (rows < 0 || K < 0) return -1;
    return ceil_div(rows, 64) * k_tiles(K) * kMx4Tile;
}

#define SDT_MX4_TYPES(X) X(f16, Mx4F16, _Float16, 0) X(bf16, Mx4BF16, __bf16, 1)

#define SDT_DEFINE(NAME, ELT, SCALAR, OUT)                                                          \
    extern "C" int mx4_quantize_##NAME(int64_t rows, int64_t K, const void* X, int64_t ldx,         \
                                       void* Q, int64_t ldq, void* S, void* stream) {               \
        return quantize<ELT>(rows, K, X, rows, ldx, nullptr, 0, Q, ldq, S, stream);                 \
    }                                                                                               \
    extern "C" int mx4_quantize_rows_##NAME(                                                        \
        int64_t rows, int64_t K, const void* X, int64_t xrows, int64_t ldx, const int32_t* index,   \
        int divisor, void* Q, int64_t ldq, void* S, void* stream) {                                 \
        if (rows > 0 && !index) return SDT_ERR_INVALID_ARG;                                         \
        return quantize<ELT>(rows, K, X, xrows, ldx, index, divisor, Q, ldq, S, stream);            \
    }                                                                                               \
    extern "C" int gemm_mx4_##NAME(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,     \
                                   const void* SA, const void* B, int64_t ldb, const void* SB,      \
                                   void* C, int64_t ldc, void* stream) {                            \
        return gemm<ELT>(M, N, K, A, lda, SA, B, ldb, SB, C, ldc, stream);                          \
    }                                                                                               \
    extern "C" int gemv_mx4_m1_##NAME(int64_t N, int64_t K, const void* x, const void* B,           \
                                      int64_t ldb, const void* SB, void* y, void* stream) {         \
        return gemv<ELT>(N, K, x, B, ldb, SB, y, stream);                                           \
    }                                                                                               \
    extern "C" int moe_gemm_mx4_##NAME(const sdt_moe_plan* plan, int64_t N, int64_t K,              \
                                       const void* A, int64_t lda, const void* SA,                  \
                                       const sdt_mx4_experts* B, const sdt_mx4_experts* up,         \
                                       void* C, int64_t ldc, void* stream) {                        \
        return moe_gemm<ELT>(plan, N, K, A, lda, SA, B, up, C, ldc, stream);                        \
    }                                                                                               \
    extern "C" int moe_combine_##NAME(const sdt_moe_plan* plan, int64_t N, const void* D,           \
                                      int64_t ldd, const float* weights, void* Y, int64_t ldy,      \
                                      void* stream) {                                               \
        return combine<SCALAR>(plan, N, D, ldd, weights, Y, ldy, stream);                           \
    }                                                                                               \
    extern "C" int moe_experts_mx4_##NAME(                                                          \
        const sdt_moe_layer* layer, const int32_t* idx, const float* weights,                       \
        const sdt_moe_plan* plan, const void* X, int64_t ldx, void* Y, int64_t ldy,                 \
        void* workspace, int64_t workspace_bytes, void* stream) {                                   \
        return moe_layer<ELT>(layer, idx, weights, plan, X, ldx, Y, ldy, workspace,                 \
                              workspace_bytes, stream);                                             \
    }
SDT_MX4_TYPES(SDT_DEFINE)
#undef SDT_DEFINE

#define SDT_DEFINE(NAME, OUT)                                                                       \
    extern "C" int mx4_dequantize_##NAME(int64_t rows, int64_t K, const void* Q, int64_t ldq,       \
                                         const void* S, void* Y, int64_t ldy, void* stream) {       \
        return dequantize<OUT>(rows, K, Q, ldq, S, Y, ldy, stream);                                 \
    }
SDT_DEFINE(f16, 0)
SDT_DEFINE(bf16, 1)
SDT_DEFINE(f32, 2)
#undef SDT_DEFINE

#define SDT_DEFINE(NAME, T)                                                                         \
    extern "C" int moe_route_##NAME(int64_t n, int64_t E, const void* logits, int64_t ld,           \
                                    const float* bias, const sdt_route* cfg, int32_t* idx,          \
                                    float* weights, void* stream) {                                 \
        return route<T>(n, E, logits, ld, bias, cfg, idx, weights, stream);                         \
    }                                                                                               \
    extern "C" int moe_route_backward_##NAME(int64_t n, int64_t E, const void* logits, int64_t ld,  \
                                             const sdt_route* cfg, const int32_t* idx,              \
                                             const float* dweights, void* dlogits, int64_t ldd,     \
                                             void* stream) {                                        \
        return route_backward<T>(n, E, logits, ld, cfg, idx, dweights, dlogits, ldd, stream);       \
    }
SDT_DEFINE(f32, float)
SDT_DEFINE(f16, _Float16)
SDT_DEFINE(bf16, __bf16)
#undef SDT_DEFINE

extern "C" int mx4_pack_scales(int64_t rows, int64_t K, const void* R, int64_t ldr, void* S,
                               void* stream) {
    if (rows < 0 || K < 0) return SDT_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return SDT_OK;
    const int64_t nb = ceil_div(K, 32);
    if (!R || !S || ldr < nb) return SDT_ERR_INVALID_ARG;
    if (K > kMaxK || rows > kMaxRows || misaligned(S, 16)) return SDT_ERR_UNSUPPORTED;
    const int64_t grid = ceil_div(rows, 64) * k_tiles(K);
    if (grid > INT_MAX) return SDT_ERR_UNSUPPORTED;
    const uint8_t* r = static_cast<const uint8_t*>(R);
    uint8_t* s = static_cast<uint8_t*>(S);
    int n = (int)nb, nkt = (int)k_tiles(K);
    void* args[] = {&r, &ldr, &rows, &n, &nkt, &s};
    return launched(hipLaunchKernel(reinterpret_cast<const void*>(&mx4_pack_scales_kernel),
                                    dim3((unsigned)grid), dim3(256), args, 0,
                                    static_cast<hipStream_t>(stream)));
}

extern "C" int64_t sdt_moe_plan_rows(int64_t tokens, int topk, int experts) {
    if (tokens < 0 || topk < 1 || experts < 1 || tokens > INT_MAX) return -1;
    const int64_t R = tokens * topk;
    const int64_t rows = (R + 63 * std::min<int64_t>(experts, R)) / 64 * 64;
    return rows > INT_MAX ? -1 : rows;
}

extern "C" int moe_plan(const int32_t* idx, const sdt_moe_plan* plan, void* stream) {
    int64_t rows;
    int rc = check_plan(plan, &rows);
    if (rc != SDT_OK) return rc;
    if (plan->tokens > 0 && !idx) return SDT_ERR_INVALID_ARG;
    if (misaligned(idx, 4)) return SDT_ERR_UNSUPPORTED;
    PlanParams p = plan_params(idx, plan, rows);
    return launch(reinterpret_cast<const void*>(&moe_plan_kernel), p.E, 1024, p, stream);
}

extern "C" int64_t sdt_moe_experts_workspace_size(int64_t tokens, int topk, int experts, int64_t N,
                                                  int64_t K) {
    const int64_t rows = sdt_moe_plan_rows(tokens, topk, experts);
    if (rows < 0 || N < 0 || K < 0) return -1;
    if (N > kMaxK || K > kMaxK) return -1;
    return layer_layout(rows, N, K).bytes;
}
