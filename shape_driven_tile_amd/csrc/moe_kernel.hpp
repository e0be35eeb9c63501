// Expert routing for gfx950: the choice of experts and its gradient, the plan
// that sorts the chosen slots by expert, and the weighted sum of the experts'
// outputs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace sdt {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 64;
constexpr int kMaxGroups = 64;

struct RouteParams {
    const void* logits;
    int64_t ld;
    const float* bias;
    int32_t* idx;
    float* weights;
    int64_t T;
    int E, topk, score, groups, kept, group_top, renormalize;
    float scale;
    // backward
    const float* dweights;
    void* dlogits;
    int64_t ldd;
};

template <typename T>
__device__ __forceinline__ float route_load(const void* p, int64_t i) {
    if constexpr (std::is_same_v<T, float>) return static_cast<const float*>(p)[i];
    if constexpr (std::is_same_v<T, _Float16>) return (float)static_cast<const _Float16*>(p)[i];
    if constexpr (std::is_same_v<T, __bf16>) return (float)static_cast<const __bf16*>(p)[i];
}

template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m));
    return v;
}

// Keys whose unsigned order is the order of the doubles (-0 as +0, a NaN as
// -infinity).  0 is below every key: an expert that may not be chosen.
__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) v = -__builtin_inf();
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value(uint64_t k) {
    return __builtin_bit_cast(double, (k >> 63) ? (k & 0x7fffffffffffffffull) : ~k);
}

// (key, index) of the largest key over the wave, the lowest index among equals.
__device__ __forceinline__ void wave_best(uint64_t& k, int& i) {
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) {
        const uint64_t ok = __shfl_xor((unsigned long long)k, m);
        const int oi = __shfl_xor(i, m);
        if (ok > k || (ok == k && oi < i)) {
            k = ok;
            i = oi;
        }
    }
}

// One wave per token; lane l holds experts l, l + 64, ... (EPL of them).
// Every score is formed from the logits in registers; the choice is topk
// rounds of a wave-wide maximum on 64-bit keys.  Keys come from the logits in
// fp32 or, with a bias or worths summed over two, from scores in 64 bits, so
// that two experts tie only where their definitions do.
template <typename T, int EPL>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteParams p) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= p.T) return;
    const float ninf = -__builtin_inff();
    float x[EPL];
    float top = ninf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = j * 64 + lane;
        x[j] = e < p.E ? route_load<T>(p.logits, t * p.ld + e) : ninf;
        if (x[j] != x[j]) x[j] = ninf;
        top = fmaxf(top, x[j]);
    }
    top = wave_max(top);
    // scores: softmax's numerators (the largest logit's is 1, also an infinite
    // one's) or sigmoids
    const bool wide = p.bias != nullptr || p.group_top == 2;
    float s[EPL];
    double sd[EPL];
    float total = 0.0f;
    double totald = 0.0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        sd[j] = 0.0;
        if (p.score == 0) {
            s[j] = x[j] == ninf ? 0.0f : x[j] == top ? 1.0f : expf(x[j] - top);
            total += s[j];
            if (wide) {
                sd[j] = x[j] == ninf ? 0.0 : x[j] == top ? 1.0 : exp((double)x[j] - (double)top);
                totald += sd[j];
            }
        } else {
            s[j] = x[j] == ninf ? 0.0f : 1.0f / (1.0f + expf(-x[j]));
            if (wide) sd[j] = x[j] == ninf ? 0.0 : 1.0 / (1.0 + exp(-(double)x[j]));
        }
    }
    if (p.score == 0) {
        total = wave_sum(total);
        const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) s[j] *= inv;
        if (wide) {
            totald = wave_sum(totald);
#pragma unroll
            for (int j = 0; j < EPL; ++j) sd[j] = totald > 0.0 ? sd[j] / totald : 0.0;
        }
    }
    uint64_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = j * 64 + lane;
        const double c = p.bias != nullptr ? sd[j] + (e < p.E ? (double)p.bias[e] : 0.0) : (double)x[j];
        key[j] = e < p.E ? order_key(c) : 0;
    }
    if (p.groups > 1) {
        // a group's worth: its best value, or the sum of its two best
        const int per = p.E / p.groups;
        uint64_t worth = 0;               // lane g: group g's
        for (int g = 0; g < p.groups; ++g) {
            uint64_t b1 = 0, b2 = 0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                const int e = j * 64 + lane;
                if (e / per == g && e < p.E) {
                    const uint64_t v = p.bias != nullptr || p.group_top == 1 ? key[j] : order_key(sd[j]);
                    if (v > b1) {
                        b2 = b1;
                        b1 = v;
                    } else if (v > b2) {
                        b2 = v;
                    }
                }
            }
#pragma unroll
            for (int m = 32; m > 0; m >>= 1) {
                const uint64_t o1 = __shfl_xor((unsigned long long)b1, m);
                const uint64_t o2 = __shfl_xor((unsigned long long)b2, m);
                const uint64_t lo = o1 < b1 ? o1 : b1;
                b1 = o1 < b1 ? b1 : o1;
                b2 = b2 > o2 ? b2 : o2;
                b2 = b2 > lo ? b2 : lo;
            }
            const uint64_t w = p.group_top == 1 ? b1 : order_key(key_value(b1) + key_value(b2));
            if (lane == g) worth = w;
        }
        uint64_t keptmask = 0;
        for (int r = 0; r < p.kept; ++r) {
            uint64_t k = worth;
            int i = lane;
            wave_best(k, i);
            keptmask |= 1ull << i;
            if (lane == i) worth = 0;
        }
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = j * 64 + lane;
            if (e < p.E && !((keptmask >> (e / per)) & 1)) key[j] = 0;
        }
    }
    // topk rounds; lane r keeps the r-th choice
    int mine = 0;
    float w = 0.0f;
    for (int r = 0; r < p.topk; ++r) {
        uint64_t k = key[0];
        int i = lane;
#pragma unroll
        for (int j = 1; j < EPL; ++j)
            if (key[j] > k) {
                k = key[j];
                i = j * 64 + lane;
            }
        wave_best(k, i);
        float sv = 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (i == j * 64 + lane) {
                key[j] = 0;
                sv = s[j];
            }
        sv = __shfl(sv, i & 63);
        if (lane == r) {
            mine = i;
            w = sv;
        }
    }
    if (p.renormalize) {
        const float sum = wave_sum(w);
        w = sum > 0.0f ? w / sum : 0.0f;
    }
    if (lane < p.topk) {
        p.idx[t * p.topk + lane] = mine;
        p.weights[t * p.topk + lane] = w * p.scale;
    }
}

// The gradient of the logits, one wave per token.  With p_j the chosen scores
// over their sum S (renormalised) or the scores: ds_j = scale / S * (dw_j -
// sum_i dw_i p_i), or scale * dw_j; a sigmoid's dl = s (1 - s) ds.  Softmax:
// dl = s (ds - sum ds s); renormalised, that sum is zero by construction and
// s_j / S = p_j, so dl_j = scale p_j (dw_j - sum dw p) on the chosen and
// exactly zero elsewhere.
template <typename T, int EPL>
__global__ __launch_bounds__(256) void moe_route_backward_kernel(RouteParams p) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= p.T) return;
    const float ninf = -__builtin_inff();
    float x[EPL], s[EPL], ds[EPL];
    float top = ninf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = j * 64 + lane;
        x[j] = e < p.E ? route_load<T>(p.logits, t * p.ld + e) : ninf;
        if (x[j] != x[j]) x[j] = ninf;
        top = fmaxf(top, x[j]);
        ds[j] = 0.0f;
    }
    float total = 0.0f;
    if (p.score == 0) {
        top = wave_max(top);
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            s[j] = x[j] == ninf ? 0.0f : x[j] == top ? 1.0f : expf(x[j] - top);
            total += s[j];
        }
        total = wave_sum(total);
        const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) s[j] *= inv;
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) s[j] = x[j] == ninf ? 0.0f : 1.0f / (1.0f + expf(-x[j]));
    }
    // the weights' gradients to their experts' lanes (an expert named twice
    // gets the sum, in slot order), and the chosen scores' sums
    int e_r = -1;
    float dw_r = 0.0f;
    if (lane < p.topk) {
        e_r = p.idx[t * p.topk + lane];
        dw_r = p.dweights[t * p.topk + lane];
    }
    float S = 0.0f, inner = 0.0f;
    float n[EPL];                          // times an expert was chosen
#pragma unroll
    for (int j = 0; j < EPL; ++j) n[j] = 0.0f;
    for (int r = 0; r < p.topk; ++r) {
        const int e = __shfl(e_r, r);
        const float dw = __shfl(dw_r, r);
        if (e < 0 || e >= p.E) continue;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (e == j * 64 + lane) {
                ds[j] += dw;
                n[j] += 1.0f;
                S += s[j];
                inner += dw * s[j];
            }
    }
    float out[EPL];
    if (p.renormalize) {
        S = wave_sum(S);
        inner = wave_sum(inner);
        const float inv = S > 0.0f ? 1.0f / S : 0.0f;
        const float mean = inner * inv;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const float d = p.scale * (s[j] * inv) * (ds[j] - n[j] * mean);
            out[j] = p.score == 0 ? d : d * (1.0f - s[j]);
        }
    } else {
        inner = wave_sum(inner);
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            out[j] = p.scale * (p.score == 0 ? s[j] * (ds[j] - inner) : s[j] * (1.0f - s[j]) * ds[j]);
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = j * 64 + lane;
        if (e < p.E) static_cast<T*>(p.dlogits)[t * p.ldd + e] = (T)out[j];
    }
}

struct PlanParams {
    const int32_t* idx;
    int32_t *counts, *offsets, *rows, *pos, *tiles;
    int R, E, cap;
};

// One workgroup per expert.  Each counts every expert's slots in LDS (integer
// adds: any order gives the same counts), so each knows where its segment
// starts; then it passes over the slots once more and places its own in order.
// No workgroup needs another's result.  Bound by the latency of reading idx
// twice: every wave owns a contiguous sixteenth of the slots and reads four to a
// lane, kPlanLoads loads in flight, so neither pass has a barrier inside.
constexpr int kPlanLoads = 8;

struct SlotQuad {
    int32_t v[4];
};

__global__ __launch_bounds__(1024) void moe_plan_kernel(PlanParams p) {
    __shared__ int hist[kMaxExperts];
    __shared__ int wcount[16], wbefore[16];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int e = blockIdx.x;
    for (int i = t; i < p.E; i += 1024) hist[i] = 0;
    __syncthreads();
    // this wave's quads of slots
    const int quads = (int)(((int64_t)p.R + 3) / 4);
    const int per = (quads + 15) / 16;
    const int first = min(wave * per, quads), last = min(first + per, quads);
    auto load = [&](int q0, SlotQuad (&v)[kPlanLoads]) {
#pragma unroll
        for (int u = 0; u < kPlanLoads; ++u) {
            const int q = q0 + u * 64 + lane;
            const int64_t i = (int64_t)q * 4;
            if (q < last && i + 3 < p.R) {
                __builtin_memcpy(&v[u], p.idx + i, 16);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[u].v[c] = q < last && i + c < p.R ? p.idx[i + c] : -1;
            }
        }
    };
    int mine = 0;                              // slots of this wave that chose e
    for (int q0 = first; q0 < last; q0 += 64 * kPlanLoads) {
        SlotQuad v[kPlanLoads];
        load(q0, v);
#pragma unroll
        for (int u = 0; u < kPlanLoads; ++u) {
            if (q0 + u * 64 >= last) break;
            const int q = q0 + u * 64 + lane;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int x = v[u].v[c];
                const int64_t i = (int64_t)q * 4 + c;
                mine += __popcll(__ballot(x == e));
                if (q < last && i < p.R) {
                    if (x >= 0 && x < p.E)
                        atomicAdd(&hist[x], 1);
                    else if (e == 0)
                        p.pos[i] = -1;
                }
            }
        }
    }
    if (lane == 0) wcount[wave] = mine;
    __syncthreads();
    // rows before this expert's
    int before = 0;
    for (int i = t; i < e; i += 1024) before += (hist[i] + 63) & ~63;
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) before += __shfl_xor(before, m);
    if (lane == 0) wbefore[wave] = before;
    __syncthreads();
    int start = 0, row0 = 0, count = 0;
    for (int w = 0; w < 16; ++w) {
        start += wbefore[w];
        if (w < wave) row0 += wcount[w];
        count += wcount[w];
    }
    const int end = start + ((count + 63) & ~63);
    if (t == 0) {
        p.counts[e] = count;
        p.offsets[e] = start;
        if (e == p.E - 1) p.offsets[p.E] = end;
    }
    for (int i = start + count + t; i < end; i += 1024) p.rows[i] = -1;
    for (int i = start / 64 + t; i < end / 64; i += 1024) p.tiles[i] = e;
    if (e == p.E - 1) {
        for (int i = end + t; i < p.cap; i += 1024) p.rows[i] = -1;
        for (int i = end / 64 + t; i < p.cap / 64; i += 1024) p.tiles[i] = -1;
    }
    if (mine == 0) return;
    int row = start + row0;                    // of this wave's next slot
    const uint64_t below = (1ull << lane) - 1;
    for (int q0 = first; q0 < last; q0 += 64 * kPlanLoads) {
        SlotQuad v[kPlanLoads];
        load(q0, v);
#pragma unroll
        for (int u = 0; u < kPlanLoads; ++u) {
            if (q0 + u * 64 >= last) break;
            const int i = (int)((uint32_t)(q0 + u * 64 + lane) * 4u);   // used where it is a slot
            int at = row, all = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint64_t mask = __ballot(v[u].v[c] == e);
                at += __popcll(mask & below);
                all += __popcll(mask);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (v[u].v[c] == e) {
                    p.rows[at] = i + c;
                    p.pos[i + c] = at;
                    ++at;
                }
            row += all;
        }
    }
}

struct CombineParams {
    const uint16_t* D;
    int64_t ldd;
    const int32_t* pos;
    const float* weights;
    uint16_t* Y;
    int64_t ldy;
    int64_t T;
    int topk, N, nch;      // nch: chunks of 8 columns
};

// Eight columns of one token per thread.
template <typename S>
__global__ __launch_bounds__(256) void moe_combine_kernel(CombineParams p) {
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = id / p.nch;
    if (t >= p.T) return;
    const int n = (int)(id - t * p.nch) * 8;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    typedef S vec8 __attribute__((ext_vector_type(8)));
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    for (int j = 0; j < p.topk; ++j) {
        const int row = p.pos[t * p.topk + j];
        if (row < 0) continue;
        const float w = p.weights[t * p.topk + j];
        const uint16_t* d = p.D + row * p.ldd + n;
        if (n + 7 < p.N) {
            const vec8 v = __builtin_bit_cast(vec8, *reinterpret_cast<const u4*>(d));
#pragma unroll
            for (int c = 0; c < 8; ++c) acc[c] += w * (float)v[c];
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (n + c < p.N) acc[c] += w * (float)__builtin_bit_cast(S, d[c]);
        }
    }
    uint16_t h[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const S v = (S)acc[c];
        h[c] = __builtin_bit_cast(uint16_t, v);
    }
    uint16_t* y = p.Y + t * p.ldy + n;
    if (n + 7 < p.N) {
        *reinterpret_cast<u4*>(y) = __builtin_bit_cast(u4, h);
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (n + c < p.N) y[c] = h[c];
    }
}

}  // namespace sdt
