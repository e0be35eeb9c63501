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

// One step of a reduction towards lane 63: lanes without a source, or of rows
// outside ROWS, get `none`.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t none, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false);
}
template <typename V, typename F>
__device__ __forceinline__ V wave_reduce(V v, F f) {
    v = f(v, std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xf>{});   // row_shr:1
    v = f(v, std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xf>{});
    v = f(v, std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xf>{});
    v = f(v, std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xf>{});
    v = f(v, std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});   // row_bcast:15
    return f(v, std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});  // :31
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __builtin_bit_cast(float, lane_value(__builtin_bit_cast(uint32_t, v), lane));
}
// Over the wave, known to every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = wave_reduce(v, [](uint32_t x, auto c, auto r) {
        const uint32_t o = dpp<decltype(c)::value, decltype(r)::value>(0, x);
        return x > o ? x : o;
    });
    return lane_value(v, 63);
}
__device__ __forceinline__ float wave_max(float v) {
    v = wave_reduce(v, [](float x, auto c, auto r) {
        const uint32_t o = dpp<decltype(c)::value, decltype(r)::value>(0xff800000u,
                                                                       __builtin_bit_cast(uint32_t, x));
        return fmaxf(x, __builtin_bit_cast(float, o));
    });
    return lane_value(v, 63);
}
__device__ __forceinline__ float wave_sum(float v) {
    v = wave_reduce(v, [](float x, auto c, auto r) {
        const uint32_t o = dpp<decltype(c)::value, decltype(r)::value>(0, __builtin_bit_cast(uint32_t, x));
        return x + __builtin_bit_cast(float, o);
    });
    return lane_value(v, 63);
}
__device__ __forceinline__ double wave_sum(double v) {
    v = wave_reduce(v, [](double x, auto c, auto r) {
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const uint64_t lo = dpp<decltype(c)::value, decltype(r)::value>(0, (uint32_t)u);
        const uint64_t hi = dpp<decltype(c)::value, decltype(r)::value>(0, (uint32_t)(u >> 32));
        return x + __builtin_bit_cast(double, (hi << 32) | lo);
    });
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = lane_value((uint32_t)u, 63), hi = lane_value((uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, (hi << 32) | lo);
}

// Keys whose unsigned order is the order of the values (-0 as +0, a NaN as
// -infinity).  0 is below every key: an expert that may not be chosen.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) v = -__builtin_inff();
    const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) v = -__builtin_inf();
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double key_value(uint64_t k) {
    return __builtin_bit_cast(double, (k >> 63) ? (k & 0x7fffffffffffffffull) : ~k);
}

// The lowest lane that holds the wave's largest key.
__device__ __forceinline__ int best_lane(uint32_t k) {
    const uint32_t top = wave_max(k);
    return __builtin_ctzll(__ballot(k == top));
}
__device__ __forceinline__ int best_lane(uint64_t k) {
    const uint32_t hi = (uint32_t)(k >> 32);
    const uint32_t tophi = wave_max(hi);
    const uint32_t lo = hi == tophi ? (uint32_t)k : 0u;
    const uint32_t toplo = wave_max(lo);
    return __builtin_ctzll(__ballot(hi == tophi && (uint32_t)k == toplo));
}

// Scores.  A softmax's numerator: the largest logit's is 1, also an infinite one's.
__device__ __forceinline__ float softmax_numerator(float x, float top) {
    return x == -__builtin_inff() ? 0.0f : x == top ? 1.0f : expf(x - top);
}
// A sigmoid and 1 - it, from e = exp(-|x|) in [0, 1], so that neither overflows or is
// a difference (the reciprocal, of a number in [1, 2], is a step off at most).
struct Sigmoid {
    float s, c;
};
__device__ __forceinline__ Sigmoid sigmoid(float x) {
    const float e = expf(-fabsf(x));
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    return x >= 0.0f ? Sigmoid{r, e * r} : Sigmoid{e * r, r};
}
// A score for a sum that it is divided by: over a common factor, exp(m - top) / sum
// for a softmax and exp(m) for sigmoids of an m < 0, with m the largest logit in the
// sum (top: of the row), so that scores far below 1 keep their ratios.  Zero where 64
// bits hold no more of the score itself, a softmax 745 below the row's largest and
// a sigmoid below -709: a logit of a type's lowest value is a mask, whatever it is
// compared with.
__device__ __forceinline__ float softmax_share(float x, float top, float m) {
    return x - top < -745.0f ? 0.0f : softmax_numerator(x, m);
}
__device__ __forceinline__ float sigmoid_share(float x, float m, const Sigmoid& g) {
    if (!(m < 0.0f)) return g.s;
    return x < -709.0f ? 0.0f : expf(x - m) * g.c;   // 1 / (1 + exp(x)) = 1 - sigmoid(x)
}

// One wave per token; lane l holds experts l EPL .. + EPL - 1, so the lowest
// lane among equals has the lowest expert.  Renormalised weights are formed from
// the chosen logits, a lane each; the choice is topk rounds of a wave-wide maximum,
// six steps of lane-crossing operands (DPP) on 32-bit keys.  Keys come from the
// logits in fp32 or (WIDE), with a bias or worths summed over two, from scores in
// 64 bits, so that two experts tie only where their definitions do.  Bound by
// the rounds' instructions: 16384 tokens, 8 of 128 experts (bf16): 35 us with
// lane exchanges through LDS on 64-bit keys, 9.8 us so (a score for every expert
// instead of the chosen: 10.4).
template <typename T, int EPL, bool WIDE>
__global__ __launch_bounds__(256) void moe_route_kernel(RouteParams p) {
    typedef std::conditional_t<WIDE, uint64_t, uint32_t> Key;
    __shared__ Key shared_keys[4][EPL * 64];      // groups: a wave's keys by expert
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= p.T) return;
    const float ninf = -__builtin_inff();
    const int e0 = lane * EPL;
    float x[EPL];
    float top = ninf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        x[j] = e0 + j < p.E ? route_load<T>(p.logits, t * p.ld + e0 + j) : ninf;
        if (x[j] != x[j]) x[j] = ninf;
        top = fmaxf(top, x[j]);
    }
    // what the chosen take to their weights: the score, or the logit where the scores
    // are renormalised
    float v[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) v[j] = x[j];
    double sd[WIDE ? EPL : 1];
    if (p.score == 0) {
        top = wave_max(top);
        if (!p.renormalize) {
            float total = 0.0f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                v[j] = softmax_numerator(x[j], top);
                total += v[j];
            }
            total = wave_sum(total);
            const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) v[j] *= inv;
        }
        if constexpr (WIDE) {
            double totald = 0.0;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                sd[j] = x[j] == ninf ? 0.0 : x[j] == top ? 1.0 : exp((double)x[j] - (double)top);
                totald += sd[j];
            }
            totald = wave_sum(totald);
#pragma unroll
            for (int j = 0; j < EPL; ++j) sd[j] = totald > 0.0 ? sd[j] / totald : 0.0;
        }
    } else {
        if (!p.renormalize)
#pragma unroll
            for (int j = 0; j < EPL; ++j) v[j] = sigmoid(x[j]).s;
        if constexpr (WIDE)
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                sd[j] = x[j] == ninf ? 0.0 : 1.0 / (1.0 + exp(-(double)x[j]));
    }
    Key key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        const int e = e0 + j;
        if constexpr (WIDE) {
            const double c =
                p.bias != nullptr ? sd[j] + (e < p.E ? (double)p.bias[e] : 0.0) : (double)x[j];
            key[j] = e < p.E ? order_key(c) : 0;
        } else {
            key[j] = e < p.E ? order_key(x[j]) : 0;
        }
    }
    if (p.groups > 1) {
        // A group's worth: its best value, or the sum of its two best.  `parts` lanes
        // scan a group, then merge.
        const int per = p.E / p.groups;
        Key* mine = shared_keys[wave];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            Key v = key[j];
            if constexpr (WIDE)
                if (p.bias == nullptr && p.group_top == 2) v = order_key(sd[j]);
            mine[e0 + j] = v;
        }
        // other lanes' keys: LDS runs a wave's accesses in order, the fence keeps
        // the compiler from reordering them
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int shift = 31 - __builtin_clz(64 / p.groups);     // parts = 1 << shift
        const int g = lane >> shift, part = lane & ((1 << shift) - 1);
        Key b1 = 0, b2 = 0;
        if (g < p.groups)
            for (int i = part; i < per; i += 1 << shift) {
                const Key v = mine[g * per + i];
                const Key lo = v < b1 ? v : b1;
                b1 = v > b1 ? v : b1;
                b2 = lo > b2 ? lo : b2;
            }
        for (int m = 1; m < 1 << shift; m <<= 1) {
            Key o1, o2;
            if constexpr (WIDE) {
                o1 = __shfl_xor((unsigned long long)b1, m);
                o2 = __shfl_xor((unsigned long long)b2, m);
            } else {
                o1 = (uint32_t)__shfl_xor((int)b1, m);
                o2 = (uint32_t)__shfl_xor((int)b2, m);
            }
            const Key lo = o1 < b1 ? o1 : b1;
            b1 = o1 < b1 ? b1 : o1;
            b2 = b2 > o2 ? b2 : o2;
            b2 = b2 > lo ? b2 : lo;
        }
        Key worth = b1;
        if constexpr (WIDE)
            if (p.group_top == 2) worth = order_key(key_value(b1) + key_value(b2));
        if (part != 0 || g >= p.groups) worth = 0;
        uint64_t keptmask = 0;
        for (int r = 0; r < p.kept; ++r) {
            const int l = best_lane(worth);
            keptmask |= 1ull << (l >> shift);
            if (lane == l) worth = 0;
        }
        int eg = e0 / per, rem = e0 - eg * per;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            if (e0 + j >= p.E || !((keptmask >> eg) & 1)) key[j] = 0;
            if (++rem == per) {
                rem = 0;
                ++eg;
            }
        }
    }
    // topk rounds over the lanes' best; lane r keeps the r-th choice
    int mine = 0;
    float w = ninf;
    for (int r = 0; r < p.topk; ++r) {
        Key best = key[0];
        int at = 0;
        float chosen = v[0];
#pragma unroll
        for (int j = 1; j < EPL; ++j)
            if (key[j] > best) {
                best = key[j];
                at = j;
                chosen = v[j];
            }
        const int l = best_lane(best);
        const int e = l * EPL + (int)lane_value((uint32_t)at, l);
        chosen = lane_value(chosen, l);
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (e0 + j == e) key[j] = 0;
        if (lane == r) {
            mine = e;
            w = chosen;
        }
    }
    if (p.renormalize) {
        // without a bias the first choice has the largest logit
        const float m = p.bias == nullptr ? lane_value(w, 0) : wave_max(w);
        w = p.score == 0 ? softmax_share(w, top, m) : sigmoid_share(w, m, sigmoid(w));
        const float sum = wave_sum(w);           // lanes past topk: of -infinity, 0
        w = sum > 0.0f ? w / sum : 0.0f;
    }
    if (lane < p.topk) {
        p.idx[t * p.topk + lane] = mine;
        p.weights[t * p.topk + lane] = w * p.scale;
    }
}

// The gradient of the logits, one wave per token.  With p_r the chosen scores over
// their sum and dw_r their weights' gradients:
//   renormalised: the logit of slot r gets scale p_r (dw_r - sum_i p_i dw_i), for a
//   sigmoid times 1 - s_r (softmax: s_r / sum = p_r), other logits exactly zero;
//   sigmoid: scale s_r (1 - s_r) dw_r, others zero;
//   softmax: every logit gets scale s_j (dw_j - sum_i s_i dw_i), dw_j = 0 where not
//   chosen, the sum of its slots' where chosen more than once.
// The sums' weights add up to 1, so any constant may be taken from all dw: with the
// one of the largest score nothing is left to cancel where that score is next to 1.
// The first two are worked out a slot a lane and then go to the lanes that hold the
// experts' outputs (EPL each, in order), in slot order.
// 16384 tokens, 8 of 128 experts (bf16): 8.2 us, bound by its instructions (memory
// alone would be 2).  A softmax needs the row's largest logit, so the row is there,
// and up to four logits a lane a slot's comes from its lane (65536 tokens, 2 of 200:
// 26.3 us, from memory 28.1); a sigmoid reads the slots' alone (16384, 8 of 256: 9.9
// us, the rows 10.6).
template <typename T, int EPL>
__global__ __launch_bounds__(256) void moe_route_backward_kernel(RouteParams p) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= p.T) return;
    const float ninf = -__builtin_inff();
    const int e0 = lane * EPL;
    int er = -1;                               // this lane's slot
    float dw = 0.0f, xr = ninf;
    if (lane < p.topk) {
        er = p.idx[t * p.topk + lane];
        dw = p.dweights[t * p.topk + lane];
        if (er < 0 || er >= p.E) er = -1;
    }
    float out[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) out[j] = 0.0f;
    // v of every slot to its expert
    auto scatter = [&](float v) {
        for (int r = 0; r < p.topk; ++r) {
            const int e = (int)lane_value((uint32_t)er, r);
            const float vr = lane_value(v, r);
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                if (e == e0 + j) out[j] += vr;
        }
    };
    // the slots' gradients from their scores q over the largest, which has the logit m
    auto renormalized = [&](float q, float m, float factor) {
        const uint64_t largest = __ballot(er >= 0 && xr == m);
        const float d = dw - (largest ? lane_value(dw, __builtin_ctzll(largest)) : 0.0f);
        if (er < 0) q = 0.0f;
        const float S = wave_sum(q);
        const float inner = wave_sum(er >= 0 ? q * d : 0.0f);
        const float inv = S > 0.0f ? 1.0f / S : 0.0f;
        scatter(p.scale * factor * (q * inv) * (d - inner * inv));
    };
    auto slot_from_memory = [&]() {
        if (er >= 0) xr = route_load<T>(p.logits, t * p.ld + er);
        if (xr != xr) xr = ninf;
    };
    if (p.score != 0) {
        slot_from_memory();
        const Sigmoid g = sigmoid(xr);
        if (p.renormalize) {
            const float m = wave_max(xr);
            renormalized(sigmoid_share(xr, m, g), m, g.c);
        } else {
            scatter(p.scale * (g.s * g.c) * dw);
        }
    } else {
        float x[EPL];
        float top = ninf;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            x[j] = e0 + j < p.E ? route_load<T>(p.logits, t * p.ld + e0 + j) : ninf;
            if (x[j] != x[j]) x[j] = ninf;
            top = fmaxf(top, x[j]);
        }
        top = wave_max(top);
        if (p.renormalize) {
            if constexpr (EPL <= 4) {          // the logit is in the lane of its expert
#pragma unroll
                for (int j = 0; j < EPL; ++j) {
                    const float got = __shfl(x[j], er < 0 ? 0 : er / EPL);
                    if (er >= 0 && er % EPL == j) xr = got;
                }
            } else {
                slot_from_memory();
            }
            const float m = wave_max(xr);
            renormalized(softmax_share(xr, top, m), m, 1.0f);
        } else {
            scatter(dw);
            bool largest = false;
            float pivot = 0.0f;
#pragma unroll
            for (int j = EPL - 1; j >= 0; --j)
                if (x[j] == top) {
                    largest = true;
                    pivot = out[j];
                }
            pivot = lane_value(pivot, __builtin_ctzll(__ballot(largest)));
            float S = 0.0f, inner = 0.0f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                x[j] = softmax_numerator(x[j], top);
                out[j] -= pivot;
                S += x[j];
                inner += x[j] * out[j];
            }
            S = wave_sum(S);
            inner = wave_sum(inner);
            const float inv = S > 0.0f ? 1.0f / S : 0.0f;
            const float mean = inner * inv;
#pragma unroll
            for (int j = 0; j < EPL; ++j) out[j] = p.scale * (x[j] * inv) * (out[j] - mean);
        }
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j)
        if (e0 + j < p.E) static_cast<T*>(p.dlogits)[t * p.ldd + e0 + j] = (T)out[j];
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
    constexpr int NW = 16;
    __shared__ int hist[kMaxExperts];
    __shared__ int wcount[NW], wbefore[NW];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int e = blockIdx.x;
    for (int i = t; i < p.E; i += NW * 64) hist[i] = 0;
    __syncthreads();
    // this wave's quads of slots
    const int quads = (int)(((int64_t)p.R + 3) / 4);
    const int per = (quads + NW - 1) / NW;
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
    SlotQuad v[kPlanLoads];
    for (int q0 = first; q0 < last; q0 += 64 * kPlanLoads) {
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
    for (int i = t; i < e; i += NW * 64) before += (hist[i] + 63) & ~63;
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) before += __shfl_xor(before, m);
    if (lane == 0) wbefore[wave] = before;
    __syncthreads();
    int start = 0, row0 = 0, count = 0;
    for (int w = 0; w < NW; ++w) {
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
    for (int i = start + count + t; i < end; i += NW * 64) p.rows[i] = -1;
    for (int i = start / 64 + t; i < end / 64; i += NW * 64) p.tiles[i] = e;
    if (e == p.E - 1) {
        for (int i = end + t; i < p.cap; i += NW * 64) p.rows[i] = -1;
        for (int i = end / 64 + t; i < p.cap / 64; i += NW * 64) p.tiles[i] = -1;
    }
    if (mine == 0) return;
    int row = start + row0;                    // of this wave's next slot
    const uint64_t below = (1ull << lane) - 1;
    for (int q0 = first; q0 < last; q0 += 64 * kPlanLoads) {
        if (last - first > 64 * kPlanLoads) load(q0, v);   // else they are still there
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

// Eight columns of one token per thread, the rows of four slots loaded together.
// Bound by reading D (4096 tokens, 6 rows of 2048 each: 19 us, 5.2 TB/s).
template <typename S>
__global__ __launch_bounds__(256) void moe_combine_kernel(CombineParams p) {
    constexpr int G = 4;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = id / p.nch;
    if (t >= p.T) return;
    const int n = (int)(id - t * p.nch) * 8;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    typedef S vec8 __attribute__((ext_vector_type(8)));
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    for (int j0 = 0; j0 < p.topk; j0 += G) {
        int row[G];
        float w[G];
#pragma unroll
        for (int u = 0; u < G; ++u) {
            const bool in = j0 + u < p.topk;
            row[u] = in ? p.pos[t * p.topk + j0 + u] : -1;
            w[u] = in ? p.weights[t * p.topk + j0 + u] : 0.0f;
        }
        if (n + 7 < p.N) {
            u4 v[G];
#pragma unroll
            for (int u = 0; u < G; ++u) {
                v[u] = u4{0, 0, 0, 0};
                if (row[u] >= 0) v[u] = *reinterpret_cast<const u4*>(p.D + row[u] * p.ldd + n);
            }
#pragma unroll
            for (int u = 0; u < G; ++u)
                if (row[u] >= 0) {
                    const vec8 x = __builtin_bit_cast(vec8, v[u]);
#pragma unroll
                    for (int c = 0; c < 8; ++c) acc[c] += w[u] * (float)x[c];
                }
        } else {
            for (int u = 0; u < G; ++u)
                if (row[u] >= 0)
                    for (int c = 0; c < 8; ++c)
                        if (n + c < p.N) {
                            const uint16_t d = p.D[row[u] * p.ldd + n + c];
                            acc[c] += w[u] * (float)__builtin_bit_cast(S, d);
                        }
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
