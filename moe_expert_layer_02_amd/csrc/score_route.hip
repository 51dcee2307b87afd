// Routing by scores: s = softmax(l) or sigmoid(l) in fp64, selection by s + bias
// (the bias balances the experts' load and never enters a weight), group limit,
// top-k, weights from the unbiased scores.
//
// Decisions are those of fp64, so that two choices that differ by more than a few
// 1e-16 rank the same here as in any other fp64 evaluation; equal choices go to the
// lower id.  Evaluating every score and comparing in fp64 (route_fp64: a wavefront per
// token, lane l with experts [l npl, l npl + npl), npl = ceil(E / 64) <= 8) is bound by
// the vector units: 37 us for 16384 tokens of 256 experts whose logits take 3.5 us to
// read.  So a first pass ranks in fp32 and keeps its result only where no decision was
// close, route_fp64 taking the other tokens; weights are fp64 in both.  With a wavefront
// per token (route_fp32) that took 29 us, with four tokens per wavefront, up to 256
// experts and 14 choices, 13.6 us (1150 vector instructions per four tokens).
#include <type_traits>

#include "internal.h"

namespace moe355 {
namespace {

constexpr int SR_MAX_NPL = 8;
constexpr int SR_MAX_GROUPS = 64;
constexpr int SR_WAVES = 4;

struct ScoreParams {
    const void* logits;
    int64_t stride;
    const float* bias;
    int T, E, k, score, n_group, topk_group, renorm;
    float scale;
    int32_t* ids;
    float* w;
};

// Order-preserving map of a double to uint64 (-0.0 folded onto +0.0 first).
__device__ __forceinline__ uint64_t f64_order_key(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// Token t in fp64.  One wavefront; c: [E] doubles of LDS of its own.
template <bool BF16, int NPL>
__device__ void route_fp64(const ScoreParams& p, int t, double* c) {
    const int lane = threadIdx.x & (WAVE - 1);
    const int E = p.E, npl = (E + WAVE - 1) / WAVE;

    float l[NPL];
    double s[NPL], choice[NPL];
    bool live[NPL], have[NPL];
    float mx = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane * npl + i;
        have[i] = i < npl && e < E;
        l[i] = -__builtin_inff();
        if (have[i]) {
            const int64_t at = static_cast<int64_t>(t) * p.stride + e;
            l[i] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p.logits)[at])
                        : static_cast<const float*>(p.logits)[at];
            if (!(l[i] == l[i])) l[i] = -__builtin_inff();   // NaN: not selectable
        }
        mx = fmaxf(mx, l[i]);
    }
    if (p.score == MOE355_SCORE_SOFTMAX) {
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) mx = fmaxf(mx, __shfl_xor(mx, m, WAVE));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            // the maximum itself is e^0 also where it is +inf; a row of -inf has no mass
            s[i] = l[i] == -__builtin_inff() ? 0.0
                   : l[i] == mx              ? 1.0
                                             : exp(static_cast<double>(l[i]) - static_cast<double>(mx));
            sum += s[i];
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) sum += __shfl_xor(sum, m, WAVE);
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] = 1.0 / (1.0 + exp(-static_cast<double>(l[i])));
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const float b = p.bias && have[i] ? p.bias[lane * npl + i] : 0.0f;
        live[i] = have[i] && l[i] > -__builtin_inff() && b > -__builtin_inff();
        choice[i] = live[i] ? s[i] + static_cast<double>(b) : -__builtin_inf();
    }

    uint64_t kept = ~0ull;
    const int gsize = E / p.n_group;
    if (p.topk_group < p.n_group) {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (have[i]) c[lane * npl + i] = choice[i];
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
        __builtin_amdgcn_wave_barrier();
        // lane g: the sum of group g's up to two best live choices
        double a1 = -__builtin_inf(), a2 = -__builtin_inf();
        if (lane < p.n_group)
            for (int i = 0; i < gsize; ++i) {
                const double v = c[lane * gsize + i];
                a2 = fmax(a2, fmin(a1, v));
                a1 = fmax(a1, v);
            }
        const double score = a2 > -__builtin_inf() ? a1 + a2 : a1;
        int rank = 0;
        for (int g = 0; g < p.n_group; ++g) {
            const double o = __shfl(score, g, WAVE);
            if (o > score || (o == score && g < lane)) ++rank;
        }
        kept = __ballot(lane < p.n_group && rank < p.topk_group);
    }

    // key 0: not there or in a group left out; 1: not selectable (last resort, by id)
    uint64_t key[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = lane * npl + i;
        const bool in = have[i] && ((kept >> (p.topk_group < p.n_group ? e / gsize : 0)) & 1);
        key[i] = !in ? 0ull : live[i] ? f64_order_key(choice[i]) : 1ull;
    }
    int my_e = 0;
    double my_s = 0.0;
    for (int r = 0; r < p.k; ++r) {
        uint64_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < NPL; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint64_t top = wave_max_u64(best);
        const uint64_t who = __ballot(best == top);
        const int owner = __ffsll(static_cast<unsigned long long>(who)) - 1;   // the lowest lane has the lowest ids
        double v = 0.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (i == at) {
                v = live[i] ? s[i] : 0.0;
                if (lane == owner) key[i] = 0ull;
            }
        v = __shfl(v, owner, WAVE);
        const int e = __shfl(lane * npl + at, owner, WAVE);
        if (lane == r) {
            my_e = e;
            my_s = v;
        }
    }
    double sum = 0.0;
    for (int r = 0; r < p.k; ++r) sum += __shfl(my_s, r, WAVE);
    if (lane < p.k) {
        const double w = p.renorm ? my_s / (sum + 1e-20) : my_s;
        p.ids[static_cast<int64_t>(t) * p.k + lane] = my_e;
        p.w[static_cast<int64_t>(t) * p.k + lane] = static_cast<float>(w * static_cast<double>(p.scale));
    }
}

// e^x for x <= 0 by 2^(x log2 e) on the hardware: relative error below 1.8e-7 |x| +
// 2.4e-7 (the product's two roundings and the instruction's 1 ulp).
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// The fp32 pass: false if a decision was close.  ids and weights as route_fp64
// leaves them.  LPG: lanes per group (0: no group limit).
template <bool BF16, int NPL>
__device__ __forceinline__ bool route_fp32(const ScoreParams& p, int t, bool vec, int lpg) {
    const int lane = threadIdx.x & (WAVE - 1);
    const int E = p.E, e0 = lane * NPL;
    float l[NPL];
    const int64_t at = static_cast<int64_t>(t) * p.stride + e0;
    if (vec) {   // rows of whole, aligned lanes: one load
        if (e0 < E) {
            if constexpr (BF16) {
                uint16_t v[NPL];
                __builtin_memcpy(v, __builtin_assume_aligned(static_cast<const uint16_t*>(p.logits) + at, 2 * NPL), 2 * NPL);
#pragma unroll
                for (int i = 0; i < NPL; ++i) l[i] = bf16_to_f32(v[i]);
            } else {
                __builtin_memcpy(l, __builtin_assume_aligned(static_cast<const float*>(p.logits) + at, NPL >= 4 ? 16 : 4 * NPL), 4 * NPL);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (e0 + i < E)
                l[i] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p.logits)[at + i])
                            : static_cast<const float*>(p.logits)[at + i];
    }
    float b[NPL];
    bool plain = true;   // every logit of the row is finite and its bias moderate
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        b[i] = 0.0f;
        if (e0 + i < E) {
            if (p.bias) b[i] = p.bias[e0 + i];
            plain = plain && __builtin_fabsf(l[i]) < 1e30f && __builtin_fabsf(b[i]) < 64.0f;
        } else {
            l[i] = -3.0e38f;
        }
    }
    if (__ballot(!plain)) return false;

    // Scores, and a bound es of their error.  Sigmoid: s (1 - s) times the relative error of
    // e^-l, where s (1 - s) |l| <= 0.23, and the sum's and reciprocal's roundings: below 5e-7.
    // Softmax, d below the maximum, r = 1 / sum: r e^-d (1.8e-7 d + 2.4e-7 + 8e-7 for the
    // sum), largest at d = 0: below 1.5e-6 r.
    float s[NPL], mx = l[0], es = 5e-7f, total = 1.0f;
    const bool soft = p.score == MOE355_SCORE_SOFTMAX;
    if (soft) {
#pragma unroll
        for (int i = 1; i < NPL; ++i) mx = fmaxf(mx, l[i]);
        // order-preserving keys of finite floats: the integer maximum
        mx = __uint_as_float([&] {
            const uint32_t k = wave_max_u32(f32_order_key(mx));
            return (k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k;
        }());
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            s[i] = exp_fast(l[i] - mx);
            sum += s[i];
        }
        total = wave_sum_dpp_f32(sum);
        const float r = 1.0f / total;
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] *= r;
        es = 1.5e-6f * r;
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + exp_fast(-l[i]));
    }
    uint32_t key[NPL];   // of the choices; 0: no expert, or one of a group left out
#pragma unroll
    for (int i = 0; i < NPL; ++i) key[i] = e0 + i < E ? f32_order_key(s[i] + b[i]) : 0u;
    auto value = [](uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k); };

    if (lpg) {
        // the two best keys of the group, by exchanges inside its lanes
        uint32_t a1 = key[0], a2 = 0u;
#pragma unroll
        for (int i = 1; i < NPL; ++i) {
            a2 = max(a2, min(a1, key[i]));
            a1 = max(a1, key[i]);
        }
        for (int m = 1; m < lpg; m <<= 1) {
            const uint32_t o1 = __shfl_xor(a1, m, WAVE), o2 = __shfl_xor(a2, m, WAVE);
            a2 = max(min(a1, o1), max(a2, o2));
            a1 = max(a1, o1);
        }
        const float g = value(a1) + value(a2);
        const int mine = lane / lpg;
        int rank = 0;
        float lowest_in = 3.0e38f, highest_out = -3.0e38f;
        for (int q = 0; q < p.n_group; ++q) {
            const float o = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), q * lpg));
            if (o > g || (o == g && q < mine)) ++rank;
        }
        const bool kept = mine < p.n_group && rank < p.topk_group;
        for (int q = 0; q < p.n_group; ++q) {
            const float o = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), q * lpg));
            if (__builtin_amdgcn_readlane(kept ? 1 : 0, q * lpg)) lowest_in = fminf(lowest_in, o);
            else highest_out = fmaxf(highest_out, o);
        }
        // four scores' errors, and the roundings of sums with biases below 64
        if (!(lowest_in - highest_out > 4.0f * es + (p.bias ? 1.6e-5f : 5e-7f))) return false;
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = kept ? key[i] : 0u;
    }

    int my_e = 0;
    float my_l = 0.0f, last_c = 0.0f, last_l = 0.0f, last_b = 0.0f;
    for (int r = 0; r <= p.k; ++r) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < NPL; ++i) m = max(m, key[i]);
        const uint32_t top = wave_max_u32(m);
        if (top == 0u) break;   // fewer than k + 1 candidates (never fewer than k)
        const uint64_t who = __ballot(m == top);
        const int owner = __ffsll(static_cast<unsigned long long>(who)) - 1;   // the lowest lane has the lowest ids
        int at_i = NPL - 1;
        float li = l[NPL - 1], bi = b[NPL - 1];
#pragma unroll
        for (int i = NPL - 2; i >= 0; --i)
            if (key[i] == top) {
                at_i = i;
                li = l[i];
                bi = b[i];
            }
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = lane == owner && i == at_i ? 0u : key[i];
        const float lo = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(li), owner));
        const float bo = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(bi), owner));
        const int e = __builtin_amdgcn_readlane(e0 + at_i, owner);
        const float c = value(top);
        // two scores' errors, and the roundings of the two sums with a bias
        const float near = 2.0f * es + 2.4e-7f * fmaxf(__builtin_fabsf(last_c), __builtin_fabsf(c));
        // the (k + 1)th has to be clear of the kth: behind a tie there may be a third, equal in fp32
        if (r > 0 && !(last_c - c > near) && !(r < p.k && lo == last_l && bo == last_b)) return false;
        last_c = c;
        last_l = lo;
        last_b = bo;
        if (lane == r) {
            my_e = e;
            my_l = lo;
        }
    }

    // weights in fp64
    double sc;
    if (soft) {
        sc = exp(static_cast<double>(my_l) - static_cast<double>(mx));
        if (p.renorm) {
            // the row's sum cancels but for the 1e-20 beside it, where fp32 does as long as the
            // chosen hold some mass
            const float mass = wave_sum_dpp_f32(lane < p.k ? static_cast<float>(sc) : 0.0f);
            if (!(mass > 1e-6f)) return false;
            sc /= static_cast<double>(total);
        } else {
            double z = 0.0;
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (e0 + i < E) z += exp(static_cast<double>(l[i]) - static_cast<double>(mx));
#pragma unroll
            for (int m = 32; m >= 1; m >>= 1) z += __shfl_xor(z, m, WAVE);
            sc /= z;
        }
    } else {
        sc = 1.0 / (1.0 + exp(-static_cast<double>(my_l)));
    }
    if (lane >= p.k) sc = 0.0;
    if (p.renorm) {
        double sum = sc;   // the first 32 lanes hold the chosen
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor(sum, m, WAVE);
        sc = sc / (sum + 1e-20);
    }
    if (lane < p.k) {
        p.ids[static_cast<int64_t>(t) * p.k + lane] = my_e;
        p.w[static_cast<int64_t>(t) * p.k + lane] = static_cast<float>(sc * static_cast<double>(p.scale));
    }
    return true;
}

template <bool BF16, int NPL>
__global__ void __launch_bounds__(SR_WAVES* WAVE) score_route_kernel(ScoreParams p, bool fast, bool vec, int lpg) {
    extern __shared__ double choice_lds[];   // [SR_WAVES][E], used when groups limit the choice
    const int wv = threadIdx.x / WAVE;
    const int t = blockIdx.x * SR_WAVES + wv;
    if (t >= p.T) return;   // whole wavefronts leave; there is no block barrier
    if (fast && route_fp32<BF16, NPL>(p, t, vec, lpg)) return;
    route_fp64<BF16, NPL>(p, t, choice_lds + static_cast<int64_t>(wv) * p.E);
}

// ---- up to 256 experts and 14 choices: four tokens per wavefront ---------------------------
// A token has a row of 16 lanes, NE = 4, 8 or 16 experts a lane, and most
// instructions serve four tokens.  The fp32 pass as above, on keys whose low bits
// hold the entry's place in its lane: a lane sorts its keys once (a merge network of
// minima and maxima), and a round takes the largest head of the row by four DPP
// maxima over the upper bits, the lowest lane's among equals, and moves that lane on.
// So entries with equal upper bits come in order of their ids.  The k + 2 best of these
// keys are ranked by fp64 choices, and the next one bounds all that is left, equal logits
// apart: few tokens are too close for that and are decided by route_fp64, whose 5 to 8 us
// (one wavefront, from cold) show at the end of a launch.

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xf, 0xf, false));
}
template <int CTRL>
__device__ __forceinline__ float dppf(float v) { return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v))); }
// exchanges that meet every lane of a row of 16: neighbours, pairs, halves, ends
constexpr int QP1 = 0xB1, QP2 = 0x4E, HALF_MIRROR = 0x141, MIRROR = 0x140, ROW_SHL1 = 0x101, ROW_ROR = 0x120;
template <typename F>
__device__ __forceinline__ uint32_t row_all_u32(uint32_t v, F f) {
    v = f(v, dpp_u32<QP1>(v));
    v = f(v, dpp_u32<QP2>(v));
    v = f(v, dpp_u32<HALF_MIRROR>(v));
    return f(v, dpp_u32<MIRROR>(v));
}
template <typename F>
__device__ __forceinline__ float row_all_f32(float v, F f) {
    v = f(v, dppf<QP1>(v));
    v = f(v, dppf<QP2>(v));
    v = f(v, dppf<HALF_MIRROR>(v));
    return f(v, dppf<MIRROR>(v));
}
__device__ __forceinline__ double row_sum_f64(double v) {
    auto step = [&](auto C) {
        constexpr int CTRL = decltype(C)::value;
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint64_t o = static_cast<uint64_t>(dpp_u32<CTRL>(static_cast<uint32_t>(u >> 32))) << 32 | dpp_u32<CTRL>(static_cast<uint32_t>(u));
        v += __builtin_bit_cast(double, o);
    };
    step(std::integral_constant<int, QP1>{});
    step(std::integral_constant<int, QP2>{});
    step(std::integral_constant<int, HALF_MIRROR>{});
    step(std::integral_constant<int, MIRROR>{});
    return v;
}

// e^x in fp64: x = n ln 2 + r, |r| <= 0.35, Taylor's series to r^13 (the next term is
// below 5e-18); 0 and infinity beyond +-800.
__device__ __forceinline__ double exp_f64(double x) {
    x = fmin(fmax(x, -800.0), 800.0);
    const double n = rint(x * 1.4426950408889634);
    const double r = fma(n, -2.3190468138462996e-17, fma(n, -0.6931471805599453, x));   // ln 2 in two parts
    double y = 1.0 / 6227020800.0;
    y = fma(y, r, 1.0 / 479001600.0);
    y = fma(y, r, 1.0 / 39916800.0);
    y = fma(y, r, 1.0 / 3628800.0);
    y = fma(y, r, 1.0 / 362880.0);
    y = fma(y, r, 1.0 / 40320.0);
    y = fma(y, r, 1.0 / 5040.0);
    y = fma(y, r, 1.0 / 720.0);
    y = fma(y, r, 1.0 / 120.0);
    y = fma(y, r, 1.0 / 24.0);
    y = fma(y, r, 1.0 / 6.0);
    y = fma(y, r, 0.5);
    y = fma(y, r, 1.0);
    y = fma(y, r, 1.0);
    return ldexp(y, static_cast<int>(n));
}

// The rank of this lane's group among the row's (LPG lanes each), and whether another
// group has the same score.
template <int LPG, int D = 1>
__device__ __forceinline__ void group_rank(float g, int& rank, bool& same) {
    if constexpr (D * LPG < 16) {
        const float o = dppf<ROW_ROR + D * LPG>(g);
        rank += o > g ? 1 : 0;
        same = same || o == g;
        group_rank<LPG, D + 1>(g, rank, same);
    }
}

// D: places of a lane that can be looked at, k + 3 or all of its NE.  vec: quads of logits and biases are aligned.
template <bool BF16, int NE, int D>
__global__ void __launch_bounds__(SR_WAVES* WAVE) score_route_rows_kernel(ScoreParams p, bool vec, int lpg) {
    extern __shared__ double choice_lds[];
    __shared__ int32_t sel[SR_WAVES][4][16];
    const int wv = threadIdx.x / WAVE, lane = threadIdx.x & (WAVE - 1);
    const int row = lane >> 4, j = lane & 15, e0 = j * NE;
    const int t0 = (blockIdx.x * SR_WAVES + wv) * 4;
    if (t0 >= p.T) return;   // whole wavefronts leave
    const int E = p.E;
    const bool soft = p.score == MOE355_SCORE_SOFTMAX;
    const int64_t at = static_cast<int64_t>(min(t0 + row, p.T - 1)) * p.stride;

    // All loads of a lane in flight together: places past the row's end read its last
    // experts and are replaced.
    float l[NE], b[NE];
    if (vec) {   // E is a multiple of 4
#pragma unroll
        for (int q = 0; q < NE; q += 4) {
            const int64_t from = at + min(e0 + q, E - 4);
            if constexpr (BF16) {
                const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.logits) + from);
                l[q] = __uint_as_float(v.x << 16);
                l[q + 1] = __uint_as_float(v.x & 0xFFFF0000u);
                l[q + 2] = __uint_as_float(v.y << 16);
                l[q + 3] = __uint_as_float(v.y & 0xFFFF0000u);
            } else {
                const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + from);
                l[q] = v.x;
                l[q + 1] = v.y;
                l[q + 2] = v.z;
                l[q + 3] = v.w;
            }
        }
        if (p.bias) {
#pragma unroll
            for (int q = 0; q < NE; q += 4) {
                const float4 v = *reinterpret_cast<const float4*>(p.bias + min(e0 + q, E - 4));
                b[q] = v.x;
                b[q + 1] = v.y;
                b[q + 2] = v.z;
                b[q + 3] = v.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const int64_t from = at + min(e0 + i, E - 1);
            l[i] = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p.logits)[from])
                        : static_cast<const float*>(p.logits)[from];
        }
        if (p.bias) {
#pragma unroll
            for (int i = 0; i < NE; ++i) b[i] = p.bias[min(e0 + i, E - 1)];
        }
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        l[i] = e0 + i < E ? l[i] : -3.0e38f;
        b[i] = p.bias && e0 + i < E ? b[i] : 0.0f;
    }
    // infinities and NaN (also where a lane's product with 0 shows them), large biases
    float odd = 0.0f, bmax = 0.0f;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
        odd = fmaf(l[i], 0.0f, odd);
        odd = fmaf(b[i], 0.0f, odd);
        bmax = fmaxf(bmax, __builtin_fabsf(b[i]));
    }
    bool fail = !(odd == 0.0f) || bmax >= 64.0f;

    float s[NE], mx = 0.0f, es = 5e-7f, total = 1.0f;   // errors: see route_fp32
    if (soft) {
        mx = l[0];
#pragma unroll
        for (int i = 1; i < NE; ++i) mx = fmaxf(mx, l[i]);
        mx = row_all_f32(mx, [](float x, float y) { return fmaxf(x, y); });
        fail = fail || mx < -1.0e38f;   // the filler of short rows would count
        total = 0.0f;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            s[i] = exp_fast(l[i] - mx);
            total += s[i];
        }
        total = row_all_f32(total, [](float x, float y) { return x + y; });
        const float r = 1.0f / total;
#pragma unroll
        for (int i = 0; i < NE; ++i) s[i] *= r;
        es = 1.5e-6f * r;
    } else {
#pragma unroll
        for (int i = 0; i < NE; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + exp_fast(-l[i]));
    }
    // keys: the choice without its last bits (1.9e-6 of it at NE = 16) and the place from the end
    uint32_t key[NE];
#pragma unroll
    for (int i = 0; i < NE; ++i)
        key[i] = (f32_order_key(e0 + i < E ? s[i] + b[i] : -3.0e38f) & ~static_cast<uint32_t>(NE - 1)) |
                 static_cast<uint32_t>(NE - 1 - i);
    constexpr uint32_t NONE = 0x02000000u;   // keys of the filler and 0 are below, those of choices above
    auto value = [](uint32_t k) {
        k &= ~static_cast<uint32_t>(NE - 1);
        return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
    };

    bool in_kept = true;
    if (lpg) {
        uint32_t a1 = key[0], a2 = 0u;
#pragma unroll
        for (int i = 1; i < NE; ++i) {
            a2 = max(a2, min(a1, key[i]));
            a1 = max(a1, key[i]);
        }
        auto merge = [&](uint32_t o1, uint32_t o2) {
            a2 = max(min(a1, o1), max(a2, o2));
            a1 = max(a1, o1);
        };
        if (lpg >= 2) merge(dpp_u32<QP1>(a1), dpp_u32<QP1>(a2));
        if (lpg >= 4) merge(dpp_u32<QP2>(a1), dpp_u32<QP2>(a2));
        if (lpg >= 8) merge(dpp_u32<HALF_MIRROR>(a1), dpp_u32<HALF_MIRROR>(a2));
        const bool group = e0 < E;
        const float g = group ? value(a1) + value(a2) : -2.0e38f;
        int rank = 0;
        bool same = false;
        if (lpg == 1) group_rank<1>(g, rank, same);
        else if (lpg == 2) group_rank<2>(g, rank, same);
        else if (lpg == 4) group_rank<4>(g, rank, same);
        else group_rank<8>(g, rank, same);
        const bool kept = group && rank < p.topk_group;
        const float low = row_all_f32(kept ? g : 3.0e38f, [](float x, float y) { return fminf(x, y); });
        const float high = row_all_f32(group && !kept ? g : -3.0e38f, [](float x, float y) { return fmaxf(x, y); });
        // Four scores' errors; with choices below m: the keys' lost bits, always towards
        // minus infinity, 2 * 15 * 2^-23 m between two groups' sums, and the roundings of
        // four choices (2^-24 m each) and two sums (2^-24 2 m each), 4.1e-6 m in all.
        const float m = 1.0f + row_all_f32(bmax, [](float x, float y) { return fmaxf(x, y); });
        fail = fail || (group && same) || !(low - high > 4.0f * es + 4.5e-6f * m);
#pragma unroll
        for (int i = 0; i < NE; ++i) key[i] = kept ? key[i] : 0u;
        in_kept = kept;
    }

    // descending merge sort network (odd-even merges)
#pragma unroll
    for (int w = 1; w < NE; w *= 2)
#pragma unroll
        for (int d = w; d >= 1; d /= 2)
#pragma unroll
            for (int x = d % w; x + d < NE; x += 2 * d)
#pragma unroll
                for (int i = 0; i < d; ++i)
                    if (x + i + d < NE && (x + i) / (2 * w) == (x + i + d) / (2 * w)) {
                        const uint32_t hi = max(key[x + i], key[x + i + d]), lo = min(key[x + i], key[x + i + d]);
                        key[x + i] = hi;
                        key[x + i + d] = lo;
                    }

    const uint64_t rowbits = 0xFFFFull << (16 * row);
    const uint64_t below = rowbits & ((1ull << lane) - 1);
    uint32_t my_top = 0u;
    for (int r = 0; r < p.k + 2; ++r) {
        const uint32_t head = key[0] & ~static_cast<uint32_t>(NE - 1);
        const uint32_t top = row_all_u32(head, [](uint32_t x, uint32_t y) { return max(x, y); });
        const uint64_t holders = __ballot(head == top);
        const bool own = head == top && top >= NONE && (holders & below) == 0;
        if (own) sel[wv][row][r] = e0 + NE - 1 - static_cast<int>(key[0] & (NE - 1));
        my_top = j == r ? top : my_top;
        const uint32_t moved = own ? 0xFFFFFFFFu : 0u;
#pragma unroll
        for (int q = 0; q + 1 < D; ++q) key[q] = (key[q] & ~moved) | (key[q + 1] & moved);
        key[D - 1] &= ~moved;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wavefront's own LDS writes
    // Lanes 0 to k + 1: the candidates, from which fp64 takes k.  All that is left is below
    // the largest head, give or take its error.
    const bool cand = my_top >= NONE && j < p.k + 2;
    const uint32_t left = row_all_u32(key[0], [](uint32_t x, uint32_t y) { return max(x, y); });
    const int e = cand ? sel[wv][row][j] : E - 1;
    const float le = BF16 ? bf16_to_f32(static_cast<const uint16_t*>(p.logits)[at + e])
                          : static_cast<const float*>(p.logits)[at + e];
    const float be = p.bias ? p.bias[e] : 0.0f;
    fail = fail || (j < p.k && !cand);

    // scores in fp64
    double sc;
    if (soft) {
        sc = exp_f64(static_cast<double>(le) - static_cast<double>(mx));
        if (p.renorm && !p.bias) {
            // the row's sum cancels but for the 1e-20 beside it, where fp32 does as long as the
            // chosen hold some mass, and does not change the order
            const float mass = row_all_f32(cand ? static_cast<float>(sc) : 0.0f, [](float x, float y) { return fmaxf(x, y); });
            fail = fail || !(mass > 1e-6f);
            sc /= static_cast<double>(total);
        } else {
            double z = 0.0;
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (e0 + i < E) z += exp_f64(static_cast<double>(l[i]) - static_cast<double>(mx));
            sc /= row_sum_f64(z);
        }
    } else {
        sc = 1.0 / (1.0 + exp_f64(-static_cast<double>(le)));
    }

    // The candidates' order: mostly that of the keys.  Two that are not equal in logit and
    // bias have to be further apart than two evaluations in fp64 can differ.
    const double choice = sc + static_cast<double>(be);
    auto order = [&](double oc, float ol, float ob, int oe, bool there, bool& before) {
        const bool equal = ol == le && ob == be;
        const double apart = 1e-14 * (__builtin_fabs(oc) + __builtin_fabs(choice) + __builtin_fabsf(ob) + __builtin_fabsf(be));
        before = there && (equal ? oe < e : oc > choice);
        return !there || equal || __builtin_fabs(oc - choice) > apart;
    };
    int rank = j;
    {
        const uint64_t u = __builtin_bit_cast(uint64_t, choice);
        const uint64_t o = static_cast<uint64_t>(dpp_u32<ROW_SHL1>(static_cast<uint32_t>(u >> 32))) << 32 |
                           dpp_u32<ROW_SHL1>(static_cast<uint32_t>(u));
        const bool there = dpp_u32<ROW_SHL1>(cand ? 1u : 0u) != 0u && cand;
        bool swapped;
        const bool clear = order(__builtin_bit_cast(double, o), dppf<ROW_SHL1>(le), dppf<ROW_SHL1>(be),
                                 static_cast<int>(dpp_u32<ROW_SHL1>(static_cast<uint32_t>(e))), there, swapped);
        fail = fail || !clear;
        if (__ballot(swapped)) {
            rank = 0;
            for (int d = 1; d < 16; ++d) {
                const int src = (lane & ~15) | ((j + d) & 15);
                bool before;
                const double oc = __shfl(choice, src, WAVE);
                const float ol = __shfl(le, src, WAVE), ob = __shfl(be, src, WAVE);
                const int oe = __shfl(e, src, WAVE), there2 = __shfl(cand ? 1 : 0, src, WAVE);
                const bool apart = order(oc, ol, ob, oe, there2 && cand, before);
                fail = fail || !apart;
                rank += before ? 1 : 0;
            }
        }
    }
    const bool chosen = cand && rank < p.k;
    const float rest = value(left);
    // two scores' errors, the keys' lost bits (1.8e-6 of the value), roundings
    const float near = 2.0f * es + 4.2e-6f * fmaxf(__builtin_fabsf(rest), __builtin_fabsf(static_cast<float>(choice)));
    const uint64_t tight = __ballot(chosen && left >= NONE && !(static_cast<float>(choice) - rest > near));
    if (tight) {
        // Equal logits may run on behind the candidates (bf16 has few values); their ids are
        // higher.  Everything else that could belong to the chosen has to be a candidate.
        const uint64_t last = __ballot(chosen && rank == p.k - 1) & rowbits;
        const int src = last ? __ffsll(static_cast<unsigned long long>(last)) - 1 : lane;
        const float lk = __shfl(le, src, WAVE), bk = __shfl(be, src, WAVE);
        const float ck = __shfl(static_cast<float>(choice), src, WAVE);
        const float limit = ck - 2.0f * es - 4.4e-6f * __builtin_fabsf(ck);
        int others = cand && value(my_top) > limit && !(le == lk && be == bk) ? -1 : 0;
#pragma unroll
        for (int i = 0; i < NE; ++i)
            others += in_kept && e0 + i < E && value(f32_order_key(s[i] + b[i])) > limit && !(l[i] == lk && b[i] == bk) ? 1 : 0;
        others = static_cast<int>(row_all_u32(static_cast<uint32_t>(others), [](uint32_t x, uint32_t y) { return x + y; }));
        fail = fail || ((tight & rowbits) != 0 && others != 0);
    }

    if (p.renorm) sc = sc / (row_sum_f64(chosen ? sc : 0.0) + 1e-20);
    const uint64_t failed = __ballot(fail);
    if (chosen && t0 + row < p.T && (failed & rowbits) == 0) {
        p.ids[static_cast<int64_t>(t0 + row) * p.k + rank] = e;
        p.w[static_cast<int64_t>(t0 + row) * p.k + rank] = static_cast<float>(sc * static_cast<double>(p.scale));
    }
    for (int r = 0; r < 4; ++r)
        if ((failed >> (16 * r) & 0xFFFFull) && t0 + r < p.T)
            route_fp64<BF16, NE / 4>(p, t0 + r, choice_lds + static_cast<int64_t>(wv) * E);
}

template <bool BF16>
void launch_score_route(const ScoreParams& p, hipStream_t stream) {
    const unsigned blocks = (static_cast<unsigned>(p.T) + SR_WAVES - 1) / SR_WAVES;
    const bool limit = p.topk_group < p.n_group;
    const size_t lds = limit ? SR_WAVES * static_cast<size_t>(p.E) * sizeof(double) : 0;
    const int npl = (p.E + WAVE - 1) / WAVE;
    const int NPL = npl <= 1 ? 1 : npl <= 2 ? 2 : npl <= 4 ? 4 : SR_MAX_NPL;
    // the fp32 pass gives lane l experts [l NPL, l NPL + NPL); a group limit has to fall
    // on whole lanes, a power of two of them
    const int gsize = p.E / p.n_group, lpg = limit ? gsize / NPL : 0;
    const bool fast = !limit || (gsize % NPL == 0 && (lpg & (lpg - 1)) == 0);
    const int width = BF16 ? 2 * NPL : NPL >= 4 ? 16 : 4 * NPL;   // alignment of a lane's load
    const bool vec = p.E % NPL == 0 && p.stride * (BF16 ? 2 : 4) % width == 0 &&
                     reinterpret_cast<uintptr_t>(p.logits) % width == 0;
    // up to 256 experts and 14 choices: four tokens per wavefront, lane j of a row with
    // experts [j NE, j NE + NE)
    const int NE = p.E <= 64 ? 4 : p.E <= 128 ? 8 : 16, lpg_rows = limit ? gsize / NE : 0;
    if (p.E <= 256 && p.k <= 14 && (!limit || (gsize % NE == 0 && (lpg_rows & (lpg_rows - 1)) == 0))) {
        const bool quads = p.E % 4 == 0 && p.stride % 4 == 0 &&
                           reinterpret_cast<uintptr_t>(p.logits) % (BF16 ? 8 : 16) == 0 &&
                           reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
        const unsigned groups = (static_cast<unsigned>(p.T) + 4 * SR_WAVES - 1) / (4 * SR_WAVES);
        auto kr = NE == 4   ? score_route_rows_kernel<BF16, 4, 4>
                  : NE == 8 ? score_route_rows_kernel<BF16, 8, 8>
                  : p.k <= 8 ? score_route_rows_kernel<BF16, 16, 11>
                             : score_route_rows_kernel<BF16, 16, 16>;
        kr<<<groups, SR_WAVES * WAVE, lds, stream>>>(p, quads, lpg_rows);
        return;
    }
    auto k = NPL == 1 ? score_route_kernel<BF16, 1>
             : NPL == 2 ? score_route_kernel<BF16, 2>
             : NPL == 4 ? score_route_kernel<BF16, 4>
                        : score_route_kernel<BF16, SR_MAX_NPL>;
    k<<<blocks, SR_WAVES * WAVE, lds, stream>>>(p, fast, vec, lpg);
}

}  // namespace
}  // namespace moe355

using namespace moe355;

extern "C" moe355_status moe355_route_scored(const moe355_router_desc* r, const void* logits,
                                             int32_t logits_type, int64_t logits_stride,
                                             const float* bias, int32_t T, int32_t* topk_ids,
                                             float* topk_w, hipStream_t stream) {
    MOE355_REQUIRE(r, MOE355_EINVAL, "route_scored: null router descriptor");
    const int E = r->n_experts, k = r->top_k;
    MOE355_REQUIRE(E >= 1 && k >= 1 && k <= E, MOE355_EINVAL, "route_scored: E=%d k=%d", E, k);
    MOE355_REQUIRE(E <= WAVE * SR_MAX_NPL && k <= 32, MOE355_ENOTSUP,
                   "route_scored: E=%d (at most %d), k=%d (at most 32)", E, WAVE * SR_MAX_NPL, k);
    MOE355_REQUIRE(r->score == MOE355_SCORE_SOFTMAX || r->score == MOE355_SCORE_SIGMOID, MOE355_EINVAL,
                   "route_scored: score=%d", r->score);
    MOE355_REQUIRE(r->n_group >= 1 && r->topk_group >= 1 && r->topk_group <= r->n_group &&
                       E % r->n_group == 0,
                   MOE355_EINVAL, "route_scored: n_group=%d topk_group=%d (E=%d)", r->n_group,
                   r->topk_group, E);
    MOE355_REQUIRE(r->n_group <= SR_MAX_GROUPS, MOE355_ENOTSUP, "route_scored: n_group=%d (at most %d)",
                   r->n_group, SR_MAX_GROUPS);
    MOE355_REQUIRE(r->n_group == 1 || E / r->n_group >= 2, MOE355_ENOTSUP,
                   "route_scored: groups of %d expert", E / r->n_group);
    MOE355_REQUIRE(k <= r->topk_group * (E / r->n_group), MOE355_EINVAL,
                   "route_scored: k=%d exceeds the kept groups' %d experts", k,
                   r->topk_group * (E / r->n_group));
    MOE355_REQUIRE(r->scale == r->scale && __builtin_fabsf(r->scale) < __builtin_inff(), MOE355_EINVAL,
                   "route_scored: scale is not finite");
    MOE355_REQUIRE(logits_type == MOE355_F32 || logits_type == MOE355_BF16, MOE355_EINVAL,
                   "route_scored: logits_type=%d", logits_type);
    MOE355_REQUIRE(T >= 0, MOE355_EINVAL, "route_scored: T=%d", T);
    MOE355_REQUIRE(T <= 1 || logits_stride >= E, MOE355_EINVAL, "route_scored: row stride %lld < E=%d",
                   static_cast<long long>(logits_stride), E);
    if (T == 0) return ok();
    MOE355_REQUIRE(logits && topk_ids && topk_w, MOE355_EINVAL, "route_scored: null pointer");
    const ScoreParams p{logits, logits_stride, bias, T, E, k, r->score, r->n_group, r->topk_group,
                        r->renorm, r->scale, topk_ids, topk_w};
    if (logits_type == MOE355_BF16) launch_score_route<true>(p, stream);
    else launch_score_route<false>(p, stream);
    return check_launch("route_scored");
}
