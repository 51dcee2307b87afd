// Routing by scores: s = softmax(l) or sigmoid(l) in fp64, selection by s + bias
// (the bias balances the experts' load and never enters a weight), group limit,
// top-k, weights from the unbiased scores.
//
// One wavefront per token.  Lane l owns experts [l*npl, l*npl + npl), npl =
// ceil(E / 64) <= 8.  Decisions are made in fp64, so that two choices that differ
// by more than a few 1e-16 rank the same here as in any other fp64 evaluation;
// equal choices go to the lower id.
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

template <bool BF16, int NPL>
__global__ void __launch_bounds__(SR_WAVES* WAVE) score_route_kernel(ScoreParams p) {
    extern __shared__ double choice_lds[];   // [SR_WAVES][E], used when groups limit the choice
    const int lane = threadIdx.x & (WAVE - 1), wv = threadIdx.x / WAVE;
    const int t = blockIdx.x * SR_WAVES + wv;
    if (t >= p.T) return;   // whole wavefronts leave; there is no block barrier below
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
        double* c = choice_lds + static_cast<int64_t>(wv) * E;
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

template <bool BF16>
void launch_score_route(const ScoreParams& p, hipStream_t stream) {
    const unsigned blocks = (static_cast<unsigned>(p.T) + SR_WAVES - 1) / SR_WAVES;
    const size_t lds = p.topk_group < p.n_group ? SR_WAVES * static_cast<size_t>(p.E) * sizeof(double) : 0;
    const int npl = (p.E + WAVE - 1) / WAVE;
    auto k = npl <= 1 ? score_route_kernel<BF16, 1>
             : npl <= 2 ? score_route_kernel<BF16, 2>
             : npl <= 4 ? score_route_kernel<BF16, 4>
                        : score_route_kernel<BF16, SR_MAX_NPL>;
    k<<<blocks, SR_WAVES * WAVE, lds, stream>>>(p);
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
