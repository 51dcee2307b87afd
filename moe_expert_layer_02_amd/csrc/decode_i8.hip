// Decode expert FFN over int8 experts: out[t] = sum_j w[t, j] down_e(silu(gate_e
// x_t) (up_e x_t)), both products in int8 with one scale per row of activations
// and one per weight row; at most 256 routed pairs per call.
//
// v_mfma_i32_16x16x64_i8 with the weights as the first operand (16 rows x 64
// inputs) and up to 16 pairs of the expert as the second, so one pass over an
// expert's bytes serves its pairs; bound by the weight bytes of the distinct
// experts.  Four launches: quantise x, gate/up (h in bf16 by pair), quantise h,
// down with the combine.  A down block owns 16 output rows of every token: the
// pairs' results meet in LDS and are summed j ascending, so no atomics and a
// deterministic output.
#include "i8.h"

namespace moe355 {
namespace {

constexpr int MAX_PAIRS = 256;
constexpr int DN_WAVES = 8;

struct DecodeI8 {
    const int32_t* ids;
    const float* topk_w;
    const uint8_t* pool;        // this layer's experts
    const uint8_t* slots;       // cache slots (null: everything from the pool)
    int n_slots;
    const int32_t* uniq;        // the call's lists (null: grouped here from ids)
    const int32_t* counts;
    const int4* plan;
    int capacity;
    int64_t S;
    int64_t q_off[3], s_off[3];
    int T, k, H, I, E, pairs;
    const int8_t* xq;
    const float* xs;
    uint16_t* h;
    const int8_t* hq;
    const float* hs;
    uint16_t* out;
};

// Where an expert's bytes are: its cache slot, or the pool.
__device__ __forceinline__ const uint8_t* blob_of(const DecodeI8& p, int e, int slot) {
    return p.slots && slot >= 0 && slot < p.n_slots ? p.slots + static_cast<int64_t>(slot) * p.S
                                                    : p.pool + static_cast<int64_t>(e) * p.S;
}

// Pairs of expert e in ascending order into list; their number.  One wavefront;
// ids: the call's ids (LDS), -1 past the pairs.
__device__ __forceinline__ int pairs_of(const int32_t* ids, int e, int lane, int32_t* list) {
    int n = 0;
#pragma unroll
    for (int g = 0; g < MAX_PAIRS / WAVE; ++g) {
        const bool hit = ids[g * WAVE + lane] == e;
        const uint64_t m = __ballot(hit);
        if (hit) list[n + __popcll(m & ((1ull << lane) - 1))] = g * WAVE + lane;
        n += __popcll(m);
    }
    return n;
}

// One 16-row tile against one group of 16 columns over inputs [k0, k1) in steps
// of 64, `step` apart.  w: this lane's row and 16-byte chunk; x: this lane's
// column and chunk.
__device__ __forceinline__ i32x4 dot_tile(const uint8_t* w, const int8_t* x, int k0, int k1, int step, i32x4 acc) {
#pragma unroll 8
    for (int k = k0; k < k1; k += step)
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const i32x4*>(w + k),
                                                    *reinterpret_cast<const i32x4*>(x + k), acc, 0, 0, 0);
    return acc;
}

__global__ void __launch_bounds__(256) gate_up_i8_kernel(DecodeI8 p) {
    __shared__ int32_t ids[MAX_PAIRS];
    __shared__ int32_t list[MAX_PAIRS];
    __shared__ int32_t count;
    __shared__ i32x4 part[4][2][WAVE];
    const int tid = threadIdx.x, lane = tid & (WAVE - 1);
    const int wv = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int u = blockIdx.y, f0 = blockIdx.x * 16;
    int e, slot = -1;
    if (p.uniq) {
        if (u >= p.counts[0]) return;
        e = p.uniq[u];
        slot = p.plan[u].x;
    } else {
        e = p.ids[u];
    }
    if (e < 0 || e >= p.E) return;
    ids[tid] = tid < p.pairs ? p.ids[tid] : -1;
    __syncthreads();
    if (wv == 0) {
        const int n = pairs_of(ids, e, lane, list);
        if (lane == 0) count = n;
    }
    __syncthreads();
    // without lists the first pair of an expert does it
    if (count == 0 || (!p.uniq && list[0] != u)) return;
    const int n = count;
    const uint8_t* blob = blob_of(p, e, slot);
    const int row = lane & 15, quad = lane >> 4;
    const uint8_t* wg = blob + p.q_off[0] + static_cast<int64_t>(f0 + row) * p.H + quad * 16;
    const uint8_t* wu = blob + p.q_off[1] + static_cast<int64_t>(f0 + row) * p.H + quad * 16;
    const float* gs = reinterpret_cast<const float*>(blob + p.s_off[0]) + f0;
    const float* us = reinterpret_cast<const float*>(blob + p.s_off[1]) + f0;
    for (int g = 0; g < n; g += 16) {
        const int tok = list[min(g + row, n - 1)] / p.k;
        const int8_t* x = p.xq + static_cast<int64_t>(tok) * p.H + quad * 16;
        part[wv][0][lane] = dot_tile(wg, x, wv * 64, p.H, 256, i32x4{});
        part[wv][1][lane] = dot_tile(wu, x, wv * 64, p.H, 256, i32x4{});
        __syncthreads();
        // element i of lane l: row 4 (l / 16) + i, column l % 16
        const int f = tid & 15, c = tid >> 4;
        if (g + c < n) {
            const int at = (f >> 2) * 16 + c, i = f & 3;
            int a = 0, b = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                a += reinterpret_cast<const int*>(&part[w][0][at])[i];
                b += reinterpret_cast<const int*>(&part[w][1][at])[i];
            }
            const int pair = list[g + c];
            p.h[static_cast<int64_t>(pair) * p.I + f0 + f] = swiglu_bf16(a, b, p.xs[pair / p.k], gs[f], us[f]);
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(DN_WAVES* WAVE) down_i8_kernel(DecodeI8 p) {
    __shared__ int32_t ids[MAX_PAIRS];
    __shared__ int32_t item[MAX_PAIRS];
    __shared__ int32_t n_items;
    __shared__ int32_t lists[DN_WAVES][MAX_PAIRS];
    __shared__ float y[MAX_PAIRS][16];
    const int tid = threadIdx.x, lane = tid & (WAVE - 1);
    const int wv = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int r0 = blockIdx.x * 16;
    if (tid < MAX_PAIRS) {
        const int id = tid < p.pairs ? p.ids[tid] : -1;
        ids[tid] = id >= 0 && id < p.E ? id : -1;
    }
    __syncthreads();
    if (!p.uniq && wv == 0) {   // the first pair of every expert, in order
        int n = 0;
        for (int g = 0; g < p.pairs; g += WAVE) {
            const int q = g + lane, id = ids[q];
            bool first = id >= 0;
            for (int j = 0; j < q && first; ++j) first = ids[j] != id;
            const uint64_t m = __ballot(first);
            if (first) item[n + __popcll(m & ((1ull << lane) - 1))] = id;
            n += __popcll(m);
        }
        if (lane == 0) n_items = n;
    }
    __syncthreads();
    const int items = p.uniq ? min(p.counts[0], p.capacity) : n_items;
    const int row = lane & 15, quad = lane >> 4;
    for (int u = wv; u < items; u += DN_WAVES) {
        const int e = p.uniq ? p.uniq[u] : item[u];
        if (e < 0 || e >= p.E) continue;
        const uint8_t* blob = blob_of(p, e, p.uniq ? p.plan[u].x : -1);
        const int n = pairs_of(ids, e, lane, lists[wv]);
        __builtin_amdgcn_wave_barrier();
        const uint8_t* w = blob + p.q_off[2] + static_cast<int64_t>(r0 + row) * p.I + quad * 16;
        const float4 ds = *reinterpret_cast<const float4*>(blob + p.s_off[2] + (r0 + quad * 4) * 4);
        for (int g = 0; g < n; g += 16) {
            const int pair = lists[wv][min(g + row, n - 1)];
            const i32x4 acc = dot_tile(w, p.hq + static_cast<int64_t>(pair) * p.I + quad * 16, 0, p.I, 64, i32x4{});
            const float s = p.hs[pair];
            if (g + row < n)
                *reinterpret_cast<float4*>(&y[pair][quad * 4]) =
                    make_float4(static_cast<float>(acc[0]) * s * ds.x, static_cast<float>(acc[1]) * s * ds.y,
                                static_cast<float>(acc[2]) * s * ds.z, static_cast<float>(acc[3]) * s * ds.w);
        }
    }
    __syncthreads();
    for (int i = tid; i < p.T * 16; i += DN_WAVES * WAVE) {
        const int t = i / 16, r = i % 16;
        float a = 0.0f;
        for (int j = 0; j < p.k; ++j)
            if (ids[t * p.k + j] >= 0) a = fmaf(p.topk_w[t * p.k + j], y[t * p.k + j][r], a);
        p.out[static_cast<int64_t>(t) * p.H + r0 + r] = f32_to_bf16(a);
    }
}

int64_t align256(int64_t n) { return (n + 255) & ~int64_t{255}; }

struct DecodeWs {
    int64_t xq, xs, h, hq, hs, bytes;
};
DecodeWs decode_ws(const moe355_layer_desc* d, int T) {
    const int64_t pairs = static_cast<int64_t>(T) * d->top_k;
    DecodeWs w;
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t here = at;
        at += align256(n);
        return here;
    };
    w.xq = take(static_cast<int64_t>(T) * d->hidden);
    w.xs = take(4ll * T);
    w.h = take(2 * pairs * d->inter);
    w.hq = take(pairs * d->inter);
    w.hs = take(4 * pairs);
    w.bytes = at;
    return w;
}

}  // namespace

size_t decode_i8_ws_bytes(const moe355_layer_desc* d, int T) {
    return static_cast<size_t>(decode_ws(d, T).bytes);
}

}  // namespace moe355

using namespace moe355;

extern "C" moe355_status moe355_expert_ffn_decode_i8(const moe355_layer_desc* d, const void* x_bf16, int32_t T,
                                                     const int32_t* topk_ids, const float* topk_w,
                                                     const moe355_cache* cache, const uint8_t* pool, int32_t layer,
                                                     const moe355_classify_out* exp, void* out_bf16, void* ws,
                                                     size_t ws_bytes, hipStream_t stream) {
    moe355_status st = check_desc_i8(d, "expert_ffn_decode_i8");
    if (st) return st;
    MOE355_REQUIRE(T >= 0, MOE355_EINVAL, "expert_ffn_decode_i8: T=%d", T);
    if (T == 0) return ok();
    MOE355_REQUIRE(static_cast<int64_t>(T) * d->top_k <= MAX_PAIRS, MOE355_ENOTSUP,
                   "expert_ffn_decode_i8: T*k=%lld > %d", static_cast<long long>(T) * d->top_k, MAX_PAIRS);
    MOE355_REQUIRE(x_bf16 && topk_ids && topk_w && pool && out_bf16, MOE355_EINVAL,
                   "expert_ffn_decode_i8: null pointer");
    MOE355_REQUIRE(reinterpret_cast<uintptr_t>(x_bf16) % 16 == 0 && reinterpret_cast<uintptr_t>(pool) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(ws) % 256 == 0,
                   MOE355_EINVAL, "expert_ffn_decode_i8: x and pool at multiples of 16 bytes, ws of 256");
    MOE355_REQUIRE(layer >= 0, MOE355_EINVAL, "expert_ffn_decode_i8: layer=%d", layer);
    const I8Layout L = i8_layout(d);
    const int pairs = T * d->top_k;
    if (cache) {
        st = check_cache(cache);
        if (st) return st;
        MOE355_REQUIRE(exp, MOE355_EINVAL, "expert_ffn_decode_i8: a cache needs the call's lists");
        MOE355_REQUIRE(cache->n_experts == d->n_experts && layer < cache->n_layers && cache->slot_bytes == L.bytes &&
                           cache->slot_data && reinterpret_cast<uintptr_t>(cache->slot_data) % 16 == 0,
                       MOE355_EINVAL, "expert_ffn_decode_i8: cache of %d experts, %d layers, %lld-byte slots for E=%d, layer %d, S=%lld",
                       cache->n_experts, cache->n_layers, static_cast<long long>(cache->slot_bytes), d->n_experts,
                       layer, static_cast<long long>(L.bytes));
    }
    if (exp) {
        MOE355_REQUIRE(exp->uniq && exp->counts && exp->plan, MOE355_EINVAL,
                       "expert_ffn_decode_i8: null list");
        const int most = pairs < d->n_experts ? pairs : d->n_experts;
        MOE355_REQUIRE(exp->capacity >= most, MOE355_ECAPACITY,
                       "expert_ffn_decode_i8: lists of %d experts, the call may need %d", exp->capacity, most);
    }
    const DecodeWs w = decode_ws(d, T);
    MOE355_REQUIRE(ws && ws_bytes >= static_cast<size_t>(w.bytes), MOE355_ECAPACITY,
                   "expert_ffn_decode_i8: workspace %zu < %lld bytes", ws_bytes, static_cast<long long>(w.bytes));
    uint8_t* base = static_cast<uint8_t*>(ws);
    int8_t* xq = reinterpret_cast<int8_t*>(base + w.xq);
    float* xs = reinterpret_cast<float*>(base + w.xs);
    int8_t* hq = reinterpret_cast<int8_t*>(base + w.hq);
    float* hs = reinterpret_cast<float*>(base + w.hs);
    DecodeI8 p{};
    p.ids = topk_ids;
    p.topk_w = topk_w;
    p.pool = pool + static_cast<int64_t>(layer) * d->n_experts * L.bytes;
    if (cache) {
        p.slots = cache->slot_data;
        p.n_slots = cache->n_slots;
    }
    if (exp) {
        p.uniq = exp->uniq;
        p.counts = exp->counts;
        p.plan = reinterpret_cast<const int4*>(exp->plan);
        p.capacity = exp->capacity;
    }
    p.S = L.bytes;
    for (int m = 0; m < 3; ++m) {
        p.q_off[m] = L.q[m];
        p.s_off[m] = L.s[m];
    }
    p.T = T;
    p.k = d->top_k;
    p.H = d->hidden;
    p.I = d->inter;
    p.E = d->n_experts;
    p.pairs = pairs;
    p.xq = xq;
    p.xs = xs;
    p.h = reinterpret_cast<uint16_t*>(base + w.h);
    p.hq = hq;
    p.hs = hs;
    p.out = static_cast<uint16_t*>(out_bf16);
    st = launch_quant_rows(x_bf16, p.H, T, p.H, xq, p.H, xs, stream, "expert_ffn_decode_i8 quantise x");
    if (st) return st;
    const int items = exp ? (pairs < p.E ? pairs : p.E) : pairs;
    gate_up_i8_kernel<<<dim3(p.I / 16, items), 256, 0, stream>>>(p);
    st = check_launch("expert_ffn_decode_i8 gate_up");
    if (st) return st;
    st = launch_quant_rows(p.h, p.I, pairs, p.I, hq, p.I, hs, stream, "expert_ffn_decode_i8 quantise h");
    if (st) return st;
    down_i8_kernel<<<p.H / 16, DN_WAVES * WAVE, 0, stream>>>(p);
    return check_launch("expert_ffn_decode_i8 down");
}
