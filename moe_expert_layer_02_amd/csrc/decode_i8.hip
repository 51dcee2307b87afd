// Decode expert FFN over int8 experts: out[t] = sum_j w[t, j] down_e(silu(gate_e
// x_t) (up_e x_t)), both products in int8 with one scale per row of activations
// and one per weight row; at most 256 routed pairs per call.
//
// v_mfma_i32_16x16x64_i8 with the weights as the first operand (16 rows x 64
// inputs) and up to 16 pairs of the expert as the second, so one pass over an
// expert's bytes serves its pairs; bound by the weight bytes of the distinct
// experts (16 tokens of 6 experts, H 4096, I 2048: 355 us, 5.7 TB/s of expert bytes), and
// by the chain of launches and loads where those are few (one token of 8 experts, H 2048,
// I 512: 12.5 us for 25 MB).
//
// Two kernels: gate/up (h in bf16 by pair) and down with the combine.  A down block
// owns 16 output rows of every token: the pairs' results meet in LDS and are summed
// j ascending, so no atomics and a deterministic output.  A small call quantises x
// and h inside them, every block for itself (the rows are read from the L2 while
// the weights are on their way); otherwise each has a launch of its own before it,
// since a block would spend longer on all rows than the launch takes.
#include "i8.h"

namespace moe355 {
namespace {

constexpr int MAX_PAIRS = 256;
constexpr int MAX_EXPERTS_I8 = 1024;
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
    const uint16_t* x;
    int early;                  // weights are requested before the pairs are known
    int lds_rows;               // bytes of one quantised row in LDS (0: rows are quantised already)
};

// A small call: rows quantised by every block.  Gate/up: one row per wavefront of its
// four (H = 2048, I = 512, 8 experts a token: one token 12.5 us against 13.9 with a launch
// before it, four 30.7 against 32.0; INLINE_H bounds the rows' LDS); down: at most this
// many values of h (4096: 12.5 us against 13.4; 8192 even; 16384: 27.5 against 25.5).
constexpr int INLINE_TOKENS = 4, INLINE_H = 8192, INLINE_VALUES = 12288;
// Calls of so few pairs and gate/up blocks (two per CU) request weights first: 256 blocks
// 12.5 us against 13.1, 512 20.3 against 20.9; 768 (H = 4096, I = 2048) 39.4 against 36.1.
constexpr int EARLY_PAIRS = 16, EARLY_BLOCKS = 512;

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

// N steps of 64 inputs of one operand's tile, requested at once: from k0 on, `step`
// apart.  p: this lane's row (or column) and 16-byte chunk.
template <int N>
struct Steps {
    i32x4 v[N];
    __device__ __forceinline__ void load(const void* p, int k0, int n, int step) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = k0 + i * step < n ? *reinterpret_cast<const i32x4*>(static_cast<const uint8_t*>(p) + k0 + i * step) : i32x4{};
    }
    // the products with the other operand (zero past the end on both sides)
    __device__ __forceinline__ i32x4 dot(const Steps& x, i32x4 acc) const {
#pragma unroll
        for (int i = 0; i < N; ++i) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(v[i], x.v[i], acc, 0, 0, 0);
        return acc;
    }
};

// N: steps of gate and of up that a wavefront has in flight.  A small call has few
// blocks and takes 8; where blocks queue, 4 leave room for twice the blocks per CU.
template <int N>
__global__ void __launch_bounds__(256) gate_up_i8_kernel(DecodeI8 p) {
    extern __shared__ __attribute__((aligned(16))) int8_t rows[];   // small call: the tokens' codes
    __shared__ int32_t ids[MAX_PAIRS];
    __shared__ int32_t list[MAX_PAIRS];
    __shared__ int32_t count;
    __shared__ float row_scales[INLINE_TOKENS];
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
    // In a call of few pairs the weights are requested before anything else is known
    // about the expert's pairs; in a larger one many pairs share an expert, and the first
    // of them has to be found before (loading first read 1.2 times the bytes at 96 pairs).
    const bool early = p.uniq || p.early;
    auto find_pairs = [&]() {
        __syncthreads();
        if (wv == 0) {
            const int n = pairs_of(ids, e, lane, list);
            if (lane == 0) count = n;
        }
    };
    if (!early) {
        find_pairs();
        __syncthreads();
        if (list[0] != u) return;
    }
    const uint8_t* blob = blob_of(p, e, slot);
    const int row = lane & 15, quad = lane >> 4;
    const uint8_t* wg = blob + p.q_off[0] + static_cast<int64_t>(f0 + row) * p.H + quad * 16;
    const uint8_t* wu = blob + p.q_off[1] + static_cast<int64_t>(f0 + row) * p.H + quad * 16;
    Steps<N> g0, u0;
    g0.load(wg, wv * 64, p.H, 256);
    u0.load(wu, wv * 64, p.H, 256);
    const float gs = reinterpret_cast<const float*>(blob + p.s_off[0])[f0 + (tid & 15)];
    const float us = reinterpret_cast<const float*>(blob + p.s_off[1])[f0 + (tid & 15)];
    if (early) find_pairs();
    if (p.lds_rows && wv < p.T) {
        const float s = quant_row(p.x + static_cast<int64_t>(wv) * p.H, p.H, rows + wv * p.lds_rows, lane);
        if (lane == 0) row_scales[wv] = s;
    }
    __syncthreads();
    // without lists the first pair of an expert does it
    if (count == 0 || (!p.uniq && list[0] != u)) return;
    const int n = count;
    for (int g = 0; g < n; g += 16) {
        const int tok = list[min(g + row, n - 1)] / p.k;
        const int8_t* x = (p.lds_rows ? rows + tok * p.lds_rows : p.xq + static_cast<int64_t>(tok) * p.H) + quad * 16;
        Steps<N> a, b, xs;
        xs.load(x, wv * 64, p.H, 256);
        i32x4 ga = g0.dot(xs, i32x4{}), ua = u0.dot(xs, i32x4{});
        for (int k = wv * 64 + N * 256; k < p.H; k += N * 256) {
            xs.load(x, k, p.H, 256);
            a.load(wg, k, p.H, 256);
            b.load(wu, k, p.H, 256);
            ga = a.dot(xs, ga);
            ua = b.dot(xs, ua);
        }
        part[wv][0][lane] = ga;
        part[wv][1][lane] = ua;
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
            const int pair = list[g + c], t = pair / p.k;
            p.h[static_cast<int64_t>(pair) * p.I + f0 + f] = swiglu_bf16(a, b, p.lds_rows ? row_scales[t] : p.xs[t], gs, us);
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(DN_WAVES* WAVE) down_i8_kernel(DecodeI8 p) {
    extern __shared__ __attribute__((aligned(16))) int8_t rows[];   // small call: the pairs' codes
    __shared__ int32_t ids[MAX_PAIRS];
    __shared__ int32_t item[MAX_PAIRS];
    __shared__ int32_t first[MAX_EXPERTS_I8];   // the first pair of every expert named
    __shared__ int32_t n_items;
    __shared__ int32_t lists[DN_WAVES][MAX_PAIRS];
    __shared__ float hscale[MAX_PAIRS];
    __shared__ float y[MAX_PAIRS][16];
    const int tid = threadIdx.x, lane = tid & (WAVE - 1);
    const int wv = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int r0 = blockIdx.x * 16;
    int my_id = -1;
    if (tid < MAX_PAIRS) {
        my_id = tid < p.pairs ? p.ids[tid] : -1;
        if (my_id >= p.E || my_id < 0) my_id = -1;
        ids[tid] = my_id;
        if (my_id >= 0) first[my_id] = MAX_PAIRS;
    }
    __syncthreads();
    if (!p.uniq) {
        if (my_id >= 0) atomicMin(&first[my_id], tid);
        __syncthreads();
        if (wv == 0) {   // the experts in the order of their first pairs
            int n = 0;
#pragma unroll
            for (int g = 0; g < MAX_PAIRS; g += WAVE) {
                const int id = ids[g + lane];
                const bool is = id >= 0 && first[id] == g + lane;
                const uint64_t m = __ballot(is);
                if (is) item[n + __popcll(m & ((1ull << lane) - 1))] = id;
                n += __popcll(m);
            }
            if (lane == 0) n_items = n;
        }
        __syncthreads();
    }
    const int items = p.uniq ? min(p.counts[0], p.capacity) : n_items;
    const int row = lane & 15, quad = lane >> 4;
    auto blob_of_item = [&](int u) {   // null: none
        const int e = u < items ? (p.uniq ? p.uniq[u] : item[u]) : -1;
        if (e < 0 || e >= p.E) return static_cast<const uint8_t*>(nullptr);
        return blob_of(p, e, p.uniq ? p.plan[u].x : -1);
    };
    auto tile_of = [&](const uint8_t* blob) {   // this lane's row and chunk
        return blob + p.q_off[2] + static_cast<int64_t>(r0 + row) * p.I + quad * 16;
    };
    // A wavefront's items are one stream of chunks of 8 steps; the next chunk (of this
    // item or the first of the next) is requested before this one's products.
    const uint8_t *blob = blob_of_item(wv), *w = blob ? tile_of(blob) : nullptr;
    constexpr int CHUNK = 8;
    Steps<CHUNK> cur;
    if (w) cur.load(w, 0, p.I, 64);
    if (p.lds_rows) {
        for (int q = wv; q < p.pairs; q += DN_WAVES) {
            if (ids[q] < 0) continue;
            const float s = quant_row(p.h + static_cast<int64_t>(q) * p.I, p.I, rows + q * p.lds_rows, lane);
            if (lane == 0) hscale[q] = s;
        }
        __syncthreads();
    }
    for (int u = wv; u < items; u += DN_WAVES) {
        const uint8_t *next_blob = blob_of_item(u + DN_WAVES), *next_w = next_blob ? tile_of(next_blob) : nullptr;
        if (w) {
            const int e = p.uniq ? p.uniq[u] : item[u];
            const int n = pairs_of(ids, e, lane, lists[wv]);
            __builtin_amdgcn_wave_barrier();
            const float4 ds = *reinterpret_cast<const float4*>(blob + p.s_off[2] + (r0 + quad * 4) * 4);
            auto x_of = [&](int pair) {
                return (p.lds_rows ? rows + pair * p.lds_rows : p.hq + static_cast<int64_t>(pair) * p.I) + quad * 16;
            };
            auto put = [&](int g, int pair, i32x4 acc) {
                const float s = p.lds_rows ? hscale[pair] : p.hs[pair];
                if (g + row < n)
                    *reinterpret_cast<float4*>(&y[pair][quad * 4]) =
                        make_float4(static_cast<float>(acc[0]) * s * ds.x, static_cast<float>(acc[1]) * s * ds.y,
                                    static_cast<float>(acc[2]) * s * ds.z, static_cast<float>(acc[3]) * s * ds.w);
            };
            const int pair0 = n ? lists[wv][min(row, n - 1)] : 0;   // n = 0: lists of other ids; nothing is kept
            i32x4 acc = {};
            for (int k = 0; k < p.I; k += CHUNK * 64) {
                // loads complete in order: the columns first, or they would wait for the weights
                Steps<CHUNK> next, x;
                x.load(x_of(pair0), k, p.I, 64);
                __builtin_amdgcn_sched_barrier(0);
                if (k + CHUNK * 64 < p.I) next.load(w, k + CHUNK * 64, p.I, 64);
                else if (next_w) next.load(next_w, 0, p.I, 64);
                __builtin_amdgcn_sched_barrier(0);
                acc = cur.dot(x, acc);
                cur = next;
            }
            if (n) put(0, pair0, acc);
            for (int g = 16; g < n; g += 16) {   // more than 16 pairs: the tile again, from the caches
                const int pair = lists[wv][min(g + row, n - 1)];
                i32x4 more = {};
                for (int k = 0; k < p.I; k += CHUNK * 64) {
                    Steps<CHUNK> a, x;
                    x.load(x_of(pair), k, p.I, 64);
                    a.load(w, k, p.I, 64);
                    more = a.dot(x, more);
                }
                put(g, pair, more);
            }
        } else if (next_w) {
            cur.load(next_w, 0, p.I, 64);
        }
        w = next_w;
        blob = next_blob;
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
    p.x = static_cast<const uint16_t*>(x_bf16);
    // rows in LDS lie 16 bytes further apart than their length, so that columns fall in
    // different banks
    const bool inline_x = T <= INLINE_TOKENS && p.H <= INLINE_H;
    if (!inline_x) {
        st = launch_quant_rows(x_bf16, p.H, T, p.H, xq, p.H, xs, stream, "expert_ffn_decode_i8 quantise x");
        if (st) return st;
    }
    const int items = exp ? (pairs < p.E ? pairs : p.E) : pairs;
    p.lds_rows = inline_x ? p.H + 16 : 0;
    p.early = pairs <= EARLY_PAIRS && p.I / 16 * items <= EARLY_BLOCKS;
    auto gate_up = p.early ? gate_up_i8_kernel<8> : gate_up_i8_kernel<4>;
    gate_up<<<dim3(p.I / 16, items), 256, static_cast<size_t>(p.lds_rows) * T, stream>>>(p);
    st = check_launch("expert_ffn_decode_i8 gate_up");
    if (st) return st;
    const bool inline_h = pairs * p.I <= INLINE_VALUES;
    if (!inline_h) {
        st = launch_quant_rows(p.h, p.I, pairs, p.I, hq, p.I, hs, stream, "expert_ffn_decode_i8 quantise h");
        if (st) return st;
    }
    p.lds_rows = inline_h ? p.I + 16 : 0;
    down_i8_kernel<<<p.H / 16, DN_WAVES * WAVE, static_cast<size_t>(p.lds_rows) * pairs, stream>>>(p);
    return check_launch("expert_ffn_decode_i8 down");
}
