// Int8 matrix products on the CDNA4 matrix cores: C[m, n] = sa[m] sb[n] sum_k
// A[m, k] B[n, k], the sum exact in int32 (v_mfma_i32_32x32x32_i8), in three
// forms that share one K loop:
//   dense    C = A . B^T (moe355_matmul_i8);
//   gate/up  a grouped product over expert buckets whose epilogue forms
//            h = silu(g) u (moe355_expert_ffn_prefill_i8);
//   down     the grouped product of h, one row of y per (token, slot) pair.
//
// Tile: 128 rows x 256 weight rows per block of four wavefronts; a wavefront owns
// all 128 rows and 64 weight rows (2 column tiles of 32; eight 32x32
// accumulators).  The activations are the first operand, so an accumulator holds
// rows (tokens) in its registers and a weight row per lane.  K runs in stages of
// 64: A (8 KB) and B (16 KB) go global -> LDS by direct loads into a ring of three
// slots, two stages ahead.  Two blocks share a CU, so one block's epilogue and
// waits run under the other's products.
#include "i8.h"
#include "lds_dma.h"

namespace moe355 {
namespace {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int SLOT_A = BM * BK, SLOT = (BM + BN) * BK;   // bytes
constexpr int RING = 3;
constexpr int LOADS = SLOT / 1024 / 4;                   // direct loads per wavefront and stage
constexpr int NXCD = 8;

enum Kind { DENSE, GATE_UP, DOWN };

struct GemmParams {
    const int8_t* a;        // rows of codes
    int64_t lda;
    const float* as;
    const int8_t* b;        // dense: weight rows; grouped: expert blobs
    int64_t ldb;
    const float* bs;
    int M, N, K;            // dense sizes; grouped: N = I (gate/up) or H (down), K = H or I
    void* out;
    int out_bf16;
    int64_t ldo;
    // grouped
    int64_t S;
    int64_t q_off[2], s_off[2];
    const int32_t* perm;
    const int32_t* ids;
    const int32_t* tile_e;
    const int32_t* tile_p0;
    const int32_t* tile_rows;
    const int32_t* n_tiles;
    int pairs, k;
};

// 16-byte chunk c of LDS row r sits at position c ^ swz(r) of the row's four, so
// that the 16 rows a quarter of a read covers fall in different banks.
__device__ __forceinline__ int swz(int r) { return (r >> 2) & 3; }

// The K loop.  aoff / boff: byte offsets (from abase / bbase) of the chunk each
// lane fetches for its 2 A loads and 4 B loads of a stage; ks stages; ktail: K of
// the last stage (64, or less in the dense form).
template <int NMT>
__device__ __forceinline__ void k_loop(uint8_t* ring, uint32_t ring_lds, const void* abase, const void* bbase,
                                       const uint32_t (&aoff)[2], const uint32_t (&boff)[4], int ks, int ktail,
                                       int wv, int lane, i32x16 (&R)[4][2]) {
    const int ln = lane & 31, hh = lane >> 5;
    auto load_stage = [&](int kk, int slot) {
        const uint32_t sl = ring_lds + slot * SLOT;
        const uint32_t ko = kk * BK;
        // a chunk past the last stage's K is fetched from the row's start instead
        // (in bounds; its A side is cleared before use)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = (lane & 3) ^ swz(16 * j + lane / 4);
            const uint32_t in = kk < ks - 1 || c * 16 < ktail ? ko : static_cast<uint32_t>(-(c * 16));
            dma16(abase, aoff[j] + in, sl + (2 * wv + j) * 1024);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = (lane & 3) ^ swz(16 * j + lane / 4);
            const uint32_t in = kk < ks - 1 || c * 16 < ktail ? ko : static_cast<uint32_t>(-(c * 16));
            dma16(bbase, boff[j] + in, sl + SLOT_A + (4 * wv + j) * 1024);
        }
    };
    load_stage(0, 0);
    load_stage(min(1, ks - 1), 1);
    int slot = 0;
    for (int kk = 0; kk < ks; ++kk) {
        stage_barrier<LOADS>();   // stage kk has landed everywhere and stage kk - 1 is read out
        const int s2 = slot == 0 ? 2 : slot - 1;
        load_stage(min(kk + 2, ks - 1), s2);   // past the end the last stage again: uniform counts
        uint8_t* sp = ring + slot * SLOT;
        if (ktail < BK && kk == ks - 1) {
            for (int i = threadIdx.x; i < BM * 4; i += 256) {
                const int r = i >> 2, c = i & 3;
                if (c * 16 >= ktail)
                    *reinterpret_cast<uint4*>(sp + r * BK + ((c ^ swz(r)) << 4)) = make_uint4(0, 0, 0, 0);
            }
            __syncthreads();
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int c = 2 * s + hh;
            i32x4 b[2], a[NMT];
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) {
                const int r = 64 * wv + 32 * ct + ln;
                b[ct] = *reinterpret_cast<const i32x4*>(sp + SLOT_A + r * BK + ((c ^ swz(r)) << 4));
            }
#pragma unroll
            for (int mt = 0; mt < NMT; ++mt) {
                const int r = 32 * mt + ln;
                a[mt] = *reinterpret_cast<const i32x4*>(sp + r * BK + ((c ^ swz(r)) << 4));
            }
#pragma unroll
            for (int mt = 0; mt < NMT; ++mt)
#pragma unroll
                for (int ct = 0; ct < 2; ++ct)
                    R[mt][ct] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[mt], b[ct], R[mt][ct], 0, 0, 0);
        }
        slot = slot == 2 ? 0 : slot + 1;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // the repeated loads have landed
}

template <int KIND>
__global__ void __launch_bounds__(256, 2) gemm_i8_kernel(GemmParams p) {
    __shared__ __attribute__((aligned(1024))) uint8_t ring[RING * SLOT];
    __shared__ __attribute__((aligned(16))) float rscale[BM];
    __shared__ int32_t rrow[BM];   // gate/up: source row; down: pair id, or -1 for a row that is not stored
    const int tid = threadIdx.x, lane = tid & (WAVE - 1);
    const int wv = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int ln = lane & 31, hh = lane >> 5;
    const uint32_t ring_lds = lds_addr(ring);

    // Tiles of one XCD (block id mod 8) are consecutive: neighbours share an
    // expert's weights or activation rows in that XCD's L2.
    const int per_n = KIND == GATE_UP ? BN / 2 : BN;
    const int NT = (p.N + per_n - 1) / per_n;
    const int MT = KIND == DENSE ? (p.M + BM - 1) / BM : ld_const(p.n_tiles);
    const int64_t total = static_cast<int64_t>(MT) * NT;
    const int xcd = blockIdx.x % NXCD, at = blockIdx.x / NXCD;
    const int64_t t0 = total * xcd / NXCD, t1 = total * (xcd + 1) / NXCD;
    if (t0 + at >= t1) return;
    const int64_t t = t0 + at;
    const int mtile = static_cast<int>(t / NT), nt = static_cast<int>(t % NT);

    const void* abase;
    const void* bbase;
    const float* bs[2];
    int rows, m0 = 0, e = 0, p0 = 0;
    if (KIND == DENSE) {
        m0 = mtile * BM;
        rows = min(BM, p.M - m0);
        abase = uniform_ptr(p.a + static_cast<int64_t>(m0) * p.lda);
        bbase = uniform_ptr(p.b + static_cast<int64_t>(nt) * BN * p.ldb);
        bs[0] = p.bs;
    } else {
        e = ld_const(p.tile_e + mtile);
        p0 = ld_const(p.tile_p0 + mtile);
        rows = ld_const(p.tile_rows + mtile);
        const int8_t* blob = p.b + static_cast<int64_t>(e) * p.S;
        abase = uniform_ptr(KIND == GATE_UP ? p.a : p.a + static_cast<int64_t>(p0) * p.lda);
        bbase = uniform_ptr(blob + p.q_off[0] + (KIND == DOWN ? static_cast<int64_t>(nt) * BN * p.ldb : 0));
        bs[0] = reinterpret_cast<const float*>(blob + p.s_off[0]);
        bs[1] = reinterpret_cast<const float*>(blob + p.s_off[1]);
    }
    const int nmt = __builtin_amdgcn_readfirstlane((rows + 31) / 32);

    if (tid < BM) {
        const int r = min(tid, rows - 1);
        if (KIND == DENSE) {
            rscale[tid] = p.as[m0 + r];
        } else {
            // a position whose pair is not one of this expert's (ids changed or out of
            // range) is computed from row 0 and never used
            int pair = p.perm[p0 + r];
            if (pair < 0 || pair >= p.pairs || p.ids[pair] != e) pair = -1;
            if (KIND == GATE_UP) {
                const int tok = pair < 0 ? 0 : pair / p.k;
                rrow[tid] = tok;
                rscale[tid] = p.as[tok];
            } else {
                rrow[tid] = tid < rows ? pair : -1;
                rscale[tid] = p.as[p0 + r];
            }
        }
    }
    __syncthreads();

    // Load sources.  LDS row 64 w + 32 ct + i of B is weight row n0 + 64 w + 2 i + ct
    // (so a lane ends with two neighbouring outputs), or for gate/up row f0 + 32 w + i
    // of gate (ct = 0) and up (ct = 1).  Rows past the end repeat the last one.
    uint32_t aoff[2], boff[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = 32 * wv + 16 * j + lane / 4, c = (lane & 3) ^ swz(r);
        const uint32_t row = KIND == GATE_UP ? static_cast<uint32_t>(rrow[r]) : static_cast<uint32_t>(min(r, rows - 1));
        aoff[j] = row * static_cast<uint32_t>(p.lda) + c * 16;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = 64 * wv + 16 * j + lane / 4, c = (lane & 3) ^ swz(r);
        const int ct = (r >> 5) & 1, i = r & 31;
        if (KIND == GATE_UP) {
            const int f = min(nt * (BN / 2) + 32 * wv + i, p.N - 1);
            boff[j] = static_cast<uint32_t>(f) * static_cast<uint32_t>(p.ldb) + c * 16 +
                      (ct ? static_cast<uint32_t>(p.q_off[1] - p.q_off[0]) : 0u);
        } else {
            const int n = min(64 * wv + 2 * i + ct, p.N - 1 - nt * BN);
            boff[j] = static_cast<uint32_t>(n) * static_cast<uint32_t>(p.ldb) + c * 16;
        }
    }

    i32x16 R[4][2];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int ct = 0; ct < 2; ++ct) R[mt][ct] = i32x16{};
    const int ks = (p.K + BK - 1) / BK, ktail = p.K - (ks - 1) * BK;
    switch (nmt) {
        case 1: k_loop<1>(ring, ring_lds, abase, bbase, aoff, boff, ks, ktail, wv, lane, R); break;
        case 2: k_loop<2>(ring, ring_lds, abase, bbase, aoff, boff, ks, ktail, wv, lane, R); break;
        case 3: k_loop<3>(ring, ring_lds, abase, bbase, aoff, boff, ks, ktail, wv, lane, R); break;
        default: k_loop<4>(ring, ring_lds, abase, bbase, aoff, boff, ks, ktail, wv, lane, R); break;
    }

    // Element i of an accumulator is row 8 (i / 4) + 4 hh + i % 4 of its 32.
    if (KIND == GATE_UP) {
        const int f = nt * (BN / 2) + 32 * wv + ln;
        if (f >= p.N) return;
        const float gs = bs[0][f], us = bs[1][f];
        uint16_t* h = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(p0) * p.ldo + f;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = 32 * mt + 8 * (i >> 2) + 4 * hh + (i & 3);
                if (r < rows) h[static_cast<int64_t>(r) * p.ldo] = swiglu_bf16(R[mt][0][i], R[mt][1][i], rscale[r], gs, us);
            }
    } else {
        const int n = nt * BN + 64 * wv + 2 * ln;
        if (n >= p.N) return;
        const bool two = n + 1 < p.N;
        const float s0 = bs[0][n], s1 = bs[0][two ? n + 1 : n];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int r = 32 * mt + 8 * (i >> 2) + 4 * hh + (i & 3);
                if (r >= rows) continue;
                int64_t orow = m0 + r;
                if (KIND == DOWN) {
                    orow = rrow[r];
                    if (orow < 0) continue;
                }
                const float v0 = static_cast<float>(R[mt][0][i]) * rscale[r] * s0;
                const float v1 = static_cast<float>(R[mt][1][i]) * rscale[r] * s1;
                const int64_t o = orow * p.ldo + n;
                if (KIND == DOWN || p.out_bf16) {
                    uint16_t* y = static_cast<uint16_t*>(p.out) + o;
                    if (KIND == DOWN) {
                        // y in bf16: one more rounding of 2^-9 per expert output, for half the
                        // traffic of the [pairs, H] intermediate
                        *reinterpret_cast<uint32_t*>(y) = f32_to_bf16(v0) | static_cast<uint32_t>(f32_to_bf16(v1)) << 16;
                    } else {
                        y[0] = f32_to_bf16(v0);
                        if (two) y[1] = f32_to_bf16(v1);
                    }
                } else {
                    float* y = static_cast<float*>(p.out) + o;
                    y[0] = v0;
                    if (two) y[1] = v1;
                }
            }
    }
}

// Tile plan of a grouped call: tile j covers tile_rows[j] positions of expert
// tile_e[j]'s bucket from tile_p0[j].  Offsets are clamped to the call's pairs.
__global__ void __launch_bounds__(1024) plan_i8_kernel(const int32_t* __restrict__ offsets, int E, int pairs,
                                                       int max_tiles, int32_t* __restrict__ tile_e,
                                                       int32_t* __restrict__ tile_p0,
                                                       int32_t* __restrict__ tile_rows,
                                                       int32_t* __restrict__ n_tiles) {
    __shared__ int32_t wave_tot[16];
    const int e = threadIdx.x, lane = e & (WAVE - 1), w = e / WAVE;
    const int beg = e < E ? min(max(offsets[e], 0), pairs) : 0;
    const int end = e < E ? min(max(offsets[e + 1], beg), pairs) : 0;
    const int nt = (end - beg + BM - 1) / BM;
    int inc = nt;
#pragma unroll
    for (int d = 1; d < WAVE; d <<= 1) {
        const int o = __shfl_up(inc, d, WAVE);
        if (lane >= d) inc += o;
    }
    if (lane == WAVE - 1) wave_tot[w] = inc;
    __syncthreads();
    int base = 0, all = 0;
    for (int i = 0; i < 16; ++i) {
        if (i < w) base += wave_tot[i];
        all += wave_tot[i];
    }
    base += inc - nt;
    for (int i = 0; i < nt && base + i < max_tiles; ++i) {
        tile_e[base + i] = e;
        tile_p0[base + i] = beg + i * BM;
        tile_rows[base + i] = min(BM, end - beg - i * BM);
    }
    if (e == 0) *n_tiles = min(all, max_tiles);
}

// out[t] = sum over j ascending of w[t, j] y[t k + j] in fp32, rounded to bf16
// once; a slot whose id is out of range adds nothing.  Eight columns a thread.
__global__ void __launch_bounds__(256) combine_i8_kernel(const uint16_t* __restrict__ y,
                                                         const int32_t* __restrict__ ids,
                                                         const float* __restrict__ w, int k, int E, int H,
                                                         int64_t n8, uint16_t* __restrict__ out) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n8) return;
    const int H8 = H / 8;
    const int64_t t = i / H8;
    const int c = static_cast<int>(i - t * H8) * 8;
    float a[8] = {};
    for (int j = 0; j < k; ++j) {
        const int id = ids[t * k + j];
        if (id < 0 || id >= E) continue;
        const float wj = w[t * k + j];
        const uint4 v = *reinterpret_cast<const uint4*>(y + (t * k + j) * H + c);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            a[2 * q] = fmaf(wj, __uint_as_float(u[q] << 16), a[2 * q]);
            a[2 * q + 1] = fmaf(wj, __uint_as_float(u[q] & 0xFFFF0000u), a[2 * q + 1]);
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = f32_to_bf16(a[2 * q]) | static_cast<uint32_t>(f32_to_bf16(a[2 * q + 1])) << 16;
    *reinterpret_cast<uint4*>(out + t * H + c) = make_uint4(o[0], o[1], o[2], o[3]);
}

int64_t align256(int64_t n) { return (n + 255) & ~int64_t{255}; }

int max_tiles(int pairs, int E) { return pairs / BM + (pairs < E ? pairs : E); }

// Regions of a prefill workspace.
struct PrefillWs {
    int64_t tiles, xq, xs, h, hq, hs, y, bytes;
};
PrefillWs prefill_ws(const moe355_layer_desc* d, int T) {
    const int64_t th = static_cast<int64_t>(T) * d->hidden, tk = static_cast<int64_t>(T) * d->top_k;
    PrefillWs w;
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t here = at;
        at += align256(n);
        return here;
    };
    w.tiles = take((3ll * max_tiles(static_cast<int>(tk), d->n_experts) + 1) * 4);
    w.xq = take(th);
    w.xs = take(4ll * T);
    w.h = take(2 * tk * d->inter);
    w.hq = take(tk * d->inter);
    w.hs = take(4 * tk);
    w.y = take(2 * tk * d->hidden);
    w.bytes = at;
    return w;
}

unsigned grid_of(int64_t tiles) { return static_cast<unsigned>((tiles + NXCD - 1) / NXCD * NXCD); }

}  // namespace

size_t prefill_i8_ws_bytes(const moe355_layer_desc* d, int T) {
    if (static_cast<int64_t>(T) * d->top_k >= (1ll << 28)) return 0;
    return static_cast<size_t>(prefill_ws(d, T).bytes);
}

}  // namespace moe355

using namespace moe355;

extern "C" moe355_status moe355_matmul_i8(const int8_t* a, int64_t a_stride, const float* a_scale,
                                          const int8_t* b, int64_t b_stride, const float* b_scale, int32_t M,
                                          int32_t N, int32_t K, void* out, int32_t out_type,
                                          int64_t out_stride, hipStream_t stream) {
    MOE355_REQUIRE(M >= 0 && N >= 1 && K >= 1, MOE355_EINVAL, "matmul_i8: M=%d N=%d K=%d", M, N, K);
    MOE355_REQUIRE(out_type == MOE355_F32 || out_type == MOE355_BF16, MOE355_EINVAL, "matmul_i8: out_type=%d",
                   out_type);
    MOE355_REQUIRE(K % 16 == 0 && K <= 65536, MOE355_ENOTSUP, "matmul_i8: K=%d (a multiple of 16 up to 65536)", K);
    if (M == 0) return ok();
    MOE355_REQUIRE(a && a_scale && b && b_scale && out, MOE355_EINVAL, "matmul_i8: null pointer");
    MOE355_REQUIRE((M == 1 || (a_stride >= K && out_stride >= N)) && (N == 1 || b_stride >= K), MOE355_EINVAL,
                   "matmul_i8: row strides %lld, %lld, %lld of K=%d, K, N=%d values",
                   static_cast<long long>(a_stride), static_cast<long long>(b_stride),
                   static_cast<long long>(out_stride), K, N);
    if (M == 1) a_stride = K;
    if (N == 1) b_stride = K;
    if (M == 1) out_stride = N;
    MOE355_REQUIRE(a_stride % 16 == 0 && b_stride % 16 == 0 && reinterpret_cast<uintptr_t>(a) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(b) % 16 == 0,
                   MOE355_ENOTSUP, "matmul_i8: rows of codes must start at multiples of 16 bytes");
    // a tile's rows are addressed by 32-bit offsets from its first one
    MOE355_REQUIRE(a_stride < (1ll << 23) && b_stride < (1ll << 23), MOE355_ENOTSUP,
                   "matmul_i8: row strides %lld, %lld of 2^23 bytes or more", static_cast<long long>(a_stride),
                   static_cast<long long>(b_stride));
    const int64_t tiles = static_cast<int64_t>((M + BM - 1) / BM) * ((N + BN - 1) / BN);
    MOE355_REQUIRE(tiles < (1ll << 31) - NXCD, MOE355_ENOTSUP, "matmul_i8: %lld tiles", static_cast<long long>(tiles));
    GemmParams p{};
    p.a = a;
    p.lda = a_stride;
    p.as = a_scale;
    p.b = b;
    p.ldb = b_stride;
    p.bs = b_scale;
    p.M = M;
    p.N = N;
    p.K = K;
    p.out = out;
    p.out_bf16 = out_type == MOE355_BF16;
    p.ldo = out_stride;
    gemm_i8_kernel<DENSE><<<grid_of(tiles), 256, 0, stream>>>(p);
    return check_launch("matmul_i8");
}

extern "C" moe355_status moe355_expert_ffn_prefill_i8(const moe355_layer_desc* d, const void* x_bf16, int32_t T,
                                                      const int32_t* topk_ids, const float* topk_w,
                                                      const uint8_t* layer_w, const int32_t* perm,
                                                      const int32_t* offsets, void* out_bf16, void* ws,
                                                      size_t ws_bytes, hipStream_t stream) {
    moe355_status st = check_desc_i8(d, "expert_ffn_prefill_i8");
    if (st) return st;
    MOE355_REQUIRE(T >= 0 && static_cast<int64_t>(T) * d->top_k < (1ll << 28), MOE355_EINVAL,
                   "expert_ffn_prefill_i8: T=%d", T);
    if (T == 0) return ok();
    MOE355_REQUIRE(x_bf16 && topk_ids && topk_w && layer_w && perm && offsets && out_bf16, MOE355_EINVAL,
                   "expert_ffn_prefill_i8: null pointer");
    MOE355_REQUIRE(reinterpret_cast<uintptr_t>(x_bf16) % 16 == 0 && reinterpret_cast<uintptr_t>(layer_w) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(out_bf16) % 16 == 0 && reinterpret_cast<uintptr_t>(ws) % 256 == 0,
                   MOE355_EINVAL, "expert_ffn_prefill_i8: x, layer_w and out at multiples of 16 bytes, ws of 256");
    MOE355_REQUIRE(d->n_experts <= 1024, MOE355_ENOTSUP, "expert_ffn_prefill_i8: E=%d > 1024", d->n_experts);
    // x's codes and one expert's blob are addressed by 32-bit offsets
    MOE355_REQUIRE(static_cast<int64_t>(T) * d->hidden <= 0xFFFFFFFFll, MOE355_ENOTSUP,
                   "expert_ffn_prefill_i8: T*H=%lld beyond 2^32", static_cast<long long>(T) * d->hidden);
    const PrefillWs w = prefill_ws(d, T);
    MOE355_REQUIRE(ws && ws_bytes >= static_cast<size_t>(w.bytes), MOE355_ECAPACITY,
                   "expert_ffn_prefill_i8: workspace %zu < %lld bytes", ws_bytes, static_cast<long long>(w.bytes));
    const I8Layout L = i8_layout(d);
    const int H = d->hidden, I = d->inter, pairs = T * d->top_k;
    const int mt = max_tiles(pairs, d->n_experts);
    uint8_t* base = static_cast<uint8_t*>(ws);
    int32_t* tiles = reinterpret_cast<int32_t*>(base + w.tiles);
    int8_t* xq = reinterpret_cast<int8_t*>(base + w.xq);
    float* xs = reinterpret_cast<float*>(base + w.xs);
    int8_t* hq = reinterpret_cast<int8_t*>(base + w.hq);
    float* hs = reinterpret_cast<float*>(base + w.hs);
    uint16_t* h = reinterpret_cast<uint16_t*>(base + w.h);
    uint16_t* y = reinterpret_cast<uint16_t*>(base + w.y);

    plan_i8_kernel<<<1, 1024, 0, stream>>>(offsets, d->n_experts, pairs, mt, tiles, tiles + mt, tiles + 2 * mt,
                                           tiles + 3 * mt);
    st = check_launch("expert_ffn_prefill_i8 plan");
    if (st) return st;
    st = launch_quant_rows(x_bf16, H, T, H, xq, H, xs, stream, "expert_ffn_prefill_i8 quantise x");
    if (st) return st;
    GemmParams p{};
    p.S = L.bytes;
    p.b = reinterpret_cast<const int8_t*>(layer_w);
    p.perm = perm;
    p.ids = topk_ids;
    p.tile_e = tiles;
    p.tile_p0 = tiles + mt;
    p.tile_rows = tiles + 2 * mt;
    p.n_tiles = tiles + 3 * mt;
    p.pairs = pairs;
    p.k = d->top_k;
    GemmParams g = p;
    g.a = xq;
    g.lda = H;
    g.as = xs;
    g.ldb = H;
    g.N = I;
    g.K = H;
    g.out = h;
    g.ldo = I;
    for (int m = 0; m < 2; ++m) {
        g.q_off[m] = L.q[m];
        g.s_off[m] = L.s[m];
    }
    gemm_i8_kernel<GATE_UP><<<grid_of(static_cast<int64_t>(mt) * ((I + BN / 2 - 1) / (BN / 2))), 256, 0, stream>>>(g);
    st = check_launch("expert_ffn_prefill_i8 gate_up");
    if (st) return st;
    st = launch_quant_rows(h, I, pairs, I, hq, I, hs, stream, "expert_ffn_prefill_i8 quantise h");
    if (st) return st;
    GemmParams dn = p;
    dn.a = hq;
    dn.lda = I;
    dn.as = hs;
    dn.ldb = I;
    dn.N = H;
    dn.K = I;
    dn.out = y;
    dn.ldo = H;
    dn.q_off[0] = dn.q_off[1] = L.q[2];
    dn.s_off[0] = dn.s_off[1] = L.s[2];
    gemm_i8_kernel<DOWN><<<grid_of(static_cast<int64_t>(mt) * ((H + BN - 1) / BN)), 256, 0, stream>>>(dn);
    st = check_launch("expert_ffn_prefill_i8 down");
    if (st) return st;
    const int64_t n8 = static_cast<int64_t>(T) * H / 8;
    combine_i8_kernel<<<static_cast<unsigned>((n8 + 255) / 256), 256, 0, stream>>>(
        y, topk_ids, topk_w, d->top_k, d->n_experts, H, n8, static_cast<uint16_t*>(out_bf16));
    return check_launch("expert_ffn_prefill_i8 combine");
}
