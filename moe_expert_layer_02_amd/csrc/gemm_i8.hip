// Int8 matrix products on the CDNA4 matrix cores: C[m, n] = sa[m] sb[n] sum_k
// A[m, k] B[n, k], the sum exact in int32 (v_mfma_i32_32x32x32_i8), in three
// forms that share one K loop:
//   dense    C = A . B^T (moe355_matmul_i8);
//   gate/up  a grouped product over expert buckets whose epilogue forms
//            h = silu(g) u (moe355_expert_ffn_prefill_i8);
//   down     the grouped product of h, one row of y per (token, slot) pair.
//
// Tile: 256 rows (short tiles: 64) x 256 weight rows per block of eight wavefronts, two
// per SIMD; a wavefront owns half the rows and 64 weight rows (eight 32x32 accumulators,
// or two).  The activations are the first operand, so an accumulator holds rows
// (tokens) in its registers and a weight row per lane.
//
// K runs in stages of 128, whose rows are whole 128-byte lines: direct loads to
// LDS of 128-byte row pieces reach 23.8 TB/s over the chip, of 64-byte pieces
// 14.7 (one cache request each either way).  Two slots of 64 KB (three of 40 KB) hold
// the stage in use and the next (two).  Blocks are persistent (one per CU): the stages
// of a block's tiles form one stream, so the next tile's first stages load under the
// epilogue of the one before.
//
// Short tiles serve small products, where few blocks wait for their loads and the
// matrix cores for both: a tile of K = 4096 takes 24 us against 51 of a tall one, one of
// K = 512 takes 7.6 against 15.  Per row the tall ones read half as much, so they win
// from three rounds of short tiles over the CUs on (3000 x 4096 x 4096: 67 us against
// 82), and in the grouped products from about 96 pairs per expert on (64 experts of
// 2048 x 768: 92 us short and 111 tall at 32 pairs, 128 and 141 at 96, 149 and 148 at 128).
//
// What bounds the tall ones: LDS reads (3200 cycles a stage of 2048 MFMA cycles) and
// power; the same loop on registers and LDS alone sustains 2.9 POP/s on random codes (4.9
// on zeros).  Measured: 16384 x 4096 x 4096 in 293 us with the quantisation of A before
// it, 1.88 POP/s; gate/up of 98304 pairs, H 4096, I 2048, 1.89 ms, 1.75 POP/s; down 1.06 ms.
#include <type_traits>

#include "i8.h"
#include "lds_dma.h"

namespace moe355 {
namespace {

constexpr int BN = 256, BK = 128;
constexpr int THREADS = 512;
constexpr int NXCD = 8;
constexpr int TALL = 256, SHORT = 64;   // rows of a tile
constexpr int TALL_COST = 2, SHORT_COST = 1;   // of a round of tiles: 51 us and 24 us at K = 4096
constexpr int SHORT_PAIRS = 96;         // pairs per expert up to which a chunk takes them

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
    int paired;             // dense: two neighbouring outputs go out in one store
    int64_t ldo;
    // grouped
    int64_t S;
    int64_t q_off[2], s_off[2];
    const int32_t* row;     // of each position: gate/up its token, down its row of y
    const int32_t* tile_e;
    const int32_t* tile_p0;
    const int32_t* tile_rows;
    const int32_t* n_tiles;
};

// 16-byte chunk c of LDS row r sits at position c ^ swz(r) of the row's eight, so
// that the 16 rows a quarter of a read covers fall in different banks.
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

// The operands of one K step (32 inputs) of a wavefront.
struct Frag {
    i32x4 a[4], b[2];
};

// A tile: its weight column block, rows, expert and first row (dense) or position.
struct Tile {
    int nt, rows, e, m0;
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

// A direct load of base + voff (per lane) into LDS at lds + AT.
template <int AT>
__device__ __forceinline__ void dma16_at(const void* base, uint32_t voff, uint32_t lds) {
    asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(voff), "s"(base), "s"(lds), "n"(AT) : "memory", "scc");
}

template <int KIND, int BM>
__global__ void __launch_bounds__(THREADS, 2) gemm_i8_kernel(GemmParams p) {
    constexpr int SLOTS = BM == TALL ? 2 : 3;
    constexpr int SLOT_A = BM * BK, SLOT = (BM + BN) * BK;   // bytes
    // direct loads of each operand per wavefront and stage
    constexpr int PA = SLOT_A / 1024 / (THREADS / WAVE), PB = BN * BK / 1024 / (THREADS / WAVE);
    constexpr int MT_W = BM / 64;              // row tiles of 32 of a wavefront
    constexpr int GROUP_M = 1024 / BM;         // dense: 1024 rows of tiles at a time, weight columns outermost
    __shared__ __attribute__((aligned(1024))) uint8_t ring[SLOTS * SLOT];
    __shared__ __attribute__((aligned(16))) float rscale[2][BM];   // scales of the rows of this tile and the next
    __shared__ __attribute__((aligned(16))) int64_t rrow[2][BM];   // down: byte offsets of their rows of y
    const int tid = threadIdx.x;
    const int wv = __builtin_amdgcn_readfirstlane(tid / WAVE);
    // The lane index is made opaque again for every tile, so that the compiler
    // recomputes what derives from it instead of keeping it in registers (they would
    // not suffice, and a spill's reload waits for every memory operation in flight).
    int lane = tid & (WAVE - 1), ln = 0, hh = 0, la = 0, lb = 0;   // la, lb: LDS rows of load piece 0; piece j: + 8 j
    auto refresh_lane = [&]() {
        asm volatile("" : "+v"(lane));
        ln = lane & 31;
        hh = lane >> 5;
        la = 8 * PA * wv + lane / 8;
        lb = 8 * PB * wv + lane / 8;
    };
    refresh_lane();
    const int wm = wv >> 2, wn = wv & 3;   // the wavefront's half of the rows and 64 weight rows
    const uint32_t ring_lds = lds_addr(ring);

    // Tiles of one XCD (block id mod 8) are consecutive: neighbours share an
    // expert's weights or activation rows in that XCD's L2.
    constexpr int PER_N = KIND == GATE_UP ? BN / 2 : BN;
    const int NT = (p.N + PER_N - 1) / PER_N;
    const int MT = KIND == DENSE ? static_cast<int>((static_cast<int64_t>(p.M) + BM - 1) / BM) : ld_const(p.n_tiles);
    const int64_t total = static_cast<int64_t>(MT) * NT;
    const int xcd = blockIdx.x % NXCD, step_t = gridDim.x / NXCD;
    const int t_end = static_cast<int>(total * (xcd + 1) / NXCD);
    int t = static_cast<int>(total * xcd / NXCD) + blockIdx.x / NXCD;
    if (t >= t_end) return;
    const int ks = max(SLOTS, (p.K + BK - 1) / BK);

    auto tile_at = [&](int i) {
        Tile x;
        int mt;
        if (KIND == DENSE) {
            const int g = i / (GROUP_M * NT), in = i - g * GROUP_M * NT;
            const int gm = min(GROUP_M, MT - g * GROUP_M);
            x.nt = in / gm;
            mt = g * GROUP_M + (in - x.nt * gm);
            x.m0 = mt * BM;
            x.rows = min(BM, p.M - x.m0);
            x.e = 0;
        } else {
            mt = i / NT;
            x.nt = i - mt * NT;
            x.e = ld_const(p.tile_e + mt);
            x.m0 = ld_const(p.tile_p0 + mt);
            x.rows = ld_const(p.tile_rows + mt);
        }
        return x;
    };
    auto blob_at = [&](const Tile& x) { return p.b + static_cast<int64_t>(x.e) * p.S; };

    // Load sources of the tile the stream has reached.  LDS row 64 w + 32 ct + i of B
    // is weight row n0 + 64 w + 2 i + ct (so a lane ends with two neighbouring
    // outputs), or for gate/up row f0 + 32 w + i of gate (ct = 0) and up (ct = 1).
    // Rows past the end repeat the last one.
    const void *abase, *bbase;
    uint32_t aoff[PA], boff[PB];
    bool a_rows = true;   // some of the wavefront's A rows exist (the others are not loaded, nor used)
    auto set_source = [&](const Tile& x, const int (&tok)[PA]) {
        if (KIND == DENSE) {
            abase = uniform_ptr(p.a + static_cast<int64_t>(x.m0) * p.lda);
            bbase = uniform_ptr(p.b + static_cast<int64_t>(x.nt) * BN * p.ldb);
        } else {
            abase = uniform_ptr(KIND == GATE_UP ? p.a : p.a + static_cast<int64_t>(x.m0) * p.lda);
            bbase = uniform_ptr(blob_at(x) + p.q_off[0] + (KIND == DOWN ? static_cast<int64_t>(x.nt) * BN * p.ldb : 0));
        }
        a_rows = 8 * PA * wv < x.rows;
#pragma unroll
        for (int j = 0; j < PA; ++j) {
            const int r = la + 8 * j;
            const int row = KIND == GATE_UP ? tok[j] : min(r, x.rows - 1);
            aoff[j] = static_cast<uint32_t>(row) * static_cast<uint32_t>(p.lda) + ((lane & 7) ^ swz(r)) * 16;
        }
#pragma unroll
        for (int j = 0; j < PB; ++j) {
            const int r = lb + 8 * j, c = ((lane & 7) ^ swz(r)) * 16;
            const int w = r >> 6, ct = (r >> 5) & 1, i = r & 31;
            if (KIND == GATE_UP) {
                const int f = min(x.nt * (BN / 2) + 32 * w + i, p.N - 1);
                boff[j] = static_cast<uint32_t>(f) * static_cast<uint32_t>(p.ldb) + c +
                          (ct ? static_cast<uint32_t>(p.q_off[1] - p.q_off[0]) : 0u);
            } else {
                const int n = min(64 * w + 2 * i + ct, p.N - 1 - x.nt * BN);
                boff[j] = static_cast<uint32_t>(n) * static_cast<uint32_t>(p.ldb) + c;
            }
        }
    };
    // Stage kk into a slot.  The offsets stay in their
    // registers; the bases move.  (Four instructions a load: with the addresses and the
    // tail's test formed per load, the last load of a stage went out half a stage late.)
    auto load_full = [&](int kk, int slot) {
        const uint32_t sa = ring_lds + slot * SLOT + PA * wv * 1024, sb = ring_lds + slot * SLOT + PB * wv * 1024;
        const int8_t *ab = static_cast<const int8_t*>(abase) + kk * BK, *bb = static_cast<const int8_t*>(bbase) + kk * BK;
        dma16_at<SLOT_A>(bb, boff[0], sb);
        dma16_at<SLOT_A + 1024>(bb, boff[1], sb);
        dma16_at<SLOT_A + 2 * 1024>(bb, boff[2], sb);
        dma16_at<SLOT_A + 3 * 1024>(bb, boff[3], sb);
        if (a_rows) {
            dma16_at<0>(ab, aoff[0], sa);
            if constexpr (PA == 4) {
                dma16_at<1024>(ab, aoff[1], sa);
                dma16_at<2 * 1024>(ab, aoff[2], sa);
                dma16_at<3 * 1024>(ab, aoff[3], sa);
            }
        }
    };
    // A stage that ends past K: a chunk past it is fetched from the row's start instead
    // (in bounds; its A side is cleared before use).
    auto load_tail = [&](int kk, int slot) {
        const uint32_t sa = ring_lds + slot * SLOT + PA * wv * 1024, sb = ring_lds + slot * SLOT + PB * wv * 1024;
#pragma unroll
        for (int j = 0; j < PA; ++j) {
            const int c = ((lane & 7) ^ swz(la + 8 * j)) * 16;
            dma16(abase, aoff[j] + (kk * BK + c < p.K ? kk * BK : static_cast<uint32_t>(-c)), sa + j * 1024);
        }
#pragma unroll
        for (int j = 0; j < PB; ++j) {
            const int c = ((lane & 7) ^ swz(lb + 8 * j)) * 16;
            dma16(bbase, boff[j] + (kk * BK + c < p.K ? kk * BK : static_cast<uint32_t>(-c)), sb + j * 1024 + SLOT_A);
        }
    };
    auto load_stage = [&](int kk, int slot) {
        if ((kk + 1) * BK > p.K) load_tail(kk, slot);
        else load_full(kk, slot);
    };
    auto clear_tail = [&](int kk, int slot) {   // A chunks past K of stage kk
        uint8_t* sp = ring + slot * SLOT;
        for (int i = tid; i < BM * 8; i += THREADS) {
            const int r = i >> 3, c = i & 7;
            if (kk * BK + c * 16 >= p.K)
                *reinterpret_cast<uint4*>(sp + r * BK + ((c ^ swz(r)) << 4)) = make_uint4(0, 0, 0, 0);
        }
        __syncthreads();
    };
    auto read_op = [&](int slot, int s, int i, Frag& f) {   // operand i (of 2 + MT_W) of step s
        const uint8_t* sp = ring + slot * SLOT;
        const int c = ((2 * s + hh) ^ swz(ln)) << 4;        // rows differ from ln by multiples of 32
        if (i < 2) f.b[i] = *reinterpret_cast<const i32x4*>(sp + SLOT_A + (64 * wn + 32 * i + ln) * BK + c);
        else f.a[i - 2] = *reinterpret_cast<const i32x4*>(sp + (BM / 2 * wm + 32 * (i - 2) + ln) * BK + c);
    };

    // The scales (and rows of y) of a tile's rows, one row per thread, and the tokens
    // behind the LDS rows this lane loads of it.
    float my_scale = 0.0f;
    int my_row = 0, tok[PA] = {};
    auto request_rows = [&](const Tile& x) {
        const int r = x.m0 + min(tid & (BM - 1), x.rows - 1);
        my_scale = p.as[KIND == GATE_UP ? p.row[r] : r];
        if (KIND == DOWN) my_row = p.row[r];
    };
    auto keep_rows = [&](int at) {
        if (tid < BM) {
            rscale[at][tid] = my_scale;
            if (KIND == DOWN) rrow[at][tid] = 2 * p.ldo * my_row;
        }
    };
    auto request_tokens = [&](const Tile& x) {
        if (KIND == GATE_UP) {
#pragma unroll
            for (int j = 0; j < PA; ++j) tok[j] = p.row[x.m0 + min(la + 8 * j, x.rows - 1)];
        }
    };
    auto next_of = [&](int i) { return i + step_t < t_end ? i + step_t : i; };   // at the end the tile itself

    Tile cur = tile_at(t), nxt = tile_at(next_of(t));
    request_tokens(cur);
    request_rows(cur);
    set_source(cur, tok);
    keep_rows(0);
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) load_stage(i, i);
    int slot = 0, lk = SLOTS;   // slot of the stage in use; next stage to load of the tile in aoff / boff
    auto after = [&](int i) { return i + 1 < SLOTS ? i + 1 : 0; };   // the next slot
    Frag f[2];
    stage_barrier<PB * (SLOTS - 1)>();   // stage 0 has landed everywhere (each later one is at least PB loads)
    if (p.K < BK) clear_tail(0, 0);
#pragma unroll
    for (int i = 0; i < 2 + MT_W; ++i) read_op(0, 0, i, f[0]);
    bool stores_after = false;   // at least 16 MT_W stores were issued after the last loads
    int par = 0;                 // this tile's half of rscale and rrow

    for (; t < t_end; t += step_t) {
        refresh_lane();
        request_rows(nxt);
        request_tokens(nxt);
        i32x16 R[MT_W][2];
#pragma unroll
        for (int mt = 0; mt < MT_W; ++mt)
#pragma unroll
            for (int ct = 0; ct < 2; ++ct) R[mt][ct] = i32x16{};
        // Rows of the wavefront that exist: row tiles of 32 without any are skipped.
        const int live = __builtin_amdgcn_readfirstlane(cur.rows - BM / 2 * wm);
        // The four K steps of a stage: while a step's MFMAs run, the next step's
        // operands are read from LDS into the other register set.  The stage's barrier
        // stands before its last step, whose operands are in registers by then: past it
        // the next stage has landed and this one is read out, so the last step covers the
        // first reads of the next stage and the issue of the loads after that.
        // No scalar load may be pending in the loop: they complete out of order, so every
        // wait for an LDS read would have to wait for all of them.
        __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0)
#pragma nounroll
        for (int kk = 0; kk < ks; ++kk) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s == 3) {
                    if (lk == ks) {   // the stream enters the next tile
                        set_source(nxt, tok);
                        lk = 0;
                    }
                    // the loads have landed; of a tile's first stage they are older than the
                    // stores of the epilogue before, which may still be on their way
                    if (kk == 0 && stores_after) stage_barrier<BM == TALL ? 32 : 16>();
                    else stage_barrier<PB * (SLOTS - 2)>();
                    // the next stage ends past K: the last of this tile, or (K < 128) the first of the next
                    const int nk = kk + 1 < ks ? kk + 1 : 0;
                    if ((nk + 1) * BK > p.K) clear_tail(nk, after(slot));
                    // what was requested about the next tile's rows has landed by now
                    if (kk == 1) keep_rows(par ^ 1);
                }
#pragma unroll
                for (int mt = 0; mt < MT_W; ++mt) {
                    __builtin_amdgcn_sched_barrier(0);
                    if (32 * mt < live) {
#pragma unroll
                        for (int ct = 0; ct < 2; ++ct)
                            R[mt][ct] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f[s & 1].a[mt], f[s & 1].b[ct], R[mt][ct], 0, 0, 0);
                    }
                    if (s == 3 && mt == 0) load_stage(lk, slot);
#pragma unroll
                    for (int j = 2 * mt; j < (mt + 1 < MT_W ? 2 * mt + 2 : 2 + MT_W); ++j) {
                        if (s < 3) read_op(slot, s + 1, j, f[(s + 1) & 1]);
                        else read_op(after(slot), 0, j, f[0]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            ++lk;
            slot = after(slot);
        }

        refresh_lane();
        const Tile now = cur;
        cur = nxt;
        nxt = tile_at(next_of(next_of(t)));
        const int half = par;
        par ^= 1;
        // Element i of an accumulator is row 8 (i / 4) + 4 hh + i % 4 of its 32.
        // 16 MT_W stores where every row is live and the wavefront's first output exists
        stores_after = live >= BM / 2 && now.nt * PER_N + (PER_N / 4) * wn < p.N;
        const float* bs0 = KIND == DENSE ? p.bs : reinterpret_cast<const float*>(blob_at(now) + p.s_off[0]);
        const int r0 = BM / 2 * wm + 4 * hh;
        // Loaded scales are waited for here: left to the rows' conditional blocks, every one
        // of them would wait for all of the stores before it.
        auto landed = [](float a, float b) { asm volatile("" ::"v"(a), "v"(b)); };
        // Scales and row offsets are read for four rows at a time and outside the rows'
        // conditions (behind each one, a partial tile spent an LDS trip per row).
        auto each_row = [&](auto put) {   // put(mt, element, row past r0, its scale, its offset in y)
            auto rows = [&](auto ALLc) {
#pragma unroll
                for (int mt = 0; mt < MT_W; ++mt) {
                    if (!decltype(ALLc)::value && 32 * mt >= live) continue;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int r = 32 * mt + 8 * g;
                        float rs[4];
                        int64_t ro[4] = {};
                        __builtin_memcpy(rs, __builtin_assume_aligned(&rscale[half][r0 + r], 16), 16);
                        if (KIND == DOWN) __builtin_memcpy(ro, __builtin_assume_aligned(&rrow[half][r0 + r], 16), 32);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (decltype(ALLc)::value || r0 + r + i < now.rows) put(mt, 4 * g + i, r + i, rs[i], ro[i]);
                    }
                }
            };
            if (live >= BM / 2) rows(std::true_type{});
            else if (live > 0) rows(std::false_type{});
        };
        if (KIND == GATE_UP) {
            const float* bs1 = reinterpret_cast<const float*>(blob_at(now) + p.s_off[1]);
            const int fe = now.nt * (BN / 2) + 32 * wn + ln;
            if (fe < p.N) {
                const float gs = bs0[fe], us = bs1[fe];
                landed(gs, us);
                uint16_t* h = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(now.m0 + r0) * p.ldo + fe;
                each_row([&](int mt, int i, int r, float xs, int64_t) {
                    h[static_cast<int64_t>(r) * p.ldo] = swiglu_bf16(R[mt][0][i], R[mt][1][i], xs, gs, us);
                });
            }
        } else {
            const int n = now.nt * BN + 64 * wn + 2 * ln;
            if (n < p.N) {
                const bool two = n + 1 < p.N;
                const float s0 = bs0[n], s1 = bs0[two ? n + 1 : n];
                landed(s0, s1);
                each_row([&](int mt, int i, int r, float rs, int64_t ro) {
                    const float v0 = static_cast<float>(R[mt][0][i]) * rs * s0;
                    const float v1 = static_cast<float>(R[mt][1][i]) * rs * s1;
                    if (KIND == DOWN) {
                        // y in bf16: one more rounding of 2^-9 per expert output, for half the
                        // traffic of the [pairs, H] intermediate
                        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + ro + 2 * n) = pack_bf16(v0, v1);
                        return;
                    }
                    const int64_t o = static_cast<int64_t>(now.m0 + r0 + r) * p.ldo + n;
                    if (p.out_bf16) {
                        uint16_t* y = static_cast<uint16_t*>(p.out) + o;
                        if (p.paired) {
                            *reinterpret_cast<uint32_t*>(y) = pack_bf16(v0, v1);
                        } else {
                            y[0] = f32_to_bf16(v0);
                            if (two) y[1] = f32_to_bf16(v1);
                        }
                    } else {
                        float* y = static_cast<float*>(p.out) + o;
                        if (p.paired) {
                            *reinterpret_cast<float2*>(y) = make_float2(v0, v1);
                        } else {
                            y[0] = v0;
                            if (two) y[1] = v1;
                        }
                    }
                });
            }
        }
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // the loads past the last tile have landed
}

// Dense product of few rows: bound by reading the weights once and by latency, not by
// the matrix cores.  A block owns 16 weight rows and up to 16 NT rows of A; its eight
// wavefronts split K (v_mfma_i32_16x16x64_i8, the weights as the first operand) and
// meet in LDS.  1 x 4096 x 4096: 5.0 us, 3.4 TB/s of weights (22 us by tiles).
constexpr int FEW_WAVES = 8;
constexpr int64_t FEW_OUTPUTS = 1 << 19;
template <int NT>
__global__ void __launch_bounds__(FEW_WAVES* WAVE) few_rows_i8_kernel(GemmParams p) {
    __shared__ i32x4 part[FEW_WAVES][NT][WAVE];
    const int tid = threadIdx.x, lane = tid & (WAVE - 1);
    const int wv = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int row = lane & 15, quad = lane >> 4;
    const int n0 = blockIdx.x * 16, m0 = blockIdx.y * 16 * NT;
    const int8_t* w = p.b + static_cast<int64_t>(min(n0 + row, p.N - 1)) * p.ldb + quad * 16;
    const int8_t* x[NT];
    i32x4 acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        x[t] = p.a + static_cast<int64_t>(min(m0 + 16 * t + row, p.M - 1)) * p.lda + quad * 16;
        acc[t] = i32x4{};
    }
    // steps of 64 inputs, FEW_WAVES apart; AHEAD of them requested at once.  A lane whose
    // 16 inputs lie past K takes zeros.
    constexpr int AHEAD = NT >= 4 ? 4 : 8;
    for (int k0 = wv * 64; k0 < p.K; k0 += AHEAD * FEW_WAVES * 64) {
        i32x4 b[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int k = k0 + i * FEW_WAVES * 64;
            b[i] = k + quad * 16 < p.K ? *reinterpret_cast<const i32x4*>(w + k) : i32x4{};
        }
        i32x4 a[AHEAD][NT];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int k = k0 + i * FEW_WAVES * 64;
#pragma unroll
            for (int t = 0; t < NT; ++t) a[i][t] = k + quad * 16 < p.K ? *reinterpret_cast<const i32x4*>(x[t] + k) : i32x4{};
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[i], a[i][t], acc[t], 0, 0, 0);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) part[wv][t][lane] = acc[t];
    __syncthreads();
    // element i of lane l: weight row 4 (l / 16) + i, row of A l % 16
    for (int o = tid; o < NT * 256; o += FEW_WAVES * WAVE) {
        const int n = o & 15, m = (o >> 4) & 15, t = o >> 8;
        if (n0 + n >= p.N || m0 + 16 * t + m >= p.M) continue;
        int sum = 0;
#pragma unroll
        for (int q = 0; q < FEW_WAVES; ++q) sum += reinterpret_cast<const int*>(&part[q][t][(n >> 2) * 16 + m])[n & 3];
        const int r = m0 + 16 * t + m;
        const float v = static_cast<float>(sum) * p.as[r] * p.bs[n0 + n];
        const int64_t at = static_cast<int64_t>(r) * p.ldo + n0 + n;
        if (p.out_bf16) static_cast<uint16_t*>(p.out)[at] = f32_to_bf16(v);
        else static_cast<float*>(p.out)[at] = v;
    }
}

// What the products need beside the weights, in one launch: the tile list (block 0),
// what each position of the buckets stands for, and x's codes and scales.
//
// Tiles are cut to about equal size per bucket, so that blocks that take the same
// number of tiles end together.  A position's token, and its row of y: a position whose
// pair is not one of the bucket's expert (ids out of range leave such positions behind)
// computes token 0 into a row of y that nobody reads.  Quantisation: one wavefront per
// row, as quantize_i8.
constexpr int PREP = 1024;
struct PrepParams {
    const int32_t *offsets, *perm, *ids;
    int E, k, pairs, bm, max_tiles, row_blocks;
    int32_t *tile_e, *tile_p0, *tile_rows, *n_tiles, *tok, *yrow;
    const uint16_t* x;
    int T, H;
    int8_t* xq;
    float* xs;
};
__global__ void __launch_bounds__(PREP) prep_i8_kernel(PrepParams p) {
    __shared__ int32_t wave_tot[PREP / WAVE];
    const int lane = threadIdx.x & (WAVE - 1), w = threadIdx.x / WAVE;
    if (static_cast<int>(blockIdx.x) > p.row_blocks) {
        const int64_t t = static_cast<int64_t>(blockIdx.x - p.row_blocks - 1) * (PREP / WAVE) + w;
        if (t >= p.T) return;
        const float scale = quant_row(p.x + t * p.H, p.H, p.xq + t * p.H, lane);
        if (lane == 0) p.xs[t] = scale;
        return;
    }
    if (blockIdx.x > 0) {
        const int64_t i = static_cast<int64_t>(blockIdx.x - 1) * PREP + threadIdx.x;
        if (i >= p.pairs) return;
        const int pair = p.perm[i];
        bool ok = pair >= 0 && pair < p.pairs;
        const int e = ok ? p.ids[pair] : -1;
        ok = e >= 0 && e < p.E && p.offsets[e] <= i && i < p.offsets[e + 1];
        p.tok[i] = ok ? pair / p.k : 0;
        p.yrow[i] = ok ? pair : p.pairs;
        return;
    }
    const int e = threadIdx.x;
    const int beg = e < p.E ? min(max(p.offsets[e], 0), p.pairs) : 0;
    const int end = e < p.E ? min(max(p.offsets[e + 1], beg), p.pairs) : 0;
    const int nt = (end - beg + p.bm - 1) / p.bm;
    const int per = nt ? ((end - beg + nt - 1) / nt + 31) / 32 * 32 : 0;
    int inc = nt;
#pragma unroll
    for (int d = 1; d < WAVE; d <<= 1) {
        const int o = __shfl_up(inc, d, WAVE);
        if (lane >= d) inc += o;
    }
    if (lane == WAVE - 1) wave_tot[w] = inc;
    __syncthreads();
    int base = 0, all = 0;
    for (int i = 0; i < PREP / WAVE; ++i) {
        if (i < w) base += wave_tot[i];
        all += wave_tot[i];
    }
    base += inc - nt;
    for (int i = 0; i < nt && base + i < p.max_tiles; ++i) {
        p.tile_e[base + i] = e;
        p.tile_p0[base + i] = beg + i * per;
        p.tile_rows[base + i] = min(per, end - beg - i * per);
    }
    if (e == 0) *p.n_tiles = min(all, p.max_tiles);
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

// Rows of a tile of the grouped products.
int tile_rows(int pairs, int E) { return pairs <= SHORT_PAIRS * E ? SHORT : TALL; }

// Room for the tile list: the short tiles' bound for either, so that a workspace for a
// long chunk also holds a shorter one's list.
int max_tiles(int pairs, int E) { return pairs / SHORT + (pairs < E ? pairs : E); }

// Regions of a prefill workspace.
struct PrefillWs {
    int64_t tiles, tok, yrow, xq, xs, h, hq, hs, y, bytes;
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
    w.tok = take(4 * tk);
    w.yrow = take(4 * tk);
    w.xq = take(th);
    w.xs = take(4ll * T);
    w.h = take(2 * tk * d->inter);
    w.hq = take(tk * d->inter);
    w.hs = take(4 * tk);
    w.y = take(2 * (tk + 1) * d->hidden);   // one row more: see prep_i8_kernel
    w.bytes = at;
    return w;
}

// Which dense form: up to 2^19 outputs, or 64 rows, no tiles (M = 256, N = 2048, K = 4096:
// 20.8 us against 24.8 of the short tiles; M = 192, N = 4096: 29.6 against 25.2).
bool few_rows(int M, int N) { return M <= 64 || static_cast<int64_t>(M) * N <= FEW_OUTPUTS; }

// CUs, down to a multiple of the XCDs.
int cus() {
    static const int n = [] {
        int dev = 0, c = 0;
        if (hipGetDevice(&dev) != hipSuccess ||
            hipDeviceGetAttribute(&c, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
            c = 256;
        return c < NXCD ? NXCD : c / NXCD * NXCD;
    }();
    return n;
}

// One block per CU; fewer where there are fewer tiles.
unsigned grid_of(int64_t tiles) {
    const int64_t need = (tiles + NXCD - 1) / NXCD * NXCD;
    return static_cast<unsigned>(need < cus() ? need : cus());
}

// Dense tiles: the tall ones if their rounds over the CUs cost no more.
bool tall_tiles(int64_t tall, int64_t low) {
    return (tall + cus() - 1) / cus() * TALL_COST < (low + cus() - 1) / cus() * SHORT_COST;
}

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
    const int64_t columns = (N + BN - 1) / BN;
    const int64_t tall = (static_cast<int64_t>(M) + TALL - 1) / TALL * columns;
    const int64_t tiles = (static_cast<int64_t>(M) + SHORT - 1) / SHORT * columns;
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
    p.paired = N % 2 == 0 && out_stride % 2 == 0 && reinterpret_cast<uintptr_t>(out) % (p.out_bf16 ? 4 : 8) == 0;
    if (few_rows(M, N)) {
        const dim3 grid((N + 15) / 16, (M + 63) / 64);
        if (M <= 16) few_rows_i8_kernel<1><<<grid, FEW_WAVES * WAVE, 0, stream>>>(p);
        else if (M <= 32) few_rows_i8_kernel<2><<<grid, FEW_WAVES * WAVE, 0, stream>>>(p);
        else few_rows_i8_kernel<4><<<grid, FEW_WAVES * WAVE, 0, stream>>>(p);
        return check_launch("matmul_i8");
    }
    if (tall_tiles(tall, tiles)) gemm_i8_kernel<DENSE, TALL><<<grid_of(tall), THREADS, 0, stream>>>(p);
    else gemm_i8_kernel<DENSE, SHORT><<<grid_of(tiles), THREADS, 0, stream>>>(p);
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

    int32_t* tok = reinterpret_cast<int32_t*>(base + w.tok);
    int32_t* yrow = reinterpret_cast<int32_t*>(base + w.yrow);
    PrepParams r{};
    r.offsets = offsets;
    r.perm = perm;
    r.ids = topk_ids;
    r.E = d->n_experts;
    r.k = d->top_k;
    r.pairs = pairs;
    r.bm = tile_rows(pairs, d->n_experts);
    r.max_tiles = mt;
    r.row_blocks = (pairs + PREP - 1) / PREP;
    r.tile_e = tiles;
    r.tile_p0 = tiles + mt;
    r.tile_rows = tiles + 2 * mt;
    r.n_tiles = tiles + 3 * mt;
    r.tok = tok;
    r.yrow = yrow;
    r.x = static_cast<const uint16_t*>(x_bf16);
    r.T = T;
    r.H = H;
    r.xq = xq;
    r.xs = xs;
    prep_i8_kernel<<<1 + r.row_blocks + (T + PREP / WAVE - 1) / (PREP / WAVE), PREP, 0, stream>>>(r);
    st = check_launch("expert_ffn_prefill_i8 prepare");
    if (st) return st;
    GemmParams p{};
    p.S = L.bytes;
    p.b = reinterpret_cast<const int8_t*>(layer_w);
    p.tile_e = tiles;
    p.tile_p0 = tiles + mt;
    p.tile_rows = tiles + 2 * mt;
    p.n_tiles = tiles + 3 * mt;
    GemmParams g = p;
    g.row = tok;
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
    const bool tall = tile_rows(pairs, d->n_experts) == TALL;
    (tall ? gemm_i8_kernel<GATE_UP, TALL> : gemm_i8_kernel<GATE_UP, SHORT>)
        <<<grid_of(static_cast<int64_t>(mt) * ((I + BN / 2 - 1) / (BN / 2))), THREADS, 0, stream>>>(g);
    st = check_launch("expert_ffn_prefill_i8 gate_up");
    if (st) return st;
    st = launch_quant_rows(h, I, pairs, I, hq, I, hs, stream, "expert_ffn_prefill_i8 quantise h");
    if (st) return st;
    GemmParams dn = p;
    dn.row = yrow;
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
    (tall ? gemm_i8_kernel<DOWN, TALL> : gemm_i8_kernel<DOWN, SHORT>)
        <<<grid_of(static_cast<int64_t>(mt) * ((H + BN - 1) / BN)), THREADS, 0, stream>>>(dn);
    st = check_launch("expert_ffn_prefill_i8 down");
    if (st) return st;
    const int64_t n8 = static_cast<int64_t>(T) * H / 8;
    combine_i8_kernel<<<static_cast<unsigned>((n8 + 255) / 256), 256, 0, stream>>>(
        y, topk_ids, topk_w, d->top_k, d->n_experts, H, n8, static_cast<uint16_t*>(out_bf16));
    return check_launch("expert_ffn_prefill_i8 combine");
}
