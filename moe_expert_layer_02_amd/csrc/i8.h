// Shared pieces of the int8 operators (quantisation, dense product, expert FFN).
#pragma once

#include "internal.h"

namespace moe355 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// Codes and scales of `rows` rows (the kernel behind moe355_quantize_i8).
moe355_status launch_quant_rows(const void* x, int64_t ldx, int64_t rows, int cols, int8_t* q, int64_t ldq,
                                float* scales, hipStream_t stream, const char* what);

// Largest magnitude among 8 packed bf16 values, as bf16 bits (order-preserving:
// a NaN's bits lie above infinity's, so neither is lost).
__device__ __forceinline__ uint32_t bf16x8_top(uint4 v) {
    const u16x2_t m = bf16_mag_max(v, u16x2_t{0, 0});
    return max(static_cast<uint32_t>(m.x), static_cast<uint32_t>(m.y));
}

// A row's factors from its largest magnitude (bf16 bits): codes = rint(x r).  A
// row below 2^-100 counts as zero (127 / a would overflow); a row that holds an
// infinity or NaN gets codes 0 and the scale NaN, so its products are NaN.
struct RowScale {
    float r, scale;
};
__device__ __forceinline__ RowScale row_scale(uint32_t top) {
    const float a = __uint_as_float(top << 16);
    if (top >= 0x7F80u) return {0.0f, __builtin_nanf("")};
    if (a < 0x1p-100f) return {0.0f, 0.0f};
    return {127.0f / a, a / 127.0f};
}

// One code.  r = 0 marks a row whose codes are 0 (also where x is not finite).
__device__ __forceinline__ int quant1(float x, float r) {
    const float v = rintf(x * r);
    return r == 0.0f ? 0 : static_cast<int>(v);
}

// Eight bf16 values to eight codes.
__device__ __forceinline__ uint2 quant8(uint4 v, float r) {
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = static_cast<uint32_t>(quant1(__uint_as_float(in[i] << 16), r));
        const uint32_t hi = static_cast<uint32_t>(quant1(__uint_as_float(in[i] & 0xFFFF0000u), r));
        c[i] = (lo & 0xFFu) | (hi & 0xFFu) << 8;
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// One row of n bf16 values (16-byte aligned, n a multiple of 8) to codes by one
// wavefront; the row's scale on every lane.
__device__ __forceinline__ float quant_row(const uint16_t* x, int n, int8_t* q, int lane) {
    constexpr int HELD = 4;   // vectors a lane keeps between the two passes (2048 columns); the others are read again
    uint4 v[HELD];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int c = (i * WAVE + lane) * 8;
        v[i] = c < n ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
    }
    for (int c = (HELD * WAVE + lane) * 8; c < n; c += WAVE * 8)
        top = max(top, bf16x8_top(*reinterpret_cast<const uint4*>(x + c)));
#pragma unroll
    for (int i = 0; i < HELD; ++i) top = max(top, bf16x8_top(v[i]));
    const RowScale rs = row_scale(wave_max_u32(top));
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int c = (i * WAVE + lane) * 8;
        if (c < n) *reinterpret_cast<uint2*>(q + c) = quant8(v[i], rs.r);
    }
    for (int c = (HELD * WAVE + lane) * 8; c < n; c += WAVE * 8)
        *reinterpret_cast<uint2*>(q + c) = quant8(*reinterpret_cast<const uint4*>(x + c), rs.r);
    return rs.scale;
}

// fp32 to bf16 bits, to nearest (ties to even); NaN stays NaN.
__device__ __forceinline__ uint16_t f32_to_bf16(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}

// silu(g) u = g u / (1 + e^-g).  h is kept in bf16 between the two products of an
// int8 layer: half the traffic of fp32, and its 2^-9 is far below the code step it
// meets next.
__device__ __forceinline__ float swiglu(float g, float u) {
    return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}
// h of one element from the two int32 sums and their scales.
__device__ __forceinline__ uint16_t swiglu_bf16(int ga, int ua, float xs, float gs, float us) {
    const float g = static_cast<float>(ga) * xs * gs, u = static_cast<float>(ua) * xs * us;
    return f32_to_bf16(swiglu(g, u));
}

// One int8 expert blob: byte offsets of the codes and scales of gate, up, down.
struct I8Layout {
    int64_t bytes;
    int64_t q[3], s[3];
};
inline I8Layout i8_layout(const moe355_layer_desc* d) {
    const int64_t H = d->hidden, I = d->inter;
    I8Layout L;
    L.q[0] = 0;
    L.s[0] = I * H;
    L.q[1] = L.s[0] + 4 * I;
    L.s[1] = L.q[1] + I * H;
    L.q[2] = L.s[1] + 4 * I;
    L.s[2] = L.q[2] + H * I;
    L.bytes = L.s[2] + 4 * H;
    return L;
}

moe355_status check_desc_i8(const moe355_layer_desc* d, const char* what);
size_t prefill_i8_ws_bytes(const moe355_layer_desc* d, int T);
size_t decode_i8_ws_bytes(const moe355_layer_desc* d, int T);

}  // namespace moe355
