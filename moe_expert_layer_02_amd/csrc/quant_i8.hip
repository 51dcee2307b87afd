// Symmetric int8 quantisation of bf16 rows: a = max |x|, r = 127 / a, code =
// rint(x r), scale = a / 127, every step rounded once to fp32, so the codes are
// defined bit for bit (|x r| <= 127 (1 + 2^-23) rounds to at most 127).
//
// One wavefront per row: the row stays in registers between the maximum and the
// codes (up to 4096 columns; longer rows are read twice).  Bound by memory: 2
// bytes read and 1 written per value (16384 x 4096: 37 us, 5.4 TB/s).
#include "i8.h"

namespace moe355 {
namespace {

constexpr int QWAVES = 4;

// NV > 0: vectors of 8 columns per lane held in registers; 0: any width, read
// twice; -1: any width and alignment, one value at a time.
template <int NV>
__global__ void __launch_bounds__(QWAVES* WAVE) quant_rows_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                                  int64_t rows, int cols,
                                                                  int8_t* __restrict__ q, int64_t ldq,
                                                                  float* __restrict__ scales) {
    const int lane = threadIdx.x & (WAVE - 1);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * QWAVES + threadIdx.x / WAVE;
    if (row >= rows) return;
    const uint16_t* xr = x + row * ldx;
    int8_t* qr = q + row * ldq;
    uint32_t top = 0;
    if constexpr (NV > 0) {
        uint4 v[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * WAVE + lane) * 8;
            v[i] = c < cols ? *reinterpret_cast<const uint4*>(xr + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) top = max(top, bf16x8_top(v[i]));
        const RowScale rs = row_scale(wave_max_u32(top));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (i * WAVE + lane) * 8;
            if (c < cols) *reinterpret_cast<uint2*>(qr + c) = quant8(v[i], rs.r);
        }
        if (lane == 0) scales[row] = rs.scale;
    } else if constexpr (NV == 0) {
        for (int c = lane * 8; c < cols; c += WAVE * 8)
            top = max(top, bf16x8_top(*reinterpret_cast<const uint4*>(xr + c)));
        const RowScale rs = row_scale(wave_max_u32(top));
        for (int c = lane * 8; c < cols; c += WAVE * 8)
            *reinterpret_cast<uint2*>(qr + c) = quant8(*reinterpret_cast<const uint4*>(xr + c), rs.r);
        if (lane == 0) scales[row] = rs.scale;
    } else {
        for (int c = lane; c < cols; c += WAVE) top = max(top, static_cast<uint32_t>(xr[c]) & 0x7FFFu);
        const RowScale rs = row_scale(wave_max_u32(top));
        for (int c = lane; c < cols; c += WAVE)
            qr[c] = static_cast<int8_t>(quant1(bf16_to_f32(xr[c]), rs.r));
        if (lane == 0) scales[row] = rs.scale;
    }
}

}  // namespace

moe355_status launch_quant_rows(const void* x, int64_t ldx, int64_t rows, int cols, int8_t* q, int64_t ldq,
                                float* scales, hipStream_t stream, const char* what) {
    if (rows == 0) return MOE355_OK;
    const uint16_t* xb = static_cast<const uint16_t*>(x);
    const bool vec = cols % 8 == 0 && ldx % 8 == 0 && ldq % 8 == 0 &&
                     reinterpret_cast<uintptr_t>(x) % 16 == 0 && reinterpret_cast<uintptr_t>(q) % 8 == 0;
    const int nv = (cols + WAVE * 8 - 1) / (WAVE * 8);
    auto k = !vec      ? quant_rows_kernel<-1>
             : nv <= 1 ? quant_rows_kernel<1>
             : nv <= 2 ? quant_rows_kernel<2>
             : nv <= 4 ? quant_rows_kernel<4>
             : nv <= 8 ? quant_rows_kernel<8>
                       : quant_rows_kernel<0>;
    k<<<static_cast<unsigned>((rows + QWAVES - 1) / QWAVES), QWAVES * WAVE, 0, stream>>>(xb, ldx, rows, cols, q,
                                                                                       ldq, scales);
    return check_launch(what);
}

}  // namespace moe355

using namespace moe355;

extern "C" moe355_status moe355_quantize_i8(const void* x_bf16, int64_t x_stride, int64_t rows, int32_t cols,
                                            int8_t* codes, int64_t codes_stride, float* scales,
                                            hipStream_t stream) {
    MOE355_REQUIRE(rows >= 0 && cols >= 1, MOE355_EINVAL, "quantize_i8: rows=%lld cols=%d",
                   static_cast<long long>(rows), cols);
    MOE355_REQUIRE(rows <= 1 || (x_stride >= cols && codes_stride >= cols), MOE355_EINVAL,
                   "quantize_i8: row strides %lld and %lld below cols=%d", static_cast<long long>(x_stride),
                   static_cast<long long>(codes_stride), cols);
    if (rows == 0) return ok();
    MOE355_REQUIRE(x_bf16 && codes && scales, MOE355_EINVAL, "quantize_i8: null pointer");
    MOE355_REQUIRE(rows <= 0x7FFFFFFFll, MOE355_ENOTSUP, "quantize_i8: rows=%lld",
                   static_cast<long long>(rows));
    return launch_quant_rows(x_bf16, x_stride, rows, cols, codes, codes_stride, scales, stream, "quantize_i8");
}
