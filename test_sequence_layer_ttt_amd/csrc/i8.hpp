// Arguments of the 8-bit integer product and the quantiser of its rows
// (i8_quantize.hip, i8_gemm.hip). All strides are in elements, the innermost
// dimension contiguous.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ttt {

struct I8QuantArgs {
    int M, K, io;
    const void *x;  // [M,K]
    int64_t xr;
    int8_t *q;  // [M,K], rows of qr
    int64_t qr;
    float *scale;  // [M]
};

struct I8Args {
    int M, K, N, out_io;  // tokens, contraction, features
    const int8_t *x;      // [M,K]
    int64_t xr;
    const float *xs;  // [M]
    const int8_t *w;  // [N,K]
    int64_t wr;
    const float *ws, *bias;  // [N]; bias may be null
    void *y;                 // [M,N]
    int64_t yr;
    // as the layer's views: three of [B,H,L,64] instead of y, N = 192 H, M = B L
    int L = 0, H = 0;
    void *v[3] = {};
    bool vec = false;  // y in 16-byte accesses (set by the launch)
};

// rows of K bytes, two operands' (rows 0: none), into rows of `pad` (a multiple of 128) with zeros behind
struct I8PadArgs {
    int rows[2];
    const int8_t *src[2];
    int64_t stride[2];
    int8_t *dst[2];
    int K, pad;
};

// Which operands launch_i8_project cannot take as they stand: with M > 64, rows that are not whole
// 16-byte chunks at 16-byte addresses, or 8 MB and more apart.
void i8_unaligned(const I8Args &a, bool *x, bool *w);
hipError_t launch_i8_pad(const I8PadArgs &a, hipStream_t stream);
hipError_t launch_i8_quantize(const I8QuantArgs &a, hipStream_t stream);
hipError_t launch_i8_project(const I8Args &a, hipStream_t stream);
// from features x [M,K] of io, rows of xr (a.x, a.xr, a.xs unused), where in_one says so
bool i8_features_in_one(const I8Args &a);
hipError_t launch_i8_features(const I8Args &a, int io, const void *x, int64_t xr, hipStream_t stream);

}  // namespace ttt
