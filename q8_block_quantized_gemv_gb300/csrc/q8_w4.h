// Shared by the kernels over 4-bit weights: the tiled form, the view of a call, and the launches.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/q8_gemv.h"

namespace q8 {

constexpr int kW4Strip = 32;  // columns of a strip

// Bytes of a unit (one group of a strip): codes, 32 scales, 32 zero points where there are any.
__host__ __device__ constexpr int w4_unit(int group, bool zeros) { return 16 * group + 64 + (zeros ? 32 : 0); }

// Where the word of rows 8t .. 8t + 7 of the group's 32-row block b, column c of the strip, stands in its unit.
__host__ __device__ constexpr int w4_word(int group, int b, int t, int c) {
    const int j = c >> 4, h = (c >> 3) & 1, lane = 4 * (c & 7) + t;
    return group == 32 ? 256 * j + 8 * lane + 4 * h : 512 * (2 * (b >> 1) + j) + 16 * lane + 4 * (2 * (b & 1) + h);
}

// What follows the product: nothing, the gated pair (parts 0 and 1 are the gate and the up projection), the residual.
enum W4Epilogue { kW4Store = 0, kW4Glu = 1, kW4Residual = 2 };

struct W4Part {
    const unsigned char *w;
    float *y;  // fp32 [m][Np]; the gated pair's may be null
    int N, Np;
    int strip_end;  // strips of the parts up to this one
};

struct W4Args {
    const uint16_t *x;  // bf16 [m][K]
    int m, K, group, unit;
    int zeros, bf16;  // flags of the weights
    int nparts, epi;
    uint16_t *ybf;     // the gated pair's bf16 output, or null
    const float *res;  // the residual, fp32 [m][Np]
    W4Part part[Q8_MAX_PARTS];
};

constexpr int kW4StreamRows = 16;  // most rows of a stream; more take the GEMM
constexpr unsigned kW4Fault = 16u;  // bit of the fault word: a bounded wait ran out
cudaError_t launch_w4_stream(const W4Args &a, bool constant_weights, cudaStream_t stream);  // q8_w4_stream.cu
cudaError_t launch_w4_gemm(const W4Args &a, bool constant_weights, cudaStream_t stream);    // q8_w4_gemm.cu
cudaError_t read_w4_fault(unsigned *out, bool clear);       // of both
cudaError_t read_w4_gemm_fault(unsigned *out, bool clear);

}  // namespace q8
