// Products over 4-bit weights, first form: a warp computes one strip of 32 columns for eight rows, a lane a column, on the
// CUDA cores.  Right for every size; neither reads the weight once for all rows nor fills the SMs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "q8_w4.h"

namespace q8 {
namespace {

constexpr int kRows = 8;

__device__ __forceinline__ float scale_value(uint16_t s, int bf16) {
    return bf16 ? __uint_as_float((uint32_t)s << 16) : __half2float(__ushort_as_half(s));
}

__device__ void product(const W4Args &a, const unsigned char *strip, int row0, int c, float (&acc)[kRows]) {
    for (int r = 0; r < kRows; ++r) acc[r] = 0.0f;
    for (int g = 0; g < a.K / a.group; ++g, strip += a.unit) {
        const int zero = a.zeros ? strip[16 * a.group + 64 + c] : 8;
        float part[kRows] = {};
        for (int b = 0; b < a.group / 32; ++b)
            for (int t = 0; t < 4; ++t) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(strip + w4_word(a.group, b, t, c));
                const uint16_t *x = a.x + (size_t)row0 * a.K + g * a.group + 32 * b + 8 * t;
                for (int i = 0; i < 8; ++i) {
                    const float v = (float)((int)((w >> (4 * (i >> 1) + 16 * (i & 1))) & 15u) - zero);
                    for (int r = 0; r < kRows; ++r)
                        if (row0 + r < a.m) part[r] = fmaf(__uint_as_float((uint32_t)x[(size_t)r * a.K + i] << 16), v, part[r]);
                }
            }
        const float s = scale_value(*reinterpret_cast<const uint16_t *>(strip + 16 * a.group + 2 * c), a.bf16);
        for (int r = 0; r < kRows; ++r) acc[r] = fmaf(s, part[r], acc[r]);
    }
}

__global__ void __launch_bounds__(128) simple_kernel(const __grid_constant__ W4Args a) {
    const int c = threadIdx.x & 31, strips = a.epi == kW4Glu ? a.part[0].strip_end : a.part[a.nparts - 1].strip_end;
    const int strip = blockIdx.x * 4 + (threadIdx.x >> 5), row0 = blockIdx.y * kRows;
    if (strip >= strips) return;
    int p = 0;
    while (strip >= a.part[p].strip_end) ++p;
    const int local = strip - (p ? a.part[p - 1].strip_end : 0), n = local * kW4Strip + c;
    const size_t at = (size_t)local * (a.K / a.group) * a.unit;
    float acc[kRows], up[kRows];
    product(a, a.part[p].w + at, row0, c, acc);
    if (a.epi == kW4Glu) product(a, a.part[1].w + at, row0, c, up);
    for (int r = 0; r < kRows && row0 + r < a.m; ++r) {
        const size_t to = (size_t)(row0 + r) * a.part[p].Np + n;
        float v = acc[r];
        if (a.epi == kW4Glu) v = v / (1.0f + expf(-v)) * up[r];
        if (a.epi == kW4Residual && n < a.part[p].N) v += a.res[to];
        if (n >= a.part[p].N) v = 0.0f;
        if (a.part[p].y) a.part[p].y[to] = v;
        if (a.ybf) a.ybf[to] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
}

}  // namespace

cudaError_t launch_w4_gemm(const W4Args &a, bool, cudaStream_t stream) {
    const int strips = a.epi == kW4Glu ? a.part[0].strip_end : a.part[a.nparts - 1].strip_end;
    simple_kernel<<<dim3((unsigned)(strips + 3) / 4, (unsigned)(a.m + kRows - 1) / kRows), 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace q8
