// The 8-bit integer product for gfx950: Y = act(X Wq^T dx dw + bias) * mul + res
// on v_mfma_i32_16x16x64_i8, sums exact in int32.
#include "int8.hpp"

namespace ql {

namespace {

template <bool F16>
QL_DEV float value16(uint16_t v) { return lo16<F16>(v); }

// Output (t, n): what the epilogue reads, loaded ahead, and the rounding at the end.
struct EpiOperands {
    float xs, ws;
    uint16_t bias, mul, res;
};
QL_DEV EpiOperands epi_load(const Int8Args& a, int64_t t, int64_t n) {
    const int64_t at = t * a.N + n;
    EpiOperands o;
    o.xs = a.xs[t];
    o.ws = a.ws[n];
    o.bias = a.ep.bias ? a.ep.bias[n] : 0;
    o.mul = a.ep.mul ? a.ep.mul[at] : 0;
    o.res = a.ep.res ? a.ep.res[at] : 0;
    return o;
}
template <bool F16>
QL_DEV uint16_t epi_value(const Int8Args& a, const EpiOperands& o, int sum) {
    float z = int8_scaled(sum, o.xs, o.ws);
    if (a.ep.bias) z += value16<F16>(o.bias);
    z = act_of(a.ep.act, z);
    if (a.ep.mul) z *= value16<F16>(o.mul);
    if (a.ep.res) z += value16<F16>(o.res);
    return (uint16_t)(pack16x2<F16>(z, 0.0f) & 0xFFFFu);
}

constexpr int kSkinnyWaves = 8;

}  // namespace

// 16 NT tokens x 16 channels per workgroup, K split over its eight waves in
// steps of 128 bytes; the waves' sums are added in LDS.
template <bool F16, int NT>
__global__ __launch_bounds__(64 * kSkinnyWaves) void k_int8_skinny(Int8Args a) {
    __shared__ int sums[kSkinnyWaves][NT][16][16];
    const int lane = (int)threadIdx.x & 63, wv = (int)threadIdx.x >> 6;
    const int l16 = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, t0 = (int64_t)blockIdx.y * (16 * NT);
    const int64_t n = n0 + l16 < a.N ? n0 + l16 : a.N - 1;
    const int8_t* wr = a.w + n * a.P + g * 16;
    const int8_t* xr[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int64_t t = t0 + 16 * i + l16;
        xr[i] = a.x + (t < a.T ? t : a.T - 1) * a.P + g * 16;
    }
    i32x4_t acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = i32x4_t{0, 0, 0, 0};
#pragma unroll 2
    for (int k = wv * 128; k < a.P; k += 128 * kSkinnyWaves) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const i32x4_t wf = *reinterpret_cast<const i32x4_t*>(wr + k + 64 * j);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(*reinterpret_cast<const i32x4_t*>(xr[i] + k + 64 * j), wf,
                                                               acc[i], 0, 0, 0);
        }
    }
    // lane holds tokens 4 g .. 4 g + 3 of channel l16
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) sums[wv][i][4 * g + q][l16] = acc[i][q];
    __syncthreads();
    for (int e = (int)threadIdx.x; e < NT * 256; e += 64 * kSkinnyWaves) {
        const int64_t t = t0 + e / 16, nn = n0 + e % 16;
        if (t >= a.T || nn >= a.N) continue;
        int v = 0;
#pragma unroll
        for (int w = 0; w < kSkinnyWaves; ++w) v += sums[w][e / 256][e / 16 % 16][e % 16];
        a.y[t * a.N + nn] = epi_value<F16>(a, epi_load(a, t, nn), v);
    }
}

size_t int8_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_int8(const Int8Args& a, void*, hipStream_t s, bool f16) {
    const auto go = [&](auto kern, int nt) {
        hipLaunchKernelGGL(kern, dim3((unsigned)ceil_div(a.N, 16), (unsigned)ceil_div(a.T, 16 * nt)),
                           dim3(64 * kSkinnyWaves), 0, s, a);
    };
    if (a.T <= 16) f16 ? go(k_int8_skinny<true, 1>, 1) : go(k_int8_skinny<false, 1>, 1);
    else f16 ? go(k_int8_skinny<true, 4>, 4) : go(k_int8_skinny<false, 4>, 4);
    return hipGetLastError();
}

}  // namespace ql
