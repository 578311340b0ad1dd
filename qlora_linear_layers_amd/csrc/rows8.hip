// Rows in 8 bits with one scale each, for gfx950: the quantizer and the way
// back.  Both are bound by HBM; a row is read once into its team's registers
// (rows.hpp), so that the maximum and the codes come from one pass.
#include "rows.hpp"

namespace ql {

// 2048 x 22016 values, 135 MB: 23.4 us, 5.8 TB/s; 7 x 11008 4.1 us, its latencies.
template <bool F16, int LANES, int CH>
__global__ __launch_bounds__(team_threads(LANES)) void k_rows8_quantize(const uint16_t* __restrict__ x, int64_t R,
                                                                        int K, int P, int8_t* __restrict__ codes,
                                                                        float* __restrict__ scale) {
    __shared__ float slot[32];
    const int lane = (int)threadIdx.x & (LANES - 1);
    const int64_t row = (int64_t)blockIdx.x * (team_threads(LANES) / LANES) + threadIdx.x / LANES;
    const bool ok = row < R;
    const uint16_t* xr = x + (ok ? row : R - 1) * K;
    u32x4_t v[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) v[j] = row_load(xr, lane + j * LANES, K);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p) m = abs_max2(v[j][p], m);
    m = team_umax<LANES>(m, slot);
    float d, inv;
    ck_scale<F16>(m, d, inv);
    if (!ok) return;
    int8_t* cr = codes + row * P;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = lane + j * LANES;
        if (c * 8 < P)
            *reinterpret_cast<u32x2_t*>(cr + c * 8) =
                u32x2_t{ck_codes4<F16>(v[j][0], v[j][1], inv), ck_codes4<F16>(v[j][2], v[j][3], inv)};
    }
    if (lane == 0) scale[row] = d;
}

// The values back: 21.0 us for the same size, 6.4 TB/s.
template <bool F16, int LANES, int CH>
__global__ __launch_bounds__(team_threads(LANES)) void k_rows8_dequantize(const int8_t* __restrict__ codes,
                                                                          const float* __restrict__ scale, int64_t R,
                                                                          int K, int P, uint16_t* __restrict__ out) {
    const int lane = (int)threadIdx.x & (LANES - 1);
    const int64_t row = (int64_t)blockIdx.x * (team_threads(LANES) / LANES) + threadIdx.x / LANES;
    if (row >= R) return;
    const float d = scale[row];
    const int8_t* cr = codes + row * P;
    u32x2_t c[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int e0 = (lane + j * LANES) * 8;
        if (e0 < K) c[j] = *reinterpret_cast<const u32x2_t*>(cr + e0);
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int ch = lane + j * LANES;
        if (ch * 8 < K) row_store(out + row * K, ch, K, ck_pack8<F16>(c[j], d));
    }
}

// Team of a row of K values: one wave up to 2048 values, else 256 threads, and
// 1024 where 256 would hold more than eight chunks each.
template <class Go>
static void for_team(int64_t K, Go go) {
    const int64_t c = ceil_div(K, 8);
    if (c <= 64) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    else if (c <= 128) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    else if (c <= 256) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
    else if (c <= 512) go(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    else if (c <= 1024) go(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
    else if (c <= 2048) go(std::integral_constant<int, 256>{}, std::integral_constant<int, 8>{});
    else if (c <= 4096) go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
    else go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 8>{});
}

hipError_t launch_rows8_quantize(const uint16_t* x, int64_t R, int64_t K, int8_t* codes, float* scale, hipStream_t s,
                                 bool f16) {
    for_team(K, [&](auto lanes, auto ch) {
        constexpr int L = decltype(lanes)::value, C = decltype(ch)::value;
        const dim3 g((unsigned)ceil_div(R, team_threads(L) / L)), b(team_threads(L));
        const int P = (int)rows8_pitch(K);
        if (f16) hipLaunchKernelGGL((k_rows8_quantize<true, L, C>), g, b, 0, s, x, R, (int)K, P, codes, scale);
        else hipLaunchKernelGGL((k_rows8_quantize<false, L, C>), g, b, 0, s, x, R, (int)K, P, codes, scale);
    });
    return hipGetLastError();
}

hipError_t launch_rows8_dequantize(const int8_t* codes, const float* scale, int64_t R, int64_t K, uint16_t* out,
                                   hipStream_t s, bool f16) {
    for_team(K, [&](auto lanes, auto ch) {
        constexpr int L = decltype(lanes)::value, C = decltype(ch)::value;
        const dim3 g((unsigned)ceil_div(R, team_threads(L) / L)), b(team_threads(L));
        const int P = (int)rows8_pitch(K);
        if (f16) hipLaunchKernelGGL((k_rows8_dequantize<true, L, C>), g, b, 0, s, codes, scale, R, (int)K, P, out);
        else hipLaunchKernelGGL((k_rows8_dequantize<false, L, C>), g, b, 0, s, codes, scale, R, (int)K, P, out);
    });
    return hipGetLastError();
}

}  // namespace ql
