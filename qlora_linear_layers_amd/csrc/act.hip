// 8-bit activation checkpoints and the elementwise part of the epilogue's
// backward, for gfx950.  All of it is bound by HBM: each kernel reads every
// input once and writes every output once, 16 bytes of 16-bit values per lane.
#include "act.hpp"
#include "plan.hpp"

namespace ql {

namespace {

constexpr int kThreads = 256;
constexpr int kCkChunks = 4;                       // 8-value chunks per thread
constexpr int64_t kCkPerWg = (int64_t)kThreads * 8 * kCkChunks;

// Values 8 ch .. 8 ch + 7 of x[numel], zeros past the end
QL_DEV u32x4_t chunk_of(const uint16_t* x, int64_t ch, int64_t numel) {
    const int64_t e0 = ch * 8;
    if (e0 + 8 <= numel) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(x) + ch);
    u32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e0 + e < numel) v[e >> 1] |= (uint32_t)x[e0 + e] << (16 * (e & 1));
    return v;
}

}  // namespace

// Checkpoint of x[numel]: eight lanes hold one block of 64, whose largest |x|
// is an integer max over the lanes.  Only the last block can be partial.
template <bool F16>
__global__ __launch_bounds__(kThreads) void k_act8_quantize(const uint16_t* __restrict__ x, int64_t numel,
                                                            int8_t* __restrict__ codes, float* __restrict__ scale) {
    const int64_t ch0 = (int64_t)blockIdx.x * (kThreads * kCkChunks) + threadIdx.x;
    u32x4_t v[kCkChunks];
#pragma unroll
    for (int j = 0; j < kCkChunks; ++j) v[j] = chunk_of(x, ch0 + j * kThreads, numel);
#pragma unroll
    for (int j = 0; j < kCkChunks; ++j) {
        const int64_t e0 = (ch0 + j * kThreads) * 8;
        uint32_t m = 0;
#pragma unroll
        for (int p = 0; p < 4; ++p) m = abs_max2(v[j][p], m);
        float d, inv;
        ck_scale<F16>(max_of_8_lanes(m), d, inv);
        const u32x2_t c = {ck_codes4<F16>(v[j][0], v[j][1], inv), ck_codes4<F16>(v[j][2], v[j][3], inv)};
        if (e0 + 8 <= numel) {
            __builtin_nontemporal_store(c, reinterpret_cast<u32x2_t*>(codes + e0));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e0 + e < numel) codes[e0 + e] = (int8_t)(c[e >> 2] >> (8 * (e & 3)));
        }
        if ((threadIdx.x & 7) == 0 && e0 < numel) scale[e0 >> 6] = d;
    }
}

template <bool F16>
__global__ __launch_bounds__(kThreads) void k_act8_dequantize(const int8_t* __restrict__ codes,
                                                              const float* __restrict__ scale, int64_t numel,
                                                              uint16_t* __restrict__ out) {
    const int64_t ch0 = (int64_t)blockIdx.x * (kThreads * kCkChunks) + threadIdx.x;
    u32x2_t c[kCkChunks];
    float d[kCkChunks];
#pragma unroll
    for (int j = 0; j < kCkChunks; ++j) {
        const int64_t e0 = (ch0 + j * kThreads) * 8;
        c[j] = u32x2_t{0, 0};
        d[j] = 0.0f;
        if (e0 + 8 <= numel) {
            c[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(codes + e0));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e0 + e < numel) c[j][e >> 2] |= (uint32_t)(uint8_t)codes[e0 + e] << (8 * (e & 3));
        }
        if (e0 < numel) d[j] = scale[e0 >> 6];
    }
#pragma unroll
    for (int j = 0; j < kCkChunks; ++j) {
        const int64_t e0 = (ch0 + j * kThreads) * 8;
        float v[8];
        ck_values4(c[j][0], d[j], v);
        ck_values4(c[j][1], d[j], v + 4);
        const u32x4_t o = pack8<F16>(v);
        if (e0 + 8 <= numel) {
            __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>(out + e0));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e0 + e < numel) out[e0 + e] = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// ------------------------------------------------------------------ backward of the epilogue

namespace {

// eight values of a saved [T][N] activation at element `at` (at % 8 == 0)
template <bool F16>
QL_DEV void saved8(const Saved& s, int64_t at, float (&v)[8]) {
    if (s.codes) {
        const u32x2_t c = *reinterpret_cast<const u32x2_t*>(s.codes + at);
        const float d = s.scale[at >> 6];
        ck_values4(c[0], d, v);
        ck_values4(c[1], d, v + 4);
    } else {
        unpack8<F16>(*reinterpret_cast<const u32x4_t*>(s.v + at), v);
    }
}

}  // namespace

// A workgroup owns 128 columns (16 lanes of 8) and one range of rows, 16 rows
// per step.  Column sums stay in registers over the steps; the 16 row slots of
// a column are then added in LDS in slot order, so d_bias is deterministic.
template <int ACT, bool F16>
__global__ __launch_bounds__(kThreads) void k_act_bwd(ActBwd a) {
    const int cl = threadIdx.x & 15, slot = threadIdx.x >> 4;
    const int64_t n = (int64_t)blockIdx.x * 128 + cl * 8;
    const int64_t r0 = (int64_t)blockIdx.y * a.rows;
    const int64_t r1 = r0 + a.rows < a.T ? r0 + a.rows : a.T;
    const bool nok = n < a.N;
    const bool has_z = a.z.v || a.z.codes, has_mul = a.mul.v || a.mul.codes;
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
    if (nok) {
#pragma unroll 2
        for (int64_t t = r0 + slot; t < r1; t += 16) {
            const int64_t at = t * a.N + n;
            float dy[8], z[8], u[8];
            unpack8<F16>(*reinterpret_cast<const u32x4_t*>(a.dy + at), dy);
            if (has_z) {
                saved8<F16>(a.z, at, z);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = 0.0f;
            }
            if (has_mul) saved8<F16>(a.mul, at, u);
            float h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float d;
                act_slope<ACT>(z[e], h[e], d);
                h[e] *= dy[e];
                if (has_mul) dy[e] *= u[e];
                dy[e] *= d;
                sum[e] += dy[e];
            }
            if (a.dmul) *reinterpret_cast<u32x4_t*>(a.dmul + at) = pack8<F16>(h);
            if (a.dz) *reinterpret_cast<u32x4_t*>(a.dz + at) = pack8<F16>(dy);
        }
    }
    if (!a.part) return;
    __shared__ float red[16][128 + 4];
#pragma unroll
    for (int e = 0; e < 8; ++e) red[slot][cl * 8 + e] = sum[e];
    __syncthreads();
    if (threadIdx.x < 128) {
        const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
        float v = red[0][threadIdx.x];
#pragma unroll
        for (int q = 1; q < 16; ++q) v += red[q][threadIdx.x];
        if (c < a.N) a.part[(int64_t)blockIdx.y * a.N + c] = v;
    }
}

// d_bias[n] = RNE_16(sum over the row ranges, in range order)
template <bool F16>
__global__ __launch_bounds__(kThreads) void k_bias_fin(const float* __restrict__ part, int64_t ranges, int64_t N,
                                                       uint16_t* __restrict__ out) {
    const int64_t n = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (n >= N) return;
    float v = 0.0f;
#pragma unroll 8
    for (int64_t q = 0; q < ranges; ++q) v += part[q * N + n];
    out[n] = (uint16_t)(pack16x2<F16>(v, 0.0f) & 0xFFFFu);
}

// ------------------------------------------------------------------ launchers

hipError_t launch_act8_quantize(const uint16_t* x, int64_t numel, int8_t* codes, float* scale, hipStream_t s,
                                bool f16) {
    const dim3 g((unsigned)ceil_div(numel, kCkPerWg));
    if (f16) hipLaunchKernelGGL(k_act8_quantize<true>, g, dim3(kThreads), 0, s, x, numel, codes, scale);
    else hipLaunchKernelGGL(k_act8_quantize<false>, g, dim3(kThreads), 0, s, x, numel, codes, scale);
    return hipGetLastError();
}

hipError_t launch_act8_dequantize(const int8_t* codes, const float* scale, int64_t numel, uint16_t* out, hipStream_t s,
                                  bool f16) {
    const dim3 g((unsigned)ceil_div(numel, kCkPerWg));
    if (f16) hipLaunchKernelGGL(k_act8_dequantize<true>, g, dim3(kThreads), 0, s, codes, scale, numel, out);
    else hipLaunchKernelGGL(k_act8_dequantize<false>, g, dim3(kThreads), 0, s, codes, scale, numel, out);
    return hipGetLastError();
}

hipError_t launch_act_bwd(const ActBwd& a, uint16_t* d_bias, hipStream_t s, bool f16) {
    const int64_t ranges = ceil_div(a.T, a.rows);
    const dim3 g((unsigned)ceil_div(a.N, 128), (unsigned)ranges);
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, g, dim3(kThreads), 0, s, a); };
    switch (a.act) {
        case kActRelu: f16 ? go(k_act_bwd<kActRelu, true>) : go(k_act_bwd<kActRelu, false>); break;
        case kActSilu: f16 ? go(k_act_bwd<kActSilu, true>) : go(k_act_bwd<kActSilu, false>); break;
        case kActGelu: f16 ? go(k_act_bwd<kActGelu, true>) : go(k_act_bwd<kActGelu, false>); break;
        case kActGeluTanh: f16 ? go(k_act_bwd<kActGeluTanh, true>) : go(k_act_bwd<kActGeluTanh, false>); break;
        default: f16 ? go(k_act_bwd<kActNone, true>) : go(k_act_bwd<kActNone, false>); break;
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !d_bias) return e;
    const dim3 bg((unsigned)ceil_div(a.N, kThreads));
    if (f16) hipLaunchKernelGGL(k_bias_fin<true>, bg, dim3(kThreads), 0, s, a.part, ranges, a.N, d_bias);
    else hipLaunchKernelGGL(k_bias_fin<false>, bg, dim3(kThreads), 0, s, a.part, ranges, a.N, d_bias);
    return hipGetLastError();
}

}  // namespace ql
