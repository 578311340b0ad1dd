// Rows of 16-bit values held in a team's registers, and the 8-bit row format,
// shared by the norm (norm.hip) and the row quantizer (rows8.hip).
//
// A team of LANES threads owns one row; lane l holds the 8-value chunks l,
// l + LANES, ... (CH of them), zeros past the row's end.  Teams of one wave
// share a 256-thread workgroup; larger ones are the workgroup.  A row starts at
// any even address (odd row lengths): its chunks are 16-byte loads and stores of
// 2-byte alignment, which the hardware takes, and only the row's last, partial
// chunk goes element by element.  (Loading the row's last eight values instead and
// shifting them spared odd rows a wait per operand, 777 x 4099 backward 24.4 -> 19.6 us,
// and cost all others its instructions and registers, 4096 x 4096 31.3 -> 34.4.)
#pragma once

#include "act.hpp"
#include "common.hpp"
#include "plan.hpp"

namespace ql {

constexpr int64_t kRows8Pitch = 128;
__host__ __device__ inline int64_t rows8_pitch(int64_t K) { return (K + kRows8Pitch - 1) / kRows8Pitch * kRows8Pitch; }

constexpr int team_threads(int lanes) { return lanes < 256 ? 256 : lanes; }

typedef u32x4_t u32x4_a2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_a4 __attribute__((aligned(4)));

// Values 8 c .. 8 c + 7 of a row of D, zeros past its end
QL_DEV u32x4_t row_load(const uint16_t* row, int c, int D) {
    const int e0 = c * 8;
    if (e0 + 8 <= D) return *reinterpret_cast<const u32x4_a2*>(row + e0);
    u32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e0 + e < D) v[e >> 1] |= (uint32_t)row[e0 + e] << (16 * (e & 1));
    return v;
}

QL_DEV void row_store(uint16_t* row, int c, int D, const u32x4_t& v) {
    const int e0 = c * 8;
    if (e0 + 8 <= D) {
        *reinterpret_cast<u32x4_a2*>(row + e0) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e0 + e < D) row[e0 + e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
}

// The same for data that is not needed again soon: the caches let go of it first.
QL_DEV u32x4_t row_load_far(const uint16_t* row, int c, int D) {
    if (c * 8 + 8 <= D) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(row + c * 8));
    return row_load(row, c, D);
}
QL_DEV void row_store_far(uint16_t* row, int c, int D, const u32x4_t& v) {
    if (c * 8 + 8 <= D) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2*>(row + c * 8));
    else row_store(row, c, D, v);
}

// ------------------------------------------------------------------ reductions over a team

template <class F>
QL_DEV float row16_reduce(float v, F f) {                 // over the 16 lanes of a DPP row, in all of them
    v = f(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, false)));    // lane ^ 1
    v = f(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, false)));    // lane ^ 2
    v = f(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, false)));   // the other quad
    v = f(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, false)));   // the other eight
    return v;
}
QL_DEV float lane_value(float v, int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); }

QL_DEV float wave_sum(float v) {
    v = row16_reduce(v, [](float a, float b) { return a + b; });
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
// of values ordered as integers (magnitudes; a NaN's bits are the largest)
QL_DEV uint32_t wave_umax(uint32_t m) {
    m = max_of_8_lanes(m);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xF, 0xF, false));
    const auto at = [&](int l) { return (uint32_t)__builtin_amdgcn_readlane((int)m, l); };
    return max(max(at(0), at(16)), max(at(32), at(48)));
}

// Over a team; every thread of the workgroup calls these the same number of
// times.  `slot` is LDS of 32 words that no other reduction in flight uses (a
// caller alternates between two: a wave can only enter the next reduction's
// slot after the barrier of this one, so two are enough).
template <int LANES>
QL_DEV float team_sum(float v, float* slot) {
    v = wave_sum(v);
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < LANES / 64; ++w) v += slot[w];
    }
    return v;
}
template <int LANES>
QL_DEV void team_sum2(float& a, float& b, float* slot) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0) {
            slot[threadIdx.x >> 6] = a;
            slot[16 + (threadIdx.x >> 6)] = b;
        }
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < LANES / 64; ++w) {
            a += slot[w];
            b += slot[16 + w];
        }
    }
}
template <int LANES>
QL_DEV uint32_t team_umax(uint32_t m, float* slot) {
    m = wave_umax(m);
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = __uint_as_float(m);
        __syncthreads();
        m = 0;
#pragma unroll
        for (int w = 0; w < LANES / 64; ++w) m = max(m, __float_as_uint(slot[w]));
    }
    return m;
}

// ------------------------------------------------------------------ 8-bit rows
//
// One scale per row: with c = max|x|, d = fl32(c / 127) and codes
// q = fl32(x fl32(127 / c)) rounded to an integer, ties to even (the checkpoint's
// rounding, act.hpp).  c < 2^-120, where 127 / c leaves the fp32 range: zeros.
// An inf or a NaN in the row: d = NaN.

// scale and factor from the bits of fp32 c = max|x| (a NaN's are above inf's)
QL_DEV void rows8_scale(uint32_t cbits, float& d, float& inv) {
    const float c = __uint_as_float(cbits);
    const bool zero = c < 0x1p-120f;
    d = zero ? 0.0f : __fdiv_rn(c, 127.0f);
    inv = zero ? 0.0f : __fdiv_rn(127.0f, c);
    if (cbits >= 0x7F800000u) {
        d = __uint_as_float(0x7FC00000u);
        inv = 0.0f;
    }
}

// codes of eight fp32 values, value 0 in the low byte
QL_DEV u32x2_t rows8_codes(const float (&v)[8], float inv) {
    u32x2_t o;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const uint32_t q0 = ck_code(v[4 * p], inv), q1 = ck_code(v[4 * p + 1], inv);
        const uint32_t q2 = ck_code(v[4 * p + 2], inv), q3 = ck_code(v[4 * p + 3], inv);
        o[p] = __builtin_amdgcn_perm(q1, q0, 0x0C0C0400u) | __builtin_amdgcn_perm(q3, q2, 0x04000C0Cu);
    }
    return o;
}

// ------------------------------------------------------------------ launches

struct NormArgs {
    const uint16_t* x;
    const uint16_t* res;      // or null, as w, h, y and codes
    const void* w;            // [D], fp32 if w32, else of the 16-bit type
    uint16_t* h;
    uint16_t* y;
    int8_t* codes;
    float* scale;
    int64_t T;
    int D, w32;
    float eps;
    bool far;                 // set by the launch: h is written past the caches
};
struct NormBwd {
    const uint16_t* dy;
    const uint16_t* h;
    const void* w;
    const uint16_t* add;
    uint16_t* dx;
    void* dw;                 // null = not asked for
    float* part;              // [rmsnorm_bwd_partials][D] of dw
    int64_t T;
    int D, w32;
    float eps;
};

hipError_t launch_rmsnorm(NormArgs a, hipStream_t s, bool f16);
int64_t rmsnorm_bwd_partials(int64_t T, int64_t D);    // fp32 partial rows of dw
hipError_t launch_rmsnorm_bwd(const NormBwd& a, hipStream_t s, bool f16);
hipError_t launch_rows8_quantize(const uint16_t* x, int64_t R, int64_t K, int8_t* codes, float* scale, hipStream_t s,
                                 bool f16);
hipError_t launch_rows8_dequantize(const int8_t* codes, const float* scale, int64_t R, int64_t K, uint16_t* out,
                                   hipStream_t s, bool f16);

}  // namespace ql
