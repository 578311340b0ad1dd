// Activations, the 8-bit activation checkpoint and the output epilogue, shared
// by the kernels that end a projection (gemm.hip, gemv.hip) and by act.hip.
//
// Activation functions and their slopes (p = act(z) / z for the last three):
//   silu       p = 1 / (1 + e^-z)                      act' = p + z p (1 - p)
//   gelu       p = Phi(z) = erfc(-z / sqrt 2) / 2      act' = p + z e^(-z^2/2) / sqrt(2 pi)
//   gelu_tanh  p = 1 / (1 + e^(-2u)),  u = sqrt(2/pi) (z + 0.044715 z^3)
//                                                      act' = p + z p (1 - p) 2 u'
// (0.5 (1 + tanh u) is the logistic function of 2u).  Everything is fp32; exp
// and the reciprocal are the hardware's (about 1 ulp, plus |z| 2^-24 for the
// scaled argument of exp), far inside the 16-bit rounding of the results.
//
// Phi uses e^(x^2) erfc(x) as a polynomial of degree 7 in t = 1 / (1 + x/2),
// x = |z| / sqrt 2: a least-squares fit reweighted until the relative error is
// level over 0 <= x <= 12 (4.2e-7).  With fp32 arithmetic Phi's relative error
// is below 1.4e-6 for z > -5 and 7.1e-6 for z > -12, and the factor e^(-z^2/2)
// is shared with the slope; about 20 instructions, without branches.
#pragma once

#include "common.hpp"

namespace ql {

enum Act : int { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4 };
constexpr int kActs = 5;

// 1 / (1 + e^-z): e^-z = inf gives 0 and e^-z = 0 gives 1
QL_DEV float logistic(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhC = 0.79788456080286536f, kTanhA = 0.044715f;   // sqrt(2/pi)

// Phi(z), and e = e^(-z^2/2)
QL_DEV float normal_cdf(float z, float& e) {
    e = __builtin_amdgcn_exp2f(z * z * (-0.5f * 1.44269504088896341f));
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.5f * 0.70710678118654752f, 1.0f));
    float r = 0.5f * 0.09769358485937119f;                       // half of the fit: erfc / 2
    r = fmaf(r, t, 0.5f * -0.39232999086380005f);
    r = fmaf(r, t, 0.5f * 0.44363337755203247f);
    r = fmaf(r, t, 0.5f * -0.00581517955288291f);
    r = fmaf(r, t, 0.5f * 0.30132532119750977f);
    r = fmaf(r, t, 0.5f * 0.27252811193466187f);
    r = fmaf(r, t, 0.5f * 0.2830007076263428f);
    r = fmaf(r, t, 0.5f * -3.552611087798141e-05f);
    const float h = r * e;
    return z < 0.0f ? h : 1.0f - h;
}

template <int ACT>
QL_DEV float act_value(float z) {
    if constexpr (ACT == kActRelu) return z <= 0.0f ? 0.0f : z;
    else if constexpr (ACT == kActSilu) return z * logistic(z);
    else if constexpr (ACT == kActGelu) { float e; return z * normal_cdf(z, e); }
    else if constexpr (ACT == kActGeluTanh) return z * logistic(2.0f * kTanhC * z * fmaf(kTanhA * z, z, 1.0f));
    else return z;
}

// act(z) and act'(z).  relu'(0) = 0.  A NaN comes out of both, relu's too, so that
// it is not lost on the way to the gradients.  The silu slope adds v (1 - p) to p,
// in that order: p + v first would lose p to v's rounding where z is large.  The
// tanh form's slope is constant beyond |z| = 32 (0 or 1 in fp32), and z is held
// inside that range there so that its z^3 does not overflow into inf * 0.
template <int ACT>
QL_DEV void act_slope(float z, float& v, float& d) {
    if constexpr (ACT == kActRelu) {
        v = z <= 0.0f ? 0.0f : z;
        d = z <= 0.0f ? 0.0f : z > 0.0f ? 1.0f : z;
    } else if constexpr (ACT == kActSilu) {
        const float p = logistic(z);
        v = z * p;
        d = fmaf(v, 1.0f - p, p);
    } else if constexpr (ACT == kActGelu) {
        float e;
        const float p = normal_cdf(z, e);
        v = z * p;
        d = fmaf(z * kInvSqrt2Pi, e, p);
    } else if constexpr (ACT == kActGeluTanh) {
        const float c = z > 32.0f ? 32.0f : z < -32.0f ? -32.0f : z;
        const float p = logistic(2.0f * kTanhC * c * fmaf(kTanhA * c, c, 1.0f));
        v = z * p;
        d = fmaf(c * p * (1.0f - p), 2.0f * kTanhC * fmaf(3.0f * kTanhA * c, c, 1.0f), p);
    } else {
        v = z;
        d = 1.0f;
    }
}

// act(v[e]) for a uniform activation
template <int N>
QL_DEV void act_values(int act, float (&v)[N]) {
    switch (act) {
        case kActRelu:
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = act_value<kActRelu>(v[e]);
            break;
        case kActSilu:
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = act_value<kActSilu>(v[e]);
            break;
        case kActGelu:
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = act_value<kActGelu>(v[e]);
            break;
        case kActGeluTanh:
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = act_value<kActGeluTanh>(v[e]);
            break;
        default: break;
    }
}

// ------------------------------------------------------------------ 8-bit checkpoints
//
// Blocks of 64 consecutive values (row-major).  With c = max|x| of a block:
//   d = fl32(c / 127),  q = fl32(x fl32(127 / c)) rounded to an integer, ties to even,
// and the block stands for q d.  The scale and the factor are divided exactly
// (IEEE).  Rounding the product to fp32 first puts the exact ties of 127 x / c
// (c a multiple of 127 units) back on the tie, which an fma would miss by the
// factor's rounding; adding 1.5 * 2^23, whose ulp is 1, then leaves q in two's
// complement in the low byte.  |x| <= c keeps |q| <= 127.  A block whose c is below 2^-120
// (where 127 / c leaves the fp32 range) is stored as zeros (d = 0), and one
// that holds an inf or a NaN gets d = NaN, so it reads back as NaN and an
// overflow is not lost in the checkpoint.

// largest |x| bit pattern of the type that is finite
template <bool F16>
constexpr uint32_t kFiniteBits = F16 ? 0x7BFFu : 0x7F7Fu;

// scale d and the factor 127 / c of a block from the largest |x| bit pattern
template <bool F16>
QL_DEV void ck_scale(uint32_t m, float& d, float& inv) {
    const float c = F16 ? lo16<true>(m) : __uint_as_float(m << 16);
    const bool zero = c < 0x1p-120f;
    d = zero ? 0.0f : __fdiv_rn(c, 127.0f);
    inv = zero ? 0.0f : __fdiv_rn(127.0f, c);
    if (m > kFiniteBits<F16>) {
        d = __uint_as_float(0x7FC00000u);
        inv = 0.0f;
    }
}

// largest |x| bit pattern of a packed pair (both formats order like integers)
QL_DEV uint32_t abs_max2(uint32_t v, uint32_t m) { return max(m, max(v & 0x7FFFu, (v >> 16) & 0x7FFFu)); }

// max over the eight lanes of an aligned cluster (quad swaps, then the mirror
// that pairs the two quads)
QL_DEV uint32_t max_of_8_lanes(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x141, 0xF, 0xF, false));
    return m;
}

// fp32 whose low byte is the code of x (two roundings: not to be contracted)
QL_DEV uint32_t ck_code(float x, float inv) {
#pragma clang fp contract(off)
    const float n = x * inv;
    return __float_as_uint(n + 12582912.0f);
}

// codes of four values (two packed pairs), value 0 in the low byte
template <bool F16>
QL_DEV uint32_t ck_codes4(uint32_t a, uint32_t b, float inv) {
    const uint32_t q0 = ck_code(lo16<F16>(a), inv), q1 = ck_code(hi16<F16>(a), inv);
    const uint32_t q2 = ck_code(lo16<F16>(b), inv), q3 = ck_code(hi16<F16>(b), inv);
    // perm bytes 0..3 come from the second operand, 4..7 from the first
    const uint32_t lo = __builtin_amdgcn_perm(q1, q0, 0x0C0C0400u), hi = __builtin_amdgcn_perm(q3, q2, 0x04000C0Cu);
    return lo | hi;
}

// the four values fl32(q d) of a code dword
QL_DEV void ck_values4(uint32_t codes, float d, float* v) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = (float)(int8_t)(codes >> (8 * e)) * d;
}

template <bool F16>
QL_DEV u32x4_t pack8(const float (&v)[8]) {
    u32x4_t o;
#pragma unroll
    for (int p = 0; p < 4; ++p) o[p] = pack16x2<F16>(v[2 * p], v[2 * p + 1]);
    return o;
}
template <bool F16>
QL_DEV void unpack8(const u32x4_t& q, float (&v)[8]) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        v[2 * p] = lo16<F16>(q[p]);
        v[2 * p + 1] = hi16<F16>(q[p]);
    }
}

// RNE_16(fl32(q d)) of eight codes: the operand that a checkpoint puts into a
// matrix product
template <bool F16>
QL_DEV u32x4_t ck_pack8(const u32x2_t& codes, float d) {
    float v[8];
    ck_values4(codes[0], d, v);
    ck_values4(codes[1], d, v + 4);
    return pack8<F16>(v);
}

// ------------------------------------------------------------------ epilogue of the forward

// Z = product + bias, Y = act(Z) * mul + residual, all in fp32 with one
// rounding at each output.  z: Z in 16 bits; zc / zs: the checkpoint of that
// 16-bit Z.  Y may be the buffer of mul or residual (every element is read
// before the same thread writes it).
struct Epilogue {
    int act;
    const uint16_t* bias;     // [N], or null (as the other pointers)
    const uint16_t* mul;      // [T][N]
    const uint16_t* res;      // [T][N]
    uint16_t* z;              // [T][N]
    int8_t* zc;               // [T][N]
    float* zs;                // [T][N / 64]
};

// The epilogue of eight consecutive columns n .. n + 7 of row t (n % 8 == 0):
// product sums in v, the operands' eight 16-bit values in bq, mq, rq (unused
// where the operand is absent).  Eight consecutive lanes hold one 64-column
// block.
template <bool F16>
QL_DEV void epilogue8(const Epilogue& ep, float (&v)[8], const u32x4_t& bq, const u32x4_t& mq, const u32x4_t& rq,
                      int64_t t, int64_t n, int64_t N, uint16_t* y) {
    const int64_t at = t * N + n;
    float w[8];
    if (ep.bias) {
        unpack8<F16>(bq, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += w[e];
    }
    if (ep.z || ep.zc) {
        const u32x4_t zq = pack8<F16>(v);
        if (ep.z) *reinterpret_cast<u32x4_t*>(ep.z + at) = zq;
        if (ep.zc) {
            uint32_t m = 0;
#pragma unroll
            for (int p = 0; p < 4; ++p) m = abs_max2(zq[p], m);
            float d, inv;
            ck_scale<F16>(max_of_8_lanes(m), d, inv);
            *reinterpret_cast<u32x2_t*>(ep.zc + at) =
                u32x2_t{ck_codes4<F16>(zq[0], zq[1], inv), ck_codes4<F16>(zq[2], zq[3], inv)};
            if ((n & 63) == 0) ep.zs[at >> 6] = d;
        }
    }
    act_values(ep.act, v);
    if (ep.mul) {
        unpack8<F16>(mq, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= w[e];
    }
    if (ep.res) {
        unpack8<F16>(rq, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += w[e];
    }
    *reinterpret_cast<u32x4_t*>(y + at) = pack8<F16>(v);
}

// ------------------------------------------------------------------ backward of the epilogue

// One saved activation: 16-bit values, or a checkpoint (codes and scales).
struct Saved {
    const uint16_t* v;
    const int8_t* codes;
    const float* scale;
    bool present() const { return v || codes; }
};

// dZ = dY * mul * act'(Z) (16-bit, dz; null when dZ is dY itself), dmul = dY *
// act(Z) (null if not asked for), and fp32 column sums of dZ over each row
// range, part[range][N] (null without a bias gradient).
struct ActBwd {
    int act;
    const uint16_t* dy;
    Saved z, mul;
    uint16_t* dz;
    uint16_t* dmul;
    float* part;
    int64_t T, N, rows;       // rows: rows of one range (a multiple of 64)
    int blocks;               // workgroups of the elementwise pass, 0 = none
};

// Rows of one range: 64, or more where that would be over 64 ranges (the
// partials of the bias gradient are summed range by range).
constexpr int64_t kActBwdMaxRanges = 64;
inline int64_t act_bwd_rows(int64_t T) {
    return ((T + kActBwdMaxRanges - 1) / kActBwdMaxRanges + 63) / 64 * 64;
}
inline int64_t act_bwd_ranges(int64_t T) { return (T + act_bwd_rows(T) - 1) / act_bwd_rows(T); }

// d_bias[n] = RNE_16 of the sum of part[range][n] in range order, 256 columns
// per workgroup
struct BiasFin {
    const float* part;
    int64_t ranges, N;
    uint16_t* out;            // null = no job
};
inline int bias_fin_blocks(const BiasFin& b) { return b.out ? (int)((b.N + 255) / 256) : 0; }
template <bool F16>
QL_DEV void bias_fin(const BiasFin& b, int bid) {
    const int64_t n = (int64_t)bid * 256 + threadIdx.x;
    if (n >= b.N) return;
    float v = 0.0f;
#pragma unroll 8
    for (int64_t q = 0; q < b.ranges; ++q) v += b.part[q * b.N + n];
    b.out[n] = (uint16_t)(pack16x2<F16>(v, 0.0f) & 0xFFFFu);
}

hipError_t launch_act8_quantize(const uint16_t* x, int64_t numel, int8_t* codes, float* scale, hipStream_t s, bool f16);
hipError_t launch_act8_dequantize(const int8_t* codes, const float* scale, int64_t numel, uint16_t* out, hipStream_t s,
                                  bool f16);
// Splits of the two down projections of a backward and their fp32 partials.
struct DownPair {
    int s_g, s_p;
    float *gpart, *ppart;
};

// the elementwise pass, with the block scales of the dX product as extra
// workgroups of the same launch (either may be absent)
hipError_t launch_act_bwd(const ActBwd& a, const ScalesJob& sj, hipStream_t s, bool f16);
hipError_t launch_bias_fin(const BiasFin& b, hipStream_t s, bool f16);

}  // namespace ql
