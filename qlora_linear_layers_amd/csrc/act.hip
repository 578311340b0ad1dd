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
// is an integer max over the lanes (DPP swaps, no LDS), and a thread takes four
// 8-value chunks 256 threads apart, so every wave instruction covers contiguous
// bytes.  Only the last block can be partial.  2048 x 22016 values, 138 MB read
// and written: 23.6 us, 5.85 TB/s, the rate of a large copy; the counted HBM
// bytes are 1.001 of these.
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

// The values back: 23.3 us for the same size (5.9 TB/s).
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

// A saved activation as buffers: 16-bit values, or codes and scales; an absent
// one has empty buffers and reads zeros.  Eight values at element `at`
// (a multiple of 8), loaded raw and turned into fp32 later.
struct SavedRow {
    u32x4_t q;                // 16-bit values, or the codes in the first two dwords
    uint32_t d;
};
struct SavedBuf {
    rsrc_t rv, rd;
    bool q8;
    QL_DEV SavedBuf(const Saved& s, int64_t numel) : q8(s.codes != nullptr) {
        rv = q8 ? make_rsrc(s.codes, numel) : make_rsrc(s.v, s.v ? numel * 2 : 0);
        rd = make_rsrc(s.scale, q8 ? numel / 16 : 0);
    }
    QL_DEV SavedRow load(bool ok, uint32_t at) const {
        SavedRow r;
        if (q8) {
            const u32x2_t c = bload8(rv, ok ? at : kOOB, 0);
            r.q = u32x4_t{c[0], c[1], 0, 0};
            r.d = bload4(rd, ok ? at / 64 * 4 : kOOB, 0);
        } else {
            r.q = bload16(rv, ok ? at * 2 : kOOB, 0);
            r.d = 0;
        }
        return r;
    }
    template <bool F16>
    QL_DEV void values(const SavedRow& r, float (&v)[8]) const {
        if (q8) {
            ck_values4(r.q[0], __uint_as_float(r.d), v);
            ck_values4(r.q[1], __uint_as_float(r.d), v + 4);
        } else {
            unpack8<F16>(r.q, v);
        }
    }
};

}  // namespace

// A workgroup owns 128 columns (16 lanes of 8) and one range of rows, 16 row
// slots of two rows each per step: the loads of a step's rows are all issued
// before the first is used.  Column sums stay in registers over the steps; the
// 16 row slots of a column are then added in LDS in slot order, so d_bias is
// deterministic.  dmul, which nothing here reads again, is stored past the
// caches.
//
// Bound by HBM with the VALU behind it (about 25 instruction slots per element
// for silu, exp and the reciprocal counting four each): 2048 x 11008 with Z and
// mul as checkpoints, 183 MB, takes 38 us (4.8 TB/s).  Forming
// s dZ B^T in the same pass was slower: the registers of its fragments leave
// two workgroups a CU, too few to cover the memory latency (80 us for both
// against 41 + 21).
template <int ACT, bool F16>
QL_DEV void act_bwd_block(const ActBwd& a, int bid, float* red) {
    constexpr int U = 2;
    // workgroups are dealt round-robin to the 8 XCDs: neighbouring column blocks,
    // which share the cache lines of the scales, go to one XCD
    const int per = a.blocks >> 3;
    const int b = bid < 8 * per ? (bid & 7) * per + (bid >> 3) : bid;
    const int cb = (int)ceil_div(a.N, 128);
    const int bx = b % cb, by = b / cb;
    const int cl = threadIdx.x & 15, slot = threadIdx.x >> 4;
    const int64_t n = (int64_t)bx * 128 + cl * 8;
    const int64_t r0 = (int64_t)by * a.rows;
    const int64_t r1 = r0 + a.rows < a.T ? r0 + a.rows : a.T;
    const bool nok = n < a.N;
    const bool has_mul = a.mul.v || a.mul.codes;
    const rsrc_t rdy = make_rsrc(a.dy, a.T * a.N * 2);
    const SavedBuf zb(a.z, a.T * a.N), ub(a.mul, a.T * a.N);
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
#pragma unroll 1
    for (int64_t t0 = r0 + slot; t0 < r1; t0 += 16 * U) {
        u32x4_t dyq[U];
        SavedRow zr[U], ur[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + 16 * u;
            const bool ok = nok && t < r1;
            const uint32_t at = (uint32_t)(t * a.N + n);
            dyq[u] = bload16(rdy, ok ? at * 2 : kOOB, 0);
            zr[u] = zb.load(ok, at);
            ur[u] = ub.load(ok, at);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + 16 * u;
            const bool ok = nok && t < r1;
            float dy[8], z[8], m[8], h[8];
            unpack8<F16>(dyq[u], dy);
            zb.template values<F16>(zr[u], z);
            if (has_mul) ub.template values<F16>(ur[u], m);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float d;
                act_slope<ACT>(z[e], h[e], d);
                h[e] *= dy[e];
                if (has_mul) dy[e] *= m[e];
                dy[e] *= d;
            }
            if (a.part) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += dy[e];
            }
            if (ok) {
                if (a.dmul) __builtin_nontemporal_store(pack8<F16>(h), reinterpret_cast<u32x4_t*>(a.dmul + t * a.N + n));
                if (a.dz) *reinterpret_cast<u32x4_t*>(a.dz + t * a.N + n) = pack8<F16>(dy);
            }
        }
    }
    if (!a.part) return;
    constexpr int kRow = 128 + 4;
#pragma unroll
    for (int e = 0; e < 8; ++e) red[slot * kRow + cl * 8 + e] = sum[e];
    __syncthreads();
    if (threadIdx.x < 128) {
        const int64_t c = (int64_t)bx * 128 + threadIdx.x;
        float v = red[threadIdx.x];
#pragma unroll
        for (int q = 1; q < 16; ++q) v += red[q * kRow + threadIdx.x];
        if (c < a.N) a.part[(int64_t)by * a.N + c] = v;
    }
}

constexpr int kActBwdLds = 16 * 132 * 4;
static_assert(kScalesLds <= kActBwdLds, "the job shares the workgroup's LDS");

template <int ACT, bool F16>
__global__ __launch_bounds__(kThreads) void k_act_bwd(ActBwd a, ScalesJob sj) {
    __shared__ __align__(16) uint8_t lds[kActBwdLds];
    const int bid = (int)blockIdx.x;
    if (bid < a.blocks) act_bwd_block<ACT, F16>(a, bid, reinterpret_cast<float*>(lds));
    else scales_job(sj, bid - a.blocks, (lds8_t*)lds);
}

template <bool F16>
__global__ __launch_bounds__(kThreads) void k_bias_fin(BiasFin b) {
    bias_fin<F16>(b, (int)blockIdx.x);
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

hipError_t launch_act_bwd(const ActBwd& a, const ScalesJob& sj, hipStream_t s, bool f16) {
    const int n = a.blocks + sj.blocks;
    if (n == 0) return hipSuccess;
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3((unsigned)n), dim3(kThreads), 0, s, a, sj); };
    switch (a.act) {
        case kActRelu: f16 ? go(k_act_bwd<kActRelu, true>) : go(k_act_bwd<kActRelu, false>); break;
        case kActSilu: f16 ? go(k_act_bwd<kActSilu, true>) : go(k_act_bwd<kActSilu, false>); break;
        case kActGelu: f16 ? go(k_act_bwd<kActGelu, true>) : go(k_act_bwd<kActGelu, false>); break;
        case kActGeluTanh: f16 ? go(k_act_bwd<kActGeluTanh, true>) : go(k_act_bwd<kActGeluTanh, false>); break;
        default: f16 ? go(k_act_bwd<kActNone, true>) : go(k_act_bwd<kActNone, false>); break;
    }
    return hipGetLastError();
}

hipError_t launch_bias_fin(const BiasFin& b, hipStream_t s, bool f16) {
    const dim3 g((unsigned)bias_fin_blocks(b));
    if (f16) hipLaunchKernelGGL(k_bias_fin<true>, g, dim3(kThreads), 0, s, b);
    else hipLaunchKernelGGL(k_bias_fin<false>, g, dim3(kThreads), 0, s, b);
    return hipGetLastError();
}

}  // namespace ql
