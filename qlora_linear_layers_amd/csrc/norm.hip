// Root-mean-square norm with the residual's addition, and its backward, for
// gfx950.  With r = (mean(h^2) + eps)^(-1/2), n = h r and g = dy w:
//   y  = n w
//   dx = r (g - n mean(g n)) + dx_add,   dw = sum over rows of dy n
// (d r / d h_j = -r^3 h_j / D, so the norm's slope takes from g its part along n;
// mean(g n) is r mean(g h), so that one pass over a row gives both sums).  Both are
// bound by HBM: a row stays in its team's registers (rows.hpp), every input is read
// once and every output written once; only the backward of rows past 12288 values
// reads them twice.
#include <algorithm>

#include "rows.hpp"

namespace ql {

namespace {

// Eight weights as they are stored: 16-bit in lo, fp32 in lo and hi, ones
// without a weight and zeros past the end.
struct WChunk {
    u32x4_t lo, hi;
};
template <bool F16>
QL_DEV WChunk weight_load(const void* w, int w32, int c, int D) {
    WChunk k;
    const int e0 = c * 8;
    if (!w) {
        k.lo = k.hi = u32x4_t{0x3F800000u, 0x3F800000u, 0x3F800000u, 0x3F800000u};
    } else if (!w32) {
        k.lo = row_load(static_cast<const uint16_t*>(w), c, D);
        k.hi = u32x4_t{0, 0, 0, 0};
    } else {
        const uint32_t* p = static_cast<const uint32_t*>(w) + e0;
        if (e0 + 8 <= D) {
            k.lo = *reinterpret_cast<const u32x4_t*>(p);
            k.hi = *reinterpret_cast<const u32x4_t*>(p + 4);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                k.lo[e] = e0 + e < D ? p[e] : 0u;
                k.hi[e] = e0 + 4 + e < D ? p[4 + e] : 0u;
            }
        }
    }
    return k;
}
template <bool F16>
QL_DEV void weight_values(const WChunk& k, bool wide, float (&v)[8]) {
    if (wide) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = __uint_as_float(k.lo[e]);
            v[4 + e] = __uint_as_float(k.hi[e]);
        }
    } else {
        unpack8<F16>(k.lo, v);
    }
}

// Rows whose squares leave fp32 are summed again scaled by a power of two (exact), eps with
// its square:
//   above (the sum and eps over 2^128): 2^-72; the sum of an inf stays inf (r = 0), of a NaN NaN;
//   below (both under 2^-40): 2^64.  Squares of values below 2^-63 lose bits, and the
//     hardware's rsq takes an argument below 2^-126 as 0, whose root would make a row of zeros
//     0 * inf.  Scaled, eps alone is at least 2^-21.
constexpr float kHuge = 0x1p-72f, kTiny = 0x1p64f;

// the power of two for a row's unscaled sum of squares (the same in the whole team)
QL_DEV float row_scale(float ss, float eps) {
    const float both = ss + eps;
    return !(both < __builtin_inff()) ? kHuge : both < 0x1p-40f ? kTiny : 1.0f;
}

// 1 / sqrt of the mean square of the row times `pre`, eps scaled with it
QL_DEV float inv_rms(float ss, int D, float eps, float pre) {
    return __builtin_amdgcn_rsqf(ss / (float)D + eps * pre * pre);
}

}  // namespace

// y = n w of a row per team.  With a residual, calls in a row over eight sets of inputs (more
// than the caches hold): 2048 x 8192 to 16 bits (134 MB) 23.8 us, 5.6 TB/s, to 8 bits (117 MB)
// 23.5, 2048 x 4096 13.4 and 13.2, 8192 x 1024 13.0.  Over three sets, which the last cache
// mostly holds, 2048 x 8192 takes 19.9 and 19.8 (21.0 with h stored through the caches).
template <bool F16, bool Q8, int LANES, int CH>
__global__ __launch_bounds__(team_threads(LANES)) void k_rmsnorm(NormArgs a) {
    __shared__ float slots[2][32];
    const int lane = (int)threadIdx.x & (LANES - 1), D = a.D;
    const int64_t row = (int64_t)blockIdx.x * (team_threads(LANES) / LANES) + threadIdx.x / LANES;
    const bool ok = row < a.T;
    const int64_t at = (ok ? row : a.T - 1) * D;
    u32x4_t h[CH];
    WChunk w[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) h[j] = row_load(a.x + at, lane + j * LANES, D);
    if (a.res) {
        u32x4_t q[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j) q[j] = row_load(a.res + at, lane + j * LANES, D);
#pragma unroll
        for (int j = 0; j < CH; ++j) w[j] = weight_load<F16>(a.w, a.w32, lane + j * LANES, D);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float u[8], v[8];
            unpack8<F16>(h[j], u);
            unpack8<F16>(q[j], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] += v[e];
            h[j] = pack8<F16>(u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < CH; ++j) w[j] = weight_load<F16>(a.w, a.w32, lane + j * LANES, D);
    }
    if (a.h && ok) {
        if (a.far) {
#pragma unroll
            for (int j = 0; j < CH; ++j) row_store_far(a.h + at, lane + j * LANES, D, h[j]);
        } else {
#pragma unroll
            for (int j = 0; j < CH; ++j) row_store(a.h + at, lane + j * LANES, D, h[j]);
        }
    }
    const auto squares = [&](float pre) {
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float v[8];
            unpack8<F16>(h[j], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(v[e] * pre, v[e] * pre, s);
        }
        return s;
    };
    float ss = team_sum<LANES>(squares(1.0f), slots[0]);
    const float pre = row_scale(ss, a.eps);
    if (pre != 1.0f) {
        if constexpr (LANES > 64) __syncthreads();      // slots[0] is read
        ss = team_sum<LANES>(squares(pre), slots[0]);
    }
    const float r = inv_rms(ss, D, a.eps, pre);
    const bool wide = a.w32 || !a.w;
    const auto normed = [&](int j, float (&y)[8]) {
        float g[8];
        unpack8<F16>(h[j], y);
        weight_values<F16>(w[j], wide, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * pre * r * g[e];
    };
    if (a.y && ok) {
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float y[8];
            normed(j, y);
            row_store(a.y + at, lane + j * LANES, D, pack8<F16>(y));
        }
    }
    if constexpr (Q8) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float y[8];
            normed(j, y);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if ((lane + j * LANES) * 8 + e < D) m = max(m, __float_as_uint(y[e]) & 0x7FFFFFFFu);
        }
        m = team_umax<LANES>(m, slots[1]);
        float d, inv;
        rows8_scale(m, d, inv);
        if (ok) {
            const int P = (int)rows8_pitch(D);
            int8_t* cr = a.codes + row * P;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int c = lane + j * LANES;
                float y[8];
                normed(j, y);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = c * 8 + e < D ? y[e] : 0.0f;
                if (c * 8 < P) *reinterpret_cast<u32x2_t*>(cr + c * 8) = rows8_codes(y, inv);
            }
            if (lane == 0) a.scale[row] = d;
        }
    }
}

// dx of a row per team and step, the teams striding over the rows.  A lane holds the
// same columns of every row, so its share of dw stays in registers, and one fp32
// partial row per workgroup is written at the end (DW).  Rows up to 12288 values are
// held in registers, the next row's loads issued before this row's sums (kHold); longer
// ones are read again after the sums, from the caches.  With dw, three chunks a thread of
// held rows spill 60 to 72 bytes a lane at 256 registers, four chunks of 1024 threads 260 to
// 320 at 128.
//
// 4096 x 8192 with dx_add and fp32 weights, 268 MB: 46.6 us, 5.8 TB/s (FAR; 48.4 through the
// caches), and 4.7 us for the sum of the partials.  One workgroup a CU (256): through the
// caches with two 61.9 us in all, against 55.7, with three 68.7 (more partials, and the held
// rows leave no registers for a second one).  Up to 6144 values, where 256 threads hold a row,
// that is one wave a SIMD: 2048 x 4096 with dx_add 20.7 us in all against 11.3 for its 67 MB.
template <bool F16, bool DW, bool FAR, int LANES, int CH>
__global__ __launch_bounds__(team_threads(LANES)) void k_rmsnorm_bwd(NormBwd a, int64_t teams) {
    __shared__ float slots[2][32];
    constexpr int kTeams = team_threads(LANES) / LANES;
    constexpr bool kHold = LANES < 1024;
    const int lane = (int)threadIdx.x & (LANES - 1), D = a.D;
    const int64_t team = (int64_t)blockIdx.x * kTeams + threadIdx.x / LANES;
    const bool wide = a.w32 || !a.w;
    constexpr int kRegs = kHold ? CH : 1;
    WChunk w[kRegs];
    u32x4_t hn[kRegs], dyn[kRegs], an[kRegs];
    float dw[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        if constexpr (kHold) w[j] = weight_load<F16>(a.w, a.w32, lane + j * LANES, D);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[j][e] = 0.0f;
    }
    const float invD = 1.0f / (float)D;
    const auto load = [&](int64_t row) {
        const int64_t at = row * D;
        const auto get = [&](const uint16_t* p, int c) { return FAR ? row_load_far(p, c, D) : row_load(p, c, D); };
#pragma unroll
        for (int j = 0; j < CH; ++j) hn[j] = get(a.h + at, lane + j * LANES);
#pragma unroll
        for (int j = 0; j < CH; ++j) dyn[j] = get(a.dy + at, lane + j * LANES);
        if (a.add) {
#pragma unroll
            for (int j = 0; j < CH; ++j) an[j] = get(a.add + at, lane + j * LANES);
        }
    };
    if constexpr (kHold)
        if (team < a.T) load(team);
    int par = 0;
#pragma unroll 1
    for (int64_t row = team; row < a.T; row += teams) {
        const int64_t at = row * D;
        u32x4_t hq[kRegs], dyq[kRegs], aq[kRegs];
        if constexpr (kHold) {
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                hq[j] = hn[j];
                dyq[j] = dyn[j];
                aq[j] = an[j];
            }
            if (row + teams < a.T) load(row + teams);
        }
        // chunk j: h, dy and the weights in fp32
        const auto chunk = [&](int j, float (&h)[8], float (&dy)[8], float (&g)[8]) {
            const int c = lane + j * LANES;
            if constexpr (kHold) {
                unpack8<F16>(hq[j], h);
                unpack8<F16>(dyq[j], dy);
                weight_values<F16>(w[j], wide, g);
            } else {
                const u32x4_t hc = row_load(a.h + at, c, D), dyc = row_load(a.dy + at, c, D);
                const WChunk wc = weight_load<F16>(a.w, a.w32, c, D);
                unpack8<F16>(hc, h);
                unpack8<F16>(dyc, dy);
                weight_values<F16>(wc, wide, g);
            }
        };
        // over the row's values: f(sum, h, dy w)
        const auto sum = [&](auto f) {
            float s = 0.0f;
            const auto add = [&](int j) {
                float h[8], dy[8], g[8];
                chunk(j, h, dy, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) s = f(s, h[e], dy[e] * g[e]);
            };
            if constexpr (kHold) {
#pragma unroll
                for (int j = 0; j < CH; ++j) add(j);
            } else {
#pragma unroll 1
                for (int j = 0; j < CH; ++j) add(j);
            }
            return s;
        };
        float ss = 0.0f, gh = 0.0f;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            float h[8], dy[8], g[8];
            chunk(j, h, dy, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(h[e], h[e], ss);
                gh = fmaf(dy[e] * g[e], h[e], gh);
            }
        }
        team_sum2<LANES>(ss, gh, slots[par]);
        const float pre = row_scale(ss, a.eps);
        float r = inv_rms(ss, D, a.eps, 1.0f);
        float m = gh * r * invD;                        // mean(g n)
        // The squares or g h leave fp32: first r, then the mean from n itself.  The branch below
        // costs least as an unlikely one where the row is held (2048 x 4096 19.2 -> 19.4 us for
        // the whole case, 2048 x 11008 unchanged), and as a uniform one where it is read again
        // (1000 x 20000 104 -> 98 us, as an unlikely one 112: the registers spill elsewhere).
        const bool rare = pre != 1.0f || !(fabsf(m) < __builtin_inff());
        const auto again = [&]() {
            if constexpr (LANES > 64) __syncthreads();
            ss = team_sum<LANES>(sum([&](float s, float h, float) { return fmaf(h * pre, h * pre, s); }), slots[par]);
            r = inv_rms(ss, D, a.eps, pre);
            if constexpr (LANES > 64) __syncthreads();
            m = team_sum<LANES>(sum([&](float s, float h, float g) { return fmaf(g, h * pre * r * invD, s); }), slots[par]);
        };
        if constexpr (kHold) {
            if (__builtin_expect(rare, 0)) again();
        } else {
            if (__builtin_amdgcn_readfirstlane(rare)) again();
        }
        par ^= 1;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            // the packed values are what stays in registers over the sums, not their fp32 forms
            if constexpr (kHold) asm("" : "+v"(hq[j]), "+v"(dyq[j]));
            else asm volatile("" ::: "memory");
            const int c = lane + j * LANES;
            float h[8], dy[8], g[8];
            chunk(j, h, dy, g);
            u32x4_t add = {0, 0, 0, 0};
            if (a.add) {
                if constexpr (kHold) add = aq[j];
                else add = row_load(a.add + at, c, D);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = h[e] * pre * r;
                if constexpr (DW) dw[j][e] = fmaf(dy[e], n, dw[j][e]);
                h[e] = (dy[e] * g[e] - n * m) * r * pre;
            }
            if (a.add) {
                unpack8<F16>(add, dy);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] += dy[e];
            }
            row_store(a.dx + at, c, D, pack8<F16>(h));
        }
    }
    if constexpr (DW) {
        float* const part = a.part + (int64_t)blockIdx.x * D;
        if constexpr (kTeams > 1) {
            // the workgroup's teams are added in team order
            __shared__ float all[kTeams][LANES * CH * 8];
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) all[threadIdx.x / LANES][(lane + j * LANES) * 8 + e] = dw[j][e];
            __syncthreads();
            for (int c = (int)threadIdx.x; c < D; c += team_threads(LANES)) {
                float v = all[0][c];
#pragma unroll
                for (int q = 1; q < kTeams; ++q) v += all[q][c];
                part[c] = v;
            }
        } else {
#pragma unroll
            for (int j = 0; j < CH; ++j) {
                const int e0 = (lane + j * LANES) * 8;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e0 + e < D) part[e0 + e] = dw[j][e];
            }
        }
    }
}

// dw: 64 columns per workgroup, 16 waves that each add every sixteenth partial;
// their sums are added in wave order.  Bound by latency: 8.4 MB in 4.8 us (D = 8192).
template <bool F16>
__global__ __launch_bounds__(1024) void k_rmsnorm_dw(const float* __restrict__ part, int64_t groups, int D, int w32,
                                                     void* __restrict__ dw) {
    __shared__ float sum[16][64];
    const int c = (int)blockIdx.x * 64 + ((int)threadIdx.x & 63), wv = (int)threadIdx.x >> 6;
    float v = 0.0f;
    if (c < D) {
#pragma unroll 8
        for (int64_t q = wv; q < groups; q += 16) v += part[q * D + c];
    }
    sum[wv][threadIdx.x & 63] = v;
    __syncthreads();
    if (wv == 0 && c < D) {
#pragma unroll
        for (int q = 1; q < 16; ++q) v += sum[q][threadIdx.x];
        if (w32) static_cast<float*>(dw)[c] = v;
        else static_cast<uint16_t*>(dw)[c] = (uint16_t)(pack16x2<F16>(v, 0.0f) & 0xFFFFu);
    }
}

// ------------------------------------------------------------------ launchers

namespace {

// Team of a row: one wave up to 2048 values, 256 threads up to 6144, 512 up to 8192,
// else 1024 (2048 x 8192: 256 threads 28.4 us, 512 26.0, 1024 26.2 to 8 bits and 28.7 to
// 16).
template <class Go>
void for_norm_team(int64_t D, Go go) {
    const int64_t c = ceil_div(D, 8);
    if (c <= 64) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
    else if (c <= 128) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
    else if (c <= 256) go(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
    else if (c <= 512) go(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
    else if (c <= 768) go(std::integral_constant<int, 256>{}, std::integral_constant<int, 3>{});
    else if (c <= 1024) go(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
    else if (c <= 2048) go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
}

// What passes by the caches, so that what the next kernel needs stays in them.
//
// Forward: h, which a block reads again behind its products or in the backward, where it is
// larger than the L2 caches of the eight XCDs together.  us with it stored through / past the
// caches, with a consumer of y (16 bits) behind each call: 1722 x 8192 (27 MiB of h) 27.3 /
// 26.9, 2048 x 8192 35.8 / 31.9, 4096 x 8192 67.1 / 62.5; 3444 x 4096 29.2 / 27.0, 4096 x 4096
// 35.3 / 31.0; y in 8 bits 26.9 / 25.0, 31.3 / 28.7 and 59.2 / 56.2; odd rows gain alike (4000 x
// 4099 46.0 / 40.0).  Where h is read at once instead, storing it past the caches costs: 1024 x
// 8192 17.0 / 18.5, 2048 x 8192 34.6 / 35.9, 4096 x 8192 67.6 / 68.4.
//
// Backward: its rows, read for the last time, where the call touches more than the 256 MiB
// cache behind them.  With dx_add (8 bytes a value) 3444 x 8192 (215 MiB) 44.5 / 44.0, 4096 x
// 8192 51.5 / 49.3, 8192 x 8192 103 / 88; 27554 x 1024 40.2 / 41.0, 38967 x 1024 58.4 / 54.5.
// Without (6 bytes) 4870 x 8192 (228 MiB) 46.9 / 47.0, 5792 x 8192 54.1 / 53.3, 8192 x 8192 80.8 /
// 69.4.  Not for rows of odd alignment, whose lines are read twice: 8200 x 4099 174 / 198, 4100 x
// 8194 97 / 102.  A template argument there: a branch around the loads cost 57 us against 49.6.
constexpr int64_t kL2Bytes = int64_t(32) << 20, kCacheBytes = int64_t(256) << 20;

// The backward holds rows of up to 12288 values in 512 threads (us, 1024 threads that read
// the row twice / 512 that hold it: 2048 x 11008 68.9 / 55.5, 4096 x 8448 with a consumer of dx
// 133.8 / 98.4; with four chunks a thread, 4096 x 16384, more registers spill: 133.6 / 159.9).
template <class Go>
void for_bwd_team(int64_t D, Go go) {
    const int64_t c = ceil_div(D, 8);
    if (c > 1024 && c <= 1536) go(std::integral_constant<int, 512>{}, std::integral_constant<int, 3>{});
    else for_norm_team(D, go);
}

// Workgroups of the backward (one a CU) and its teams
constexpr int64_t kBwdGroups = 256;
int64_t bwd_per(int64_t D) { return D <= 2048 ? 4 : 1; }
int64_t bwd_groups(int64_t T, int64_t D) { return std::min(kBwdGroups, ceil_div(T, bwd_per(D))); }

}  // namespace

hipError_t launch_rmsnorm(NormArgs a, hipStream_t s, bool f16) {
    a.far = a.T * a.D * 2 >= kL2Bytes;
    for_norm_team(a.D, [&](auto lanes, auto ch) {
        constexpr int L = decltype(lanes)::value, C = decltype(ch)::value;
        const dim3 g((unsigned)ceil_div(a.T, team_threads(L) / L)), b(team_threads(L));
        if (a.codes) {
            if (f16) hipLaunchKernelGGL((k_rmsnorm<true, true, L, C>), g, b, 0, s, a);
            else hipLaunchKernelGGL((k_rmsnorm<false, true, L, C>), g, b, 0, s, a);
        } else {
            if (f16) hipLaunchKernelGGL((k_rmsnorm<true, false, L, C>), g, b, 0, s, a);
            else hipLaunchKernelGGL((k_rmsnorm<false, false, L, C>), g, b, 0, s, a);
        }
    });
    return hipGetLastError();
}

int64_t rmsnorm_bwd_partials(int64_t T, int64_t D) { return bwd_groups(T, D); }

hipError_t launch_rmsnorm_bwd(const NormBwd& a, hipStream_t s, bool f16) {
    const int64_t groups = bwd_groups(a.T, a.D), teams = groups * bwd_per(a.D);
    const bool far = a.T * a.D * (a.add ? 8 : 6) >= kCacheBytes && a.D % 8 == 0;
    for_bwd_team(a.D, [&](auto lanes, auto ch) {
        constexpr int L = decltype(lanes)::value, C = decltype(ch)::value;
        const dim3 g((unsigned)groups), b(team_threads(L));
        const auto go = [&](auto kern) { hipLaunchKernelGGL(kern, g, b, 0, s, a, teams); };
        const auto of = [&](auto f) {
            constexpr bool F = decltype(f)::value && L < 1024;
            if (a.dw) f16 ? go(k_rmsnorm_bwd<true, true, F, L, C>) : go(k_rmsnorm_bwd<false, true, F, L, C>);
            else f16 ? go(k_rmsnorm_bwd<true, false, F, L, C>) : go(k_rmsnorm_bwd<false, false, F, L, C>);
        };
        far ? of(std::true_type{}) : of(std::false_type{});
    });
    if (a.dw) {
        const dim3 g((unsigned)ceil_div(a.D, 64));
        if (f16) hipLaunchKernelGGL(k_rmsnorm_dw<true>, g, dim3(1024), 0, s, a.part, groups, a.D, a.w32, a.dw);
        else hipLaunchKernelGGL(k_rmsnorm_dw<false>, g, dim3(1024), 0, s, a.part, groups, a.D, a.w32, a.dw);
    }
    return hipGetLastError();
}

}  // namespace ql
