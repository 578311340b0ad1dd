// The rank-r products of the LoRA branch on gfx950 (Volcengine article
// section 3.4 for the layer; the gradients follow by differentiation, and
// only the adapters receive them, "从LoRA到QLoRA" section 3.1):
//
//   down projections   P = s X A      [T, r]   (forward and backward)
//                      G = s dY B^T   [T, r]   (backward)
//   adapter gradients  dA = X^T G     [K, r]
//                      dB = P^T dY    [r, N]
//
// All four are bound by reading the big operand (X or dY) once from HBM; the
// r-wide operands are small and stay in L2.  They use v_mfma_f32_16x16x32_bf16
// (lane l holds 8 consecutive reduction elements of row / column l % 16, group
// l / 16; the 4 results of lane l are column l % 16, rows 4 (l / 16) .. +3).
//
// k_down: a workgroup owns 64 rows of X (or dY) and a range of the reduction,
// staged through LDS in whole cache lines; the ranges of one row tile are
// added in a fixed order by k_down_fin.  P and G leave as bf16 hi +
// lo pairs (hi = RNE(v), lo = RNE(v - hi)), row-major for the GEMM kernels and
// transposed for k_grad.
//
// k_grad: the adapter-gradient block product of grad.hpp, one 128-column x
// 64-rank block per workgroup; token ranges of different workgroups produce
// fp32 partials that k_grad_finalize sums in split order.  Every result is
// deterministic.
#include <type_traits>

#include "act.hpp"
#include "common.hpp"
#include "grad.hpp"
#include "plan.hpp"

namespace ql {

namespace {

constexpr int kThreads = 256;

template <bool F16>
QL_DEV f32x4_t mfma16(const bf16x8_t& a, const bf16x8_t& b, const f32x4_t& c) {
    return mfma16x16x32<F16>(a, b, c);
}

QL_DEV bf16x8_t as_bf16x8(const u32x4_t& v) { return __builtin_bit_cast(bf16x8_t, v); }

// hi = RNE_16(v), lo = RNE_16(v - hi) as 16-bit patterns (bf16, or fp16 when F16)
template <bool F16>
QL_DEV void split_hi_lo(float v, uint16_t& hi, uint16_t& lo) {
    const uint32_t hb = pack16x2<F16>(v, 0.0f) & 0xFFFFu;
    hi = (uint16_t)hb;
    lo = (uint16_t)(pack16x2<F16>(v - lo16<F16>(hb), 0.0f) & 0xFFFFu);
}

}  // namespace

// ------------------------------------------------------------------ down projections

struct DownArgs {
    const uint16_t* s;    // [T][L] bf16 (X or dY)
    const int8_t* sc;     // or its 8-bit checkpoint: codes [T][L] and
    const float* sd;      // scales [T][L / 64]
    const uint16_t* m;    // B [m_rows = r][ldm = N] bf16, or with TM A [L = K][m_rows = r]; ranks r .. r_pad-1 read as zero
    int64_t T, L, ldm, m_rows, r_pad;
    float scale;
    uint16_t* hi;         // [T][r_pad]
    uint16_t* lo;
    uint16_t* hit;        // [r_pad][ldt] (tokens [0, T8), T8 = T rounded up to 8) or null
    uint16_t* lot;
    int64_t T8, ldt;
    float* part;          // [splits][T][r_pad] fp32 partial sums (splits > 1)
    int splits;
    bool tm;              // M is A [K][r] (TM)
    ScalesJob sj;         // the dX kernel's transposed block scales, as extra workgroups (sj.blocks may be 0)
};

// v (already scaled) -> hi/lo at row t, column j of both layouts
template <bool F16>
QL_DEV void down_out(const DownArgs& a, int64_t t, int j, float v, bool rowmajor) {
    uint16_t h, lw;
    split_hi_lo<F16>(v, h, lw);
    if (rowmajor) {
        if (t < a.T) {
            a.hi[t * a.r_pad + j] = h;
            a.lo[t * a.r_pad + j] = lw;
        }
    } else if (t < a.T8) {          // tokens [T, T8) are zeros (their S rows read as zero)
        a.hit[j * a.ldt + t] = h;
        a.lot[j * a.ldt + t] = lw;
    }
}

// sum[ROWS][R] (row stride R + 4) of rows t0 .. t0+ROWS-1 -> both output layouts
template <int R, int ROWS, bool F16>
QL_DEV void down_emit(const DownArgs& a, const float* sum, int64_t t0) {
    for (int e = threadIdx.x; e < ROWS * R; e += kThreads) {      // [T][r_pad], j fastest
        const int tl = e / R, j = e % R;
        down_out<F16>(a, t0 + tl, j, sum[tl * (R + 4) + j] * a.scale, true);
    }
    if (a.hit)
        for (int e = threadIdx.x; e < ROWS * R; e += kThreads) {  // [r_pad][ldt], t fastest
            const int j = e / ROWS, tl = e % ROWS;
            down_out<F16>(a, t0 + tl, j, sum[tl * (R + 4) + j] * a.scale, false);
        }
}

// out[t][j] = scale * sum_l S[t][l] M[j][l].  A workgroup owns 64 rows t
// (wave w: rows 16w .. 16w+15, all r_pad columns) and one of `splits` ranges
// of the reduction, walked in rounds of 64: each round's 64 rows of S and
// r_pad rows of M (128 contiguous bytes per row) are loaded PD rounds ahead
// into registers, written to a swizzled LDS buffer and read back as MFMA
// fragments, so every global load fetches whole cache lines and M is read
// once per 64 rows.  With several splits each workgroup stores an fp32
// partial (whole rows, through LDS) and k_down_fin adds them in split order.
//
// Q8: S is an 8-bit checkpoint.  A round is one block of 64 codes per row, so a
// thread loads the eight codes of its 16-byte chunk and the row's scale, and
// rounds the eight values q d to 16 bits on their way to LDS, so no 16-bit copy
// of a checkpointed X exists.  A round costs what a 16-bit one does and carries
// half the bytes: 4096 x 11008 in 8 bits takes 25 us where 4096 x 4096 in 16 takes
// 10.  No single part of a round bounds it (leaving out the MFMAs, the M tile or
// any of the loads saves 1 to 3 us of 22 each); it is the chain of instructions and
// barriers.
//
// TM: M is stored with the reduction as the row index (A [K][r]).  A thread
// loads the same eight ranks of two consecutive k and writes the pairs (k, k + 1)
// as dwords of the [rank][k] tile, so A needs no transposed copy.
template <int RT, bool F16, bool TM, bool Q8>
QL_DEV void down_block(const DownArgs& a, int bid, uint8_t* smem_raw) {
    constexpr int PD = RT <= 4 ? 4 : 2;
    constexpr int NX = 2;            // 16-byte chunks of the 64 x 64 S tile per thread
    constexpr int NM = RT / 2;       // 16-byte chunks of the r_pad x 64 M tile per thread
    constexpr int R = RT * 16;
    lds8_t* smem = (lds8_t*)(smem_raw);
    constexpr uint32_t kXT = 64 * 128, kMT = R * 128, kBuf = kXT + kMT;
    const int tiles = (int)ceil_div(a.T, 64);
    const int l = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int tile = bid % tiles, split = bid / tiles;
    const int64_t t0 = (int64_t)tile * 64;
    const int nr_all = (int)(a.L / 64);
    const int r0 = split * nr_all / a.splits, r1 = (split + 1) * nr_all / a.splits;
    const int nr = r1 - r0;

    const rsrc_t rx = Q8 ? make_rsrc(a.sc, a.T * a.L) : make_rsrc(a.s, a.T * a.L * 2);
    [[maybe_unused]] const rsrc_t rd = make_rsrc(a.sd, Q8 ? a.T * a.L / 16 : 0);
    const rsrc_t rm = make_rsrc(a.m, a.m_rows * (TM ? a.L : a.ldm) * 2);
    const uint32_t mrow = (uint32_t)(a.m_rows * 2);                   // TM: bytes of a row of A
    const uint32_t mround = TM ? 64u * mrow : 128u;                   // bytes of M between rounds
    uint32_t xo[NX], mo[NM];
    [[maybe_unused]] uint32_t dof[NX];
#pragma unroll
    for (int u = 0; u < NX; ++u) {
        const int q = threadIdx.x + u * kThreads;
        const int64_t t = t0 + (q >> 3);
        xo[u] = t < a.T ? (uint32_t)((t * a.L + (int64_t)r0 * 64 + (q & 7) * 8) * (Q8 ? 1 : 2)) : kOOB;
        if constexpr (Q8) dof[u] = t < a.T ? (uint32_t)((t * (a.L / 64) + r0) * 4) : kOOB;
    }
#pragma unroll
    for (int u = 0; u < NM; ++u) {
        if constexpr (TM) {
            // unit u / 2 of the thread: k pair and rank chunk; u & 1: the pair's row
            const int e = threadIdx.x + (u >> 1) * kThreads;
            const int pair = e / (2 * RT), jc = (e % (2 * RT)) * 8;
            mo[u] = jc < a.m_rows ? (uint32_t)(((int64_t)r0 * 64 + 2 * pair + (u & 1)) * mrow + jc * 2) : kOOB;
        } else {
            const int q = threadIdx.x + u * kThreads;
            const int64_t j = q >> 3;
            mo[u] = j < a.m_rows ? (uint32_t)((j * a.ldm + (int64_t)r0 * 64 + (q & 7) * 8) * 2) : kOOB;
        }
    }
    using xreg_t = std::conditional_t<Q8, u32x2_t, u32x4_t>;
    xreg_t xr[PD][NX];
    [[maybe_unused]] uint32_t dr[PD][NX];
    u32x4_t mr[PD][NM];
    auto load = [&](int i, int slot) {           // round i of this split (zeros past nr)
        const bool ok = i < nr;
        const uint32_t so = ok ? (uint32_t)i * 128u : 0u, sm = ok ? (uint32_t)i * mround : 0u;
#pragma unroll
        for (int u = 0; u < NX; ++u) {
            if constexpr (Q8) {
                xr[slot][u] = bload8(rx, ok ? xo[u] : kOOB, so >> 1);
                dr[slot][u] = bload4(rd, ok ? dof[u] : kOOB, so >> 5);
            } else {
                xr[slot][u] = bload16(rx, ok ? xo[u] : kOOB, so);
            }
        }
#pragma unroll
        for (int u = 0; u < NM; ++u) mr[slot][u] = bload16(rm, ok ? mo[u] : kOOB, sm);
    };
    auto store = [&](int slot, lds8_t* buf) {
#pragma unroll
        for (int u = 0; u < NX; ++u) {
            const int q = threadIdx.x + u * kThreads;
            u32x4_t v;
            if constexpr (Q8) v = ck_pack8<F16>(xr[slot][u], __uint_as_float(dr[slot][u]));
            else v = xr[slot][u];
            *reinterpret_cast<lds_u32x4_t*>(buf + lds_off(q >> 3, q & 7)) = v;
        }
        if constexpr (TM) {
#pragma unroll
            for (int u = 0; u < NM; u += 2) {
                const int e = threadIdx.x + (u >> 1) * kThreads;
                const int pair = e / (2 * RT), jc = (e % (2 * RT)) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t sel = (i & 1) ? 0x07060302u : 0x05040100u;
                    *reinterpret_cast<lds_u32_t*>(buf + kXT + lds_off(jc + i, pair >> 2) + (pair & 3) * 4) =
                        __builtin_amdgcn_perm(mr[slot][u + 1][i >> 1], mr[slot][u][i >> 1], sel);
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < NM; ++u) {
                const int q = threadIdx.x + u * kThreads;
                *reinterpret_cast<lds_u32x4_t*>(buf + kXT + lds_off(q >> 3, q & 7)) = mr[slot][u];
            }
        }
    };

    f32x4_t acc[RT];
#pragma unroll
    for (int jt = 0; jt < RT; ++jt) acc[jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    // Up to 128 ranks the fragments of a round (64 ranks) or step are read before
    // its first MFMA: the compiler would otherwise reuse one register set and
    // wait out an LDS latency in front of every MFMA (5-10% of the launch).
    // Above that they do not fit the registers.
    auto compute = [&](const lds8_t* buf) {
        auto xfrag = [&](int st) {
            return *reinterpret_cast<const lds_bf16x8_t*>(buf + lds_off(16 * w + (l & 15), 4 * st + (l >> 4)));
        };
        auto mfrag = [&](int st, int jt) {
            return *reinterpret_cast<const lds_bf16x8_t*>(buf + kXT + lds_off(16 * jt + (l & 15), 4 * st + (l >> 4)));
        };
        if constexpr (RT <= 8) {
            constexpr int G = RT <= 4 ? 2 : 1;   // steps read together
#pragma unroll
            for (int s0 = 0; s0 < 2; s0 += G) {
                bf16x8_t xv[G], mv[G][RT];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    xv[g] = xfrag(s0 + g);
#pragma unroll
                    for (int jt = 0; jt < RT; ++jt) mv[g][jt] = mfrag(s0 + g, jt);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int jt = 0; jt < RT; ++jt) acc[jt] = mfma16<F16>(xv[g], mv[g][jt], acc[jt]);
            }
        } else {
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                const bf16x8_t xv = xfrag(st);
#pragma unroll
                for (int jt = 0; jt < RT; ++jt) acc[jt] = mfma16<F16>(xv, mfrag(st, jt), acc[jt]);
            }
        }
    };
    // the loop runs whole groups of PD rounds (rounds past nr load zeros), so
    // it has no branches and the loads stay in flight across it
#pragma unroll
    for (int p = 0; p < PD; ++p) load(p, p);
    for (int i = 0; i < nr; i += PD) {
#pragma unroll
        for (int p = 0; p < PD; ++p) {
            lds8_t* buf = smem + ((i + p) & 1) * kBuf;
            store(p, buf);
            load(i + p + PD, p);
            __syncthreads();
            compute(buf);
        }
    }

    // the tile's sums [64][R] in LDS (the round buffers are free after a barrier)
    __syncthreads();
    float* sum = reinterpret_cast<float*>(smem_raw);
#pragma unroll
    for (int jt = 0; jt < RT; ++jt)
#pragma unroll
        for (int v = 0; v < 4; ++v) sum[(16 * w + 4 * (l >> 4) + v) * (R + 4) + 16 * jt + (l & 15)] = acc[jt][v];
    __syncthreads();
    if (a.splits == 1) {
        down_emit<R, 64, F16>(a, sum, t0);
        return;
    }
    float* out = a.part + (int64_t)split * a.T * a.r_pad;     // whole rows, 16 bytes per lane
    for (int e = threadIdx.x; e < 16 * R; e += kThreads) {
        const int tl = e / (R / 4), j = 4 * (e % (R / 4));
        const int64_t t = t0 + tl;
        if (t < a.T) {
            const float* src = sum + tl * (R + 4) + j;
            *reinterpret_cast<f32x4_t*>(out + t * a.r_pad + j) = f32x4_t{src[0], src[1], src[2], src[3]};
        }
    }
}

template <int RT, bool F16, bool TM>
__global__ __launch_bounds__(kThreads, 2) void k_down(DownArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const int n = (int)ceil_div(a.T, 64) * a.splits, bid = (int)blockIdx.x;
    if (bid >= n) {                             // block-scale workgroups of the same launch, dispatched
        scales_job(a.sj, bid - n, (lds8_t*)smem_raw);     // after the longer projection workgroups
        return;
    }
    down_block<RT, F16, TM, false>(a, bid, smem_raw);
}

// Both down projections of a backward in one launch, then the sums of the bias
// gradient: workgroups [0, n0) take a0 (s dZ B^T), [n0, n0 + n1) a1 (s X A, X a
// checkpoint when Q8), the rest 256 columns of the bias gradient each.
template <int RT, bool F16, bool Q8>
__global__ __launch_bounds__(kThreads, 2) void k_down2(DownArgs a0, DownArgs a1, int n0, int n1, BiasFin bf) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const int bid = (int)blockIdx.x;
    if (bid < n0) down_block<RT, F16, false, false>(a0, bid, smem_raw);
    else if (bid < n0 + n1) down_block<RT, F16, true, Q8>(a1, bid - n0, smem_raw);
    else bias_fin<F16>(bf, bid - n0 - n1);
}

// Split-ordered sum of the k_down partials of 16 rows, then both layouts.
template <int RT, bool F16>
QL_DEV void down_fin_block(const DownArgs& a, int bid, uint8_t* smem_raw) {
    constexpr int R = RT * 16;
    float* sum = reinterpret_cast<float*>(smem_raw);           // [16][R + 4]
    const int64_t t0 = (int64_t)bid * 16;
    for (int e = threadIdx.x; e < 4 * R; e += kThreads) {
        const int tl = e / (R / 4), j = 4 * (e % (R / 4));
        const int64_t t = t0 + tl;
        f32x4_t s4 = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s0 = 0; s0 < a.splits; s0 += 8) {                // eight loads issued together
            f32x4_t v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int sp = s0 + q;
                v[q] = (sp < a.splits && t < a.T)
                           ? *reinterpret_cast<const f32x4_t*>(a.part + ((int64_t)sp * a.T + t) * a.r_pad + j)
                           : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) s4 += v[q];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) sum[tl * (R + 4) + j + c] = s4[c];
    }
    __syncthreads();
    down_emit<R, 16, F16>(a, sum, t0);
}

// workgroups [0, n0) take a0, the rest a1 (n0 workgroups alone for one problem)
template <int RT, bool F16>
__global__ __launch_bounds__(kThreads) void k_down_fin(DownArgs a0, DownArgs a1, int n0) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const int bid = (int)blockIdx.x;
    if (bid < n0) down_fin_block<RT, F16>(a0, bid, smem_raw);
    else down_fin_block<RT, F16>(a1, bid - n0, smem_raw);
}

// ------------------------------------------------------------------ adapter gradients

// One launch serves both adapter gradients: workgroups [0, blocks0) take
// problem a0 (dA = X^T G), the rest problem a1 (dB = P^T dY); blockIdx.y
// picks the 64 ranks.  Q8: a0's X is an 8-bit checkpoint.
template <bool F16, bool Q8>
__global__ __launch_bounds__(kThreads, 1) void k_grad(GradArgs a0, GradArgs a1, int blocks0) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const bool second = (int)blockIdx.x >= blocks0;
    const GradArgs& a = second ? a1 : a0;
    const int bx = second ? (int)blockIdx.x - blocks0 : (int)blockIdx.x;
    float* red = reinterpret_cast<float*>(smem_raw);
    if constexpr (Q8) {
        if (!second) {
            grad_block<F16, true>(a0, bx % a0.cblocks, bx / a0.cblocks, (int64_t)blockIdx.y * 64, red);
            return;
        }
    }
    grad_block<F16, false>(a, bx % a.cblocks, bx / a.cblocks, (int64_t)blockIdx.y * 64, red);
}

// dA[k][j] (transpose = 0) or dB[j][n] (transpose = 1): RNE_bf16 of the
// split-ordered sum of part[s][c][j], j < r.  One workgroup per 16 columns c;
// a thread sums four consecutive j with its split loads issued in batches of
// eight.  The transposed output goes through an LDS tile so that its stores
// run along c.  Workgroups [0, blocks0) serve the first problem, the rest the
// second.
struct GradFin {
    const float* part;
    int splits;
    int64_t C, r_pad, r;
    uint16_t* out;
    int transpose;
};

template <bool F16>
__global__ __launch_bounds__(256) void k_grad_finalize(GradFin f0, GradFin f1, int blocks0) {
    __shared__ uint16_t tile[256][16 + 2];              // [j][c] for the transposed output
    const bool second = (int)blockIdx.x >= blocks0;
    const GradFin& f = second ? f1 : f0;
    const int64_t c0 = (int64_t)(second ? (int)blockIdx.x - blocks0 : (int)blockIdx.x) * 16;
    const int64_t stride = f.C * f.r_pad;
    const int q = (int)(f.r_pad / 4);
    for (int e = threadIdx.x; e < 16 * q; e += 256) {
        const int cl = e / q, j = 4 * (e % q);
        const int64_t c = c0 + cl;
        f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
        if (c < f.C) {
            const float* src = f.part + c * f.r_pad + j;
            int s = 0;
            for (; s + 8 <= f.splits; s += 8) {
                f32x4_t v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) v[u] = *reinterpret_cast<const f32x4_t*>(src + (int64_t)(s + u) * stride);
#pragma unroll
                for (int u = 0; u < 8; ++u) sum += v[u];
            }
            for (; s < f.splits; ++s) sum += *reinterpret_cast<const f32x4_t*>(src + (int64_t)s * stride);
        }
        const uint32_t p01 = pack16x2<F16>(sum[0], sum[1]), p23 = pack16x2<F16>(sum[2], sum[3]);
        if (!f.transpose) {
            if (c < f.C && j < f.r) *reinterpret_cast<u32x2_t*>(f.out + c * f.r + j) = u32x2_t{p01, p23};
        } else {
            tile[j][cl] = (uint16_t)p01;
            tile[j + 1][cl] = (uint16_t)(p01 >> 16);
            tile[j + 2][cl] = (uint16_t)p23;
            tile[j + 3][cl] = (uint16_t)(p23 >> 16);
        }
    }
    if (!f.transpose) return;
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * f.r; e += 256) {
        const int j = e / 16, cl = e % 16;
        const int64_t c = c0 + cl;
        if (c < f.C) f.out[j * f.C + c] = tile[j][cl];
    }
}

// ------------------------------------------------------------------ launchers

namespace {

template <class F>
hipError_t set_smem(F* f, size_t bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(f), hipFuncAttributeMaxDynamicSharedMemorySize,
                               (int)bytes);
}

template <int RT, bool F16>
hipError_t down_rt(const DownArgs& a, hipStream_t s) {
    constexpr int R = RT * 16;
    const size_t bufs = (size_t)2 * (64 + R) * 128, sums = (size_t)64 * (R + 4) * 4;
    const size_t lds = bufs > sums ? bufs : sums;
    const unsigned tiles = (unsigned)ceil_div(a.T, 64);
    auto go = [&](auto kern) {
        hipError_t e = set_smem(kern, lds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3(tiles * (unsigned)a.splits + (unsigned)a.sj.blocks), dim3(kThreads), lds, s, a);
        return hipGetLastError();
    };
    hipError_t e = a.tm ? go(k_down<RT, F16, true>) : go(k_down<RT, F16, false>);
    if (e != hipSuccess) return e;
    if (a.splits > 1) {
        const size_t fl = (size_t)16 * (R + 4) * 4;
        const int n = (int)ceil_div(a.T, 16);
        hipLaunchKernelGGL((k_down_fin<RT, F16>), dim3((unsigned)n), dim3(kThreads), fl, s, a, a, n);
    }
    return hipGetLastError();
}

// a0 and (when `second`) a1 in one k_down2 launch, the split sums of both in one more
template <int RT, bool F16>
hipError_t down2_rt(const DownArgs& a0, const DownArgs& a1, bool second, const BiasFin& bf, hipStream_t s) {
    constexpr int R = RT * 16;
    const size_t bufs = (size_t)2 * (64 + R) * 128, sums = (size_t)64 * (R + 4) * 4;
    const size_t lds = bufs > sums ? bufs : sums;
    const int tiles = (int)ceil_div(a0.T, 64), n0 = tiles * a0.splits, n1 = second ? tiles * a1.splits : 0;
    auto go = [&](auto kern) {
        hipError_t e = set_smem(kern, lds);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3((unsigned)(n0 + n1 + bias_fin_blocks(bf))), dim3(kThreads), lds, s, a0, a1, n0,
                           n1, bf);
        return hipGetLastError();
    };
    hipError_t e = a1.sc ? go(k_down2<RT, F16, true>) : go(k_down2<RT, F16, false>);
    if (e != hipSuccess) return e;
    const int f = (int)ceil_div(a0.T, 16), f0 = a0.splits > 1 ? f : 0, f1 = second && a1.splits > 1 ? f : 0;
    if (f0 + f1 > 0) {
        const size_t fl = (size_t)16 * (R + 4) * 4;
        hipLaunchKernelGGL((k_down_fin<RT, F16>), dim3((unsigned)(f0 + f1)), dim3(kThreads), fl, s, a0, a1, f0);
    }
    return hipGetLastError();
}

template <bool F16>
hipError_t down2_t(const DownArgs& a0, const DownArgs& a1, bool second, const BiasFin& bf, hipStream_t s) {
    switch (a0.r_pad / 16) {
        case 4: return down2_rt<4, F16>(a0, a1, second, bf, s);
        case 8: return down2_rt<8, F16>(a0, a1, second, bf, s);
        case 12: return down2_rt<12, F16>(a0, a1, second, bf, s);
        case 16: return down2_rt<16, F16>(a0, a1, second, bf, s);
        default: return hipErrorInvalidValue;
    }
}

template <bool F16>
hipError_t down_t(const DownArgs& a, hipStream_t s) {
    switch (a.r_pad / 16) {
        case 4: return down_rt<4, F16>(a, s);
        case 8: return down_rt<8, F16>(a, s);
        case 12: return down_rt<12, F16>(a, s);
        case 16: return down_rt<16, F16>(a, s);
        default: return hipErrorInvalidValue;
    }
}

hipError_t down(const DownArgs& a, hipStream_t s, bool f16) { return f16 ? down_t<true>(a, s) : down_t<false>(a, s); }

// One k_grad launch over up to two problems (`n1` = 0: a0 alone).
hipError_t grad(const GradArgs& a0, int n0, const GradArgs& a1, int n1, int64_t r_pad, hipStream_t s, bool f16) {
    auto go = [&](auto kern) {
        hipError_t e = set_smem(kern, kGradSmem);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(kern, dim3((unsigned)(n0 + n1), (unsigned)(r_pad / 64)), dim3(kThreads), kGradSmem, s,
                           a0, a1, n0);
        return hipGetLastError();
    };
    if (a0.sc) return f16 ? go(k_grad<true, true>) : go(k_grad<false, true>);
    return f16 ? go(k_grad<true, false>) : go(k_grad<false, false>);
}

// One k_grad_finalize launch for dA (fa, when has_a) and dB (fb, when has_b).
hipError_t grad_finalize(GradFin fa, bool has_a, const GradFin& fb, bool has_b, const LoraPlan& pl, hipStream_t s,
                         bool f16) {
    const int ba = has_a ? (int)ceil_div(pl.K, 16) : 0;
    const int bb = has_b ? (int)ceil_div(pl.N, 16) : 0;
    if (!has_a) fa = fb;                   // a single problem runs as the first one
    if (f16)
        hipLaunchKernelGGL(k_grad_finalize<true>, dim3((unsigned)(ba + bb)), dim3(256), 0, s, fa, fb,
                           has_a ? ba : bb);
    else
        hipLaunchKernelGGL(k_grad_finalize<false>, dim3((unsigned)(ba + bb)), dim3(256), 0, s, fa, fb,
                           has_a ? ba : bb);
    return hipGetLastError();
}

}  // namespace

namespace {

// s X A -> P (hi/lo [T][r_pad]; also transposed when `transposed`)
DownArgs down_x_args(const Saved& x, const uint16_t* lora_a, float scaling, const LoraPlan& pl, uint8_t* ws,
                     bool transposed) {
    return DownArgs{x.v, x.codes, x.scale, lora_a, pl.T, pl.K, pl.r, pl.r, pl.r_pad, scaling,
                    reinterpret_cast<uint16_t*>(ws + pl.off_ps_hi), reinterpret_cast<uint16_t*>(ws + pl.off_ps_lo),
                    transposed ? reinterpret_cast<uint16_t*>(ws + pl.off_pst_hi) : nullptr,
                    transposed ? reinterpret_cast<uint16_t*>(ws + pl.off_pst_lo) : nullptr, pl.T8, pl.ld_t,
                    reinterpret_cast<float*>(ws + pl.off_dpart), pl.s_down_x, true, ScalesJob{}};
}

// s dY B^T -> G (hi/lo [T][r_pad], also transposed when `transposed`)
DownArgs down_dy_args(const uint16_t* dy, const uint16_t* lora_b, float scaling, const LoraPlan& pl, uint8_t* ws,
                      bool transposed) {
    return DownArgs{dy, nullptr, nullptr, lora_b, pl.T, pl.N, pl.N, pl.r, pl.r_pad, scaling,
                    reinterpret_cast<uint16_t*>(ws + pl.off_gs_hi), reinterpret_cast<uint16_t*>(ws + pl.off_gs_lo),
                    transposed ? reinterpret_cast<uint16_t*>(ws + pl.off_gst_hi) : nullptr,
                    transposed ? reinterpret_cast<uint16_t*>(ws + pl.off_gst_lo) : nullptr, pl.T8, pl.ld_t,
                    reinterpret_cast<float*>(ws + pl.off_dpart), pl.s_down_dy, false, ScalesJob{}};
}

}  // namespace

hipError_t launch_lora_down_x(const uint16_t* x, const uint16_t* lora_a, float scaling, const LoraPlan& pl,
                              uint8_t* ws, bool transposed, hipStream_t s, bool f16) {
    return down(down_x_args(Saved{x, nullptr, nullptr}, lora_a, scaling, pl, ws, transposed), s, f16);
}

// `scales` (if not NULL) runs as extra workgroups of the same launch.
hipError_t launch_lora_down_dy(const uint16_t* dy, const uint16_t* lora_b, float scaling, const LoraPlan& pl,
                               uint8_t* ws, bool transposed, hipStream_t s, bool f16, const ScalesJob* scales) {
    DownArgs a = down_dy_args(dy, lora_b, scaling, pl, ws, transposed);
    if (scales) a.sj = *scales;
    return down(a, s, f16);
}

// G and, with `x` present, P, both transposed too then; and the bias gradient.
// `splits` ranges of each reduction, whose partials are at gpart and ppart.
hipError_t launch_lora_down_pair(const uint16_t* dz, const uint16_t* lora_a, const uint16_t* lora_b, const Saved& x,
                                 float scaling, const LoraPlan& pl, uint8_t* ws, const DownPair& dp,
                                 const BiasFin& bf, hipStream_t s, bool f16) {
    const bool second = x.present();
    DownArgs a0 = down_dy_args(dz, lora_b, scaling, pl, ws, second);
    DownArgs a1 = down_x_args(x, lora_a, scaling, pl, ws, true);
    a0.part = dp.gpart;
    a0.splits = dp.s_g;
    a1.part = dp.ppart;
    a1.splits = dp.s_p;
    return f16 ? down2_t<true>(a0, a1, second, bf, s) : down2_t<false>(a0, a1, second, bf, s);
}

// dA = X^T G and dB = P^T dY from the transposed intermediates in ws.
hipError_t launch_lora_grads(const Saved& x, const uint16_t* dy, const LoraPlan& pl, uint8_t* ws,
                             uint16_t* d_lora_a, uint16_t* d_lora_b, hipStream_t s, bool f16) {
    float* pda = reinterpret_cast<float*>(ws + pl.off_pda);
    float* pdb = reinterpret_cast<float*>(ws + pl.off_pdb);
    GradFin fa{pda, pl.s_da, pl.K, pl.r_pad, pl.r, d_lora_a, 0};
    GradFin fb{pdb, pl.s_db, pl.N, pl.r_pad, pl.r, d_lora_b, 1};
    // dA and dB in one launch (either may be absent)
    const GradArgs ga{x.v, x.codes, x.scale, reinterpret_cast<const uint16_t*>(ws + pl.off_gst_hi),
                      reinterpret_cast<const uint16_t*>(ws + pl.off_gst_lo), pda, pl.T, pl.T8, pl.ld_t, pl.K,
                      pl.r_pad, (int)ceil_div(pl.K, 128), pl.cpw_da};
    const GradArgs gb{dy, nullptr, nullptr, reinterpret_cast<const uint16_t*>(ws + pl.off_pst_hi),
                      reinterpret_cast<const uint16_t*>(ws + pl.off_pst_lo), pdb, pl.T, pl.T8, pl.ld_t, pl.N,
                      pl.r_pad, (int)ceil_div(pl.N, 128), pl.cpw_db};
    const int na = d_lora_a ? ga.cblocks * pl.s_da : 0, nb = d_lora_b ? gb.cblocks * pl.s_db : 0;
    {
        hipError_t e = na ? grad(ga, na, gb, nb, pl.r_pad, s, f16) : grad(gb, nb, gb, 0, pl.r_pad, s, f16);
        if (e != hipSuccess) return e;
    }
    return grad_finalize(fa, d_lora_a != nullptr, fb, d_lora_b != nullptr, pl, s, f16);
}

// The fused backward's gradient problems: S = X against G^T for dA and S = dY
// against P^T for dB, one group of fz_tpg 256-token tiles per split, partials
// in the fused region of ws.
FusedGrads fused_grads_for(const uint16_t* x, const uint16_t* dy, const LoraPlan& pl, uint8_t* ws, bool da,
                           bool db) {
    FusedGrads f{};
    f.tpg = pl.fz_tpg;
    f.groups = pl.s_fz;
    f.waves = 0;                                   // set by the dX launcher from its grid
    if (da)
        f.ga = GradArgs{x, nullptr, nullptr, reinterpret_cast<const uint16_t*>(ws + pl.off_gst_hi),
                        reinterpret_cast<const uint16_t*>(ws + pl.off_gst_lo), reinterpret_cast<float*>(ws + pl.off_fza),
                        pl.T, pl.T8, pl.ld_t, pl.K, pl.r_pad, (int)ceil_div(pl.K, 128), 8};
    if (db)
        f.gb = GradArgs{dy, nullptr, nullptr, reinterpret_cast<const uint16_t*>(ws + pl.off_pst_hi),
                        reinterpret_cast<const uint16_t*>(ws + pl.off_pst_lo), reinterpret_cast<float*>(ws + pl.off_fzb),
                        pl.T, pl.T8, pl.ld_t, pl.N, pl.r_pad, (int)ceil_div(pl.N, 128), 8};
    return f;
}

// dA and dB from the fused backward's partials (one per 256-token tile).
hipError_t launch_fused_grads_finalize(const LoraPlan& pl, uint8_t* ws, uint16_t* d_lora_a, uint16_t* d_lora_b,
                                       hipStream_t s, bool f16) {
    const GradFin fa{reinterpret_cast<const float*>(ws + pl.off_fza), pl.s_fz, pl.K, pl.r_pad, pl.r, d_lora_a, 0};
    const GradFin fb{reinterpret_cast<const float*>(ws + pl.off_fzb), pl.s_fz, pl.N, pl.r_pad, pl.r, d_lora_b, 1};
    return grad_finalize(fa, d_lora_a != nullptr, fb, d_lora_b != nullptr, pl, s, f16);
}

}  // namespace ql
