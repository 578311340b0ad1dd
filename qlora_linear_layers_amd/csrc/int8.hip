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

// Eight channels n .. n + 7 of token t: 16-byte accesses of 2-byte alignment, or
// element by element where the last of them lie past N.
struct EpiRow {
    u32x4_t w0, w1, bias, mul, res;
    float xs;
};
QL_DEV EpiRow epi_row_load(const Int8Args& a, int64_t t, int64_t n) {
    const int64_t at = t * a.N + n;
    EpiRow o;
    o.xs = a.xs[t];
    o.w0 = *reinterpret_cast<const u32x4_t*>(a.ws + n);
    o.w1 = *reinterpret_cast<const u32x4_t*>(a.ws + n + 4);
    o.bias = o.mul = o.res = u32x4_t{0, 0, 0, 0};
    if (a.ep.bias) o.bias = *reinterpret_cast<const u32x4_t*>(a.ep.bias + n);
    if (a.ep.mul) o.mul = *reinterpret_cast<const u32x4_a2*>(a.ep.mul + at);
    if (a.ep.res) o.res = *reinterpret_cast<const u32x4_a2*>(a.ep.res + at);
    return o;
}
template <bool F16>
QL_DEV void epi_row_store(const Int8Args& a, const EpiRow& o, int64_t t, int64_t n, const int (&sum)[8]) {
    float v[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = int8_scaled(sum[e], o.xs, __uint_as_float(e < 4 ? o.w0[e] : o.w1[e - 4]));
    if (a.ep.bias) {
        unpack8<F16>(o.bias, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += w[e];
    }
    act_values(a.ep.act, v);
    if (a.ep.mul) {
        unpack8<F16>(o.mul, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= w[e];
    }
    if (a.ep.res) {
        unpack8<F16>(o.res, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += w[e];
    }
    *reinterpret_cast<u32x4_a2*>(a.y + t * a.N + n) = pack8<F16>(v);
}
template <bool F16>
QL_DEV void int8_epilogue8(const Int8Args& a, int64_t t, int64_t n, const int (&sum)[8]) {
    if (n + 8 <= a.N) {
        epi_row_store<F16>(a, epi_row_load(a, t, n), t, n, sum);
    } else {
#pragma unroll 1
        for (int e = 0; n + e < a.N; ++e) {
            int v = sum[0];
#pragma unroll
            for (int q = 1; q < 8; ++q) v = e == q ? sum[q] : v;
            a.y[t * a.N + n + e] = epi_value<F16>(a, epi_load(a, t, n + e), v);
        }
    }
}

// Workgroup -> (channel tile, token tile).  Workgroups are dealt round-robin to
// the 8 XCDs: each XCD gets a contiguous range of tiles, walked in bands of four
// token tiles, so that the workgroups that share an L2 share operands.
QL_DEV void int8_tile_of(int pid, int gn, int gt, int& tn, int& tt) {
    const int g = gn * gt, per = g >> 3;
    const int l = pid < 8 * per ? (pid & 7) * per + (pid >> 3) : pid;
    constexpr int kBand = 4;
    const int band = l / (kBand * gn), within = l % (kBand * gn);
    const int bw = gt - band * kBand < kBand ? gt - band * kBand : kBand;
    tn = within / bw;
    tt = band * kBand + within % bw;
}

// Scheduling hint of one step: an LDS read behind every MFMA until they are out.
template <int kMfma, int kReads>
QL_DEV void int8_interleave() {
#pragma unroll
    for (int j = 0; j < kMfma; ++j) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);               // MFMA
        if (j < kReads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // DS read
    }
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

// ------------------------------------------------------------------ tiles
//
// BN channels x BM tokens per workgroup of four waves (WN x WM of them), K in
// tiles of 128 bytes, double-buffered in LDS and filled by loads that go there
// directly.  LDS rows are 128 bytes with their 16-byte chunks XOR-swizzled
// (lds_off); a direct load writes 64 consecutive chunks (eight rows), so the
// swizzle is applied to the chunk that a lane reads from memory.  Rows past N or T
// repeat the last one (their outputs are not stored).

typedef __attribute__((address_space(3))) i32x4_t lds_i32x4_t;

template <int BN, int BM, int WN, int WM>
struct Int8Tile {
    static constexpr int kLoads = (BN + BM) / 32;             // direct loads per thread and k tile
    static constexpr int kStage = (BN + BM) * 128;
    static constexpr int NI = BN / WN / 32, NJ = BM / WM / 32;  // 32 x 32 MFMA tiles of a wave
    rsrc_t rw, rx;
    uint32_t voff[kLoads];
    int wave;

    QL_DEV void init(const Int8Args& a, int64_t n0, int64_t t0) {
        wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        const int64_t rn = a.N - n0 < BN ? a.N - n0 : BN, rt = a.T - t0 < BM ? a.T - t0 : BM;
        rw = make_rsrc(a.w + n0 * a.P, rn * a.P);
        rx = make_rsrc(a.x + t0 * a.P, rt * a.P);
        const int l = (int)threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = (i * 4 + wave) * 8 + (l >> 3);      // row of the stage: W rows, then X rows
            const int row = i < BN / 32 ? (q < rn ? q : (int)rn - 1) : (q - BN < rt ? q - BN : (int)rt - 1);
            voff[i] = (uint32_t)row * (uint32_t)a.P + ((uint32_t)((l & 7) ^ ((q ^ (q >> 3)) & 7)) << 4);
        }
    }
    QL_DEV void load(lds8_t* stage, int kt) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(i < BN / 32 ? rw : rx, stage + (i * 4 + wave) * 1024, 16, voff[i],
                                                     kt * 128, 0, 0);
    }
};

QL_DEV i32x4_t int8_frag(const lds8_t* base, int row, int chunk) {
    return *reinterpret_cast<const lds_i32x4_t*>(base + lds_off(row, chunk));
}

// s0, s1: the two stages, LDS variables of their own, so that the compiler knows
// that a load into one is no hazard for reads of the other.
template <bool F16, int BN, int BM, int WN, int WM>
QL_DEV void int8_tile(const Int8Args& a, lds8_t* s0, lds8_t* s1) {
    using Tile = Int8Tile<BN, BM, WN, WM>;
    constexpr int NI = Tile::NI, NJ = Tile::NJ;
    const int gn = (int)ceil_div(a.N, BN), gt = (int)ceil_div(a.T, BM);
    int tn, tt;
    int8_tile_of((int)blockIdx.x, gn, gt, tn, tt);
    const int64_t n0 = (int64_t)tn * BN, t0 = (int64_t)tt * BM;
    Tile tl;
    tl.init(a, n0, t0);
    const int lane = (int)threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wn = tl.wave % WN, wm = tl.wave / WN;
    const int rowa = wn * (BN / WN) + r, rowb = BN + wm * (BM / WM) + r;
    i32x16_t acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;
    const int KT = a.P / 128;

    i32x4_t fa[2][NI], fb[2][NJ];
    const auto read = [&](int set, const lds8_t* st, int step) {
#pragma unroll
        for (int i = 0; i < NI; ++i) fa[set][i] = int8_frag(st, rowa + 32 * i, 2 * step + h);
#pragma unroll
        for (int j = 0; j < NJ; ++j) fb[set][j] = int8_frag(st, rowb + 32 * j, 2 * step + h);
    };
    const auto mfma = [&](int set, int j) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[set][i], fb[set][j], acc[i][j], 0, 0, 0);
    };
    const auto tile = [&](lds8_t* cur, lds8_t* nxt, int kt) {
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            read((s + 1) & 1, cur, s + 1);
#pragma unroll
            for (int j = 0; j < NJ; ++j) mfma(s & 1, j);
            int8_interleave<NI * NJ, NI + NJ>();
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < NJ / 2; ++j) mfma(1, j);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0070);                   // vmcnt(0) lgkmcnt(0): the next stage is loaded, this one read
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        tl.load(cur, kt + 2 < KT ? kt + 2 : KT - 1);          // past the end: the last one again, which nothing reads
        read(0, nxt, 0);
#pragma unroll
        for (int j = NJ / 2; j < NJ; ++j) mfma(1, j);
        __builtin_amdgcn_sched_barrier(0);
    };
    tl.load(s0, 0);
    tl.load(s1, KT > 1 ? 1 : 0);
    __builtin_amdgcn_s_waitcnt(0x0070);
    __syncthreads();
    read(0, s0, 0);
    int kt = 0;
#pragma unroll 1
    for (; kt + 1 < KT; kt += 2) {
        tile(s0, s1, kt);
        tile(s1, s0, kt + 1);
    }
    if (kt < KT) tile(s0, s1, kt);

    // Epilogue: 32 tokens of every wave at a time through LDS (sums of 32 WM tokens
    // x BN channels, 4-channel chunks swizzled by the token), then whole rows: eight
    // channels per thread.
    constexpr int kRow = BN * 4, kTok = 32 * WM;
    static_assert(kTok * kRow <= Tile::kStage, "one pass of the epilogue fits a stage");
    lds8_t* const st = s0;
    __builtin_amdgcn_s_waitcnt(0x0070);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        __syncthreads();
        const int tk = wm * 32 + r;
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = (wn * (BN / WN) + 32 * i + 8 * g + 4 * h) >> 2;
                *reinterpret_cast<lds_i32x4_t*>(st + tk * kRow + ((c ^ (tk & 31)) << 4)) =
                    i32x4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
            }
        __syncthreads();
#pragma unroll 4
        for (int u = (int)threadIdx.x; u < kTok * BN / 8; u += 256) {
            const int tk2 = u / (BN / 8), c8 = u % (BN / 8);
            const int64_t t = t0 + (tk2 >> 5) * (BM / WM) + 32 * j + (tk2 & 31), n = n0 + c8 * 8;
            if (t >= a.T || n >= a.N) continue;
            const i32x4_t lo = *reinterpret_cast<const lds_i32x4_t*>(st + tk2 * kRow + (((2 * c8) ^ (tk2 & 31)) << 4));
            const i32x4_t hi = *reinterpret_cast<const lds_i32x4_t*>(st + tk2 * kRow + (((2 * c8 + 1) ^ (tk2 & 31)) << 4));
            const int sum[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            int8_epilogue8<F16>(a, t, n, sum);
        }
    }
}

template <bool F16, int BN, int BM, int WN, int WM>
__global__ __launch_bounds__(256) void k_int8_tile(Int8Args a) {
    __shared__ __align__(1024) uint8_t s0[(BN + BM) * 128];
    __shared__ __align__(1024) uint8_t s1[(BN + BM) * 128];
    int8_tile<F16, BN, BM, WN, WM>(a, (lds8_t*)s0, (lds8_t*)s1);
}

size_t int8_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_int8(const Int8Args& a, void*, hipStream_t s, bool f16) {
    const auto go = [&](auto kern, int nt) {
        hipLaunchKernelGGL(kern, dim3((unsigned)ceil_div(a.N, 16), (unsigned)ceil_div(a.T, 16 * nt)),
                           dim3(64 * kSkinnyWaves), 0, s, a);
    };
    const auto tiles = [&](auto kern, int bn, int bm) {
        hipLaunchKernelGGL(kern, dim3((unsigned)(ceil_div(a.N, bn) * ceil_div(a.T, bm))), dim3(256), 0, s, a);
    };
    if (a.T > 512) {
        f16 ? tiles(k_int8_tile<true, 256, 256, 2, 2>, 256, 256) : tiles(k_int8_tile<false, 256, 256, 2, 2>, 256, 256);
        return hipGetLastError();
    }
    if (a.T > 64) {
        f16 ? tiles(k_int8_tile<true, 128, 128, 2, 2>, 128, 128) : tiles(k_int8_tile<false, 128, 128, 2, 2>, 128, 128);
        return hipGetLastError();
    }
    if (a.T <= 16) f16 ? go(k_int8_skinny<true, 1>, 1) : go(k_int8_skinny<false, 1>, 1);
    else f16 ? go(k_int8_skinny<true, 4>, 4) : go(k_int8_skinny<false, 4>, 4);
    return hipGetLastError();
}

}  // namespace ql
