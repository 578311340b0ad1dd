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

// Scheduling hint of kMfma MFMAs: the LDS reads and the loads into LDS spread evenly
// behind them.
template <int kMfma, int kReads, int kLoads>
QL_DEV void int8_interleave() {
#pragma unroll
    for (int j = 0; j < kMfma; ++j) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                   // MFMA
#pragma unroll
        for (int q = j * kReads / kMfma; q < (j + 1) * kReads / kMfma; ++q)
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);               // LDS read
#pragma unroll
        for (int q = j * kLoads / kMfma; q < (j + 1) * kLoads / kMfma; ++q)
            __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);               // load
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
// tiles of 128 bytes, whole cache lines: two buffers in LDS, filled by loads that go
// there directly.  A wave takes the fragments of a whole K tile into registers during
// the tile's first quarter, so that its buffer is free from then on and the loads of
// the tile after next are under way for 1.5 tiles.  LDS rows are 128 bytes with their
// 16-byte chunks XOR-swizzled (lds_off); a direct load writes 64 consecutive chunks
// (eight rows), so the swizzle is applied to the chunk that a lane reads from memory.
// Rows past N or T repeat the last one (their outputs are not stored).

typedef __attribute__((address_space(3))) i32x4_t lds_i32x4_t;
constexpr int kTileK = 128;

template <int BN, int BM, int WN, int WM>
struct Int8Tile {
    static constexpr int kLoads = (BN + BM) / 32;             // direct loads per thread and K tile
    static constexpr int kBuf = (BN + BM) * kTileK;
    static constexpr int NI = BN / WN / 32, NJ = BM / WM / 32;  // 32 x 32 MFMA tiles of a wave
    rsrc_t rw, rx;
    uint32_t voff[kLoads];
    int wave;

    QL_DEV void init(const Int8Args& a, int64_t n0, int64_t t0) {
        wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        // 32-bit: scalar units have no 64-bit compare, and a descriptor that goes through
        // vector registers costs a loop around every load
        const int rn = min((int)a.N - (int)n0, BN), rt = min((int)a.T - (int)t0, BM);
        rw = make_rsrc(a.w + n0 * a.P, rn * a.P);
        rx = make_rsrc(a.x + t0 * a.P, rt * a.P);
        const int l = (int)threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = (i * 4 + wave) * 8 + (l >> 3);      // row of the buffer: W rows, then X rows
            const int row = i < BN / 32 ? min(q, rn - 1) : min(q - BN, rt - 1);
            voff[i] = (uint32_t)row * (uint32_t)a.P + ((uint32_t)((l & 7) ^ ((q ^ (q >> 3)) & 7)) << 4);
        }
    }
    // loads i0 .. i1 - 1 of K tile kt
    QL_DEV void load(lds8_t* buf, int kt, int i0, int i1) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i >= i0 && i < i1)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(i < BN / 32 ? rw : rx, buf + (i * 4 + wave) * 1024, 16,
                                                         voff[i], kt * kTileK, 0, 0);
    }
};

QL_DEV i32x4_t int8_frag(const lds8_t* base, int row, int chunk) {
    return *reinterpret_cast<const lds_i32x4_t*>(base + lds_off(row, chunk));
}

// A wave's own wait, then the barrier.  __syncthreads would wait for the loads in
// flight, too (its fence covers what they write to LDS); the empty asm keeps the
// compiler from moving memory accesses over the barrier instead.
template <int kWait>
QL_DEV void wait_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(kWait);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
constexpr int kWaitLds = 0xC07F;                               // lgkmcnt(0)
constexpr int wait_loads(int n) { return 0x0F70 | (n & 15) | (n >> 4) << 14; }   // vmcnt(n)

// s0, s1: the buffers, LDS variables of their own, so that the compiler knows that a
// load into one is no hazard for reads of the other.
template <bool F16, int ACT, int BN, int BM, int WN, int WM>
QL_DEV void int8_tile(const Int8Args& a, lds8_t* s0, lds8_t* s1) {
    using Tile = Int8Tile<BN, BM, WN, WM>;
    constexpr int NI = Tile::NI, NJ = Tile::NJ;
    const int gn = ((int)a.N + BN - 1) / BN, gt = ((int)a.T + BM - 1) / BM;
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
    const int KT = a.P / kTileK;

    i32x4_t fa[4][NI], fb[4][NJ];                             // of the four steps of 32 K bytes
    const auto read = [&](int s, const lds8_t* buf) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) fb[s][j] = int8_frag(buf, rowb + 32 * j, 2 * s + h);
#pragma unroll
        for (int i = 0; i < NI; ++i) fa[s][i] = int8_frag(buf, rowa + 32 * i, 2 * s + h);
    };
    const auto mfma = [&](int s, int j0, int j1) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (j >= j0 && j < j1)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[s][i], fb[s][j], acc[i][j], 0, 0, 0);
    };
    constexpr int kL = Tile::kLoads, kF = NI + NJ, kM = NI * NJ, kEarly = kL / 3;
    // One K tile: on entry step 0's fragments are read.
    const auto tile = [&](lds8_t* cur, lds8_t* nxt, int kt) {
        const int ahead = kt + 2 < KT ? kt + 2 : KT - 1;      // past the end: the last one again, which nothing reads
        read(1, cur);
        read(2, cur);
        read(3, cur);
        mfma(0, 0, NJ);
        int8_interleave<kM, 3 * kF, 0>();
        __builtin_amdgcn_sched_barrier(0);
        mfma(1, 0, NJ / 2);
        wait_barrier<kWaitLds>();                             // everyone has read all of cur
        tl.load(cur, ahead, 0, kEarly);
        mfma(1, NJ / 2, NJ);
        int8_interleave<kM / 2, 0, kEarly>();
        __builtin_amdgcn_sched_barrier(0);
        tl.load(cur, ahead, kEarly, kL);
        mfma(2, 0, NJ);
        int8_interleave<kM, 0, kL - kEarly>();
        wait_barrier<wait_loads(kL)>();                       // nxt has landed, the loads just issued may fly
        read(0, nxt);
        mfma(3, 0, NJ);
        int8_interleave<kM, kF, 0>();
        __builtin_amdgcn_sched_barrier(0);
    };
    tl.load(s0, 0, 0, kL);
    tl.load(s1, KT > 1 ? 1 : 0, 0, kL);
    wait_barrier<wait_loads(kL)>();
    read(0, s0);
    int kt = 0;
#pragma unroll 1
    for (; kt + 1 < KT; kt += 2) {
        tile(s0, s1, kt);
        tile(s1, s0, kt + 1);
    }
    if (kt < KT) tile(s0, s1, kt);

    // Epilogue, each wave for itself: 32 tokens at a time through LDS of its own
    // (sums, 4-channel chunks swizzled by the token), then rows: eight channels per
    // lane, the same ones for every token, as 16-byte accesses of 2-byte alignment; the
    // lanes whose last channels lie past N go element by element.  The first operand
    // (mul, or res) is loaded for the whole wave tile before anything waits: loaded a few
    // rows at a time, four waves a CU cover too little of the memory latency (the epilogue
    // of a 256 x 256 tile then took as long as 45 K tiles).
    constexpr int kCh = BN / WN, kRow = kCh * 4, kPer = kCh / 8, kItems = 32 * kPer / 64, kStep = 64 / kPer;
    static_assert(64 * kRow <= Tile::kBuf, "32 tokens of two waves fit a buffer");
    lds8_t* const st = (tl.wave < 2 ? s0 : s1) + (tl.wave & 1) * 32 * kRow;
    const int c8 = lane % kPer, tk0 = lane / kPer, N = (int)a.N;
    const int n = (int)n0 + wn * kCh + c8 * 8, tw = (int)t0 + wm * (BM / WM), left = (int)a.T - tw;
    const bool full = n + 8 <= N;
    // rows of the wave tile: a uniform base and 32-bit byte offsets
    const int64_t base = (int64_t)tw * N;
    const auto row8 = [&](const uint16_t* p, int tk) -> const u32x4_a2* {
        return reinterpret_cast<const u32x4_a2*>(reinterpret_cast<const uint8_t*>(p + base) + ((uint32_t)tk * N + n) * 2u);
    };
    const uint16_t* const p1 = a.ep.mul ? a.ep.mul : a.ep.res;
    const uint16_t* const p2 = a.ep.mul ? a.ep.res : nullptr;
    __builtin_amdgcn_s_waitcnt(0x0070);                       // the loads past the end have landed, every read is done
    __syncthreads();
    u32x4_t q1[NJ][kItems];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int u = 0; u < kItems; ++u) {
            const int tk = 32 * j + tk0 + u * kStep;
            q1[j][u] = u32x4_t{0, 0, 0, 0};
            if (p1 && full && tk < left) q1[j][u] = *row8(p1, tk);
        }
    float ws[8], xs[NJ];
    u32x4_t bias = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) ws[e] = n + e < N ? a.ws[n + e] : 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j) xs[j] = 32 * j + r < left ? a.xs[tw + 32 * j + r] : 0.0f;
    if (a.ep.bias && full) bias = *reinterpret_cast<const u32x4_t*>(a.ep.bias + n);
    const bool edge = (int)n0 + (wn + 1) * kCh > N;              // some lanes are not full
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = 8 * i + 2 * g + h;
                *reinterpret_cast<lds_i32x4_t*>(st + r * kRow + ((c ^ (r & (kCh / 4 - 1))) << 4)) =
                    i32x4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
            }
#pragma unroll
        for (int u = 0; u < kItems; ++u) {
            const int tk = tk0 + u * kStep, sw = tk & (kCh / 4 - 1);
            const i32x4_t lo = *reinterpret_cast<const lds_i32x4_t*>(st + tk * kRow + (((2 * c8) ^ sw) << 4));
            const i32x4_t hi = *reinterpret_cast<const lds_i32x4_t*>(st + tk * kRow + (((2 * c8 + 1) ^ sw) << 4));
            const float x = __shfl(xs[j], tk);
            float v[8], w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = int8_scaled(e < 4 ? lo[e] : hi[e - 4], x, ws[e]);
            if (a.ep.bias) {
                unpack8<F16>(bias, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += w[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = act_value<ACT>(v[e]);
            if (p1) {
                unpack8<F16>(q1[j][u], w);
                if (a.ep.mul) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= w[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += w[e];
                }
            }
            if (full && 32 * j + tk < left) {
                if (p2) {
                    const u32x4_t q2 = *row8(p2, 32 * j + tk);
                    unpack8<F16>(q2, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] += w[e];
                }
                *const_cast<u32x4_a2*>(row8(a.y, 32 * j + tk)) = pack8<F16>(v);
            }
        }
        if (edge && !full) {
#pragma unroll 1
            for (int tk = tk0; tk < 32 && 32 * j + tk < left; tk += kStep)
#pragma unroll 1
                for (int e = 0; n + e < N; ++e) {
                    const int c = 2 * c8 + (e >> 2);
                    const int sum = *reinterpret_cast<const __attribute__((address_space(3))) int*>(
                        st + tk * kRow + ((c ^ (tk & (kCh / 4 - 1))) << 4) + (e & 3) * 4);
                    const int64_t t = tw + 32 * j + tk;
                    a.y[t * N + n + e] = epi_value<F16>(a, epi_load(a, t, n + e), sum);
                }
        }
    }
}

template <bool F16, int ACT, int BN, int BM, int WN, int WM>
__global__ __launch_bounds__(256) void k_int8_tile(Int8Args a) {
    __shared__ __align__(1024) uint8_t s0[(BN + BM) * kTileK], s1[(BN + BM) * kTileK];
    int8_tile<F16, ACT, BN, BM, WN, WM>(a, (lds8_t*)s0, (lds8_t*)s1);
}

template <int BN, int BM, int WN, int WM, bool F16>
void launch_tiles(const Int8Args& a, hipStream_t s) {
    const dim3 g((unsigned)(ceil_div(a.N, BN) * ceil_div(a.T, BM)));
    switch (a.ep.act) {
        case kActRelu: hipLaunchKernelGGL((k_int8_tile<F16, kActRelu, BN, BM, WN, WM>), g, dim3(256), 0, s, a); break;
        case kActSilu: hipLaunchKernelGGL((k_int8_tile<F16, kActSilu, BN, BM, WN, WM>), g, dim3(256), 0, s, a); break;
        case kActGelu: hipLaunchKernelGGL((k_int8_tile<F16, kActGelu, BN, BM, WN, WM>), g, dim3(256), 0, s, a); break;
        case kActGeluTanh:
            hipLaunchKernelGGL((k_int8_tile<F16, kActGeluTanh, BN, BM, WN, WM>), g, dim3(256), 0, s, a);
            break;
        default: hipLaunchKernelGGL((k_int8_tile<F16, kActNone, BN, BM, WN, WM>), g, dim3(256), 0, s, a); break;
    }
}

size_t int8_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_int8(const Int8Args& a, void*, hipStream_t s, bool f16) {
    const auto go = [&](auto kern, int nt) {
        hipLaunchKernelGGL(kern, dim3((unsigned)ceil_div(a.N, 16), (unsigned)ceil_div(a.T, 16 * nt)),
                           dim3(64 * kSkinnyWaves), 0, s, a);
    };
    if (a.T > 64) {
        if (ceil_div(a.N, 256) * ceil_div(a.T, 256) >= 256)
            f16 ? launch_tiles<256, 256, 2, 2, true>(a, s) : launch_tiles<256, 256, 2, 2, false>(a, s);
        else
            f16 ? launch_tiles<128, 128, 2, 2, true>(a, s) : launch_tiles<128, 128, 2, 2, false>(a, s);
        return hipGetLastError();
    }
    if (a.T <= 16) f16 ? go(k_int8_skinny<true, 1>, 1) : go(k_int8_skinny<false, 1>, 1);
    else f16 ? go(k_int8_skinny<true, 4>, 4) : go(k_int8_skinny<false, 4>, 4);
    return hipGetLastError();
}

}  // namespace ql
