// The 8-bit integer product for gfx950: with sums exact in int32,
//   Y = act((sum_k xq wq) dx dw + bias) * mul + res.
// Few tokens: k_int8_skinny (v_mfma_i32_16x16x64_i8 fed from global memory).  Else LDS
// tiles on v_mfma_i32_32x32x32_i8: k_int8_tile, with k_int8_fin where a reduction is
// split.  Int8Plan at the end chooses.
#include "int8.hpp"

namespace ql {

namespace {

template <bool F16>
QL_DEV float value16(uint16_t v) { return lo16<F16>(v); }

// Output (t, n): what the epilogue reads, loaded ahead, and the rounding at the end.
// The loads have no branches (a missing operand is read from the weight's scales and
// not used), so that nothing waits for them until the end.
struct EpiOperands {
    float xs, ws;
    uint16_t bias, mul, res;
};
QL_DEV EpiOperands epi_load(const Int8Args& a, int64_t t, int64_t n) {
    const int64_t at = t * a.N + n;
    const uint16_t* const none = reinterpret_cast<const uint16_t*>(a.ws);
    return {a.xs[t], a.ws[n], *(a.ep.bias ? a.ep.bias + n : none), *(a.ep.mul ? a.ep.mul + at : none),
            *(a.ep.res ? a.ep.res + at : none)};
}
// The epilogue's steps are rounded one by one, here as in k_int8_tile and k_int8_fin:
// contracted into fmas in some places and not in others, the bits of an output would
// depend on the kernel that forms it and on N % 8.
template <bool F16>
QL_DEV uint16_t epi_value(const Int8Args& a, const EpiOperands& o, int sum) {
#pragma clang fp contract(off)
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

}  // namespace

// 16 NT tokens x 16 channels per workgroup, K dealt to its waves in steps of 128 bytes
// (neighbouring waves read neighbouring steps), whose sums are added in LDS.  A wave
// keeps the loads of D steps in flight; what the epilogue reads is loaded first of all,
// so that its latency passes meanwhile.
//
// Bound by the weight's bytes: one token through 8192 -> 22016 (180 MB) takes 31.6 us,
// 5.7 TB/s, through 4096 -> 11008 (45 MB) 9.6 us, of which about 2.5 pass before the first
// and after the last load.  16 waves with two steps each in flight; 8 waves with four 9.7
// and 32.9 us, 8 with six 12.5 (one workgroup less a CU), 16 with four 17.3, 4 with eight
// 10.7 and 34.6.
constexpr int kSkinnyWaves = 16, kSkinnySteps = 2;
template <bool F16, int NT>
__global__ __launch_bounds__(64 * kSkinnyWaves) void k_int8_skinny(Int8Args a) {
    constexpr int WAVES = kSkinnyWaves, D = kSkinnySteps, kThreads = 64 * WAVES, kOut = (NT * 256 + kThreads - 1) / kThreads;
    __shared__ int sums[WAVES][NT][16][16];
    const int lane = (int)threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int n0 = (int)blockIdx.x * 16, t0 = (int)blockIdx.y * (16 * NT), N = (int)a.N, T = (int)a.T;
    EpiOperands op[kOut];
#pragma unroll
    for (int q = 0; q < kOut; ++q) {
        const int e = (int)threadIdx.x + q * kThreads;
        op[q] = epi_load(a, min(t0 + e / 16, T - 1), min(n0 + e % 16, N - 1));
    }
    const int8_t* wr = a.w + (int64_t)min(n0 + l16, N - 1) * a.P + g * 16;
    const int8_t* xr[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) xr[i] = a.x + (int64_t)min(t0 + 16 * i + l16, T - 1) * a.P + g * 16;
    const int steps = a.P / 128;
    i32x4_t wf[D][2], xf[D][2][NT], acc[NT];
    const auto load = [&](int u, int s) {
        const int k = s * 128;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            wf[u][j] = *reinterpret_cast<const i32x4_t*>(wr + k + 64 * j);
#pragma unroll
            for (int i = 0; i < NT; ++i) xf[u][j][i] = *reinterpret_cast<const i32x4_t*>(xr[i] + k + 64 * j);
        }
        asm volatile("" ::: "memory");                        // loads stay here, they do not sink to their uses
    };
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = i32x4_t{0, 0, 0, 0};
    const auto mul = [&](int u) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < NT; ++i)
                acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xf[u][j][i], wf[u][j], acc[i], 0, 0, 0);
    };
#pragma unroll
    for (int u = 0; u < D; ++u) load(u, min(wv + u * WAVES, steps - 1));   // past the end: the last step again, not multiplied
    int s = wv;
#pragma unroll 1
    for (; s + (2 * D - 1) * WAVES < steps; s += D * WAVES)
#pragma unroll
        for (int u = 0; u < D; ++u) {
            mul(u);
            load(u, s + (u + D) * WAVES);
        }
    // fewer than 2 D steps are left, the first D of them loaded
#pragma unroll
    for (int u = 0; u < D; ++u)
        if (s + u * WAVES < steps) {
            mul(u);
            if (s + (u + D) * WAVES < steps) load(u, s + (u + D) * WAVES);
        }
#pragma unroll
    for (int u = 0; u < D - 1; ++u)
        if (s + (u + D) * WAVES < steps) mul(u);
    // lane holds tokens 4 g .. 4 g + 3 of channel l16
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) sums[wv][i][4 * g + q][l16] = acc[i][q];
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kOut; ++q) {
        const int e = (int)threadIdx.x + q * kThreads;
        const int t = t0 + e / 16, n = n0 + e % 16;
        if (e >= NT * 256 || t >= T || n >= N) continue;
        int v = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v += sums[w][e / 256][e / 16 % 16][e % 16];
        a.y[(int64_t)t * N + n] = epi_value<F16>(a, op[q], v);
    }
}

// ------------------------------------------------------------------ tiles
//
// BN channels x BM tokens per workgroup of four waves (WN x WM of them), K in tiles of
// 128 bytes, whole cache lines, in S buffers of LDS that are filled by loads that go
// there directly.
//   S = 2 (256 x 256, and 128 x 128 with two workgroups a CU): a wave takes the fragments
//     of a whole K tile into registers during the tile's first quarter, so that its
//     buffer is free from then on and the loads of the tile after next are under way for
//     1.5 tiles.
//   S = 4 (128 x 128 and 128 x 64 where they are at most one a CU): loads run three tiles
//     ahead.  Two waves a SIMD, each with one half of every K tile, gained 3% there
//     (1024 tokens of 4096 x 4096 20.9 -> 20.3 us) and lost as much in split products.
// 2048 tokens through 8192 -> 22016 with silu and mul: 328 to 345 us by the card, 2.2 POP/s, MFMA busy
// 0.66 of the cycles, no bank conflicts; on zeros 319 us where values took 354, so a part
// of the rest is the card's power (an MFMA-only loop reaches 4.94 POP/s on zeros, 3.5 on
// values).  128 x 128 tiles, one a CU: 0.34 to 0.42 us a K tile, 32 KB each out of L2.
// LDS rows are 128 bytes with their 16-byte chunks XOR-swizzled (lds_off); a direct load
// writes 64 consecutive chunks (eight rows), so the swizzle is applied to the chunk that
// a lane reads from memory.  Rows past N or T repeat the last one (their outputs are not
// stored).

typedef __attribute__((address_space(3))) i32x4_t lds_i32x4_t;
constexpr int kTileK = 128;

template <int BN, int BM, int WN, int WM>
struct Int8Tile {
    static_assert(WN * WM == 4 && BN % 32 == 0 && BM % 32 == 0, "four waves, whole loads");
    static constexpr int kLoads = (BN + BM) / 32;             // direct loads per thread and K tile
    static constexpr int kLoadsW = BN / 32;                   // those of W come first
    static constexpr int kBuf = (BN + BM) * kTileK;
    static constexpr int NI = BN / WN / 32, NJ = BM / WM / 32;  // 32 x 32 MFMA tiles of a wave
    rsrc_t rw, rx;
    uint32_t voff[kLoads];
    int wave;

    QL_DEV void init(const Int8Args& a, int64_t n0, int64_t t0, int k0) {
        wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
        // 32-bit: scalar units have no 64-bit compare, and a descriptor that goes through
        // vector registers costs a loop around every load
        const int rn = min((int)a.N - (int)n0, BN), rt = min((int)a.T - (int)t0, BM);
        rw = make_rsrc(a.w + n0 * a.P + k0, rn * a.P - k0);
        rx = make_rsrc(a.x + t0 * a.P + k0, rt * a.P - k0);
        const int l = (int)threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int q = (i * 4 + wave) * 8 + (l >> 3);      // row of the buffer: W rows, then X rows
            const int row = i < kLoadsW ? min(q, rn - 1) : min(q - BN, rt - 1);
            voff[i] = (uint32_t)row * (uint32_t)a.P + ((uint32_t)((l & 7) ^ ((q ^ (q >> 3)) & 7)) << 4);
        }
    }
    // loads i0 .. i1 - 1 of K tile kt
    QL_DEV void load(lds8_t* buf, int kt, int i0, int i1) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (i >= i0 && i < i1)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(i < kLoadsW ? rw : rx, buf + (i * 4 + wave) * 1024, 16,
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

// buf: the S buffers, LDS variables of their own, so that the compiler knows that a
// load into one is no hazard for reads of another.
// kActPart for ACT: the K tiles of one split, whose sums go to a.part.
constexpr int kActPart = -1;
template <bool F16, int ACT, int BN, int BM, int WN, int WM, int S>
QL_DEV void int8_tile(const Int8Args& a, lds8_t* const (&buf)[S]) {
#pragma clang fp contract(off)
    using Tile = Int8Tile<BN, BM, WN, WM>;
    constexpr int NI = Tile::NI, NJ = Tile::NJ;
    const int gn = ((int)a.N + BN - 1) / BN, gt = ((int)a.T + BM - 1) / BM;
    // the splits of a tile are the outermost index: workgroups of one split share operands
    int tn, tt, sp = 0, kt0 = 0, KT = a.P / kTileK;
    if constexpr (ACT == kActPart) {
        const int g = gn * gt;
        sp = (int)blockIdx.x / g;
        int8_tile_of((int)blockIdx.x % g, gn, gt, tn, tt);
        kt0 = KT * sp / a.splits;
        KT = KT * (sp + 1) / a.splits - kt0;
    } else {
        int8_tile_of((int)blockIdx.x, gn, gt, tn, tt);
    }
    const int64_t n0 = (int64_t)tn * BN, t0 = (int64_t)tt * BM;
    Tile tl;
    tl.init(a, n0, t0, kt0 * kTileK);
    const int lane = (int)threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int wn = tl.wave % WN, wm = tl.wave / WN;
    const int rowa = wn * (BN / WN) + r, rowb = BN + wm * (BM / WM) + r;
    // The epilogue, each wave for itself: 32 tokens at a time through LDS of its own
    // (sums, 4-channel chunks swizzled by the token), then rows: eight channels per
    // lane, the same ones for every token, as 16-byte accesses of 2-byte alignment; the
    // lanes whose last channels lie past N go element by element.  The first operand
    // (mul, or res) is loaded for the whole wave tile ahead of the staging: loaded a few
    // rows at a time, four waves a CU cover too little of the memory latency (the epilogue
    // of a 256 x 256 tile then took as long as 45 K tiles).  Where a CU holds one small
    // tile, it is loaded before the first K tile.
    constexpr int kCh = BN / WN, kRow = kCh * 4, kPer = kCh / 8, kItems = 32 * kPer / 64, kStep = 64 / kPer;
    static_assert(64 * kRow <= Tile::kBuf, "32 tokens of two waves fit a buffer");
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
    constexpr bool kEarly = ACT != kActPart && S == 4;
    u32x4_t q1[NJ][kItems], bias;
    float ws[8], xs[NJ];
    const auto operands = [&]() {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int u = 0; u < kItems; ++u) {
                const int tk = 32 * j + tk0 + u * kStep;
                q1[j][u] = u32x4_t{0, 0, 0, 0};
                if (p1 && full && tk < left) q1[j][u] = *row8(p1, tk);
            }
#pragma unroll
        for (int e = 0; e < 8; ++e) ws[e] = n + e < N ? a.ws[n + e] : 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) xs[j] = 32 * j + r < left ? a.xs[tw + 32 * j + r] : 0.0f;
        bias = u32x4_t{0, 0, 0, 0};
        if (a.ep.bias && full) bias = *reinterpret_cast<const u32x4_t*>(a.ep.bias + n);
    };
    if constexpr (kEarly) operands();

    i32x16_t acc[NI][NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[i][j][q] = 0;

    constexpr int kS = 4;                                     // steps of 32 K bytes of a K tile
    i32x4_t fa[kS][NI], fb[kS][NJ];
    const auto read = [&](int s, const lds8_t* buf) {
        const int c = 2 * s + h;
#pragma unroll
        for (int j = 0; j < NJ; ++j) fb[s][j] = int8_frag(buf, rowb + 32 * j, c);
#pragma unroll
        for (int i = 0; i < NI; ++i) fa[s][i] = int8_frag(buf, rowa + 32 * i, c);
    };
    const auto mfma = [&](int s, int j0, int j1) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (j >= j0 && j < j1)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[s][i], fb[s][j], acc[i][j], 0, 0, 0);
    };
    constexpr int kL = Tile::kLoads, kF = NI + NJ, kM = NI * NJ;
    // Loads issued before the barrier (and, with two buffers, by the end of step 1).
    // They keep the address unit busy for half of the time that the MFMAs of a 256 x 256
    // tile take, and a wave that waits for it cannot issue MFMAs: they are spread over the
    // tile (2048 tokens through 8192 -> 22016: 334 us, against 358 with all of them by the
    // end of step 2).
    constexpr int kL1 = kL / 5, kB = S == 2 ? 3 * kL / 5 : (kS - 1) * kL / kS;
    // One K tile: on entry step 0's fragments are read.  With two buffers the tile after
    // next goes where this one was, once everyone has read all of it; with more of them a
    // later one goes to `prev`, the buffer before this one, which the barrier of the last
    // tile has freed.
    const auto tile = [&](lds8_t* prev, lds8_t* cur, lds8_t* nxt, int kt) {
        // past the end: the last one again, which nothing reads
        const int ahead = min(kt + (S == 2 ? 2 : S - 1), KT - 1);
#pragma unroll
        for (int s = 1; s < kS; ++s) read(s, cur);
        if constexpr (S == 2) {
            mfma(0, 0, NJ);
            int8_interleave<kM, (kS - 1) * kF, 0>();
            __builtin_amdgcn_sched_barrier(0);
            mfma(1, 0, NJ / 2);
            wait_barrier<kWaitLds>();                         // everyone has read all of cur
            tl.load(cur, ahead, 0, kL1);
            mfma(1, NJ / 2, NJ);
            int8_interleave<kM / 2, 0, kL1>();
            __builtin_amdgcn_sched_barrier(0);
            tl.load(cur, ahead, kL1, kB);
            mfma(2, 0, NJ);
            int8_interleave<kM, 0, kB - kL1>();
            wait_barrier<wait_loads(kB)>();                   // nxt has landed, the loads just issued may fly
            read(0, nxt);
            tl.load(cur, ahead, kB, kL);
            mfma(3, 0, NJ);
            int8_interleave<kM, kF, kL - kB>();
        } else {
#pragma unroll
            for (int s = 0; s < kS - 1; ++s) {
                tl.load(prev, ahead, s * kL / kS, (s + 1) * kL / kS);
                mfma(s, 0, NJ);
                if (s == 0) int8_interleave<kM, 3 * kF, kL / kS>();
                else int8_interleave<kM, 0, kL / kS>();
                __builtin_amdgcn_sched_barrier(0);
            }
            wait_barrier<wait_loads((S - 3) * kL + kB) & ~0x0F00>();   // nxt has landed, all of cur is read
            read(0, nxt);
            tl.load(prev, ahead, kB, kL);
            mfma(kS - 1, 0, NJ);
            int8_interleave<kM, kF, kL - kB>();
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr int kFirst = S == 2 ? 2 : S - 1;                // tiles loaded before the first
    static_assert(kFirst * kL < 64, "the loads in flight fit the counter");
#pragma unroll
    for (int q = 0; q < kFirst; ++q) tl.load(buf[q], min(q, KT - 1), 0, kL);
    wait_barrier<wait_loads((kFirst - 1) * kL)>();
    read(0, buf[0]);
    int kt = 0;
#pragma unroll 1
    for (; kt + S <= KT; kt += S)
#pragma unroll
        for (int q = 0; q < S; ++q) tile(buf[(q + S - 1) % S], buf[q], buf[(q + 1) % S], kt + q);
#pragma unroll
    for (int q = 0; q < S - 1; ++q)
        if (kt + q < KT) tile(buf[(q + S - 1) % S], buf[q], buf[q + 1], kt + q);

    lds8_t* const st = (tl.wave < 2 ? buf[0] : buf[1]) + (tl.wave & 1) * 32 * kRow;
    __builtin_amdgcn_s_waitcnt(0x0070);                       // the loads past the end have landed, every read is done
    __syncthreads();
    const auto stage = [&](int j) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int c = 8 * i + 2 * g + h;
                *reinterpret_cast<lds_i32x4_t*>(st + r * kRow + ((c ^ (r & (kCh / 4 - 1))) << 4)) =
                    i32x4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
            }
    };
    const auto staged = [&](int tk, int c) {                  // channels 4 c .. 4 c + 3 of token tk
        return *reinterpret_cast<const lds_i32x4_t*>(st + tk * kRow + ((c ^ (tk & (kCh / 4 - 1))) << 4));
    };
    if constexpr (ACT == kActPart) {
        const int NP = (N + 7) & ~7;
        int* const part = a.part + (int64_t)sp * a.T * NP;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            stage(j);
#pragma unroll
            for (int u = 0; u < kItems; ++u) {
                const int tk = tk0 + u * kStep;
                if (n >= N || 32 * j + tk >= left) continue;
                i32x4_t* const o = reinterpret_cast<i32x4_t*>(part + (int64_t)(tw + 32 * j + tk) * NP + n);
                o[0] = staged(tk, 2 * c8);
                o[1] = staged(tk, 2 * c8 + 1);
            }
        }
        return;
    } else {
    if constexpr (!kEarly) operands();
    const bool edge = (int)n0 + (wn + 1) * kCh > N;              // some lanes are not full
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        stage(j);
#pragma unroll
        for (int u = 0; u < kItems; ++u) {
            const int tk = tk0 + u * kStep;
            const i32x4_t lo = staged(tk, 2 * c8), hi = staged(tk, 2 * c8 + 1);
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
}

template <bool F16, int ACT, int BN, int BM, int WN, int WM, int S>
__global__ __launch_bounds__(256) void k_int8_tile(Int8Args a) {
    constexpr int kBuf = (BN + BM) * kTileK;
    __shared__ __align__(1024) uint8_t s0[kBuf], s1[kBuf];
    if constexpr (S == 4) {
        __shared__ __align__(1024) uint8_t s2[kBuf], s3[kBuf];
        int8_tile<F16, ACT, BN, BM, WN, WM, 4>(a, {(lds8_t*)s0, (lds8_t*)s1, (lds8_t*)s2, (lds8_t*)s3});
    } else {
        int8_tile<F16, ACT, BN, BM, WN, WM, 2>(a, {(lds8_t*)s0, (lds8_t*)s1});
    }
}

template <int BN, int BM, int WN, int WM, int S, bool F16>
void launch_tiles(const Int8Args& a, hipStream_t s) {
    const dim3 g((unsigned)(ceil_div(a.N, BN) * ceil_div(a.T, BM)));
    const auto go = [&](auto kern) { hipLaunchKernelGGL(kern, g, dim3(256), 0, s, a); };
    switch (a.ep.act) {
        case kActRelu: go(k_int8_tile<F16, kActRelu, BN, BM, WN, WM, S>); break;
        case kActSilu: go(k_int8_tile<F16, kActSilu, BN, BM, WN, WM, S>); break;
        case kActGelu: go(k_int8_tile<F16, kActGelu, BN, BM, WN, WM, S>); break;
        case kActGeluTanh: go(k_int8_tile<F16, kActGeluTanh, BN, BM, WN, WM, S>); break;
        default: go(k_int8_tile<F16, kActNone, BN, BM, WN, WM, S>); break;
    }
}

// The sums of all splits, and the epilogue: eight channels of a token per thread, one
// wave per workgroup, so that few tokens spread over the CUs.  The number of splits is a
// template argument and the operands of the epilogue come before the sums, so that every
// load of a thread is in flight at once: 61 x 4097 of five splits (5 MB) 3.3 us, with a
// loop over the splits and the operands after it 5.1.  Channels behind the last whole
// eight go one by one.
template <bool F16, int S>
__global__ __launch_bounds__(64) void k_int8_fin(Int8Args a) {
#pragma clang fp contract(off)
    const int N = (int)a.N, NP = (N + 7) & ~7;
    const int n = ((int)blockIdx.x * 64 + (int)threadIdx.x) * 8;
    const int64_t t = blockIdx.y;
    if (n >= N) return;
    const int64_t step = a.T * NP, o = t * N + n;
    const i32x4_t* const p = reinterpret_cast<const i32x4_t*>(a.part + t * NP + n);
    i32x4_t lo[S], hi[S];
#pragma unroll
    for (int q = 0; q < S; ++q) {
        lo[q] = p[q * step / 4];
        hi[q] = p[q * step / 4 + 1];
    }
    const auto add = [&]() {
#pragma unroll
        for (int q = 1; q < S; ++q) {
            lo[0] += lo[q];
            hi[0] += hi[q];
        }
    };
    if (n + 8 > N) {
        add();
#pragma unroll 1
        for (int e = 0; n + e < N; ++e) {
            int v = lo[0][0];
#pragma unroll
            for (int q = 1; q < 8; ++q) v = e == q ? (q < 4 ? lo[0][q] : hi[0][q - 4]) : v;
            a.y[o + e] = epi_value<F16>(a, epi_load(a, t, n + e), v);
        }
        return;
    }
    const float xs = a.xs[t];
    const u32x4_t w0 = *reinterpret_cast<const u32x4_t*>(a.ws + n), w1 = *reinterpret_cast<const u32x4_t*>(a.ws + n + 4);
    u32x4_t bias = {0, 0, 0, 0}, mul = bias, res = bias;
    if (a.ep.bias) bias = *reinterpret_cast<const u32x4_t*>(a.ep.bias + n);
    if (a.ep.mul) mul = *reinterpret_cast<const u32x4_a2*>(a.ep.mul + o);
    if (a.ep.res) res = *reinterpret_cast<const u32x4_a2*>(a.ep.res + o);
    add();
    float v[8], w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = int8_scaled(e < 4 ? lo[0][e] : hi[0][e - 4], xs, __uint_as_float(e < 4 ? w0[e] : w1[e - 4]));
    if (a.ep.bias) {
        unpack8<F16>(bias, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += w[e];
    }
    act_values(a.ep.act, v);
    if (a.ep.mul) {
        unpack8<F16>(mul, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= w[e];
    }
    if (a.ep.res) {
        unpack8<F16>(res, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += w[e];
    }
    *reinterpret_cast<u32x4_a2*>(a.y + o) = pack8<F16>(v);
}

namespace {

// Which kernel takes a product, and the splits of its reduction.
constexpr int kInt8MaxSplits = 8;
enum class Int8Route { Skinny, Tile64, Tile128, Tile256 };
struct Int8Plan {
    Int8Route route;
    int splits;
    size_t bytes;
    Int8Plan(int64_t T, int64_t K, int64_t N) : route(Int8Route::Skinny), splits(1), bytes(0) {
        if (T <= 16 || (T <= kInt8SkinnyT && N <= 4096 && T * K <= kInt8SkinnyTK)) return;
        const int64_t kt = rows8_pitch(K) / kTileK;
        // A round of 256 x 256 tiles (one a CU) takes as long as 1.5 rounds of 128 x 128
        // tiles (two a CU), whose last round need not be full.  256 / 128, us: 1536 tokens
        // through 8192 -> 8192 (192 / 768 tiles) 105 / 111, 1024 through 4096 -> 11008 (172 /
        // 688) 60 / 59, 2048 through 11008 -> 4096 (128 / 512) 117 / 98.
        if (768 * ceil_div(ceil_div(N, 256) * ceil_div(T, 256), 256) <= ceil_div(N, 128) * ceil_div(T, 128)) {
            route = Int8Route::Tile256;
            return;
        }
        route = T <= 64 ? Int8Route::Tile64 : Int8Route::Tile128;
        // Splits: rounds of K tiles at 0.34 us, and for the int32 sums, written and read
        // back, 0.4 us a MB and 1.5 us of a launch (the time of a K tile is that of operands in
        // the caches: 512 tokens through a cold 11008 -> 4096, 43 K tiles a workgroup, take 27 to
        // 33 us).  Against 0.25 us a MB and 2 of a launch,
        // us: 128 tokens through 11008 -> 4096 18.9 / 20.2 (6 / 8 splits), 256 through 4096 ->
        // 1024 11.7 / 13.2; with 2.5 of a launch 256 through 4096 -> 4096 stay unsplit, 16.8
        // against 15.3, 300 through 5120 -> 5120 21.7 against 20.0.
        const int64_t tiles = ceil_div(N, 128) * ceil_div(T, T <= 64 ? 64 : 128);
        const auto cost = [&](int64_t s) {
            return (double)ceil_div(tiles * s, 256) * (double)ceil_div(kt, s) * 0.34 +
                   (s > 1 ? 1.5 + 0.4e-6 * (double)(s * T * N * 4) : 0.0);
        };
        for (int s = 2; s <= kInt8MaxSplits && kt / s >= 2 && tiles * s <= 256; ++s)
            if (cost(s) < cost(splits)) splits = s;
        if (splits == 1) return;
        bytes = align256((size_t)splits * T * ((N + 7) & ~int64_t(7)) * 4);
    }
};

}  // namespace

size_t int8_workspace(int64_t T, int64_t K, int64_t N) { return Int8Plan(T, K, N).bytes; }

template <bool F16>
static hipError_t launch_int8_of(const Int8Args& a, const Int8Plan& pl, hipStream_t s) {
    const auto skinny = [&](auto kern, int nt) {
        hipLaunchKernelGGL(kern, dim3((unsigned)ceil_div(a.N, 16), (unsigned)ceil_div(a.T, 16 * nt)),
                           dim3(64 * kSkinnyWaves), 0, s, a);
    };
    const auto part = [&](auto kern, int bm) {
        hipLaunchKernelGGL(kern, dim3((unsigned)(ceil_div(a.N, 128) * ceil_div(a.T, bm) * pl.splits)), dim3(256), 0, s, a);
    };
    if (pl.route == Int8Route::Skinny) {
        if (a.T > 16) skinny(k_int8_skinny<F16, 2>, 2);
        else skinny(k_int8_skinny<F16, 1>, 1);
    } else if (pl.splits > 1) {
        if (pl.route == Int8Route::Tile64) part(k_int8_tile<false, kActPart, 128, 64, 2, 2, 4>, 64);
        else part(k_int8_tile<false, kActPart, 128, 128, 2, 2, 4>, 128);
        const auto fin = [&](auto kern) {
            hipLaunchKernelGGL(kern, dim3((unsigned)ceil_div(a.N, 512), (unsigned)a.T), dim3(64), 0, s, a);
        };
        switch (pl.splits) {
            case 2: fin(k_int8_fin<F16, 2>); break;
            case 3: fin(k_int8_fin<F16, 3>); break;
            case 4: fin(k_int8_fin<F16, 4>); break;
            case 5: fin(k_int8_fin<F16, 5>); break;
            case 6: fin(k_int8_fin<F16, 6>); break;
            case 7: fin(k_int8_fin<F16, 7>); break;
            default: fin(k_int8_fin<F16, 8>); break;
        }
    } else if (pl.route == Int8Route::Tile256) {
        launch_tiles<256, 256, 2, 2, 2, F16>(a, s);
    } else if (pl.route == Int8Route::Tile64) {
        launch_tiles<128, 64, 2, 2, 4, F16>(a, s);
    } else if (ceil_div(a.N, 128) * ceil_div(a.T, 128) > 256) {
        launch_tiles<128, 128, 2, 2, 2, F16>(a, s);
    } else {
        launch_tiles<128, 128, 2, 2, 4, F16>(a, s);
    }
    return hipGetLastError();
}

hipError_t launch_int8(Int8Args a, int64_t K, void* ws, hipStream_t s, bool f16) {
    const Int8Plan pl(a.T, K, a.N);
    a.part = static_cast<int*>(ws);
    a.splits = pl.splits;
    return f16 ? launch_int8_of<true>(a, pl, s) : launch_int8_of<false>(a, pl, s);
}

}  // namespace ql
