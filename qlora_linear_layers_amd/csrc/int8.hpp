// The 8-bit integer product: arguments, epilogue and launch.
#pragma once

#include "act.hpp"
#include "common.hpp"
#include "rows.hpp"

namespace ql {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

struct Int8Args {
    const int8_t* x;          // [T][P]
    const float* xs;          // [T]
    const int8_t* w;          // [N][P]
    const float* ws;          // [N]
    uint16_t* y;              // [T][N]
    Epilogue ep;              // z, zc and zs unused
    int64_t T, N;
    int P;                    // pitch of a row: K rounded up to 128, zeros past K
    int splits;               // of the reduction, and their int32 sums [splits][T][N rounded up to 8]
    int* part;
};

// Z = sum dx dw.  The smaller scale first: sum * min stays finite and keeps its
// bits wherever the result does (a sum of 0 stays 0 where the scales' product
// would overflow), and a NaN in either scale comes through.
QL_DEV float int8_scaled(int sum, float xs, float ws) {
    const bool lt = xs < ws;
    return ((float)sum * (lt ? xs : ws)) * (lt ? ws : xs);
}

QL_DEV float act_of(int act, float z) {
    switch (act) {
        case kActRelu: return act_value<kActRelu>(z);
        case kActSilu: return act_value<kActSilu>(z);
        case kActGelu: return act_value<kActGelu>(z);
        case kActGeluTanh: return act_value<kActGeluTanh>(z);
        default: return z;
    }
}

// Up to 16 tokens a product runs on the decode kernel (no LDS tiles), and up to 32
// where its workgroups are one a CU and read little of X: each of them reads all of it.
// Decode kernel / split 64-token tiles, us: 17 tokens through 4096 -> 4096 6.7 / 8.5, 32
// tokens 7.9 / 9.1, 20 tokens through 8192 -> 4096 11.0 / 11.2, 24 tokens 11.6 / 10.9, 32
// tokens through 11008 -> 4096 16.8 / 13.4, 17 tokens through 4096 -> 11008 16.6 / 12.3, 16
// tokens 13.2 / 12.2.  Up to a microsecond is given away for one launch and no workspace,
// which a call from the host (8 against 14 us of its own) gains back.
constexpr int64_t kInt8SkinnyT = 32, kInt8SkinnyTK = 196608;

size_t int8_workspace(int64_t T, int64_t K, int64_t N);
hipError_t launch_int8(Int8Args a, int64_t K, void* ws, hipStream_t s, bool f16);

}  // namespace ql
