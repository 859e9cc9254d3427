// int8.hip - products of 8-bit integers with a scale per row and per output channel, grouped by
// expert: y[n][m] = sx[n] sw[e][m] sum_k x[n][k] w[e][m][k] for the rows n of expert e.
//
// The sum runs in the integer matrix instructions (16x16x64: int8 operands, int32 accumulators)
// and is exact in any order, so every variant and split gives the same bits; only the two scales
// and the SwiGLU are fp32 arithmetic. Weights are the A operand and rows the B operand: a lane's
// accumulators are four consecutive channels of one row, stored as one piece.
#include "device_common.h"
#include "kernels.h"

namespace moe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void mma_i8(i32x4_t &acc, const uint4 &a, const uint4 &b) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a),
                                                __builtin_bit_cast(i32x4_t, b), acc, 0, 0, 0);
}

// Row tiles of the experts in order: expert e's rows [lo, hi) in tiles of `per` rows. Every wave
// finds tile u by itself: lane l sums the tiles of experts 4l .. 4l + 3, a wave scan places them.
struct RowTile {
    int e, start, n;  // n = 0: there is no tile u
};
__device__ RowTile find_tile(const int32_t *offsets, int E, int n_rows, int per, int u) {
    if (!offsets) return {0, u * per, max(0, min(per, n_rows - u * per))};
    const int lane = lane_id();
    int lo[4], hi[4], nt[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = min(4 * lane + i, E);  // past the last expert: an empty range
        lo[i] = min(max(offsets[e], 0), n_rows);
        hi[i] = min(max(offsets[min(e + 1, E)], lo[i]), n_rows);
        nt[i] = (hi[i] - lo[i] + per - 1) / per;
        sum += nt[i];
    }
    const int incl = wave_inclusive_sum(sum);
    int at = incl - sum;
    RowTile r = {0, 0, 0};
    const uint64_t mine = __ballot(u >= at && u < incl);
    if (!mine) return r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (u >= at && u < at + nt[i]) {
            r.e = 4 * lane + i;
            r.start = lo[i] + (u - at) * per;
            r.n = min(per, hi[i] - r.start);
        }
        at += nt[i];
    }
    const int src = __ffsll((unsigned long long)mine) - 1;
    r.e = __builtin_amdgcn_readlane(r.e, src);
    r.start = __builtin_amdgcn_readlane(r.start, src);
    r.n = __builtin_amdgcn_readlane(r.n, src);
    return r;
}

__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(uint16_t *p, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(p) = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// z = fp32(sum) * x_scale * w_scale of four channels.
__device__ __forceinline__ void scaled(const i32x4_t &acc, float sx, const float *sw, float (&z)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) z[r] = (float)acc[r] * sx * sw[r];
}

// Tiles of 64 rows by 64 output channels, 16 channels per wave (with SwiGLU: 16 gate and the 16
// matching up channels).
constexpr int kTRows = 64, kTCols = 64;
template <bool kSwiglu, class O>
__global__ __launch_bounds__(256) void i8_tile_kernel(I8Params p) {
    constexpr int kA = kSwiglu ? 2 : 1;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, q = lane >> 4;
    const int Mo = kSwiglu ? p.M / 2 : p.M;
    const int cb = (Mo + kTCols - 1) / kTCols;
    const int u = blockIdx.x / cb, m0 = (blockIdx.x % cb) * kTCols + wave * kTile;
    const RowTile t = find_tile(p.offsets, p.E, p.n_rows, kTRows, u);
    if (t.n <= 0 || m0 >= Mo) return;
    const int mrow = min(m0 + col, Mo - 1);
    const int8_t *w[kA];
#pragma unroll
    for (int a = 0; a < kA; ++a) w[a] = p.w + ((size_t)t.e * p.M + a * Mo + mrow) * p.K;
    const int8_t *x[kTRows / kTile];
#pragma unroll
    for (int i = 0; i < kTRows / kTile; ++i)
        x[i] = p.x + (size_t)(t.start + min(i * kTile + col, t.n - 1)) * p.K;
    i32x4_t acc[kA][kTRows / kTile] = {};
    for (int k = q * 16; k < (p.K + 63) / 64 * 64; k += 64) {
        const bool in = k < p.K;
        const uint4 z = {0, 0, 0, 0};
        uint4 a[kA];
#pragma unroll
        for (int i = 0; i < kA; ++i) a[i] = in ? load16(w[i] + k) : z;
#pragma unroll
        for (int j = 0; j < kTRows / kTile; ++j) {
            const uint4 b = in ? load16(x[j] + k) : z;
#pragma unroll
            for (int i = 0; i < kA; ++i) mma_i8(acc[i][j], a[i], b);
        }
    }
    const int mc = m0 + 4 * q;
    if (mc >= Mo) return;  // Mo is a multiple of 8: a lane's four channels are all in or all out
    const float *sw = p.w_scale + (size_t)t.e * p.M + mc;
#pragma unroll
    for (int j = 0; j < kTRows / kTile; ++j) {
        const int n = j * kTile + col;
        if (n >= t.n) continue;
        const float sx = p.x_scale[t.start + n];
        float z[4];
        scaled(acc[0][j], sx, sw, z);
        if constexpr (kSwiglu) {
            float up[4];
            scaled(acc[1][j], sx, sw + Mo, up);
#pragma unroll
            for (int r = 0; r < 4; ++r) z[r] = z[r] / (1.0f + expf(-z[r])) * up[r];
        }
        store4(reinterpret_cast<O *>(p.y) + (size_t)(t.start + n) * Mo + mc, z);
    }
}

}  // namespace

hipError_t launch_matmul_i8(const I8Params &p, bool swiglu, int y_dtype, hipStream_t s) {
    const int Mo = swiglu ? p.M / 2 : p.M;
    // most row tiles n_rows rows of E experts can make: full ones, and a part of one per expert
    const long tiles = p.offsets ? p.n_rows / kTRows + (p.E < p.n_rows ? p.E : p.n_rows)
                                 : (p.n_rows + kTRows - 1) / kTRows;
    const long grid = tiles * ((Mo + kTCols - 1) / kTCols);
    if (grid > 0x7FFFFFFFl) return hipErrorInvalidValue;
    auto go = [&](auto o) {
        using O = decltype(o);
        if (swiglu) launch_k(i8_tile_kernel<true, O>, (unsigned)grid, 256, 0, s, p);
        else launch_k(i8_tile_kernel<false, O>, (unsigned)grid, 256, 0, s, p);
    };
    if (y_dtype == 0) go(float{});
    else go(uint16_t{});
    return hipGetLastError();
}

}  // namespace moe
