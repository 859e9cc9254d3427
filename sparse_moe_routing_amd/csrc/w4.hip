// w4.hip - products with 4-bit weights and a scale (and a zero point) per group of columns, grouped by
// expert: y[n][m] = sum_g s[g][m] sum_{k in g} x[n][k] (c[m][k] - z[g][m]) for the rows n of expert e.
//
// Nothing is rounded on the way to the sums: a code less 8 is a whole number of -8..7, exact in bf16,
// and a bf16 row element is an operand as it stands; fp32 rows go in as three bf16 parts that add up to
// all of their 24 bits. A group's sum runs in the matrix instructions (16x16x32, fp32 sums), the
// scale is applied to it in fp32: s (sum x (c - 8) - (z - 8) sum x). Rows are the A operand and
// channels the B operand: a lane's accumulators are four rows of one channel, so that one scale
// serves all of a lane's sums.
#include <math.h>

#include "device_common.h"
#include "expert_tiles.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kStepK = 32;  // columns of one matrix instruction; a scale's group is 1, 2 or 4 of them

// Eight codes (one word, column j in bits 4j .. 4j + 3) as (code - 8) / 16 in bf16, in order. With
// bit 3 turned over a code is a signed 4-bit number, which one instruction converts to fp32 as
// that number / 16: at most four significant bits, so that the upper half is the exact bf16.
__device__ __forceinline__ uint4 codes8(uint32_t w) {
    const uint32_t a = w ^ 0x88888888u, b = a >> 4;
    auto f = [](uint32_t v) __attribute__((always_inline)) {
        return __float_as_uint(__builtin_amdgcn_cvt_off_f32_i4((int)v));
    };
    auto two = [&](uint32_t lo, uint32_t hi) __attribute__((always_inline)) {
        return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
    };
    return uint4{two(f(a), f(b)), two(f((a >> 8) & 0xFFu), f((b >> 8) & 0xFFu)),
                 two(f((a >> 16) & 0xFFu), f((b >> 16) & 0xFFu)), two(f(a >> 24), f(b >> 24))};
}

// A row fragment: eight consecutive elements as loaded, and as bf16 operands that add up to them.
template <class X>
struct Rows8;
template <>
struct Rows8<uint16_t> {
    static constexpr int kParts = 1;
    uint4 v;
    __device__ __forceinline__ void parts(uint4 (&o)[1]) const { o[0] = v; }
};
template <>
struct Rows8<float> {
    static constexpr int kParts = 3;
    uint4 v[2];
    // x = hi + mid + lo, each of at most 8 significant bits (cut off, not rounded)
    __device__ __forceinline__ void parts(uint4 (&o)[3]) const {
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        uint32_t m[8], l[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float rest = __uint_as_float(w[i]) - __uint_as_float(w[i] & 0xFFFF0000u);
            m[i] = __float_as_uint(rest);
            l[i] = __float_as_uint(rest - __uint_as_float(m[i] & 0xFFFF0000u));
        }
        auto pack = [](const uint32_t (&u)[8]) __attribute__((always_inline)) {
            return uint4{__builtin_amdgcn_perm(u[1], u[0], 0x07060302u), __builtin_amdgcn_perm(u[3], u[2], 0x07060302u),
                         __builtin_amdgcn_perm(u[5], u[4], 0x07060302u), __builtin_amdgcn_perm(u[7], u[6], 0x07060302u)};
        };
        o[0] = pack(w);
        o[1] = pack(m);
        o[2] = pack(l);
    }
};

__device__ __forceinline__ void mma(f32x4_t &acc, const uint4 &a, const uint4 &b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                  acc, 0, 0, 0);
}
// -1/16 in every element: its products sum the rows' elements, as the zero point takes them.
constexpr uint32_t kMinus16th = 0xBD80BD80u;

// One wave: 16 rows and 16 output channels.
template <class X, bool kSwiglu>
__global__ __launch_bounds__(256) void w4_tile_kernel(W4Params p) {
    constexpr int kN = kSwiglu ? 2 : 1;  // channel tiles of a wave
    const int lane = lane_id(), col = lane & 15, q = lane >> 4;
    const int Mo = kSwiglu ? p.M / 2 : p.M, S = (Mo + kTile - 1) / kTile;
    TileScan sc;
    int tiles = (p.n_rows + kTile - 1) / kTile;
    if (p.offsets) {
        sc = scan_tiles(p.offsets, p.E, p.n_rows, kTile);
        tiles = sc.total;
    }
    const int64_t units = (int64_t)tiles * S;
    for (int64_t u = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); u < units;
         u += (int64_t)gridDim.x * 4) {
        Unit v;
        if (p.offsets) v = pick_unit(sc, lane, (int)u, S, kTile);
        else {
            const int ti = (int)(u / S);
            v = Unit{{0, ti * kTile, min(kTile, p.n_rows - ti * kTile)}, (int)(u - (int64_t)ti * S) * kTile};
        }
        const int m = min(v.m0 + col, Mo - 1);
        const X *x = reinterpret_cast<const X *>(p.x) + (size_t)(v.t.start + min(col, v.t.n - 1)) * p.K + 8 * q;
        const uint8_t *w = p.w + ((size_t)v.t.e * p.M + m) * (p.K / 2) + 4 * q;
        const size_t sb = (size_t)v.t.e * (p.K / p.group) * p.M + m;
        f32x4_t acc[kN] = {};
        for (int k = 0; k < p.K; k += kStepK) {
            Rows8<X> r;
            r = *reinterpret_cast<const Rows8<X> *>(x + k);
            uint4 a[Rows8<X>::kParts];
            r.parts(a);
            const size_t sg = sb + (size_t)(k / p.group) * p.M;
            f32x4_t rows = {};
            if (p.zero)
#pragma unroll
                for (int i = 0; i < Rows8<X>::kParts; ++i)
                    mma(rows, a[i], uint4{kMinus16th, kMinus16th, kMinus16th, kMinus16th});
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const uint4 b = codes8(*reinterpret_cast<const uint32_t *>(w + (size_t)j * Mo * (p.K / 2) + k / 2));
                f32x4_t sum = {};
#pragma unroll
                for (int i = 0; i < Rows8<X>::kParts; ++i) mma(sum, a[i], b);
                const size_t at = sg + (size_t)j * Mo;
                const float s = 16.0f * (p.scale_f32 ? reinterpret_cast<const float *>(p.scale)[at]
                                                     : bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(p.scale)[at]));
                if (p.zero) sum += (float)((int)p.zero[at] - 8) * rows;
                acc[j] += s * sum;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 4 * q + i;
            if (n >= v.t.n || v.m0 + col >= Mo) continue;
            float z = acc[0][i];
            if constexpr (kSwiglu) z = (z < kFarGate ? silu_far(z) : silu(z)) * acc[1][i];
            const size_t at = (size_t)(v.t.start + n) * Mo + m;
            if (p.y_f32) reinterpret_cast<float *>(p.y)[at] = z;
            else reinterpret_cast<uint16_t *>(p.y)[at] = (uint16_t)(pack_bf16(z, 0.0f) & 0xFFFFu);
        }
    }
}

}  // namespace

hipError_t launch_matmul_w4(const W4Params &p, int x_dtype, bool swiglu, hipStream_t s) {
    const int Mo = swiglu ? p.M / 2 : p.M;
    const long tiles = p.offsets ? p.n_rows / kTile + (p.E < p.n_rows ? p.E : p.n_rows) : (p.n_rows + kTile - 1) / kTile;
    const long blocks = (tiles * ((Mo + kTile - 1) / kTile) + 3) / 4;
    const unsigned grid = (unsigned)(blocks < 16384 ? blocks : 16384);
    if (x_dtype == 0) {
        if (swiglu) launch_k(w4_tile_kernel<float, true>, grid, 256, 0, s, p);
        else launch_k(w4_tile_kernel<float, false>, grid, 256, 0, s, p);
    } else {
        if (swiglu) launch_k(w4_tile_kernel<uint16_t, true>, grid, 256, 0, s, p);
        else launch_k(w4_tile_kernel<uint16_t, false>, grid, 256, 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace moe
