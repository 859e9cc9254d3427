// expert_tiles.h - what the products grouped by expert share: how their rows are cut into tiles and
// units, the SwiGLU epilogue, loads straight into LDS.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>

#include "device_common.h"

namespace moe {

constexpr int kXcds = 8;

// Row tiles of the experts in order: expert e's rows [lo, hi) in as few tiles of at most `per` rows
// as hold them, of even sizes (multiples of 16 but for the last). Every wave finds its units by
// itself: lane l sums the tiles of experts 4l .. 4l + 3, a wave scan places them.
struct RowTile {
    int e, start, n;  // n = 0: there is no such tile
};
struct TileScan {
    int lo[4], nt[4], hi[4], at;  // ranges and tiles of the lane's experts, tiles before them
    int total;
};
__device__ __forceinline__ TileScan scan_tiles(const int32_t *offsets, int E, int n_rows, int per) {
    TileScan s;
    const int lane = lane_id();
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = min(4 * lane + i, E);  // past the last expert: an empty range
        s.lo[i] = min(max(offsets[e], 0), n_rows);
        s.hi[i] = min(max(offsets[min(e + 1, E)], s.lo[i]), n_rows);
        s.nt[i] = (s.hi[i] - s.lo[i] + per - 1) / per;
        sum += s.nt[i];
    }
    const int incl = wave_inclusive_sum(sum);
    s.at = incl - sum;
    s.total = __builtin_amdgcn_readlane(incl, kWave - 1);
    return s;
}
// One unit of work: a row tile and its first output channel.
struct Unit {
    RowTile t;
    int m0;
};
// Unit u of S blocks of `cols` output channels per tile. An expert's units run channel block by
// channel block, its tiles next to each other: they read the same weights at about the same time.
__device__ __forceinline__ Unit pick_unit(const TileScan &s, int lane, int u, int S, int cols) {
    int at = s.at, e = 0, start = 0, n = 0, c = 0;
    bool mine = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int nt = s.nt[i];
        if (u >= at * S && u < (at + nt) * S) {
            mine = true;
            e = 4 * lane + i;
            c = (u - at * S) / nt;
            const int rows = s.hi[i] - s.lo[i], part = ((rows + nt - 1) / nt + 15) & ~15;
            start = s.lo[i] + (u - at * S - c * nt) * part;
            n = min(part, s.hi[i] - start);
        }
        at += nt;
    }
    const uint64_t who = __ballot(mine);
    if (!who) return {{0, 0, 0}, 0};
    const int src = __ffsll((unsigned long long)who) - 1;
    return {{__builtin_amdgcn_readlane(e, src), __builtin_amdgcn_readlane(start, src),
             __builtin_amdgcn_readlane(n, src)},
            __builtin_amdgcn_readlane(c, src) * cols};
}

__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(uint16_t *p, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(p) = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// silu(z) = z / (1 + e^-z). e^-z = 2^t (1 + c), t the rounded product -z log2(e) and c the part that
// the rounding and the constant left off, so that the error stays a few steps of fp32 however large
// z is. The bound on the exponent keeps t and c finite.
constexpr float kLog2e = 1.44269502f, kLog2eRest = 1.92596299e-8f, kLn2 = 0.693147182f;
__device__ __forceinline__ float exp_rest(float a, float t) {
    return fmaf(a, kLog2eRest, fmaf(a, kLog2e, -t)) * kLn2;
}
// Gates from kFarGate up: about ten instructions. Below it 1 + e^-z passes 2^126 and its reciprocal,
// which the hardware gives as 0, is no normal number any more.
constexpr float kFarGate = -87.0f;
__device__ __forceinline__ float silu(float z) {
    const float a = __builtin_amdgcn_fmed3f(-z, -150.0f, 150.0f);
    const float t = a * kLog2e;
    const float e = __builtin_amdgcn_exp2f(t) * (1.0f + exp_rest(a, t));
    return z * __builtin_amdgcn_rcpf(1.0f + e);
}
// Gates below kFarGate, where 1 + e^-z is e^-z to far less than a step: z e^z, a normal number down to
// z = -91.9. e^z is multiplied in by halves, which are normal where the result is not yet 0. (Past
// -1000 it is 0 whatever z is; -infinity gives NaN, as the quotient above.)
__device__ __forceinline__ float silu_far(float z) {
    const float a = fmaxf(z, -1000.0f);
    const float t = a * kLog2e, h = __builtin_amdgcn_exp2f(0.5f * t);
    return z * h * (1.0f + exp_rest(a, t)) * h;
}
// z = silu(z) up of four channels. Far gates are as good as never met: one test for all four.
__device__ __forceinline__ void swiglu4(float (&z)[4], const float (&up)[4]) {
    float s[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] = silu(z[r]);
    if (__builtin_expect(fminf(fminf(z[0], z[1]), fminf(z[2], z[3])) < kFarGate, 0)) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (z[r] < kFarGate) s[r] = silu_far(z[r]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) z[r] = s[r] * up[r];
}

template <int kAux>
__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t r, void *seg, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)seg, 16, (int)off,
                                             0, 0, kAux);
}
__device__ __forceinline__ void to_lds4(__amdgpu_buffer_rsrc_t r, void *seg, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)seg, 4, (int)off,
                                             0, 0, 0);
}

// Lanes of a wave exchange values through LDS: fenced at wavefront scope, without which the
// compiler may forward a lane's own earlier store to its load.
__device__ __forceinline__ void wave_exchange() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// CUs of the current device (looked up once per device).
inline int num_cus() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < kXcds)
            n = 256;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace moe
