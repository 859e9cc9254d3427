// w4_core.h - what the kernels of the products with 4-bit weights share: operand forms, units of work.
#pragma once

#include "device_common.h"
#include "expert_tiles.h"
#include "kernels.h"
#include "w4_choice.h"

namespace moe {

constexpr int kStepK = 32;  // columns of one matrix instruction; a scale's group is 1, 2 or 4 of them

// Operand forms by the rows' type. codes(w): eight codes (one word, column j in bits 4j .. 4j + 3) as bf16
// numbers kUnit (code - kFrom); parts(): a row fragment, eight consecutive elements as loaded, as bf16
// operands that add up to it, its columns in the order that codes() leaves. What a zero point z adds
// is kUnit (kFrom - z) times the rows' sums, which the matrix instructions form as the products with
// kMinus: rows' = -kUnit sum x, so that a group's sum is  codes' sum + (z - kFrom) rows'.
__device__ __forceinline__ uint32_t halves(uint32_t hi, uint32_t lo, uint32_t sel) { return __builtin_amdgcn_perm(hi, lo, sel); }
constexpr uint32_t kLow = 0x05040100u, kHigh = 0x07060302u;  // both low halves, both high halves

template <class X>
struct Form;

// bf16 rows: a code goes into the mantissa of 16, which makes 16 + code in one instruction for two codes
// and one shift. The sums are up to five times as large as with code - 8, and so are their roundings:
// 2^-22 or so of the result, far below a bf16 element's own half step of 2^-9. (Converting the codes
// takes 14 instructions for eight in place of 8.) Columns j and j + 4 come out side by side.
template <>
struct Form<uint16_t> {
    static constexpr int kParts = 1, kPer = 1;  // operands and 16-byte pieces of a fragment
    static constexpr int kSplit = 2;            // parts of a slab that the scheduler keeps apart
    static constexpr float kFrom = -16.0f, kUnit = 1.0f;
    static constexpr uint32_t kMinus = 0xBF80BF80u;     // -1
    static constexpr uint32_t kMinus24 = 0xC1C0C1C0u;   // 8 - kFrom of them
    // (the constants are kept in registers: with two literals the and and the or stay two instructions)
    uint32_t bits = 0x00780078u, from16 = 0x41804180u;
    __device__ __forceinline__ Form() { asm("" : "+s"(bits), "+v"(from16)); }
    __device__ __forceinline__ uint4 codes(uint32_t w) const {
        return uint4{((w << 3) & bits) | from16, ((w >> 1) & bits) | from16, ((w >> 5) & bits) | from16,
                     ((w >> 9) & bits) | from16};
    }
    __device__ static __forceinline__ uint4 order(const uint4 &v) {
        return uint4{halves(v.z, v.x, kLow), halves(v.z, v.x, kHigh), halves(v.w, v.y, kLow), halves(v.w, v.y, kHigh)};
    }
    __device__ static __forceinline__ void parts(const uint4 (&v)[1], uint4 (&o)[1]) { o[0] = v[0]; }
};

// fp32 rows: x = hi + mid + lo, each of at most 8 significant bits (cut off, not rounded). Their sums keep
// what an fp32 product would: with bit 3 turned over a code is a signed 4-bit number, which one
// instruction converts to fp32 as that number / 16, exact in its upper half.
template <>
struct Form<float> {
    static constexpr int kParts = 3, kPer = 2, kSplit = 4;
    static constexpr float kFrom = 8.0f, kUnit = 1.0f / 16.0f;
    static constexpr uint32_t kMinus = 0xBD80BD80u;  // -1/16
    static constexpr uint32_t kMinus24 = 0;          // 8 - kFrom is 0
    __device__ __forceinline__ uint4 codes(uint32_t w) const {
        const uint32_t a = w ^ 0x88888888u, b = a >> 4;
        auto f = [](uint32_t v) __attribute__((always_inline)) {
            return __float_as_uint(__builtin_amdgcn_cvt_off_f32_i4((int)v));
        };
        return uint4{halves(f(b), f(a), kHigh), halves(f((b >> 8) & 0xFFu), f((a >> 8) & 0xFFu), kHigh),
                     halves(f((b >> 16) & 0xFFu), f((a >> 16) & 0xFFu), kHigh), halves(f(b >> 24), f(a >> 24), kHigh)};
    }
    __device__ static __forceinline__ uint4 order(const uint4 &v) { return v; }
    __device__ static __forceinline__ void parts(const uint4 (&v)[2], uint4 (&o)[3]) {
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        uint32_t m[8], l[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float rest = __uint_as_float(w[i]) - __uint_as_float(w[i] & 0xFFFF0000u);
            m[i] = __float_as_uint(rest);
            l[i] = __float_as_uint(rest - __uint_as_float(m[i] & 0xFFFF0000u));
        }
        auto pack = [](const uint32_t (&u)[8]) __attribute__((always_inline)) {
            return uint4{halves(u[1], u[0], kHigh), halves(u[3], u[2], kHigh), halves(u[5], u[4], kHigh),
                         halves(u[7], u[6], kHigh)};
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
__device__ __forceinline__ uint4 all(uint32_t v) { return uint4{v, v, v, v}; }

// A slab is a whole cache line of a channel's codes.
constexpr int kSlabB = 128;                // bytes of a channel's codes in a slab
constexpr int kSlabK = 2 * kSlabB;         // columns
static_assert(kSlabK == kW4StreamColumns, "the choice counts these slabs");
constexpr uint32_t kPast = 0xFFFFFFF0u;    // a buffer offset past every range

// Position of 16-byte piece pc (0..7) of staged row r: rows 2m and 2m + 1 rotate by m, so that the 16 rows
// of one operand read lie on distinct banks.
__device__ __forceinline__ int spos(int r, int pc) { return r * kSlabB + ((pc ^ (r >> 1)) & 7) * 16; }

// pick_unit with the units of a tile of kGrain rows found first and placed by scalars: few divisions.
template <int kGrain>
__device__ __forceinline__ Unit find_unit(const TileScan &s, int lane, int u, int S, int cols) {
    int at = s.at, e = 0, nt = 1, before = 0, lo = 0, hi = 0;
    bool mine = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (u >= at * S && u < (at + s.nt[i]) * S)
            mine = true, e = 4 * lane + i, nt = s.nt[i], before = at, lo = s.lo[i], hi = s.hi[i];
        at += s.nt[i];
    }
    const uint64_t who = __ballot(mine);
    if (!who) return {{0, 0, 0}, 0};
    const int src = __ffsll((unsigned long long)who) - 1;
    e = __builtin_amdgcn_readlane(e, src);
    nt = __builtin_amdgcn_readlane(nt, src);
    lo = __builtin_amdgcn_readlane(lo, src);
    hi = __builtin_amdgcn_readlane(hi, src);
    const int in = u - __builtin_amdgcn_readlane(before, src) * S;
    if (nt == 1) return {{e, lo, hi - lo}, in * cols};
    const uint32_t c = (uint32_t)in / (uint32_t)nt;
    const int part = (int)(((uint32_t)(hi - lo + nt - 1) / (uint32_t)nt + kGrain - 1) & ~(kGrain - 1));
    const int start = lo + (in - (int)c * nt) * part;
    return {{e, start, min(part, hi - start)}, (int)c * cols};
}

// The most row tiles of `per` rows that n_rows rows of E experts can make.
inline long most_tiles(const W4Params &p, int per) {
    if (!p.offsets) return (p.n_rows + per - 1) / per;
    const long parts = p.n_rows / per + (p.E < p.n_rows ? p.E : p.n_rows);
    return parts < p.n_rows ? parts : p.n_rows;
}

}  // namespace moe
