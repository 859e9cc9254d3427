// w4.hip - products with 4-bit weights and a scale (and a zero point) per group of columns, grouped by
// expert: y[n][m] = sum_g s[g][m] sum_{k in g} x[n][k] (c[m][k] - z[g][m]) for the rows n of expert e.
//
// Nothing is rounded on the way to the sums: a code is a whole number, exact in bf16, and a bf16 row
// element is an operand as it stands; fp32 rows go in as three bf16 parts that add up to all of their 24
// bits. A group's sum runs in the matrix instructions (16x16x32, fp32 sums), the zero point and the scale
// are applied to it in fp32: s (sum x (c - b) - (z - b) sum x), b a constant of the operand's form.
// Rows are the A operand and channels the B operand: a lane's accumulators are four rows of one
// channel, so that one scale serves all of a lane's sums.
#include <math.h>

#include "device_common.h"
#include "expert_tiles.h"
#include "kernels.h"

namespace moe {

namespace {

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
    static constexpr int kParts = 3, kPer = 2;
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

// One wave: 16 rows and 16 output channels.
template <class X, bool kSwiglu>
__global__ __launch_bounds__(256) void w4_tile_kernel(W4Params p) {
    using F = Form<X>;
    const F form;
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
            uint4 v8[F::kPer], a[F::kParts];
#pragma unroll
            for (int i = 0; i < F::kPer; ++i) v8[i] = F::order(load16(x + k + 4 * i));
            F::parts(v8, a);
            const size_t sg = sb + (size_t)(k / p.group) * p.M;
            f32x4_t rows = {};
#pragma unroll
            for (int i = 0; i < F::kParts; ++i) mma(rows, a[i], all(F::kMinus));
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const uint4 b = form.codes(*reinterpret_cast<const uint32_t *>(w + (size_t)j * Mo * (p.K / 2) + k / 2));
                f32x4_t sum = {};
#pragma unroll
                for (int i = 0; i < F::kParts; ++i) mma(sum, a[i], b);
                const size_t at = sg + (size_t)j * Mo;
                const float s = p.scale_f32 ? reinterpret_cast<const float *>(p.scale)[at]
                                            : bf16_bits_to_f32(reinterpret_cast<const uint16_t *>(p.scale)[at]);
                sum += ((p.zero ? (float)p.zero[at] : 8.0f) - F::kFrom) * rows;
                acc[j] += s * sum;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = 4 * q + i;
            if (n >= v.t.n || v.m0 + col >= Mo) continue;
            float z = acc[0][i] / F::kUnit;
            if constexpr (kSwiglu) z = (z < kFarGate ? silu_far(z) : silu(z)) * (acc[1][i] / F::kUnit);
            const size_t at = (size_t)(v.t.start + n) * Mo + m;
            if (p.y_f32) reinterpret_cast<float *>(p.y)[at] = z;
            else reinterpret_cast<uint16_t *>(p.y)[at] = (uint16_t)(pack_bf16(z, 0.0f) & 0xFFFFu);
        }
    }
}

// ------------------------------------------------------------------------- few rows per expert
// With a few rows per expert the time is the one read of the weights. A wave takes up to 4 kR rows of one
// expert and 32 weight channels (with SwiGLU 16 gate and the matching 16 up channels) and streams the
// channels' codes in slabs of 128 bytes (256 columns), whole cache lines loaded straight into its own
// ring of slab buffers, with the slab's scales and zero points beside them. The rows come through
// buffer loads into registers; rows past the tile's read as zero without a memory access.
// One-wave blocks fill a CU's LDS. They are persistent: a wave walks its units, and the ring takes the
// next unit's first slabs while the last slabs and the results of the present one are worked on.
// kKS waves make a block and split K between them (their sums join in LDS, in order) where there is so
// little to stream that single waves would not cover the chip; each such block takes one unit.
//
// Of every four operand rows 4a .. 4a + 3 the tile's tokens fill only kR; the others hold the same
// tokens' columns of the next steps, so that a slab of 4 rows takes two loads in place of eight. Operand row
// 4a + kR b + r holds token a + 4 r, b steps on. All four are multiplied with a step's codes, and
// of the four sums of a lane those are taken whose columns are the step's: a sum is only continued by
// a step of the same place. The rows' own sums, for the zero points, need one instruction for 4 / kR steps.
constexpr int kSCh = 32;                   // weight channels of a wave
constexpr int kSlabB = 128;                // bytes of a channel's codes in a slab
constexpr int kSlabK = 2 * kSlabB;         // columns
constexpr int kSteps = kSlabK / kStepK;    // matrix instructions per 16 channels and slab
constexpr int kCodeBytes = kSCh * kSlabB;  // a slab's codes
constexpr int kScaleBytes = kWave * 16;    // room for its scales: at most 8 groups of 32 fp32 numbers
constexpr int kZeroBytes = kWave * 4;      // and zero points
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

// kGen: fp32 scales or zero points; otherwise bf16 scales alone.
template <class X, bool kSwiglu, int kR, int kKS, bool kGen>
__global__ __launch_bounds__(kKS *kWave) __attribute__((amdgpu_waves_per_eu(2))) void w4_stream_kernel(W4Params p) {
    using F = Form<X>;
    constexpr int kPer = F::kPer;
    constexpr int kXL = 2 * kR;          // row fragments of a slab
    // slabs in flight: their rows' registers set the limit
    constexpr int kRing = kKS > 1 ? 2 : kXL * kPer >= 8 ? 3 : 4;
    constexpr int kSlot = kCodeBytes + kScaleBytes + (kGen ? kZeroBytes : 0);
    // one object per ring slot, so that the compiler can tell loads into one from reads of another
    __shared__ __align__(16) unsigned char ring0[kKS][kSlot], ring1[kKS][kSlot], ring2[kRing > 2 ? kKS : 1][kRing > 2 ? kSlot : 16],
        ring3[kRing > 3 ? kKS : 1][kRing > 3 ? kSlot : 16];
    constexpr int kCols = kSwiglu ? kSCh / 2 : kSCh;  // output channels of a block
    constexpr int kRows = 4 * kR;
    constexpr bool kWalk = kKS == 1;
    const F form;
    const int lane = lane_id(), wave = kKS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
    const int col = lane & 15, q = lane >> 4;
    auto slot = [&](auto ic) __attribute__((always_inline)) -> unsigned char * {
        constexpr int B = decltype(ic)::value;
        return B == 0 ? ring0[wave] : B == 1 ? ring1[wave] : B == 2 ? ring2[wave] : ring3[wave];
    };
    const int Mo = kSwiglu ? p.M / 2 : p.M, KB = p.K / 2;
    const int S = (Mo + kCols - 1) / kCols;
    TileScan sc;
    int tiles = (p.n_rows + kRows - 1) / kRows;
    if (p.offsets) {
        sc = scan_tiles(p.offsets, p.E, p.n_rows, kRows);
        tiles = sc.total;
    }
    const int units = tiles * S, per = (units + kXcds - 1) / kXcds;
    const int first = (blockIdx.x % kXcds) * per, last = min(first + per, units), step = gridDim.x / kXcds;
    int u = first + blockIdx.x / kXcds;
    if (u >= last) return;  // uniform
    auto unit = [&](int i) __attribute__((always_inline)) {
        if (p.offsets) return find_unit<kRows>(sc, lane, i, S, kCols);
        const int ti = i / S;
        return Unit{{0, ti * kRows, min(kRows, p.n_rows - ti * kRows)}, (i - ti * S) * kCols};
    };
    // this wave's slabs: s0 .. s0 + share - 1, in whole turns of the ring
    const int nslab = (p.K + kSlabK - 1) / kSlabK;
    const int share = (nslab + kKS - 1) / kKS, s0 = wave * share;
    const int turns = (share + kRing - 1) / kRing * kRing;
    // segment a of a slab: staged rows 8a .. 8a + 7 (SwiGLU: rows 16 .. 31 are the up channels)
    uint32_t woff[kSCh / 8];
    int wk[kSCh / 8];
#pragma unroll
    for (int a = 0; a < kSCh / 8; ++a) {
        const int R = 8 * a + (lane >> 3), c = kSwiglu ? (R & 15) + (R >> 4) * Mo : R;
        wk[a] = (((lane & 7) ^ (R >> 1)) & 7) * 16;
        woff[a] = (uint32_t)c * KB + wk[a];
    }
    // row fragment j: step j (4 / kR) + xs of token a + 4 (b4 % kR)
    const int b4 = col & 3, xs = b4 / kR;
    const uint32_t xoff = ((uint32_t)((col >> 2) + 4 * (b4 % kR)) * p.K + xs * kStepK + 8 * q) * sizeof(X);
    // scales: groups of a slab, 32 channels each (SwiGLU: 16 gate, 16 up), in 16-byte pieces
    const int gl = p.group == 128 ? 2 : p.group == 64 ? 1 : 0;  // log2 of the steps of a group
    const int slabg = kSteps >> gl, groups = p.K / p.group;
    const bool wide = kGen && p.scale_f32;
    const int sb = wide ? 4 : 2;                                // bytes of a scale
    const int sg = lane >> (wide ? 3 : 2), sp = lane & (wide ? 7 : 3), shalf = wide ? 4 : 2;
    const uint32_t soff = (uint32_t)(sg * p.M + (kSwiglu && sp >= shalf ? Mo : 0)) * sb + (kSwiglu ? sp % shalf : sp) * 16;
    const int zg = lane >> 3, zp = lane & 7;
    const uint32_t zoff = (uint32_t)(zg * p.M + (kSwiglu && zp >= 4 ? Mo : 0) + (kSwiglu ? zp % 4 : zp) * 4);
    // reading them: the word of the lane's channel, and which half of it (fp32: all)
    const int s_word = col * sb & ~3, s_shift = wide || (col & 1) ? 0 : 16;
    const uint32_t s_mask = wide ? ~0u : 0xFFFF0000u;
    const float z_bias = (p.zero ? 0.0f : 8.0f) - F::kFrom;  // without zero points 0s are loaded
    uint4 xr[kRing][kXL][kPer];
    // where a unit's operands lie, from this wave's first slab on; a unit that does not exist has none
    struct From {
        const unsigned char *x, *w, *s, *z;
        uint32_t nx, nw, ns;  // bytes of rows and codes, scales in number
    };
    auto from = [&](const Unit &v, bool any) __attribute__((always_inline)) {
        const size_t at = (size_t)v.t.e * groups * p.M + v.m0;
        return From{reinterpret_cast<const unsigned char *>(p.x) + (size_t)v.t.start * p.K * sizeof(X),
                    p.w + ((size_t)v.t.e * p.M + v.m0) * KB,
                    reinterpret_cast<const unsigned char *>(p.scale) + at * sb, p.zero + (p.zero ? at : 0),
                    any ? (uint32_t)v.t.n * (uint32_t)p.K * (uint32_t)sizeof(X) : 0u,
                    any ? (uint32_t)(p.M - v.m0) * (uint32_t)KB : 0u,
                    any ? (uint32_t)groups * (uint32_t)p.M - (uint32_t)v.m0 : 0u};
    };
    // the wave's slab i of a unit: always the same number of loads (they are counted); pieces at or past
    // K, slabs past the share and units that do not exist read as zero
    auto issue = [&](auto ic, const From &f, int i) __attribute__((always_inline)) {
        constexpr int B = decltype(ic)::value;
        const int s = s0 + i;
        const int left = i < share ? KB - s * kSlabB : 0;      // bytes of a channel's codes from this slab on
        const int gleft = i < share ? groups - s * slabg : 0;  // groups from this slab on
        const uint32_t wb = (uint32_t)s * kSlabB, xb = wb * 2 * (uint32_t)sizeof(X), gb = (uint32_t)(s * slabg) * p.M;
        // (the saturating difference is a vector instruction: brought back to a scalar)
        auto rest = [](uint32_t all, uint32_t at) __attribute__((always_inline)) {
            return (uint32_t)__builtin_amdgcn_readfirstlane((int)(all > at ? all - at : 0u));
        };
        const __amdgpu_buffer_rsrc_t rw = buffer_rsrc(f.w + wb, rest(f.nw, wb)), rx = buffer_rsrc(f.x + xb, rest(f.nx, xb));
        auto loads = [&](auto full) __attribute__((always_inline)) {
            constexpr bool kFull = decltype(full)::value;
#pragma unroll
            for (int a = 0; a < kSCh / 8; ++a)
                to_lds16<kBufNT>(rw, slot(ic) + a * 1024, kFull || wk[a] < left ? woff[a] : kPast);
#pragma unroll
            for (int j = 0; j < kXL; ++j)
#pragma unroll
                for (int h = 0; h < kPer; ++h)
                    xr[B][j][h] = __builtin_bit_cast(
                        uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                   rx,
                                   (int)(kFull || (j * (4 / kR) + xs) * (kStepK / 2) < left
                                             ? xoff + (uint32_t)(j * (4 / kR) * kStepK * (int)sizeof(X) + 16 * h)
                                             : kPast),
                                   0, 0));
        };
        to_lds16<0>(buffer_rsrc(f.s + (size_t)gb * sb, rest(f.ns, gb) * sb), slot(ic) + kCodeBytes, sg < slabg && sg < gleft ? soff : kPast);
        if constexpr (kGen)
            to_lds4(buffer_rsrc(f.z + (p.zero ? gb : 0), p.zero ? rest(f.ns, gb) : 0u), slot(ic) + kCodeBytes + kScaleBytes,
                    zg < slabg && zg < gleft ? zoff : kPast);
        if (left >= kSlabB) loads(std::true_type{});
        else loads(std::false_type{});
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    // loads of the younger slabs may be outstanding when a slab is used
    constexpr int kYoung = (kRing - 1) * (kSCh / 8 + 1 + (kGen ? 1 : 0) + kXL * kPer);
    static_assert(kYoung < 64, "vmcnt has six bits");
    constexpr int kWait = (kYoung & 15) | 0x0F70 | ((kYoung >> 4) << 14);

    Unit cur = unit(u);
    From at = from(cur, true);
    issue(I0{}, at, 0);
    issue(I1{}, at, 1);
    if constexpr (kRing > 2) issue(I2{}, at, 2);
    if constexpr (kRing > 3) issue(I3{}, at, 3);
    for (;;) {
        u += step;
        const bool more = kWalk && u < last;
        const Unit nxt = more ? unit(u) : cur;
        const From next = from(nxt, more);
        float acc[2][kR] = {};
        // one slab, a scale per kG steps
        auto work = [&](auto ic, auto gc) __attribute__((always_inline)) {
            constexpr int B = decltype(ic)::value, kG = 1 << decltype(gc)::value;
            constexpr int kPack = 4 / kR;                          // steps in a row fragment
            constexpr int kPos = kG < kPack ? kG : kPack;          // of them, those of one group
            constexpr int kFrags = kG < kPack ? 1 : kG / kPack;    // fragments of a group
            constexpr bool kMinus = kGen || F::kMinus24 != 0;
            f32x4_t sum[2][kPos], rows = {};
            uint4 a[kFrags][F::kParts];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                if (s == kSteps / 2) __builtin_amdgcn_sched_barrier(0);  // registers
                if (s % (kPack * kFrags) == 0) {
                    rows = f32x4_t{};
#pragma unroll
                    for (int f = 0; f < kFrags; ++f) {
                        uint4 v[kPer];
#pragma unroll
                        for (int h = 0; h < kPer; ++h) v[h] = F::order(xr[B][s / kPack + f][h]);
                        F::parts(v, a[f]);
                        if constexpr (kMinus)
#pragma unroll
                            for (int i = 0; i < F::kParts; ++i) mma(rows, a[f][i], all(kGen ? F::kMinus : F::kMinus24));
                    }
                }
                const int pos = s % kPos, frag = s / kPack % kFrags;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (s % kG < kPos) sum[t][pos] = kMinus && !kGen ? rows : f32x4_t{};
                    const uint4 b = form.codes(*reinterpret_cast<const uint32_t *>(slot(ic) + t * kTile * kSlabB + spos(col, s) + 4 * q));
#pragma unroll
                    for (int i = 0; i < F::kParts; ++i) mma(sum[t][pos], a[frag][i], b);
                    if (s % kG != kG - 1) continue;
                    const int at = s / kG * kSCh + t * kTile;
                    const unsigned char *aux = slot(ic) + kCodeBytes;
                    float scale, z = 0.0f;
                    if constexpr (kGen) {
                        scale = __uint_as_float((*reinterpret_cast<const uint32_t *>(aux + at * sb + s_word) << s_shift) & s_mask);
                        z = (float)(int)aux[kScaleBytes + at + col] + z_bias;
                    } else {
                        scale = bf16_bits_to_f32(*reinterpret_cast<const uint16_t *>(aux + (at + col) * 2));
                    }
#pragma unroll
                    for (int r = 0; r < kR; ++r) {
                        const int e = (s - (kPos - 1)) % kPack * kR + r;  // where the group's first step stands
                        float v = sum[t][(s - (kPos - 1)) % kPos][e], w = rows[e];
#pragma unroll
                        for (int i = 1; i < kPos; ++i) {
                            v += sum[t][(s - (kPos - 1) + i) % kPos][e + i * kR];
                            w += rows[e + i * kR];
                        }
                        acc[t][r] = fmaf(scale, kGen ? fmaf(z, w, v) : v, acc[t][r]);
                    }
                }
            }
        };
        auto turn = [&](auto ic, int i) __attribute__((always_inline)) {
            __builtin_amdgcn_s_waitcnt(kWait);
            __builtin_amdgcn_sched_barrier(0);  // the loads counted above stay on their side of it
            if (gl == 2) work(ic, I2{});
            else if (gl == 1) work(ic, I1{});
            else work(ic, I0{});
            // The refill goes into the slot that was read: it is requested once the reads have returned
            // (one past K is answered without a memory access, so latency orders nothing).
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0xC07F);  // LDS reads: none outstanding; loads: not waited for
            __builtin_amdgcn_sched_barrier(0);
            const bool here = i + kRing < turns;  // uniform
            issue(ic, here ? at : next, here ? i + kRing : i + kRing - turns);
        };
        int i = 0;
        do {
            turn(I0{}, i);
            turn(I1{}, i + 1);
            if constexpr (kRing > 2) turn(I2{}, i + 2);
            if constexpr (kRing > 3) turn(I3{}, i + 3);
        } while ((i += kRing) < turns);
        bool mine = true;
        if constexpr (kKS > 1) {  // join the waves' sums in wave 0, in order
            __shared__ float red[kKS - 1][2][kR][kWave];
            mine = wave == 0;
            if (!mine) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < kR; ++r) red[wave - 1][t][r][lane] = acc[t][r];
            }
            __syncthreads();
            if (mine) {
#pragma unroll
                for (int w = 0; w < kKS - 1; ++w)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int r = 0; r < kR; ++r) acc[t][r] += red[w][t][r][lane];
            }
        }
        if (mine) {
#pragma unroll
            for (int r = 0; r < kR; ++r) {
                const int n = q + 4 * r;
                if (n >= cur.t.n) continue;
#pragma unroll
                for (int t = 0; t < (kSwiglu ? 1 : 2); ++t) {
                    const int m = cur.m0 + t * kTile + col;
                    if (m >= Mo) continue;
                    float z = acc[t][r] / F::kUnit;
                    if constexpr (kSwiglu) z = (z < kFarGate ? silu_far(z) : silu(z)) * (acc[1][r] / F::kUnit);
                    const size_t at = (size_t)(cur.t.start + n) * Mo + m;
                    if (p.y_f32) reinterpret_cast<float *>(p.y)[at] = z;
                    else reinterpret_cast<uint16_t *>(p.y)[at] = (uint16_t)(pack_bf16(z, 0.0f) & 0xFFFFu);
                }
            }
        }
        if (!more) break;
        cur = nxt;
        at = next;
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // no load into this block's LDS outlives it
}

}  // namespace

namespace {

// The most row tiles of `per` rows that n_rows rows of E experts can make.
long most_tiles(const W4Params &p, int per) {
    if (!p.offsets) return (p.n_rows + per - 1) / per;
    const long parts = p.n_rows / per + (p.E < p.n_rows ? p.E : p.n_rows);
    return parts < p.n_rows ? parts : p.n_rows;
}

template <class X, int kR, int kKS>
void launch_stream(const W4Params &p, bool swiglu, unsigned grid, hipStream_t s) {
    const bool gen = p.zero || p.scale_f32;
    if (gen && swiglu) launch_k(w4_stream_kernel<X, true, kR, kKS, true>, grid, kKS * kWave, 0, s, p);
    else if (gen) launch_k(w4_stream_kernel<X, false, kR, kKS, true>, grid, kKS * kWave, 0, s, p);
    else if (swiglu) launch_k(w4_stream_kernel<X, true, kR, kKS, false>, grid, kKS * kWave, 0, s, p);
    else launch_k(w4_stream_kernel<X, false, kR, kKS, false>, grid, kKS * kWave, 0, s, p);
}

constexpr int kStreamBlocks = 8;  // one-wave blocks per CU (LDS)
constexpr int kSplit = 8;         // waves that split K where there are few units

}  // namespace

hipError_t launch_matmul_w4(const W4Params &p, int x_dtype, bool swiglu, hipStream_t s) {
    const int Mo = swiglu ? p.M / 2 : p.M, cus = num_cus();
    const double experts = p.offsets ? (p.E < p.n_rows ? p.E : p.n_rows) : 1, rows = p.n_rows / experts;
    if (rows <= 16) {
        const int r = rows <= 3 ? 1 : rows <= 7 || x_dtype == 0 ? 2 : 4;
        const int cols = swiglu ? kSCh / 2 : kSCh, S = (Mo + cols - 1) / cols;
        const long units = most_tiles(p, 4 * r) * S;
        const bool split = units <= 2 * cus && p.K > kSlabK;
        const long room = (long)cus * kStreamBlocks;
        const long blocks = units <= room || split ? units : room;
        const unsigned grid = (unsigned)((blocks + kXcds - 1) / kXcds * kXcds);
        auto go = [&](auto x, auto rc) {
            using X = decltype(x);
            constexpr int kR = decltype(rc)::value;
            if (split) launch_stream<X, kR, kSplit>(p, swiglu, grid, s);
            else launch_stream<X, kR, 1>(p, swiglu, grid, s);
        };
        using R1 = std::integral_constant<int, 1>;
        using R2 = std::integral_constant<int, 2>;
        using R4 = std::integral_constant<int, 4>;
        if (x_dtype == 0) r == 1 ? go(float{}, R1{}) : go(float{}, R2{});
        else r == 1 ? go(uint16_t{}, R1{}) : r == 2 ? go(uint16_t{}, R2{}) : go(uint16_t{}, R4{});
        return hipGetLastError();
    }
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
