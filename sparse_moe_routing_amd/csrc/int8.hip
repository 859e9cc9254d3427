// int8.hip - products of 8-bit integers with a scale per row and per output channel, grouped by
// expert: y[n][m] = sx[n] sw[e][m] sum_k x[n][k] w[e][m][k] for the rows n of expert e.
//
// The sum runs in the integer matrix instructions (16x16x64: int8 operands, int32 accumulators)
// and is exact in any order, so every variant and split gives the same bits; only the two scales
// and the SwiGLU are fp32 arithmetic. Weights are the A operand and rows the B operand: a lane's
// accumulators are four consecutive channels of one row, stored as one piece.
#include <math.h>

#include <atomic>

#include "device_common.h"
#include "kernels.h"

namespace moe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void mma_i8(i32x4_t &acc, const uint4 &a, const uint4 &b) {
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a),
                                                __builtin_bit_cast(i32x4_t, b), acc, 0, 0, 0);
}

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

// z = fp32(sum) * x_scale * w_scale of four channels.
__device__ __forceinline__ void scaled(const i32x4_t &acc, float sx, const float *sw, float (&z)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) z[r] = (float)acc[r] * sx * sw[r];
}

// ------------------------------------------------------------------------- large row counts
// The wide form: a block multiplies up to 320 rows of one expert by 256 weight channels (with
// SwiGLU: 128 gate channels and the 128 up channels that go with them). K is staged in slabs of 128
// bytes per row, whole cache lines loaded straight into LDS (buffer loads with the LDS flag: no registers held
// while in flight), double-buffered: the next slab's loads are in flight during the current slab's
// matrix instructions. Eight waves, two per SIMD: wave w takes the channels of half w % 2 and a
// quarter of the tile's 16-row subtiles, at most five, so that a tile of n rows costs ceil(n / 64)
// subtiles of matrix work per wave whatever n is. Waves w and w + 4, on the same SIMD, run one
// phase apart: while one reads its operands from LDS the other multiplies (one of many calls in a row:
// 65536 rows of 256 experts of 2048 x 1024 194 us in step, 185 so; dense 8192 x 4096 x 4096 131, 126).
//
// A block's 144 KB of slabs leave one block per CU, so nothing else would cover a unit's start and
// end: the blocks are persistent, one per CU, and the last slab of a unit is multiplied (and its
// results are scaled and stored) while the first slab and the scales of the block's next unit load.
//
// Bounds come from the buffer resources: the row resource covers exactly the tile's n rows and the
// weight resource the expert's remaining channels, so that loads past either return zeros without
// a memory access; pieces past K in the last slab are sent past the range in the same way.
//
// Why these sizes: per slab a CU moves 72 KB into LDS and reads 208 KB of operands for 640 matrix
// instructions; 320 x 256 is the patch with the least LDS traffic per product whose sums still fit
// two waves' registers, and at 65536 rows of 256 experts most experts' rows fit one tile, so that
// their weights cross HBM once. Measured, single calls after the caches were filled with other data:
// 65536 rows of 256 experts of 2048 x 1024 with SwiGLU 173 us (1.6 Pop/s; 644 MiB read, the least
// there is; matrix units busy 38 %, waits 38 %); dense 8192 x 4096 x 4096 125 us (2.2 Pop/s). Other
// shapes, each against this one as it was then: 256-row tiles took 10 % longer, 128-channel blocks 14 %,
// four waves of 128 x 128 39 %.
//
// With fewer rows per expert a slab's matrix work is over long before the next slab has landed, and
// one slab ahead is not enough to keep the weights coming. The deep form (kDeep) takes at most 128
// rows a tile; the LDS saved holds a third pair of slab buffers, so that two slabs are in flight
// behind the one in use. A wave counts its loads (always the same number per slab, past the operands
// they read zero), waits for all but the youngest slab's, and there is one barrier per slab. Measured,
// 256 experts of 2048 x 1024 with SwiGLU, 31 rows each: 94 us (562 MB, 6.0 TB/s; the wide form 110),
// skewed 67 (90); dense 512 x 4096 x 4096 27 (39).
constexpr int kBWaves = 8;
constexpr int kBRows = 320, kBCh = 256;   // rows and weight channels per block
constexpr int kSlabB = 128;               // bytes (K elements) of a staged row
constexpr int kBA = kBCh / 2 / kTile;     // channel subtiles per wave (8)
constexpr int kDeepRows = 128;            // rows per block of the deep form
constexpr int kWSegs = kBCh * kSlabB / 1024 / kBWaves;    // 1 KB weight segments per wave (4)
constexpr int kXcds = 8;
constexpr uint32_t kPast = 0xFFFFFFF0u;   // a buffer offset past every range
constexpr uint32_t kFar = 0x80000000u;    // the same with any row's offset added (they stay below 2^30)

// Position of 16-byte piece pc (0..7) of staged row r: rows 2m and 2m + 1 rotate by m, so the 16
// rows of one operand read lie on distinct bank groups; rows 16 apart keep their pieces' order.
__device__ __forceinline__ int spos(int r, int pc) { return r * kSlabB + ((pc ^ (r >> 1)) & 7) * 16; }

// The slab buffers are separate objects, so that the compiler can tell loads into one from operand
// reads of the other.
__shared__ __align__(16) unsigned char b_w0[kBCh * kSlabB], b_w1[kBCh * kSlabB];
__shared__ __align__(16) unsigned char b_x0[kBRows * kSlabB], b_x1[kBRows * kSlabB];
// The deep form's three.
__shared__ __align__(16) unsigned char d_w0[kBCh * kSlabB], d_w1[kBCh * kSlabB], d_w2[kBCh * kSlabB];
__shared__ __align__(16) unsigned char d_x0[kDeepRows * kSlabB], d_x1[kDeepRows * kSlabB],
    d_x2[kDeepRows * kSlabB];
// Scales of the current and the next unit: rows, then staged weight rows.
__shared__ __align__(16) float b_scale[2][kBRows + kBCh];

template <int kAux>
__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t r, void *seg, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)seg, 16, (int)off,
                                             0, 0, kAux);
}
__device__ __forceinline__ void to_lds4(__amdgpu_buffer_rsrc_t r, void *seg, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)seg, 4, (int)off,
                                             0, 0, 0);
}

// The scan of the row tiles, kept out of the registers of the products (written by wave 0).
__shared__ TileScan b_scan[kWave];

// Lanes of a wave exchange values through LDS: fenced at wavefront scope, without which the
// compiler may forward a lane's own earlier store to its load.
__device__ __forceinline__ void wave_exchange() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <bool kSwiglu, class O, bool kOnce, bool kDeep>
struct BlockProduct {
    // 1 KB row segments per wave (5, deep: 2)
    static constexpr int kXSegs = (kDeep ? kDeepRows : kBRows) * kSlabB / 1024 / kBWaves;
    static constexpr int kCols = kSwiglu ? kBCh / 2 : kBCh;  // output channels of a block
    static constexpr int kAux = kOnce ? kBufNT : 0;          // cache policy of the weights
    const I8Params &p;
    int lane, wave, ch, th, Mo;
    int nslab;

    __device__ __forceinline__ BlockProduct(const I8Params &p_) : p(p_) {
        lane = lane_id();
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        ch = wave & 1;
        th = (wave >> 1) & 3;
        Mo = kSwiglu ? p.M / 2 : p.M;
        nslab = (p.K + kSlabB - 1) / kSlabB;
    }
    // The lane number, made anew: what is computed from it stays next to its use instead of in
    // registers across the products, which need them all.
    __device__ __forceinline__ int here() const {
        int l = lane;
        asm volatile("" : "+v"(l));
        return l;
    }
    // weight channel (past m0) of staged row R; SwiGLU: each half of 128 staged rows holds 64 gate
    // channels, then the 64 matching up channels
    __device__ __forceinline__ int channel(int R) const {
        return kSwiglu ? (R >> 7) * 64 + (R & 63) + ((R >> 6) & 1) * Mo : R;
    }
    // Slab s of an operand: segment g holds rows 8g .. 8g + 7; lane l of its load writes position
    // l % 8 of row l / 8, so it reads the piece that the row's rotation puts there. row(g): the
    // segment's first row in memory, negative when the whole segment is past the operand (it is
    // not loaded: its results are dropped). Pieces at or past K read as zero.
    template <int kSegs, int kAuxBits, class Row>
    __device__ __forceinline__ void issue(__amdgpu_buffer_rsrc_t r, unsigned char *buf, int s, Row row) const {
        const int l = here(), pc = ((l & 7) ^ (l >> 4)) * 16, left = p.K - s * kSlabB;
        const uint32_t at = (uint32_t)(l >> 3) * p.K;
        const uint32_t even = pc < left ? at + pc : kFar, odd = (pc ^ 64) < left ? at + (pc ^ 64) : kFar;
#pragma unroll
        for (int a = 0; a < kSegs; ++a) {
            const int g = kSegs * wave + a, first = row(g);
            if (kDeep || first >= 0)  // uniform; the deep form counts its loads, past the operand they read zero
                to_lds16<kAuxBits>(r, buf + g * 1024, (g & 1 ? odd : even) + (uint32_t)(first * p.K + s * kSlabB));
        }
    }
    __device__ __forceinline__ void issue_x(const Unit &u, unsigned char *xb, int s) const {
        const __amdgpu_buffer_rsrc_t r =
            buffer_rsrc(p.x + (size_t)u.t.start * p.K, (uint32_t)u.t.n * (uint32_t)p.K);
        issue<kXSegs, 0>(r, xb, s, [&](int g) { return kDeep || 8 * g < u.t.n ? 8 * g : -1; });
    }
    __device__ __forceinline__ void issue_w(const Unit &u, unsigned char *wb, int s) const {
        const __amdgpu_buffer_rsrc_t r =
            buffer_rsrc(p.w + ((size_t)u.t.e * p.M + u.m0) * p.K, (uint32_t)(p.M - u.m0) * (uint32_t)p.K);
        issue<kWSegs, kAux>(r, wb, s, [&](int g) {
            const int c = channel(8 * g);
            return kDeep || c < p.M - u.m0 ? c : -1;
        });
    }
    // 64 scales per load: waves 0..4 those of the rows, waves 4..7 those of the weight rows
    __device__ __forceinline__ void issue_scales(const Unit &u, float *to) const {
        const int i = 64 * wave + here();
        if (wave < kBRows / 64)
            to_lds4(buffer_rsrc(p.x_scale + u.t.start, (uint32_t)u.t.n * 4), to + 64 * wave, i * 4);
        if (wave >= 4) {
            const int R = i - 256;
            to_lds4(buffer_rsrc(p.w_scale + (size_t)u.t.e * p.M + u.m0, (uint32_t)(p.M - u.m0) * 4),
                         to + kBRows + 64 * (wave - 4), (uint32_t)channel(R) * 4);
        }
    }
    // A block barrier that leaves loads in flight. kRead: after this wave's LDS reads have returned
    // (what they read may be overwritten); kLoads: after its loads, all but the youngest kYoung, have
    // landed in LDS.
    template <bool kRead, bool kLoads, int kYoung = 0>
    __device__ __forceinline__ void phase_end() const {
        static_assert(kYoung < 16, "the counter's low bits");
        if constexpr (kRead || kLoads)
            __builtin_amdgcn_s_waitcnt((kRead ? 0x0070 : 0x0F70) | (kLoads ? kYoung : 0xC00F));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
    }

    // The unit's products, scaled and stored; its slab 0 and scales are in LDS at entry. next() (if
    // more): the block's next unit, whose slab 0 and scales (to nscale) are requested on the way.
    template <int kN, class Next>
    __device__ __forceinline__ void run(const Unit &u, Next next, bool more, const float *scale,
                                        float *nscale) const {
        i32x4_t acc[kBA][kN] = {};
        const bool busy = th * kN * kTile < u.t.n;  // uniform: the wave has rows
        uint4 a[kBA], b[kN];
        auto read = [&](const unsigned char *wb, const unsigned char *xb, int h) __attribute__((always_inline)) {
            if (!kDeep && !busy) return;
            const int l = here(), rd = spos(l & 15, l >> 4);
#pragma unroll
            for (int i = 0; i < kBA; ++i) a[i] = load16(wb + (ch * kBA + i) * kTile * kSlabB + (rd ^ 64 * h));
#pragma unroll
            for (int j = 0; j < kN; ++j) b[j] = load16(xb + (th * kN + j) * kTile * kSlabB + (rd ^ 64 * h));
        };
        auto mult = [&]() __attribute__((always_inline)) {
            if (!kDeep && !busy) return;
#pragma unroll
            for (int j = 0; j < kN; ++j)
#pragma unroll
                for (int i = 0; i < kBA; ++i) mma_i8(acc[i][j], a[i], b[j]);
        };
        // A slab in four phases (operands of each half, products of each half) that the waves of the
        // second half of the block go through one phase later. refill() requests what comes into
        // the slab's buffer next: after the phase in which the later waves read its second half,
        // for both kinds of waves. The other buffer's loads were requested four phases earlier and
        // are waited for at the same place.
        auto slab = [&](auto late, const unsigned char *wb, const unsigned char *xb, bool there,
                        auto refill) __attribute__((always_inline)) {
            constexpr bool kLate = decltype(late)::value;
            if (there) read(wb, xb, 0);
            phase_end<true, false>();
            if (there) mult();
            phase_end<false, false>();
            if (there) read(wb, xb, 1);
            phase_end<true, kLate>();
            if (kLate) refill();
            if (there) mult();
            phase_end<false, !kLate>();
            if (!kLate) refill();
        };
        // The deep form: three buffers, two slabs ahead, a barrier per slab. Slab s of a turn of three
        // lies in buffer s % 3; in a unit's last turn the first two buffers take the next unit's
        // first slabs, the third is left for the results.
        auto deep = [&]() __attribute__((always_inline)) {
            constexpr int kLoads = kXSegs + kWSegs;  // loads of a slab
            issue_x(u, d_x2, 2);
            issue_w(u, d_w2, 2);
            Unit nxt = u;
            if (more) nxt = next();
            auto work = [&](const unsigned char *wb, const unsigned char *xb) __attribute__((always_inline)) {
                read(wb, xb, 0);
                mult();
                read(wb, xb, 1);
                mult();
            };
            auto fill = [&](const Unit &v, unsigned char *wb, unsigned char *xb, int s, bool any)
                            __attribute__((always_inline)) {
                issue_x(v, xb, any ? s : nslab);  // (past K: zeros)
                issue_w(v, wb, any ? s : nslab);
            };
            int s = 0;
            for (; s + 3 < nslab; s += 3) {
                work(d_w0, d_x0);
                phase_end<true, true, kLoads>();
                fill(u, d_w0, d_x0, s + 3, true);
                work(d_w1, d_x1);
                phase_end<true, true, kLoads>();
                fill(u, d_w1, d_x1, s + 4, true);
                work(d_w2, d_x2);
                phase_end<true, true, kLoads>();
                fill(u, d_w2, d_x2, s + 5, true);
            }
            work(d_w0, d_x0);
            phase_end<true, true, kLoads>();
            issue_scales(nxt, nscale);
            fill(nxt, d_w0, d_x0, 0, more);
            if (s + 1 < nslab) work(d_w1, d_x1);
            phase_end<true, true, kLoads>();
            fill(nxt, d_w1, d_x1, 1, more);
            if (s + 2 < nslab) work(d_w2, d_x2);
            phase_end<true, true, kLoads>();
        };
        auto slabs = [&](auto late) __attribute__((always_inline)) {
            constexpr bool kLate = decltype(late)::value;
            if (kLate) phase_end<false, false>();
            for (int s = 0; s < nslab; s += 2) {
                slab(late, b_w0, b_x0, true, [&]() __attribute__((always_inline)) {
                    if (s + 2 < nslab) {
                        issue_x(u, b_x0, s + 2);
                        issue_w(u, b_w0, s + 2);
                    } else if (more) {
                        const Unit nxt = next();  // (looked up here: registers)
                        issue_x(nxt, b_x0, 0);
                        issue_w(nxt, b_w0, 0);
                        issue_scales(nxt, nscale);
                    }
                });
                slab(late, b_w1, b_x1, s + 1 < nslab, [&]() __attribute__((always_inline)) {
                    if (s + 3 < nslab) {
                        issue_x(u, b_x1, s + 3);
                        issue_w(u, b_w1, s + 3);
                    }
                });
            }
            if (!kLate) phase_end<false, false>();  // both kinds end together
        };
        // the deep form takes its scales to registers here: later the next unit's are on their way
        float sxs[kN], sws[kBA][4];
        if constexpr (kDeep) {
            const int l = here();
#pragma unroll
            for (int j = 0; j < kN; ++j) sxs[j] = scale[(th * kN + j) * kTile + (l & 15)];
#pragma unroll
            for (int i = 0; i < kBA; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) sws[i][r] = scale[kBRows + (ch * kBA + i) * kTile + 4 * (l >> 4) + r];
            deep();
        } else {
            if (1 < nslab) {
                issue_x(u, b_x1, 1);
                issue_w(u, b_w1, 1);
            }
            if (wave >= kBWaves / 2) slabs(std::true_type{});
            else slabs(std::false_type{});
        }
        // Results: the last weight buffer is free now, the next unit's first slab has landed. A wave
        // turns 16 rows at a time in its 4 KB of that buffer, so that rows leave in whole 16-byte
        // pieces, 256 bytes of a row side by side; pieces rotate by the row (no bank conflicts).
        if (busy) {
            constexpr int kOut = kSwiglu ? kBA / 2 : kBA;                  // output subtiles per wave
            constexpr int kPart = 4096 / (kTile * (int)sizeof(O)) / kTile; // subtiles per turn of 4 KB
            constexpr int kSub = kOut < kPart ? kOut : kPart;
            constexpr int kRowB = kSub * kTile * (int)sizeof(O);           // bytes of a row per turn
            constexpr int kPcs = kRowB / 16;                               // 16-byte pieces of it
            const int l = here();
            const int lc = l & 15, lq = l >> 4;
            unsigned char *stage = (kDeep ? d_w2 : b_w1) + wave * 4096;
            const float *sw = scale + kBRows + ch * kBA * kTile + 4 * lq;
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const int n0 = (th * kN + j) * kTile;
                const float sx = kDeep ? sxs[j] : scale[n0 + lc];
#pragma unroll
                for (int i0 = 0; i0 < kOut; i0 += kSub) {
#pragma unroll
                    for (int i = i0; i < i0 + kSub; ++i) {
                        float z[4];
                        scaled(acc[i][j], sx, kDeep ? sws[i] : sw + i * kTile, z);
                        if constexpr (kSwiglu) {
                            float up[4];
                            scaled(acc[kOut + i][j], sx, kDeep ? sws[kOut + i] : sw + (kOut + i) * kTile, up);
                            swiglu4(z, up);
                        }
                        const int at = ((i - i0) * kTile + 4 * lq) * (int)sizeof(O);
                        store4(reinterpret_cast<O *>(stage + lc * kRowB +
                                                     (((at >> 4) ^ lc) & (kPcs - 1)) * 16 + (at & 15)),
                               z);
                    }
                    wave_exchange();
#pragma unroll
                    for (int g = 0; g < kTile * kPcs / kWave; ++g) {
                        const int r = (g * kWave + l) / kPcs, pc = l & (kPcs - 1);
                        const int m = u.m0 + (ch * kOut + i0) * kTile + pc * 16 / (int)sizeof(O);
                        const uint4 v = load16(stage + r * kRowB + ((pc ^ r) & (kPcs - 1)) * 16);
                        if (n0 + r < u.t.n && m < Mo)
                            *reinterpret_cast<uint4 *>(reinterpret_cast<O *>(p.y) +
                                                       (size_t)(u.t.start + n0 + r) * Mo + m) = v;
                    }
                    wave_exchange();
                }
            }
        }
        phase_end<true, false>();  // the last buffers may be filled again
    }
};

// kOnce (by expert): the tiles that read an expert's weights run side by side, mostly there is one:
// the weights are streamed past the caches. Otherwise (one matrix) the units of a group of kGroup
// row tiles run channel block by channel block, so that the 32 CUs of an XCD work on a near-square
// patch and share both operands in L2.
constexpr int kGroup = 4;
template <bool kSwiglu, class O, bool kOnce, bool kDeep>
__global__ __launch_bounds__(kBWaves *kWave) __attribute__((amdgpu_waves_per_eu(2, 2))) void i8_block_kernel(
    I8Params p) {
    using B = BlockProduct<kSwiglu, O, kOnce, kDeep>;
    const B b(p);
    const int S = (b.Mo + B::kCols - 1) / B::kCols;
    int tiles = (p.n_rows + p.tile_rows - 1) / p.tile_rows;
    if (p.offsets) {
        const TileScan sc = scan_tiles(p.offsets, p.E, p.n_rows, p.tile_rows);
        tiles = sc.total;
        if (threadIdx.x < kWave) b_scan[threadIdx.x] = sc;
        __syncthreads();
    }
    // blocks b, b + 8, ... run on one XCD and share one contiguous eighth of the units, in order
    const int units = tiles * S, per = (units + kXcds - 1) / kXcds;
    const int first = (blockIdx.x % kXcds) * per, last = min(first + per, units);
    auto unit = [&](int i) __attribute__((always_inline)) {
        if (p.offsets) {
            const int l = b.here();
            return pick_unit(b_scan[l], l, i, S, B::kCols);
        }
        const int g = i / (kGroup * S), in = i - g * kGroup * S, h = min(kGroup, tiles - g * kGroup);
        const int c = in / h, ti = g * kGroup + in - c * h;
        return Unit{{0, ti * p.tile_rows, min(p.tile_rows, p.n_rows - ti * p.tile_rows)}, c * B::kCols};
    };
    const int step = gridDim.x / kXcds;
    int i = first + blockIdx.x / kXcds;
    if (i >= last) return;  // uniform
    Unit u = unit(i);
    b.issue_scales(u, b_scale[0]);
    b.issue_x(u, kDeep ? d_x0 : b_x0, 0);
    b.issue_w(u, kDeep ? d_w0 : b_w0, 0);
    if constexpr (kDeep) {
        b.issue_x(u, d_x1, 1);
        b.issue_w(u, d_w1, 1);
    }
    b.template phase_end<true, true, kDeep ? B::kXSegs + kWSegs : 0>();
    for (int par = 0;; par ^= 1) {
        i += step;
        const bool more = i < last;
        auto next = [&]() __attribute__((always_inline)) { return unit(i); };
        const int sub = (u.t.n + 4 * kTile - 1) / (4 * kTile);  // row subtiles per wave
        const float *scale = b_scale[par];
        float *nscale = b_scale[par ^ 1];
        if (sub == 1) b.template run<1>(u, next, more, scale, nscale);
        else if (kDeep || sub == 2) b.template run<2>(u, next, more, scale, nscale);
        else if constexpr (kDeep) return;  // (not reached)
        else if (sub == 3) b.template run<3>(u, next, more, scale, nscale);
        else if (sub == 4) b.template run<4>(u, next, more, scale, nscale);
        else b.template run<5>(u, next, more, scale, nscale);
        if (!more) break;
        u = next();
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // no load into this block's LDS outlives it
}

// ------------------------------------------------------------------------- few rows per expert
// With a few rows per expert the time is the one read of the weights. A wave takes up to 16 kNB
// rows of one expert and 32 weight channels (with SwiGLU 16 gate and the matching 16 up channels)
// and streams the channels in slabs of 128 bytes, whole cache lines loaded straight into its own
// ring of kRing slab buffers: neither registers nor a block barrier hold the stream back. The
// rows come through buffer loads into registers in operand order; rows past the tile's read as
// zero without a memory access, so one or two rows cost one or two lines per step.
// Ten one-wave blocks fill a CU's LDS. They are persistent: a wave walks its units, and the ring
// takes the next unit's first slabs while the last slabs and the results of the present one are
// worked on, so that the stream does not stop between them.
// kKS waves make a block and split K between them (their integer sums join in LDS, exact in any
// order) where there is so little to stream that single waves would not cover the chip; each such
// block takes one unit.
// Measured: 256 rows over about 163 of 256 experts of 2048 x 1024 with SwiGLU 53 us (331 MiB read, 6.5
// TB/s, the rate of reads alone; plain instead of non-temporal loads 63, slabs of half cache lines 65
// and more); one row of 4096 x 4096 7 us.
constexpr int kSCh = 32, kRing = 4;
constexpr int kSlabBytes = kSCh * kSlabB;  // one wave's slab (4 KB)
constexpr int kStreamBlocks = 10;          // one-wave blocks per CU

template <bool kSwiglu, class O, int kNB, int kKS>
__global__ __launch_bounds__(kKS *kWave) void i8_stream_kernel(I8Params p) {
    // one object per ring slot, so that the compiler can tell loads into one from reads of another
    __shared__ __align__(16) unsigned char ring0[kKS][kSlabBytes], ring1[kKS][kSlabBytes],
        ring2[kKS][kSlabBytes], ring3[kKS][kSlabBytes];
    constexpr int kCols = kSwiglu ? kSCh / 2 : kSCh;  // output channels of a block
    constexpr int kRows = kTile * kNB;
    constexpr bool kWalk = kKS == 1;
    const int lane = lane_id(), wave = kKS > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
    const int col = lane & 15, q = lane >> 4;
    auto slot = [&](auto ic) __attribute__((always_inline)) -> unsigned char * {
        constexpr int B = decltype(ic)::value;
        return B == 0 ? ring0[wave] : B == 1 ? ring1[wave] : B == 2 ? ring2[wave] : ring3[wave];
    };
    const int Mo = kSwiglu ? p.M / 2 : p.M;
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
        if (p.offsets) return pick_unit(sc, lane, i, S, kCols);
        const int ti = i / S;
        return Unit{{0, ti * kRows, min(kRows, p.n_rows - ti * kRows)}, (i - ti * S) * kCols};
    };
    // this wave's slabs: s0 .. s0 + share - 1, in whole turns of the ring
    const int nslab = (p.K + kSlabB - 1) / kSlabB;
    const int share = (nslab + kKS - 1) / kKS, s0 = wave * share;
    const int turns = (share + kRing - 1) / kRing * kRing;
    // segment a of a slab: staged rows 8a .. 8a + 7 (SwiGLU: rows 16 .. 31 are the up channels)
    uint32_t woff[kSCh / 8], xoff[kNB];
    int wk[kSCh / 8];
#pragma unroll
    for (int a = 0; a < kSCh / 8; ++a) {
        const int R = 8 * a + (lane >> 3), c = kSwiglu ? (R & 15) + (R >> 4) * Mo : R;
        wk[a] = (((lane & 7) ^ (R >> 1)) & 7) * 16;
        woff[a] = (uint32_t)c * p.K + wk[a];
    }
#pragma unroll
    for (int j = 0; j < kNB; ++j) xoff[j] = (uint32_t)(j * kTile + col) * p.K + q * 16;
    uint4 xr[kRing][kNB][2];
    // the wave's slab i of unit v: always the same number of loads (they are counted); pieces at or
    // past K, slabs past the share and units that do not exist (any = false) read as zero
    auto issue = [&](auto ic, const Unit &v, int i, bool any) __attribute__((always_inline)) {
        constexpr int B = decltype(ic)::value;
        const __amdgpu_buffer_rsrc_t rx =
            buffer_rsrc(p.x + (size_t)v.t.start * p.K, (uint32_t)v.t.n * (uint32_t)p.K);
        const __amdgpu_buffer_rsrc_t rw =
            buffer_rsrc(p.w + ((size_t)v.t.e * p.M + v.m0) * p.K, (uint32_t)(p.M - v.m0) * (uint32_t)p.K);
        const uint32_t k0 = (uint32_t)(s0 + i) * kSlabB;
        const int left = any && i < share ? p.K - (int)k0 : 0;  // bytes of K from this slab on
#pragma unroll
        for (int a = 0; a < kSCh / 8; ++a)
            to_lds16<kBufNT>(rw, slot(ic) + a * 1024, wk[a] < left ? woff[a] + k0 : kPast);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < kNB; ++j)
                xr[B][j][h] = __builtin_bit_cast(
                    uint4, __builtin_amdgcn_raw_buffer_load_b128(
                               rx, (int)((4 * h + q) * 16 < left ? xoff[j] + k0 + h * 64 : kPast), 0, 0));
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;
    // loads of the three younger slabs may be outstanding when a slab is used
    constexpr int kYoung = (kRing - 1) * (kSCh / 8 + 2 * kNB);
    static_assert(kYoung < 64, "vmcnt has six bits");
    constexpr int kWait = (kYoung & 15) | 0x0F70 | ((kYoung >> 4) << 14);

    Unit cur = unit(u);
    issue(I0{}, cur, 0, true);
    issue(I1{}, cur, 1, true);
    issue(I2{}, cur, 2, true);
    issue(I3{}, cur, 3, true);
    for (;;) {
        u += step;
        const bool more = kWalk && u < last;
        const Unit nxt = more ? unit(u) : cur;
        // the unit's scales, requested before its products: rows and channels past it read as zero
        // (their results are not stored)
        float sx[kNB], sw[2][4];
        {
            const __amdgpu_buffer_rsrc_t r = buffer_rsrc(p.x_scale + cur.t.start, (uint32_t)cur.t.n * 4);
            const __amdgpu_buffer_rsrc_t c =
                buffer_rsrc(p.w_scale + (size_t)cur.t.e * p.M + cur.m0, (uint32_t)(p.M - cur.m0) * 4);
#pragma unroll
            for (int j = 0; j < kNB; ++j) sx[j] = __uint_as_float(bload4(r, (uint32_t)(j * kTile + col) * 4));
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sw[i][k] = __uint_as_float(bload4(c, (uint32_t)(i * (kSwiglu ? Mo : kTile) + 4 * q + k) * 4));
        }
        i32x4_t acc[2][kNB] = {};
        auto turn = [&](auto ic, int i) __attribute__((always_inline)) {
            constexpr int B = decltype(ic)::value;
            __builtin_amdgcn_s_waitcnt(kWait);
            __builtin_amdgcn_sched_barrier(0);  // the loads counted above stay on their side of it
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 a[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) a[k] = load16(slot(ic) + k * kTile * kSlabB + spos(col, 4 * h + q));
#pragma unroll
                for (int j = 0; j < kNB; ++j)
#pragma unroll
                    for (int k = 0; k < 2; ++k) mma_i8(acc[k][j], a[k], xr[B][j][h]);
            }
            // The refill goes into the slot that was read: it is requested once the reads have returned
            // (one past K is answered without a memory access, so latency orders nothing).
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0xC07F);  // LDS reads: none outstanding; loads: not waited for
            __builtin_amdgcn_sched_barrier(0);
            const bool here = i + kRing < turns;  // uniform
            issue(ic, here ? cur : nxt, here ? i + kRing : i + kRing - turns, here || more);
        };
        int i = 0;
        do {
            turn(I0{}, i);
            turn(I1{}, i + 1);
            turn(I2{}, i + 2);
            turn(I3{}, i + 3);
        } while ((i += kRing) < turns);
        bool mine = true;
        if constexpr (kKS > 1) {  // join the waves' sums in wave 0
            __shared__ __align__(16) int red[kKS - 1][2][kNB][kWave][4];
            mine = wave == 0;
            if (!mine) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int j = 0; j < kNB; ++j)
                        *reinterpret_cast<i32x4_t *>(red[wave - 1][k][j][lane]) = acc[k][j];
            }
            __syncthreads();
            if (mine) {
#pragma unroll
                for (int w = 0; w < kKS - 1; ++w)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int j = 0; j < kNB; ++j)
                            acc[k][j] += *reinterpret_cast<const i32x4_t *>(red[w][k][j][lane]);
            }
        }
        if (mine) {
#pragma unroll
            for (int j = 0; j < kNB; ++j) {
                const int n = j * kTile + col;
                if (n >= cur.t.n) continue;
                O *y = reinterpret_cast<O *>(p.y) + (size_t)(cur.t.start + n) * Mo;
#pragma unroll
                for (int k = 0; k < (kSwiglu ? 1 : 2); ++k) {
                    const int mc = cur.m0 + k * kTile + 4 * q;
                    if (mc >= Mo) continue;  // Mo is a multiple of 8: four channels are all in or all out
                    float z[4];
                    scaled(acc[k][j], sx[j], sw[k], z);
                    if constexpr (kSwiglu) {
                        float up[4];
                        scaled(acc[1][j], sx[j], sw[1], up);
                        swiglu4(z, up);
                    }
                    store4(y + mc, z);
                }
            }
        }
        if (!more) break;
        cur = nxt;
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // no load into this block's LDS outlives it
}

}  // namespace

namespace {

// CUs of the current device (looked up once per device).
int num_cus() {
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

// The most row tiles of `per` rows that n_rows rows of E experts can make.
long most_tiles(const I8Params &p, int per) {
    if (!p.offsets) return (p.n_rows + per - 1) / per;
    const long parts = p.n_rows / per + (p.E < p.n_rows ? p.E : p.n_rows);
    return parts < p.n_rows ? parts : p.n_rows;
}

// About how many there will be: the experts' counts are on the device, so even routing is taken, and
// `more` of a tile more per expert once its rows come near a tile's. n_rows is the caller's capacity, so
// where an expert shard passes that of all pairs, an expert is taken to have as many rows more.
double likely_tiles(const I8Params &p, int per, double more) {
    if (!p.offsets) return (p.n_rows + per - 1) / per;
    const double experts = p.E < p.n_rows ? p.E : p.n_rows, each = p.n_rows / experts / per;
    return experts * (each + more > 1.0 ? each + more : 1.0);
}

// Which kernel, and how it is cut, from estimates of all in us. The constants are rates measured on
// MI355X. Stream waves take their weights and rows in at 8.5 TB/s in all, with a start and end worth
// 3 KB each. HBM gives 6.4 TB/s to those of 16 rows, 6.1 to those of 32 and to the deep block form,
// 5.2 to the wide one, and an expert's weights are read once per tile. A slab of a block costs 0.33 us and 5.5 ns a row, at
// least 0.78 (deep) or 1.2 (wide); a unit's end 3 or 2 us and its results' stores.
// Measured where the choice turns (us; 16-row waves, 32-row waves, deep, wide): 256 experts of 2048 x
// 1024 with SwiGLU, even routing, 6 rows an expert: 83, 85, 87, 97; 8 rows: 84, 88, 89, 99; 12 rows:
// 96, 91, 90, 99; 31 rows: 184, 149, 94, 110; 94 rows: deep 115, wide 124; 144 rows: 199, 140. The same
// with skewed routing, where hot experts have many tiles: 49, 47, 44, 54; 57, 55, 45, 55; 75, 68, 48,
// 64; 142, 120, 67, 91; 112, 125; 153, 149. Dense 4096 x 4096, 128 rows: 27, 16, 27, 41; 256 rows: 47,
// 31, 27, 42; 2048 rows: deep 41, wide 48; 4096 rows: 76, 64.
struct Choice {
    bool block;
    int row_tiles, k_split, tile_rows;  // stream: 16-row tiles per wave, waves per block; block: rows
};
Choice choose(const I8Params &p, bool swiglu, int out_bytes, int cus) {
    const int Mo = swiglu ? p.M / 2 : p.M, nslab = (p.K + kSlabB - 1) / kSlabB;
    const double experts = p.offsets ? (p.E < p.n_rows ? p.E : p.n_rows) : 1;
    const double weights = (double)p.M * p.K, rows = p.n_rows / experts;
    const double others = (double)p.n_rows * (p.K + (double)Mo * out_bytes);
    auto most = [](double a, double b) { return a > b ? a : b; };
    auto least = [](double a, double b) { return a < b ? a : b; };
    Choice c{true, 1, 1, kBRows};
    double best = 0;
    const int cols = swiglu ? kBCh / 2 : kBCh, S = (Mo + cols - 1) / cols;
    // dense: the row tile whose rounds over the CUs take least; by expert: the largest of either form
    for (int r = p.offsets ? kDeepRows : 64; r <= kBRows; r += p.offsets ? kBRows - kDeepRows : 64) {
        const bool deep = r <= kDeepRows;
        const double tiles = likely_tiles(p, r, 0.35), n = least(rows, r);
        const double unit = nslab * most(deep ? 0.78 : 1.2, 0.33 + 0.0055 * n) + (deep ? 3.0 : 2.0) +
                            n * cols * out_bytes / 22e3;
        const double reads = (p.offsets ? tiles : 1.0) * weights + others;
        const double us = most(ceil(tiles * S / cus) * unit, reads / (deep ? 6.1e6 : 5.2e6));
        if (best == 0 || us <= best) best = us, c.tile_rows = r;
    }
    const int scols = swiglu ? kSCh / 2 : kSCh, SS = (Mo + scols - 1) / scols;
    for (int nb = 1; nb <= 2; ++nb) {
        const double waves = likely_tiles(p, nb * kTile, nb == 1 ? 0.6 : 0.75) * SS;
        // fewer waves than CUs: their K is split four ways
        const int split = waves <= cus ? 4 : 1;
        const double us = most(waves * ((kSCh + least(rows, nb * kTile)) * p.K + 3000) / 8.5e6,
                               most((experts * weights + others) / (nb == 1 ? 6.4e6 : 6.1e6), 0.35 * nslab / split));
        if (us < best) best = us, c.block = false, c.row_tiles = nb, c.k_split = split;
    }
    return c;
}

}  // namespace

hipError_t launch_matmul_i8(const I8Params &p, bool swiglu, int y_dtype, hipStream_t s) {
    const int Mo = swiglu ? p.M / 2 : p.M, cus = num_cus();
    const Choice c = choose(p, swiglu, y_dtype == 0 ? 4 : 2, cus);
    // the output type and the epilogue
    auto typed = [&](auto go) {
        if (y_dtype == 0) swiglu ? go(float{}, std::true_type{}) : go(float{}, std::false_type{});
        else swiglu ? go(uint16_t{}, std::true_type{}) : go(uint16_t{}, std::false_type{});
    };
    if (c.block) {
        const int cols = swiglu ? kBCh / 2 : kBCh;
        const long units = most_tiles(p, c.tile_rows) * ((Mo + cols - 1) / cols);
        const unsigned grid = (unsigned)((units < cus ? units : cus) + kXcds - 1) / kXcds * kXcds;
        I8Params b = p;
        b.tile_rows = c.tile_rows;
        typed([&](auto o, auto glu) {
            using O = decltype(o);
            constexpr bool kGlu = decltype(glu)::value;
            const bool deep = c.tile_rows <= kDeepRows;
            if (p.offsets && deep) launch_k(i8_block_kernel<kGlu, O, true, true>, grid, kBWaves * kWave, 0, s, b);
            else if (p.offsets) launch_k(i8_block_kernel<kGlu, O, true, false>, grid, kBWaves * kWave, 0, s, b);
            else if (deep) launch_k(i8_block_kernel<kGlu, O, false, true>, grid, kBWaves * kWave, 0, s, b);
            else launch_k(i8_block_kernel<kGlu, O, false, false>, grid, kBWaves * kWave, 0, s, b);
        });
        return hipGetLastError();
    }
    const int cols = swiglu ? kSCh / 2 : kSCh;
    const long units = most_tiles(p, c.row_tiles * kTile) * ((Mo + cols - 1) / cols);
    // a wave walks units of about 64 KB of weights in all: shorter walks pay their starts too often
    // (512 x 2048, 2 rows an expert: 45 us for one unit a wave, 39 for four), longer ones even out
    // badly at the end (42 for eight); more only while the chip has no room for more waves. With K split
    // a block per unit: choose() splits only where there are at most twice as many as CUs
    const long walk = p.K < 2048 ? 2048 / p.K : 1, room = (long)cus * kStreamBlocks;
    const long blocks = units <= room || c.k_split > 1 ? units : (units + walk - 1) / walk > room ? (units + walk - 1) / walk : room;
    const unsigned grid = (unsigned)((blocks + kXcds - 1) / kXcds * kXcds);
    typed([&](auto o, auto glu) {
        using O = decltype(o);
        constexpr bool kGlu = decltype(glu)::value;
        if (c.row_tiles == 1 && c.k_split == 1) launch_k(i8_stream_kernel<kGlu, O, 1, 1>, grid, kWave, 0, s, p);
        else if (c.row_tiles == 1) launch_k(i8_stream_kernel<kGlu, O, 1, 4>, grid, 4 * kWave, 0, s, p);
        else if (c.k_split == 1) launch_k(i8_stream_kernel<kGlu, O, 2, 1>, grid, kWave, 0, s, p);
        else launch_k(i8_stream_kernel<kGlu, O, 2, 4>, grid, 4 * kWave, 0, s, p);
    });
    return hipGetLastError();
}

}  // namespace moe
