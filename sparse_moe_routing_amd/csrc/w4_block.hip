// w4_block.hip - products with 4-bit weights for many rows (w4.hip has the arithmetic and the forms for
// few).
//
// A block multiplies up to 256 rows of one expert by 256 weight channels (with SwiGLU 128 gate channels
// and the 128 up channels that go with them). Rows are staged in LDS in slabs of 128 bytes a row, codes
// in slabs of 128 bytes a channel (four of the rows' slabs in bf16, eight in fp32), whole cache lines loaded
// straight into LDS, both double-buffered; the codes are turned into operands by the wave that
// multiplies them, on their way from LDS to the registers, so that LDS carries them as 4 bits. Eight waves,
// two per SIMD: wave w takes the channels of half w % 2 and a quarter of the tile's 16-row subtiles, at
// most four.
//
// The blocks are persistent, one per CU: the last slab of a unit is multiplied, and its results are stored,
// while the first slabs of the block's next unit load.
#include <math.h>

#include "w4_core.h"

namespace moe {

namespace {

constexpr int kBWaves = 8;
constexpr int kBRows = 256, kBCh = 256;      // rows and weight channels of a block
constexpr int kBA = kBCh / 2 / kTile;        // channel subtiles of a wave
constexpr int kBXSegs = kBRows / 8 / kBWaves;  // 1 KB segments of rows per wave and slab

template <class X, bool kSwiglu, bool kGen>
struct W4Block {
    using F = Form<X>;
    static constexpr int kCols = kSwiglu ? kBCh / 2 : kBCh;     // output channels
    static constexpr int kXK = kSlabB / (int)sizeof(X);         // columns of a slab of rows
    static constexpr int kXS = kXK / kStepK;                    // its steps
    static constexpr int kSub = kSlabK / kXK;                   // slabs of rows per slab of codes
    static constexpr int kGroupB = kGen ? 4 * kBCh : 2 * kBCh;  // bytes of a group's scales
    static constexpr int kScaleB = 8 * kGroupB, kZeroB = kGen ? 8 * kBCh : 0;

    const W4Params &p;
    F form;
    int lane, wave, ch, th, Mo, KB, gl, groups, slabg, sb;
    int nslab, nsuper;  // slabs of rows and of codes in K

    __device__ __forceinline__ W4Block(const W4Params &p_) : p(p_) {
        lane = lane_id();
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        ch = wave & 1;
        th = wave >> 1;
        Mo = kSwiglu ? p.M / 2 : p.M;
        KB = p.K / 2;
        gl = p.group == 128 ? 2 : p.group == 64 ? 1 : 0;
        groups = p.K / p.group;
        slabg = 8 >> gl;
        sb = kGen && p.scale_f32 ? 4 : 2;
        nslab = (p.K + kXK - 1) / kXK;
        nsuper = (p.K + kSlabK - 1) / kSlabK;
    }
    // The lane number, made anew: what is computed from it stays next to its use instead of in registers
    // across the products, which need them all.
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
    // Slab s of a unit's rows: segment g holds rows 8g .. 8g + 7; segments past the tile are not loaded.
    __device__ __forceinline__ void issue_x(const Unit &u, unsigned char *buf, int s) const {
        const int l = here(), XB = p.K * (int)sizeof(X), pc = ((l & 7) ^ (l >> 4)) * 16, left = XB - s * kSlabB;
        const __amdgpu_buffer_rsrc_t r = buffer_rsrc(reinterpret_cast<const unsigned char *>(p.x) + (size_t)u.t.start * XB,
                                                     (uint32_t)u.t.n * (uint32_t)XB);
        const uint32_t at = (uint32_t)(l >> 3) * XB + (uint32_t)s * kSlabB;
        // (even and odd segments rotate differently; pieces past K read as zero)
        const uint32_t even = pc < left ? at + pc : 0x80000000u, odd = (pc ^ 64) < left ? at + (pc ^ 64) : 0x80000000u;
#pragma unroll
        for (int a = 0; a < kBXSegs; ++a) {
            const int g = kBXSegs * wave + a;
            if (8 * g < u.t.n) to_lds16<0>(r, buf + g * 1024, (g & 1 ? odd : even) + (uint32_t)(8 * g) * XB);
        }
    }
    // Quarter h of slab S of a unit's codes: one segment of eight channels per wave.
    __device__ __forceinline__ void issue_c(const Unit &u, unsigned char *buf, int S, int h) const {
        const int l = here(), g = 8 * h + wave, left = KB - S * kSlabB;
        const int pc = ((l & 7) ^ (l >> 4) ^ (g & 1 ? 4 : 0)) * 16;
        const __amdgpu_buffer_rsrc_t r =
            buffer_rsrc(p.w + ((size_t)u.t.e * p.M + u.m0) * KB, (uint32_t)(p.M - u.m0) * (uint32_t)KB);
        const uint32_t at = (uint32_t)(channel(8 * g) + (l >> 3)) * KB + (uint32_t)S * kSlabB + pc;
        to_lds16<0>(r, buf + g * 1024, pc < left ? at : kPast);
    }
    // The scales and zero points of slab S of the codes: [group][staged row].
    __device__ __forceinline__ void issue_s(const Unit &u, unsigned char *sbuf, unsigned char *zbuf, int S) const {
        const int l = here();
        const size_t at = (size_t)u.t.e * groups * p.M + u.m0;
        const uint32_t n = (uint32_t)groups * (uint32_t)p.M - (uint32_t)u.m0;
        const __amdgpu_buffer_rsrc_t r = buffer_rsrc(reinterpret_cast<const unsigned char *>(p.scale) + at * sb, n * sb);
        if constexpr (kGen) {  // a group per wave
            const int g = S * slabg + wave;
            const bool on = wave < slabg && g < groups;
            const int R = l * (16 / sb);
            to_lds16<0>(r, sbuf + wave * kGroupB, on && R < kBCh ? (uint32_t)(g * p.M + channel(R)) * sb : kPast);
            to_lds4(buffer_rsrc(p.zero + (p.zero ? at : 0), p.zero ? n : 0u), zbuf + wave * kBCh,
                    on ? (uint32_t)(g * p.M + channel(4 * l)) : kPast);
        } else if (wave < 4) {  // two groups per wave
            const int in = 2 * wave + (l >> 5), g = S * slabg + in;
            to_lds16<0>(r, sbuf + wave * 1024, in < slabg && g < groups ? (uint32_t)(g * p.M + channel((l & 31) * 8)) * 2 : kPast);
        }
    }
    // A block barrier; the wave's loads have landed and its LDS reads have returned.
    __device__ __forceinline__ void top() const {
        __builtin_amdgcn_s_waitcnt(0x0070);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
    }
    // A staged scale, as read and as a number.
    __device__ __forceinline__ uint32_t scale_bits(const unsigned char *sbuf, int g, int R) const {
        if constexpr (kGen) return *reinterpret_cast<const uint32_t *>(sbuf + g * kGroupB + (R * sb & ~3));
        else return *reinterpret_cast<const uint16_t *>(sbuf + g * kGroupB + R * 2);
    }
    __device__ __forceinline__ float scale_of(uint32_t bits, int R) const {
        if constexpr (kGen) return __uint_as_float(sb == 4 ? bits : (R & 1) ? bits & 0xFFFF0000u : bits << 16);
        else return bf16_bits_to_f32(bits);
    }

    // The products of slab h of the slab of codes in cb with the slab of rows in xb. kFlush: steps that
    // share a scale (at most those of a slab of rows).
    template <int kN, int kFlush>
    __device__ __forceinline__ void slab(f32x4_t (&acc)[kBA][kN], const unsigned char *xb, const unsigned char *cb,
                                         const unsigned char *sbuf, const unsigned char *zbuf, int h) const {
        constexpr int kGroups = kXS / kFlush;  // groups of a slab of rows
        constexpr bool kMinus = kGen || F::kMinus24 != 0;
        constexpr int kVPerM = F::kParts == 3 ? 2 : 4;
        const int l = here(), col = l & 15, q = l >> 4;
        uint4 x[kN][kXS][F::kParts];
        f32x4_t rows[kN][kGroups];
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const unsigned char *row = xb + (th * kN + j) * kTile * kSlabB;
#pragma unroll
            for (int s = 0; s < kXS; ++s) {
                uint4 v[F::kPer];
#pragma unroll
                for (int i = 0; i < F::kPer; ++i) v[i] = F::order(load16(row + spos(col, (4 * s + q) * F::kPer + i)));
                F::parts(v, x[j][s]);
                if constexpr (kMinus) {
                    if (s % kFlush == 0) rows[j][s / kFlush] = f32x4_t{};
#pragma unroll
                    for (int i = 0; i < F::kParts; ++i)
                        mma(rows[j][s / kFlush], x[j][s][i], all(kGen ? F::kMinus : F::kMinus24));
                }
            }
        }
        const int R0 = ch * kBA * kTile + col, step = h * kXS;
        const float z_bias = (p.zero ? 0.0f : 8.0f) - F::kFrom;
        // A channel subtile's codes are read two subtiles ahead and made operands one ahead; a sum is scaled
        // just before its registers take the next one, kN matrix instructions after its last: so
        // the matrix instructions always have something beside them.
        struct Bits {
            uint32_t s[kGroups];
            int z[kGroups];
        };
        struct Scales {
            float s[kGroups], z[kGroups];
        };
        auto words = [&](int i, uint32_t (&w)[kXS]) __attribute__((always_inline)) {
#pragma unroll
            for (int s = 0; s < kXS; ++s)
                w[s] = *reinterpret_cast<const uint32_t *>(cb + (ch * kBA + i) * kTile * kSlabB + spos(col, step + s) + 4 * q);
        };
        auto bits = [&](int i, Bits &v) __attribute__((always_inline)) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int at = (step + g * kFlush) >> gl, R = R0 + i * kTile;
                v.s[g] = scale_bits(sbuf, at, R);
                v.z[g] = kGen ? (int)zbuf[at * kBCh + R] : 0;
            }
        };
        uint32_t w[2][kXS];
        Bits raw[2];
        Scales sc[2];
        uint4 ops[2][kXS];
        f32x4_t sum[kN];
        auto scaled = [&](int i, int g, int j) __attribute__((always_inline)) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float v = sum[j][r];
                acc[i][j][r] = fmaf(sc[i & 1].s[g], kGen ? fmaf(sc[i & 1].z[g], rows[j][g][r], v) : v, acc[i][j][r]);
            }
        };
        words(0, w[0]);
        words(1, w[1]);
        bits(0, raw[0]);
#pragma unroll
        for (int s = 0; s < kXS; ++s) ops[0][s] = form.codes(w[0][s]);
#pragma unroll
        for (int i = 0; i < kBA; ++i) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                sc[i & 1].s[g] = scale_of(raw[i & 1].s[g], col);
                sc[i & 1].z[g] = (float)raw[i & 1].z[g] + z_bias;
            }
            if (i + 1 < kBA) bits(i + 1, raw[(i + 1) & 1]);
            if (i + 2 < kBA) words(i + 2, w[i & 1]);
#pragma unroll
            for (int s = 0; s < kXS; ++s) {
                if (i + 1 < kBA && s == kXS - 1)
#pragma unroll
                    for (int s2 = 0; s2 < kXS; ++s2) ops[(i + 1) & 1][s2] = form.codes(w[(i + 1) & 1][s2]);
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    if (s % kFlush == 0) {
                        if (s > 0) scaled(i, s / kFlush - 1, j);
                        else if (i > 0) scaled(i - 1, kGroups - 1, j);
                        sum[j] = kMinus && !kGen ? rows[j][s / kFlush] : f32x4_t{};
                    }
#pragma unroll
                    for (int k = 0; k < F::kParts; ++k) mma(sum[j], x[j][s][k], ops[i & 1][s]);
                }
            }
            // their order: a few vector instructions before each matrix instruction
#pragma unroll
            for (int m = 0; m < kXS * kN * F::kParts; ++m) {
                __builtin_amdgcn_sched_group_barrier(0x002, kVPerM, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < kN; ++j) scaled(kBA - 1, kGroups - 1, j);
    }
};

template <class X, bool kSwiglu, bool kGen>
__global__ __launch_bounds__(kBWaves *kWave) __attribute__((amdgpu_waves_per_eu(2, 2))) void w4_block_kernel(W4Params p) {
    using B = W4Block<X, kSwiglu, kGen>;
    // The buffers are separate objects, so that the compiler can tell loads into one from reads of the other.
    __shared__ __align__(16) unsigned char x0[kBRows * kSlabB], x1[kBRows * kSlabB], c0[kBCh * kSlabB], c1[kBCh * kSlabB];
    __shared__ __align__(16) unsigned char s0[B::kScaleB], s1[B::kScaleB], z0[kGen ? B::kZeroB : 16], z1[kGen ? B::kZeroB : 16];
    // the scan of the row tiles, kept out of the registers of the products
    __shared__ TileScan scans[kWave];
    const B b(p);
    const int S = (b.Mo + B::kCols - 1) / B::kCols;
    int tiles = (p.n_rows + p.tile_rows - 1) / p.tile_rows;
    if (p.offsets) {
        const TileScan sc = scan_tiles(p.offsets, p.E, p.n_rows, p.tile_rows);
        tiles = sc.total;
        if (threadIdx.x < kWave) scans[threadIdx.x] = sc;
        __syncthreads();
    }
    // blocks b, b + 8, ... run on one XCD and share one contiguous eighth of the units, in order
    const int units = tiles * S, per = (units + kXcds - 1) / kXcds;
    const int first = (blockIdx.x % kXcds) * per, last = min(first + per, units), step = gridDim.x / kXcds;
    auto unit = [&](int i) __attribute__((always_inline)) {
        if (p.offsets) {
            const int l = b.here();
            return find_unit<16>(scans[l], l, i, S, B::kCols);
        }
        // dense: groups of four row tiles run channel block by channel block, so that the CUs of an XCD
        // work on a near-square patch and share both operands in L2
        constexpr int kGroup = 4;
        const int g = i / (kGroup * S), in = i - g * kGroup * S, h = min(kGroup, tiles - g * kGroup);
        const int c = in / h, ti = g * kGroup + in - c * h;
        return Unit{{0, ti * p.tile_rows, min(p.tile_rows, p.n_rows - ti * p.tile_rows)}, c * B::kCols};
    };
    int i = first + blockIdx.x / kXcds;
    if (i >= last) return;  // uniform
    Unit u = unit(i);
    b.issue_s(u, s0, z0, 0);
#pragma unroll
    for (int h = 0; h < 4; ++h) b.issue_c(u, c0, 0, h);
    b.issue_x(u, x0, 0);
    for (;;) {
        i += step;
        const bool more = i < last;
        const Unit nxt = more ? unit(i) : u;
        auto run = [&](auto nc, auto fc) __attribute__((always_inline)) {
            constexpr int kN = decltype(nc)::value, kFlush = decltype(fc)::value;
            f32x4_t acc[kBA][kN] = {};
            // One slab of codes (S, in cb) with its slabs of rows; the next slab of codes comes into ncb. Past
            // K nothing is multiplied, but the buffers take their turns, so that a unit starts with the
            // first of each.
            auto super = [&](int S, const unsigned char *cb, const unsigned char *sbuf, const unsigned char *zbuf,
                             unsigned char *ncb, unsigned char *nsb, unsigned char *nzb) __attribute__((always_inline)) {
                const bool end = S + 2 > b.nsuper && (S & 1);  // the unit's last slab of codes, or the turn behind it
                const bool load = !end || more;
                const Unit &nu = end ? nxt : u;
                const int nS = end ? 0 : S + 1;
                auto turn = [&](int h, const unsigned char *xb, unsigned char *nxb, bool close) __attribute__((always_inline)) {
                    const int s = S * B::kSub + h;
                    b.top();
                    if (h == 0 && load) b.issue_s(nu, nsb, nzb, nS);
                    // the next slab of rows: the unit's, or behind its last turn the next unit's first
                    if (!(close && end)) {
                        if (s + 1 < b.nslab) b.issue_x(u, nxb, s + 1);
                    } else if (more) {
                        b.issue_x(nxt, nxb, 0);
                    }
                    if (h < 4 && load) b.issue_c(nu, ncb, nS, h);
                    if (s < b.nslab && b.th * kN * kTile < u.t.n) b.template slab<kN, kFlush>(acc, xb, cb, sbuf, zbuf, h);
                };
                for (int h = 0; h < B::kSub; h += 2) {
                    turn(h, x0, x1, false);
                    turn(h + 1, x1, x0, h + 2 == B::kSub);
                }
            };
            for (int S2 = 0; S2 < b.nsuper; S2 += 2) {
                super(S2, c0, s0, z0, c1, s1, z1);
                super(S2 + 1, c1, s1, z1, c0, s0, z0);
            }
            // results
            const int l = b.here(), col = l & 15, q = l >> 4;
            constexpr int kOut = kSwiglu ? kBA / 2 : kBA;
#pragma unroll
            for (int j = 0; j < kN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int n = (b.th * kN + j) * kTile + 4 * q + r;
                    if (n >= u.t.n) continue;
#pragma unroll
                    for (int a = 0; a < kOut; ++a) {
                        const int m = u.m0 + (b.ch * kOut + a) * kTile + col;
                        if (m >= b.Mo) continue;
                        float z = acc[a][j][r] / B::F::kUnit;
                        if constexpr (kSwiglu) z = (z < kFarGate ? silu_far(z) : silu(z)) * (acc[kOut + a][j][r] / B::F::kUnit);
                        const size_t at = (size_t)(u.t.start + n) * b.Mo + m;
                        if (p.y_f32) reinterpret_cast<float *>(p.y)[at] = z;
                        else reinterpret_cast<uint16_t *>(p.y)[at] = (uint16_t)(pack_bf16(z, 0.0f) & 0xFFFFu);
                    }
                }
        };
        auto sized = [&](auto fc) __attribute__((always_inline)) {
            const int sub = (u.t.n + 4 * kTile - 1) / (4 * kTile);  // row subtiles per wave
            if (sub == 1) run(std::integral_constant<int, 1>{}, fc);
            else if (sub == 2) run(std::integral_constant<int, 2>{}, fc);
            else if (sub == 3) run(std::integral_constant<int, 3>{}, fc);
            else run(std::integral_constant<int, 4>{}, fc);
        };
        if constexpr (B::kXS > 1) {
            if (b.gl > 0) sized(std::integral_constant<int, 2>{});
            else sized(std::integral_constant<int, 1>{});
        } else {
            sized(std::integral_constant<int, 1>{});
        }
        if (!more) break;
        u = nxt;
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // no load into this block's LDS outlives it
}

}  // namespace

hipError_t launch_w4_block(const W4Params &p, int x_dtype, bool swiglu, hipStream_t s) {
    const int cus = num_cus(), Mo = swiglu ? p.M / 2 : p.M, cols = swiglu ? kBCh / 2 : kBCh;
    const long units = most_tiles(p, p.tile_rows) * ((Mo + cols - 1) / cols);
    const unsigned grid = (unsigned)((units < cus ? units : cus) + kXcds - 1) / kXcds * kXcds;
    const bool gen = p.zero || p.scale_f32;
    auto go = [&](auto x) {
        using X = decltype(x);
        if (gen && swiglu) launch_k(w4_block_kernel<X, true, true>, grid, kBWaves * kWave, 0, s, p);
        else if (gen) launch_k(w4_block_kernel<X, false, true>, grid, kBWaves * kWave, 0, s, p);
        else if (swiglu) launch_k(w4_block_kernel<X, true, false>, grid, kBWaves * kWave, 0, s, p);
        else launch_k(w4_block_kernel<X, false, false>, grid, kBWaves * kWave, 0, s, p);
    };
    if (x_dtype == 0) go(float{});
    else go(uint16_t{});
    return hipGetLastError();
}

}  // namespace moe
