// w4_block.h - products with 4-bit weights for many rows (w4.hip has the arithmetic and the forms for
// few).
//
// A block multiplies the rows of one expert, up to 256 of them, by 256 weight channels (with SwiGLU 128 gate
// channels and the 128 up channels that go with them), 64 columns at a time: a slab. Rows are loaded
// straight into LDS, whole cache lines, double-buffered. Codes come to registers, whole cache lines of
// four slabs at once, and each wave turns an eighth of a slab's into operands, which it puts into LDS for
// all of them while the slab before is multiplied: every code is converted once per block.
// Eight waves, two per SIMD: wave w takes the channels of half w % 2 and a quarter of the tile's 16-row
// subtiles, at most kMaxN.
//
// Nothing is rounded on the way to the sums: an operand is the whole number code - zero (that / 16 without zero
// points), and each group's sums are scaled in fp32, so that a row's results are as exact here as in the forms
// for few rows. (Scales rounded into bf16 operands let the sums stay in the matrix instructions over all of K
// and 320 rows fit a block: 257 us in place of the 281 below, 332 in place of the 475. But that moved a bf16
// result by up to 2^-8 sum |x w|, and only where many rows came with it: 0.0026 of the norm after SwiGLU
// in place of 0.0017.)
//
// Instructions bound it: a SIMD takes two vector instructions beside each matrix instruction of 16 cycles
// for nothing, and every further one costs nearly its own time. With groups of 64 or more the scaling is two
// for each matrix instruction (four rows of a channel, two steps), the conversion comes on top. Up to 256 rows, 192
// with zero points or fp32 scales, 128 of fp32 rows: what the registers hold.
// Measured (us): 8192 x 4096 x 4096 with the codes turned over by each multiplying wave 318, with one
// conversion a block 281 to 304 (of 281, by leaving work out: 234 without the loads of the rows, 261 without those of
// the codes, 247 without the conversion, 189 without all three). 65536 rows over 256 experts of 2048 x 1024 with
// SwiGLU 470 to 480. 8192 x 4096 x 4096 with zero points 419; of fp32 rows (three products for one: the floor is
// three times as high) 700, with zero points and fp32 scales 765.
//
// The blocks are persistent, one per CU: the last slab of a unit is multiplied, and its results are stored,
// while the first slabs of the block's next unit load.
#pragma once

#include <math.h>

#include "w4_core.h"

namespace moe {

namespace {

constexpr int kBWaves = 8;
constexpr int kBCh = 256;              // weight channels of a block
constexpr int kBA = kBCh / 2 / kTile;  // channel subtiles of a wave
constexpr int kBK = 64;                // columns of a slab
constexpr int kBS = kBK / kStepK;      // its steps

template <class X, bool kGen>
struct W4Block {
    using F = Form<X>;
    static constexpr int kPer = F::kPer;                        // 128-byte pieces of a row in a slab
    // row subtiles of a wave and rows of a block (registers: products with zero points need most)
    static constexpr int kRows = w4_block_rows(kPer > 1, kGen), kMaxN = kRows / (4 * kTile);
    static constexpr int kSub = 4, kLineB = kSub * kBK / 2;     // slabs whose codes a wave loads at once: a cache line's
    static constexpr int kXSegs = kRows / 8 / kBWaves;          // 1 KB segments of rows per wave and piece
    static constexpr int kGroupB = kGen ? 4 * kBCh : 2 * kBCh;  // bytes of a group's scales
    static constexpr int kPairGroups = 4;                       // most groups of two slabs
    static constexpr int kScaleB = kPairGroups * kGroupB;
    static constexpr float kUnit = kGen ? 1.0f : 1.0f / 16.0f;  // of a code in the operands

    const W4Params &p;
    int lane, wave, ch, th, cols, Mo, KB, gl, groups, sb;  // cols: output channels of a block
    int nslab, nsuper;  // slabs, and slabs of whole lines of codes, in K

    __device__ __forceinline__ W4Block(const W4Params &p_) : p(p_) {
        lane = lane_id();
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        ch = wave & 1;
        th = wave >> 1;
        cols = p.swiglu ? kBCh / 2 : kBCh;
        Mo = p.swiglu ? p.M / 2 : p.M;
        KB = p.K / 2;
        gl = p.group == 128 ? 2 : p.group == 64 ? 1 : 0;
        groups = p.K / p.group;
        sb = kGen && p.scale_f32 ? 4 : 2;
        nslab = (p.K + kBK - 1) / kBK;
        nsuper = (p.K + kSub * kBK - 1) / (kSub * kBK);
    }
    // The lane number, made anew: what is computed from it stays next to its use instead of in registers
    // across the products, which need them all.
    __device__ __forceinline__ int here() const {
        int l = lane;
        asm volatile("" : "+v"(l));
        return l;
    }
    // Where the lane reads operands of a subtile's first step (the second: ^ 64), and where its own come in.
    __device__ __forceinline__ int read_at() const {
        const int l = here();
        return spos(l & 15, l >> 4);
    }
    __device__ __forceinline__ int made_at() const {
        const int l = here();
        return spos(32 * wave + (l >> 1), 4 * (l & 1));
    }
    // weight channel (past m0) of staged row R; SwiGLU: each half of 128 staged rows holds 64 gate
    // channels, then the 64 matching up channels
    __device__ __forceinline__ int channel(int R) const {
        return p.swiglu ? (R >> 7) * 64 + (R & 63) + ((R >> 6) & 1) * Mo : R;
    }
    // Slab s of a unit's rows (any: there is one): segment g holds rows 8g .. 8g + 7; a wave takes kSegs of them,
    // every eighth. Rows past the tile and pieces past K read as zero without a memory access. Even and odd
    // segments rotate differently.
    template <int kSegs>
    __device__ __forceinline__ void issue_x(const Unit &u, unsigned char *buf, int s, bool any) const {
        const int l = here(), XB = p.K * (int)sizeof(X), pc = ((l & 7) ^ (l >> 4)) * 16;
#pragma unroll
        for (int h = 0; h < kPer; ++h) {
            const int from = (s * kPer + h) * kSlabB, left = any ? XB - from : 0;
            const __amdgpu_buffer_rsrc_t r = buffer_rsrc(reinterpret_cast<const unsigned char *>(p.x) + (size_t)u.t.start * XB + from,
                                                         left > 0 ? (uint32_t)(u.t.n * XB - from) : 0u);
            const uint32_t row = (uint32_t)(l >> 3) * XB;
            const int mine = pc ^ (wave & 1 ? 64 : 0);
            const uint32_t at = mine < left ? row + (uint32_t)mine : 0x80000000u;
#pragma unroll
            for (int a = 0; a < kSegs; ++a) {
                const int g = kBWaves * a + wave;
                to_lds16<0>(r, buf + (h * kRows / 8 + g) * 1024, at + (uint32_t)(8 * g) * XB);
            }
        }
    }
    // The codes of line S that this wave converts (staged row 32 wave + l / 2, 32 columns of each slab), with
    // their zero points.
    struct Codes {
        uint4 c;
        uint32_t z;
    };
    __device__ __forceinline__ void issue_c(const Unit &u, Codes (&c)[kSub], int S) const {
        const int l = here(), left = KB - S * kLineB, m = channel(32 * wave + (l >> 1));
        const __amdgpu_buffer_rsrc_t r =
            buffer_rsrc(p.w + ((size_t)u.t.e * p.M + u.m0) * KB, (uint32_t)(p.M - u.m0) * (uint32_t)KB);
        const uint32_t at = (uint32_t)m * KB + (uint32_t)S * kLineB + (l & 1) * 16;
#pragma unroll
        for (int h = 0; h < kSub; ++h)
            c[h].c = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                                   r, (int)(h * 32 + (l & 1) * 16 < left ? at + h * 32 : kPast), 0, 0));
        if constexpr (kGen) {
            const size_t z_at = (size_t)u.t.e * groups * p.M + u.m0;
            const __amdgpu_buffer_rsrc_t rz = buffer_rsrc(p.zero + (p.zero ? z_at : 0),
                                                          p.zero ? (uint32_t)groups * (uint32_t)p.M - (uint32_t)u.m0 : 0u);
#pragma unroll
            for (int h = 0; h < kSub; ++h) {
                const int g = (2 * (kSub * S + h) + (l & 1)) >> gl;
                c[h].z = bload1(rz, g < groups ? (uint32_t)(g * p.M + m) : kPast);
            }
        }
    }
    // What is added to the lane's codes of a slab (as signed numbers, times 16) with zero points.
    __device__ __forceinline__ float offset(const Codes &c) const { return kGen && p.zero ? 8.0f - (float)(int)c.z : 0.0f; }
    // Codes 4 half .. 4 half + 3 of a word as operands, whole numbers, from the conversion of signed 4-bit numbers
    // (/ 16), one a code.
    __device__ __forceinline__ void operands(uint32_t w, float z, int half, uint32_t (&o)[4]) const {
        const uint32_t a = (w ^ 0x88888888u) >> (16 * half), b = a >> 4;
        auto f = [&](uint32_t v) __attribute__((always_inline)) {
            const float c = __builtin_amdgcn_cvt_off_f32_i4((int)v);
            return __float_as_uint(kGen ? fmaf(c, 16.0f, z) : c);
        };
        o[2 * half] = halves(f(b & 0xFFu), f(a & 0xFFu), kHigh);
        o[2 * half + 1] = halves(f((b >> 8) & 0xFFu), f((a >> 8) & 0xFFu), kHigh);
    }
    __device__ __forceinline__ uint32_t word(const Codes &c, int t) const { return t == 0 ? c.c.x : t == 1 ? c.c.y : t == 2 ? c.c.z : c.c.w; }
    // Piece t (0..3) of the lane's 32 operands of a slab, into LDS. (Written in assembly: before an LDS write
    // of its own the compiler waits for every load into LDS, other buffers' too; meet() waits for the writes.)
    __device__ __forceinline__ void store(unsigned char *ab, int t, const uint32_t (&o)[4]) const {
        const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char *)ab + (uint32_t)(made_at() ^ (16 * t));
        const u32x4_t v = {o[0], o[1], o[2], o[3]};
        asm volatile("ds_write_b128 %0, %1" ::"v"(at), "v"(v));
    }
    __device__ __forceinline__ void convert(Codes c, unsigned char *ab) const {
        // (made anew: or the compiler does this work in front of the branch, for the waves that multiply too)
        asm volatile("" : "+v"(c.c.x), "+v"(c.c.y), "+v"(c.c.z), "+v"(c.c.w));
        const float k = offset(c);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            uint32_t o[4];
            operands(word(c, t), k, 0, o);
            operands(word(c, t), k, 1, o);
            store(ab, t, o);
        }
    }
    // The scales of slabs 2P and 2P + 1: [group][staged row], the groups of two slabs.
    __device__ __forceinline__ void issue_s(const Unit &u, unsigned char *sbuf, int P) const {
        const int l = here(), in = kGen ? wave : 2 * wave + (l >> 5);
        const size_t at = (size_t)u.t.e * groups * p.M + u.m0;
        const uint32_t n = (uint32_t)groups * (uint32_t)p.M - (uint32_t)u.m0;
        const __amdgpu_buffer_rsrc_t r = buffer_rsrc(reinterpret_cast<const unsigned char *>(p.scale) + at * sb, n * sb);
        const int g = ((4 * P) >> gl) + in, R = kGen ? l * (16 / sb) : (l & 31) * 8;
        if (wave < kPairGroups * kGroupB / 1024)
            to_lds16<0>(r, sbuf + wave * 1024, in < 4 >> gl && g < groups && R < kBCh ? (uint32_t)(g * p.M + channel(R)) * sb : kPast);
    }
    // A block barrier; the wave's loads have landed, its LDS reads have returned and its writes are done.
    __device__ __forceinline__ void meet() const {
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

    // The products of slab h of a line: rows in xb, operands in ab. kFlush: steps that share a scale (at most
    // those of a slab). Beside them the codes c of the slab behind become operands in nab. An operand is read one
    // subtile ahead; a sum is scaled just before its registers take the next one, kN matrix
    // instructions after its last: so the matrix instructions always have something beside them.
    template <int kN, int kFlush>
    __device__ __forceinline__ void slab(f32x4_t (&acc)[kBA][kN], const unsigned char *xb, const unsigned char *ab,
                                         const unsigned char *sbuf, int h, const Codes &c, unsigned char *nab) const {
        constexpr int kGroups = kBS / kFlush;  // groups of a slab
        constexpr int kVPerM = F::kParts == 3 ? 2 : 3;
        const int l = here(), col = l & 15, q = l >> 4, rd = read_at();
        const unsigned char *mine = ab + ch * kBA * kTile * kSlabB;
        f32x4_t sum[kN];
        uint4 x[kN][kBS][F::kParts], b[2][kBS];
        uint32_t raw[2][kGroups];
        float scale[2][kGroups];
        auto weights = [&](int i) __attribute__((always_inline)) {
#pragma unroll
            for (int s = 0; s < kBS; ++s) b[i & 1][s] = load16(mine + i * kTile * kSlabB + (rd ^ (64 * s)));
        };
        const int R0 = ch * kBA * kTile + col, step = h % 2 * kBS;
        auto bits = [&](int i) __attribute__((always_inline)) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) raw[i & 1][g] = scale_bits(sbuf, (step + g * kFlush) >> gl, R0 + i * kTile);
        };
        auto scaled = [&](int i, int g, int j) __attribute__((always_inline)) {
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(scale[i & 1][g], sum[j][r], acc[i][j][r]);
        };
        const float k = offset(c);
        uint32_t made[4];
        weights(0);
        bits(0);
#pragma unroll
        for (int s = 0; s < kBS; ++s)
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                // (fp32: a step's columns lie in piece s of a row)
                const unsigned char *row = xb + ((kPer > 1 ? s * kRows : 0) + (th * kN + j) * kTile) * kSlabB;
                uint4 v[kPer];
#pragma unroll
                for (int e = 0; e < kPer; ++e) v[e] = load16(row + (kPer > 1 ? spos(col, 2 * q + e) : rd ^ (64 * s)));
                F::parts(v, x[j][s]);
            }
#pragma unroll
        for (int i = 0; i < kBA; ++i) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g) scale[i & 1][g] = scale_of(raw[i & 1][g], col);
            if (i + 1 < kBA) bits(i + 1);
            if (i + 1 < kBA) weights(i + 1);
            if (i % 2 == 1) {
                operands(word(c, i / 2), k, 0, made);
                operands(word(c, i / 2), k, 1, made);
                store(nab, i / 2, made);
            }
#pragma unroll
            for (int s = 0; s < kBS; ++s)
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    if (s % kFlush == 0) {
                        if (s > 0) scaled(i, s / kFlush - 1, j);
                        else if (i > 0) scaled(i - 1, kGroups - 1, j);
                        sum[j] = f32x4_t{};
                    }
#pragma unroll
                    for (int e = 0; e < F::kParts; ++e) mma(sum[j], x[j][s][e], b[i & 1][s]);
                }
            // their order: the reads ahead first, then a few vector instructions before each matrix instruction
            if (i + 1 < kBA) __builtin_amdgcn_sched_group_barrier(0x100, kBS + kGroups, 0);
#pragma unroll
            for (int m = 0; m < kBS * kN * F::kParts; ++m) {
                __builtin_amdgcn_sched_group_barrier(0x002, kVPerM, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < kN; ++j) scaled(kBA - 1, kGroups - 1, j);
    }
};

template <class X, bool kGen>
__global__ __launch_bounds__(kBWaves *kWave) __attribute__((amdgpu_waves_per_eu(2, 2))) void w4_block_kernel(W4Params p) {
    using B = W4Block<X, kGen>;
    // The buffers are separate objects, so that the compiler can tell loads into one from reads of the other.
    __shared__ __align__(16) unsigned char x0[B::kRows * B::kPer * kSlabB], x1[B::kRows * B::kPer * kSlabB], a0[kBCh * kSlabB], a1[kBCh * kSlabB];
    __shared__ __align__(16) unsigned char s0[B::kScaleB], s1[B::kScaleB];
    // the scan of the row tiles, kept out of the registers of the products
    __shared__ TileScan scans[kWave];
    const B b(p);
    const int S = (b.Mo + b.cols - 1) / b.cols;
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
            return find_unit<16>(scans[l], l, i, S, b.cols);
        }
        // dense: groups of four row tiles run channel block by channel block, so that the CUs of an XCD
        // work on a near-square patch and share both operands in L2
        constexpr int kGroup = 4;
        const int g = i / (kGroup * S), in = i - g * kGroup * S, h = min(kGroup, tiles - g * kGroup);
        const int c = in / h, ti = g * kGroup + in - c * h;
        return Unit{{0, ti * p.tile_rows, min(p.tile_rows, p.n_rows - ti * p.tile_rows)}, c * b.cols};
    };
    int i = first + blockIdx.x / kXcds;
    if (i >= last) return;  // uniform
    Unit u = unit(i);
    constexpr int kSub = B::kSub;
    typename B::Codes codes[kSub], ncodes[kSub];
    b.issue_s(u, s0, 0);
    b.issue_c(u, codes, 0);
    b.template issue_x<B::kXSegs>(u, x0, 0, true);
    b.convert(codes[0], a0);
    for (;;) {
        i += step;
        const bool more = i < last;
        const Unit nxt = more ? unit(i) : u;
        auto run = [&](auto nc, auto fc) __attribute__((always_inline)) {
            constexpr int kN = decltype(nc)::value, kFlush = decltype(fc)::value;
            const bool busy = b.th * kN * kTile < u.t.n;  // uniform: the wave has rows
            f32x4_t acc[kBA][kN] = {};
            // Line S of the codes: kSub slabs. Past K nothing is multiplied, but the buffers take their turns.
            for (int S = 0; S < b.nsuper; ++S) {
                const bool end = S + 1 >= b.nsuper;
                auto turn = [&](auto hc, const unsigned char *xb, unsigned char *nxb, const unsigned char *ab, unsigned char *nab,
                                const unsigned char *sbuf) __attribute__((always_inline)) {
                    constexpr int h = decltype(hc)::value;
                    const int s = S * kSub + h;
                    const typename B::Codes &c = h < kSub - 1 ? codes[(h + 1) % kSub] : ncodes[0];
                    b.meet();
                    // the next slab of rows: the unit's, or behind its last turn the next unit's first
                    const bool over = h == kSub - 1 && end;
                    if (over) b.template issue_x<B::kXSegs>(nxt, nxb, 0, more);
                    else b.template issue_x<kN>(u, nxb, s + 1, s + 1 < b.nslab);
                    if (h == 1) b.issue_s(u, s1, 2 * S + 1);
                    if (h == kSub - 2) b.issue_c(end ? nxt : u, ncodes, end ? 0 : S + 1);
                    if (h == 3) b.issue_s(end ? nxt : u, s0, end ? 0 : 2 * S + 2);
                    if (busy && s < b.nslab) {
                        b.template slab<kN, kFlush>(acc, xb, ab, sbuf, h, c, nab);
                    } else {
                        b.convert(c, nab);
                    }
                };
                turn(std::integral_constant<int, 0>{}, x0, x1, a0, a1, s0);
                turn(std::integral_constant<int, 1>{}, x1, x0, a1, a0, s0);
                turn(std::integral_constant<int, 2>{}, x0, x1, a0, a1, s1);
                turn(std::integral_constant<int, 3>{}, x1, x0, a1, a0, s1);
#pragma unroll
                for (int h = 0; h < kSub; ++h) codes[h] = ncodes[h];
            }
            // results
            const int l = b.here(), col = l & 15, q = l >> 4, out = p.swiglu ? kBA / 2 : kBA;
#pragma unroll
            for (int j = 0; j < kN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int n = (b.th * kN + j) * kTile + 4 * q + r;
                    if (n >= u.t.n) continue;
#pragma unroll
                    for (int a = 0; a < kBA; ++a) {
                        const int m = u.m0 + (b.ch * out + a) * kTile + col;
                        if (a >= out || m >= b.Mo) continue;
                        float z = acc[a][j][r] / B::kUnit;
                        if (a < kBA / 2 && p.swiglu)
                            z = (z < kFarGate ? silu_far(z) : silu(z)) * (acc[(a + kBA / 2) % kBA][j][r] / B::kUnit);
                        const size_t at = (size_t)(u.t.start + n) * b.Mo + m;
                        if (p.y_f32) reinterpret_cast<float *>(p.y)[at] = z;
                        else reinterpret_cast<uint16_t *>(p.y)[at] = (uint16_t)(pack_bf16(z, 0.0f) & 0xFFFFu);
                    }
                }
        };
        auto sized = [&](auto fc) __attribute__((always_inline)) {
            const int sub = (u.t.n + 4 * kTile - 1) / (4 * kTile);  // row subtiles per wave
            if (sub == 1) run(std::integral_constant<int, 1>{}, fc);
            else if (B::kMaxN == 2 || sub == 2) run(std::integral_constant<int, 2>{}, fc);
            else if constexpr (B::kMaxN > 2) {
                if (B::kMaxN == 3 || sub == 3) run(std::integral_constant<int, 3>{}, fc);
                else if constexpr (B::kMaxN > 3) run(std::integral_constant<int, 4>{}, fc);
            }
        };
        if (b.gl > 0) sized(std::integral_constant<int, 2>{});
        else sized(std::integral_constant<int, 1>{});
        if (!more) break;
        u = nxt;
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // no load into this block's LDS outlives it
}

}  // namespace

template <class X>
static hipError_t launch_form(const W4Params &p, hipStream_t s) {
    auto go = [&](auto gen) -> hipError_t {
        constexpr bool kGen = decltype(gen)::value;
        constexpr int kRows = W4Block<X, kGen>::kRows;
        if (p.tile_rows < 1 || p.tile_rows > kRows) return hipErrorInvalidValue;  // the buffers hold no more
        const int cus = num_cus(), Mo = p.swiglu ? p.M / 2 : p.M, cols = p.swiglu ? kBCh / 2 : kBCh;
        const long units = most_tiles(p, p.tile_rows) * ((Mo + cols - 1) / cols);
        const unsigned grid = (unsigned)((units < cus ? units : cus) + kXcds - 1) / kXcds * kXcds;
        launch_k(w4_block_kernel<X, kGen>, grid, kBWaves * kWave, 0, s, p);
        return hipGetLastError();
    };
    return p.zero || p.scale_f32 ? go(std::true_type{}) : go(std::false_type{});
}

}  // namespace moe
