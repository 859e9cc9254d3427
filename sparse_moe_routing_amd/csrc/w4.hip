// w4.hip - products with 4-bit weights and a scale (and a zero point) per group of columns, grouped by
// expert: y[n][m] = sum_g s[g][m] sum_{k in g} x[n][k] (c[m][k] - z[g][m]) for the rows n of expert e.
//
// Nothing is rounded on the way to the sums: a code is a whole number, exact in
// bf16, and a bf16 row element is an operand as it stands; fp32 rows go in as three bf16 parts that add up to all
// of their 24 bits. A group's sum runs in the matrix instructions (16x16x32, fp32 sums), the zero point and the
// scale are applied to it in fp32: in the form for few rows as s (sum x (c - b) - (z - b) sum x), b a constant of
// the operand's form.
// Rows are the A operand and channels the B operand: a lane's accumulators are four rows of one
// channel, so that one scale serves all of a lane's sums.
// The form for many rows is in w4_block.h. Which one runs is chosen in w4_choice.h, from estimated times.
#include "w4_core.h"

namespace moe {

namespace {

// ------------------------------------------------------------------------- few rows per expert
// With a few rows per expert the time is the one read of the weights: HBM bounds it. Measured (us, one
// call over changing operands): 256 experts of 2048 x 1024 with 32 tokens' 256 rows 35 to 38 (178 MB, 5.0 TB/s), one
// row of 4096 x 65536 with zero points 45 (147 MB, 3.3 TB/s: its 2048 units are eight to a CU, which holds seven of
// their blocks, so that the last eighth runs by itself), 4 rows of 2048 x 1024 8.4 and 32 rows of 4096 x 4096 10.1 (a launch and one chain
// of loads).
//
// A wave takes up to 4 kR rows of one
// expert and 32 weight channels (with SwiGLU 16 gate and the matching 16 up channels) and streams the
// channels' codes in slabs of 128 bytes (256 columns), whole cache lines loaded straight into its own
// ring of slab buffers, with the slab's scales and zero points beside them. The rows come through
// buffer loads into registers; rows past the tile's read as zero without a memory access.
// Eight one-wave blocks are launched for a CU, which its LDS holds at once; of those with a ring of four and zero points
// or fp32 scales (21 KB each) it holds seven, and the last one's units follow when one of them has ended. They are
// persistent: a wave walks its units, and the ring takes the next unit's first slabs while the last slabs and
// the results of the present one are worked on. A unit takes whole turns of the ring: with K = 512 half of the slabs of a
// ring of four, and a third of those of a ring of three, are zeros.
// kKS waves make a block and split K between them (their sums join in LDS, in order) where there is so
// little to stream that single waves would not cover the chip; each such block takes one unit.
//
// Of every four operand rows 4a .. 4a + 3 the tile's tokens fill only kR; the others hold the same
// tokens' columns of the next steps, so that a slab of 4 rows takes two loads in place of eight. Operand row
// 4a + kR b + r holds token a + 4 r, b steps on. All four are multiplied with a step's codes, and
// of the four sums of a lane those are taken whose columns are the step's: a sum is only continued by
// a step of the same place. The rows' own sums, for the zero points, need one instruction for 4 / kR steps.
// (Against one 16 x 16 tile a wave with the rows loaded as they lie: one row 183 -> 45 us, 32 tokens over 256
// experts 148 -> 36. Moving the sums between lanes in place of choosing among them takes 49 for the latter, two
// tiles of 16 rows a wave spill.)
constexpr int kSCh = kW4StreamChannels;    // weight channels of a wave
constexpr int kSteps = kSlabK / kStepK;    // matrix instructions per 16 channels and slab
constexpr int kCodeBytes = kSCh * kSlabB;  // a slab's codes
constexpr int kScaleBytes = kWave * 16;    // room for its scales: at most 8 groups of 32 fp32 numbers
constexpr int kZeroBytes = kWave * 4;      // and zero points
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
                if (s % (kSteps / F::kSplit) == 0 && s > 0) __builtin_amdgcn_sched_barrier(0);  // registers
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

template <class X, int kR, int kKS>
void launch_stream(const W4Params &p, bool swiglu, unsigned grid, hipStream_t s) {
    const bool gen = p.zero || p.scale_f32;
    if (gen && swiglu) launch_k(w4_stream_kernel<X, true, kR, kKS, true>, grid, kKS * kWave, 0, s, p);
    else if (gen) launch_k(w4_stream_kernel<X, false, kR, kKS, true>, grid, kKS * kWave, 0, s, p);
    else if (swiglu) launch_k(w4_stream_kernel<X, true, kR, kKS, false>, grid, kKS * kWave, 0, s, p);
    else launch_k(w4_stream_kernel<X, false, kR, kKS, false>, grid, kKS * kWave, 0, s, p);
}

}  // namespace

hipError_t launch_matmul_w4(const W4Params &p, int x_dtype, hipStream_t s) {
    const bool swiglu = p.swiglu;
    const int Mo = swiglu ? p.M / 2 : p.M, cus = num_cus();
    const W4Choice c = w4_choose(W4Sizes{p.n_rows, p.E, p.M, p.K, p.group, p.offsets != nullptr, x_dtype == 0, p.scale_f32 != 0,
                                         p.zero != nullptr, p.y_f32 != 0, swiglu}, cus);
    if (c.r == 0) {
        W4Params b = p;
        b.tile_rows = c.tile_rows;
        if (x_dtype == 0) return launch_w4_block_f32(b, s);
        return launch_w4_block_bf16(b, s);
    }
    const int cols = swiglu ? kSCh / 2 : kSCh, S = (Mo + cols - 1) / cols;
    const long units = most_tiles(p, 4 * c.r) * S, room = (long)cus * kW4StreamBlocks;
    const long blocks = units <= room || c.split ? units : room;
    const unsigned grid = (unsigned)((blocks + kXcds - 1) / kXcds * kXcds);
    auto go = [&](auto x, auto rc) {
        using X = decltype(x);
        constexpr int kR = decltype(rc)::value;
        if (c.split) launch_stream<X, kR, kW4Split>(p, swiglu, grid, s);
        else launch_stream<X, kR, 1>(p, swiglu, grid, s);
    };
    using R1 = std::integral_constant<int, 1>;
    using R2 = std::integral_constant<int, 2>;
    using R4 = std::integral_constant<int, 4>;
    if (x_dtype == 0) c.r == 1 ? go(float{}, R1{}) : go(float{}, R2{});
    else c.r == 1 ? go(uint16_t{}, R1{}) : c.r == 2 ? go(uint16_t{}, R2{}) : go(uint16_t{}, R4{});
    return hipGetLastError();
}

}  // namespace moe
