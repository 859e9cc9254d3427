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
__device__ __forceinline__ RowTile pick_tile(const TileScan &s, int per, int u) {
    int at = s.at, e = 0, start = 0, n = 0;
    bool mine = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (u >= at && u < at + s.nt[i]) {
            mine = true;
            e = 4 * lane_id() + i;
            start = s.lo[i] + (u - at) * per;
            n = min(per, s.hi[i] - start);
        }
        at += s.nt[i];
    }
    const uint64_t who = __ballot(mine);
    if (!who) return {0, 0, 0};
    const int src = __ffsll((unsigned long long)who) - 1;
    return {__builtin_amdgcn_readlane(e, src), __builtin_amdgcn_readlane(start, src),
            __builtin_amdgcn_readlane(n, src)};
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
    const RowTile t = p.offsets ? pick_tile(scan_tiles(p.offsets, p.E, p.n_rows, kTRows), kTRows, u)
                                : RowTile{0, u * kTRows, min(kTRows, p.n_rows - u * kTRows)};
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

// ------------------------------------------------------------------------- large row counts
// A block multiplies up to 320 rows of one expert by 256 weight channels (with SwiGLU: 128 gate
// channels and the 128 up channels that go with them). K is staged in slabs of 128 bytes per row,
// loaded straight into LDS (buffer loads with the LDS flag: no registers held while in flight),
// double-buffered: the next slab's loads are in flight during the current slab's matrix
// instructions, one block barrier per slab. Eight waves, two per SIMD: wave w takes the channels
// of half w % 2 and a quarter of the tile's 16-row subtiles, at most five, so that a tile of n rows
// costs ceil(n / 64) subtiles of matrix work per wave whatever n is.
//
// Bounds come from the buffer resources: the row resource covers exactly the tile's n rows and the
// weight resource the expert's remaining channels, so that loads past either return zeros without
// a memory access; pieces past K in the last slab are sent past the range in the same way.
constexpr int kBWaves = 8;
constexpr int kBRows = 320, kBCh = 256;   // rows and weight channels per block
constexpr int kSlabB = 128;               // bytes (K elements) of a staged row
constexpr int kBA = kBCh / 2 / kTile;     // channel subtiles per wave (8)
constexpr int kXSegs = kBRows * kSlabB / 1024 / kBWaves;  // 1 KB row segments per wave (5)
constexpr int kWSegs = kBCh * kSlabB / 1024 / kBWaves;    // 1 KB weight segments per wave (4)
constexpr int kXcds = 8;
constexpr uint32_t kPast = 0xFFFFFFF0u;   // a buffer offset past every range

// Position of 16-byte piece pc (0..7) of staged row r: rows 2m and 2m + 1 rotate by m, so the 16
// rows of one operand read lie on distinct bank groups; rows 16 apart keep their pieces' order.
__device__ __forceinline__ int spos(int r, int pc) { return r * kSlabB + ((pc ^ (r >> 1)) & 7) * 16; }

// The slab buffers are separate objects, so that the compiler can tell loads into one from operand
// reads of the other.
__shared__ __align__(16) unsigned char b_w0[kBCh * kSlabB], b_w1[kBCh * kSlabB];
__shared__ __align__(16) unsigned char b_x0[kBRows * kSlabB], b_x1[kBRows * kSlabB];

__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t r, unsigned char *seg, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)seg, 16,
                                             (int)off, 0, 0, 0);
}

template <bool kSwiglu, class O, int kN>
__device__ __forceinline__ void block_product(const I8Params &p, const RowTile &t, int m0) {
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, q = lane >> 4;
    const int ch = wave & 1, th = (wave >> 1) & 3;
    const int Mo = kSwiglu ? p.M / 2 : p.M;
    const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(p.x + (size_t)t.start * p.K, (uint32_t)t.n * (uint32_t)p.K);
    const __amdgpu_buffer_rsrc_t rw =
        buffer_rsrc(p.w + ((size_t)t.e * p.M + m0) * p.K, (uint32_t)(p.M - m0) * (uint32_t)p.K);
    // weight channel (past m0) of staged row R; SwiGLU: each half of 128 staged rows holds 64 gate
    // channels, then the 64 matching up channels
    auto channel = [&](int R) {
        return kSwiglu ? (R >> 7) * 64 + (R & 63) + ((R >> 6) & 1) * Mo : R;
    };
    const int lr = lane >> 3;
    uint32_t xoff[kXSegs], woff[kWSegs];
    // lane l of a segment's load writes position l % 8 of row l / 8, so it reads the piece that the
    // row's rotation puts there: a function of the row modulo 16
#pragma unroll
    for (int a = 0; a < kXSegs; ++a) {
        const int R = 8 * (kXSegs * wave + a) + lr;
        xoff[a] = (uint32_t)R * p.K + (((lane & 7) ^ (R >> 1)) & 7) * 16;
    }
#pragma unroll
    for (int a = 0; a < kWSegs; ++a) {
        const int R = 8 * (kWSegs * wave + a) + lr;
        woff[a] = (uint32_t)channel(R) * p.K + (((lane & 7) ^ (R >> 1)) & 7) * 16;
    }
    const int nslab = (p.K + kSlabB - 1) / kSlabB;
    const bool ragged = p.K % kSlabB != 0;
    auto issue = [&](unsigned char *wb, unsigned char *xb, int s) __attribute__((always_inline)) {
        const bool tail = ragged && s == nslab - 1;  // uniform
#pragma unroll
        for (int a = 0; a < kXSegs; ++a) {
            const int R = 8 * (kXSegs * wave + a);
            if (R >= t.n) continue;  // uniform: whole segments past the tile (their results are dropped)
            uint32_t off = xoff[a] + s * kSlabB;
            if (tail && s * kSlabB + (((lane & 7) ^ ((R + lr) >> 1)) & 7) * 16 >= p.K) off = kPast;
            to_lds16(rx, xb + (kXSegs * wave + a) * 1024, off);
        }
#pragma unroll
        for (int a = 0; a < kWSegs; ++a) {
            const int R = 8 * (kWSegs * wave + a);
            uint32_t off = woff[a] + s * kSlabB;
            if (tail && s * kSlabB + (((lane & 7) ^ ((R + lr) >> 1)) & 7) * 16 >= p.K) off = kPast;
            to_lds16(rw, wb + (kWSegs * wave + a) * 1024, off);
        }
    };
    i32x4_t acc[kBA][kN] = {};
    const int rd[2] = {spos(col, q), spos(col, 4 + q)};
    const bool busy = th * kN * kTile < t.n;  // uniform: the wave has rows
    auto mult = [&](const unsigned char *wb, const unsigned char *xb) __attribute__((always_inline)) {
        if (!busy) return;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            uint4 a[kBA], b[kN];
#pragma unroll
            for (int i = 0; i < kBA; ++i) a[i] = load16(wb + (ch * kBA + i) * kTile * kSlabB + rd[s]);
#pragma unroll
            for (int j = 0; j < kN; ++j) b[j] = load16(xb + (th * kN + j) * kTile * kSlabB + rd[s]);
#pragma unroll
            for (int j = 0; j < kN; ++j)
#pragma unroll
                for (int i = 0; i < kBA; ++i) mma_i8(acc[i][j], a[i], b[j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto turn = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's loads are in LDS
        __syncthreads();
    };
    issue(b_w0, b_x0, 0);
    turn();
    for (int s = 0; s < nslab; s += 2) {
        if (s + 1 < nslab) issue(b_w1, b_x1, s + 1);
        mult(b_w0, b_x0);
        turn();
        if (s + 2 < nslab) issue(b_w0, b_x0, s + 2);
        if (s + 1 < nslab) mult(b_w1, b_x1);
        turn();
    }
    if (!busy) return;
    constexpr int kOut = kSwiglu ? kBA / 2 : kBA;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        const int n = (th * kN + j) * kTile + col;
        if (n >= t.n) continue;
        const float sx = p.x_scale[t.start + n];
        O *y = reinterpret_cast<O *>(p.y) + (size_t)(t.start + n) * Mo;
#pragma unroll
        for (int i = 0; i < kOut; ++i) {
            const int mc = m0 + (ch * kOut + i) * kTile + 4 * q;
            if (mc >= Mo) continue;
            const float *sw = p.w_scale + (size_t)t.e * p.M + mc;
            float z[4];
            scaled(acc[i][j], sx, sw, z);
            if constexpr (kSwiglu) {
                float up[4];
                scaled(acc[kOut + i][j], sx, sw + Mo, up);
#pragma unroll
                for (int r = 0; r < 4; ++r) z[r] = z[r] / (1.0f + expf(-z[r])) * up[r];
            }
            store4(y + mc, z);
        }
    }
}

template <bool kSwiglu, class O>
__global__ __launch_bounds__(kBWaves *kWave) __attribute__((amdgpu_waves_per_eu(2, 2))) void i8_block_kernel(
    I8Params p) {
    constexpr int kCols = kSwiglu ? kBCh / 2 : kBCh;  // output channels of a block
    const int Mo = kSwiglu ? p.M / 2 : p.M;
    const int S = (Mo + kCols - 1) / kCols;
    TileScan sc;
    int tiles = (p.n_rows + kBRows - 1) / kBRows;
    if (p.offsets) {
        sc = scan_tiles(p.offsets, p.E, p.n_rows, kBRows);
        tiles = sc.total;
    }
    // unit = (row tile, channel block), the channel blocks of a tile next to each other; blocks
    // b, b + 8, ... run on one XCD and take one contiguous eighth of the units
    const int units = tiles * S, per = (units + kXcds - 1) / kXcds;
    const int idx = blockIdx.x / kXcds, u = (blockIdx.x % kXcds) * per + idx;
    if (idx >= per || u >= units) return;  // uniform
    const int ti = u / S, m0 = (u - ti * S) * kCols;
    const RowTile t = p.offsets ? pick_tile(sc, kBRows, ti)
                                : RowTile{0, ti * kBRows, min(kBRows, p.n_rows - ti * kBRows)};
    const int sub = (t.n + 4 * kTile - 1) / (4 * kTile);  // row subtiles per wave
    if (sub == 1) block_product<kSwiglu, O, 1>(p, t, m0);
    else if (sub == 2) block_product<kSwiglu, O, 2>(p, t, m0);
    else if (sub == 3) block_product<kSwiglu, O, 3>(p, t, m0);
    else if (sub == 4) block_product<kSwiglu, O, 4>(p, t, m0);
    else block_product<kSwiglu, O, 5>(p, t, m0);
}

}  // namespace

hipError_t launch_matmul_i8(const I8Params &p, bool swiglu, int y_dtype, hipStream_t s) {
    const int Mo = swiglu ? p.M / 2 : p.M;
    // most row tiles n_rows rows of E experts can make: full ones, and a part of one per expert
    const long tiles = p.offsets ? p.n_rows / kTRows + (p.E < p.n_rows ? p.E : p.n_rows)
                                 : (p.n_rows + kTRows - 1) / kTRows;
    if (p.n_rows >= 16 * (long)p.E) {
        const int cols = swiglu ? kBCh / 2 : kBCh;
        const long t2 = p.offsets ? p.n_rows / kBRows + (p.E < p.n_rows ? p.E : p.n_rows)
                                  : (p.n_rows + kBRows - 1) / kBRows;
        const long grid = (t2 * ((Mo + cols - 1) / cols) + kXcds - 1) / kXcds * kXcds;
        auto go = [&](auto o) {
            using O = decltype(o);
            if (swiglu) launch_k(i8_block_kernel<true, O>, (unsigned)grid, kBWaves * kWave, 0, s, p);
            else launch_k(i8_block_kernel<false, O>, (unsigned)grid, kBWaves * kWave, 0, s, p);
        };
        if (y_dtype == 0) go(float{});
        else go(uint16_t{});
        return hipGetLastError();
    }
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
