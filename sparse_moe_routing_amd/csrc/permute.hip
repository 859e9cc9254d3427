// permute.hip - rows sorted by expert and back, their gradients, and rows as 8-bit integers.
//
//   permute            xs[r_k] = x[t]                       r_k = rows[8t + k], k = 0..7
//   permute_backward   dx[t] = sum_k dxs[r_k]
//   unpermute          y[t] = sum_k w_k ys[r_k] + g sh[t]
//   unpermute_backward dys[r_k] = w_k dy[t], dw_k = <dy[t], ys[r_k]>, dsh[t] = g dy[t],
//                      dg = <dy[t], sh[t]>
// All of them run token by token over the inverse table `rows`: every element of x, dy, y, dx is
// touched once, every sorted row once, no atomics, and a token's sums run in rank order whatever
// the batch. They move bytes and little else, so what bounds them is HBM at large T and the
// latency of one dependent chain (table entry, row, result) at decode. A block works on one row whatever
// its width: rows of a few hundred bytes leave most of its lanes idle (8192 tokens of 64 bf16: the sort
// 6.4 us, 1.5 TB/s, 65536 rows as integers 21 us; of 256: 8.6 us, 4.4 TB/s, and 26 us).
//
// Two measures are quoted: "alone" is a single call after the caches were filled with other data,
// "in a row" one of many calls over changing operands, where a call's last stores leave the caches
// under the next one.
#include "device_common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kRowThreads = 256;

// Eight consecutive elements (the unit of all row kernels) as fp32 and back.
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t *p, float (&v)[8]) {
    const uint4 a = load16(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
// The same from a buffer resource at a byte offset: past its range (an empty range: a dropped pair)
// zeros, without a memory access.
template <int kAux>
__device__ __forceinline__ uint4 row_piece(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, kAux));
}
template <class E>
struct Piece8;  // eight elements as loaded
template <>
struct Piece8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t h) {
        a = row_piece<kBufNT>(r, h * 4);
        b = row_piece<kBufNT>(r, h * 4 + 16);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    }
};
template <>
struct Piece8<uint16_t> {
    uint4 a;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t h) { a = row_piece<kBufNT>(r, h * 2); }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
// Row r of a sorted buffer; a dropped pair (r < 0) has an empty range.
template <class E>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_rsrc(const E *rows, int r, int H) {
    return buffer_rsrc(rows + (size_t)max(r, 0) * H, r >= 0 ? (uint32_t)(H * sizeof(E)) : 0u);
}

// The eight sorted rows of token t; -1 for an entry outside [0, n_rows).
__device__ __forceinline__ void token_rows(const int32_t *rows, int t, int n_rows, int (&r)[kTopK]) {
#pragma unroll
    for (int k = 0; k < kTopK; ++k) {
        const int v = rows[(size_t)t * kTopK + k];
        r[k] = v >= 0 && v < n_rows ? v : -1;
    }
}

// Stores of the sorted rows. kStream: past the caches. A prefill chunk's eight copies of its rows are
// more than the 256 MB behind the L2s hold, and written through the caches they only push each
// other out (in a row, T = 8192 rows of 2048 bf16: 61.8 us, 51.5 streamed; the return's gradient of
// 4097 tokens 69.6 and 65.5, now 63); a decode round's rows are read back at once and stay in them.
constexpr size_t kStreamBytes = (size_t)64 << 20;
template <bool kStream>
__device__ __forceinline__ void put16(void *p, const uint4 &v) {
    if constexpr (kStream)
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4_t, v), reinterpret_cast<u32x4_t *>(p));
    else
        *reinterpret_cast<uint4 *>(p) = v;
}
template <bool kStream>
__device__ __forceinline__ void put8(float *p, const float (&v)[8]) {
    put16<kStream>(p, __builtin_bit_cast(uint4, make_float4(v[0], v[1], v[2], v[3])));
    put16<kStream>(p + 4, __builtin_bit_cast(uint4, make_float4(v[4], v[5], v[6], v[7])));
}
template <bool kStream>
__device__ __forceinline__ void put8(uint16_t *p, const float (&v)[8]) {
    put16<kStream>(p, uint4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                            pack_bf16(v[6], v[7])});
}

// One block per token: its row is read once and stored to its eight places from registers (T = 8192 of
// 2048 bf16: 288 MiB moved in 61 us alone, 4.9 TB/s, nearly all of it stores, 52 in a row; one launch
// at T = 4: 5 us).
template <class E, bool kStream>
__global__ __launch_bounds__(kRowThreads) void permute_kernel(const E *x, const int32_t *rows, int H,
                                                              int n_rows, E *xs) {
    constexpr int kPer = 16 / sizeof(E);
    const int t = blockIdx.x;
    int r[kTopK];
    token_rows(rows, t, n_rows, r);
    for (int h = threadIdx.x * kPer; h < H; h += kRowThreads * kPer) {
        const uint4 v = load16(x + (size_t)t * H + h);
#pragma unroll
        for (int k = 0; k < kTopK; ++k)
            if (r[k] >= 0) put16<kStream>(xs + (size_t)r[k] * H + h, v);
    }
}

// One block per token again: the sum over its eight sorted rows is formed where they arrive, in fp32
// and in rank order, and rounded once. kWeighted: unpermute (weights, optional shared row);
// otherwise permute_backward. T = 8192 of 2048 bf16: 322 MiB in 59 us and 289 MiB in 53 us, alone (58
// and 52 in a row), 5.7 TB/s, between the rates of a large copy (5.1) and of reads alone (6.5).
template <class E, class O, bool kWeighted>
__global__ __launch_bounds__(kRowThreads) void unpermute_kernel(const E *ys, const int32_t *rows,
                                                                const float *w, const E *shared,
                                                                const float *gate, int H, int n_rows,
                                                                O *y) {
    const int t = blockIdx.x;
    int r[kTopK];
    token_rows(rows, t, n_rows, r);
    float wk[kTopK];
#pragma unroll
    for (int k = 0; k < kTopK; ++k) wk[k] = kWeighted ? w[(size_t)t * kTopK + k] : 1.0f;
    const float g = kWeighted && shared ? gate[t] : 0.0f;
    for (int h = threadIdx.x * 8; h < H; h += kRowThreads * 8) {
        // every load is issued before the first is used
        Piece8<E> in[kTopK + 1];
#pragma unroll
        for (int k = 0; k < kTopK; ++k) in[k].load(row_rsrc(ys, r[k], H), h);
        if (kWeighted) in[kTopK].load(row_rsrc(shared, shared ? t : -1, H), h);
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, v[8];
#pragma unroll
        for (int k = 0; k < kTopK; ++k) {
            if (r[k] < 0) continue;  // (its weight is not looked at)
            in[k].get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = kWeighted ? fmaf(wk[k], v[i], acc[i]) : acc[i] + v[i];
        }
        if (kWeighted && shared) {
            in[kTopK].get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(g, v[i], acc[i]);
        }
        put8<false>(y + (size_t)t * H + h, acc);
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// One block per token: dy[t] is read once for its eight scaled copies and its nine dot products with
// the same rows (fp32 sums: lanes, a butterfly over the wave, then the four waves in order, the
// same for every batch). T = 4097 of 2048 bf16: 321 MiB in 67 us alone, 5.0 TB/s, half of it stores
// (63 in a row).
template <class E, class O, bool kStream>
__global__ __launch_bounds__(kRowThreads) void unpermute_bwd_kernel(const O *dy, const E *ys,
                                                                    const int32_t *rows, const float *w,
                                                                    const E *shared, const float *gate,
                                                                    int H, int n_rows, E *dys, float *dw,
                                                                    E *dshared, float *dgate) {
    __shared__ float part[kRowThreads / kWave][kTopK + 1];
    const int t = blockIdx.x, tid = threadIdx.x;
    int r[kTopK];
    token_rows(rows, t, n_rows, r);
    float wk[kTopK], dot[kTopK + 1];
#pragma unroll
    for (int k = 0; k < kTopK; ++k) wk[k] = w[(size_t)t * kTopK + k];
#pragma unroll
    for (int k = 0; k <= kTopK; ++k) dot[k] = 0.0f;
    const float g = shared ? gate[t] : 0.0f;
    for (int h = tid * 8; h < H; h += kRowThreads * 8) {
        Piece8<E> in[kTopK + 1];
#pragma unroll
        for (int k = 0; k < kTopK; ++k) in[k].load(row_rsrc(ys, r[k], H), h);
        in[kTopK].load(row_rsrc(shared, shared ? t : -1, H), h);
        float d[8], v[8];
        load8(dy + (size_t)t * H + h, d);
#pragma unroll
        for (int k = 0; k < kTopK; ++k) {
            if (r[k] < 0) continue;
            in[k].get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[k] = fmaf(d[i], v[i], dot[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = wk[k] * d[i];
            put8<kStream>(dys + (size_t)r[k] * H + h, v);
        }
        if (shared) {
            in[kTopK].get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[kTopK] = fmaf(d[i], v[i], dot[kTopK]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = g * d[i];
            put8<false>(dshared + (size_t)t * H + h, v);
        }
    }
#pragma unroll
    for (int k = 0; k <= kTopK; ++k) {
        const float s = wave_sum(dot[k]);
        if ((tid & 63) == 0) part[tid >> 6][k] = s;
    }
    __syncthreads();
    if (tid <= kTopK) {
        float s = 0.0f;
        for (int i = 0; i < kRowThreads / kWave; ++i) s += part[i][tid];
        if (tid < kTopK) dw[(size_t)t * kTopK + tid] = s;
        else if (shared) dgate[t] = s;
    }
}

// Rows as 8-bit integers. scale = amax / 127 (IEEE division); the code is the integer nearest to
// the exact quotient v / scale, ties to even. Halves are common here: with bf16 rows v / amax has
// few bits, and 127 v / amax often ends in exactly .5. v * (1 / scale) is within 2^-16 of the
// quotient, so its rounding is the quotient's unless it lies that near a half; those few values
// take code_of: a first guess q at most one off, whose residual v - q * scale (one fused operation,
// exact next to a half: q has 8 bits, the difference cancels) is compared with scale / 2.
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
    if (amax_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);  // an infinity or a NaN
    if (amax_bits == 0) return 1.0f;
    return fmaxf(__uint_as_float(amax_bits) / 127.0f, 1.17549435e-38f);
}
__device__ __forceinline__ int code_of(float v, float scale, float inv) {
    float q = rintf(v * inv);
    const float d = fmaf(-q, scale, v), half = 0.5f * scale;
    const bool odd = (((int)q) & 1) != 0;
    if (d > half || (d == half && odd)) q += 1.0f;
    else if (d < -half || (d == -half && odd)) q -= 1.0f;
    return (int)q;
}
// Sixteen codes. Adding 1.5 * 2^23 rounds to an integer (ties to even) and leaves it, in two's
// complement, in the sum's low bits.
__device__ __forceinline__ uint4 codes16(const float (&v)[16], float scale, float inv) {
    constexpr float kRound = 12582912.0f;
    uint32_t c[16];
    float far = 0.0f;  // the largest distance from the chosen integer
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const float t = fmaf(v[j], inv, kRound);
        far = fmaxf(far, fabsf(fmaf(v[j], inv, kRound - t)));
        c[j] = __float_as_uint(t);
    }
    if (far > 0.4999f) {
#pragma unroll
        for (int j = 0; j < 16; ++j) c[j] = (uint32_t)code_of(v[j], scale, inv);
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // the low bytes of four codes
        w[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[4 * i + 3], c[4 * i + 2], 0x0C0C0400u),
                                     __builtin_amdgcn_perm(c[4 * i + 1], c[4 * i], 0x0C0C0400u), 0x05040100u);
    return uint4{w[0], w[1], w[2], w[3]};
}

// One block per row (kSort: per token, its row written to each of its kept sorted rows), 16
// elements per thread and turn, as many waves as one turn fills (at most four); the row stays in
// registers between its maximum and its codes, so that it is read once. Measured alone: 8192 rows of
// 4096 bf16 22.5 us (96 MiB, 4.5 TB/s; a block's loads, its maximum and its stores follow each other,
// and only the other blocks of the CU fill the gaps), 8192 rows of 2048 sorted to 65536 33 us (163 MiB,
// 5.2 TB/s).
template <class E, bool kSort, int kTurns>
__global__ __launch_bounds__(kRowThreads) void quantize_kernel(const E *x, const int32_t *rows, int K,
                                                               int n_rows, int8_t *q, float *scale) {
    __shared__ uint32_t s_max[kRowThreads / kWave];
    const int t = blockIdx.x, tid = threadIdx.x, nt = blockDim.x;
    float v[kTurns][16];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int h = (i * nt + tid) * 16;
        if (h < K) {
            float a[8], b[8];
            load8(x + (size_t)t * K + h, a);
            load8(x + (size_t)t * K + h + 8, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[i][j] = a[j];
                v[i][8 + j] = b[j];
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
        }
    }
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    if (nt > kWave) {  // uniform
        if ((tid & 63) == 0) s_max[tid >> 6] = m;
        __syncthreads();
        for (int i = 0; i < nt / kWave; ++i) m = max(m, s_max[i]);
    }
    const float sc = row_scale(m);
    const bool finite = m < 0x7F800000u;
    const float inv = 1.0f / sc;
    int r[kTopK];
    if constexpr (kSort) {
        token_rows(rows, t, n_rows, r);
        if (tid == 0) {
#pragma unroll
            for (int k = 0; k < kTopK; ++k)
                if (r[k] >= 0) scale[r[k]] = sc;
        }
    } else if (tid == 0) {
        scale[t] = sc;
    }
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
        const int h = (i * nt + tid) * 16;
        if (h >= K) continue;
        const uint4 c = finite ? codes16(v[i], sc, inv) : uint4{0, 0, 0, 0};
        if constexpr (kSort) {
#pragma unroll
            for (int k = 0; k < kTopK; ++k)
                if (r[k] >= 0) *reinterpret_cast<uint4 *>(q + (size_t)r[k] * K + h) = c;
        } else {
            *reinterpret_cast<uint4 *>(q + (size_t)t * K + h) = c;
        }
    }
}

}  // namespace

hipError_t launch_permute(const void *x, const int32_t *rows, int T, int H, int n_rows, int dtype,
                          void *xs, hipStream_t s) {
    auto go = [&](auto e, auto stream) {
        using E = decltype(e);
        launch_k(permute_kernel<E, decltype(stream)::value>, T, kRowThreads, 0, s, (const E *)x, rows, H,
                 n_rows, (E *)xs);
    };
    const bool stream = (size_t)T * kTopK * H * (dtype == 0 ? 4 : 2) >= kStreamBytes;
    if (dtype == 0) stream ? go(float{}, std::true_type{}) : go(float{}, std::false_type{});
    else stream ? go(uint16_t{}, std::true_type{}) : go(uint16_t{}, std::false_type{});
    return hipGetLastError();
}

hipError_t launch_unpermute(const UnpermuteParams &p, int dtype, int y_dtype, hipStream_t s) {
    auto go = [&](auto e, auto o) {
        using E = decltype(e);
        using O = decltype(o);
        if (p.w)
            launch_k(unpermute_kernel<E, O, true>, p.T, kRowThreads, 0, s, (const E *)p.ys, p.rows, p.w,
                     (const E *)p.shared, p.gate, p.H, p.n_rows, (O *)p.y);
        else if constexpr (std::is_same<E, O>::value)
            launch_k(unpermute_kernel<E, O, false>, p.T, kRowThreads, 0, s, (const E *)p.ys, p.rows, p.w,
                     (const E *)p.shared, p.gate, p.H, p.n_rows, (O *)p.y);
    };
    if (dtype == 0 && y_dtype == 0) go(float{}, float{});
    else if (dtype == 0) go(float{}, uint16_t{});
    else if (y_dtype == 0) go(uint16_t{}, float{});
    else go(uint16_t{}, uint16_t{});
    return hipGetLastError();
}

hipError_t launch_unpermute_backward(const UnpermuteBwdParams &p, int dtype, int y_dtype, hipStream_t s) {
    auto go = [&](auto e, auto o) {
        using E = decltype(e);
        using O = decltype(o);
        auto run = [&](auto stream) {
            launch_k(unpermute_bwd_kernel<E, O, decltype(stream)::value>, p.T, kRowThreads, 0, s,
                     (const O *)p.dy, (const E *)p.ys, p.rows, p.w, (const E *)p.shared, p.gate, p.H,
                     p.n_rows, (E *)p.dys, p.dw, (E *)p.dshared, p.dgate);
        };
        if ((size_t)p.T * kTopK * p.H * sizeof(E) >= kStreamBytes) run(std::true_type{});
        else run(std::false_type{});
    };
    if (dtype == 0 && y_dtype == 0) go(float{}, float{});
    else if (dtype == 0) go(float{}, uint16_t{});
    else if (y_dtype == 0) go(uint16_t{}, float{});
    else go(uint16_t{}, uint16_t{});
    return hipGetLastError();
}

hipError_t launch_quantize_i8(const void *x, const int32_t *rows, int n, int K, int n_rows, int dtype,
                              int8_t *q, float *scale, hipStream_t s) {
    const int units = K / 16, threads = units >= kRowThreads ? kRowThreads : (units + kWave - 1) / kWave * kWave;
    auto go = [&](auto e) {
        using E = decltype(e);
        auto run = [&](auto sort, auto turns) {
            launch_k(quantize_kernel<E, decltype(sort)::value, decltype(turns)::value>, n, threads, 0, s,
                     (const E *)x, rows, K, n_rows, q, scale);
        };
        using One = std::integral_constant<int, 1>;
        using Four = std::integral_constant<int, 4>;  // 256 threads x 16 elements x 4 = 16384
        if (units <= kRowThreads) rows ? run(std::true_type{}, One{}) : run(std::false_type{}, One{});
        else rows ? run(std::true_type{}, Four{}) : run(std::false_type{}, Four{});
    };
    if (dtype == 0) go(float{});
    else go(uint16_t{});
    return hipGetLastError();
}

}  // namespace moe
