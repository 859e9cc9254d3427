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
// latency of one dependent chain (table entry, row, result) at decode.
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
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = uint4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                          pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

// The eight sorted rows of token t; -1 for an entry outside [0, n_rows).
__device__ __forceinline__ void token_rows(const int32_t *rows, int t, int n_rows, int (&r)[kTopK]) {
#pragma unroll
    for (int k = 0; k < kTopK; ++k) {
        const int v = rows[(size_t)t * kTopK + k];
        r[k] = v >= 0 && v < n_rows ? v : -1;
    }
}

// One block per token.
template <class E>
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
            if (r[k] >= 0) *reinterpret_cast<uint4 *>(xs + (size_t)r[k] * H + h) = v;
    }
}

// kWeighted: unpermute (weights, optional shared row); otherwise permute_backward.
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
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, v[8];
#pragma unroll
        for (int k = 0; k < kTopK; ++k) {
            if (r[k] < 0) continue;
            load8(ys + (size_t)r[k] * H + h, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = kWeighted ? fmaf(wk[k], v[i], acc[i]) : acc[i] + v[i];
        }
        if (kWeighted && shared) {
            load8(shared + (size_t)t * H + h, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(g, v[i], acc[i]);
        }
        store8(y + (size_t)t * H + h, acc);
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

template <class E, class O>
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
        float d[8], v[8];
        load8(dy + (size_t)t * H + h, d);
#pragma unroll
        for (int k = 0; k < kTopK; ++k) {
            if (r[k] < 0) continue;
            load8(ys + (size_t)r[k] * H + h, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[k] = fmaf(d[i], v[i], dot[k]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = wk[k] * d[i];
            store8(dys + (size_t)r[k] * H + h, v);
        }
        if (shared) {
            load8(shared + (size_t)t * H + h, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[kTopK] = fmaf(d[i], v[i], dot[kTopK]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = g * d[i];
            store8(dshared + (size_t)t * H + h, v);
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
// the exact quotient v / scale: q = rint(v * (1 / scale)) is at most one off, and the residual
// v - q * scale, one fused operation, is exact next to a half (q has 8 bits, the difference cancels),
// so comparing it with scale / 2 settles the rounding, ties to even. Halves are common here: with
// bf16 rows v / amax has few bits, and 127 v / amax often ends in exactly .5.
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

// One block per row (kSort: per token, its row written to each of its kept sorted rows), 16
// elements per thread and turn; the row stays in registers between its maximum and its codes.
constexpr int kQTurns = 4;  // 256 threads x 16 elements x 4 = 16384
template <class E, bool kSort>
__global__ __launch_bounds__(kRowThreads) void quantize_kernel(const E *x, const int32_t *rows, int K,
                                                               int n_rows, int8_t *q, float *scale) {
    __shared__ uint32_t s_max[kRowThreads / kWave];
    const int t = blockIdx.x, tid = threadIdx.x;
    float v[kQTurns][2][8];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kQTurns; ++i) {
        const int h = (i * kRowThreads + tid) * 16;
        if (h < K) {
            load8(x + (size_t)t * K + h, v[i][0]);
            load8(x + (size_t)t * K + h + 8, v[i][1]);
#pragma unroll
            for (int j = 0; j < 16; ++j) m = max(m, __float_as_uint(v[i][j >> 3][j & 7]) & 0x7FFFFFFFu);
        }
    }
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    if ((tid & 63) == 0) s_max[tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRowThreads / kWave; ++i) m = max(m, s_max[i]);
    const float sc = row_scale(m);
    const bool finite = m < 0x7F800000u;
    const float inv = 1.0f / sc;
    int r[kTopK];
    if constexpr (kSort) {
        token_rows(rows, t, n_rows, r);
        if (tid < kTopK && r[tid & 7] >= 0) scale[r[tid & 7]] = sc;
    } else if (tid == 0) {
        scale[t] = sc;
    }
#pragma unroll
    for (int i = 0; i < kQTurns; ++i) {
        const int h = (i * kRowThreads + tid) * 16;
        if (h >= K) continue;
        uint32_t w[4] = {0, 0, 0, 0};
        if (finite) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                w[j >> 2] |= ((uint32_t)code_of(v[i][j >> 3][j & 7], sc, inv) & 0xFFu) << (8 * (j & 3));
        }
        const uint4 c = uint4{w[0], w[1], w[2], w[3]};
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
    if (dtype == 0)
        launch_k(permute_kernel<float>, T, kRowThreads, 0, s, (const float *)x, rows, H, n_rows, (float *)xs);
    else
        launch_k(permute_kernel<uint16_t>, T, kRowThreads, 0, s, (const uint16_t *)x, rows, H, n_rows,
                 (uint16_t *)xs);
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
        launch_k(unpermute_bwd_kernel<E, O>, p.T, kRowThreads, 0, s, (const O *)p.dy, (const E *)p.ys,
                 p.rows, p.w, (const E *)p.shared, p.gate, p.H, p.n_rows, (E *)p.dys, p.dw,
                 (E *)p.dshared, p.dgate);
    };
    if (dtype == 0 && y_dtype == 0) go(float{}, float{});
    else if (dtype == 0) go(float{}, uint16_t{});
    else if (y_dtype == 0) go(uint16_t{}, float{});
    else go(uint16_t{}, uint16_t{});
    return hipGetLastError();
}

hipError_t launch_quantize_i8(const void *x, const int32_t *rows, int n, int K, int n_rows, int dtype,
                              int8_t *q, float *scale, hipStream_t s) {
    auto go = [&](auto e) {
        using E = decltype(e);
        if (rows)
            launch_k(quantize_kernel<E, true>, n, kRowThreads, 0, s, (const E *)x, rows, K, n_rows, q, scale);
        else
            launch_k(quantize_kernel<E, false>, n, kRowThreads, 0, s, (const E *)x, rows, K, n_rows, q, scale);
    };
    if (dtype == 0) go(float{});
    else go(uint16_t{});
    return hipGetLastError();
}

}  // namespace moe
