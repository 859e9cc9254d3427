// balance.hip - what trains the router: the balance loss of a routing with its gradient, and the
// gradient of the selection's weights, both in the logits.
//
//   P[t] = softmax(z[t][0..E-1]);  c_e = pairs (t, k) with ids[t][k] = e;  N = counted tokens
//   L = E sum_e (c_e / 8N) (1/N sum_t P[t][e])
//   dL/dz[t][j] = E / N P[t][j] (f_j - sum_e f_e P[t][e]),  f_e = c_e / 8N
// sum_e P = 1, so that a number taken off all f_e changes nothing. The gradient is formed with the whole numbers d_e =
// c_e - floor(8N / E) in place of f_e (the shares of a nearly even routing are nearly 1 / E), and for each token the
// mean m = sum_e P d_e is taken off them, then what is left of it: P_j ((d_j - m) - sum_e P (d_e - m)). The
// rounding of m cancels in that, and a token that is sure of expert j keeps its small d_j - m: with m taken off once, u |d_j| is
// left in its place (a tenth of it at 1 - P_j = 1e-6).
//
//   w = softmax over the eight chosen logits, g = sigmoid(z[t][E]):
//   dz[t][ids_k] = w_k (dw_k - sum_j w_j dw_j);  dz[t][E] = g (1 - g) dg;  0 elsewhere
//
// All of them read or write the logits' array once and compute a few instructions per element: HBM
// bounds them for large T, a launch and one dependent chain for small ones. Measured (us; loss and gradient
// from Python one after the other): 192 tokens of 256 fp32 logits 18 (two launches), 8192 22 to 23 (three; 25 MB),
// 131072 of bf16 logits in padded sequences 54. On the GPU, after the caches were filled with other data, the
// latter is 23 for the sums (38 MB of the tokens that count; waits are 66 % of the waves' cycles: a pass asks for its
// logits when its mask has come back, two latencies behind each other), 7.6 for joining them, 30.6 for the
// gradient (the same 36 MB again, 67 MB of stores).
#include "device_common.h"
#include "kernels.h"
#include "select_core.h"

namespace moe {

namespace {

constexpr int kRowLanes = 16;  // lanes that share a token; a wave takes four tokens at a time
constexpr int kMaxE = 256;
constexpr int kBalWaves = 16;
constexpr int kBalTokens = kBalWaves * (kWave / kRowLanes);  // tokens of one pass of a block

// Sum and maximum over the 16 lanes of a token (every lane gets it), by lane moves in a fixed order.
__device__ __forceinline__ float row_sum(float v) {
    v += __uint_as_float(partner32<0>(__float_as_uint(v)));
    v += __uint_as_float(partner32<1>(__float_as_uint(v)));
    v += __uint_as_float(partner32<2>(__float_as_uint(v)));
    v += __uint_as_float(partner32<3>(__float_as_uint(v)));
    return v;
}
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, __uint_as_float(partner32<0>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(partner32<1>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(partner32<2>(__float_as_uint(v))));
    v = fmaxf(v, __uint_as_float(partner32<3>(__float_as_uint(v))));
    return v;
}

// A token's logits as the 16 lanes that share it hold them: kI for each. One by one (kV = 1: lane l holds experts
// l, l + 16, ...), or where rows begin on 16-byte boundaries in whole 16-byte pieces of kV experts.
template <class Z, int kI, int kV>
struct Logits {
    static constexpr int kPieces = kI / kV;
    using piece_t = typename std::conditional<kV == 1, Z, uint4>::type;
    piece_t v[kPieces];
    __device__ static __forceinline__ int expert(int i, int l) { return i / kV * kV * kRowLanes + l * kV + i % kV; }
    // nothing is read of a token that is not on, nor past the E experts' pieces
    __device__ __forceinline__ void load(const Z *z, bool on, int E, int l) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int e = expert(j * kV, l);
            v[j] = piece_t{};
            if (on && e < E) v[j] = *reinterpret_cast<const piece_t *>(z + e);
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (kV == 1) {
            if constexpr (sizeof(Z) == 4) return v[i];
            else return bf16_bits_to_f32(v[i]);
        } else {
            const uint4 &p = v[i / kV];
            const uint32_t w[4] = {p.x, p.y, p.z, p.w};
            if constexpr (sizeof(Z) == 4) return __uint_as_float(w[i % kV]);
            else return __uint_as_float(i % 2 ? w[i % kV / 2] & 0xFFFF0000u : w[i % kV / 2] << 16);
        }
    }
};

// The probabilities of the token. A token whose logits are all -infinity, or that is not on, has
// probabilities 0. A NaN among the logits, or a logit of +infinity, makes them NaN. 2^x of the rounded z
// log2(e): a probability e^-a carries a relative error of about a 2^-24 on top of the rounding of 2^x
// itself, less than a hundred steps where it is still a normal number, and next to none where it is large.
template <class Z, int kI, int kV>
__device__ __forceinline__ void token_probs(const Logits<Z, kI, kV> &z, bool on, int E, int l, float (&p)[kI]) {
    constexpr float kL2e = 1.44269502f;
    const float kNone = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kI; ++i) p[i] = on && Logits<Z, kI, kV>::expert(i, l) < E ? z.get(i) : kNone;
    float m = kNone;
#pragma unroll
    for (int i = 0; i < kI; ++i) m = fmaxf(m, p[i]);
    m = row_max(m);
    const bool none = m == kNone;
    const float base = none ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kI; ++i) {
        p[i] = __builtin_amdgcn_exp2f((p[i] - base) * kL2e);
        s += p[i];
    }
    s = row_sum(s);
    const float inv = none ? 0.0f : __builtin_amdgcn_rcpf(s);
#pragma unroll
    for (int i = 0; i < kI; ++i) p[i] *= inv;
}

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t *p, float v) { *p = (uint16_t)(pack_bf16(v, 0.0f) & 0xFFFFu); }
template <int kV, class Z>
__device__ __forceinline__ void put_piece(Z *p, const float *v) {
    if constexpr (kV == 1) put(p, v[0]);
    else if constexpr (kV == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint4 *>(p) =
            uint4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
}

// The loss from the sums of all tokens: thread e < E holds expert e's. For a block of whole waves.
__device__ __forceinline__ void write_loss(const BalanceParams &p, int e, double probs, int count, int tokens) {
    __shared__ double part[kBalWaves];
    const bool mine = e < p.E;
    const double n = tokens > 0 ? (double)tokens : 1.0;
    double v = mine ? (double)count * probs : 0.0;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) v += __shfl_xor(v, d, kWave);
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = v;
    if (mine) p.counts[e] = count;
    __syncthreads();
    if (threadIdx.x == 0) {
        double sum = 0.0;
        for (int i = 0; i < (int)blockDim.x / kWave; ++i) sum += part[i];
        *p.loss = (float)(sum * p.E / (kTopK * n * n));
        *p.tokens = tokens;
    }
}

// A block's share of the tokens: sums of their probabilities and counts of their pairs. One block: the
// loss at once; more: the block's row of the partial sums (balance_join_kernel adds them up in order). One block
// takes up to 512 tokens: a second launch costs about what its eight passes do (7.6 us for the join on its own, 11.2 for
// the one block over 192 tokens). 16 lanes a token keep a token's sums within lane moves of one row of lanes, and a
// block's 16 waves take 64 tokens a pass.
template <class Z, int kI, int kV>
__global__ __launch_bounds__(kBalWaves *kWave) void balance_kernel(BalanceParams p) {
    __shared__ float sums[kBalWaves][kMaxE];
    __shared__ int hist[kMaxE];
    __shared__ int counted;
    const int lane = lane_id(), wave = threadIdx.x / kWave, l = lane & (kRowLanes - 1), sub = lane / kRowLanes;
    if (threadIdx.x < kMaxE) hist[threadIdx.x] = 0;
    if (threadIdx.x == 0) counted = 0;
    const Z *z = reinterpret_cast<const Z *>(p.logits);
    float acc[kI] = {};
    int n = 0;
    // four tokens a wave, the next four's logits and ids on their way (lanes 0 .. 31: a pair each)
    using L = Logits<Z, kI, kV>;
    const int step = (int)gridDim.x * kBalTokens;
    auto counts = [&](int t) { return t < p.T && (!p.mask || p.mask[t]); };
    auto pair = [&](int t, uint64_t who) {
        const int k = t - sub + lane / kTopK;  // the pair's token
        return lane < 4 * kTopK && (who >> (lane / kTopK * kRowLanes) & 1) ? p.ids[(size_t)k * kTopK + (lane & (kTopK - 1))] : -1;
    };
    int t = blockIdx.x * kBalTokens + wave * (kWave / kRowLanes) + sub;
    bool on = counts(t);
    uint64_t who = __ballot(on);
    L cur;
    cur.load(z + (size_t)(on ? t : 0) * p.R, on, p.E, l);
    int id = pair(t, who);
    __syncthreads();
    while (t - sub < p.T) {  // uniform
        const int next = t + step;
        const bool non = counts(next);
        const uint64_t nwho = __ballot(non);
        L nxt;
        nxt.load(z + (size_t)(non ? next : 0) * p.R, non, p.E, l);
        const int nid = pair(next, nwho);
        if (who) {  // uniform: padding costs nothing
            float q[kI];
            token_probs(cur, on, p.E, l, q);
#pragma unroll
            for (int i = 0; i < kI; ++i) acc[i] += q[i];
            if (id >= 0 && id < p.E) atomicAdd(&hist[id], 1);
            n += __popcll(who) / kRowLanes;
        }
        t = next;
        on = non;
        who = nwho;
        id = nid;
        cur = nxt;
    }
    if (lane == 0) atomicAdd(&counted, n);
#pragma unroll
    for (int i = 0; i < kI; ++i) {  // the wave's four tokens' lanes
        acc[i] += __uint_as_float(partner32<4>(__float_as_uint(acc[i])));
        acc[i] += __uint_as_float(partner32<5>(__float_as_uint(acc[i])));
        if (lane < kRowLanes) sums[wave][L::expert(i, l)] = acc[i];
    }
    __syncthreads();
    const int e = threadIdx.x;
    const bool mine = e < p.E;
    double s = 0.0;
    if (mine)
#pragma unroll
        for (int w = 0; w < kBalWaves; ++w) s += (double)sums[w][e];
    if (gridDim.x == 1) {
        write_loss(p, e, s, mine ? hist[e] : 0, counted);
        return;
    }
    if (mine) {
        p.part[(size_t)blockIdx.x * p.E + e] = (float)s;
        p.part_counts[(size_t)blockIdx.x * p.E + e] = hist[e];
    }
    if (threadIdx.x == 0) p.part_tokens[blockIdx.x] = counted;
}

// The blocks' sums, joined in order, and the loss. (Four experts a thread and 16 rows at a time take longer: 10.1 us
// against 7.6 for 128 rows, both after the caches were filled with other data.)
__global__ __launch_bounds__(4 * kMaxE) void balance_join_kernel(BalanceParams p) {
    __shared__ double sums[3][kMaxE];
    __shared__ int counts[3][kMaxE];
    __shared__ int counted;
    const int e = threadIdx.x & (kMaxE - 1), g = threadIdx.x / kMaxE;
    if (threadIdx.x == 0) counted = 0;
    __syncthreads();
    double s = 0.0;
    int c = 0;
    if (e < p.E)
#pragma unroll 16
        for (int b = g; b < p.blocks; b += 4) {
            s += (double)p.part[(size_t)b * p.E + e];
            c += p.part_counts[(size_t)b * p.E + e];
        }
    for (int b = threadIdx.x; b < p.blocks; b += 4 * kMaxE) atomicAdd(&counted, p.part_tokens[b]);
    if (g > 0) sums[g - 1][e] = s, counts[g - 1][e] = c;
    __syncthreads();
    if (g == 0)
#pragma unroll
        for (int i = 0; i < 3; ++i) s += sums[i][e], c += counts[i][e];
    write_loss(p, g == 0 ? e : kMaxE, s, c, counted);
}

// dlogits, 16 lanes a token; columns past the experts and tokens that do not count get 0. At most four blocks per
// CU (what its registers hold at once), each walking its tokens: 131072 bf16 tokens with padding 27 us, with 2048
// blocks 31, with 4096 41 (all before the mean was taken off twice, which takes 2 to 3).
template <class Z, int kI, int kV>
__global__ __launch_bounds__(256) void balance_backward_kernel(BalanceBwdParams p) {
    const int lane = lane_id(), l = lane & (kRowLanes - 1), per = 256 / kRowLanes;
    const Z *z = reinterpret_cast<const Z *>(p.logits);
    Z *dz = reinterpret_cast<Z *>(p.dlogits);
    // the next token's logits on their way, the first while the counts come
    using L = Logits<Z, kI, kV>;
    auto counts = [&](int64_t t) { return t < p.T && (!p.mask || p.mask[t]); };
    int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / kRowLanes;
    bool on = counts(t);
    L cur;
    cur.load(z + (size_t)(t < p.T ? t : 0) * p.R, on, p.E, l);
    const int n = *p.tokens;
    int c[kI];  // (without branches: all of them on their way at once)
#pragma unroll
    for (int i = 0; i < kI; ++i) c[i] = p.counts[min(L::expert(i, l), p.E - 1)];
    float d[kI];
    const double even = floor((double)kTopK * n / p.E);
#pragma unroll
    for (int i = 0; i < kI; ++i)  // whole numbers, exact below 2^24
        d[i] = L::expert(i, l) < p.E ? (float)((double)c[i] - even) : 0.0f;
    const float factor = n > 0 ? (float)((double)*p.dloss * p.E / ((double)kTopK * n * n)) : 0.0f;
    while (t - lane / kRowLanes < p.T) {  // uniform
        const int64_t next = t + (int64_t)gridDim.x * per;
        const bool there = t < p.T, non = counts(next);
        L nxt;
        nxt.load(z + (size_t)(next < p.T ? next : 0) * p.R, non, p.E, l);
        const size_t at = (size_t)(there ? t : 0) * p.R;
        float q[kI] = {}, mean = 0.0f, rest = 0.0f;
        if (__any(on)) {  // padding is only cleared
            token_probs(cur, on, p.E, l, q);
#pragma unroll
            for (int i = 0; i < kI; ++i) mean = fmaf(q[i], d[i], mean);
            mean = row_sum(mean);
#pragma unroll
            for (int i = 0; i < kI; ++i) rest = fmaf(q[i], d[i] - mean, rest);
            rest = row_sum(rest);
        }
        if (there) {
#pragma unroll
            for (int i = 0; i < kI; ++i) q[i] = on ? factor * (q[i] * ((d[i] - mean) - rest)) : 0.0f;
#pragma unroll
            for (int i = 0; i < kI; i += kV) {
                const int e = L::expert(i, l);
                if (e + kV <= p.E) put_piece<kV>(dz + at + e, q + i);
                else
#pragma unroll
                    for (int k = 0; k < kV; ++k)
                        if (e + k < p.E) put(dz + at + e + k, q[i + k]);
            }
            for (int c = p.E + l; c < p.R; c += kRowLanes) put(dz + at + c, 0.0f);
        }
        t = next;
        on = non;
        cur = nxt;
    }
}

// The gradient of the selection's weights: a block builds the rows of kSelTokens tokens in LDS and
// stores them as one aligned run. Eight lanes a token, one per rank; an expert that a token names more
// than once takes the sum of its ranks, in order. The stores bound it: 131072 tokens of 257 columns 26.8 us
// (135 MB of them, 5.5 TB/s with the reads). 32 tokens are whole waves' worth of lanes, and their R 4 bytes begin every block's
// run on a multiple of 16 whatever R is.
constexpr int kSelTokens = 32;
__global__ __launch_bounds__(kSelTokens *kTopK) void select_backward_kernel(SelectBwdParams p) {
    __shared__ __align__(16) float rows[kSelTokens * (kMaxE + 1)];
    const int R = p.E + (p.gate ? 1 : 0), tid = threadIdx.x;
    const int t0 = blockIdx.x * kSelTokens, n = min(kSelTokens, p.T - t0);
    const int k = tid & (kTopK - 1), j = tid / kTopK;
    const bool on = j < n;
    const size_t pair = (size_t)t0 * kTopK + tid;
    const float w = on ? p.w[pair] : 0.0f, dw = on ? p.dw[pair] : 0.0f;
    const int id = on ? p.ids[pair] : -1;
    const float g = on && k == 0 && p.gate ? p.gate[t0 + j] : 0.0f;
    const float dg = on && k == 0 && p.gate ? p.dgate[t0 + j] : 0.0f;
    for (int i = tid * 4; i < kSelTokens * R; i += kSelTokens * kTopK * 4)
        *reinterpret_cast<float4 *>(rows + i) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float dot = w * dw;
    dot += __uint_as_float(partner32<0>(__float_as_uint(dot)));
    dot += __uint_as_float(partner32<1>(__float_as_uint(dot)));
    dot += __uint_as_float(partner32<2>(__float_as_uint(dot)));
    const float v = w * (dw - dot);
    float sum = 0.0f;
    bool first = true;
#pragma unroll
    for (int r = 0; r < kTopK; ++r) {
        const bool same = __shfl(id, r, kTopK) == id;
        const float o = __shfl(v, r, kTopK);
        if (same) sum += o;
        if (same && r < k) first = false;
    }
    __syncthreads();
    if (on && first && id >= 0 && id < p.E) rows[j * R + id] = sum;
    if (on && k == 0 && p.gate) rows[j * R + p.E] = g * (1.0f - g) * dg;
    __syncthreads();
    float *out = p.dlogits + (size_t)t0 * R;  // t0 R 4 bytes: a multiple of 16
    const int total = n * R;
    for (int i = tid * 4; i + 4 <= total; i += kSelTokens * kTopK * 4)
        *reinterpret_cast<float4 *>(out + i) = *reinterpret_cast<const float4 *>(rows + i);
    const int rest = total & ~3;
    if (rest + tid < total) out[rest + tid] = rows[rest + tid];
}

// logits type, elements per lane and how they are taken: in whole pieces where rows of both arrays begin on their boundaries
template <class Go>
void typed(int dtype, int E, int R, const void *one, const void *two, Go go) {
    const int bytes = dtype == 0 ? 4 : 2;
    const bool whole = (size_t)R * bytes % 16 == 0 && (uintptr_t)one % 16 == 0 && (uintptr_t)two % 16 == 0;
    auto wide = [&](auto z, auto kv) {
        if (E <= 64 && decltype(kv)::value <= 4) {
            if constexpr (decltype(kv)::value <= 4) go(z, std::integral_constant<int, 4>{}, kv);
        } else if (E <= 128) go(z, std::integral_constant<int, 8>{}, kv);
        else go(z, std::integral_constant<int, 16>{}, kv);
    };
    using V1 = std::integral_constant<int, 1>;
    using V4 = std::integral_constant<int, 4>;
    using V8 = std::integral_constant<int, 8>;
    if (dtype == 0) whole ? wide(float{}, V4{}) : wide(float{}, V1{});
    else whole ? wide(uint16_t{}, V8{}) : wide(uint16_t{}, V1{});
}

}  // namespace

int balance_blocks(int T) {
    const int one = 8 * kBalTokens;  // up to here the block does all in one launch
    if (T <= one) return 1;
    // a block per CU: 131072 tokens of bf16 logits 22.6 us and 7.6 for the join, with twice the blocks 25.5 and 12.9
    const int b = (T + kBalTokens - 1) / kBalTokens;
    return b < 256 ? b : 256;
}

hipError_t launch_balance(const BalanceParams &p, int dtype, hipStream_t s) {
    typed(dtype, p.E, p.R, p.logits, nullptr, [&](auto z, auto ki, auto kv) {
        launch_k(balance_kernel<decltype(z), decltype(ki)::value, decltype(kv)::value>, p.blocks, kBalWaves * kWave, 0, s, p);
    });
    if (p.blocks > 1) launch_k(balance_join_kernel, 1, 4 * kMaxE, 0, s, p);
    return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceBwdParams &p, int dtype, hipStream_t s) {
    const int per = 256 / kRowLanes, all = (p.T + per - 1) / per;
    typed(dtype, p.E, p.R, p.logits, p.dlogits, [&](auto z, auto ki, auto kv) {
        launch_k(balance_backward_kernel<decltype(z), decltype(ki)::value, decltype(kv)::value>, all < 1024 ? all : 1024, 256, 0, s, p);
    });
    return hipGetLastError();
}

hipError_t launch_select_backward(const SelectBwdParams &p, hipStream_t s) {
    launch_k(select_backward_kernel, (p.T + kSelTokens - 1) / kSelTokens, kSelTokens * kTopK, 0, s, p);
    return hipGetLastError();
}

}  // namespace moe
