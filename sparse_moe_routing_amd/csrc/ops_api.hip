// ops_api.hip - the C ABI of the separate row operators, the products with 8-bit and 4-bit weights and
// the router's training operators (include/moe.h): argument checks, all on the host before anything is enqueued.
#include <initializer_list>

#include "../../include/moe.h"
#include "device_common.h"
#include "kernels.h"

using namespace moe;

namespace {

constexpr int kMaxTokens = 1 << 20;
constexpr int kMaxRows = kMaxTokens * 8;
constexpr int kMaxWidth = 16384;
constexpr int kMaxChannels = 65536;
constexpr int kMaxExperts = 256;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool row_dtype(int d) { return d == MOE_F32 || d == MOE_BF16; }
int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// MOE_OK, or why T tokens with rows of `width` elements in n_rows sorted rows are refused.
int check_shape(int32_t T, int32_t n_rows, int32_t width, int multiple) {
    if (T < 0 || n_rows < 0) return MOE_ERR_INVALID_ARG;
    if (T > kMaxTokens || n_rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (width < multiple || width > kMaxWidth || width % multiple) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// A matrix that is touched: there and 16-byte aligned. One without rows may be NULL.
bool rows_ok(const void *p, int32_t n) { return aligned(p, 16) && (p || n == 0); }
// A table or vector that is touched: there and 4-byte aligned.
bool vec_ok(const void *p, int32_t n = 1) { return aligned(p, 4) && (p || n == 0); }

// Logits, which the kernels take element by element: there and aligned to one.
bool logits_ok(const void *p, int32_t T, int dtype) { return aligned(p, dtype == MOE_F32 ? 4 : 2) && (p || T == 0); }

// n bytes at p; an operand that is not given takes none.
struct Span {
    uintptr_t at;
    size_t n;
    Span(const void *p, size_t bytes) : at((uintptr_t)p), n(p ? bytes : 0) {}
    bool meets(const Span &o) const { return n && o.n && at < o.at + o.n && o.at < at + n; }
};
// No output shares a byte with an input or another output.
bool apart(std::initializer_list<Span> out, std::initializer_list<Span> in) {
    for (const Span *o = out.begin(); o != out.end(); ++o) {
        for (const Span &i : in)
            if (o->meets(i)) return false;
        for (const Span *q = out.begin(); q != o; ++q)
            if (o->meets(*q)) return false;
    }
    return true;
}
size_t row_bytes(int32_t n, int32_t width, int dtype) { return (size_t)n * width * (dtype == MOE_F32 ? 4 : 2); }
size_t pair_bytes(int32_t T) { return (size_t)T * 32; }  // a table of T * 8 entries of 4 bytes

// The same for T tokens' logits [T][R] over E experts.
int check_router(int32_t T, int32_t E, int32_t R, int32_t dtype) {
    if (T < 0 || R < E || !row_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    if (T > kMaxTokens || E < kTopK || E > kMaxExperts || R > kMaxWidth) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int unpermute_impl(const void *ys, const int32_t *rows, const float *w, const void *shared,
                   const float *gate, int32_t T, int32_t H, int32_t n_rows, int32_t dtype, void *y,
                   int32_t y_dtype, hipStream_t stream) {
    const int st = check_shape(T, n_rows, H, 8);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!vec_ok(rows) || !rows_ok(ys, n_rows) || !rows_ok(y, T)) return MOE_ERR_INVALID_ARG;
    if (!aligned(w, 4) || (shared != nullptr) != (gate != nullptr) || !aligned(shared, 16) ||
        !aligned(gate, 4))
        return MOE_ERR_INVALID_ARG;
    if (!apart({{y, row_bytes(T, H, y_dtype)}},
               {{ys, row_bytes(n_rows, H, dtype)}, {rows, pair_bytes(T)}, {w, pair_bytes(T)},
                {shared, row_bytes(T, H, dtype)}, {gate, (size_t)T * 4}}))
        return MOE_ERR_INVALID_ARG;
    const UnpermuteParams p{ys, rows, w, shared, gate, y, T, H, n_rows};
    return hip_status(launch_unpermute(p, dtype, y_dtype, stream));
}

}  // namespace

extern "C" {

int moe_permute(const void *x, const int32_t *rows, int32_t T, int32_t H, int32_t n_rows,
                int32_t dtype, void *xs, hipStream_t stream) {
    if (!row_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const int st = check_shape(T, n_rows, H, 8);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!vec_ok(rows) || !rows_ok(x, T) || !rows_ok(xs, n_rows)) return MOE_ERR_INVALID_ARG;
    if (n_rows == 0) return MOE_OK;
    if (!apart({{xs, row_bytes(n_rows, H, dtype)}}, {{x, row_bytes(T, H, dtype)}, {rows, pair_bytes(T)}}))
        return MOE_ERR_INVALID_ARG;
    return hip_status(launch_permute(x, rows, T, H, n_rows, dtype, xs, stream));
}

int moe_permute_backward(const void *dxs, const int32_t *rows, int32_t T, int32_t H,
                         int32_t n_rows, int32_t dtype, void *dx, hipStream_t stream) {
    if (!row_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    return unpermute_impl(dxs, rows, nullptr, nullptr, nullptr, T, H, n_rows, dtype, dx, dtype,
                          stream);
}

int moe_unpermute(const void *ys, const int32_t *rows, const float *w, const void *shared,
                  const float *gate, int32_t T, int32_t H, int32_t n_rows, int32_t dtype, void *y,
                  int32_t y_dtype, hipStream_t stream) {
    if (!row_dtype(dtype) || !row_dtype(y_dtype) || (T > 0 && !w)) return MOE_ERR_INVALID_ARG;
    return unpermute_impl(ys, rows, w, shared, gate, T, H, n_rows, dtype, y, y_dtype, stream);
}

int moe_unpermute_backward(const void *dy, const void *ys, const int32_t *rows, const float *w,
                           const void *shared, const float *gate, int32_t T, int32_t H,
                           int32_t n_rows, int32_t dtype, int32_t y_dtype, void *dys, float *dw,
                           void *dshared, float *dgate, hipStream_t stream) {
    if (!row_dtype(dtype) || !row_dtype(y_dtype)) return MOE_ERR_INVALID_ARG;
    const int st = check_shape(T, n_rows, H, 8);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!rows_ok(dy, T) || !rows_ok(ys, n_rows) || !rows_ok(dys, n_rows) || !vec_ok(rows) ||
        !vec_ok(w) || !vec_ok(dw))
        return MOE_ERR_INVALID_ARG;
    const bool sh = shared != nullptr;
    if (sh != (gate != nullptr) || sh != (dshared != nullptr) || sh != (dgate != nullptr) ||
        !aligned(shared, 16) || !aligned(dshared, 16) || !aligned(gate, 4) || !aligned(dgate, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t sorted = row_bytes(n_rows, H, dtype), tokens = row_bytes(T, H, dtype);
    if (!apart({{dys, sorted}, {dw, pair_bytes(T)}, {dshared, tokens}, {dgate, (size_t)T * 4}},
               {{dy, row_bytes(T, H, y_dtype)}, {ys, sorted}, {rows, pair_bytes(T)}, {w, pair_bytes(T)},
                {shared, tokens}, {gate, (size_t)T * 4}}))
        return MOE_ERR_INVALID_ARG;
    const UnpermuteBwdParams p{dy, ys, rows, w, shared, gate, dys, dw, dshared, dgate, T, H, n_rows};
    return hip_status(launch_unpermute_backward(p, dtype, y_dtype, stream));
}

int moe_quantize_i8(const void *x, int32_t n, int32_t K, int32_t dtype, int8_t *q, float *scale,
                    hipStream_t stream) {
    if (!row_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const int st = check_shape(0, n, K, 16);
    if (st != MOE_OK) return st;
    if (n == 0) return MOE_OK;
    if (!rows_ok(x, n) || !rows_ok(q, n) || !vec_ok(scale)) return MOE_ERR_INVALID_ARG;
    if (!apart({{q, (size_t)n * K}, {scale, (size_t)n * 4}}, {{x, row_bytes(n, K, dtype)}}))
        return MOE_ERR_INVALID_ARG;
    return hip_status(launch_quantize_i8(x, nullptr, n, K, n, dtype, q, scale, stream));
}

int moe_permute_i8(const void *x, const int32_t *rows, int32_t T, int32_t H, int32_t n_rows,
                   int32_t dtype, int8_t *xs, float *xs_scale, hipStream_t stream) {
    if (!row_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    const int st = check_shape(T, n_rows, H, 16);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!vec_ok(rows) || !rows_ok(x, T) || !rows_ok(xs, n_rows) || !vec_ok(xs_scale, n_rows))
        return MOE_ERR_INVALID_ARG;
    if (n_rows == 0) return MOE_OK;
    if (!apart({{xs, (size_t)n_rows * H}, {xs_scale, (size_t)n_rows * 4}},
               {{x, row_bytes(T, H, dtype)}, {rows, pair_bytes(T)}}))
        return MOE_ERR_INVALID_ARG;
    return hip_status(launch_quantize_i8(x, rows, T, H, n_rows, dtype, xs, xs_scale, stream));
}

int moe_matmul_i8(const int8_t *x, const float *x_scale, int32_t n_rows, const int8_t *w,
                  const float *w_scale, int32_t E, int32_t M, int32_t K, const int32_t *offsets,
                  int32_t swiglu, void *y, int32_t y_dtype, hipStream_t stream) {
    if (!row_dtype(y_dtype) || (swiglu != 0 && swiglu != 1)) return MOE_ERR_INVALID_ARG;
    const int st = check_shape(0, n_rows, K, 16);
    if (st != MOE_OK) return st;
    const int m = swiglu ? 16 : 8;
    if (E < 1 || E > kMaxExperts || M < m || M > kMaxChannels || M % m) return MOE_ERR_UNSUPPORTED;
    if (!offsets && E != 1) return MOE_ERR_INVALID_ARG;
    if (n_rows == 0) return MOE_OK;
    if (!rows_ok(x, n_rows) || !vec_ok(x_scale) || !rows_ok(w, 1) || !vec_ok(w_scale) ||
        !aligned(offsets, 4) || !rows_ok(y, n_rows))
        return MOE_ERR_INVALID_ARG;
    if (!apart({{y, row_bytes(n_rows, swiglu ? M / 2 : M, y_dtype)}},
               {{x, (size_t)n_rows * K}, {x_scale, (size_t)n_rows * 4}, {w, (size_t)E * M * K},
                {w_scale, (size_t)E * M * 4}, {offsets, (size_t)(E + 1) * 4}}))
        return MOE_ERR_INVALID_ARG;
    const I8Params p{x, x_scale, w, w_scale, offsets, y, n_rows, E, M, K, 0};
    return hip_status(launch_matmul_i8(p, swiglu != 0, y_dtype, stream));
}

int moe_matmul_w4(const void *x, int32_t n_rows, int32_t dtype, const uint8_t *w, const void *scale,
                  int32_t scale_dtype, const uint8_t *zero, int32_t E, int32_t M, int32_t K, int32_t group,
                  const int32_t *offsets, int32_t swiglu, void *y, int32_t y_dtype, hipStream_t stream) {
    if (!row_dtype(dtype) || !row_dtype(scale_dtype) || !row_dtype(y_dtype) || (swiglu != 0 && swiglu != 1))
        return MOE_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return MOE_ERR_UNSUPPORTED;
    const int st = check_shape(0, n_rows, K, group);
    if (st != MOE_OK) return st;
    const int m = swiglu ? 16 : 8;
    if (E < 1 || E > kMaxExperts || M < m || M > kMaxChannels || M % m) return MOE_ERR_UNSUPPORTED;
    if (!offsets && E != 1) return MOE_ERR_INVALID_ARG;
    if (n_rows == 0) return MOE_OK;
    if (!rows_ok(x, n_rows) || !rows_ok(w, 1) || !rows_ok(scale, 1) || !aligned(zero, 16) || !aligned(offsets, 4) ||
        !rows_ok(y, n_rows))
        return MOE_ERR_INVALID_ARG;
    const size_t groups = (size_t)E * M * (K / group);
    if (!apart({{y, row_bytes(n_rows, swiglu ? M / 2 : M, y_dtype)}},
               {{x, row_bytes(n_rows, K, dtype)}, {w, (size_t)E * M * K / 2},
                {scale, groups * (scale_dtype == MOE_F32 ? 4 : 2)}, {zero, groups},
                {offsets, (size_t)(E + 1) * 4}}))
        return MOE_ERR_INVALID_ARG;
    const W4Params p{x, w, scale, zero, offsets, y, n_rows, E, M, K, group, scale_dtype == MOE_F32, y_dtype == MOE_F32, swiglu, 0};
    return hip_status(launch_matmul_w4(p, dtype, stream));
}

size_t moe_balance_workspace_bytes(int32_t T, int32_t E) {
    if (T < 0 || T > kMaxTokens || E < 1 || E > kMaxExperts) return 0;
    const int blocks = balance_blocks(T);
    return blocks > 1 ? (size_t)blocks * (2 * E + 1) * 4 : 0;
}

int moe_balance_loss(const void *logits, const int32_t *ids, const uint8_t *mask, int32_t T, int32_t E, int32_t R,
                     int32_t dtype, float *loss, int32_t *counts, int32_t *tokens, void *workspace,
                     size_t ws_bytes, hipStream_t stream) {
    const int st = check_router(T, E, R, dtype);
    if (st != MOE_OK) return st;
    if (!logits_ok(logits, T, dtype) || !vec_ok(ids, T) || !vec_ok(loss) || !vec_ok(counts) || !vec_ok(tokens))
        return MOE_ERR_INVALID_ARG;
    const size_t need = moe_balance_workspace_bytes(T, E);
    if (need && (!workspace || !aligned(workspace, 4) || ws_bytes < need)) return MOE_ERR_WORKSPACE;
    const Span ws(workspace, need);
    if (!apart({{loss, 4}, {counts, (size_t)E * 4}, {tokens, 4}, ws},
               {{logits, row_bytes(T, R, dtype)}, {ids, pair_bytes(T)}, {mask, (size_t)T}}))
        return MOE_ERR_INVALID_ARG;
    const int blocks = balance_blocks(T);
    float *part = (float *)workspace;
    int32_t *part_counts = (int32_t *)(part + (size_t)blocks * E);
    const BalanceParams p{logits, ids, mask, loss, counts, tokens, part, part_counts,
                          part_counts + (size_t)blocks * E, T, E, R, blocks};
    return hip_status(launch_balance(p, dtype, stream));
}

int moe_balance_loss_backward(const float *dloss, const void *logits, const int32_t *counts, const int32_t *tokens,
                              const uint8_t *mask, int32_t T, int32_t E, int32_t R, int32_t dtype, void *dlogits,
                              hipStream_t stream) {
    const int st = check_router(T, E, R, dtype);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!vec_ok(dloss) || !logits_ok(logits, T, dtype) || !vec_ok(counts) || !vec_ok(tokens) ||
        !logits_ok(dlogits, T, dtype))
        return MOE_ERR_INVALID_ARG;
    const size_t all = row_bytes(T, R, dtype);
    if (!apart({{dlogits, all}},
               {{dloss, 4}, {logits, all}, {counts, (size_t)E * 4}, {tokens, 4}, {mask, (size_t)T}}))
        return MOE_ERR_INVALID_ARG;
    const BalanceBwdParams p{dloss, logits, counts, tokens, mask, dlogits, T, E, R};
    return hip_status(launch_balance_backward(p, dtype, stream));
}

int moe_route_backward(const float *dw, const float *w, const int32_t *ids, const float *dgate, const float *gate,
                       int32_t T, int32_t E, float *dlogits, hipStream_t stream) {
    const int st = check_router(T, E, E, MOE_F32);
    if (st != MOE_OK) return st;
    if ((gate != nullptr) != (dgate != nullptr)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!vec_ok(dw) || !vec_ok(w) || !vec_ok(ids) || !aligned(gate, 4) || !aligned(dgate, 4) || !rows_ok(dlogits, T))
        return MOE_ERR_INVALID_ARG;
    if (!apart({{dlogits, row_bytes(T, E + (gate ? 1 : 0), MOE_F32)}},
               {{dw, pair_bytes(T)}, {w, pair_bytes(T)}, {ids, pair_bytes(T)}, {dgate, (size_t)T * 4},
                {gate, (size_t)T * 4}}))
        return MOE_ERR_INVALID_ARG;
    const SelectBwdParams p{dw, w, ids, dgate, gate, dlogits, T, E};
    return hip_status(launch_select_backward(p, stream));
}

}  // extern "C"
