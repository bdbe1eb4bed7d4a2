// C ABI of the training steps: argument checks, workspace and launch order.
#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "abi_checks.h"
#include "internal.h"

using namespace moe;

namespace {

bool all_aligned(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned16(p)) return false;
    return true;
}

const bf16* in16(const moe_bf16* p) { return reinterpret_cast<const bf16*>(p); }
bf16* out16(moe_bf16* p) { return reinterpret_cast<bf16*>(p); }

int check_status_ws(const void* ws, size_t ws_bytes) {
    if (!ws || !aligned16(ws)) return MOE_EINVAL;
    return ws_bytes < MOE_STATUS_BYTES ? MOE_EWORKSPACE : MOE_OK;
}

int check_norm(int64_t T, int d) {
    if (T < 1 || T > kMaxT || d < 16 || d > (1 << 16)) return MOE_EINVAL;
    return layernorm_supported(d) ? MOE_OK : MOE_EUNSUPPORTED;
}

// Workspace of moe_route_backward.  The weight's gradient is summed over S
// chunks of tokens, each a group of the grouped product, so that the
// ceil(d / 256) row tiles of a narrow output still occupy the SMs.
struct RouteLayout {
    int ld, S;
    int64_t chunk;
    size_t dl, wr, part, total;
};

RouteLayout route_layout(const moe_dims* d) {
    RouteLayout L{};
    L.ld = (d->E + 7) / 8 * 8;
    const int m_tiles = (d->d_model + 255) / 256;
    const int pairs = (num_sms() > 0 ? num_sms() : 148) / 2;
    // two rounds of tiles for a narrow weight (E = 8, d = 4096: 144 tiles on 74 pairs;
    // one round of 64 left a seventh of them idle), one where the partial sums are large;
    // at most 16 chunks, so below d = 2304 fewer tiles than that
    int64_t S = (L.ld <= 64 ? 2 * pairs : pairs) / m_tiles;
    const int64_t most = (d->T + 255) / 256;  // at least 256 tokens a chunk
    if (S > most) S = most;
    if (S > 16) S = 16;
    if (S < 1) S = 1;
    L.chunk = ((d->T + S - 1) / S + 63) / 64 * 64;
    L.S = static_cast<int>((d->T + L.chunk - 1) / L.chunk);
    size_t o = MOE_STATUS_BYTES;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align256(o + bytes);
        return at;
    };
    L.dl = take(static_cast<size_t>(d->T) * L.ld * 2);
    L.wr = take(static_cast<size_t>(d->d_model) * L.ld * 2);
    L.part = take(static_cast<size_t>(L.S) * d->d_model * L.ld * 4);
    L.total = o;
    return L;
}

}  // namespace

extern "C" {

int moe_layernorm(int64_t T, int d_model, const void* x, int x_is_bf16, const void* gamma, const void* beta, int w_is_bf16,
                  float eps, void* y, float* mean, float* rstd, void* stream) {
    MOE_TRY(check_norm(T, d_model));
    if (!x || !y || !(eps >= 0.0f)) return MOE_EINVAL;
    if (!all_aligned({x, y, gamma, beta})) return MOE_EUNSUPPORTED;
    return map_launch(launch_layernorm(x, x_is_bf16 != 0, gamma, beta, w_is_bf16 != 0, eps, T, d_model, y, mean, rstd,
                                       static_cast<cudaStream_t>(stream)));
}

int moe_layernorm_workspace_size(int64_t T, int d_model, size_t* bytes) {
    MOE_TRY(check_norm(T, d_model));
    if (!bytes) return MOE_EINVAL;
    *bytes = MOE_STATUS_BYTES + static_cast<size_t>(layernorm_blocks(T, d_model)) * 2 * d_model * 4;
    return MOE_OK;
}

int moe_layernorm_backward(int64_t T, int d_model, const void* dy, const void* x, int x_is_bf16, const void* gamma,
                           int w_is_bf16, const float* mean, const float* rstd, const void* dx_add, void* dx, void* dgamma,
                           void* dbeta, void* ws, size_t ws_bytes, void* stream) {
    MOE_TRY(check_norm(T, d_model));
    if (!dy || !x || !mean || !rstd || (!dx && !dgamma && !dbeta)) return MOE_EINVAL;
    if (!all_aligned({dy, x, gamma, dx_add, dx})) return MOE_EUNSUPPORTED;
    float* part = nullptr;
    if (dgamma || dbeta) {
        size_t need = 0;
        MOE_TRY(moe_layernorm_workspace_size(T, d_model, &need));
        if (!ws || !aligned16(ws)) return MOE_EINVAL;
        if (ws_bytes < need) return MOE_EWORKSPACE;
        part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + MOE_STATUS_BYTES);
    }
    return map_launch(launch_layernorm_backward(dy, x, x_is_bf16 != 0, gamma, w_is_bf16 != 0, mean, rstd, dx_add, T, d_model,
                                                dx, dgamma, dbeta, part, static_cast<cudaStream_t>(stream)));
}

int moe_ffn_train(const moe_dims* dims, const moe_bf16* x_perm, const int32_t* offsets, const moe_bf16* W1, const moe_bf16* W3,
                  const moe_bf16* W2, moe_bf16* gu, moe_bf16* h, float* y_perm, void* ws, size_t ws_bytes, void* stream) {
    MOE_TRY(check_dims(dims));
    if (!x_perm || !offsets || !W1 || !W3 || !W2 || !gu || !h || !y_perm) return MOE_EINVAL;
    if (!all_aligned({x_perm, W1, W3, W2, gu, h, y_perm})) return MOE_EUNSUPPORTED;
    MOE_TRY(check_status_ws(ws, ws_bytes));
    const int64_t A = dims->T * dims->K;
    const int E = dims->E, d = dims->d_model, f = dims->d_ff;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int* status = static_cast<int*>(ws);
    MOE_TRY(map_launch(launch_train_gate(in16(x_perm), offsets, A, E, d, f, in16(W1), in16(W3), out16(gu), out16(h), status, st)));
    return map_launch(launch_train_down(in16(h), offsets, A, E, d, f, in16(W2), y_perm, status, st));
}

int moe_ffn_backward(const moe_dims* dims, const moe_bf16* dy_perm, const moe_bf16* x_perm, const int32_t* offsets,
                     const moe_bf16* W1, const moe_bf16* W3, const moe_bf16* W2, const moe_bf16* gu, const moe_bf16* h,
                     moe_bf16* dgu, moe_bf16* dx_perm, void* dW1, void* dW3, void* dW2, int dw_is_bf16, void* ws,
                     size_t ws_bytes, void* stream) {
    MOE_TRY(check_dims(dims));
    if (!dy_perm || !offsets || !W2 || !gu || !dgu) return MOE_EINVAL;
    if ((dW1 == nullptr) != (dW3 == nullptr)) return MOE_EINVAL;
    if ((dx_perm && (!W1 || !W3)) || (dW1 && !x_perm) || (dW2 && !h)) return MOE_EINVAL;
    if (!all_aligned({dy_perm, x_perm, W1, W3, W2, gu, h, dgu, dx_perm, dW1, dW3, dW2})) return MOE_EUNSUPPORTED;
    MOE_TRY(check_status_ws(ws, ws_bytes));
    const int64_t A = dims->T * dims->K;
    const int E = dims->E, d = dims->d_model, f = dims->d_ff;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int* status = static_cast<int*>(ws);
    MOE_TRY(map_launch(launch_train_dgate(in16(dy_perm), offsets, A, E, d, f, in16(W2), in16(gu), out16(dgu), status, st)));
    if (dx_perm)
        MOE_TRY(map_launch(launch_train_dx(out16(dgu), offsets, A, E, d, f, in16(W1), in16(W3), out16(dx_perm), status, st)));
    WeightGradient w[3];
    int n = 0;
    if (dW1) {
        w[n++] = {in16(x_perm), d, out16(dgu), f, 2 * static_cast<int64_t>(f), dW1};
        w[n++] = {in16(x_perm), d, out16(dgu) + f, f, 2 * static_cast<int64_t>(f), dW3};
    }
    if (dW2) w[n++] = {in16(h), f, in16(dy_perm), d, d, dW2};
    if (n > 0) MOE_TRY(map_launch(launch_train_dw(w, n, offsets, 0, A, E, dw_is_bf16 != 0, status, st)));
    return MOE_OK;
}

int moe_train_subtiles(const moe_dims* dims, int product) {
    MOE_TRY(check_dims(dims));
    if (product < 0 || product > 4) return MOE_EINVAL;
    return train_subtiles(product, dims->T * dims->K, dims->E, dims->d_model, dims->d_ff);
}

int moe_combine_backward(const moe_dims* dims, const void* dy, int dy_is_bf16, const float* y_perm, const int32_t* inv,
                         const float* topk_w, moe_bf16* dy_perm, float* dtopk_w, void* stream) {
    MOE_TRY(check_dims(dims));
    if (!dy || !inv || !topk_w || !dy_perm || (dtopk_w && !y_perm)) return MOE_EINVAL;
    if (!all_aligned({dy, y_perm, dy_perm})) return MOE_EUNSUPPORTED;
    return map_launch(launch_combine_backward(dy, dy_is_bf16 != 0, y_perm, inv, topk_w, dims->T, dims->d_model, dims->K,
                                              out16(dy_perm), dtopk_w, static_cast<cudaStream_t>(stream)));
}

int moe_permute_backward(const moe_dims* dims, const moe_bf16* dx_perm, const int32_t* inv, void* dx, int dx_is_bf16,
                         void* stream) {
    MOE_TRY(check_dims(dims));
    if (!dx_perm || !inv || !dx) return MOE_EINVAL;
    if (!all_aligned({dx_perm, dx})) return MOE_EUNSUPPORTED;
    return map_launch(launch_permute_backward(in16(dx_perm), inv, dims->T, dims->d_model, dims->K, dx, dx_is_bf16 != 0,
                                              static_cast<cudaStream_t>(stream)));
}

int moe_route_backward_workspace_size(const moe_dims* dims, size_t* bytes) {
    MOE_TRY(check_dims(dims));
    if (!bytes) return MOE_EINVAL;
    *bytes = route_layout(dims).total;
    return MOE_OK;
}

int moe_route_backward(const moe_dims* dims, const moe_bf16* x, const moe_bf16* Wr, const float* logits,
                       const int32_t* topk_idx, const float* topk_w, const float* dtopk_w, const int32_t* counts, float aux_coef,
                       float z_coef, const moe_bf16* dx_perm, const int32_t* inv, void* dx, int dx_is_bf16, void* dWr,
                       int dw_is_bf16, float* dlogits, void* ws, size_t ws_bytes, void* stream) {
    MOE_TRY(check_dims(dims));
    if (!dx && !dWr && !dlogits) return MOE_EINVAL;
    if (dtopk_w && (!topk_idx || !topk_w)) return MOE_EINVAL;
    const bool losses = aux_coef != 0.0f || z_coef != 0.0f;
    if ((losses && !logits) || (aux_coef != 0.0f && !counts)) return MOE_EINVAL;
    if ((dx && !Wr) || (dWr && !x) || ((dx_perm == nullptr) != (inv == nullptr)) || (dx_perm && !dx)) return MOE_EINVAL;
    if (!all_aligned({x, Wr, dx_perm, dx})) return MOE_EUNSUPPORTED;
    if (!ws || !aligned16(ws)) return MOE_EINVAL;
    const RouteLayout L = route_layout(dims);
    if (ws_bytes < L.total) return MOE_EWORKSPACE;
    const int64_t T = dims->T;
    const int E = dims->E, K = dims->K, d = dims->d_model;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t* base = static_cast<uint8_t*>(ws);
    int* status = static_cast<int*>(ws);
    bf16* dl = reinterpret_cast<bf16*>(base + L.dl);
    MOE_TRY(map_launch(launch_route_backward(losses ? logits : nullptr, topk_idx, topk_w, dtopk_w, counts, aux_coef, z_coef, T, E, K,
                                             L.ld, dlogits, dx || dWr ? dl : nullptr, st)));
    if (dx) {
        const bf16* w = in16(Wr);
        if (L.ld != E) {
            bf16* padded = reinterpret_cast<bf16*>(base + L.wr);
            MOE_TRY(map_launch(launch_pad_router(w, d, E, L.ld, padded, st)));
            w = padded;
        }
        MOE_TRY(map_launch(launch_router_dx(dl, w, L.ld, in16(dx_perm), inv, T, d, K, dx, dx_is_bf16 != 0, st)));
    }
    if (dWr) {
        float* part = reinterpret_cast<float*>(base + L.part);
        const WeightGradient w{in16(x), d, dl, L.ld, L.ld, part};
        MOE_TRY(map_launch(launch_train_dw(&w, 1, nullptr, L.chunk, T, L.S, false, status, st)));
        MOE_TRY(map_launch(launch_router_weight(part, L.S, d, E, L.ld, dWr, dw_is_bf16 != 0, st)));
    }
    return MOE_OK;
}

}  // extern "C"
