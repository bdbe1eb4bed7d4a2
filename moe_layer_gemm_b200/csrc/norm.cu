// Layer norm over the last axis, forward and backward.
//
//   forward   mean = sum(x) / d,  rstd = 1 / sqrt(sum((x - mean)^2) / d + eps)
//             y = xh * gamma + beta,  xh = (x - mean) * rstd
//   backward  q = dy * gamma
//             dx = rstd * (q - sum(q) / d - xh * sum(q * xh) / d) [+ dx_add]
//             dgamma = sum over tokens of dy * xh,  dbeta = sum of dy
//
// A row is read once and stays in registers (8 consecutive values per thread
// and vector) for the two sums of the variance, the second taken about the
// mean: no cancellation of large squares.  Rows of up to 1024 values take a
// warp each, wider ones a block.  Everything is summed in fp32, in a fixed
// order.  Both directions are bound by memory.
//
// The weight's gradients run down the tokens: a backward block walks a strided
// set of rows with the two column sums of its threads' own columns in
// registers, so they cost no traffic per row; each block writes one partial
// row, and a second kernel adds the partial rows in block order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "vec.cuh"

namespace moe {

namespace {

// Sum over the TEAM threads of a row, in every one of them.  A team of one
// warp needs no shared memory; otherwise the team is the block and `red` holds
// one value per warp (a buffer of its own per call site, so one barrier does).
template <int TEAM>
__device__ __forceinline__ float team_sum(float x, float* red) {
    x = warp_sum(x);
    if (TEAM == 32) return x;
    constexpr int W = TEAM / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = x;
    __syncthreads();
    return warp_sum(lane < W ? red[lane] : 0.f);
}

// Threads of a block: a team, or 8 teams of one warp.
constexpr int block_of(int team) { return team == 32 ? 256 : team; }

template <typename X, typename W, int TEAM, int V>
__global__ void __launch_bounds__(block_of(TEAM))
layernorm_kernel(const X* x, const W* __restrict__ gamma, const W* __restrict__ beta, float eps, int64_t T, int d, X* y,
                 float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    constexpr int TEAMS = block_of(TEAM) / TEAM;
    __shared__ float red[2][32];
    const int tid = threadIdx.x % TEAM;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / TEAM;
    if (row >= T) return;  // a whole team: a block of one team always has its row
    const float inv_d = 1.0f / static_cast<float>(d);
    float v[V][8];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = (j * TEAM + tid) * 8;
        if (c < d) {
            load8(x + row * d + c, v[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[j][i];
        }
    }
    const float mean = team_sum<TEAM>(sum, red[0]) * inv_d;
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
        if ((j * TEAM + tid) * 8 < d)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[j][i] -= mean;
                sq += v[j][i] * v[j][i];
            }
    const float rstd = __frsqrt_rn(team_sum<TEAM>(sq, red[1]) * inv_d + eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = (j * TEAM + tid) * 8;
        if (c < d) {
            float g[8], b[8];
            if (gamma) load8(gamma + c, g);
            if (beta) load8(beta + c, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * rstd * (gamma ? g[i] : 1.0f) + (beta ? b[i] : 0.0f);
            put8(y + row * d + c, v[j]);
        }
    }
    if (tid == 0) {
        if (mean_out) mean_out[row] = mean;
        if (rstd_out) rstd_out[row] = rstd;
    }
}

template <typename X, typename W, int TEAM, int V>
__global__ void __launch_bounds__(block_of(TEAM))
layernorm_backward_kernel(const X* dy, const X* __restrict__ x, const W* __restrict__ gamma,
                          const float* __restrict__ mean_in, const float* __restrict__ rstd_in, const X* dx_add,
                          int64_t T, int d, X* dx, float* __restrict__ part) {
    constexpr int TEAMS = block_of(TEAM) / TEAM;
    __shared__ float red[4][32];
    const int tid = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const float inv_d = 1.0f / static_cast<float>(d);
    float dg[V][8], db[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[j][i] = db[j][i] = 0.f;
    int buf = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + team; row < T; row += static_cast<int64_t>(gridDim.x) * TEAMS) {
        const float mean = mean_in[row], rstd = rstd_in[row];
        float xh[V][8], q[V][8];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (j * TEAM + tid) * 8;
            if (c < d) {
                float g[8];
                load8(x + row * d + c, xh[j]);
                load8(dy + row * d + c, q[j]);
                if (gamma) load8(gamma + c, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    xh[j][i] = (xh[j][i] - mean) * rstd;
                    dg[j][i] += q[j][i] * xh[j][i];
                    db[j][i] += q[j][i];
                    if (gamma) q[j][i] *= g[i];
                    s1 += q[j][i];
                    s2 += q[j][i] * xh[j][i];
                }
            }
        }
        if (dx) {  // the buffers alternate, so a row's sums are read before the row after the next writes them
            s1 = team_sum<TEAM>(s1, red[buf]) * inv_d;
            s2 = team_sum<TEAM>(s2, red[buf + 1]) * inv_d;
            buf ^= 2;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (j * TEAM + tid) * 8;
                if (c < d) {
                    float add[8];
                    if (dx_add) load8(dx_add + row * d + c, add);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        q[j][i] = rstd * (q[j][i] - s1 - xh[j][i] * s2);
                        if (dx_add) q[j][i] += add[i];
                    }
                    put8(dx + row * d + c, q[j]);
                }
            }
        }
    }
    if (!part) return;
    // partial row of this block: dgamma at [2 b], dbeta at [2 b + 1]
    float* pg = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
    if (TEAM == 32) {  // the 8 warps' sums, in warp order
        __shared__ float sums[256];
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                __syncthreads();
                sums[threadIdx.x] = i < 8 ? dg[j][i & 7] : db[j][i & 7];
                __syncthreads();
                if (team == 0) {
                    float t = 0.f;
                    for (int w = 0; w < TEAMS; ++w) t += sums[w * 32 + tid];
                    const int c = (j * TEAM + tid) * 8 + (i & 7);
                    if (c < d) pg[(i < 8 ? 0 : d) + c] = t;
                }
            }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (j * TEAM + tid) * 8;
            if (c < d) {
                put8(pg + c, dg[j]);
                put8(pg + d + c, db[j]);
            }
        }
    }
}

// out[c] = sum of the blocks' partial rows: a block sums 32 columns, 8 rows of
// threads each adding every 8th partial row in order, then those 8 in order.
template <typename W>
__global__ void __launch_bounds__(256)
layernorm_weight_kernel(const float* __restrict__ part, int nb, int d, W* __restrict__ dgamma, W* __restrict__ dbeta) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;  // column of [dgamma | dbeta]
    float s = 0.f;
    if (c < 2 * d)
#pragma unroll 8
        for (int b = r; b < nb; b += 8) s += part[static_cast<int64_t>(b) * 2 * d + c];
    sums[r][lane] = s;
    __syncthreads();
    if (r == 0 && c < 2 * d) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += sums[i][lane];
        W* out = c < d ? dgamma : dbeta;
        if (out) out[c < d ? c : c - d] = static_cast<W>(t);
    }
}

constexpr int kMaxD = 16384;

template <typename X, typename W, int TEAM, int V>
int forward_as(const void* x, const void* gamma, const void* beta, float eps, int64_t T, int d, void* y, float* mean,
               float* rstd, cudaStream_t st) {
    constexpr int TEAMS = block_of(TEAM) / TEAM;
    layernorm_kernel<X, W, TEAM, V><<<static_cast<unsigned>((T + TEAMS - 1) / TEAMS), block_of(TEAM), 0, st>>>(
        static_cast<const X*>(x), static_cast<const W*>(gamma), static_cast<const W*>(beta), eps, T, d, static_cast<X*>(y), mean, rstd);
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

template <typename X, typename W>
int forward_by_width(const void* x, const void* gamma, const void* beta, float eps, int64_t T, int d, void* y, float* mean,
                     float* rstd, cudaStream_t st) {
    if (d <= 256) return forward_as<X, W, 32, 1>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    if (d <= 512) return forward_as<X, W, 32, 2>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    if (d <= 1024) return forward_as<X, W, 32, 4>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    if (d <= 2048) return forward_as<X, W, 256, 1>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    if (d <= 4096) return forward_as<X, W, 256, 2>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    if (d <= 8192) return forward_as<X, W, 512, 2>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    return forward_as<X, W, 1024, 2>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
}

struct BackwardArgs {
    const void *dy, *x, *gamma;
    const float *mean, *rstd;
    const void* dx_add;
    int64_t T;
    int d;
    void *dx, *dgamma, *dbeta;
    float* part;
};

int teams_of(int d) { return d <= 1024 ? 8 : 1; }

template <typename X, typename W, int TEAM, int V>
int backward_as(const BackwardArgs& a, cudaStream_t st) {
    const int nb = layernorm_blocks(a.T, a.d);
    float* part = a.dgamma || a.dbeta ? a.part : nullptr;
    layernorm_backward_kernel<X, W, TEAM, V><<<nb, block_of(TEAM), 0, st>>>(
        static_cast<const X*>(a.dy), static_cast<const X*>(a.x), static_cast<const W*>(a.gamma), a.mean, a.rstd,
        static_cast<const X*>(a.dx_add), a.T, a.d, static_cast<X*>(a.dx), part);
    if (cudaGetLastError() != cudaSuccess) return -3;
    if (!part) return 0;
    layernorm_weight_kernel<W><<<(2 * a.d + 31) / 32, 256, 0, st>>>(part, nb, a.d, static_cast<W*>(a.dgamma), static_cast<W*>(a.dbeta));
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

template <typename X, typename W>
int backward_by_width(const BackwardArgs& a, cudaStream_t st) {
    if (a.d <= 256) return backward_as<X, W, 32, 1>(a, st);
    if (a.d <= 512) return backward_as<X, W, 32, 2>(a, st);
    if (a.d <= 1024) return backward_as<X, W, 32, 4>(a, st);
    if (a.d <= 2048) return backward_as<X, W, 256, 1>(a, st);
    if (a.d <= 4096) return backward_as<X, W, 512, 1>(a, st);
    if (a.d <= 8192) return backward_as<X, W, 512, 2>(a, st);
    return backward_as<X, W, 1024, 2>(a, st);
}

}  // namespace

bool layernorm_supported(int d) { return d >= 16 && d <= kMaxD && d % 16 == 0; }

// Two blocks per SM: the partial rows stay few and the rows in flight many.
int layernorm_blocks(int64_t T, int d) {
    const int64_t rows = (T + teams_of(d) - 1) / teams_of(d);
    const int most = 2 * (num_sms() > 0 ? num_sms() : 148);
    return static_cast<int>(rows < most ? rows : most);
}

int launch_layernorm(const void* x, bool x_bf16, const void* gamma, const void* beta, bool w_bf16, float eps, int64_t T,
                     int d, void* y, float* mean, float* rstd, cudaStream_t st) {
    if (!layernorm_supported(d)) return -2;
    if (x_bf16)
        return w_bf16 ? forward_by_width<bf16, bf16>(x, gamma, beta, eps, T, d, y, mean, rstd, st)
                      : forward_by_width<bf16, float>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    return w_bf16 ? forward_by_width<float, bf16>(x, gamma, beta, eps, T, d, y, mean, rstd, st)
                  : forward_by_width<float, float>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
}

int launch_layernorm_backward(const void* dy, const void* x, bool x_bf16, const void* gamma, bool w_bf16, const float* mean,
                              const float* rstd, const void* dx_add, int64_t T, int d, void* dx, void* dgamma, void* dbeta,
                              float* part, cudaStream_t st) {
    if (!layernorm_supported(d)) return -2;
    const BackwardArgs a{dy, x, gamma, mean, rstd, dx_add, T, d, dx, dgamma, dbeta, part};
    if (x_bf16) return w_bf16 ? backward_by_width<bf16, bf16>(a, st) : backward_by_width<bf16, float>(a, st);
    return w_bf16 ? backward_by_width<float, bf16>(a, st) : backward_by_width<float, float>(a, st);
}

}  // namespace moe
