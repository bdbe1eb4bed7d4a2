// Layer norm over the last axis, forward and backward.
//
//   forward   mean = sum(x) / d,  rstd = 1 / sqrt(sum((x - mean)^2) / d + eps)
//             y = xh * gamma + beta,  xh = (x - mean) * rstd
//   backward  q = dy * gamma
//             dx = rstd * (q - sum(q) / d - xh * sum(q * xh) / d) [+ dx_add]
//             dgamma = sum over tokens of dy * xh,  dbeta = sum of dy
//
// A row is read once and kept for the two sums of the variance, the second
// taken about the mean: no cancellation of large squares.  Rows of up to 1024 values take a
// warp each, wider ones a block.  A block walks a strided set of rows, with the
// next ones on their way through its reductions.  Everything is summed in fp32, in a fixed
// order.  Both directions are bound by memory.
//
// The weight's gradients run down the tokens: a backward block keeps the two
// column sums of its threads' own columns in
// registers, so they cost no traffic per row; each block writes one partial
// row, and a second kernel adds the partial rows in block order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "vec.cuh"

namespace moe {

namespace {

// Sums over the TEAM threads of a row, in every one of them.  A team of one
// warp needs no shared memory; otherwise the team is the block and `red` holds
// a value per warp (a buffer of its own per use, so one barrier does).
template <int TEAM>
__device__ __forceinline__ float team_sum(float x, float* red) {
    x = warp_sum(x);
    if (TEAM == 32) return x;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < TEAM / 32; i += 4) {
        const float4 r = *reinterpret_cast<const float4*>(red + i);
        s += r.x, s += r.y, s += r.z, s += r.w;
    }
    return s;
}

// Two at once: the first exchange leaves one sum in each half of the warp.
template <int TEAM>
__device__ __forceinline__ void team_sum2(float& x, float& y, float* red) {
    const bool hi = threadIdx.x & 16;
    float v = (hi ? y : x) + __shfl_xor_sync(0xffffffffu, hi ? x : y, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (TEAM == 32) {
        x = __shfl_sync(0xffffffffu, v, 0);
        y = __shfl_sync(0xffffffffu, v, 16);
        return;
    }
    if ((threadIdx.x & 15) == 0) red[(hi ? 32 : 0) + (threadIdx.x >> 5)] = v;
    __syncthreads();
    x = y = 0.f;
#pragma unroll
    for (int i = 0; i < TEAM / 32; i += 4) {
        const float4 a = *reinterpret_cast<const float4*>(red + i), b = *reinterpret_cast<const float4*>(red + 32 + i);
        x += a.x, x += a.y, x += a.z, x += a.w;
        y += b.x, y += b.y, y += b.z, y += b.w;
    }
}

// Threads of a block: a team, or 8 teams of one warp.
constexpr int block_of(int team) { return team == 32 ? 256 : team; }

// A thread holds P pieces of 16 bytes of a row, TEAM pieces apart: E values each.
template <typename X>
constexpr int kE = 16 / static_cast<int>(sizeof(X));

__device__ __forceinline__ void unpack_piece(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float((i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}
__device__ __forceinline__ void unpack_piece(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void load_values(const bf16* p, float (&v)[8]) { load8(p, v); }
__device__ __forceinline__ void load_values(const float* p, float (&v)[8]) { load8(p, v); }
__device__ __forceinline__ void load_values(const float* p, float (&v)[4]) { unpack_piece(*reinterpret_cast<const uint4*>(p), v); }
__device__ __forceinline__ void load_values(const bf16* p, float (&v)[4]) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
}
__device__ __forceinline__ void put_piece(bf16* p, const float (&v)[8]) { put8(p, v); }
__device__ __forceinline__ void put_piece(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Rows of N tensors on their way from memory: up to S of them, each thread's
// pieces in slots of shared memory that no other thread touches, so that
// waiting for its own copies is all the synchronisation there is.
template <typename X, int TEAM, int P, int N, int S>
struct Rows {
    static constexpr int kPiece = block_of(TEAM) * 16;
    static constexpr int kBytes = S * N * P * kPiece;
    uint8_t* slots;
    int slot = 0;
    __device__ __forceinline__ uint8_t* at(int s, int n, int p) const {
        return slots + ((s * N + n) * P + p) * kPiece + threadIdx.x * 16;
    }
    __device__ __forceinline__ void fetch(int s, const X* const (&src)[N], int64_t row, int64_t T, int d, int tid) {
        if (row < T)
#pragma unroll
            for (int n = 0; n < N; ++n)
                if (src[n] != nullptr)
#pragma unroll
                    for (int p = 0; p < P; ++p) {
                        const int c = (p * TEAM + tid) * kE<X>;
                        if (c < d)
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                                         ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(at(s, n, p)))),
                                           "l"(src[n] + row * d + c) : "memory");
                    }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void start(const X* const (&src)[N], int64_t row, int64_t step, int64_t T, int d, int tid) {
#pragma unroll
        for (int s = 0; s < S; ++s) fetch(s, src, row + s * step, T, d, tid);
    }
    __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory"); }
    __device__ __forceinline__ void get(int n, int p, float (&v)[kE<X>]) const {
        unpack_piece(*reinterpret_cast<const uint4*>(at(slot, n, p)), v);
    }
    // Done with this row: its slots take the row S steps on.
    __device__ __forceinline__ void next(const X* const (&src)[N], int64_t row, int64_t step, int64_t T, int d, int tid) {
        fetch(slot, src, row + S * step, T, d, tid);
        slot = slot + 1 == S ? 0 : slot + 1;
    }
};
constexpr int rows_ahead(int row_bytes, int budget) {
    return budget / row_bytes < 1 ? 1 : (budget / row_bytes > 4 ? 4 : budget / row_bytes);
}
// Forward: a block's slots take 128 bytes a thread, 128 KB an SM at 1024 threads.
template <typename X, int TEAM, int P>
using ForwardRows = Rows<X, TEAM, P, 1, rows_ahead(P * block_of(TEAM) * 16, block_of(TEAM) * 128)>;
// Backward: two blocks of 96 KB an SM, or one of 192 KB where the column sums
// leave registers for one only.
template <typename X, int TEAM, int P>
constexpr int kBackwardBlocks = P * kE<X> * TEAM > 4096 || P * kE<X> > 16 ? 1 : 2;
template <typename X, int TEAM, int P>
using BackwardRows = Rows<X, TEAM, P, 3, rows_ahead(3 * P * block_of(TEAM) * 16, 196608 / kBackwardBlocks<X, TEAM, P>)>;

// A team's part of a weight row: it stays in registers for all of a block's
// rows (read for each row from L1, 32-bit weights cost more wavefronts than
// the row itself).
template <typename X, typename W, int TEAM, int P>
__device__ __forceinline__ void load_weight(const W* w, float fill, int d, int tid, float (&v)[P][kE<X>]) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = (p * TEAM + tid) * kE<X>;
#pragma unroll
        for (int i = 0; i < kE<X>; ++i) v[p][i] = fill;
        if (w != nullptr && c < d) load_values(w + c, v[p]);
    }
}

template <typename X, typename W, int TEAM, int P>
__global__ void __launch_bounds__(block_of(TEAM))
layernorm_kernel(const X* x, const W* __restrict__ gamma, const W* __restrict__ beta, float eps, int64_t T, int d, X* y,
                 float* __restrict__ mean_out, float* __restrict__ rstd_out) {
    constexpr int TEAMS = block_of(TEAM) / TEAM, E = kE<X>;
    __shared__ __align__(16) float red[4][32];
    extern __shared__ __align__(16) uint8_t slots[];
    const int tid = threadIdx.x % TEAM;
    const float inv_d = 1.0f / static_cast<float>(d);
    const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS;
    int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + threadIdx.x / TEAM;
    const X* const src[1] = {x};
    ForwardRows<X, TEAM, P> rows{slots};
    rows.start(src, row, step, T, d, tid);
    float g[P][E], b[P][E];
    load_weight<X, W, TEAM, P>(gamma, 1.0f, d, tid, g);
    load_weight<X, W, TEAM, P>(beta, 0.0f, d, tid, b);
    int buf = 0;
    for (; row < T; row += step) {
        rows.wait();
        float v[P][E], sum = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            rows.get(0, p, v[p]);
            if ((p * TEAM + tid) * E < d)
#pragma unroll
                for (int i = 0; i < E; ++i) sum += v[p][i];
        }
        rows.next(src, row, step, T, d, tid);
        const float mean = team_sum<TEAM>(sum, red[buf]) * inv_d;
        float sq = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p)
            if ((p * TEAM + tid) * E < d)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    v[p][i] -= mean;
                    sq += v[p][i] * v[p][i];
                }
        const float rstd = __frsqrt_rn(team_sum<TEAM>(sq, red[buf + 1]) * inv_d + eps);
        buf ^= 2;  // a row's sums are read before the row after the next writes them
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = (p * TEAM + tid) * E;
            if (c < d) {
#pragma unroll
                for (int i = 0; i < E; ++i) v[p][i] = v[p][i] * rstd * g[p][i] + b[p][i];
                put_piece(y + row * d + c, v[p]);
            }
        }
        if (tid == 0) {
            if (mean_out) mean_out[row] = mean;
            if (rstd_out) rstd_out[row] = rstd;
        }
    }
}

template <typename X, typename W, int TEAM, int P>
__global__ void __launch_bounds__(block_of(TEAM), kBackwardBlocks<X, TEAM, P>)
layernorm_backward_kernel(const X* dy, const X* __restrict__ x, const W* __restrict__ gamma,
                          const float* __restrict__ mean_in, const float* __restrict__ rstd_in, const X* dx_add,
                          int64_t T, int d, X* dx, float* __restrict__ part) {
    constexpr int TEAMS = block_of(TEAM) / TEAM, E = kE<X>;
    __shared__ __align__(16) float red[4][32];
    extern __shared__ __align__(16) uint8_t slots[];
    const int tid = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    const float inv_d = 1.0f / static_cast<float>(d);
    const int64_t step = static_cast<int64_t>(gridDim.x) * TEAMS;
    int64_t row = static_cast<int64_t>(blockIdx.x) * TEAMS + team;
    const X* const src[3] = {x, dy, dx ? dx_add : nullptr};
    BackwardRows<X, TEAM, P> rows{slots};
    rows.start(src, row, step, T, d, tid);
    float g[P][E], dg[P][E], db[P][E];
    load_weight<X, W, TEAM, P>(gamma, 1.0f, d, tid, g);
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < E; ++i) dg[p][i] = db[p][i] = 0.f;
    float mean_n = row < T ? mean_in[row] : 0.f, rstd_n = row < T ? rstd_in[row] : 0.f;
    int buf = 0;
    for (; row < T; row += step) {
        const float mean = mean_n, rstd = rstd_n;
        if (row + step < T) mean_n = mean_in[row + step], rstd_n = rstd_in[row + step];
        rows.wait();
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int p = 0; p < P; ++p)
            if ((p * TEAM + tid) * E < d) {
                float xh[E], q[E];
                rows.get(0, p, xh);
                rows.get(1, p, q);
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    xh[i] = (xh[i] - mean) * rstd;
                    dg[p][i] += q[i] * xh[i];
                    db[p][i] += q[i];
                    q[i] *= g[p][i];
                    s1 += q[i];
                    s2 += q[i] * xh[i];
                }
            }
        if (dx) {  // the buffers alternate, so a row's sums are read before the row after the next writes them
            team_sum2<TEAM>(s1, s2, red[buf]);
            s1 *= inv_d;
            s2 *= inv_d;
            buf ^= 2;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int c = (p * TEAM + tid) * E;
                if (c < d) {
                    float xh[E], q[E], add[E];
                    rows.get(0, p, xh);
                    rows.get(1, p, q);
                    if (dx_add) rows.get(2, p, add);
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        q[i] = rstd * (q[i] * g[p][i] - s1 - (xh[i] - mean) * rstd * s2);
                        if (dx_add) q[i] += add[i];
                    }
                    put_piece(dx + row * d + c, q);
                }
            }
        }
        rows.next(src, row, step, T, d, tid);
    }
    if (!part) return;
    // partial row of this block: dgamma at [2 b], dbeta at [2 b + 1]
    float* pg = part + static_cast<int64_t>(blockIdx.x) * 2 * d;
    if (TEAM == 32) {  // the 8 warps' sums, in warp order
        __shared__ float sums[256];
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int i = 0; i < 2 * E; ++i) {
                __syncthreads();
                sums[threadIdx.x] = i < E ? dg[p][i % E] : db[p][i % E];
                __syncthreads();
                if (team == 0) {
                    float t = 0.f;
                    for (int w = 0; w < TEAMS; ++w) t += sums[w * 32 + tid];
                    const int c = (p * TEAM + tid) * E + i % E;
                    if (c < d) pg[(i < E ? 0 : d) + c] = t;
                }
            }
    } else {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = (p * TEAM + tid) * E;
            if (c < d)
#pragma unroll
                for (int i = 0; i < E; i += 4) {
                    *reinterpret_cast<float4*>(pg + c + i) = make_float4(dg[p][i], dg[p][i + 1], dg[p][i + 2], dg[p][i + 3]);
                    *reinterpret_cast<float4*>(pg + d + c + i) = make_float4(db[p][i], db[p][i + 1], db[p][i + 2], db[p][i + 3]);
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

// Threads of a row: few, with many values each, since the shuffles and the
// barrier cost every thread the same.  T = 16384, d = 4096, bf16: forward 41 us
// with 128 threads (the copy bandwidth), 52 with 256; backward 92 us with 256,
// 105 with 128 (one block an SM for the registers), 132 with 512.
// Above d = 8192 the 1024 threads have 64 registers, and the backward kernels
// spill: T = 16384, d = 16384, us (floor): bf16 240 (164) forward, 739 (328)
// backward, fp32 332 (328), 861 (656); d = 10240, bf16: 213 (102), 551 (205).

// V: vectors of 8 values a thread.
template <typename X, typename W, int TEAM, int V>
int forward_as(const void* x, const void* gamma, const void* beta, float eps, int64_t T, int d, void* y, float* mean,
               float* rstd, cudaStream_t st) {
    constexpr int TEAMS = block_of(TEAM) / TEAM, P = V * 8 / kE<X>;
    static std::atomic<unsigned long long> attr_done{0};
    constexpr int bytes = ForwardRows<X, TEAM, P>::kBytes;
    const auto kernel = layernorm_kernel<X, W, TEAM, P>;
    if (smem_attr_once(reinterpret_cast<const void*>(kernel), bytes, attr_done) != 0) return -3;
    const int64_t rows = (T + TEAMS - 1) / TEAMS, most = static_cast<int64_t>(num_sms()) * (1024 / block_of(TEAM));
    kernel<<<static_cast<unsigned>(rows < most ? rows : most), block_of(TEAM), bytes, st>>>(
        static_cast<const X*>(x), static_cast<const W*>(gamma), static_cast<const W*>(beta), eps, T, d, static_cast<X*>(y), mean, rstd);
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

template <typename X, typename W>
int forward_by_width(const void* x, const void* gamma, const void* beta, float eps, int64_t T, int d, void* y, float* mean,
                     float* rstd, cudaStream_t st) {
    if (d <= 256) return forward_as<X, W, 32, 1>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    if (d <= 512) return forward_as<X, W, 32, 2>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    if (d <= 1024) return forward_as<X, W, 32, 4>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    if (d <= 2048) return forward_as<X, W, 128, 2>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    if (d <= 4096) return forward_as<X, W, 128, 4>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
    if (d <= 8192) return forward_as<X, W, 256, 4>(x, gamma, beta, eps, T, d, y, mean, rstd, st);
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
    static std::atomic<unsigned long long> attr_done{0};
    constexpr int P = V * 8 / kE<X>, bytes = BackwardRows<X, TEAM, P>::kBytes;
    const auto kernel = layernorm_backward_kernel<X, W, TEAM, P>;
    if (smem_attr_once(reinterpret_cast<const void*>(kernel), bytes, attr_done) != 0) return -3;
    kernel<<<nb, block_of(TEAM), bytes, st>>>(
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
    if (a.d <= 2048) return backward_as<X, W, 128, 2>(a, st);
    if (a.d <= 4096) return backward_as<X, W, 256, 2>(a, st);
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
