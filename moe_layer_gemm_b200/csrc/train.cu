// Gradients of the steps around the experts: combine, dispatch and router.
//
//   combine   dy_perm[r] = w[t,k] * dy[t],  dw[t,k] = <dy[t], y_perm[r]>,  r = inv[t,k]
//   dispatch  dx[t] = sum over the kept slots k of dx_perm[inv[t,k]]
//   router    dl[t,e] = sum over the slots k that chose e of w[t,k] (dw[t,k] - sum_j w[t,j] dw[t,j])
//                     + aux * E / T * p[t,e] * (f_e - sum_i f_i p[t,i])
//                     + zc * 2 / T * lse[t] * p[t,e]
// with p and lse the softmax and log-sum-exp of the unbiased logits and
// f_e = counts_e / (T K), a constant as in the balance loss itself.  Rows are
// most of their bytes.  Combine and dispatch take a token's slots one after
// the other, its own row again for each (from L1 after the first), and cover
// the latency with the SM's many blocks; the router's product with the tokens'
// rows keeps several rows in flight in a thread.  Every sum is fp32 in a fixed
// order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "vec.cuh"

namespace moe {

namespace {

constexpr int kMaxK = 16;

// A block per token, a slot after the other: with 32 registers a thread the SM's
// resident blocks keep enough rows in flight (8192 x 2048, 4 slots, a quarter
// dropped: 51 us, the copy bandwidth; four slots' loads at once in each thread
// took 79 us).  Slot k's dot product is summed per thread over its
// columns, then over the warps in order.
template <typename Y>
__global__ void __launch_bounds__(256)
combine_backward_kernel(const Y* __restrict__ dy, const float* __restrict__ y_perm, const int32_t* __restrict__ inv,
                        const float* __restrict__ w, int64_t rows, int d, int K, bf16* __restrict__ dy_perm,
                        float* __restrict__ dw) {
    __shared__ float red[kMaxK][8];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int k = 0; k < K; ++k) {
        const int64_t r = inv[t * K + k];
        float dot = 0.f;
        if (r >= 0 && r < rows) {
            const float wk = w[t * K + k];
            for (int c = threadIdx.x * 8; c < d; c += blockDim.x * 8) {
                float g[8], o[8], y[8];
                load8(dy + t * d + c, g);
                if (dw) load8(y_perm + r * d + c, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[i] = wk * g[i];
                    if (dw) dot += g[i] * y[i];
                }
                put8(dy_perm + r * d + c, o);
            }
        }
        if (dw) {
            dot = warp_sum(dot);
            if (lane == 0) red[k][warp] = dot;
        }
    }
    if (!dw) return;
    __syncthreads();
    if (threadIdx.x < K) {
        float s = 0.f;
        for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) s += red[threadIdx.x][i];
        dw[t * K + threadIdx.x] = s;
    }
}

// A block per token, slot by slot: number, then row (8192 x 2048, 4 slots, a
// quarter dropped: 26.5 us, 20.5 at the copy bandwidth; the two loads wait for
// one another, and DRAM is half idle).
template <typename X>
__global__ void __launch_bounds__(256)
permute_backward_kernel(const bf16* __restrict__ dx_perm, const int32_t* __restrict__ inv, int64_t rows, int d, int K,
                        X* __restrict__ dx) {
    const int64_t t = blockIdx.x;
    for (int c = threadIdx.x * 8; c < d; c += blockDim.x * 8) {
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < K; ++k) {
            const int64_t r = inv[t * K + k];
            if (r < 0 || r >= rows) continue;
            float v[8];
            load8(dx_perm + r * d + c, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] += v[i];
        }
        put8(dx + t * d + c, s);
    }
}

// A warp per token; lane l owns experts l, l + 32, ..., J of them.  The bf16 copy [T, ld]
// (columns E.. zero) is what the two router products multiply: a rounding of
// 2^-9 of each value, as for every other operand of the tensor cores.
template <int J>
__global__ void __launch_bounds__(256)
route_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ idx, const float* __restrict__ w,
                      const float* __restrict__ dw, const int32_t* __restrict__ counts, float aux, float zc, int64_t T, int E,
                      int K, int ld, float* __restrict__ dlogits, bf16* __restrict__ dl16) {
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (t >= T) return;
    float dl[J];
#pragma unroll
    for (int j = 0; j < J; ++j) dl[j] = 0.f;
    if (logits) {
        float l[J], p[J];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = lane + 32 * j;
            l[j] = e < E ? logits[t * E + e] : -INFINITY;
            mx = fmaxf(mx, l[j]);
        }
        mx = warp_max(mx);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            p[j] = lane + 32 * j < E ? expf(l[j] - mx) : 0.f;
            sum += p[j];
        }
        sum = warp_sum(sum);
        const float inv_sum = 1.0f / sum, lse = mx + logf(sum);
        const float invA = 1.0f / (static_cast<float>(T) * static_cast<float>(K));
        float f[J];
        float fp = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = lane + 32 * j;
            p[j] *= inv_sum;
            f[j] = counts && e < E ? static_cast<float>(counts[e]) * invA : 0.f;
            fp += f[j] * p[j];
        }
        fp = warp_sum(fp);
        const float ca = aux * static_cast<float>(E) / static_cast<float>(T), cz = 2.0f * zc / static_cast<float>(T) * lse;
#pragma unroll
        for (int j = 0; j < J; ++j) dl[j] = p[j] * (ca * (f[j] - fp) + cz);
    }
    if (dw) {
        const float wk = lane < K ? w[t * K + lane] : 0.f, dk = lane < K ? dw[t * K + lane] : 0.f;
        const int ek = lane < K ? idx[t * K + lane] : -1;
        const float g = wk * (dk - warp_sum(wk * dk));
        for (int k = 0; k < K; ++k) {
            const int e = __shfl_sync(0xffffffffu, ek, k);
            const float gk = __shfl_sync(0xffffffffu, g, k);
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (e == lane + 32 * j) dl[j] += gk;
        }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = lane + 32 * j;
        if (dlogits && e < E) dlogits[t * E + e] = dl[j];
        if (dl16 && e < ld) dl16[t * ld + e] = __float2bfloat16_rn(e < E ? dl[j] : 0.f);
    }
}

// dx = dl Wr^T + the tokens' rows.  The product has at most 256 terms and the
// rows' bytes bound the kernel, so it is built as a gather that needs many loads
// in flight: blocks of 64 tokens x 128 columns, several to an SM, multiply
// with warp-level MMAs (16 x 8 x 16; each warp 64 tokens x 16 columns) from a
// double buffer of 64-term chunks, turn the sums round in shared memory and
// then walk rows, 16 lanes reading 256 consecutive bytes.  Neighbouring blocks
// take one strip of columns after the other of the same tokens, so that a row's
// pieces are read at about the same time (T = 16384, d = 4096, E = 8, K = 2:
// 89 us, 94 with a strip's tokens in a row).  (The same sum in the
// epilogue of the CTA-pair GEMM, whose 8 epilogue warps an SM are too few to
// cover the rows' latency, took 224 us at T = 16384, d = 4096, K = 2.)
constexpr int kDxTokens = 64, kDxCols = 128, kDxK = 64;
constexpr int kDxRows = 2;  // rows of a thread in flight together (1, 2, 4: 182, 168, 174 us at T = 4096, d = 7168, K = 8)
constexpr int kDxStride = kDxK + 8;   // bf16 operands: rows 16 bytes apart modulo 128
constexpr int kDxOut = kDxCols + 4;   // fp32 sums
constexpr int kDxBuffer = (kDxTokens + kDxCols) * kDxStride;
// One buffer where the product has one chunk; the sums go where the operands were.
constexpr int dx_smem(int ld) {
    const int operands = (ld > kDxK ? 2 : 1) * kDxBuffer * 2, sums = kDxTokens * kDxOut * 4;
    return operands > sums ? operands : sums;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const bf16* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(smem_addr(p)));
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 64-term chunk at k0 of both operands into `buf`; zeros beyond T, d and ld.
__device__ __forceinline__ void stage_dx(bf16* buf, const bf16* dl, const bf16* Wr, int ld, int k0, int width, int64_t t0, int64_t T,
                                         int n0, int d) {
    for (int i = threadIdx.x; i < (kDxTokens + kDxCols) * width; i += 256) {
        const int r = i / width, c = (i - r * width) * 8;
        const bool tok = r < kDxTokens;
        const bool ok = k0 + c < ld && (tok ? t0 + r < T : n0 + r - kDxTokens < d);
        const bf16* src = tok ? dl + (t0 + r) * ld : Wr + static_cast<int64_t>(n0 + r - kDxTokens) * ld;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                     ::"r"(smem_addr(buf + r * kDxStride + c)), "l"(ok ? src + k0 + c : dl), "r"(ok ? 16 : 0) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <typename X>
__global__ void __launch_bounds__(256, 4)
router_dx_kernel(const bf16* __restrict__ dl, const bf16* __restrict__ Wr, int ld, const bf16* __restrict__ dx_perm,
                 const int32_t* __restrict__ inv, int64_t T, int d, int K, X* __restrict__ dx) {
    extern __shared__ __align__(16) uint8_t smem[];
    bf16* const operands = reinterpret_cast<bf16*>(smem);
    float* const out = reinterpret_cast<float*>(smem);  // after the product
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned strips = (static_cast<unsigned>(d) + kDxCols - 1) / kDxCols;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / strips) * kDxTokens;
    const int n0 = static_cast<int>(blockIdx.x % strips) * kDxCols;
    // a chunk's 16-byte units of a row, whole MMA steps
    auto units = [&](int k0) { return min(kDxK, (ld - k0 + 15) / 16 * 16) / 8; };
    stage_dx(operands, dl, Wr, ld, 0, units(0), t0, T, n0, d);
    // the rows this thread adds up, t0 + 16 i + tid / 16: lane k of each 16 has slot k's number
    const int64_t rows = T * K;
    int mine[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + 16 * i + (threadIdx.x >> 4);
        const int64_t r = dx_perm && (lane & 15) < K && t < T ? inv[t * K + (lane & 15)] : -1;
        mine[i] = r < rows ? static_cast<int>(r) : -1;
    }
    float acc[4][2][4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    int buf = 0;
    for (int k0 = 0; k0 < ld; k0 += kDxK, buf ^= 1) {
        const bool more = k0 + kDxK < ld;
        if (more) stage_dx(operands + (buf ^ 1) * kDxBuffer, dl, Wr, ld, k0 + kDxK, units(k0 + kDxK), t0, T, n0, d);
        if (more) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        const bf16* sa = operands + buf * kDxBuffer;
        const bf16* sb = sa + kDxTokens * kDxStride;
        for (int k = 0; k < units(k0) * 8; k += 16) {
            uint32_t b[4];  // both 8-column halves of k 0-7, then of k 8-15
            ldmatrix4(b, sb + (16 * warp + (lane & 15)) * kDxStride + k + 8 * (lane >> 4));
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                uint32_t a[4];
                ldmatrix4(a, sa + (16 * m + (lane & 15)) * kDxStride + k + 8 * (lane >> 4));
                mma_16816(acc[m][0], a, b[0], b[2]);
                mma_16816(acc[m][1], a, b[1], b[3]);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *reinterpret_cast<float2*>(out + (16 * m + 8 * h + (lane >> 2)) * kDxOut + 16 * warp + 8 * n + 2 * (lane & 3)) =
                    make_float2(acc[m][n][2 * h], acc[m][n][2 * h + 1]);
    __syncthreads();
    const int col = 8 * (threadIdx.x & 15), c = n0 + col;
    const bool in = c < d;
#pragma unroll
    for (int h = 0; h < 4; h += kDxRows) {  // rows at a time
        float s[kDxRows][8];
#pragma unroll
        for (int i = 0; i < kDxRows; ++i) load8(out + (16 * (h + i) + (threadIdx.x >> 4)) * kDxOut + col, s[i]);
        if (dx_perm)
#pragma unroll 2
            for (int k = 0; k < K; ++k) {
                int src[kDxRows];
                float v[kDxRows][8];
#pragma unroll
                for (int i = 0; i < kDxRows; ++i) src[i] = __shfl_sync(0xffffffffu, mine[h + i], (lane & 16) + k);
                // every load is issued, a dropped slot's at row 0 and unused: a branch
                // around each would wait for them in turn
#pragma unroll
                for (int i = 0; i < kDxRows; ++i) load8(dx_perm + static_cast<int64_t>(src[i] < 0 ? 0 : src[i]) * d + (in ? c : 0), v[i]);
#pragma unroll
                for (int i = 0; i < kDxRows; ++i)
#pragma unroll
                    for (int x = 0; x < 8; ++x) s[i][x] += src[i] >= 0 ? v[i][x] : 0.f;
            }
#pragma unroll
        for (int i = 0; i < kDxRows; ++i) {
            const int64_t t = t0 + 16 * (h + i) + (threadIdx.x >> 4);
            if (t < T && in) put8(dx + t * d + c, s[i]);
        }
    }
}

// Router weight [d, E] with rows of ld elements, a multiple of 16 bytes;
// columns E.. are zero.
__global__ void __launch_bounds__(256)
pad_router_kernel(const bf16* __restrict__ Wr, int64_t n, int E, int ld, bf16* __restrict__ out) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t r = i / ld;
    const int c = static_cast<int>(i - r * ld);
    out[i] = c < E ? Wr[r * E + c] : __float2bfloat16_rn(0.f);
}

// dWr [d, E] = the token chunks' partial products [S, d, ld], summed in chunk order.
template <typename W>
__global__ void __launch_bounds__(256)
router_weight_kernel(const float* __restrict__ part, int S, int64_t stride, int64_t n, int E, int ld, W* __restrict__ out) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t r = i / E;
    const int64_t at = r * ld + (i - r * E);
    float s = 0.f;
    for (int j = 0; j < S; ++j) s += part[j * stride + at];
    out[i] = static_cast<W>(s);
}

int row_threads(int d) {
    const int t = (d / 8 + 31) / 32 * 32;
    return t < 32 ? 32 : (t > 256 ? 256 : t);
}
int done() { return cudaGetLastError() == cudaSuccess ? 0 : -3; }

}  // namespace

int launch_combine_backward(const void* dy, bool dy_bf16, const float* y_perm, const int32_t* inv, const float* w, int64_t T,
                            int d, int K, bf16* dy_perm, float* dw, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(T);
    if (dy_bf16)
        combine_backward_kernel<<<grid, row_threads(d), 0, st>>>(static_cast<const bf16*>(dy), y_perm, inv, w, T * K, d, K, dy_perm, dw);
    else
        combine_backward_kernel<<<grid, row_threads(d), 0, st>>>(static_cast<const float*>(dy), y_perm, inv, w, T * K, d, K, dy_perm, dw);
    return done();
}

int launch_permute_backward(const bf16* dx_perm, const int32_t* inv, int64_t T, int d, int K, void* dx, bool dx_bf16,
                            cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(T);
    if (dx_bf16)
        permute_backward_kernel<<<grid, row_threads(d), 0, st>>>(dx_perm, inv, T * K, d, K, static_cast<bf16*>(dx));
    else
        permute_backward_kernel<<<grid, row_threads(d), 0, st>>>(dx_perm, inv, T * K, d, K, static_cast<float*>(dx));
    return done();
}

int launch_route_backward(const float* logits, const int32_t* idx, const float* w, const float* dw, const int32_t* counts,
                          float aux, float zc, int64_t T, int E, int K, int ld, float* dlogits, bf16* dl16, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>((T + 7) / 8);
    const auto kernel = E <= 32 ? route_backward_kernel<1> : (E <= 64 ? route_backward_kernel<2> : (E <= 128 ? route_backward_kernel<4> : route_backward_kernel<8>));
    kernel<<<grid, 256, 0, st>>>(logits, idx, w, dw, counts, aux, zc, T, E, K, ld, dlogits, dl16);
    return done();
}

int launch_router_dx(const bf16* dl, const bf16* Wr, int ld, const bf16* dx_perm, const int32_t* inv, int64_t T, int d, int K,
                     void* dx, bool dx_bf16, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>((T + kDxTokens - 1) / kDxTokens * ((d + kDxCols - 1) / kDxCols));
    static std::atomic<unsigned long long> done16{0}, done32{0};
    if (dx_bf16) {
        if (smem_attr_once(reinterpret_cast<const void*>(router_dx_kernel<bf16>), dx_smem(256), done16) != 0) return -3;
        router_dx_kernel<<<grid, 256, dx_smem(ld), st>>>(dl, Wr, ld, dx_perm, inv, T, d, K, static_cast<bf16*>(dx));
    } else {
        if (smem_attr_once(reinterpret_cast<const void*>(router_dx_kernel<float>), dx_smem(256), done32) != 0) return -3;
        router_dx_kernel<<<grid, 256, dx_smem(ld), st>>>(dl, Wr, ld, dx_perm, inv, T, d, K, static_cast<float*>(dx));
    }
    return done();
}

int launch_pad_router(const bf16* Wr, int d, int E, int ld, bf16* out, cudaStream_t st) {
    const int64_t n = static_cast<int64_t>(d) * ld;
    pad_router_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, st>>>(Wr, n, E, ld, out);
    return done();
}

int launch_router_weight(const float* part, int S, int d, int E, int ld, void* out, bool out_bf16, cudaStream_t st) {
    const int64_t n = static_cast<int64_t>(d) * E, stride = static_cast<int64_t>(d) * ld;
    const unsigned grid = static_cast<unsigned>((n + 255) / 256);
    if (out_bf16) router_weight_kernel<<<grid, 256, 0, st>>>(part, S, stride, n, E, ld, static_cast<bf16*>(out));
    else router_weight_kernel<<<grid, 256, 0, st>>>(part, S, stride, n, E, ld, static_cast<float*>(out));
    return done();
}

}  // namespace moe
