// Grouped matrix products of a training step on CTA pairs (tcgen05
// cta_group::2), reading the weights in their own [E, rows, cols] layout:
// an optimizer rewrites them every step, so nothing is packed beforehand.
//
// With g the experts, X_g the rows of expert g and the weights
// W1, W3 [d, f], W2 [f, d]:
//   gate    G = X W1, U = X W3, H = silu(G) * U        (one launch)
//   down    Y = H W2
//   dgate   dH = dY W2^T, then dG, dU from dH, G, U    (one launch)
//   dx      dX = dG W1^T + dU W3^T                     (one accumulation)
//   dw      dW1 = X^T dG, dW3 = X^T dU, dW2 = H^T dY   (one launch)
// and for the router, with dL [T, E] the logits' gradients:
//   router dw   dWr = x^T dL                           (token chunks as groups)
//
// Every product is D[256 x 256] tiles of a CTA pair: CTA r holds the M half r
// of A and the N half r of B, 64-deep k-blocks of 16 KB each in a ring; the
// leader issues 256 x 256 x 16 MMAs into two TMEM accumulators in turn.  A
// group's last tile of at most 128 rows takes MMAs of M = 128 and half of A;
// a CTA's 64 rows are then in TMEM lanes 0-63 with the tile's first 128 columns
// and in lanes 64-127 with the others.  What
// differs is which side of an operand is contiguous in memory: tcgen05 takes
// either from shared memory, so no operand is ever transposed:
//   K contiguous  (X, dY, dG|dU; W2 and W1, W3 as transposed weights): boxes
//                 of 64 k x 128 rows;
//   M or N contiguous (W1, W3, W2 as plain weights; every operand of a weight
//                 gradient, whose k is the token): two boxes of 64 columns x
//                 64 k.
// Out-of-range columns and weight rows are zero-filled by TMA (the weights'
// maps are 3-D, so a box never reads the next expert).  A weight gradient's
// k ends inside a box where a group ends: there the rows behind the group
// (other experts' rows, or memory nobody wrote) are cleared in shared memory,
// in both operands, before the MMA reads them.
//
// Pair protocol (each CTA has every barrier; "leader" is rank 0's copy):
//   full[s]    leader: armed for the pair's bytes, both CTAs' loads complete on it
//   empty[s]   both: the leader's MMA commit arrives on both
//   tfull[b]   both: the leader's MMA commit arrives on both
//   tempty[b]  leader: all epilogue warps of the pair arrive
//   tail[s]    both: a CTA's own loads of a k-block that its group ends in
//   clear[s]   leader: both CTAs have cleared the rows behind the group
// Only full[] and empty[] are used per k-block, and nothing a k-block waits
// for goes through the peer's threads: with each CTA's loads on its own full[]
// and a thread of the peer passing the news on, a release-arrive a k-block
// across the pair cost 1.15 us, a relaxed one 0.53 us.
// Tiles are dealt round-robin; every role derives them from the offsets.
// Every wait is bounded: one that runs out records its code and raises both
// abort flags, and all roles of the pair stop.  Then, as after a complete run,
// the two producers' counts are compared: the leader completes by hand the
// bytes of the peer's loads that it armed and the peer never issued, arms
// those that the peer issued ahead of it, and waits for all of them and for
// its MMAs before the pair frees TMEM.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kBK = 64;
constexpr uint32_t kOperand = 16384u;  // one CTA's half of an operand: 128 x 64 bf16
constexpr uint32_t kTmemCols = 512;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;   // weight gradients: one more warp, which clears tails
constexpr int kClearWarp = 2 + kEpiWarps;
constexpr int kMaxGroups = 256;
constexpr int kMaxStages = 6;
constexpr int kRaster = 3;  // tile columns walked together: the operands of the ~74 tiles in flight stay in L2

enum Epi : int { E_GATE, E_F32, E_DGATE, E_BF16, E_WGRAD };

// Operand ring, and output staging of an epilogue warp.  The saved projections'
// gradient stages two outputs beside the sums that it turns round; weight
// gradients need no table of first tiles, so their 4 KB fit beside the ring.
constexpr uint32_t ring_of(int epi) { return (epi == E_DGATE ? 10 : 12) * kOperand; }
constexpr int staging_of(int epi) { return epi == E_DGATE ? 6144 : (epi == E_WGRAD ? 4096 : 2048); }

// A weight gradient [M, N] of every group, rows of ld elements.
struct Product {
    int M, N;
    int m_tiles, n_tiles;
    int64_t ld;
    void* out;
};
constexpr int kProducts = 3;

struct Args {
    const int32_t* off;  // [G + 1] group offsets, or nullptr: groups of `chunk` rows
    int64_t cap;         // rows of the token matrices
    int64_t chunk;
    int G;
    int kb_first, kb_all;  // token-major: k-blocks of the first operand pair, and of both
    Product p[kProducts];  // weight gradients: `products` of them; token-major: p[0] without rows
    int products;
    int group_tiles;       // weight gradients: tiles of a group, all products
    bf16* h;               // E_GATE: activations out
    const bf16* gu;        // E_DGATE: saved projections [rows, 2 N]
    int out_bf16;          // E_WGRAD: bf16 output, else fp32
    int* status;
    uint32_t wait_limit;
    // A test of the timeout paths: the epilogue waits, `epi_limit` polls, for what
    // nothing completes.  The other waits keep the default limit, so that theirs
    // cannot run out first, which polls faster or slower than the epilogue's.
    int never_ready;
    uint32_t epi_limit;
};

struct Maps {
    CUtensorMap a[kProducts];
    CUtensorMap b[kProducts];
    CUtensorMap ah[2];         // token-major: a[] in boxes of 64 rows
    // outputs that leave by TMA: weight gradients [G, M, N] in boxes of 128 bytes x
    // 32 rows, E_DGATE's two in boxes of 64 bytes x 32 rows
    CUtensorMap c[kProducts];
};

// One thread of a converged warp.  The roles that issue copies and MMAs run in
// whole warps on warp-uniform values, and only these instructions are
// predicated: their operands are uniform registers, which a branch of one
// thread would have to fill from vector registers for each of them.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}
template <typename T>
__device__ __forceinline__ T uniform(T v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t out;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(addr), "r"(rank));
    return out;
}
__device__ __forceinline__ void pair_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void pair_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void store_cluster(uint32_t cluster_addr, uint32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Acquire at cluster scope: for arrivals that publish the other CTA's writes.
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
// Loads into this CTA's shared memory that complete on a barrier of either CTA.
__device__ __forceinline__ void load_2d(uint32_t one, const CUtensorMap* map, uint32_t dst, uint32_t bar, int32_t x, int32_t y) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];\n\t}"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(one) : "memory");
}
__device__ __forceinline__ void load_3d(uint32_t one, const CUtensorMap* map, uint32_t dst, uint32_t bar, int32_t x,
                                        int32_t y, int32_t z) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
                 "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];\n\t}"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(one) : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t one, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one) : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t one, uint64_t* bar) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                 "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
                 ::"r"(smem_u32(bar)), "h"(static_cast<uint16_t>(3)), "r"(one) : "memory");
}

// Operand whose M or N side is contiguous: two boxes of 64 columns x 64 k
// (rows of 128 B, 128-byte swizzle), 8 KB apart (leading offset); 8-k groups
// are 1024 B apart (stride offset).  One MMA covers 16 k: 2048 B.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(8192u >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

struct Tile {
    int g, j, n, m;    // group, product, column tile, row tile
    int64_t row0;      // token-major: first token row; weight gradient: first row of the reduction
    int rows;          // token-major: valid rows of the tile (<= 256)
    bool half;         // M = 128
    int kb;            // k-blocks
    int k_tail;        // weight gradient: valid rows of the last k-block
};

struct Sched {
    const int* off;   // clamped offsets
    const int* start; // first tile of each group
    int total;
};

template <bool WG>
__device__ __forceinline__ Tile decode(const Args& a, const Sched& sc, int tile) {
    Tile t;
    int local;
    t.j = 0;
    if (WG) {
        t.g = tile / a.group_tiles;
        local = tile - t.g * a.group_tiles;
        for (int n; t.j + 1 < a.products && local >= (n = a.p[t.j].m_tiles * a.p[t.j].n_tiles); ++t.j) local -= n;
    } else {
        int lo = 0, hi = a.G;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sc.start[mid] <= tile) lo = mid; else hi = mid;
        }
        t.g = lo;
        local = tile - sc.start[lo];
    }
    const Product& p = a.p[t.j];
    const int rows = max(0, sc.off[t.g + 1] - sc.off[t.g]);
    const int mt = WG ? p.m_tiles : (rows + 255) >> 8;
    const int band = local / (mt * kRaster);
    const int width = min(kRaster, p.n_tiles - band * kRaster);
    const int in = local - band * kRaster * mt;
    t.m = in / width;
    t.n = band * kRaster + in - t.m * width;
    if (WG) {
        t.row0 = sc.off[t.g];
        t.rows = 256;
        t.half = false;
        t.kb = (rows + kBK - 1) / kBK;
        t.k_tail = rows - (t.kb - 1) * kBK;
    } else {
        t.row0 = sc.off[t.g] + t.m * 256;
        t.rows = min(256, rows - t.m * 256);
        t.half = t.rows <= 128;
        t.kb = a.kb_all;
        t.k_tail = kBK;
    }
    return t;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&p);
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// 8 consecutive values as 16 bytes of bf16 (round to nearest even), and back.
__device__ __forceinline__ uint4 pack8(const float* v) {
    return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ void unpack8(const uint4& q, float* v) {
    v[0] = bf_lo(q.x), v[1] = bf_hi(q.x), v[2] = bf_lo(q.y), v[3] = bf_hi(q.y);
    v[4] = bf_lo(q.z), v[5] = bf_hi(q.z), v[6] = bf_lo(q.w), v[7] = bf_hi(q.w);
}

// Logistic function with the approximate reciprocal and exponential.  The
// exponential's documented error, 2 + 1.173 |x| units in the last place, is
// that of the result where x is far below 0: 2^-21 of the value at x = -1,
// 2^-18 at -20, 2^-16 at -87.  What comes of it is rounded to bf16, by up to
// 2^-8 of the value.  Below 2^-126 (x < -87.3) the reciprocal flushes to 0,
// as it does where the exponential overflows (x < -88.7).
__device__ __forceinline__ float sigmoid(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + __expf(-x)));
    return r;
}

// A wait that gives up after `limit` polls; its failure, or an abort seen, stops
// both CTAs of the pair.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, const Args& a, uint32_t limit, int code,
                                              volatile int* abort_flag, uint32_t peer_abort) {
    for (uint32_t i = 0; i < limit; ++i) {
        if (CLUSTER ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if ((i & 255u) == 255u) {
            if (*abort_flag) return false;
            if (i > 65536u) __nanosleep(64);
        }
    }
    atomicCAS(a.status, 0, code);
    *abort_flag = 1;
    store_cluster(peer_abort, 1u);
    return false;
}

// The same for a whole warp: every lane leaves with the same answer.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const Args& a, uint32_t limit, int code,
                                          volatile int* abort_flag, uint32_t peer_abort) {
    return __all_sync(0xffffffffu, wait_or_abort<CLUSTER>(bar, parity, a, limit, code, abort_flag, peer_abort)) != 0;
}

// An accumulator has a row per lane; stored from there, one instruction would
// touch 32 rows.  Each epilogue warp turns 32 rows x 64 bytes at a time round in
// 2 KB of shared memory: 16-byte chunk j of row r sits at chunk
// j ^ (r / 2 mod 4), free of bank conflicts by rows and by columns.  Then 4
// lanes hold a row's 64 bytes: lane l has rows 8 i + l / 4, i < 4, and chunk
// l % 4 of each.
__device__ __forceinline__ uint4* chunk_at(uint8_t* stg, int row, int j) {
    return reinterpret_cast<uint4*>(stg + row * 64 + ((j ^ ((row >> 1) & 3)) << 4));
}

// The staged rows to global memory: `base` is row 0's first byte; rows and
// 16-byte chunks beyond the counts are left out.
__device__ __forceinline__ void flush(uint8_t* stg, int lane, uint8_t* base, int64_t row_bytes, int rows, int chunks) {
    __syncwarp();
    const int j = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        if (r < rows && j < chunks) *reinterpret_cast<uint4*>(base + r * row_bytes + j * 16) = *chunk_at(stg, r, j);
    }
    __syncwarp();
}

// A row's 32 values, rounded to bf16.
__device__ __forceinline__ void stage_bf16(uint8_t* stg, int lane, const float* v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *chunk_at(stg, lane, j) = pack8(v + 8 * j);
}
// 16 of them as they are.
__device__ __forceinline__ void stage_f32(uint8_t* stg, int lane, const float* v) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(chunk_at(stg, lane, j)) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}

// A weight gradient's accumulators go to registers at once, which frees them
// for the next tile, and leave as TMA stores of 32 rows x 128 bytes: a tile of
// few k-blocks is bound by this epilogue (64 experts of 9 rows, 5856 x 400:
// 367 us with the stores above, 303 so).  The store clips at M and N.
template <int EPI>
struct WeightStore {
    uint32_t acc[4][32];
    __device__ __forceinline__ void fetch(uint32_t taddr) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            asm volatile(
                "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                : "=r"(acc[q][0]),"=r"(acc[q][1]),"=r"(acc[q][2]),"=r"(acc[q][3]),"=r"(acc[q][4]),"=r"(acc[q][5]),"=r"(acc[q][6]),"=r"(acc[q][7]),"=r"(acc[q][8]),"=r"(acc[q][9]),"=r"(acc[q][10]),"=r"(acc[q][11]),"=r"(acc[q][12]),"=r"(acc[q][13]),"=r"(acc[q][14]),"=r"(acc[q][15]),"=r"(acc[q][16]),"=r"(acc[q][17]),"=r"(acc[q][18]),"=r"(acc[q][19]),"=r"(acc[q][20]),"=r"(acc[q][21]),"=r"(acc[q][22]),"=r"(acc[q][23]),"=r"(acc[q][24]),"=r"(acc[q][25]),"=r"(acc[q][26]),"=r"(acc[q][27]),"=r"(acc[q][28]),"=r"(acc[q][29]),"=r"(acc[q][30]),"=r"(acc[q][31])
                : "r"(taddr + 32u * q));
#pragma unroll
        for (int q = 0; q < 4; ++q)  // nothing that uses them can move ahead of the wait
            asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(acc[q][0]),"+r"(acc[q][1]),"+r"(acc[q][2]),"+r"(acc[q][3]),"+r"(acc[q][4]),"+r"(acc[q][5]),"+r"(acc[q][6]),"+r"(acc[q][7]),"+r"(acc[q][8]),"+r"(acc[q][9]),"+r"(acc[q][10]),"+r"(acc[q][11]),"+r"(acc[q][12]),"+r"(acc[q][13]),"+r"(acc[q][14]),"+r"(acc[q][15]),"+r"(acc[q][16]),"+r"(acc[q][17]),"+r"(acc[q][18]),"+r"(acc[q][19]),"+r"(acc[q][20]),"+r"(acc[q][21]),"+r"(acc[q][22]),"+r"(acc[q][23]),"+r"(acc[q][24]),"+r"(acc[q][25]),"+r"(acc[q][26]),"+r"(acc[q][27]),"+r"(acc[q][28]),"+r"(acc[q][29]),"+r"(acc[q][30]),"+r"(acc[q][31]));
    }
    // To columns col0 .. col0 + 127 of rows row .. row + 31 of matrix g.
    __device__ __forceinline__ void store(const CUtensorMap* map, uint8_t* stg, int lane, bool as_bf16, int N, int col0, int row, int g) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int col = col0 + 32 * (as_bf16 ? q & ~1 : q);
            if (col >= N) return;
            if (!as_bf16 || !(q & 1)) {  // the box that was last stored from here has been read
                if (lane == 0) bulk_wait_read<0>();
                __syncwarp();
            }
            uint8_t* row_at = stg + lane * 128;
            if (as_bf16) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(acc[q][8 * j + i]);
                    *reinterpret_cast<uint4*>(row_at + (((4 * (q & 1) + j) ^ (lane & 7)) << 4)) = pack8(v);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4*>(row_at + ((j ^ (lane & 7)) << 4)) =
                        make_uint4(acc[q][4 * j], acc[q][4 * j + 1], acc[q][4 * j + 2], acc[q][4 * j + 3]);
            }
            if (!as_bf16 || (q & 1)) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(stg)), "r"(col), "r"(row), "r"(g) : "memory");
                    bulk_commit();
                }
            }
        }
    }
};

// A warp's part of a 256-column sub-tile: 32 rows (`rows` of them valid) from
// output row `row0`, `n` chunks of 32 columns from `col0` up to the width N
// (E_GATE: of each projection; U's accumulator columns are 64 behind G's).
// `taddr` is its first accumulator column.
// E_DGATE reads the saved projections at the same places; `load` (before the
// accumulator is ready) fetches the first 32 columns' worth.
template <int EPI>
struct Epilogue {
    const Args& a;
    const CUtensorMap* c;  // E_DGATE: the two outputs
    uint8_t* stg;
    int lane;
    uint4 g[EPI == E_DGATE ? 4 : 1], u[EPI == E_DGATE ? 4 : 1];

    // Every load is issued, at a place clamped into the tensor where its row or
    // column is out: a branch around each would wait for them in turn.
    __device__ __forceinline__ void load(const Product& p, int64_t row0, int rows, int col) {
        if constexpr (EPI == E_DGATE) {
            const int c = min(col + 8 * (lane & 3), p.N - 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = min(8 * i + (lane >> 2), rows - 1);
                const bf16* at = a.gu + (row0 + r) * p.ld + c;
                g[i] = __ldcs(reinterpret_cast<const uint4*>(at));
                u[i] = __ldcs(reinterpret_cast<const uint4*>(at + p.N));
            }
        }
    }

    __device__ __forceinline__ void run(const Product& p, uint32_t taddr, int64_t row0, int rows, int col0, int n) {
        if constexpr (EPI == E_GATE) {
#pragma unroll 1
            for (int q = 0; q < n; ++q) {
                const int col = col0 + 32 * q, chunks = (p.N - col) / 8;
                if (col >= p.N) return;
                float v[32], w[32];
                tmem_ld32(taddr + static_cast<uint32_t>(32 * q), v);
                tmem_ld32(taddr + static_cast<uint32_t>(64 + 32 * q), w);
                uint8_t* gu = reinterpret_cast<uint8_t*>(static_cast<bf16*>(p.out) + row0 * p.ld + col);
                stage_bf16(stg, lane, v);
                flush(stg, lane, gu, p.ld * 2, rows, chunks);
                stage_bf16(stg, lane, w);
                flush(stg, lane, gu + static_cast<int64_t>(p.N) * 2, p.ld * 2, rows, chunks);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= sigmoid(v[i]) * w[i];
                stage_bf16(stg, lane, v);
                flush(stg, lane, reinterpret_cast<uint8_t*>(a.h + row0 * p.N + col), static_cast<int64_t>(p.N) * 2, rows, chunks);
            }
        } else if constexpr (EPI == E_DGATE) {
#pragma unroll 1
            for (int q = 0; q < n; ++q) {
                const int col = col0 + 32 * q, cc = col + 8 * (lane & 3);
                if (col >= p.N) return;
                float acc[4][8];
                {
                    float v[32];
                    tmem_ld32(taddr + static_cast<uint32_t>(32 * q), v);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {  // 16 columns at a time; lanes l % 4 = 2 h, 2 h + 1 take them
                        stage_f32(stg, lane, v + 16 * h);
                        __syncwarp();
                        if (((lane >> 1) & 1) == h) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int r = 8 * i + (lane >> 2), j = 2 * (lane & 1);
                                const float4 x = *reinterpret_cast<const float4*>(chunk_at(stg, r, j));
                                const float4 y = *reinterpret_cast<const float4*>(chunk_at(stg, r, j + 1));
                                acc[i][0] = x.x, acc[i][1] = x.y, acc[i][2] = x.z, acc[i][3] = x.w;
                                acc[i][4] = y.x, acc[i][5] = y.y, acc[i][6] = y.z, acc[i][7] = y.w;
                            }
                        }
                        __syncwarp();
                    }
                }
                uint4 gn[4], un[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) gn[i] = g[i], un[i] = u[i];
                if (q + 1 < n && col + 32 < p.N) load(p, row0, rows, col + 32);
                // 32 rows of the tile leave as one TMA store of each gradient (the boxes'
                // 64-byte swizzle is the staging's), fewer row by row: a box would
                // reach into the next group
                uint8_t* const out = stg + 2048;
                if (rows == 32) {
                    if (lane == 0) bulk_wait_read<0>();  // the chunk before has been read
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 8 * i + (lane >> 2);
                    float gv[8], uv[8], dg[8], du[8];
                    unpack8(gn[i], gv);
                    unpack8(un[i], uv);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const float sg = sigmoid(gv[x]), silu = gv[x] * sg;
                        // s (1 + g (1 - s)) = s + g s - g s s
                        dg[x] = acc[i][x] * uv[x] * (sg + fmaf(-silu, sg, silu));
                        du[x] = acc[i][x] * silu;
                    }
                    if (rows == 32) {
                        *chunk_at(out, r, lane & 3) = pack8(dg);
                        *chunk_at(out + 2048, r, lane & 3) = pack8(du);
                    } else if (r < rows && cc < p.N) {
                        bf16* dst = static_cast<bf16*>(p.out) + (row0 + r) * p.ld + cc;
                        *reinterpret_cast<uint4*>(dst) = pack8(dg);
                        *reinterpret_cast<uint4*>(dst + p.N) = pack8(du);
                    }
                }
                if (rows == 32) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&c[0], out, col, static_cast<int32_t>(row0));
                        tma_store_2d(&c[1], out + 2048, col, static_cast<int32_t>(row0));
                        bulk_commit();
                    }
                }
            }
        } else {
            const bool as_bf16 = EPI == E_BF16;
            const int bytes = as_bf16 ? 2 : 4;
            uint8_t* out = static_cast<uint8_t*>(p.out) + row0 * p.ld * bytes;
#pragma unroll 1
            for (int q = 0; q < n; ++q) {
                const int col = col0 + 32 * q;
                if (col >= p.N) return;
                float v[32];
                tmem_ld32(taddr + static_cast<uint32_t>(32 * q), v);
                if (as_bf16) {
                    stage_bf16(stg, lane, v);
                    flush(stg, lane, out + col * 2, p.ld * 2, rows, (p.N - col) / 8);
                } else {
                    stage_f32(stg, lane, v);
                    flush(stg, lane, out + static_cast<int64_t>(col) * 4, p.ld * 4, rows, (p.N - col) / 4);
                    stage_f32(stg, lane, v + 16);
                    flush(stg, lane, out + static_cast<int64_t>(col) * 4 + 64, p.ld * 4, rows, (p.N - col) / 4 - 4);
                }
            }
        }
    }

    // A weight gradient of an expert without rows.
    __device__ __forceinline__ void zero(const Product& p, int64_t row0, int rows, int col0) {
        const int per = a.out_bf16 ? 8 : 4;
        for (int r = 0; r < rows; ++r)
            for (int c = col0 + per * lane; c < p.N && c < col0 + 128; c += 32 * per) {
                const int64_t at = (row0 + r) * p.ld + c;
                uint8_t* dst = static_cast<uint8_t*>(p.out) + at * (a.out_bf16 ? 2 : 4);
                *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
            }
    }
};

// SUB: 256-column sub-tiles of a tile, each with an accumulator of its own.  With
// one, the two accumulators alternate and a tile's epilogue runs under the
// next tile's MMAs.  With two, both belong to the tile: a k-block of A serves
// twice the MMAs, so a ring of the same size reaches twice as far ahead and
// 3/4 of the bytes are loaded; in exchange the next tile waits for the
// epilogue, except that up to a ring of its k-blocks are multiplied into the
// first accumulator while the second is still being read.
template <int EPI, bool B_MN, int SUB>  // weight gradients: SUB = 1
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(EPI == E_WGRAD ? kThreads + 32 : kThreads, 1)
train_gemm_kernel(const __grid_constant__ Maps maps, const Args a) {
    constexpr bool WG = EPI == E_WGRAD;
    constexpr uint32_t kStageBytes = (1 + SUB) * kOperand;
    constexpr uint32_t kRingBytes = ring_of(EPI);
    constexpr int kStages = kRingBytes / kStageBytes;
    constexpr int kSubCols = EPI == E_GATE ? 128 : 256;  // output columns of a sub-tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRingBytes + kEpiWarps * staging_of(EPI));
    uint64_t* empty = full + kStages;
    uint64_t* tail = empty + kStages;
    uint64_t* clear = tail + kStages;
    uint64_t* tfull = clear + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint64_t* never = drain + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(never + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint32_t* issued = tmem_slot + 2;  // [rank][stage uses issued, stages whose last use was a tail], [rank][use_bytes]
    int* off = reinterpret_cast<int*>(issued + 4 + 2 * kMaxStages);
    int* start = off + kMaxGroups + 1;  // token-major only

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cta_rank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&tail[s], 1);
            mbar_init(&clear[s], 2);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * kEpiWarps);
        }
        mbar_init(drain, 1);
        mbar_init(never, 1);
        *abort_flag = 0;
        fence_mbar_init();
        for (int i = 0; i < (WG ? a.products : 2); ++i) {
            tma_prefetch_desc(&maps.a[i]);
            tma_prefetch_desc(&maps.b[i]);
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    __syncwarp();
    pair_arrive();  // this CTA's barriers exist; the other's are waited for below
    // Under programmatic launch all of the above ran while the previous kernel
    // of the stream finished; the next one may do the same from here on.
    pdl_wait();
    pdl_trigger();
    // Offsets clamped to the matrices' rows: no value in the array is ever an address.
    for (int g = threadIdx.x; g <= a.G; g += blockDim.x) {
        const int64_t o = a.off != nullptr ? static_cast<int64_t>(a.off[g]) : static_cast<int64_t>(g) * a.chunk;
        off[g] = static_cast<int>(o < 0 ? 0 : (o > a.cap ? a.cap : o));
    }
    __syncthreads();
    if (!WG && warp == 0) {  // tiles before each group; one whose end lies before its start is empty
        int carry = 0;
        for (int g0 = 0; g0 < a.G; g0 += 32) {
            const int g = g0 + lane;
            const int n = g < a.G ? ((max(0, off[g + 1] - off[g]) + 255) >> 8) * a.p[0].n_tiles : 0;
            int incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            if (g < a.G) start[g] = carry + incl - n;
            carry += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) start[a.G] = carry;
    }
    tc_fence_before();
    __syncthreads();
    pair_wait();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const Sched sc{off, start, WG ? a.G * a.group_tiles : start[a.G]};
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const uint32_t peer_abort = peer_addr(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u);

    if (warp == 0) {
        // ---------------------------------------------------- producer (both CTAs)
        const uint32_t one = elect_one();
        const uint32_t leader_full = peer_addr(smem_u32(full), 0), own_tail = peer_addr(smem_u32(tail), rank);
        uint32_t s = 0, ph = 0, uses = 0, tails = 0, tail_ph = 0;
        uint32_t* use_bytes = issued + 4 + kMaxStages * rank;  // this CTA's bytes of each stage's last use
        bool ok = true;
        for (int tile = pair; ok && tile < sc.total; tile += npairs) {
            Tile t = decode<WG>(a, sc, tile);
            t.j = uniform(t.j);
            t.g = uniform(t.g);
            t.m = uniform(t.m);
            t.n = uniform(t.n);
            t.kb = uniform(t.kb);
            t.k_tail = uniform(t.k_tail);
            const int row0 = uniform(static_cast<int>(t.row0));
            const bool half = uniform(static_cast<int>(t.half)) != 0;
            const int col0 = t.n * SUB * kSubCols;
            const int subs = min(SUB, (a.p[t.j].N - col0 + kSubCols - 1) / kSubCols);
            const int n0 = col0 + (EPI == E_GATE ? 64 : 128) * static_cast<int>(rank);
            const uint32_t bytes = static_cast<uint32_t>(subs) * kOperand + (half ? kOperand / 2 : kOperand);
            for (int kb = 0; kb < t.kb; ++kb) {
                if (!warp_wait(&empty[s], ph ^ 1u, a, a.wait_limit, DEV_TIMEOUT_PRODUCER_EMPTY, abort_flag, peer_abort)) {
                    ok = false;
                    break;
                }
                const uint32_t sa = smem_u32(smem + s * kStageBytes);
                uint32_t bar = leader_full + 8u * s;
                if (WG && kb == t.kb - 1 && t.k_tail < kBK) {
                    bar = own_tail + 8u * s;
                    if (one) mbar_arrive_expect_tx(&tail[s], bytes);
                    if (leader && one) mbar_arrive(&full[s]);
                    tails |= 1u << s;
                    tail_ph ^= 1u << s;
                } else {
                    if (leader && one) mbar_arrive_expect_tx(&full[s], 2 * bytes);
                    tails &= ~(1u << s);
                }
                if (one) use_bytes[s] = bytes;
                if (WG) {
                    const int y = row0 + kb * kBK;
                    const int m0 = t.m * 256 + 128 * static_cast<int>(rank);
                    load_2d(one, &maps.a[t.j], sa, bar, m0, y);
                    load_2d(one, &maps.a[t.j], sa + 8192, bar, m0 + 64, y);
                    load_2d(one, &maps.b[t.j], sa + kOperand, bar, n0, y);
                    load_2d(one, &maps.b[t.j], sa + kOperand + 8192, bar, n0 + 64, y);
                } else {
                    const int second = kb >= a.kb_first ? 1 : 0;
                    const int k0 = (kb - (second ? a.kb_first : 0)) * kBK;
                    load_2d(one, half ? &maps.ah[second] : &maps.a[second], sa, bar, k0,
                            row0 + (half ? 64 : 128) * static_cast<int>(rank));
                    const CUtensorMap* b = &maps.b[second];
                    for (int j = 0; j < subs; ++j) {
                        const uint32_t sb = sa + (1 + j) * kOperand;
                        const int n = n0 + kSubCols * j;
                        if (EPI == E_GATE) {  // the same 64 columns of both projections
                            load_3d(one, &maps.b[0], sb, bar, n, k0, t.g);
                            load_3d(one, &maps.b[1], sb + 8192, bar, n, k0, t.g);
                        } else if (B_MN) {
                            load_3d(one, b, sb, bar, n, k0, t.g);
                            load_3d(one, b, sb + 8192, bar, n + 64, k0, t.g);
                        } else {
                            load_3d(one, b, sb, bar, k0, n, t.g);
                        }
                    }
                }
                ++uses;
                if (++s == kStages) { s = 0; ph ^= 1u; }
            }
        }
        if (one) {
            // this CTA's own tails have landed (a phase never used counts as complete)
            for (int i = 0; WG && i < kStages; ++i)
                mbar_drain(&tail[i], ((tail_ph >> i) & 1u) ^ 1u, a.status, DEV_TIMEOUT_DRAIN, a.wait_limit);
            const uint32_t rec = peer_addr(smem_u32(issued), 0);
            store_cluster(rec + 8u * rank, uses);
            store_cluster(rec + 8u * rank + 4u, tails);
            if (!leader)
                for (int i = 0; i < kStages; ++i) store_cluster(rec + 4u * (4 + kMaxStages + i), use_bytes[i]);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------- MMA issuer (leader)
        // By the whole warp where a tile has one sub-tile of columns: 60 small experts'
        // backward takes 960 us, 974 by one thread.  The wide tiles' eight MMAs a k-block
        // keep the tensor cores fed from one thread, which is the faster there: forward of
        // the Mixtral-shaped batch 8.16 ms, 8.43 by the warp.
        constexpr bool kWarp = SUB == 1;
        if (leader && (kWarp || lane == 0)) {
            const uint32_t one = kWarp ? elect_one() : 1u;
            auto wait = [&](auto cluster, uint64_t* bar, uint32_t parity, int code) -> bool {
                constexpr bool kCluster = decltype(cluster)::value;
                if (kWarp) return warp_wait<kCluster>(bar, parity, a, a.wait_limit, code, abort_flag, peer_abort);
                return wait_or_abort<kCluster>(bar, parity, a, a.wait_limit, code, abort_flag, peer_abort);
            };
            auto same = [&](int v) { return kWarp ? uniform(v) : v; };
            // idesc: D fp32, A and B bf16, bits 15 and 16 set where A, B are M-, N-contiguous
            constexpr uint32_t major = (WG ? (1u << 15) : 0u) | (B_MN ? (1u << 16) : 0u);
            // descriptors of the ring's first byte; a stage, a sub-tile and a step of 16 k add to their address field
            const uint32_t ring = smem_u32(smem);
            const uint64_t desc_a = WG ? desc_mn(ring) : umma_desc_sw128(ring);
            const uint64_t desc_b = (B_MN ? desc_mn(ring) : umma_desc_sw128(ring)) + (kOperand >> 4);
            uint32_t s = 0, ph = 0, tail_ph = 0, uses1 = 0;  // uses1: tiles that filled the second of two sub-tiles
            int it = 0;
            bool ok = true;
            // Wait until k-block kb of the tile is in stage s of both CTAs, a tail's
            // rows behind the group cleared; the 16-k steps to multiply, 0: abort.
            auto arrived = [&](const Tile& t, int kb) -> int {
                int steps = kBK / 16;
                if (WG && kb == t.kb - 1 && t.k_tail < kBK) {
                    const uint32_t tph = (tail_ph >> s) & 1u;
                    tail_ph ^= 1u << s;
                    if (!wait(std::true_type{}, &clear[s], tph, DEV_TIMEOUT_MMA_FULL)) return 0;
                    steps = (t.k_tail + 15) / 16;
                }
                if (!wait(std::false_type{}, &full[s], ph, DEV_TIMEOUT_MMA_FULL)) return 0;
                tc_fence_after();
                return steps;
            };
            // Stage `st`'s k-block into accumulator `buf` with sub-tile j of B.
            auto multiply = [&](uint32_t idesc, uint32_t st, int j, int buf, int steps, bool first) {
                const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf) * 256u;
                const uint64_t da = desc_a + st * (kStageBytes >> 4);
                const uint64_t db = desc_b + st * (kStageBytes >> 4) + static_cast<uint32_t>(j) * (kOperand >> 4);
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk) {
                    if (WG && kk >= steps) break;
                    mma_pair(one, d_tmem, da + kk * ((WG ? 2048 : 32) >> 4), db + kk * ((B_MN ? 2048 : 32) >> 4), idesc, (!first || kk > 0) ? 1u : 0u);
                }
            };
            for (int tile = pair; ok && tile < sc.total; tile += npairs) {
                Tile t = decode<WG>(a, sc, tile);
                t.kb = same(t.kb);
                t.k_tail = same(t.k_tail);
                if (t.kb == 0) continue;
                const uint32_t idesc = (same(static_cast<int>(t.half)) ? umma_idesc_bf16(128, 256) : umma_idesc_bf16(256, 256)) | major;
                const int subs = SUB == 1 ? 1 : same(min(SUB, (a.p[t.j].N - t.n * SUB * kSubCols + kSubCols - 1) / kSubCols));
                int kb = 0;
                const int buf0 = SUB == 1 ? it & 1 : 0;
                const uint32_t use = static_cast<uint32_t>(SUB == 1 ? it >> 1 : it);
                if (!wait(std::true_type{}, &tempty[buf0], (use & 1u) ^ 1u, DEV_TIMEOUT_MMA_TEMPTY)) break;
                tc_fence_after();
                if (SUB == 2 && subs == 2) {
                    // the second accumulator may still be read: go ahead in the first
                    // with the k-blocks that the ring holds (whole ones, before the last)
                    const uint32_t s0 = s, want = (uses1 & 1u) ^ 1u;
                    while (kb < kStages && kb < t.kb - 1 && !try_wait_cluster(&tempty[1], want)) {
                        if (!arrived(t, kb)) {
                            ok = false;
                            break;
                        }
                        multiply(idesc, s, 0, 0, kBK / 16, kb == 0);
                        ++kb;
                        if (++s == kStages) { s = 0; ph ^= 1u; }
                    }
                    if (!ok || !wait(std::true_type{}, &tempty[1], want, DEV_TIMEOUT_MMA_TEMPTY)) break;
                    tc_fence_after();
                    uint32_t st = s0;
                    for (int b = 0; b < kb; ++b) {
                        multiply(idesc, st, 1, 1, kBK / 16, b == 0);
                        commit_pair(one, &empty[st]);
                        if (++st == kStages) st = 0;
                    }
                }
                for (; kb < t.kb; ++kb) {
                    const int steps = arrived(t, kb);
                    if (!steps) {
                        ok = false;
                        break;
                    }
                    multiply(idesc, s, 0, buf0, steps, kb == 0);
                    if (SUB == 2 && subs == 2) {
                        if (kb == t.kb - 1) commit_pair(one, &tfull[0]);  // its epilogue runs under the last MMAs
                        multiply(idesc, s, 1, 1, steps, kb == 0);
                    }
                    commit_pair(one, &empty[s]);
                    if (++s == kStages) { s = 0; ph ^= 1u; }
                }
                if (ok) commit_pair(one, &tfull[SUB == 2 && subs == 2 ? 1 : buf0]);
                ++it;
                uses1 += subs == 2 ? 1u : 0u;
            }
            // every MMA issued is complete before TMEM is freed
            if (one) {  // the thread that issued them
                asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                             ::"r"(smem_u32(drain)) : "memory");
                mbar_drain(drain, 0, a.status, DEV_TIMEOUT_DRAIN, a.wait_limit);
            }
        }
        __syncwarp();
    } else if (WG && warp == kClearWarp) {
        // ---------------------------------------------------- tails (both CTAs)
        // A group ends inside a tile's last box: clear the rows behind it, up to
        // the last 16-row step that is multiplied, once the box has landed.
        const uint32_t leader_clear = peer_addr(smem_u32(clear), 0);
        uint32_t s = 0, tail_ph = 0;
        for (int tile = pair; tile < sc.total; tile += npairs) {
            const Tile t = decode<WG>(a, sc, tile);
            if (t.kb == 0) continue;
            s = (s + static_cast<uint32_t>(t.kb)) % kStages;
            if (t.k_tail == kBK) continue;
            const uint32_t st = (s + kStages - 1) % kStages;
            const uint32_t tph = (tail_ph >> st) & 1u;
            tail_ph ^= 1u << st;
            if (!warp_wait(&tail[st], tph, a, a.wait_limit, DEV_TIMEOUT_MMA_FULL, abort_flag, peer_abort)) break;
            const int from = t.k_tail * 8, to = (t.k_tail + 15) / 16 * 128;  // 16-byte units of a 64-column box
            uint4* box = reinterpret_cast<uint4*>(smem + st * kStageBytes);
            for (int i = from + lane; i < to; i += 32)
                for (int b = 0; b < 4; ++b) box[b * 512 + i] = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive_cluster(leader_clear + 8u * st);
        }
    } else {
        // ---------------------------------------------------- epilogue (both CTAs)
        // Warp quarter q holds rows 32 q .. of this CTA's 128 and the two warps of
        // a quarter take the two column halves; of M = 128, quarters q and q + 2
        // hold rows 32 q .. of 64 and a column half each, shared by their warps.
        const int q = warp & 3, half = (warp - 2) >> 2;
        const uint32_t leader_tempty = peer_addr(smem_u32(tempty), 0);
        uint8_t* const stg = smem + kRingBytes + (warp - 2) * staging_of(EPI);
        Epilogue<EPI> epi{a, maps.c, stg, lane};
        int it = 0;
        uint32_t uses1 = 0;
        bool ok = true;
        for (int tile = pair; ok && tile < sc.total; tile += npairs) {
            const Tile t = decode<WG>(a, sc, tile);
            const int r0 = t.half ? static_cast<int>(rank) * 64 + (q & 1) * 32 : static_cast<int>(rank) * 128 + q * 32;
            // its first column of a sub-tile, that column's accumulator, and its 32-column chunks
            const int part = t.half ? (q >> 1) * (kSubCols / 2) + half * (kSubCols / 4) : half * (kSubCols / 2);
            const int part_acc = t.half ? half * (kSubCols / 4) : half * 128;
            const int part_n = (kSubCols / 64) / (t.half ? 2 : 1);
            const Product& p = a.p[t.j];
            const int rows = max(0, min(32, (WG ? p.M - t.m * 256 : t.rows) - r0));
            const int64_t row0 = WG ? static_cast<int64_t>(t.g) * p.M + t.m * 256 + r0 : t.row0 + r0;
            const int tile_col = t.n * SUB * kSubCols;
            const int subs = SUB == 1 ? 1 : min(SUB, (p.N - tile_col + kSubCols - 1) / kSubCols);
            for (int j = 0; j < subs; ++j) {
                const int col0 = tile_col + j * kSubCols + part;
                if (WG && t.kb == 0) {
                    epi.zero(p, row0, rows, col0);
                    continue;
                }
                const int buf = SUB == 1 ? it & 1 : j;
                const uint32_t use = SUB == 1 ? static_cast<uint32_t>(it >> 1) : (j ? uses1 : static_cast<uint32_t>(it));
                const bool mine = rows > 0 && col0 < p.N;
                if (mine && !WG) epi.load(p, row0, rows, col0);
                if (!warp_wait(a.never_ready ? never : &tfull[buf], a.never_ready ? 0u : use & 1u, a, a.epi_limit, DEV_TIMEOUT_EPI_TFULL,
                               abort_flag, peer_abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t taddr = tmem_base + static_cast<uint32_t>(buf) * 256u + (static_cast<uint32_t>(q * 32) << 16) +
                                       static_cast<uint32_t>(part_acc);
                if constexpr (WG) {
                    WeightStore<EPI> w;
                    w.fetch(taddr);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_cluster(leader_tempty + 8u * buf);
                    if (mine) w.store(&maps.c[t.j], stg, lane, a.out_bf16, p.N, col0, t.m * 256 + r0, t.g);
                } else {
                    if (mine) epi.run(p, taddr, row0, rows, col0, part_n);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_cluster(leader_tempty + 8u * buf);
                }
            }
            if (!(WG && t.kb == 0)) {
                ++it;
                uses1 += subs == 2 ? 1u : 0u;
            }
        }
        if ((WG || EPI == E_DGATE) && lane == 0) bulk_wait_all();
    }

    // No copy is in flight when the pair ends.  A complete run issued the same
    // uses on both sides and multiplied them all; after an abort the leader
    // makes up for the difference (at most the ring, since a use waits for its
    // stage) and waits for what was issued.
    auto reconcile = [&]() {
        const uint32_t mine = issued[0], theirs = issued[2];
        const uint32_t *my_bytes = issued + 4, *their_bytes = my_bytes + kMaxStages;
        const uint32_t first = mine > kStages ? mine - kStages : 0u;
        for (uint32_t u = theirs > first ? theirs : first; u < mine; ++u)
            if (!((issued[1] >> (u % kStages)) & 1u)) mbar_complete_tx(&full[u % kStages], my_bytes[u % kStages]);
        for (uint32_t u = mine; u < theirs && u < mine + kStages; ++u) {
            if ((issued[3] >> (u % kStages)) & 1u) mbar_arrive(&full[u % kStages]);
            else mbar_arrive_expect_tx(&full[u % kStages], their_bytes[u % kStages]);
        }
        const uint32_t last = theirs > mine ? theirs : mine;
        for (uint32_t u = last > kStages ? last - kStages : 0u; u < last; ++u)
            mbar_drain(&full[u % kStages], (u / kStages) & 1u, a.status, DEV_TIMEOUT_DRAIN, a.wait_limit);
    };
    tc_fence_before();
    __syncthreads();
    // All roles of both CTAs have stopped; neither CTA's memory goes while the
    // other may still use it.
    pair_arrive();
    pair_wait();
    if (*abort_flag) {  // raised in both CTAs or in neither: whoever raised it told both before this barrier
        if (leader && threadIdx.x == 0) reconcile();
        __syncthreads();
        pair_arrive();
        pair_wait();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
    }
}

PFN_cuTensorMapEncodeTiled_v12000 map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// bf16 matrix [rows, cols] with row stride ld (elements), boxes of 64 columns x box_rows.
bool map_matrix(CUtensorMap* m, const bf16* base, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows) {
    auto enc = map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows < 1 ? 1 : rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    cuuint32_t box[2] = {64u, box_rows}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<bf16*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// bf16 matrices [mats, rows, cols], boxes of 64 columns x box_rows of one matrix.
bool map_weights(CUtensorMap* m, const bf16* base, int64_t mats, int64_t rows, int64_t cols, uint32_t box_rows) {
    auto enc = map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(mats)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 2, static_cast<cuuint64_t>(rows) * cols * 2};
    cuuint32_t box[3] = {64u, box_rows, 1u}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output matrices [mats, rows, cols], boxes of 128 bytes x 32 rows of one matrix.
bool map_output(CUtensorMap* m, void* base, bool as_bf16, int64_t mats, int64_t rows, int64_t cols) {
    auto enc = map_encoder();
    if (!enc) return false;
    const cuuint64_t size = as_bf16 ? 2 : 4;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(mats)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * size, static_cast<cuuint64_t>(rows) * cols * size};
    cuuint32_t box[3] = {as_bf16 ? 64u : 32u, 32u, 1u}, es[3] = {1, 1, 1};
    return enc(m, as_bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output rows [rows, cols] of bf16 with stride ld, boxes of 64 bytes x 32 rows.
bool map_rows_out(CUtensorMap* m, bf16* base, int64_t rows, int64_t cols, int64_t ld) {
    auto enc = map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    cuuint32_t box[2] = {32u, 32u}, es[2] = {1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int ceil_div(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

constexpr size_t smem_of(int epi) {
    return 1024 + ring_of(epi) + kEpiWarps * staging_of(epi) + (4 * kMaxStages + 6) * 8 + 8 + (4 + 2 * kMaxStages) * 4 +
           (epi == E_WGRAD ? 1 : 2) * (kMaxGroups + 1) * 4;
}
static_assert(smem_of(E_GATE) <= 232448 && smem_of(E_DGATE) <= 232448 && smem_of(E_WGRAD) <= 232448, "227 KB a CTA");

template <int EPI, bool B_MN, int SUB>
int launch_sub(const Maps& maps, const Args& a, int pairs, int64_t max_tiles, cudaStream_t st) {
    static std::atomic<unsigned long long> attr_done{0};
    const auto kernel = train_gemm_kernel<EPI, B_MN, SUB>;
    constexpr size_t kSmem = smem_of(EPI);
    if (smem_attr_once(reinterpret_cast<const void*>(kernel), static_cast<int>(kSmem), attr_done) != 0) return -3;
    if (pairs > max_tiles) pairs = static_cast<int>(max_tiles);
    // Programmatic launch: where the tiles are few, the set-up of one product's
    // kernel runs on free SMs under the previous product's end.
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(EPI == E_WGRAD ? kThreads + 32 : kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, a) == cudaSuccess ? 0 : -3;
}

// K-blocks of a tile from which it takes two sub-tiles.  The epilogue that the
// next tile then waits for has to be a small part of it.  One sub-tile against
// two, ms, from idle:
//   gate  64 k-blocks  5.67, 5.58 (Mixtral-shaped batch); 112  1.45, 1.37; 256  1.57, 1.38
//   down  32  0.83, 0.94; 128  0.89, 0.93; 160  1.11, 1.10 and 1.10, 1.02; 224  2.96, 2.82
//   dx    44  0.301, 0.314; 64  0.414, 0.405 and 0.430, 0.445; 128  0.84, 0.77; 448  5.77, 5.41
// The two others always take one.  The saved projections' gradient, whose
// epilogue reads them too, was from 0.92 to 1.09 times as fast with two at 128
// to 512 k-blocks and slower below; weight gradients were from 0.92 to 1.03
// times as fast at 32 to 1024.
constexpr int kNever = 1 << 30;
constexpr int wide_from(int epi) { return epi == E_GATE ? 64 : (epi == E_F32 ? 160 : (epi == E_BF16 ? 128 : kNever)); }
constexpr int sub_cols(int epi) { return epi == E_GATE ? 128 : 256; }

// Tiles of a launch whose tiles have `sub` sub-tiles, laid out in `a`; a
// token-major one has `row_tiles` row tiles.
int64_t lay_out(Args& a, int epi, int sub, int64_t row_tiles) {
    a.group_tiles = 0;
    for (int j = 0; j < a.products; ++j) {
        Product& p = a.p[j];
        p.n_tiles = ceil_div(p.N, sub * sub_cols(epi));
        p.m_tiles = ceil_div(p.M, 256);
        a.group_tiles += p.m_tiles * p.n_tiles;
    }
    return epi == E_WGRAD ? static_cast<int64_t>(a.G) * a.group_tiles : row_tiles * a.p[0].n_tiles;
}

// Sub-tiles of a tile.  Two need a long reduction and tiles enough for every
// pair: the pairs take their tiles in rounds, and a round of wide tiles costs
// about 0.92 of two narrow ones (0.88 to 1 in the figures above), so the wide
// tiles' rounds must be few enough.  Few tiles of two sub-tiles leave pairs
// idle.  One sub-tile against two, us, with the rounds of each:
//   down  f = 14336, d = 4096, one group of 256 rows       (1, 1)  104, 190
//         the same, 8 groups of about 256 / 512 rows       (3, 2)  381, 493; (5, 3) 603, 781
//   dx    f = 14336, d = 4096, one group of 256 rows       (1, 1)  187, 307
//         f = 8192, d = 4096, 8 groups of about 256 rows   (3, 2)  296, 369
//         f = 4096, d = 4096, one group of 4096 rows       (4, 2)  199, 192
// The row tiles are not known here: a group's last one is taken to be half full.
int sub_tiles(int epi, Args a, int pairs) {
    if (a.kb_all < wide_from(epi) || a.p[0].N <= sub_cols(epi)) return 1;
    const int64_t groups = a.G < a.cap ? a.G : a.cap, likely = (a.cap + 255) / 256 + a.G / 2;
    const int64_t row_tiles = likely > groups ? likely : groups;
    const int64_t one = (lay_out(a, epi, 1, row_tiles) + pairs - 1) / pairs, two = (lay_out(a, epi, 2, row_tiles) + pairs - 1) / pairs;
    return 92 * 2 * two <= 100 * one ? 2 : 1;
}

template <int EPI, bool B_MN>
int launch(const Maps& maps, Args a, cudaStream_t st) {
    if (a.G < 1 || a.G > kMaxGroups) return -2;
    const WaitSettings wt = wait_settings();
    a.epi_limit = wt.wait_limit ? wt.wait_limit : kWaitLimit;
    a.never_ready = wt.dep_never_ready;
    a.wait_limit = a.never_ready ? kWaitLimit : a.epi_limit;
    const int pairs = num_sms() / 2;
    if (pairs < 1) return -3;
    const int sub = sub_tiles(EPI, a, pairs);
    // at most this many row tiles: every group's last one may be partial
    const int64_t tiles = lay_out(a, EPI, sub, (a.cap + 255) / 256 + a.G);
    if constexpr (wide_from(EPI) != kNever) {
        if (sub == 2) return launch_sub<EPI, B_MN, 2>(maps, a, pairs, tiles, st);
    }
    return launch_sub<EPI, B_MN, 1>(maps, a, pairs, tiles, st);
}

// What the token-major products share.
Args token_major(const int32_t* off, int64_t rows, int E, int N, int64_t ld, void* out, int kb_first, int kb_all, int* status) {
    Args a{};
    a.off = off;
    a.cap = rows;
    a.G = E;
    a.kb_first = kb_first;
    a.kb_all = kb_all;
    a.products = 1;
    a.p[0].N = N;
    a.p[0].ld = ld;
    a.p[0].out = out;
    a.status = status;
    return a;
}

}  // namespace

int launch_train_gate(const bf16* x, const int32_t* off, int64_t rows, int E, int d, int f, const bf16* W1,
                      const bf16* W3, bf16* gu, bf16* h, int* status, cudaStream_t st) {
    Maps m;
    std::memset(&m, 0, sizeof(m));
    if (!map_matrix(&m.a[0], x, rows, d, d, 128) || !map_matrix(&m.ah[0], x, rows, d, d, 64) || !map_weights(&m.b[0], W1, E, d, f, 64) ||
        !map_weights(&m.b[1], W3, E, d, f, 64))
        return -3;
    m.a[1] = m.a[0];
    m.ah[1] = m.ah[0];
    Args a = token_major(off, rows, E, f, 2 * static_cast<int64_t>(f), gu, ceil_div(d, kBK), ceil_div(d, kBK), status);
    a.h = h;
    return launch<E_GATE, true>(m, a, st);
}

int launch_train_down(const bf16* h, const int32_t* off, int64_t rows, int E, int d, int f, const bf16* W2, float* y,
                      int* status, cudaStream_t st) {
    Maps m;
    std::memset(&m, 0, sizeof(m));
    if (!map_matrix(&m.a[0], h, rows, f, f, 128) || !map_matrix(&m.ah[0], h, rows, f, f, 64) || !map_weights(&m.b[0], W2, E, f, d, 64)) return -3;
    m.a[1] = m.a[0];
    m.ah[1] = m.ah[0];
    m.b[1] = m.b[0];
    Args a = token_major(off, rows, E, d, d, y, ceil_div(f, kBK), ceil_div(f, kBK), status);
    return launch<E_F32, true>(m, a, st);
}

int launch_train_dgate(const bf16* dy, const int32_t* off, int64_t rows, int E, int d, int f, const bf16* W2,
                       const bf16* gu, bf16* dgu, int* status, cudaStream_t st) {
    Maps m;
    std::memset(&m, 0, sizeof(m));
    if (!map_matrix(&m.a[0], dy, rows, d, d, 128) || !map_matrix(&m.ah[0], dy, rows, d, d, 64) || !map_weights(&m.b[0], W2, E, f, d, 128) ||
        !map_rows_out(&m.c[0], dgu, rows, f, 2 * static_cast<int64_t>(f)) ||
        !map_rows_out(&m.c[1], dgu + f, rows, f, 2 * static_cast<int64_t>(f)))
        return -3;
    m.a[1] = m.a[0];
    m.ah[1] = m.ah[0];
    m.b[1] = m.b[0];
    Args a = token_major(off, rows, E, f, 2 * static_cast<int64_t>(f), dgu, ceil_div(d, kBK), ceil_div(d, kBK), status);
    a.gu = gu;
    return launch<E_DGATE, false>(m, a, st);
}

int launch_train_dx(const bf16* dgu, const int32_t* off, int64_t rows, int E, int d, int f, const bf16* W1,
                    const bf16* W3, bf16* dx, int* status, cudaStream_t st) {
    Maps m;
    std::memset(&m, 0, sizeof(m));
    const int64_t ld = 2 * static_cast<int64_t>(f);
    if (!map_matrix(&m.a[0], dgu, rows, f, ld, 128) || !map_matrix(&m.a[1], dgu + f, rows, f, ld, 128) ||
        !map_matrix(&m.ah[0], dgu, rows, f, ld, 64) || !map_matrix(&m.ah[1], dgu + f, rows, f, ld, 64) ||
        !map_weights(&m.b[0], W1, E, d, f, 128) || !map_weights(&m.b[1], W3, E, d, f, 128))
        return -3;
    Args a = token_major(off, rows, E, d, d, dx, ceil_div(f, kBK), 2 * ceil_div(f, kBK), status);
    return launch<E_BF16, false>(m, a, st);
}

int launch_train_dw(const WeightGradient* w, int n, const int32_t* off, int64_t chunk, int64_t rows, int G, bool out_bf16,
                    int* status, cudaStream_t st) {
    if (n < 1 || n > kProducts) return -2;
    Maps m;
    std::memset(&m, 0, sizeof(m));
    Args a{};
    for (int j = 0; j < n; ++j) {
        if (!map_matrix(&m.a[j], w[j].left, rows, w[j].M, w[j].M, 64) || !map_matrix(&m.b[j], w[j].right, rows, w[j].N, w[j].right_ld, 64) ||
            !map_output(&m.c[j], w[j].out, out_bf16, G, w[j].M, w[j].N))
            return -3;
        a.p[j].M = w[j].M;
        a.p[j].N = w[j].N;
        a.p[j].ld = w[j].N;
        a.p[j].out = w[j].out;
    }
    a.products = n;
    a.off = off;
    a.chunk = chunk;
    a.cap = rows;
    a.G = G;
    a.out_bf16 = out_bf16 ? 1 : 0;
    a.status = status;
    return launch<E_WGRAD, true>(m, a, st);
}

int train_subtiles(int product, int64_t rows, int E, int d, int f) {
    if (wide_from(product) == kNever) return 1;
    const bool gate = product == E_GATE;  // width f, reduction over d; else the other way round
    const int k = ceil_div(gate ? d : f, kBK) * (product == E_BF16 ? 2 : 1);
    const Args a = token_major(nullptr, rows, E, gate ? f : d, 0, nullptr, k, k, nullptr);
    return sub_tiles(product, a, (num_sms() > 0 ? num_sms() : 148) / 2);
}

}  // namespace moe
