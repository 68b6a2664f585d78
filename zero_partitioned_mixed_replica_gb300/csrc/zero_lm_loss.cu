// Language-model head and loss: softmax cross entropy of hidden @ weight^T
// without the logits in memory, and its gradients.
//
// Four products of 2 n vocab d operations: the logits in the forward call, and
// in the backward call the logits again, dz @ weight and dz^T @ hidden.  One
// kernel (mm_kernel) computes all of them on the tensor cores; what differs
// is how the operands lie (a product that sums over tokens or over the
// vocabulary reads its operands along their rows, "MN-major") and what is done
// with the accumulator.  Memory: the weight once for each product, dz once
// written and twice read, everything else stays in L2 (129 MB): the products
// bound the time, at the measured 1.9 PFLOP/s of a burst.
//
// Tokens that do not count are taken out first: `gather` copies the others'
// hidden states next to one another (rows of 16-byte multiples, which TMA
// wants), so that padding costs nothing and cannot spoil a sum.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "zero_launch.h"
#include "zero_tc.cuh"

namespace zk {

constexpr int kTileK = 64;            // of K in a stage: 128 bytes
constexpr int kMmThreads = 192;       // warps 0-3: accumulator, 4: loads, 5: products
constexpr int kBoxBytes = 128 * 128;  // 128 rows of 64
constexpr int kTileN = 256;           // columns of a tile, at most

enum { EPI_STATS = 0, EPI_DZ = 1, EPI_PART = 2, EPI_OUT = 3 };
enum { ROWS_M = 1, ROWS_K = 2 };  // which extent is the number of tokens that count

// The workspace begins with what the kernels share.
struct LossHead {
    int32_t error;
    int32_t count;   // tokens that count
    uint32_t ticket;
    int32_t pad;
};

struct MmArgs {
    LossHead* head;
    int32_t rows_in;          // ROWS_M or ROWS_K
    int64_t m, n, k;          // extents (the one of rows_in at most: head->count says how many)
    int32_t bn;               // columns of a tile, a multiple of 16
    int32_t splits;           // of K
    int32_t m_group;          // row tiles that follow one another while the columns stay; 0: columns first
    int32_t n_off, k_off;     // where B's rows and K begin
    uint32_t idesc;
    // epilogue
    const int32_t* target;    // STATS, DZ: of each row
    const int32_t* row_of;    // DZ: the token of each row
    const float* lse;         // DZ: by token
    float2* parts;            // STATS: [column tile][part_rows] row maximum, sum of exponentials
    int64_t part_rows;
    float* z_target;          // STATS: the target's logit
    uint16_t* dz;             // DZ: [rows][ld]
    int64_t ld;
    float dz_scale;
    float* part;              // PART: [split][split_rows][ld]
    int64_t split_rows;
    uint16_t* out;            // OUT: [m][ld]
    float scale;
    const float* scale_dev;
    const float* share;
    int32_t add;              // PART, OUT: to what is there
    int32_t vec;              // OUT: rows begin on 32-byte boundaries, ld % 16 == 0
};

template <int CG>
struct MmShape {
    static constexpr int kA = kBoxBytes;                        // bytes of A and B in a stage
    static constexpr int kB = 2 * kBoxBytes / CG;
    static constexpr int kStages = CG == 2 ? 6 : 4;
    static constexpr int kOps = kStages * (kA + kB);
    static constexpr int kBytes = 1024 + kOps + 4 * 32 * 33 * 4 + 256;   // alignment, operands, transposition, barriers
};

struct MmTile {
    int32_t m, n, kb0, kb1;   // row tile, column tile, blocks of kTileK
};

__device__ __forceinline__ MmTile mm_tile(const MmArgs& a, int64_t t, int64_t tm, int64_t tn, int32_t kblocks) {
    const int64_t tiles = tm * tn;
    const int32_t split = (int32_t)(t / tiles);
    t -= split * tiles;
    MmTile r;
    if (a.m_group > 0) {
        const int64_t g = t / (a.m_group * tn), in = t - g * a.m_group * tn;
        const int64_t rows = min((int64_t)a.m_group, tm - g * a.m_group);
        r.n = (int32_t)(in / rows);
        r.m = (int32_t)(g * a.m_group + in - r.n * rows);
    } else {
        r.m = (int32_t)(t / tn);
        r.n = (int32_t)(t - r.m * tn);
    }
    r.kb0 = (int32_t)((int64_t)kblocks * split / a.splits);
    r.kb1 = (int32_t)((int64_t)kblocks * (split + 1) / a.splits);
    return r;
}

// Row maximum and sum of exponentials of 32 columns, into (m, s).  The difference is taken before the product with
// log2(e): exact near the maximum, however far that is from zero.
__device__ __forceinline__ void stats_chunk(float (&v)[32], float& m, float& s) {
    float top = v[0];
#pragma unroll
    for (int j = 1; j < 32; ++j) top = fmaxf(top, v[j]);
    const float next = fmaxf(m, top);
    constexpr float kLog2e = 1.4426950408889634f;
    if (next == -INFINITY) {   // nothing but -inf so far, or NaN, which the maximum passes over
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (v[j] != v[j]) s = v[j];
        return;
    }
    s = __fmul_rn(s, ex2(__fmul_rn(__fsub_rn(m, next), kLog2e)));
    float s4[4] = {};
#pragma unroll
    for (int j = 0; j < 32; ++j) s4[j & 3] = __fadd_rn(s4[j & 3], ex2(__fmul_rn(__fsub_rn(v[j], next), kLog2e)));
    s = __fadd_rn(s, __fadd_rn(__fadd_rn(s4[0], s4[1]), __fadd_rn(s4[2], s4[3])));
    m = next;
}

// out (+)= f * v for 32 columns of 32 rows of a warp; `left`: columns that exist.
template <class F>
__device__ __forceinline__ void out_chunk(const MmArgs& a, float f, float (&v)[32], int64_t row, bool row_on, int64_t col,
                                          int left, float (*sh)[33]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __fmul_rn(v[j], f);
    if (a.vec) {
        if (!row_on) return;
        uint16_t* p = a.out + row * a.ld + col;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h * 16 >= left) break;   // ld % 16 == 0: halves are whole
            uint32_t w[8];
            if (a.add) {
                ld8w(p + h * 16, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[h * 16 + 2 * j] = __fadd_rn(v[h * 16 + 2 * j], F::lo(w[j]));
                    v[h * 16 + 2 * j + 1] = __fadd_rn(v[h * 16 + 2 * j + 1], F::hi(w[j]));
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = F::pack(v[h * 16 + 2 * j], v[h * 16 + 2 * j + 1]);
            st8w(p + h * 16, w);
        }
        return;
    }
    // rows that begin anywhere: through shared memory, a row's 32 columns at a time
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 32; ++j) sh[lane][j] = v[j];
    __syncwarp();
    const uint32_t on = __ballot_sync(0xFFFFFFFFu, row_on);
    for (int r = 0; r < 32; ++r) {
        if ((on >> r & 1) && lane < left) {
            uint16_t* p = a.out + (row - lane + r) * a.ld + col + lane;
            float x = sh[r][lane];
            if (a.add) x = __fadd_rn(x, F::dec1(*p));
            *p = F::enc1(x);
        }
    }
    __syncwarp();
}

// C = A B^T of A [m, k] and B [n, k] in tiles of (128 CG) x bn, persistent.
// The loads run up to kStages blocks of K ahead of the products; two
// accumulators take turns, so that the epilogue of a tile runs under the next
// tile's products.
template <int CG, bool A_MN, bool B_MN, int EPI, class F>
__global__ void __launch_bounds__(kMmThreads, 1) mm_kernel(const __grid_constant__ CUtensorMap map_a,
                                                           const __grid_constant__ CUtensorMap map_b,
                                                           const __grid_constant__ MmArgs a) {
    using Shape = MmShape<CG>;
    constexpr int ST = Shape::kStages;
    extern __shared__ uint8_t raw[];
    uint8_t* ops = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
    float(*sh)[32][33] = reinterpret_cast<float(*)[32][33]>(ops + Shape::kOps);
    uint64_t* bars = reinterpret_cast<uint64_t*>(ops + Shape::kOps + 4 * 32 * 33 * 4);
    uint64_t* full = bars;             // [ST] in the leader: a block of both CTAs has landed
    uint64_t* empty = full + ST;       // [ST] a block has been read by the products
    uint64_t* acc_full = empty + ST;   // [2] a tile's products are done
    uint64_t* acc_empty = acc_full + 2;  // [2] in the leader: the epilogues have read the accumulator
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(acc_empty + 2);
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, 4 * CG);
        }
        fence_mbar_init();
    }
    if (warp == 5) tmem_alloc<CG>(tmem_at, 512);
    if (warp == 4 && lane == 0) {
        prefetch_map(&map_a);
        prefetch_map(&map_b);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_barrier();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;

    const int32_t count = a.head->count;
    const int64_t m_rows = a.rows_in == ROWS_M ? min((int64_t)count, a.m) : a.m;
    const int64_t k_cols = a.rows_in == ROWS_K ? min((int64_t)count, a.k) : a.k;
    const int64_t tm = (m_rows + 128 * CG - 1) / (128 * CG), tn = (a.n + a.bn - 1) / a.bn;
    const int32_t kblocks = (int32_t)((k_cols + kTileK - 1) / kTileK);
    const int64_t tiles = tm * tn * a.splits;
    const int64_t t0 = blockIdx.x / CG, step = gridDim.x / CG;
    bool ok = true;   // of this thread's waits

    if (warp == 4) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            for (int64_t t = t0; t < tiles && ok; t += step) {
                const MmTile w = mm_tile(a, t, tm, tn, kblocks);
                const int32_t ma = w.m * 128 * CG + (int32_t)rank * 128;
                const int32_t nb = w.n * a.bn + (int32_t)rank * (a.bn / CG) + a.n_off;
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                    ok = mbar_wait_cluster(empty + stage, phase ^ 1);
                    if (!ok) break;
                    const uint32_t bar = CG == 2 ? map_rank(smem_u32(full + stage), 0) : smem_u32(full + stage);
                    if (rank == 0) mbar_arrive_expect_tx(full + stage, CG * (Shape::kA + Shape::kB));
                    const uint32_t sa = smem_u32(ops) + stage * (Shape::kA + Shape::kB), sb = sa + Shape::kA;
                    const int32_t k = kb * kTileK;
                    if constexpr (A_MN) {
                        tma_load<CG>(sa, &map_a, ma, k, bar);
                        tma_load<CG>(sa + 8192, &map_a, ma + 64, k, bar);
                    } else {
                        tma_load<CG>(sa, &map_a, k, ma, bar);
                    }
                    if constexpr (B_MN) {
#pragma unroll
                        for (int j = 0; j < 4 / CG; ++j) tma_load<CG>(sb + j * 8192, &map_b, nb + 64 * j, k + a.k_off, bar);
                    } else {
                        tma_load<CG>(sb, &map_b, k + a.k_off, nb, bar);
                    }
                    if (++stage == ST) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            // until the products have read what was loaded, here and in the other CTA: neither may end before
            for (int i = 0; i < ST; ++i) {   // places never filled are free
                bool read = false;
                for (int tries = 0; tries < (ok ? 1 : kDrainTries) && !read; ++tries) read = mbar_wait_cluster(empty + stage, phase ^ 1);
                ok = ok && read;
                if (++stage == ST) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp == 5) {
        if (lane == 0 && rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int64_t done = 0;   // tiles
            for (int64_t t = t0; t < tiles && ok; t += step) {
                const MmTile w = mm_tile(a, t, tm, tn, kblocks);
                if (w.kb0 == w.kb1) continue;
                const int buf = (int)(done & 1);
                ok = mbar_wait_cluster(acc_empty + buf, (uint32_t)((done >> 1) & 1) ^ 1);
                tc_fence_after();
                for (int32_t kb = w.kb0; kb < w.kb1 && ok; ++kb) {
                    ok = mbar_wait_cluster(full + stage, phase);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t sa = smem_u32(ops) + stage * (Shape::kA + Shape::kB);
                    const uint64_t da = operand_desc(sa, A_MN), db = operand_desc(sa + Shape::kA, B_MN);
#pragma unroll
                    for (int j = 0; j < kTileK / 16; ++j)
                        tc_mma<CG>(tmem + buf * kTileN, da + j * (A_MN ? kStepMN : kStepK), db + j * (B_MN ? kStepMN : kStepK), a.idesc,
                                   kb > w.kb0 || j > 0);
                    tc_commit<CG>(empty + stage);
                    if (++stage == ST) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
                if (ok) tc_commit<CG>(acc_full + buf);
                ++done;
            }
        }
    } else {
        int64_t done = 0;
        float f = a.scale;
        if constexpr (EPI == EPI_OUT) {
            f = __fmul_rn(f, *a.share);
            if (a.scale_dev) f = __fmul_rn(f, *a.scale_dev);
        }
        for (int64_t t = t0; t < tiles && ok; t += step) {
            const MmTile w = mm_tile(a, t, tm, tn, kblocks);
            const bool any = w.kb0 < w.kb1;   // without a token that counts the sums are zeros
            const int buf = (int)(done & 1);
            const int64_t row = (int64_t)w.m * 128 * CG + rank * 128 + warp * 32 + lane;
            const int64_t n0 = (int64_t)w.n * a.bn;
            const int width = (int)min((int64_t)a.bn, a.n - n0);
            if (any) {
                ok = mbar_wait_cluster(acc_full + buf, (uint32_t)(done >> 1) & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
            }
            const uint32_t at = tmem + buf * kTileN + ((uint32_t)(warp * 32) << 16);
            [[maybe_unused]] float top = -INFINITY, sum = 0.0f, lse = 0.0f;
            [[maybe_unused]] int target = -1;
            const bool row_on = row < m_rows;
            if constexpr (EPI == EPI_STATS || EPI == EPI_DZ)
                if (row_on) target = a.target[row] - (int)n0 - (EPI == EPI_DZ ? a.n_off : 0);
            if constexpr (EPI == EPI_DZ) lse = row_on ? a.lse[a.row_of[row]] : 0.0f;
            for (int c = 0; c < width; c += 32) {
                float v[32];
                if (any) {
                    uint32_t u[32];
                    tc_ld32(at + c, u);
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                }
                const int left = width - c;
                if constexpr (EPI == EPI_STATS) {
                    if (left < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j >= left) v[j] = -INFINITY;
                    }
                    if (target >= c && target < c + 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j == target - c) a.z_target[row] = v[j];
                    }
                    stats_chunk(v, top, sum);
                } else if constexpr (EPI == EPI_DZ) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = ex2(__fmul_rn(__fsub_rn(v[j], lse), 1.4426950408889634f));
                    if (target >= c && target < c + 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j == target - c) v[j] = __fsub_rn(v[j], 1.0f);
                    }
                    if (left < 32) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (j >= left) v[j] = 0.0f;
                    }
                    uint32_t u[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        u[j] = row_on ? F::pack(__fmul_rn(v[2 * j], a.dz_scale), __fmul_rn(v[2 * j + 1], a.dz_scale)) : 0u;
                    uint16_t* p = a.dz + row * a.ld + n0 + c;
                    st8w(p, u);
                    st8w(p + 16, u + 8);
                } else if constexpr (EPI == EPI_PART) {
                    if (row_on) {
                        float* p = a.part + ((t / (tm * tn)) * a.split_rows + row) * a.ld + n0 + c;
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            if (h * 8 >= left) break;   // ld % 8 == 0
                            uint32_t u[8];
                            if (a.add) {
                                ld8w(p + h * 8, u);
#pragma unroll
                                for (int j = 0; j < 8; ++j) v[h * 8 + j] = __fadd_rn(v[h * 8 + j], __uint_as_float(u[j]));
                            }
#pragma unroll
                            for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[h * 8 + j]);
                            st8w(p + h * 8, u);
                        }
                    }
                } else {
                    out_chunk<F>(a, f, v, row, row_on, n0 + c, left, sh[warp]);
                }
            }
            if (any) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2) mbar_arrive_cluster(map_rank(smem_u32(acc_empty + buf), 0));
                    else mbar_arrive_cluster(smem_u32(acc_empty + buf));
                }
                ++done;
            }
            if constexpr (EPI == EPI_STATS)
                if (row_on) a.parts[w.n * a.part_rows + row] = make_float2(top, sum);
        }
    }
    if (!ok) atomicOr(&a.head->error, ZERO_DEVERR_WAIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_barrier();
    tc_fence_after();
    if (warp == 5) tmem_free<CG>(tmem, 512);
}

// ----------------------------------------------------------------------------
// Which tokens count
// ----------------------------------------------------------------------------
struct PickArgs {
    LossHead* head;
    const int64_t* targets;
    int32_t* slot;      // by token: its place among those that count, or -1
    int32_t* token;     // by place
    int32_t* target;    // by place
    float* losses;      // zeroed for tokens that do not count, and lse (NULL: left alone)
    float* lse;
    int64_t vocab;
    uint32_t n;
};

// One CTA walks the targets in order.
__global__ void __launch_bounds__(1024) pick_kernel(const __grid_constant__ PickArgs a) {
    __shared__ uint32_t warps[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    uint32_t base = 0;
    for (uint32_t i0 = 0; i0 < a.n; i0 += 1024) {
        const uint32_t i = i0 + threadIdx.x;
        const int64_t t = i < a.n ? a.targets[i] : -1;
        const bool on = t >= 0 && t < a.vocab;
        const uint32_t vote = __ballot_sync(0xFFFFFFFFu, on);
        if (lane == 0) warps[warp] = __popc(vote);
        __syncthreads();
        uint32_t before = lane < warp ? warps[lane] : 0, all = warps[lane];
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
            before += __shfl_xor_sync(0xFFFFFFFFu, before, s);
            all += __shfl_xor_sync(0xFFFFFFFFu, all, s);
        }
        const uint32_t at = base + before + __popc(vote & ((1u << lane) - 1));
        if (i < a.n) {
            a.slot[i] = on ? (int32_t)at : -1;
            if (on) {
                a.token[at] = (int32_t)i;
                a.target[at] = (int32_t)t;
            } else if (a.losses) {
                a.losses[i] = 0.0f;
                a.lse[i] = 0.0f;
            }
        }
        base += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        a.head->error = 0;
        a.head->count = (int32_t)base;
        a.head->ticket = 0;
    }
}

struct GatherRows {
    const LossHead* head;   // NULL: all rows, in place
    const int32_t* token;
    const uint16_t* src;
    uint16_t* dst;
    int64_t src_stride, dst_stride, rows;   // rows: of dst
    uint32_t d;
};

// Rows of d 16-bit elements, a warp each; what is behind the tokens that count
// becomes zeros, up to a whole tile.
template <int E>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ GatherRows a) {
    const int lane = threadIdx.x & 31;
    int64_t count = a.rows, end = a.rows;
    if (a.head) {
        count = a.head->count;
        end = min(a.rows, (count + 255) / 256 * 256);
    }
    const int64_t step = (int64_t)gridDim.x * kThreads / 32;
    for (int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 32; r < end; r += step) {
        const uint16_t* src = a.src + (r >= count ? 0 : a.head ? a.token[r] : r) * a.src_stride;
        uint16_t* dst = a.dst + r * a.dst_stride;
        if constexpr (E == 8) {
            for (uint32_t c = lane; c < a.d / 8; c += 32)
                reinterpret_cast<uint4*>(dst)[c] = r < count ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
        } else {
            for (uint32_t c = lane; c < a.d; c += 32) dst[c] = r < count ? __ldg(src + c) : (uint16_t)0;
        }
    }
}

// ----------------------------------------------------------------------------
// The loss from the tiles' maxima and sums
// ----------------------------------------------------------------------------
struct LossArgs {
    LossHead* head;
    const float2* parts;   // [tiles][rows]
    int64_t rows;
    int32_t tiles, blocks, reduction;
    const float* z_target;
    const int32_t* token;
    float* losses;
    float* lse;
    float* stats;
    double* block_sums;
};

// 32 tokens a block: 8 threads for each join every 8th tile, then one another
// in order.  The last CTA to end adds the blocks' sums, in order.
__global__ void __launch_bounds__(kThreads) loss_kernel(const __grid_constant__ LossArgs a) {
    __shared__ float2 sh[8][33];
    __shared__ double sums[kThreads];
    __shared__ bool last;
    constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
    const int lane = threadIdx.x & 31, part = threadIdx.x / 32;
    const int32_t count = a.head->count;
    for (int block = blockIdx.x; block < a.blocks; block += gridDim.x) {
        const int64_t row = (int64_t)block * 32 + lane;
        float m = -INFINITY, s = 0.0f;
        const auto join = [&](float2 p) {   // into (m, s)
            const float next = fmaxf(m, p.x);
            if (next == -INFINITY) {
                s = __fadd_rn(s, p.y);      // 0, or NaN
                return;
            }
            s = __fadd_rn(__fmul_rn(s, ex2(__fmul_rn(__fsub_rn(m, next), kLog2e))),
                          __fmul_rn(p.y, ex2(__fmul_rn(__fsub_rn(p.x, next), kLog2e))));
            m = next;
        };
        if (row < count)
#pragma unroll 4
            for (int t = part; t < a.tiles; t += 8) join(a.parts[(int64_t)t * a.rows + row]);
        sh[part][lane] = make_float2(m, s);
        __syncthreads();
        double loss = 0.0;
        if (part == 0) {
            if (row < count) {
                for (int p = 1; p < 8; ++p) join(sh[p][lane]);
                // log(sum exp(z)) - z_target = ln 2 (log2 s) + (m - z_target): exact where the target is the maximum
                const float ln_s = __fmul_rn(log2f(s), kLn2);
                const float one = __fadd_rn(__fsub_rn(m, a.z_target[row]), ln_s);
                const int32_t i = a.token[row];
                a.losses[i] = one;
                a.lse[i] = __fadd_rn(m, ln_s);
                loss = one;
            }
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) loss = __dadd_rn(loss, __shfl_xor_sync(0xFFFFFFFFu, loss, k));
            if (lane == 0) a.block_sums[block] = loss;
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicAdd(&a.head->ticket, 1u) == gridDim.x - 1;
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    double sum = 0.0;
    for (int b = threadIdx.x; b < a.blocks; b += kThreads) sum = __dadd_rn(sum, __ldcg(a.block_sums + b));
    sums[threadIdx.x] = sum;
    __syncthreads();
    for (int w = kThreads / 2; w > 0; w >>= 1) {
        if ((int)threadIdx.x < w) sums[threadIdx.x] = __dadd_rn(sums[threadIdx.x], sums[threadIdx.x + w]);
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const double share = a.reduction == ZERO_LOSS_MEAN ? __ddiv_rn(1.0, (double)max(count, 1)) : 1.0;
        a.stats[0] = *(volatile int32_t*)&a.head->error ? NAN : __double2float_rn(__dmul_rn(sums[0], share));
        a.stats[1] = __double2float_rn(share);
    }
}

// grad_hidden: the splits' sums times the factors, by token; zeros for tokens that do not count.
struct FinishArgs {
    const float* part;      // [splits][split_rows][ld]
    const int32_t* slot;
    uint16_t* out;          // [n][d]
    const float* share;
    const float* scale_dev;
    int64_t n, split_rows, ld;
    uint32_t d;
    int32_t splits;
    float scale;
};

template <class F, int E>
__global__ void __launch_bounds__(kThreads) finish_kernel(const __grid_constant__ FinishArgs a) {
    const int lane = threadIdx.x & 31;
    float f = __fmul_rn(a.scale, *a.share);
    if (a.scale_dev) f = __fmul_rn(f, *a.scale_dev);
    const int64_t step = (int64_t)gridDim.x * kThreads / 32;
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 32; i < a.n; i += step) {
        const int32_t at = a.slot[i];
        uint16_t* dst = a.out + i * (int64_t)a.d;
        for (uint32_t c = lane * E; c < a.d; c += 32 * E) {
            float x[E] = {};
            if (at >= 0) {
                for (int s = 0; s < a.splits; ++s) {
                    const float* p = a.part + (s * a.split_rows + at) * a.ld + c;
#pragma unroll
                    for (int e = 0; e < E; ++e) x[e] = __fadd_rn(x[e], p[e]);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = __fmul_rn(x[e], f);
            }
            if constexpr (E == 8) *reinterpret_cast<uint4*>(dst + c) = pack8<F>(x);
            else dst[c] = F::enc1(x[0]);
        }
    }
}

}  // namespace zk

using namespace zero_detail;

namespace {

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::atomic<void*> fn{nullptr};
    void* p = fn.load(std::memory_order_acquire);
    if (!p) {
        cudaDriverEntryPointQueryResult found{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(p, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(p);
}

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// rows x cols 16-bit elements, `ld` apart (ld * 2 a multiple of 16, base on a 16-byte boundary): boxes of 64 columns
// and box_rows rows, 128-byte swizzle; what lies outside reads as zero.
zero_status_t make_map(CUtensorMap* map, bool bf16, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    EncodeTiled encode = encode_tiled();
    if (!encode) return fail(ZERO_ERR_CUDA, "zero_lm_loss: no cuTensorMapEncodeTiled in the driver");
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, elem[2] = {1, 1};
    const CUresult r = encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                              const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ZERO_ERR_CUDA, "zero_lm_loss: cuTensorMapEncodeTiled failed");
    return ZERO_OK;
}

// A matrix operand: rows x cols at ld; k_inner: K runs along the rows (K-major).
struct Operand {
    const void* base;
    int64_t rows, cols, ld;
};

template <int CG, bool A_MN, bool B_MN, int EPI, class F>
zero_status_t launch_mm(const Operand& oa, const Operand& ob, zk::MmArgs a, int64_t max_tiles, cudaStream_t s, const char* what) {
    constexpr bool bf16 = std::is_same<F, zk::Bf16>::value;
    CUtensorMap ma, mb;
    zero_status_t rc = make_map(&ma, bf16, oa.base, oa.rows, oa.cols, oa.ld, A_MN ? 64 : 128);
    if (rc == ZERO_OK) rc = make_map(&mb, bf16, ob.base, ob.rows, ob.cols, ob.ld, B_MN ? 64 : 256 / CG);
    if (rc != ZERO_OK) return rc;
    a.idesc = zk::instr_desc(bf16, A_MN, B_MN, 128 * CG, a.bn);
    auto kern = zk::mm_kernel<CG, A_MN, B_MN, EPI, F>;
    constexpr int smem = zk::MmShape<CG>::kBytes;
    static std::atomic<uint64_t> allowed{0};   // by device
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (!(allowed.load(std::memory_order_relaxed) & bit) || !bit) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return after_launch(what);
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    int64_t groups = std::max(1, sm_count() / CG);
    const int32_t cap = max_ctas();
    if (cap > 0) groups = std::min<int64_t>(groups, (cap + CG - 1) / CG);
    groups = std::max<int64_t>(1, std::min(groups, max_tiles));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(groups * CG));
    cfg.blockDim = dim3(zk::kMmThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = CG;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, ma, mb, a);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(ZERO_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
    }
    return after_launch(what);
}

// Sizes and places of one call's workspace.
struct LossPlan {
    int64_t n256, ldh, ldw, vocab_tiles;
    bool copy_weight;
    int64_t piece, pieces, splits, ldo;
    // offsets: of both calls, of the forward, of the backward
    int64_t slot, token, target, hidden, weight, common;
    int64_t z_target, parts, sums, forward;
    int64_t dz, part, backward;
};

constexpr int64_t kPieceBytes = 512 << 20;

int cta_group(int64_t n) { return n <= 128 ? 1 : 2; }

LossPlan make_plan(const zero_lm_loss_args* a) {
    LossPlan p{};
    p.n256 = up(std::max<int64_t>(a->n, 1), 256);
    p.ldh = up(a->d, 8);
    p.copy_weight = (reinterpret_cast<uintptr_t>(a->weight) & 15) || a->d % 8;
    p.ldw = p.copy_weight ? p.ldh : a->d;
    p.vocab_tiles = (a->vocab + zk::kTileN - 1) / zk::kTileN;
    // dz columns at a time: few and long pieces read and write the binary32 sums of grad_hidden less often
    const int64_t all = up(a->vocab, 256);
    p.piece = a->piece > 0 ? std::min(all, up(std::min(a->piece, all), 256))
                           : std::min(all, std::max<int64_t>(4096, kPieceBytes / (2 * p.n256) / 256 * 256));
    p.pieces = (a->vocab + p.piece - 1) / p.piece;
    p.piece = up((a->vocab + p.pieces - 1) / p.pieces, 256);   // of one size
    p.pieces = (a->vocab + p.piece - 1) / p.piece;
    p.ldo = up(a->d, 8);
    // grad_hidden sums over the vocabulary: in parts, where its tiles alone would leave SMs idle
    const int cg = cta_group(a->n);
    const int64_t tiles = (p.n256 / 256) * (cg == 2 ? 1 : 1) * ((a->d + 255) / 256), slots = 152 / cg;
    p.splits = std::max<int64_t>(1, std::min<int64_t>({slots / std::max<int64_t>(tiles, 1), p.piece / 512, 64}));
    int64_t at = 256;
    const auto take = [&](int64_t bytes) { const int64_t o = at; at += up(bytes, 256); return o; };
    p.slot = take(4 * a->n);
    p.token = take(4 * a->n);
    p.target = take(4 * a->n);
    p.hidden = take(p.n256 * p.ldh * 2);
    p.weight = p.copy_weight ? take(a->vocab * p.ldw * 2) : 0;
    p.common = at;
    p.z_target = take(4 * a->n);
    p.parts = take(p.vocab_tiles * p.n256 * 8);
    p.sums = take((a->n + 31) / 32 * 8 + 8);
    p.forward = at;
    at = p.common;
    p.dz = take(p.n256 * p.piece * 2);
    p.part = take(p.splits * p.n256 * p.ldo * 4);
    p.backward = at;
    return p;
}

zero_status_t check_sizes(const char* what, const zero_lm_loss_args* a) {
    const std::string w = what;
    if (!a) return fail(ZERO_ERR_INVALID, w + ": NULL arguments");
    if (a->n < 0 || a->n > 0x7FFFFFFF) return fail(ZERO_ERR_INVALID, w + ": n must be 0 .. 2^31-1");
    if (a->d < 1 || a->d > 65536) return fail(ZERO_ERR_INVALID, w + ": d must be 1 .. 65536");
    if (a->vocab < 1 || a->vocab > 0x7FFFFFFE) return fail(ZERO_ERR_INVALID, w + ": vocab must be 1 .. 2^31-2");
    if (a->hidden_stride < a->d) return fail(ZERO_ERR_INVALID, w + ": rows overlap (hidden_stride < d)");
    if (a->dtype != ZERO_BF16 && a->dtype != ZERO_FP16) return fail(ZERO_ERR_INVALID, w + ": dtype must be ZERO_BF16 or ZERO_FP16");
    if (a->piece < 0) return fail(ZERO_ERR_INVALID, w + ": piece must be >= 0");
    if (reinterpret_cast<uintptr_t>(a->weight) & 1) return fail(ZERO_ERR_ALIGN, w + " weight: not aligned to its elements");
    return ZERO_OK;
}

zero_status_t check_at(const void* p, int size, const char* what, const char* name) {
    if (!p) return fail(ZERO_ERR_INVALID, std::string(what) + " " + name + ": NULL device pointer");
    if (reinterpret_cast<uintptr_t>(p) % size)
        return fail(ZERO_ERR_ALIGN, std::string(what) + " " + name + ": not aligned to its elements");
    return ZERO_OK;
}

template <class Kernel, class Args>
zero_status_t launch_rows(Kernel kern, int64_t rows, const Args& a, cudaStream_t s, const char* what) {
    kern<<<persistent_grid(kern, (rows * 32 + zk::kThreads - 1) / zk::kThreads), zk::kThreads, 0, s>>>(a);
    return after_launch(what);
}

// What both calls begin with: the tokens that count, their hidden states, and a weight that TMA can read.
zero_status_t gather_inputs(const zero_lm_loss_args* a, const LossPlan& p, bool forward, cudaStream_t s, const char* what) {
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    zk::PickArgs pick{};
    pick.head = reinterpret_cast<zk::LossHead*>(ws);
    pick.targets = a->targets;
    pick.slot = reinterpret_cast<int32_t*>(ws + p.slot);
    pick.token = reinterpret_cast<int32_t*>(ws + p.token);
    pick.target = reinterpret_cast<int32_t*>(ws + p.target);
    pick.losses = forward ? a->losses : nullptr;
    pick.lse = forward ? a->lse : nullptr;
    pick.vocab = a->vocab;
    pick.n = (uint32_t)a->n;
    zk::pick_kernel<<<1, 1024, 0, s>>>(pick);
    zero_status_t rc = after_launch(what);
    if (rc != ZERO_OK) return rc;
    zk::GatherRows g{};
    g.head = pick.head;
    g.token = pick.token;
    g.src = static_cast<const uint16_t*>(a->hidden);
    g.dst = reinterpret_cast<uint16_t*>(ws + p.hidden);
    g.src_stride = a->hidden_stride;
    g.dst_stride = p.ldh;
    g.rows = p.n256;
    g.d = (uint32_t)a->d;
    const bool wide = !(reinterpret_cast<uintptr_t>(a->hidden) & 15) && a->d % 8 == 0 && (a->hidden_stride % 8 == 0 || a->n == 1);
    rc = wide ? launch_rows(zk::rows_kernel<8>, p.n256, g, s, what) : launch_rows(zk::rows_kernel<1>, p.n256, g, s, what);
    if (rc != ZERO_OK || !p.copy_weight) return rc;
    zk::GatherRows w{};
    w.src = static_cast<const uint16_t*>(a->weight);
    w.dst = reinterpret_cast<uint16_t*>(ws + p.weight);
    w.src_stride = a->d;
    w.dst_stride = p.ldw;
    w.rows = a->vocab;
    w.d = (uint32_t)a->d;
    return launch_rows(zk::rows_kernel<1>, a->vocab, w, s, what);
}

// Columns of an output tile: as few tiles as there are at 256, of one width.
int32_t even_tile(int64_t n) {
    const int64_t tiles = (n + zk::kTileN - 1) / zk::kTileN;
    return (int32_t)std::min<int64_t>(zk::kTileN, up((n + tiles - 1) / tiles, 16));
}

template <int CG, class F>
zero_status_t run_forward(const zero_lm_loss_args* a, const LossPlan& p, const void* weight, cudaStream_t s, const char* what) {
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    const Operand h{ws + p.hidden, p.n256, a->d, p.ldh}, w{weight, a->vocab, a->d, p.ldw};
    zk::MmArgs m{};
    m.head = reinterpret_cast<zk::LossHead*>(ws);
    m.rows_in = zk::ROWS_M;
    m.m = a->n;
    m.n = a->vocab;
    m.k = a->d;
    m.bn = zk::kTileN;
    m.splits = 1;
    m.m_group = 32;
    m.target = reinterpret_cast<const int32_t*>(ws + p.target);
    m.parts = reinterpret_cast<float2*>(ws + p.parts);
    m.part_rows = p.n256;
    m.z_target = reinterpret_cast<float*>(ws + p.z_target);
    return launch_mm<CG, false, false, zk::EPI_STATS, F>(h, w, m, (p.n256 / 128) * p.vocab_tiles, s, what);
}

template <int CG, class F>
zero_status_t run_backward(const zero_lm_loss_args* a, const LossPlan& p, const void* weight, cudaStream_t s, const char* what) {
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    constexpr bool bf16 = std::is_same<F, zk::Bf16>::value;
    const float up_by = bf16 ? 1.0f : 16384.0f;   // of dz: fp16's normal numbers end at 2^-14
    zk::MmArgs base{};
    base.head = reinterpret_cast<zk::LossHead*>(ws);
    base.scale = (float)a->scale / up_by;
    base.scale_dev = a->scale_dev;
    base.share = a->stats + 1;
    base.splits = 1;
    zero_status_t rc = ZERO_OK;
    for (int64_t v0 = 0, i = 0; v0 < a->vocab; v0 += p.piece, ++i) {
        const int64_t cols = std::min(p.piece, a->vocab - v0);
        const Operand h{ws + p.hidden, p.n256, a->d, p.ldh}, w{weight, a->vocab, a->d, p.ldw};
        const Operand dz{ws + p.dz, p.n256, cols, p.piece};
        zk::MmArgs m = base;     // the logits of the piece, and their gradient
        m.rows_in = zk::ROWS_M;
        m.m = a->n;
        m.n = cols;
        m.k = a->d;
        m.bn = zk::kTileN;
        m.m_group = 32;
        m.n_off = (int32_t)v0;
        m.target = reinterpret_cast<const int32_t*>(ws + p.target);
        m.row_of = reinterpret_cast<const int32_t*>(ws + p.token);
        m.lse = a->lse;
        m.dz = reinterpret_cast<uint16_t*>(ws + p.dz);
        m.ld = p.piece;
        m.dz_scale = up_by;
        rc = launch_mm<CG, false, false, zk::EPI_DZ, F>(h, w, m, (p.n256 / 128) * ((cols + 255) / 256), s, what);
        if (rc != ZERO_OK) return rc;
        if (a->grad_hidden) {    // dz @ weight: K is the piece
            m = base;
            m.rows_in = zk::ROWS_M;
            m.m = a->n;
            m.n = a->d;
            m.k = cols;
            m.bn = even_tile(a->d);
            m.k_off = (int32_t)v0;
            m.splits = (int32_t)p.splits;
            m.part = reinterpret_cast<float*>(ws + p.part);
            m.split_rows = p.n256;
            m.ld = p.ldo;
            m.add = i > 0;
            rc = launch_mm<CG, false, true, zk::EPI_PART, F>(dz, w, m, (p.n256 / 128) * ((a->d + m.bn - 1) / m.bn) * p.splits, s, what);
            if (rc != ZERO_OK) return rc;
        }
        if (a->grad_weight) {    // dz^T @ hidden: K is the tokens that count
            m = base;
            m.rows_in = zk::ROWS_K;
            m.m = cols;
            m.n = a->d;
            m.k = a->n;
            m.bn = even_tile(a->d);
            m.out = static_cast<uint16_t*>(a->grad_weight) + v0 * a->d;
            m.ld = a->d;
            m.add = a->accumulate != 0;
            m.vec = (reinterpret_cast<uintptr_t>(a->grad_weight) & 31) == 0 && a->d % 16 == 0;
            rc = launch_mm<2, true, true, zk::EPI_OUT, F>(dz, h, m, ((cols + 255) / 256) * ((a->d + m.bn - 1) / m.bn), s, what);
            if (rc != ZERO_OK) return rc;
        }
    }
    if (!a->grad_hidden) return ZERO_OK;
    zk::FinishArgs f{};
    f.part = reinterpret_cast<const float*>(ws + p.part);
    f.slot = reinterpret_cast<const int32_t*>(ws + p.slot);
    f.out = static_cast<uint16_t*>(a->grad_hidden);
    f.share = a->stats + 1;
    f.scale_dev = a->scale_dev;
    f.n = a->n;
    f.split_rows = p.n256;
    f.ld = p.ldo;
    f.d = (uint32_t)a->d;
    f.splits = (int32_t)p.splits;
    f.scale = base.scale;
    const bool wide = !(reinterpret_cast<uintptr_t>(a->grad_hidden) & 15) && a->d % 8 == 0;
    return wide ? launch_rows(zk::finish_kernel<F, 8>, a->n, f, s, what) : launch_rows(zk::finish_kernel<F, 1>, a->n, f, s, what);
}

}  // namespace

extern "C" zero_status_t zero_lm_loss_query(const zero_lm_loss_args* a, int64_t* forward_bytes, int64_t* backward_bytes) {
    clear_error();
    const zero_status_t rc = check_sizes("zero_lm_loss_query", a);
    if (rc != ZERO_OK) return rc;
    const LossPlan p = make_plan(a);
    if (forward_bytes) *forward_bytes = p.forward;
    if (backward_bytes) *backward_bytes = p.backward;
    return ZERO_OK;
}

extern "C" zero_status_t zero_lm_loss_forward(const zero_lm_loss_args* a, zero_stream_t stream) {
    clear_error();
    const char* what = "zero_lm_loss_forward";
    zero_status_t rc = check_sizes(what, a);
    if (rc != ZERO_OK) return rc;
    if (a->reduction != ZERO_LOSS_MEAN && a->reduction != ZERO_LOSS_SUM)
        return fail(ZERO_ERR_INVALID, std::string(what) + ": unknown reduction");
    if ((rc = check_at(a->stats, 4, what, "stats")) != ZERO_OK) return rc;
    if (a->n > 0 && ((rc = check_at(a->hidden, 2, what, "hidden")) != ZERO_OK || (rc = check_at(a->targets, 8, what, "targets")) != ZERO_OK ||
                     (rc = check_at(a->losses, 4, what, "losses")) != ZERO_OK || (rc = check_at(a->lse, 4, what, "lse")) != ZERO_OK))
        return rc;
    if ((rc = check_at(a->weight, 2, what, "weight")) != ZERO_OK) return rc;
    if ((rc = check_dev_ptr(a->workspace, "zero_lm_loss_forward workspace")) != ZERO_OK) return rc;
    const LossPlan p = make_plan(a);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    if ((rc = gather_inputs(a, p, true, s, what)) != ZERO_OK) return rc;
    const void* weight = p.copy_weight ? ws + p.weight : a->weight;
    const bool bf16 = a->dtype == ZERO_BF16, pair = cta_group(a->n) == 2;
    rc = bf16 ? (pair ? run_forward<2, zk::Bf16>(a, p, weight, s, what) : run_forward<1, zk::Bf16>(a, p, weight, s, what))
              : (pair ? run_forward<2, zk::Fp16>(a, p, weight, s, what) : run_forward<1, zk::Fp16>(a, p, weight, s, what));
    if (rc != ZERO_OK) return rc;
    zk::LossArgs l{};
    l.head = reinterpret_cast<zk::LossHead*>(ws);
    l.parts = reinterpret_cast<const float2*>(ws + p.parts);
    l.rows = p.n256;
    l.tiles = (int32_t)p.vocab_tiles;
    l.blocks = (int32_t)((a->n + 31) / 32);
    l.reduction = a->reduction;
    l.z_target = reinterpret_cast<const float*>(ws + p.z_target);
    l.token = reinterpret_cast<const int32_t*>(ws + p.token);
    l.losses = a->losses;
    l.lse = a->lse;
    l.stats = a->stats;
    l.block_sums = reinterpret_cast<double*>(ws + p.sums);
    zk::loss_kernel<<<persistent_grid(zk::loss_kernel, std::max(1, l.blocks)), zk::kThreads, 0, s>>>(l);
    return after_launch(what);
}

extern "C" zero_status_t zero_lm_loss_backward(const zero_lm_loss_args* a, zero_stream_t stream) {
    clear_error();
    const char* what = "zero_lm_loss_backward";
    zero_status_t rc = check_sizes(what, a);
    if (rc != ZERO_OK) return rc;
    if (!std::isfinite(a->scale)) return fail(ZERO_ERR_INVALID, std::string(what) + ": scale must be finite");
    if ((rc = check_at(a->stats, 4, what, "stats")) != ZERO_OK) return rc;
    if (a->n > 0 && ((rc = check_at(a->hidden, 2, what, "hidden")) != ZERO_OK || (rc = check_at(a->targets, 8, what, "targets")) != ZERO_OK ||
                     (rc = check_at(a->lse, 4, what, "lse")) != ZERO_OK))
        return rc;
    if ((rc = check_at(a->weight, 2, what, "weight")) != ZERO_OK) return rc;
    if (a->scale_dev && (rc = check_at(a->scale_dev, 4, what, "scale_dev")) != ZERO_OK) return rc;
    if (a->grad_hidden && (rc = check_at(a->grad_hidden, 2, what, "grad_hidden")) != ZERO_OK) return rc;
    if (a->grad_weight && (rc = check_at(a->grad_weight, 2, what, "grad_weight")) != ZERO_OK) return rc;
    if ((rc = check_dev_ptr(a->workspace, "zero_lm_loss_backward workspace")) != ZERO_OK) return rc;
    if (!a->grad_hidden && !a->grad_weight) return ZERO_OK;
    const LossPlan p = make_plan(a);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    if ((rc = gather_inputs(a, p, false, s, what)) != ZERO_OK) return rc;
    const void* weight = p.copy_weight ? ws + p.weight : a->weight;
    const bool bf16 = a->dtype == ZERO_BF16, pair = cta_group(a->n) == 2;
    return bf16 ? (pair ? run_backward<2, zk::Bf16>(a, p, weight, s, what) : run_backward<1, zk::Bf16>(a, p, weight, s, what))
                : (pair ? run_backward<2, zk::Fp16>(a, p, weight, s, what) : run_backward<1, zk::Fp16>(a, p, weight, s, what));
}

extern "C" zero_status_t zero_lm_loss_device_error(const void* workspace, int32_t* bits) {
    clear_error();
    if (!bits) return fail(ZERO_ERR_INVALID, "zero_lm_loss_device_error: NULL bits");
    zero_status_t rc = check_dev_ptr(workspace, "zero_lm_loss_device_error workspace");
    if (rc != ZERO_OK) return rc;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(bits, workspace, sizeof *bits, cudaMemcpyDeviceToHost);
    return e == cudaSuccess ? ZERO_OK : fail(ZERO_ERR_CUDA, std::string("zero_lm_loss_device_error: ") + cudaGetErrorString(e));
}
