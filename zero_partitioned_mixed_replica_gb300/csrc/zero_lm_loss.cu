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
// Tokens that do not count are taken out first: pick_kernel copies the others'
// hidden states next to one another (rows of 16-byte multiples, which TMA
// wants), so that padding costs nothing and cannot spoil a sum.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "zero_launch.h"
#include "zero_tc.cuh"

namespace zk {

constexpr int kTileK = 64;            // of K in a stage: 128 bytes
constexpr int kEpiWarps = 8;          // two for each quarter of the accumulator's rows, half of the columns each
constexpr int kLoadWarp = 8, kMmaWarp = 9, kTileWarp = 10;
constexpr int kMmThreads = 32 * 11;
constexpr int kBoxBytes = 128 * 128;  // 128 rows of 64
constexpr int kTileN = 256;           // columns of a tile, at most
constexpr int kRun = 8;               // blocks of K that the tensor cores add up of a logit for few tokens, at most (MmTile)
constexpr int kFewN = 128;            // columns of a tile of logits then, at most
constexpr int kLongRun = 128;         // blocks of K that they add up of other logits, at most
constexpr int kGradRun = 512;         // and of the gradients

enum { MM_STATS = 0, MM_DZ = 1, MM_GRADS = 2 };
enum { ROWS_M = 1, ROWS_K = 2 };  // which extent is the number of tokens that count

// The workspace begins with what the kernels share.
struct LossHead {
    int32_t error;
    int32_t count;   // tokens that count
    uint32_t ticket;
    int32_t pad;
};

// One product C = A B^T, A [m, k] and B [n, k].  The last tile of a row is as
// narrow as what is left, in steps of 16 columns: at d = 1600 six tiles of 256
// and one of 64 take 0.89 of the time of seven of 240, whose loads (32 KB for
// 480 cycles of products) pass what an SM can take in (about 60 bytes a cycle).
struct MmProblem {
    int32_t rows_in;          // ROWS_M or ROWS_K
    int64_t m, n, k;          // extents (the one of rows_in at most: head->count says how many); m == 0: no product
    int32_t bn;               // columns of a tile, a multiple of 16
    int32_t splits;           // of K
    int32_t m_group;          // row tiles that follow one another while the columns stay; 0: columns first
    int32_t n_off, k_off;     // where B's rows and K begin
    uint32_t idesc;           // without the columns
};

struct MmMaps {
    CUtensorMap a[2], b[2];
};

struct MmArgs {
    LossHead* head;
    int32_t stages, b_bytes;  // b_bytes: of a widest tile's B in a stage of one CTA
    uint32_t* next;           // tiles dealt behind the first of each cluster; 0 before the launch
    MmProblem p[2];           // GRADS: dz @ weight, dz^T @ hidden; else the first alone
    // STATS, DZ
    const int32_t* target;    // of each row
    const int32_t* row_of;    // the token of each row
    const float* lse;         // DZ: by token
    float2* parts;            // STATS: [row][part_ld] maximum and sum of exponentials of half a tile's columns
    int64_t part_ld;
    float* z_target;          // STATS: the target's logit
    uint16_t* dz;             // DZ: [rows][dz_ld]
    int64_t dz_ld;
    float dz_scale;
    // GRADS
    float* part;              // binary32 sums of dz @ weight: [split][split_rows][part_cols]
    int64_t split_rows, part_cols;
    uint16_t* gh;             // not NULL: the last sums go there, at row row_of[row], instead
    uint16_t* gw;             // rows of the piece
    int64_t d;
    float scale;
    const float* scale_dev;
    const float* share;
    int32_t part_add, gw_add; // to what is there
    int32_t gw_vec;           // rows begin on 32-byte boundaries, d % 16 == 0
    float* held;              // [CTA][kHeld]: a tile's sums between its runs; NULL where none has two
};
constexpr int kHeld = 128 * kTileN;

constexpr int kMaxStages = 8;
struct MmShape {
    static constexpr int kA = kBoxBytes;                        // bytes of A in a stage; B has b_bytes
    static constexpr int kOps = 12 * kBoxBytes;                 // of all stages: 6 of 256 rows between two CTAs, 4 of one's
    static constexpr int kTurn = kEpiWarps * 32 * 17 * 4;       // transposition
    static constexpr int kSync = 512;                           // barriers, tiles dealt
    static constexpr int kBytes = 1024 + kOps + kTurn + kSync;  // and alignment
};

// The tensor cores cut the sums that they keep instead of rounding them, 16 of K at a time, all to one side: where the
// terms of a sum have one sign it comes out smaller, by about 2^-24 of itself for each 16 of K, or twice that (65536 terms
// 1.9e-4, 262144 terms 1.4e-3, several steps of fp16).  So they add runs of K, and the runs are added in binary32 with
// rounding to nearest:
//  - up to 128 tokens (CG = 1), logits: runs of up to 512 of K, added in registers.  Losses off by up to 1.8e-6
//    relatively before, below 1e-6 since, in the same time.  Tiles are then kFewN wide: for more tokens a thread would
//    hold 128 sums of a tile twice as wide, which spills;
//  - for more tokens logits in runs of up to 8192 of K (within 6e-5 for terms of one sign), the gradients of up to 32768
//    (within 1e-4, less than half of what fp16 rounds), added in `held`, each thread's own place in memory: 128 KB a CTA of
//    L2's traffic each way per run.  Gradients in runs of 8192 made the steps of 8192 tokens 3% longer, 3.01 -> 3.14 ms at
//    d 1600 and fp16.
struct alignas(16) MmTile {
    int32_t p;                // problem, or -1: no more tiles
    int32_t m, n, split;      // row tile, column tile
    int32_t kb0, kb1;         // blocks of kTileK
    int32_t width, run;       // columns that exist; blocks of a run
};

// Extents of one product, with the tokens that count.
template <int CG>
struct MmExtent {
    int64_t tm, tn, tiles;
    int32_t kblocks;

    __device__ MmExtent(const MmProblem& p, int64_t count) {
        tm = ((p.rows_in == ROWS_M ? min(count, p.m) : p.m) + 128 * CG - 1) / (128 * CG);
        tn = p.m > 0 ? (p.n + p.bn - 1) / p.bn : 0;
        kblocks = (int32_t)(((p.rows_in == ROWS_K ? min(count, p.k) : p.k) + kTileK - 1) / kTileK);
        tiles = tm * tn * p.splits;
    }
    __device__ MmTile tile(const MmProblem& p, int64_t t) const {
        MmTile r;
        const int64_t one = tm * tn;
        r.split = (int32_t)(t / one);
        t -= r.split * one;
        if (p.m_group > 0) {
            const int64_t g = t / (p.m_group * tn), in = t - g * p.m_group * tn;
            const int64_t rows = min((int64_t)p.m_group, tm - g * p.m_group);
            r.n = (int32_t)(in / rows);
            r.m = (int32_t)(g * p.m_group + in - r.n * rows);
        } else {
            r.m = (int32_t)(t / tn);
            r.n = (int32_t)(t - r.m * tn);
        }
        r.kb0 = (int32_t)((int64_t)kblocks * r.split / p.splits);
        r.kb1 = (int32_t)((int64_t)kblocks * (r.split + 1) / p.splits);
        r.width = (int32_t)min((int64_t)p.bn, p.n - (int64_t)r.n * p.bn);
        r.run = 0;
        return r;
    }
};

// The products of a launch: one, or (MM_GRADS) two.
template <int CG, int MODE>
struct MmGrid {
    MmExtent<CG> e0, e1;
    bool second;   // comes first: long tiles before short ones, so that short ones end the launch

    __device__ MmGrid(const MmArgs& a) : e0(a.p[0], a.head->count), e1(a.p[MODE == MM_GRADS], a.head->count) {
        second = MODE == MM_GRADS && e1.kblocks > e0.kblocks / a.p[0].splits;
    }
    __device__ static void set_run(MmTile& r, int32_t longest) {   // runs of about one length
        const int32_t blocks = r.kb1 - r.kb0;
        if (blocks > longest) {
            const int32_t runs = (blocks + longest - 1) / longest;
            r.run = (blocks + runs - 1) / runs;
        } else {
            r.run = max(1, blocks);
        }
    }
    __device__ int64_t all() const { return MODE == MM_GRADS ? e0.tiles + e1.tiles : e0.tiles; }
    __device__ MmTile tile(const MmArgs& a, int64_t t) const {
        if constexpr (MODE == MM_GRADS) {
            const int64_t lead = second ? e1.tiles : e0.tiles;
            const bool p1 = (t < lead) == second;
            if (t >= lead) t -= lead;
            MmTile r = p1 ? e1.tile(a.p[1], t) : e0.tile(a.p[0], t);
            r.p = p1;
            set_run(r, kGradRun);
            return r;
        } else {
            MmTile r = e0.tile(a.p[0], t);
            r.p = 0;
            set_run(r, CG == 1 ? kRun : kLongRun);
            return r;
        }
    }
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Row maximum and sum of exponentials of 32 columns, into (m, s).  The difference is taken before the product with
// log2(e): exact near the maximum, however far that is from zero.
__device__ __forceinline__ void stats_chunk(const float (&v)[32], float& m, float& s) {
    float t4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int j = 4; j < 32; ++j) t4[j & 3] = fmaxf(t4[j & 3], v[j]);
    const float next = fmaxf(m, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])));
    if (next == -INFINITY) {   // nothing but -inf so far, or NaN, which the maximum passes over
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 32; ++j) nan |= v[j] != v[j];
        if (nan) s = NAN;
        return;
    }
    s = __fmul_rn(s, ex2(__fmul_rn(__fsub_rn(m, next), kLog2e)));
    float s4[4] = {};
#pragma unroll
    for (int j = 0; j < 32; ++j) s4[j & 3] = __fadd_rn(s4[j & 3], ex2(__fmul_rn(__fsub_rn(v[j], next), kLog2e)));
    s = __fadd_rn(s, __fadd_rn(__fadd_rn(s4[0], s4[1]), __fadd_rn(s4[2], s4[3])));
    m = next;
}

// 32 columns of a row, rounded, to p (32-byte aligned), as far as `left` (a multiple of 16) columns exist.
template <class F>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&v)[32], int left, bool add) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h * 16 < left) {
            uint32_t w[8];
            if (add) {
                ld8w(p + h * 16, w);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    w[j] = pack_pair(F{}, __fadd_rn(v[h * 16 + 2 * j], F::lo(w[j])), __fadd_rn(v[h * 16 + 2 * j + 1], F::hi(w[j])));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = pack_pair(F{}, v[h * 16 + 2 * j], v[h * 16 + 2 * j + 1]);
            }
            st8w(p + h * 16, w);
        }
    }
}

// The same for rows that begin anywhere: through shared memory, two rows of 16 columns at a time.  p: the first lane's row.
template <class F>
__device__ __forceinline__ void store_turned(uint16_t* p, int64_t ld, uint32_t rows_on, const float (&v)[32], int left, bool add,
                                             float (*sh)[17]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 16; ++j) sh[lane][j] = v[h * 16 + j];
        __syncwarp();
        const int c = h * 16 + (lane & 15);
#pragma unroll 4
        for (int r = lane >> 4; r < 32; r += 2) {
            if ((rows_on >> r & 1) && c < left) {
                uint16_t* q = p + r * ld + c;
                float x = sh[r][lane & 15];
                if (add) x = __fadd_rn(x, F::dec1(*q));
                *q = F::enc1(x);
            }
        }
        __syncwarp();
    }
}

// The products of a launch, in tiles of (128 CG) x bn, persistent.  One warp
// deals tiles from a counter (SMs differ in speed by a seventh under a power
// limit, and tiles of two products in length), one loads blocks of K, six ahead
// for whole tiles, one issues the products, eight take the accumulator; two
// accumulators take turns, so that a tile's epilogue runs under the next tile's
// products.  MM_GRADS runs both products with dz, whose tiles fill one
// another's last round.
template <int CG, int MODE, class F>
__global__ void __launch_bounds__(kMmThreads, 1) mm_kernel(const __grid_constant__ MmMaps maps, const __grid_constant__ MmArgs a) {
    using Shape = MmShape;
    const int ST = a.stages;
    const uint32_t stage_bytes = Shape::kA + a.b_bytes;
    constexpr bool B_MN = MODE == MM_GRADS;
    // tiles dealt before they are begun: short tiles (logits, d of K) hide the counter's latency, long ones stay balanced
    constexpr int RING = MODE == MM_GRADS ? 2 : 3;
    extern __shared__ uint8_t raw[];
    uint8_t* ops = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
    float(*sh)[32][17] = reinterpret_cast<float(*)[32][17]>(ops + Shape::kOps);
    uint64_t* bars = reinterpret_cast<uint64_t*>(ops + Shape::kOps + Shape::kTurn);
    uint64_t* full = bars;               // [ST] in the leader: a block of both CTAs has landed
    uint64_t* empty = full + kMaxStages; // [ST] a block has been read by the products
    uint64_t* acc_full = empty + kMaxStages;  // [2] a tile's products are done
    uint64_t* acc_empty = acc_full + 2;  // [2] in the leader: the epilogues have read the accumulator
    uint64_t* tile_full = acc_empty + 2; // [RING] a tile has been dealt
    uint64_t* tile_empty = tile_full + RING;  // [RING] in the leader: all roles of both CTAs know it
    MmTile* ring = reinterpret_cast<MmTile*>(bars + 28);   // [RING]
    uint32_t* tmem_at = reinterpret_cast<uint32_t*>(ring + RING);
    static_assert(2 * kMaxStages + 4 + 2 * RING <= 28 && 28 * 8 + sizeof(MmTile) * RING + 4 <= Shape::kSync, "what the roles share");
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 2 ? cluster_rank() : 0;
    const auto leader = [](uint64_t* bar) { return CG == 2 ? map_rank(smem_u32(bar), 0) : smem_u32(bar); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + i, 1);
            mbar_init(acc_empty + i, kEpiWarps * CG);
        }
        for (int i = 0; i < RING; ++i) {
            mbar_init(tile_full + i, 1);
            mbar_init(tile_empty + i, CG * (kEpiWarps + 1) + 1);
        }
        fence_mbar_init();
    }
    if (warp == kMmaWarp) tmem_alloc<CG>(tmem_at, 512);
    if (warp == kLoadWarp && lane == 0) {
        for (int i = 0; i <= (MODE == MM_GRADS); ++i) {
            if (a.p[i].m == 0) continue;
            prefetch_map(&maps.a[i]);
            prefetch_map(&maps.b[i]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_barrier();
    tc_fence_after();
    const uint32_t tmem = *tmem_at;
    grid_wait();      // what is above ran while the kernel before this one ended
    grid_release();
    bool ok = true;   // of this thread's waits
    // the next tile; for one thread of a role
    int tile_slot = 0;
    uint32_t tile_phase = 0;
    const auto next_tile = [&]() -> MmTile {
        MmTile t;
        t.p = -1;
        ok = mbar_wait_cluster(tile_full + tile_slot, tile_phase);
        if (!ok) return t;
        const uint32_t at = smem_u32(ring + tile_slot);
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(t.p), "=r"(t.m), "=r"(t.n), "=r"(t.split) : "r"(at) : "memory");
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(t.kb0), "=r"(t.kb1), "=r"(t.width), "=r"(t.run) : "r"(at + 16) : "memory");
        mbar_arrive_remote(leader(tile_empty + tile_slot));
        if (++tile_slot == RING) {
            tile_slot = 0;
            tile_phase ^= 1;
        }
        return t;
    };

    if (warp == kTileWarp) {
        if (lane == 0 && rank == 0) {
            const MmGrid<CG, MODE> grid(a);
            const int64_t tiles = grid.all();
            int64_t t = blockIdx.x / CG;
            for (;;) {
                ok = mbar_wait_bounded(tile_empty + tile_slot, tile_phase ^ 1);
                if (!ok) break;
                MmTile w;
                w.p = -1;
                w.m = w.n = w.split = w.kb0 = w.kb1 = w.width = w.run = 0;
                if (t < tiles) w = grid.tile(a, t);
#pragma unroll
                for (int r = 0; r < CG; ++r) {
                    const uint32_t to = CG == 2 ? map_rank(smem_u32(ring + tile_slot), r) : smem_u32(ring + tile_slot);
                    const uint32_t bar = CG == 2 ? map_rank(smem_u32(tile_full + tile_slot), r) : smem_u32(tile_full + tile_slot);
                    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(w.p), "r"(w.m), "r"(w.n), "r"(w.split) : "memory");
                    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + 16), "r"(w.kb0), "r"(w.kb1), "r"(w.width), "r"(w.run) : "memory");
                    mbar_arrive_cluster(bar);
                }
                if (w.p < 0) break;
                if (++tile_slot == RING) {
                    tile_slot = 0;
                    tile_phase ^= 1;
                }
                t = gridDim.x / CG + (int64_t)atomicAdd(a.next, 1u);
            }
        }
    } else if (warp == kLoadWarp) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            const uint32_t full0 = leader(full), ops0 = smem_u32(ops);
            // one tile's blocks; what differs between the products is known at compile time
            const auto load = [&](auto a_mn_, const MmTile& w, const CUtensorMap* map_a, const CUtensorMap* map_b, const MmProblem& p) {
                constexpr bool A_MN = decltype(a_mn_)::value;
                const int32_t ma = w.m * 128 * CG + (int32_t)rank * 128;
                // logits: a box of bn / CG rows of the weight; else boxes of 64 columns, as many as the tile has
                const int32_t cols = B_MN ? (w.width + 15) / 16 * 16 / CG : p.bn / CG, k_off = p.k_off;
                const int32_t nb = w.n * p.bn + (int32_t)rank * cols + p.n_off;
                const int32_t boxes = (cols + 63) / 64;
                const uint32_t bytes = CG * (Shape::kA + (B_MN ? boxes * 8192 : cols * 128));
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                    ok = mbar_wait_bounded(empty + stage, phase ^ 1);
                    if (!ok) break;
                    const uint32_t bar = full0 + stage * 8;
                    if (rank == 0) mbar_arrive_expect_tx(full + stage, bytes);
                    const uint32_t sa = ops0 + stage * stage_bytes, sb = sa + Shape::kA;
                    const int32_t k = kb * kTileK;
                    if constexpr (A_MN) {
                        tma_load<CG>(sa, map_a, ma, k, bar);
                        tma_load<CG>(sa + 8192, map_a, ma + 64, k, bar);
                    } else {
                        tma_load<CG>(sa, map_a, k, ma, bar);
                    }
                    if constexpr (B_MN) {
#pragma unroll
                        for (int j = 0; j < 4 / CG; ++j)
                            if (j < boxes) tma_load<CG>(sb + j * 8192, map_b, nb + 64 * j, k + k_off, bar);
                    } else {
                        tma_load<CG>(sb, map_b, k + k_off, nb, bar);
                    }
                    if (++stage == ST) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            };
            for (MmTile w; (w = next_tile()).p >= 0;) {
                if constexpr (MODE == MM_GRADS) {
                    if (w.p == 0) load(std::false_type{}, w, &maps.a[0], &maps.b[0], a.p[0]);
                    else load(std::true_type{}, w, &maps.a[1], &maps.b[1], a.p[1]);
                } else {
                    load(std::false_type{}, w, &maps.a[0], &maps.b[0], a.p[0]);
                }
                if (!ok) break;
            }
            // until the products have read what was loaded, here and in the other CTA: neither may end before
            // (places never filled are free)
            const bool all = ok;
            for (int i = 0; i < ST; ++i) {
                bool read = false;
                for (int tries = 0; tries < (all ? 1 : kDrainTries) && !read; ++tries) read = mbar_wait_bounded(empty + stage, phase ^ 1);
                ok = ok && read;
                if (++stage == ST) {
                    stage = 0;
                    phase ^= 1;
                }
            }
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0 && rank == 0) {
            int stage = 0;
            uint32_t phase = 0;
            int64_t done = 0;   // accumulators
            const auto multiply = [&](auto a_mn_, int32_t kb0, int32_t kb1, uint32_t idesc, uint32_t acc) {
                constexpr bool A_MN = decltype(a_mn_)::value;
                const uint64_t da0 = operand_desc(smem_u32(ops), A_MN), db0 = operand_desc(smem_u32(ops) + Shape::kA, B_MN);
                for (int32_t kb = kb0; kb < kb1; ++kb) {
                    ok = mbar_wait_bounded(full + stage, phase);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t at = (uint64_t)(stage * (stage_bytes >> 4));
#pragma unroll
                    for (int j = 0; j < kTileK / 16; ++j)
                        tc_mma<CG>(acc, da0 + at + j * (A_MN ? kStepMN : kStepK), db0 + at + j * (B_MN ? kStepMN : kStepK), idesc,
                                   kb > kb0 || j > 0);
                    tc_commit<CG>(empty + stage);
                    if (++stage == ST) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            };
            for (MmTile w; (w = next_tile()).p >= 0;) {
                if (w.kb0 == w.kb1) continue;
                // the columns: of the last tile no more than there are (logits: what the box has loaded beyond them does no harm)
                const uint32_t columns = (uint32_t)(B_MN ? (w.width + 15) / 16 * 16 : a.p[0].bn) >> 3 << 17;
                for (int32_t k0 = w.kb0; k0 < w.kb1 && ok; k0 += w.run) {
                    const int32_t k1 = min(k0 + w.run, w.kb1);
                    const int buf = (int)(done & 1);
                    ok = mbar_wait_bounded(acc_empty + buf, (uint32_t)((done >> 1) & 1) ^ 1);
                    if (!ok) break;
                    tc_fence_after();
                    if constexpr (MODE == MM_GRADS) {
                        if (w.p == 0) multiply(std::false_type{}, k0, k1, a.p[0].idesc | columns, tmem + buf * kTileN);
                        else multiply(std::true_type{}, k0, k1, a.p[1].idesc | columns, tmem + buf * kTileN);
                    } else {
                        multiply(std::false_type{}, k0, k1, a.p[0].idesc | columns, tmem + buf * kTileN);
                    }
                    if (!ok) break;
                    tc_commit<CG>(acc_full + buf);
                    ++done;
                }
                if (!ok) break;
            }
        }
    } else {
        const int half = warp >> 2;   // of the columns; a warp reads the rows of its quarter, warp % 4
        int64_t done = 0;
        const int64_t rows0 = min((int64_t)a.head->count, a.p[0].m), rows1 = a.p[1].m;
        float f = a.scale;
        if constexpr (MODE == MM_GRADS) {
            f = __fmul_rn(f, *a.share);
            if (a.scale_dev) f = __fmul_rn(f, *a.scale_dev);
        }
        for (;;) {
            MmTile w;
            w.p = -1;
            if (lane == 0) w = next_tile();
            w.p = __shfl_sync(0xFFFFFFFFu, w.p, 0);
            if (w.p < 0) break;
            w.m = __shfl_sync(0xFFFFFFFFu, w.m, 0);
            w.n = __shfl_sync(0xFFFFFFFFu, w.n, 0);
            w.split = __shfl_sync(0xFFFFFFFFu, w.split, 0);
            w.kb0 = __shfl_sync(0xFFFFFFFFu, w.kb0, 0);
            w.kb1 = __shfl_sync(0xFFFFFFFFu, w.kb1, 0);
            w.width = __shfl_sync(0xFFFFFFFFu, w.width, 0);
            w.run = __shfl_sync(0xFFFFFFFFu, w.run, 0);
            const MmProblem& p = a.p[w.p];
            const int64_t row0 = (int64_t)w.m * 128 * CG + rank * 128 + (warp & 3) * 32, row = row0 + lane;
            const bool row_on = row < (w.p == 0 ? rows0 : rows1);
            const int64_t n0 = (int64_t)w.n * p.bn;
            constexpr int HALF = CG == 1 && MODE != MM_GRADS ? kFewN / 2 : kTileN / 2;
            const int c0 = half * HALF, c1 = half == 0 ? min(w.width, HALF) : w.width;
            // the next accumulator is full; it has been read
            const auto take = [&]() -> uint32_t {
                ok = mbar_wait_bounded(acc_full + (done & 1), (uint32_t)(done >> 1) & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                tc_fence_after();
                return tmem + (uint32_t)(done & 1) * kTileN + ((uint32_t)((warp & 3) * 32) << 16);
            };
            const auto give = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(leader(acc_empty + (done & 1)));
                ++done;
            };
            // all runs of K but the last into this thread's place, where the last finds their sums
            [[maybe_unused]] const bool runs = w.kb0 + w.run < w.kb1;
            const auto held_at = [&](int c) { return a.held + (int64_t)blockIdx.x * kHeld + warp * (kHeld / kEpiWarps) + (c - c0) * 32 + lane * 8; };
            const auto add_held = [&](int c, float (&v)[32]) {
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t u[8];
                    ld8w(held_at(c) + h * 256, u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[h * 8 + j] = __fadd_rn(__uint_as_float(u[j]), v[h * 8 + j]);
                }
            };
            const auto hold_runs = [&] {
                for (int32_t k0 = w.kb0; k0 + w.run < w.kb1; k0 += w.run) {
                    const uint32_t at = take();
                    if (!ok) return;
                    for (int c = c0; c < c1; c += 32) {
                        uint32_t u[32];
                        tc_ld32(at + c, u);
                        tc_wait_ld();
                        float v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
                        if (k0 > w.kb0) add_held(c, v);
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[h * 8 + j]);
                            st8w(held_at(c) + h * 256, u);
                        }
                    }
                    give();
                }
            };
            if constexpr (MODE != MM_GRADS) {
                const int target = row_on ? a.target[row] - (int)n0 - p.n_off : -1;
                [[maybe_unused]] float top = -INFINITY, sum = 0.0f, lse = 0.0f;
                if constexpr (MODE == MM_DZ) lse = row_on ? a.lse[a.row_of[row]] : 0.0f;
                // 32 columns of logits from c on, `left` of them (or more) in this half
                const auto use = [&](float (&v)[32], int c, int left) {
                    if constexpr (MODE == MM_STATS) {
                        if (left < 32) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j >= left) v[j] = -INFINITY;
                        }
                        if (target >= c && target < min(c + 32, c1)) {
                            // predicated stores: of a choice among registers the compiler makes an array in local memory
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %0, %1;\n\t@p st.global.f32 [%2], %3;\n\t}" ::"r"(target - c), "r"(j),
                                             "l"(a.z_target + row), "f"(v[j])
                                             : "memory");
                        }
                        stats_chunk(v, top, sum);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = ex2(__fmul_rn(__fsub_rn(v[j], lse), kLog2e));
                        if (target >= c && target < min(c + 32, c1)) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = __fsub_rn(v[j], j == target - c ? 1.0f : 0.0f);
                        }
                        if (left < 32) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (j >= left) v[j] = 0.0f;
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = row_on ? __fmul_rn(v[j], a.dz_scale) : 0.0f;
                        store_row<F>(a.dz + row * a.dz_ld + n0 + c, v, left, false);   // 16 columns at a time: bn % 16 == 0
                    }
                };
                if constexpr (CG == 1) {
                    float z[2][32];
                    for (int32_t k0 = w.kb0; k0 < w.kb1; k0 += w.run) {
                        const uint32_t at = take();
                        if (!ok) break;
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            if (c0 + g * 32 < c1) {
                                uint32_t u[32];
                                tc_ld32(at + c0 + g * 32, u);
                                tc_wait_ld();
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    z[g][j] = k0 == w.kb0 ? __uint_as_float(u[j]) : __fadd_rn(z[g][j], __uint_as_float(u[j]));
                            }
                        }
                        give();
                    }
                    if (!ok) break;
#pragma unroll
                    for (int g = 0; g < 2; ++g)
                        if (c0 + g * 32 < c1) use(z[g], c0 + g * 32, c1 - c0 - g * 32);
                } else {
                    hold_runs();
                    if (!ok) break;
                    const uint32_t at = take();
                    if (!ok) break;
                    for (int c = c0; c < c1; c += 32) {
                        uint32_t u[32];
                        tc_ld32(at + c, u);
                        tc_wait_ld();
                        float v[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
                        if (runs) add_held(c, v);
                        use(v, c, c1 - c);
                    }
                    give();
                }
                if constexpr (MODE == MM_STATS)
                    if (row_on) a.parts[row * a.part_ld + 2 * w.n + half] = make_float2(top, sum);
            } else {
                const bool any = w.kb0 < w.kb1;   // without a token that counts the sums are zeros
                hold_runs();
                if (!ok) break;
                const uint32_t at = any ? take() : 0;
                if (!ok) break;
                for (int c = c0; c < c1; c += 32) {
                    float v[32];
                    if (any) {
                        uint32_t u[32];
                        tc_ld32(at + c, u);
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(u[j]);
                        if (runs) add_held(c, v);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                    }
                    const int left = c1 - c;
                    if (w.p == 0) {
                        if (row_on) {
                            float* q = a.part + (w.split * a.split_rows + row) * a.part_cols + n0 + c;
                            if (a.part_add) {
#pragma unroll
                                for (int h = 0; h < 4; ++h) {
                                    if (h * 8 < left) {   // part_cols % 8 == 0
                                        uint32_t u[8];
                                        ld8w(q + h * 8, u);
#pragma unroll
                                        for (int j = 0; j < 8; ++j) v[h * 8 + j] = __fadd_rn(v[h * 8 + j], __uint_as_float(u[j]));
                                    }
                                }
                            }
                            if (a.gh) {
#pragma unroll
                                for (int j = 0; j < 32; ++j) v[j] = __fmul_rn(v[j], f);
                                store_row<F>(a.gh + a.row_of[row] * a.d + n0 + c, v, left, false);
                            } else {
#pragma unroll
                                for (int h = 0; h < 4; ++h) {
                                    if (h * 8 < left) {
                                        uint32_t u[8];
#pragma unroll
                                        for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[h * 8 + j]);
                                        st8w(q + h * 8, u);
                                    }
                                }
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __fmul_rn(v[j], f);
                        if (a.gw_vec) {
                            if (row_on) store_row<F>(a.gw + row * a.d + n0 + c, v, left, a.gw_add);
                        } else {
                            store_turned<F>(a.gw + row0 * a.d + n0 + c, a.d, __ballot_sync(0xFFFFFFFFu, row_on), v, left, a.gw_add, sh[warp]);
                        }
                    }
                }
                if (any) give();
            }
        }
    }
    if (!ok) atomicOr(&a.head->error, ZERO_DEVERR_WAIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_barrier();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_free<CG>(tmem, 512);
}

// ----------------------------------------------------------------------------
// Which tokens count, and their hidden states
// ----------------------------------------------------------------------------
struct PickArgs {
    LossHead* head;
    uint32_t* next;     // counters of the products' launches, zeroed
    int32_t nexts;
    const int64_t* targets;
    int32_t* slot;      // by token: its place among those that count, or -1
    int32_t* token;     // by place
    int32_t* target;    // by place
    float* losses;      // zeroed for tokens that do not count, and lse (NULL: left alone)
    float* lse;
    uint16_t* zero;     // [n][d], the same (NULL: left alone)
    const uint16_t* src;  // hidden states, src_stride apart
    uint16_t* dst;      // by place, dst_stride apart, `rows` of them
    int64_t src_stride, dst_stride, rows;
    int64_t vocab;
    uint32_t n, d, per_cta;
};

constexpr int kPickThreads = 512;

template <int E>
__device__ __forceinline__ void copy_row(uint16_t* dst, const uint16_t* src, uint32_t d, uint32_t at, uint32_t step) {
    if constexpr (E == 8) {
#pragma unroll 8
        for (uint32_t c = at; c < d / 8; c += step)
            reinterpret_cast<uint4*>(dst)[c] = src ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll 8
        for (uint32_t c = at; c < d; c += step) dst[c] = src ? __ldg(src + c) : (uint16_t)0;
    }
}

// A CTA has per_cta tokens.  It counts those before them that count (every CTA
// reads all targets: 64 KB at 8192 tokens), places its own, and copies their
// rows, a warp each; behind the last one come zeros up to a whole tile.
template <int E>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const __grid_constant__ PickArgs a) {
    constexpr int W = kPickThreads / 32;
    __shared__ uint32_t sums[2][W];
    __shared__ int32_t place[kPickThreads];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    grid_release();
    const auto counts = [&](int64_t t) { return t >= 0 && t < a.vocab; };
    const uint32_t b0 = (uint32_t)min((uint64_t)a.n, (uint64_t)blockIdx.x * a.per_cta);
    const uint32_t b1 = (uint32_t)min((uint64_t)a.n, (uint64_t)b0 + a.per_cta);
    uint32_t before = 0, all = 0;
#pragma unroll 8
    for (uint64_t i = threadIdx.x; i < a.n; i += kPickThreads) {
        const bool on = counts(__ldg(a.targets + i));
        all += on;
        before += on && i < b0;
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        before += __shfl_xor_sync(0xFFFFFFFFu, before, s);
        all += __shfl_xor_sync(0xFFFFFFFFu, all, s);
    }
    if (lane == 0) {
        sums[0][warp] = before;
        sums[1][warp] = all;
    }
    __syncthreads();
    before = all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        before += sums[0][w];
        all += sums[1][w];
    }
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) {
            a.head->error = 0;
            a.head->count = (int32_t)all;
            a.head->ticket = 0;
        }
        for (int i = threadIdx.x; i < a.nexts; i += kPickThreads) a.next[i] = 0;
    }
    for (uint32_t i0 = b0; i0 < b1; i0 += kPickThreads) {
        const uint32_t i = i0 + threadIdx.x;
        const int64_t t = i < b1 ? __ldg(a.targets + i) : -1;
        const bool on = counts(t);
        const uint32_t vote = __ballot_sync(0xFFFFFFFFu, on);
        __syncthreads();       // sums and place have been read
        if (lane == 0) sums[0][warp] = __popc(vote);
        __syncthreads();
        uint32_t at = before, in_all = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            at += w < warp ? sums[0][w] : 0;
            in_all += sums[0][w];
        }
        at += __popc(vote & ((1u << lane) - 1));
        place[threadIdx.x] = on ? (int32_t)at : -1;
        if (i < b1) {
            a.slot[i] = on ? (int32_t)at : -1;
            if (on) {
                a.token[at] = (int32_t)i;
                a.target[at] = (int32_t)t;
            } else if (a.losses) {
                a.losses[i] = 0.0f;
                a.lse[i] = 0.0f;
            }
        }
        before += in_all;
        __syncthreads();
        const uint32_t tokens = min((uint32_t)kPickThreads, b1 - i0);
        for (uint32_t j = warp; j < tokens; j += W) {
            const int32_t to = place[j];
            if (to >= 0)
                copy_row<E>(a.dst + to * a.dst_stride, a.src + (int64_t)(i0 + j) * a.src_stride, a.d, lane, 32);
            else if (a.zero)
                copy_row<1>(a.zero + (int64_t)(i0 + j) * a.d, nullptr, a.d, lane, 32);
        }
    }
    const int64_t end = min(a.rows, ((int64_t)all + 255) / 256 * 256);
    for (int64_t r = all + blockIdx.x; r < end; r += gridDim.x) copy_row<E>(a.dst + r * a.dst_stride, nullptr, a.d, threadIdx.x, kPickThreads);
}

// A matrix of rows x d, elements next to one another from anywhere on, into
// rows `ld` apart that begin on 16-byte boundaries.
struct CopyArgs {
    const uint16_t* src;
    uint16_t* dst;
    int64_t rows, ld;
    uint32_t d;
};

// 8 elements a lane, from 5 aligned words shifted by 0 or 16 bits.  A matrix that
// begins or ends in the middle of a word has the other two bytes of that word
// read and thrown away (device allocations are whole words); words wholly behind
// it are not read.  What a row's last piece has of the next row lies between d
// and ld, which no product reads.
__global__ void __launch_bounds__(kThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
    const uint32_t lane = threadIdx.x & 31, pieces = (a.d + 7) / 8;
    const int64_t step = (int64_t)gridDim.x * kThreads / 32;
    const uintptr_t end = reinterpret_cast<uintptr_t>(a.src + a.rows * (int64_t)a.d);
    for (int64_t r = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 32; r < a.rows; r += step) {
        const uint16_t* src = a.src + r * (int64_t)a.d;
        uint4* dst = reinterpret_cast<uint4*>(a.dst + r * a.ld);
#pragma unroll 2
        for (uint32_t c = lane; c < pieces; c += 32) {
            const uintptr_t at = reinterpret_cast<uintptr_t>(src + (size_t)c * 8), word = at & ~(uintptr_t)3;
            uint32_t w[5];
#pragma unroll
            for (int k = 0; k < 5; ++k) w[k] = word + 4 * k < end ? __ldg(reinterpret_cast<const uint32_t*>(word) + k) : 0u;
            const uint32_t shift = (uint32_t)(at & 3) * 8;
            dst[c] = make_uint4(__funnelshift_r(w[0], w[1], shift), __funnelshift_r(w[1], w[2], shift), __funnelshift_r(w[2], w[3], shift),
                                __funnelshift_r(w[3], w[4], shift));
        }
    }
}

// ----------------------------------------------------------------------------
// The loss from the tiles' maxima and sums
// ----------------------------------------------------------------------------
struct LossArgs {
    LossHead* head;
    const float2* parts;   // [row][tiles]
    int64_t ld;
    int32_t tiles, blocks, reduction;
    const float* z_target;
    const int32_t* token;
    float* losses;
    float* lse;
    float* stats;
    double* block_sums;
};

constexpr int kLossRows = kThreads / 32;

// A warp for each token, kLossRows of them a block: the maximum of its parts,
// then the sum at that maximum.  The last CTA to end adds the blocks' sums, in
// order.
__global__ void __launch_bounds__(kThreads) loss_kernel(const __grid_constant__ LossArgs a) {
    __shared__ double sums[kThreads];
    __shared__ bool last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    grid_wait();
    const int32_t count = a.head->count;
    for (int block = blockIdx.x; block < a.blocks; block += gridDim.x) {
        const int64_t row = (int64_t)block * kLossRows + warp;
        double loss = 0.0;
        if (row < count) {
            const float2* p = a.parts + row * a.ld;
            float m = -INFINITY, s = 0.0f;
#pragma unroll 4
            for (int t = lane; t < a.tiles; t += 32) m = fmaxf(m, __ldg(p + t).x);
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, k));
#pragma unroll 4
            for (int t = lane; t < a.tiles; t += 32) {
                const float2 x = __ldg(p + t);
                // all -inf: the sums are zeros, or NaN
                s = __fadd_rn(s, m == -INFINITY ? x.y : __fmul_rn(x.y, ex2(__fmul_rn(__fsub_rn(x.x, m), kLog2e))));
            }
#pragma unroll
            for (int k = 16; k > 0; k >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, k));
            // log(sum exp(z)) - z_target = (m - z_target) + ln 2 log2(s): exact where the target is the maximum
            const float ln_s = __fmul_rn(log2f(s), kLn2);
            const float one = __fadd_rn(__fsub_rn(m, a.z_target[row]), ln_s);
            if (lane == 0) {
                const int32_t i = a.token[row];
                a.losses[i] = one;
                a.lse[i] = __fadd_rn(m, ln_s);
            }
            loss = one;
        }
        if (lane == 0) sums[warp] = loss;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kLossRows; ++w) loss = __dadd_rn(loss, sums[w]);
            a.block_sums[block] = loss;
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
#pragma unroll 4
    for (int b = threadIdx.x; b < a.blocks; b += kThreads) sum = __dadd_rn(sum, __ldcg(a.block_sums + b));
    sums[threadIdx.x] = sum;
    __syncthreads();
    for (int w = kThreads / 2; w > 0; w >>= 1) {
        if ((int)threadIdx.x < w) sums[threadIdx.x] = __dadd_rn(sums[threadIdx.x], sums[threadIdx.x + w]);
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        const double share = a.reduction == ZERO_LOSS_MEAN ? __ddiv_rn(1.0, (double)max(count, 1)) : 1.0;
        // after an error lse is not whole either, and the backward call has no other word of it: share is a factor of each
        // of its gradients
        const bool whole = *(volatile int32_t*)&a.head->error == 0;
        a.stats[0] = whole ? __double2float_rn(__dmul_rn(sums[0], share)) : NAN;
        a.stats[1] = whole ? __double2float_rn(share) : NAN;
    }
}

// grad_hidden: the splits' sums times the factors, by token; zeros for tokens
// that do not count.  A warp takes 32 loads' width of a row: with a row each, 45
// tokens of 2048 in 17 splits took 58 us instead of 11.
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
    grid_wait();
    float f = __fmul_rn(a.scale, *a.share);
    if (a.scale_dev) f = __fmul_rn(f, *a.scale_dev);
    const int64_t step = (int64_t)gridDim.x * kThreads / 32;
    const uint32_t pieces = (a.d + 32 * E - 1) / (32 * E);
    for (int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / 32; item < a.n * pieces; item += step) {
        const int64_t i = item / pieces;
        const uint32_t c = ((uint32_t)(item - i * pieces) * 32 + lane) * E;
        if (c >= a.d) continue;
        const int32_t at = a.slot[i];
        float x[E] = {};
        if (at >= 0) {
#pragma unroll 8
            for (int s = 0; s < a.splits; ++s) {
                const float* p = a.part + (s * a.split_rows + at) * a.ld + c;
                if constexpr (E == 8) {   // ld % 8 == 0
                    const float4 u = __ldcs(reinterpret_cast<const float4*>(p)), v = __ldcs(reinterpret_cast<const float4*>(p) + 1);
                    const float y[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = __fadd_rn(x[e], y[e]);
                } else {
                    x[0] = __fadd_rn(x[0], *p);
                }
            }
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = __fmul_rn(x[e], f);
        }
        uint16_t* dst = a.out + i * (int64_t)a.d + c;
        if constexpr (E == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(pack_pair(F{}, x[0], x[1]), pack_pair(F{}, x[2], x[3]), pack_pair(F{}, x[4], x[5]),
                                                                      pack_pair(F{}, x[6], x[7]));
        else *dst = F::enc1(x[0]);
    }
}

// After a backward call whose kernels gave up waiting the gradients are not
// whole: NaN in their first rows makes the step that reads them skip.
struct VerdictArgs {
    const LossHead* head;
    uint16_t* gh;
    uint16_t* gw;
    uint32_t d;
    uint16_t nan;
};

__global__ void __launch_bounds__(32) verdict_kernel(const __grid_constant__ VerdictArgs a) {
    grid_wait();
    if (a.head->error == 0) return;
    for (uint32_t c = threadIdx.x; c < a.d; c += 32) {
        if (a.gh) a.gh[c] = a.nan;
        if (a.gw) a.gw[c] = a.nan;
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

// A matrix operand: rows x cols at ld, read in boxes of box_rows x 64.
struct Operand {
    const void* base;
    int64_t rows, cols, ld;
    int box_rows;
};

constexpr int64_t kSlots = 152;   // SMs of a GB300: what the splits of work are made for

// Tiles of a launch at most (all tokens counting).
template <int CG>
int64_t most_tiles(const zk::MmProblem& p) {
    return p.m > 0 ? (p.m + 128 * CG - 1) / (128 * CG) * ((p.n + p.bn - 1) / p.bn) * p.splits : 0;
}

template <int CG, int MODE, class F>
zero_status_t launch_mm(const Operand* oa, const Operand* ob, zk::MmArgs a, cudaStream_t s, const char* what) {
    constexpr bool bf16 = std::is_same<F, zk::Bf16>::value;
    zk::MmMaps maps{};
    for (int i = 0; i < 2; ++i) {
        zk::MmProblem& p = a.p[i];
        if (p.m == 0) {
            p.splits = p.bn = 1;
            continue;
        }
        zero_status_t rc = make_map(&maps.a[i], bf16, oa[i].base, oa[i].rows, oa[i].cols, oa[i].ld, oa[i].box_rows);
        if (rc == ZERO_OK) rc = make_map(&maps.b[i], bf16, ob[i].base, ob[i].rows, ob[i].cols, ob[i].ld, ob[i].box_rows);
        if (rc != ZERO_OK) return rc;
        p.idesc = zk::instr_desc(bf16, MODE == zk::MM_GRADS && i == 1, MODE == zk::MM_GRADS, 128 * CG, 0);
    }
    // B of a stage: the box of a logits' tile, or boxes of 64 columns; 1024 bytes are a group of the swizzle
    a.b_bytes = MODE == zk::MM_GRADS ? 2 * zk::kBoxBytes / CG : (int32_t)up(a.p[0].bn / CG * 128, 1024);
    a.stages = std::min(zk::kMaxStages, zk::MmShape::kOps / (zk::MmShape::kA + a.b_bytes));
    auto kern = zk::mm_kernel<CG, MODE, F>;
    constexpr int smem = zk::MmShape::kBytes;
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
    if (a.held) groups = std::min(groups, kSlots / CG);   // what it has places for
    groups = std::max<int64_t>(1, std::min(groups, most_tiles<CG>(a.p[0]) + most_tiles<CG>(a.p[1])));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(groups * CG));
    cfg.blockDim = dim3(zk::kMmThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, maps, a);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(ZERO_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
    }
    return after_launch(what);
}

int cta_group(int64_t n) { return n <= 128 ? 1 : 2; }

// Columns of a tile: as few tiles as there are at the widest, of one width.
int32_t even_tile(int64_t n, int64_t widest) {
    const int64_t tiles = (n + widest - 1) / widest;
    return (int32_t)std::min<int64_t>(widest, up((n + tiles - 1) / tiles, 16));
}

// Columns of a tile of logits.  Few tokens: loads bound the time, and what the
// busiest SM has of them: rounds of tiles times their rows, for single CTAs
// (CG = 1) those of the hidden states too.
int32_t logit_tile(int64_t n, int64_t vocab) {
    const int64_t cg = cta_group(n), slots = kSlots / cg, rows = (n + 128 * cg - 1) / (128 * cg);
    const int64_t widest = cg == 1 ? zk::kFewN : zk::kTileN, least = cg == 1 ? 32 : 96, more = cg == 1 ? 128 : 0;
    const auto cost = [&](int64_t bn) { return ((vocab + bn - 1) / bn * rows + slots - 1) / slots * (bn + more); };
    int64_t best = even_tile(vocab, widest);
    if ((vocab + best - 1) / best * rows < 8 * slots)
        for (int64_t bn = widest; bn >= least; bn -= 16)
            if (cost(bn) < cost(best)) best = bn;
    return (int32_t)best;
}

// Sizes and places of one call's workspace.
struct LossPlan {
    int64_t n256, ldh, ldw, part_ld;
    bool copy_weight;
    int32_t logit_bn, d_bn;
    int64_t piece, pieces, splits, ldo;
    // offsets: of both calls, of the forward, of the backward
    int64_t next, slot, token, target, hidden, weight;
    int64_t z_target, parts, sums, held_f, forward;
    int64_t dz, part, held_b, backward;   // held: 0 where no sum has two runs
};

constexpr int64_t kPieceBytes = 512 << 20;

LossPlan make_plan(const zero_lm_loss_args* a) {
    LossPlan p{};
    p.n256 = up(std::max<int64_t>(a->n, 1), 256);
    p.ldh = up(a->d, 8);
    p.copy_weight = (reinterpret_cast<uintptr_t>(a->weight) & 15) || a->d % 8;
    p.ldw = p.copy_weight ? p.ldh : a->d;
    p.logit_bn = logit_tile(a->n, a->vocab);
    p.part_ld = 2 * ((a->vocab + p.logit_bn - 1) / p.logit_bn);
    // dz columns at a time: few and long pieces read and write the binary32 sums of grad_hidden less often
    const int64_t all = up(a->vocab, 256);
    p.piece = a->piece > 0 ? std::min(all, up(std::min(a->piece, all), 256))
                           : std::min(all, std::max<int64_t>(4096, kPieceBytes / (2 * p.n256) / 256 * 256));
    p.pieces = (a->vocab + p.piece - 1) / p.piece;
    p.piece = up((a->vocab + p.pieces - 1) / p.pieces, 256);   // of one size
    p.pieces = (a->vocab + p.piece - 1) / p.piece;
    p.ldo = up(a->d, 8);
    p.d_bn = (int32_t)std::min<int64_t>(zk::kTileN, up(a->d, 16));
    // dz @ weight sums over the piece, dz^T @ hidden over the tokens, in one launch.  The first in parts, so that a tile of
    // it is at most half of what an SM has to do.
    const int64_t cg = cta_group(a->n), slots = kSlots / cg, columns = (a->d + p.d_bn - 1) / p.d_bn;
    const int64_t tiles0 = (a->n + 128 * cg - 1) / (128 * cg) * columns, kb0 = (p.piece + 63) / 64;
    const int64_t tiles1 = (p.piece + 128 * cg - 1) / (128 * cg) * columns, kb1 = (a->n + 63) / 64;
    const int64_t share = std::max<int64_t>(8, (tiles0 * kb0 + tiles1 * kb1) / slots / 2);
    p.splits = std::max<int64_t>(1, std::min<int64_t>({(kb0 + share - 1) / share, 32, (64 << 20) / (p.n256 * p.ldo * 4)}));
    const bool long_d = cg == 2 && (a->d + 63) / 64 > zk::kLongRun;
    const bool long_grads = std::max((kb0 + p.splits - 1) / p.splits, kb1) > zk::kGradRun;
    constexpr int64_t held = kSlots * zk::kHeld * 4;
    int64_t at = 256;
    const auto take = [&](int64_t bytes) { const int64_t o = at; at += up(bytes, 256); return o; };
    p.next = take(4 * (2 * p.pieces + 1));
    p.slot = take(4 * a->n);
    p.token = take(4 * a->n);
    p.target = take(4 * a->n);
    p.hidden = take(p.n256 * p.ldh * 2);
    p.weight = p.copy_weight ? take(a->vocab * p.ldw * 2) : 0;
    const int64_t common = at;
    p.z_target = take(4 * a->n);
    p.parts = take(p.part_ld * a->n * 8);
    p.sums = take((a->n + zk::kLossRows - 1) / zk::kLossRows * 8 + 8);
    p.held_f = long_d ? take(held) : 0;
    p.forward = at;
    at = common;
    p.dz = take(p.n256 * p.piece * 2);
    p.part = take(p.splits * p.n256 * p.ldo * 4);
    p.held_b = long_d || long_grads ? take(held) : 0;
    p.backward = at;
    return p;
}

zero_status_t check_sizes(const char* what, const zero_lm_loss_args* a) {
    const std::string w = what;
    if (!a) return fail(ZERO_ERR_INVALID, w + ": NULL arguments");
    constexpr int64_t kMost = 1 << 30;   // coordinates of tiles are 32-bit
    if (a->n < 0 || a->n > kMost) return fail(ZERO_ERR_INVALID, w + ": n must be 0 .. 2^30");
    if (a->d < 1 || a->d > 65536) return fail(ZERO_ERR_INVALID, w + ": d must be 1 .. 65536");
    if (a->vocab < 1 || a->vocab > kMost) return fail(ZERO_ERR_INVALID, w + ": vocab must be 1 .. 2^30");
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

bool direct_grad_hidden(const zero_lm_loss_args* a, const LossPlan& p) {
    return a->grad_hidden && p.splits == 1 && (reinterpret_cast<uintptr_t>(a->grad_hidden) & 31) == 0 && a->d % 16 == 0;
}

// What both calls begin with: the tokens that count, their hidden states, and a weight that TMA can read.
zero_status_t gather_inputs(const zero_lm_loss_args* a, const LossPlan& p, bool forward, cudaStream_t s, const char* what) {
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    zk::PickArgs k{};
    k.head = reinterpret_cast<zk::LossHead*>(ws);
    k.next = reinterpret_cast<uint32_t*>(ws + p.next);
    k.nexts = (int32_t)(2 * p.pieces + 1);
    k.targets = a->targets;
    k.slot = reinterpret_cast<int32_t*>(ws + p.slot);
    k.token = reinterpret_cast<int32_t*>(ws + p.token);
    k.target = reinterpret_cast<int32_t*>(ws + p.target);
    k.losses = forward ? a->losses : nullptr;
    k.lse = forward ? a->lse : nullptr;
    k.zero = !forward && direct_grad_hidden(a, p) ? static_cast<uint16_t*>(a->grad_hidden) : nullptr;
    k.src = static_cast<const uint16_t*>(a->hidden);
    k.dst = reinterpret_cast<uint16_t*>(ws + p.hidden);
    k.src_stride = a->hidden_stride;
    k.dst_stride = p.ldh;
    k.rows = up(std::max<int64_t>(a->n, 1), 128 * cta_group(a->n));   // whole tiles
    k.vocab = a->vocab;
    k.n = (uint32_t)a->n;
    k.d = (uint32_t)a->d;
    const bool wide = !(reinterpret_cast<uintptr_t>(a->hidden) & 15) && a->d % 8 == 0 && (a->hidden_stride % 8 == 0 || a->n == 1);
    const auto kern = wide ? zk::pick_kernel<8> : zk::pick_kernel<1>;
    // 16 tokens a CTA, but CTAs enough for the zeros behind a few tokens: 1 CTA took 30 us for 255 rows, 64 take 6
    const int grid = persistent_grid(kern, std::min<int64_t>(std::max<int64_t>((a->n + 15) / 16, 64), 2 * kSlots), 0, zk::kPickThreads);
    k.per_cta = (uint32_t)((a->n + grid - 1) / grid);
    kern<<<grid, zk::kPickThreads, 0, s>>>(k);
    const zero_status_t rc = after_launch(what);
    if (rc != ZERO_OK || !p.copy_weight) return rc;
    const zk::CopyArgs w{static_cast<const uint16_t*>(a->weight), reinterpret_cast<uint16_t*>(ws + p.weight), a->vocab, p.ldw, (uint32_t)a->d};
    return launch_rows(zk::copy_kernel, a->vocab, w, s, what);
}

zk::MmArgs mm_args(const zero_lm_loss_args* a, const LossPlan& p) {
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    zk::MmArgs m{};
    m.head = reinterpret_cast<zk::LossHead*>(ws);
    m.next = reinterpret_cast<uint32_t*>(ws + p.next);
    m.target = reinterpret_cast<const int32_t*>(ws + p.target);
    m.row_of = reinterpret_cast<const int32_t*>(ws + p.token);
    m.lse = a->lse;
    m.d = a->d;
    return m;
}

// hidden @ weight^T for `cols` columns of the vocabulary from v0 on.
template <int CG>
zk::MmProblem logits_of(const zero_lm_loss_args* a, int64_t v0, int64_t cols, int32_t bn) {
    zk::MmProblem p{};
    p.rows_in = zk::ROWS_M;
    p.m = a->n;
    p.n = cols;
    p.k = a->d;
    p.bn = bn;
    p.splits = 1;
    p.m_group = 32;   // 32 tiles of hidden states stay in L2 while the weight streams by
    p.n_off = (int32_t)v0;
    return p;
}

template <int CG, class F>
zero_status_t run_forward(const zero_lm_loss_args* a, const LossPlan& p, const void* weight, cudaStream_t s, const char* what) {
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    const Operand h{ws + p.hidden, p.n256, a->d, p.ldh, 128}, w{weight, a->vocab, a->d, p.ldw, p.logit_bn / CG};
    zk::MmArgs m = mm_args(a, p);
    m.p[0] = logits_of<CG>(a, 0, a->vocab, p.logit_bn);
    m.parts = reinterpret_cast<float2*>(ws + p.parts);
    m.part_ld = p.part_ld;
    m.z_target = reinterpret_cast<float*>(ws + p.z_target);
    m.held = p.held_f ? reinterpret_cast<float*>(ws + p.held_f) : nullptr;
    return launch_mm<CG, zk::MM_STATS, F>(&h, &w, m, s, what);
}

template <int CG, class F>
zero_status_t run_backward(const zero_lm_loss_args* a, const LossPlan& p, const void* weight, cudaStream_t s, const char* what) {
    uint8_t* ws = static_cast<uint8_t*>(a->workspace);
    constexpr bool bf16 = std::is_same<F, zk::Bf16>::value;
    const float up_by = bf16 ? 1.0f : 16384.0f;   // of dz: fp16's normal numbers end at 2^-14
    const bool direct = direct_grad_hidden(a, p);
    zk::MmArgs base = mm_args(a, p);
    base.dz = reinterpret_cast<uint16_t*>(ws + p.dz);
    base.dz_ld = p.piece;
    base.dz_scale = up_by;
    base.part = reinterpret_cast<float*>(ws + p.part);
    base.split_rows = p.n256;
    base.part_cols = p.ldo;
    base.held = p.held_b ? reinterpret_cast<float*>(ws + p.held_b) : nullptr;
    base.scale = (float)a->scale / up_by;
    base.scale_dev = a->scale_dev;
    base.share = a->stats + 1;
    base.gw_add = a->accumulate != 0;
    base.gw_vec = (reinterpret_cast<uintptr_t>(a->grad_weight) & 31) == 0 && a->d % 16 == 0;
    zero_status_t rc = ZERO_OK;
    for (int64_t i = 0; i < p.pieces; ++i) {
        const int64_t v0 = i * p.piece, cols = std::min(p.piece, a->vocab - v0);
        const int32_t bn = std::min<int32_t>(p.logit_bn, even_tile(cols, CG == 1 ? zk::kFewN : zk::kTileN));
        {   // the logits of the piece, and their gradient
            const Operand h{ws + p.hidden, p.n256, a->d, p.ldh, 128}, w{weight, a->vocab, a->d, p.ldw, bn / CG};
            zk::MmArgs m = base;
            m.next += 2 * i;
            m.p[0] = logits_of<CG>(a, v0, cols, bn);
            rc = launch_mm<CG, zk::MM_DZ, F>(&h, &w, m, s, what);
            if (rc != ZERO_OK) return rc;
        }
        const Operand oa[2] = {{ws + p.dz, p.n256, cols, p.piece, 128}, {ws + p.dz, p.n256, cols, p.piece, 64}};
        const Operand ob[2] = {{weight, a->vocab, a->d, p.ldw, 64}, {ws + p.hidden, p.n256, a->d, p.ldh, 64}};
        zk::MmArgs m = base;
        m.next += 2 * i + 1;
        if (a->grad_hidden) {    // dz @ weight: K is the piece
            m.p[0].rows_in = zk::ROWS_M;
            m.p[0].m = a->n;
            m.p[0].n = a->d;
            m.p[0].k = cols;
            m.p[0].bn = p.d_bn;
            m.p[0].k_off = (int32_t)v0;
            m.p[0].splits = (int32_t)p.splits;
            m.part_add = i > 0;
            m.gh = direct && i == p.pieces - 1 ? static_cast<uint16_t*>(a->grad_hidden) : nullptr;
        }
        if (a->grad_weight) {    // dz^T @ hidden: K is the tokens that count
            m.p[1].rows_in = zk::ROWS_K;
            m.p[1].m = cols;
            m.p[1].n = a->d;
            m.p[1].k = a->n;
            m.p[1].bn = p.d_bn;
            m.p[1].splits = 1;
            m.gw = static_cast<uint16_t*>(a->grad_weight) + v0 * a->d;
        }
        rc = launch_mm<CG, zk::MM_GRADS, F>(oa, ob, m, s, what);
        if (rc != ZERO_OK) return rc;
    }
    if (a->grad_hidden && !direct && a->n > 0) {
        zk::FinishArgs f{};
        f.part = base.part;
        f.slot = reinterpret_cast<const int32_t*>(ws + p.slot);
        f.out = static_cast<uint16_t*>(a->grad_hidden);
        f.share = base.share;
        f.scale_dev = a->scale_dev;
        f.n = a->n;
        f.split_rows = p.n256;
        f.ld = p.ldo;
        f.d = (uint32_t)a->d;
        f.splits = (int32_t)p.splits;
        f.scale = base.scale;
        const bool wide = !(reinterpret_cast<uintptr_t>(a->grad_hidden) & 15) && a->d % 8 == 0;
        const auto kern = wide ? zk::finish_kernel<F, 8> : zk::finish_kernel<F, 1>;
        const int64_t width = wide ? 32 * 8 : 32, items = a->n * ((a->d + width - 1) / width);
        rc = launch_after(kern, dim3((unsigned)persistent_grid(kern, (items + 7) / 8)), zk::kThreads, 0, s, what, f);
        if (rc != ZERO_OK) return rc;
    }
    const zk::VerdictArgs v{base.head, a->n > 0 ? static_cast<uint16_t*>(a->grad_hidden) : nullptr, static_cast<uint16_t*>(a->grad_weight),
                            (uint32_t)a->d, (uint16_t)(bf16 ? 0x7FC0 : 0x7E00)};
    return launch_after(zk::verdict_kernel, dim3(1), 32, 0, s, what, v);
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
    l.ld = p.part_ld;
    l.tiles = (int32_t)p.part_ld;
    l.blocks = (int32_t)((a->n + zk::kLossRows - 1) / zk::kLossRows);
    l.reduction = a->reduction;
    l.z_target = reinterpret_cast<const float*>(ws + p.z_target);
    l.token = reinterpret_cast<const int32_t*>(ws + p.token);
    l.losses = a->losses;
    l.lse = a->lse;
    l.stats = a->stats;
    l.block_sums = reinterpret_cast<double*>(ws + p.sums);
    return launch_after(zk::loss_kernel, dim3((unsigned)persistent_grid(zk::loss_kernel, std::max(1, l.blocks))), zk::kThreads, 0, s, what, l);
}

extern "C" zero_status_t zero_lm_loss_backward(const zero_lm_loss_args* a, zero_stream_t stream) {
    clear_error();
    const char* what = "zero_lm_loss_backward";
    zero_status_t rc = check_sizes(what, a);
    if (rc != ZERO_OK) return rc;
    if (!std::isfinite((float)a->scale)) return fail(ZERO_ERR_INVALID, std::string(what) + ": scale must be finite in binary32");
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
