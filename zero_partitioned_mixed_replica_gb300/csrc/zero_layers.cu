// Embedding lookup and layer norm, forward and backward.
//
// All four move each element once or twice and compute a handful of
// operations on it: they are bound by memory, and for few tokens by the
// latency of a launch.  Rows are read in the widest pieces that every tensor
// of the call allows (E elements: 16 bytes where all rows begin on a 16-byte
// boundary; 4 bytes, or single elements, for tensors anywhere in a flat
// buffer).
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "zero_launch.h"

namespace zk {

namespace cg = cooperative_groups;

struct Fp32 {
    using S = float;
};
template <class F>
struct Store {
    using S = uint16_t;
};
template <>
struct Store<Fp32> {
    using S = float;
};

// E elements from p, widened; p is aligned to min(16, E * size) bytes.
template <class F, int E>
__device__ __forceinline__ void ld_e(const typename Store<F>::S* __restrict__ p, float (&o)[E]) {
    if constexpr (sizeof(typename Store<F>::S) == 4) {
        if constexpr (E % 4 == 0) {
#pragma unroll
            for (int k = 0; k < E / 4; ++k) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(p) + k);
                o[4 * k] = x.x; o[4 * k + 1] = x.y; o[4 * k + 2] = x.z; o[4 * k + 3] = x.w;
            }
        } else if constexpr (E == 2) {
            const float2 x = __ldg(reinterpret_cast<const float2*>(p));
            o[0] = x.x; o[1] = x.y;
        } else {
            o[0] = __ldg(p);
        }
    } else if constexpr (E == 8) {
        unpack8<F>(__ldg(reinterpret_cast<const uint4*>(p)), o);
    } else if constexpr (E == 2) {
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(p));
        o[0] = F::lo(w);
        o[1] = F::hi(w);
    } else {
        static_assert(E == 1, "8, 2 or 1 16-bit elements");
        o[0] = F::dec1(__ldg(p));
    }
}

// The same as it lies in memory, to be widened where it is used: half the registers.
template <class F, int E>
struct Raw {
    using S = typename Store<F>::S;
    static constexpr int kWords = E * (int)sizeof(S) >= 4 ? E * (int)sizeof(S) / 4 : 1;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const S* __restrict__ p) {
        if constexpr (kWords == 4) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else {
            static_assert(kWords == 1, "16, 4 or 2 bytes");
            if constexpr (E * sizeof(S) == 4) w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
            else w[0] = __ldg(p);
        }
    }
    // What is made of the words is made from here on, not where they were loaded.
    __device__ __forceinline__ void hold() {
#pragma unroll
        for (int k = 0; k < kWords; ++k) asm volatile("" : "+r"(w[k]));
    }
    __device__ __forceinline__ void get(float (&o)[E]) const {
        if constexpr (sizeof(S) == 4) {
#pragma unroll
            for (int k = 0; k < E; ++k) o[k] = __uint_as_float(w[k]);
        } else if constexpr (E == 1) {
            o[0] = F::dec1((uint16_t)w[0]);
        } else {
#pragma unroll
            for (int k = 0; k < E / 2; ++k) {
                o[2 * k] = F::lo(w[k]);
                o[2 * k + 1] = F::hi(w[k]);
            }
        }
    }
};

// Two binary32 operations in one instruction, each rounded to nearest.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(F2 x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x.v)); }
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

template <class F, int E>
__device__ __forceinline__ void st_e(typename Store<F>::S* p, const float (&o)[E]) {
    if constexpr (sizeof(typename Store<F>::S) == 4) {
        if constexpr (E % 4 == 0) {
#pragma unroll
            for (int k = 0; k < E / 4; ++k)
                reinterpret_cast<float4*>(p)[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        } else if constexpr (E == 2) {
            *reinterpret_cast<float2*>(p) = make_float2(o[0], o[1]);
        } else {
            *p = o[0];
        }
    } else if constexpr (E == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_pair(F{}, o[0], o[1]), pack_pair(F{}, o[2], o[3]), pack_pair(F{}, o[4], o[5]),
                                                  pack_pair(F{}, o[6], o[7]));
    } else if constexpr (E == 2) {
        *reinterpret_cast<uint32_t*>(p) = pack_pair(F{}, o[0], o[1]);
    } else {
        *p = F::enc1(o[0]);
    }
}

// What is already there, added; not through the read-only path: this launch writes it.
template <class F, int E>
__device__ __forceinline__ void add_e(const typename Store<F>::S* p, float (&o)[E]) {
    if constexpr (sizeof(typename Store<F>::S) == 2 && E == 8) {
        float old[8];
        unpack8<F>(*reinterpret_cast<const uint4*>(p), old);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = __fadd_rn(old[e], o[e]);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (sizeof(typename Store<F>::S) == 4)
                o[e] = __fadd_rn(p[e], o[e]);
            else
                o[e] = __fadd_rn(F::dec1(p[e]), o[e]);
        }
    }
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xFFFFFFFFu, x, m));
    return x;
}

// ----------------------------------------------------------------------------
// Embedding
// ----------------------------------------------------------------------------
struct EmbedArgs {
    const void* weight;
    const int64_t* ids;
    void* out;
    int64_t vocab, n;
    uint32_t d, dv;      // elements and pieces of a row
    int32_t lanes_log2;  // lanes of a warp that share a row
    float scale;
};

// A row goes to 1, 2, .. 32 lanes of a warp, the fewest that cover it.  Memory
// bounds it: 8192 rows of 1600 bf16 take 8.7 us, 6.0 TB/s.
template <class F, int E>
__global__ void __launch_bounds__(kThreads) embed_kernel(const __grid_constant__ EmbedArgs a) {
    using S = typename Store<F>::S;
    const uint32_t lanes = 1u << a.lanes_log2;
    const uint32_t c0 = threadIdx.x & (lanes - 1);
    const int64_t per_grid = ((int64_t)gridDim.x * kThreads) >> a.lanes_log2;
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> a.lanes_log2; i < a.n; i += per_grid) {
        const int64_t id = __ldg(a.ids + i);
        const bool inside = id >= 0 && id < a.vocab;
        const S* src = static_cast<const S*>(a.weight) + (inside ? id : 0) * (int64_t)a.d;
        S* dst = static_cast<S*>(a.out) + i * (int64_t)a.d;
#pragma unroll 4
        for (uint32_t c = c0; c < a.dv; c += lanes) {
            float x[E] = {};
            if (inside) {
                ld_e<F, E>(src + (size_t)c * E, x);
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = __fmul_rn(x[e], a.scale);
            }
            st_e<F, E>(dst + (size_t)c * E, x);
        }
    }
}

// The tokens sorted by id, stable: a radix sort of (id, position) pairs in
// 8-bit digits by one thread-block cluster, whose CTAs exchange their digit
// counts through distributed shared memory; an id outside the vocabulary
// becomes `vocab` and sorts behind all others.  The clusters behind the first
// zero the gradient meanwhile.  SHARED: the pairs stay in the cluster's shared
// memory between the passes; under the zeroing's traffic a trip to memory takes
// 2 us, and a pass of the other form, for more tokens than that holds, makes
// three.
constexpr int kSortThreads = 1024;
constexpr uint32_t kPairsPad = 16;   // entries behind the pairs, which are read 4 at a time and 4 ahead
constexpr int kSortWarps = kSortThreads / 32;

struct SortArgs {
    const int64_t* ids;
    uint64_t* pairs[2];  // id << 32 | position; the result is in pairs[passes & 1]
    uint8_t* zero;       // zero_bytes of it are zeroed
    int64_t zero_bytes;
    int64_t vocab;
    uint32_t n;
    uint32_t per_warp;   // tokens of a warp, next to one another: a multiple of 32
    int32_t passes;
};

__device__ __forceinline__ uint64_t id_pair(const SortArgs& a, uint32_t i) {
    const int64_t id = __ldg(a.ids + i);
    const uint64_t key = id >= 0 && id < a.vocab ? (uint64_t)id : (uint64_t)a.vocab;
    return key << 32 | i;
}

template <bool SHARED>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ __align__(16) uint64_t held[];   // SHARED: [2][pairs of a CTA]
    __shared__ __align__(128) uint32_t counts[kSortWarps][256];  // of a digit in a warp's tokens; then where the next one goes
    __shared__ uint32_t total[256];                    // of a digit in this CTA's tokens
    __shared__ uint32_t warp_total[8];
    grid_release();
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ctas = cluster.num_blocks(), rank = cluster.block_rank();
    if (blockIdx.x >= ctas) {  // zero the gradient: bytes to a 16-byte boundary, 32 KB of zeros over and over, bytes
        const int64_t t = (int64_t)(blockIdx.x - ctas) * kSortThreads + threadIdx.x;
        const int64_t head = min(a.zero_bytes, (int64_t)(-reinterpret_cast<intptr_t>(a.zero) & 15));
        const int64_t whole = (a.zero_bytes - head) / 16 * 16, tail = head + whole;
        if (t < head) a.zero[t] = 0;
        if (tail + t < a.zero_bytes) a.zero[tail + t] = 0;   // fewer than 16
        for (uint32_t i = threadIdx.x; i < kSortWarps * 256; i += kSortThreads) counts[0][i] = 0;
        fence_proxy_async_smem();
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int64_t at = (int64_t)(blockIdx.x - ctas) * (int64_t)sizeof counts; at < whole; at += (int64_t)(gridDim.x - ctas) * (int64_t)sizeof counts)
                bulk_s2g(a.zero + head + at, counts, (uint32_t)min(whole - at, (int64_t)sizeof counts));
            bulk_commit();
            bulk_wait_all<0>();
        }
        return;
    }
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (rank == 0 && threadIdx.x < kPairsPad) a.pairs[a.passes & 1][(uint64_t)a.n + threadIdx.x] = ~0ull;
    const uint32_t per_cta = kSortWarps * a.per_warp, cta0 = rank * per_cta;   // at most n + 2^15
    const uint32_t w0 = min(a.n, cta0 + warp * a.per_warp), w1 = min(a.n, w0 + a.per_warp);
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = 32 + 8 * pass;
        uint64_t* mine = held + (SHARED ? (size_t)(pass & 1) * per_cta : 0);
        // 8 of a lane's pairs at a time: the counter and the ranks below go one after another
        const auto load8 = [&](uint32_t i0, uint64_t (&p)[8]) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t i = i0 + k * 32 + lane;
                p[k] = i >= w1 ? 0 : pass == 0 ? id_pair(a, i) : SHARED ? mine[i - cta0] : a.pairs[pass & 1][i];
            }
        };
        for (uint32_t d = lane; d < 256; d += 32) counts[warp][d] = 0;
        __syncwarp();
        uint64_t p[8];
        for (uint32_t i0 = w0; i0 < w1; i0 += 256) {
            load8(i0, p);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (i0 + k * 32 + lane < w1) atomicAdd(&counts[warp][(p[k] >> shift) & 255], 1u);
        }
        __syncthreads();
        if (threadIdx.x < 256) {
            uint32_t in_cta = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) in_cta += counts[w][threadIdx.x];
            total[threadIdx.x] = in_cta;
        }
        cluster.sync();
        uint32_t before = 0, all = 0, scan = 0;  // of this digit in the CTAs before this one, and in all; of the digits up to it
        if (threadIdx.x < 256) {
#pragma unroll
            for (uint32_t r = 0; r < 8; ++r) {   // ctas is 8 at most
                const uint32_t c = r < ctas ? cluster.map_shared_rank(total, r)[threadIdx.x] : 0;
                before += r < rank ? c : 0;
                all += c;
            }
            scan = all;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, scan, s);
                if (lane >= (uint32_t)s) scan += x;
            }
            if (lane == 31) warp_total[warp] = scan;
        }
        __syncthreads();
        if (threadIdx.x < 256) {
            uint32_t base = scan - all + before;
#pragma unroll
            for (uint32_t w = 0; w < 8; ++w) base += w < warp ? warp_total[w] : 0;
#pragma unroll
            for (int w0 = 0; w0 < kSortWarps; w0 += 16) {   // loads before stores, which the compiler keeps in order
                uint32_t c[16];
#pragma unroll
                for (int w = 0; w < 16; ++w) c[w] = counts[w0 + w][threadIdx.x];
#pragma unroll
                for (int w = 0; w < 16; ++w) {
                    counts[w0 + w][threadIdx.x] = base;
                    base += c[w];
                }
            }
        }
        __syncthreads();
        const bool to_memory = !SHARED || pass + 1 == a.passes;
        uint64_t* out = a.pairs[(pass + 1) & 1];
        for (uint32_t i0 = w0; i0 < w1; i0 += 256) {  // in order: equal digits keep theirs
            if (i0 > w0 || a.per_warp > 256) load8(i0, p);   // else they are there from the count
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const bool on = i0 + k * 32 + lane < w1;
                const uint32_t live = __ballot_sync(0xFFFFFFFFu, on);
                if (on) {
                    const uint32_t digit = (p[k] >> shift) & 255;
                    const uint32_t same = __match_any_sync(live, digit);
                    const uint32_t at = counts[warp][digit];
                    __syncwarp(live);
                    if (lane == (uint32_t)(__ffs(same) - 1)) counts[warp][digit] = at + __popc(same);
                    const uint32_t to = at + __popc(same & ((1u << lane) - 1));
                    if (to_memory) {
                        out[to] = p[k];
                    } else {
                        const uint32_t cta = to / per_cta;
                        uint64_t* there = cluster.map_shared_rank(held, cta);
                        there[(size_t)((pass + 1) & 1) * per_cta + (to - cta * per_cta)] = p[k];
                    }
                }
                __syncwarp();
            }
        }
        // the pairs, and the counts of all CTAs, before the next pass reads and overwrites them
        if (to_memory) __threadfence();
        cluster.sync();
    }
}

// The sorted tokens are cut into pieces of `piece` (a multiple of 8).  Lanes add
// the rows of a piece's tokens, id after id.  What begins and ends in the piece
// is a gradient's row; what reaches into another piece goes into a binary32
// row of its own (slot 0: it came from the piece before; slot 1: it begins
// here), which embed_join_kernel adds up.
struct EmbedGradArgs {
    const void* grad;
    const uint64_t* pairs;
    void* out;
    float* parts;  // [pieces][2][d]
    uint32_t n, pieces, d, dv, vocab;
    int32_t piece;
    int32_t accumulate;
    float scale;
};

template <class F, class O, int E>
__device__ __forceinline__ void embed_row(const EmbedGradArgs& a, uint32_t id, uint32_t c, float (&x)[E]) {
    typename Store<O>::S* p = static_cast<typename Store<O>::S*>(a.out) + (size_t)id * a.d + (size_t)c * E;
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = __fmul_rn(x[e], a.scale);
    if (a.accumulate) add_e<O, E>(p, x);
    st_e<O, E>(p, x);
}

// LANES lanes of a warp have a piece and as many of its columns: a whole warp
// where rows are wide, so that warps of one piece are next to one another and
// none waits for another.  4 rows are under way at a time in each of 32 warps: 8
// rows in the 16 to 24 warps that their registers allow took 1.5 times as long.
template <class F, class O, int E, int LANES>
__global__ void __launch_bounds__(kThreads, 4) embed_grad_kernel(const __grid_constant__ EmbedGradArgs a) {
    using S = typename Store<F>::S;
    const uint32_t lane = threadIdx.x & (LANES - 1);
    const uint32_t slices = (a.dv + LANES - 1) / LANES;
    const uint64_t items = (uint64_t)a.pieces * slices, step = (uint64_t)gridDim.x * (kThreads / LANES);
    grid_wait();
    grid_release();
    for (uint64_t item = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) / LANES; item < items; item += step) {
        const uint32_t q = (uint32_t)(item / slices), c = (uint32_t)(item - (uint64_t)q * slices) * LANES + lane;
        const uint32_t b = q * a.piece, e = min(a.n, b + a.piece);
        const bool on = c < a.dv;
        const uint32_t id_before = b > 0 ? (uint32_t)(__ldg(a.pairs + b - 1) >> 32) : ~0u;
        const uint32_t id_after = e < a.n ? (uint32_t)(__ldg(a.pairs + e) >> 32) : ~0u;
        // (position, id) of 4 tokens; behind the last one lie kPairsPad that are none
        uint4 pairs[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) pairs[k] = __ldg(reinterpret_cast<const uint4*>(a.pairs + b) + k);
        float sum[E] = {};
        uint32_t id = pairs[0].y;
        bool first = true;  // the piece's first id
        const auto flush = [&](uint32_t next) {
            if (on && id < a.vocab) {
                const bool came = first && id == id_before, goes = next == id;
                if (came || goes) {
                    st_e<Fp32, E>(a.parts + ((size_t)q * 2 + (came ? 0 : 1)) * a.d + (size_t)c * E, sum);
                } else {
                    embed_row<F, O, E>(a, id, c, sum);
                }
            }
            first = false;
        };
        const S* column = static_cast<const S*>(a.grad) + (on ? (size_t)c * E : 0);
        for (uint32_t i = b; i < e; i += 4) {
            Raw<F, E> raw[4];
            uint32_t ids[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                ids[k] = k & 1 ? pairs[k / 2].w : pairs[k / 2].y;
                if (ids[k] < a.vocab) raw[k].load(column + (size_t)(k & 1 ? pairs[k / 2].z : pairs[k / 2].x) * a.d);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) pairs[k] = __ldg(reinterpret_cast<const uint4*>(a.pairs + i + 4) + k);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (ids[k] < a.vocab) {
                    float x[E];
                    raw[k].get(x);
                    if (ids[k] != id) {
                        flush(ids[k]);
                        id = ids[k];
#pragma unroll
                        for (int j = 0; j < E; ++j) sum[j] = x[j];
                    } else if constexpr (E > 1) {
#pragma unroll
                        for (int j = 0; j < E; j += 2) split(add2(f2(sum[j], sum[j + 1]), f2(x[j], x[j + 1])), sum[j], sum[j + 1]);
                    } else {
                        sum[0] = __fadd_rn(sum[0], x[0]);
                    }
                }
            }
        }
        // behind the last row of an id in the vocabulary come only padding tokens, which flush nothing
        flush(id_after);
    }
}

// Adds up the parts of an id whose rows begin in piece q and go on behind it:
// slot 1 of q, slot 0 of the pieces after it.  A warp looks at a piece; what has
// more than 8 parts is added by the CTA, a warp every eighth of them, and the
// warps in order (the first token of a Zipf-distributed text is in a hundred
// pieces).
template <class F, class O, int E>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const __grid_constant__ EmbedGradArgs a) {
    constexpr uint32_t W = kThreads / 32;
    __shared__ float sh[W][32 * E];
    __shared__ uint32_t parts_of[W], id_of[W];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    grid_wait();
    for (uint32_t q0 = blockIdx.x * W; q0 + 1 < a.pieces; q0 += gridDim.x * W) {
        const uint32_t q = q0 + warp;
        uint32_t parts = 0, id = 0;
        if (q + 1 < a.pieces) {
            const uint32_t b = q * a.piece, e = b + a.piece;
            id = (uint32_t)(__ldg(a.pairs + e) >> 32);
            const uint32_t last = (uint32_t)(__ldg(a.pairs + e - 1) >> 32), before = b > 0 ? (uint32_t)(__ldg(a.pairs + b - 1) >> 32) : ~0u;
            if (id < a.vocab && last == id && before != id) {   // else nothing goes on here, or it is an earlier piece's
                uint32_t lo = e, hi = a.n;  // a place with this id, one behind its last: 32 probes at a time
                while (hi - lo > 1) {
                    const uint32_t at = lo + (uint32_t)((uint64_t)(hi - lo) * (lane + 1) / 33);
                    const uint32_t same = __popc(__ballot_sync(0xFFFFFFFFu, (uint32_t)(__ldg(a.pairs + at) >> 32) == id));
                    const uint32_t from = lo, width = hi - lo;
                    if (same > 0) lo = from + (uint32_t)((uint64_t)width * same / 33);
                    if (same < 32) hi = max(lo + 1, from + (uint32_t)((uint64_t)width * (same + 1) / 33));
                }
                parts = lo / a.piece - q + 1;
            }
        }
        if (lane == 0) {
            parts_of[warp] = parts;
            id_of[warp] = id;
        }
        __syncthreads();
        for (uint32_t c0 = blockIdx.y * 32; c0 < a.dv; c0 += 32 * gridDim.y) {
            const uint32_t c = c0 + lane;
            const auto add = [&](uint32_t from, uint32_t r0, uint32_t count, uint32_t by, float (&sum)[E]) {
#pragma unroll 4
                for (uint32_t r = r0; r < count; r += by) {
                    float x[E];
                    ld_e<Fp32, E>(a.parts + ((size_t)(from + r) * 2 + (r == 0)) * a.d + (size_t)c * E, x);
#pragma unroll
                    for (int k = 0; k < E; ++k) sum[k] = __fadd_rn(sum[k], x[k]);
                }
            };
            if (parts > 0 && parts <= W && c < a.dv) {
                float sum[E] = {};
                add(q, 0, parts, 1, sum);
                embed_row<F, O, E>(a, id, c, sum);
            }
            for (uint32_t o = 0; o < W; ++o) {
                if (parts_of[o] <= W) continue;
                float sum[E] = {};
                if (c < a.dv) add(q0 + o, warp, parts_of[o], W, sum);
#pragma unroll
                for (int k = 0; k < E; ++k) sh[warp][lane * E + k] = sum[k];
                __syncthreads();
                if (warp == 0 && c < a.dv) {
                    for (uint32_t w = 1; w < W; ++w)
#pragma unroll
                        for (int k = 0; k < E; ++k) sum[k] = __fadd_rn(sum[k], sh[w][lane * E + k]);
                    embed_row<F, O, E>(a, id_of[o], c, sum);
                }
                __syncthreads();
            }
        }
        __syncthreads();   // parts_of has been read
    }
}

// ----------------------------------------------------------------------------
// Layer norm
// ----------------------------------------------------------------------------
// Sum over the threads that share a row: a warp, or the CTA.
template <bool WARP>
__device__ __forceinline__ float row_sum(float x, float* sh) {
    x = warp_sum(x);
    if constexpr (!WARP) {
        const int warps = blockDim.x / 32;
        if ((threadIdx.x & 31) == 0) sh[threadIdx.x / 32] = x;
        __syncthreads();
        x = warp_sum((int)(threadIdx.x & 31) < warps ? sh[threadIdx.x & 31] : 0.0f);
        __syncthreads();
    }
    return x;
}

struct NormArgs {
    const void* x;
    const void* weight;
    const void* bias;
    void* y;
    float* mean;
    float* rstd;
    int64_t rows, x_stride;
    uint32_t d, dv;
    float eps;
};

// A row stays in the registers of a warp or of a CTA, NV pieces a thread.  AHEAD:
// the CTA's next row is under way during the second half of its work (9000 x 4096
// bf16: 40 us without, 31 with; single elements are no faster with it).
template <class F, int E, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? kThreads : E > 1 ? 512 : 1024) norm_kernel(const __grid_constant__ NormArgs a) {
    using S = typename Store<F>::S;
    __shared__ float sh[32];
    const uint32_t group = WARP ? 32 : blockDim.x;
    const uint32_t lane = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int64_t first = WARP ? ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 32 : blockIdx.x;
    const int64_t step = WARP ? (int64_t)gridDim.x * blockDim.x / 32 : gridDim.x;
    const float d = (float)a.d;
    constexpr bool AHEAD = !WARP && E > 1;
    const auto at = [&](int64_t row) { return static_cast<const S*>(a.x) + row * a.x_stride + (size_t)lane * E; };
    [[maybe_unused]] Raw<F, E> raw[AHEAD ? NV : 1] = {};
    const auto load = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * group < a.dv) raw[k].load(at(row) + (size_t)k * group * E);
    };
    if constexpr (AHEAD)
        if (first < a.rows) load(first);
    for (int64_t row = first; row < a.rows; row += step) {
        float x[NV][E];
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if constexpr (AHEAD) {
                raw[k].hold();
                raw[k].get(x[k]);
            } else {
                if (lane + k * group < a.dv) ld_e<F, E>(at(row) + (size_t)k * group * E, x[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * group < a.dv)
#pragma unroll
                for (int e = 0; e < E; ++e) sum = __fadd_rn(sum, x[k][e]);
        const float mean = __fdiv_rn(row_sum<WARP>(sum, sh), d);
        sum = 0.0f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * group < a.dv)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    x[k][e] = __fsub_rn(x[k][e], mean);
                    sum = __fmaf_rn(x[k][e], x[k][e], sum);
                }
        if constexpr (AHEAD)
            if (row + step < a.rows) load(row + step);
        const float var = __fdiv_rn(row_sum<WARP>(sum, sh), d);
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, a.eps)));
        if (lane == 0 && a.mean) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        S* dst = static_cast<S*>(a.y) + row * (int64_t)a.d;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t c = lane + k * group;
            if (c < a.dv) {
                float w[E], b[E] = {};
                ld_e<F, E>(static_cast<const S*>(a.weight) + (size_t)c * E, w);
                if (a.bias) ld_e<F, E>(static_cast<const S*>(a.bias) + (size_t)c * E, b);
#pragma unroll
                for (int e = 0; e < E; ++e) x[k][e] = __fmaf_rn(__fmul_rn(x[k][e], rstd), w[e], b[e]);
                st_e<F, E>(dst + (size_t)c * E, x[k]);
            }
        }
    }
}

// The same with 16-byte pieces, a warp a row: the row stays in registers as it
// lies in memory, so that 32 warps of an SM have one under way.  32768 x 1600
// bf16: 37 us, 5.7 TB/s (of 6.7), two thirds of the issue slots in
// use; 18 warps with rows widened to binary32 took 50 us, 24 that
// load a row ahead 41.
template <class F, int NV>
__global__ void __launch_bounds__(kThreads, sizeof(typename Store<F>::S) == 2 ? 4 : 2) norm_warp_kernel(const __grid_constant__ NormArgs a) {
    using S = typename Store<F>::S;
    constexpr int E = 16 / (int)sizeof(S);
    const uint32_t lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    const float d = (float)a.d;
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; row < a.rows; row += step) {
        const S* src = static_cast<const S*>(a.x) + row * a.x_stride;
        Raw<F, E> raw[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * 32 < a.dv) raw[k].load(src + (size_t)(lane + k * 32) * E);
        F2 sum = f2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * 32 < a.dv) {
                float x[E];
                raw[k].get(x);
#pragma unroll
                for (int e = 0; e < E; e += 2) sum = add2(sum, f2(x[e], x[e + 1]));
            }
        float lo, hi;
        split(sum, lo, hi);
        const float mean = __fdiv_rn(warp_sum(__fadd_rn(lo, hi)), d);
        const F2 minus = f2(-mean, -mean);
        sum = f2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < NV; ++k)
            if (lane + k * 32 < a.dv) {
                float x[E];
                raw[k].get(x);
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const F2 t = add2(f2(x[e], x[e + 1]), minus);
                    sum = fma2(t, t, sum);
                }
            }
        split(sum, lo, hi);
        const float var = __fdiv_rn(warp_sum(__fadd_rn(lo, hi)), d);
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(var, a.eps)));
        if (lane == 0 && a.mean) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
        const F2 by = f2(rstd, rstd);
        S* dst = static_cast<S*>(a.y) + row * (int64_t)a.d;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const uint32_t c = lane + k * 32;
            if (c < a.dv) {
                float x[E], w[E], b[E] = {};
                raw[k].get(x);
                ld_e<F, E>(static_cast<const S*>(a.weight) + (size_t)c * E, w);
                if (a.bias) ld_e<F, E>(static_cast<const S*>(a.bias) + (size_t)c * E, b);
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    split(fma2(mul2(add2(f2(x[e], x[e + 1]), minus), by), f2(w[e], w[e + 1]), f2(b[e], b[e + 1])), x[e], x[e + 1]);
                st_e<F, E>(dst + (size_t)c * E, x);
            }
        }
    }
}

constexpr int64_t kNormBlocks = 152;   // blocks of rows, at most: a CTA on each SM

struct NormGradArgs {
    const void* gy;
    const void* x;
    const void* weight;
    const float* mean;
    const float* rstd;
    void* gx;
    void* gw;
    void* gb;
    float* parts;  // [blocks][2][d]: sums of gy * u, of gy
    int64_t rows, gy_stride, x_stride, per_block;
    uint32_t d, dv;
    int32_t blocks, accumulate;
};

template <int G>
__device__ __forceinline__ void team_barrier(int team) {
    if constexpr (G == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(G * 32) : "memory");
}

// A CTA takes a block of rows, a team of G warps a row.  A thread keeps NV
// pieces of columns, and for all its rows their sums for the weight and bias,
// in registers; between the two passes over a row also x - mean and gy * weight
// (KEEP: up to 32 columns), while the next row's loads are under way.  What the
// time goes to are instructions (half of the issue slots; 55% of the memory's
// rate at 32768 x 1600 bf16, 65 us): widening, and 9 operations an element, two
// elements at a time.  16 columns and 16 warps: 32 columns and 8 warps issue a
// fifth less and take 71 us; the weight in registers as well leaves 12 warps and
// 77 us; rows through a ring of bulk copies in shared memory took 65 us where this
// form took 67.  A piece's next load comes after the last use of its registers:
// before it, binary32 values, which are used as they were loaded, would be copied at
// the end of the loop, which waits for them (32768 x 1600 fp32: 193 us instead of
// 111, at an odd place 480 instead of 132).
template <class F, int E, int NV, int G, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) norm_grad_kernel(const __grid_constant__ NormGradArgs a) {
    using S = typename Store<F>::S;
    constexpr int T = THREADS / 32 / G, C = NV * E;
    constexpr int P = E == 1 ? 2 : 1;   // single elements: two pieces make a pair
    constexpr bool KEEP = C <= 32;
    static_assert(T * G * 32 == THREADS && C % 2 == 0 && NV % P == 0, "whole teams, pairs of columns");
    extern __shared__ __align__(16) float sums[];   // [team][2][d]
    __shared__ float sh[2][T][G][2];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, team = warp / G, part = warp % G;
    const uint32_t tid = part * 32 + lane;          // in the team
    grid_release();
    const float inv_d = __fdiv_rn(1.0f, (float)a.d);
    // does the warp, does this lane have a piece k
    const auto any = [&](int k) { return part * 32 + k * 32 * G < a.dv; };
    const auto mine = [&](int k) { return tid + k * 32 * G < a.dv; };
    int flip = 0;
    for (int block = blockIdx.x; block < a.blocks; block += gridDim.x) {
        const int64_t r0 = block * a.per_block + team, r1 = min(a.rows, (block + 1) * a.per_block);
        F2 sw[C / 2], sb[C / 2];
#pragma unroll
        for (int j = 0; j < C / 2; ++j) sw[j] = sb[j] = f2(0.0f, 0.0f);
        const S* x_at = static_cast<const S*>(a.x) + (size_t)tid * E;
        const S* g_at = static_cast<const S*>(a.gy) + (size_t)tid * E;
        Raw<F, E> rx[KEEP ? NV : P] = {}, rg[KEEP ? NV : P] = {};
        float next_mean = 0.0f, next_rstd = 0.0f;
        const auto load = [&](int k, int at, int64_t row) {
            rx[at].load(x_at + row * a.x_stride + k * 32 * G * E);
            rg[at].load(g_at + row * a.gy_stride + k * 32 * G * E);
        };
        if (r0 < r1) {
            next_mean = __ldg(a.mean + r0);
            next_rstd = __ldg(a.rstd + r0);
            if constexpr (KEEP)
#pragma unroll
                for (int k = 0; k < NV; ++k)
                    if (mine(k)) load(k, k, r0);
        }
        for (int64_t row = r0; row < r1; row += T, flip ^= 1) {
            const float mean = next_mean, rstd = next_rstd;
            const bool more = row + T < r1;
            if (more) {
                next_mean = __ldg(a.mean + row + T);
                next_rstd = __ldg(a.rstd + row + T);
            }
            const F2 minus = f2(-mean, -mean), by = f2(rstd, rstd);
            F2 s1 = f2(0.0f, 0.0f), s2 = s1;
            // c = x - mean, h = gy * w: the sums of h, h c, gy c / std and gy
            [[maybe_unused]] F2 cs[KEEP ? C / 2 : 1], hs[KEEP ? C / 2 : 1];
#pragma unroll
            for (int k = 0; k < NV; k += P) {
                if (any(k)) {
                    float x[P][E], g[P][E], w[P][E] = {};   // zeros behind the row: they add nothing
#pragma unroll
                    for (int q = 0; q < P; ++q) {
                        const int at = KEEP ? k + q : q;
                        if constexpr (!KEEP) {
                            rx[at] = rg[at] = {};
                            if (mine(k + q)) load(k + q, at, row);
                        }
                        rx[at].hold();
                        rg[at].hold();
                        rx[at].get(x[q]);
                        rg[at].get(g[q]);
                        if (mine(k + q)) ld_e<F, E>(static_cast<const S*>(a.weight) + (size_t)(tid + (k + q) * 32 * G) * E, w[q]);
                    }
#pragma unroll
                    for (int e = 0; e < P * E; e += 2) {
                        const int j = (k * E + e) / 2, q = e / E, i = e % E, q1 = (e + 1) / E, i1 = (e + 1) % E;
                        const F2 c = add2(f2(x[q][i], x[q1][i1]), minus), gg = f2(g[q][i], g[q1][i1]);
                        sw[j] = fma2(mul2(gg, by), c, sw[j]);
                        sb[j] = add2(sb[j], gg);
                        const F2 h = mul2(gg, f2(w[q][i], w[q1][i1]));
                        s1 = add2(s1, h);
                        s2 = fma2(h, c, s2);
                        if constexpr (KEEP) {
                            cs[j] = c;
                            hs[j] = h;
                        }
                    }
                    if constexpr (KEEP) {   // the next row's, into registers that are free now
#pragma unroll
                        for (int q = 0; q < P; ++q)
                            if (more && mine(k + q)) load(k + q, k + q, row + T);
                    }
                }
            }
            float lo, hi, m1, m2;
            split(s1, lo, hi);
            m1 = __fadd_rn(lo, hi);
            split(s2, lo, hi);
            m2 = __fadd_rn(lo, hi);
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) {
                m1 = __fadd_rn(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, s));
                m2 = __fadd_rn(m2, __shfl_xor_sync(0xFFFFFFFFu, m2, s));
            }
            if constexpr (G > 1) {
                if (lane == 0) {
                    sh[flip][team][part][0] = m1;
                    sh[flip][team][part][1] = m2;
                }
                team_barrier<G>(team);   // the other half of sh is written next
                m1 = sh[flip][team][0][0];
                m2 = sh[flip][team][0][1];
#pragma unroll
                for (int p = 1; p < G; ++p) {
                    m1 = __fadd_rn(m1, sh[flip][team][p][0]);
                    m2 = __fadd_rn(m2, sh[flip][team][p][1]);
                }
            }
            // grad_x = h / std - c mean(h c) / std^3 - mean(h) / std
            const float l = -__fmul_rn(rstd, __fmul_rn(m1, inv_d));
            const float k3 = -__fmul_rn(__fmul_rn(rstd, rstd), __fmul_rn(rstd, __fmul_rn(m2, inv_d)));
            const F2 less = f2(l, l), along = f2(k3, k3);
            S* dst = static_cast<S*>(a.gx) + row * (int64_t)a.d + (size_t)tid * E;
#pragma unroll
            for (int k = 0; k < NV; k += P) {
                if (mine(k)) {
                    float o[P][E];
                    if constexpr (!KEEP) {
#pragma unroll
                        for (int q = 0; q < P; ++q) {
                            if (mine(k + q)) {
                                load(k + q, 0, row);
                                float x[E], g[E], w[E];
                                rx[0].get(x);
                                rg[0].get(g);
                                ld_e<F, E>(static_cast<const S*>(a.weight) + (size_t)(tid + (k + q) * 32 * G) * E, w);
#pragma unroll
                                for (int e = 0; e < E; ++e)
                                    o[q][e] = __fmaf_rn(__fsub_rn(x[e], mean), k3, __fmaf_rn(__fmul_rn(g[e], w[e]), rstd, l));
                            }
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < P * E; e += 2) {
                            const int j = (k * E + e) / 2;
                            split(fma2(cs[j], along, fma2(hs[j], by, less)), o[e / E][e % E], o[(e + 1) / E][(e + 1) % E]);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < P; ++q)
                        if (mine(k + q)) st_e<F, E>(dst + (k + q) * 32 * G * E, o[q]);
                }
            }
        }
        // the teams' sums, in order
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            if (mine(k)) {
                float* p = sums + (size_t)team * 2 * a.d + (size_t)(tid + k * 32 * G) * E;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float lo, hi;
                    split(sw[(k * E + e) / 2], lo, hi);
                    p[e] = (k * E + e) & 1 ? hi : lo;
                    split(sb[(k * E + e) / 2], lo, hi);
                    p[a.d + e] = (k * E + e) & 1 ? hi : lo;
                }
            }
        }
        __syncthreads();
        for (uint32_t c = threadIdx.x; c < 2 * a.d; c += THREADS) {
            float sum = sums[c];
#pragma unroll
            for (int t = 1; t < T; ++t) sum = __fadd_rn(sum, sums[(size_t)t * 2 * a.d + c]);
            a.parts[(size_t)block * 2 * a.d + c] = sum;
        }
        __syncthreads();
    }
}

// The blocks' sums: 32 columns a CTA, each warp every 32nd block, the warps in order.
template <class O>
__global__ void __launch_bounds__(1024) norm_join_kernel(const __grid_constant__ NormGradArgs a) {
    using S = typename Store<O>::S;
    __shared__ float sh[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const uint32_t per = (a.d + 31) / 32;
    grid_wait();
    for (uint32_t t = blockIdx.x; t < 2 * per; t += gridDim.x) {
        const bool bias = t >= per;
        const uint32_t c = (t - (bias ? per : 0)) * 32 + lane;
        float sum = 0.0f;
        if (c < a.d)
#pragma unroll 4
            for (int b = warp; b < a.blocks; b += 32) sum = __fadd_rn(sum, a.parts[((size_t)b * 2 + bias) * a.d + c]);
        sh[warp][lane] = sum;
        __syncthreads();
        S* p = static_cast<S*>(bias ? a.gb : a.gw);
        if (warp == 0 && c < a.d && p) {
            float o[1] = {0.0f};
            for (int w = 0; w < 32; ++w) o[0] = __fadd_rn(o[0], sh[w][lane]);
            if (a.accumulate) add_e<O, 1>(p + c, o);
            st_e<O, 1>(p + c, o);
        }
        __syncthreads();
    }
}

}  // namespace zk

using namespace zero_detail;

namespace {

int elem_size(int32_t dtype) { return dtype == ZERO_FP32 ? 4 : 2; }

bool known(int32_t dtype) { return dtype == ZERO_BF16 || dtype == ZERO_FP16 || dtype == ZERO_FP32; }

// A tensor's pointer: natural alignment.
zero_status_t check_elem_ptr(const void* p, int size, const std::string& what) {
    if (!p) return fail(ZERO_ERR_INVALID, what + ": NULL device pointer");
    if (reinterpret_cast<uintptr_t>(p) % size) return fail(ZERO_ERR_ALIGN, what + ": not aligned to its elements");
    return ZERO_OK;
}

// Elements of a piece: the widest that rows of d elements at these addresses
// and strides allow.
struct Piece {
    int64_t bits = 0;  // addresses and strides in bytes, or-ed, of what is read or written in pieces
    int64_t d;
    int size;
    explicit Piece(int64_t d_, int size_) : d(d_), size(size_) {}
    // an array of `its` bytes an element, with rows `stride` elements apart
    void add(const void* p, int its, int64_t stride) {
        // in units of `size`: an array of wider elements needs 16 bytes at most
        const int64_t a = (int64_t)reinterpret_cast<uintptr_t>(p) | (stride * its);
        bits |= its == size ? a : ((a & 15) == 0 ? 0 : (a & 7) == 0 ? 4 : size);
    }
    int elems() const {
        const int wide = 16 / size;
        if (d % wide == 0 && bits % 16 == 0) return wide;
        if (size == 2 && d % 2 == 0 && bits % 4 == 0) return 2;
        return 1;
    }
};

#define ZL_E16(F, e, ...)                                                  \
    do {                                                                   \
        if ((e) == 8) { constexpr int E = 8; using T = F; __VA_ARGS__; }   \
        else if ((e) == 2) { constexpr int E = 2; using T = F; __VA_ARGS__; } \
        else { constexpr int E = 1; using T = F; __VA_ARGS__; }            \
    } while (0)
// T: the type, E: elements of a piece
#define ZL_DISPATCH(dtype, e, ...)                                         \
    do {                                                                   \
        if ((dtype) == ZERO_BF16) ZL_E16(zk::Bf16, e, __VA_ARGS__);        \
        else if ((dtype) == ZERO_FP16) ZL_E16(zk::Fp16, e, __VA_ARGS__);   \
        else if ((e) == 4) { constexpr int E = 4; using T = zk::Fp32; __VA_ARGS__; } \
        else { constexpr int E = 1; using T = zk::Fp32; __VA_ARGS__; }     \
    } while (0)

int capped(int64_t ctas) {
    const int32_t cap = max_ctas();
    if (cap > 0 && ctas > cap) ctas = cap;
    return (int)std::max<int64_t>(1, std::min<int64_t>(ctas, 0x7FFFFFFF));
}

constexpr int64_t kMaxVocab = 0x7FFFFFFE, kMaxRows = 0x7FFFFFFF, kMaxDim = 1 << 20;

zero_status_t check_embedding(const char* what, int64_t vocab, int64_t d, int64_t n) {
    if (vocab < 1 || vocab > kMaxVocab) return fail(ZERO_ERR_INVALID, std::string(what) + ": vocab must be 1 .. 2^31-2");
    if (d < 1 || d > kMaxDim) return fail(ZERO_ERR_INVALID, std::string(what) + ": d must be 1 .. 2^20");
    if (n < 0 || n > kMaxRows) return fail(ZERO_ERR_INVALID, std::string(what) + ": n must be 0 .. 2^31-1");
    return ZERO_OK;
}

// Tokens of a piece of the sorted list: few tokens in small pieces, to fill the
// GPU; many in long ones, whose frequent ids leave fewer parts; between, of 16,
// 24 and 32 what fills the last round of 152 SMs with 32 warps best (32768
// tokens of 1600: pieces of 24, 26 us, and of 32, 32 us).
int64_t embed_piece(int64_t d, int64_t n) {
    if (n <= 8192) return 8;
    if (n > (1 << 20)) return 256;
    const int64_t slices = (d + 255) / 256;
    int64_t best = 32, least = INT64_MAX;
    for (int64_t p = 32; p >= 16; p -= 8) {
        const int64_t cost = ((n + p - 1) / p * slices + 152 * 32 - 1) / (152 * 32) * p;
        if (cost < least) {
            least = cost;
            best = p;
        }
    }
    return best;
}

struct EmbedWorkspace {
    int64_t pairs0, pairs1, parts, bytes;
    explicit EmbedWorkspace(int64_t d, int64_t n) {
        const auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
        const int64_t pieces = (n + embed_piece(d, n) - 1) / embed_piece(d, n);
        pairs0 = 0;
        pairs1 = up((n + zk::kPairsPad) * 8);
        parts = 2 * pairs1;
        bytes = parts + up(pieces * 2 * d * 4) + 256;
    }
};

}  // namespace

extern "C" zero_status_t zero_embedding_forward(const void* weight, const int64_t* ids, int64_t vocab, int64_t d, int64_t n,
                                                int32_t dtype, double scale, void* out, zero_stream_t stream) {
    clear_error();
    const char* what = "zero_embedding_forward";
    zero_status_t rc = check_embedding(what, vocab, d, n);
    if (rc != ZERO_OK) return rc;
    if (!known(dtype)) return fail(ZERO_ERR_INVALID, "zero_embedding_forward: unknown dtype");
    if (!std::isfinite((float)scale)) return fail(ZERO_ERR_INVALID, "zero_embedding_forward: scale must be finite in binary32");
    if (n == 0) return ZERO_OK;
    const int size = elem_size(dtype);
    if ((rc = check_elem_ptr(weight, size, "zero_embedding_forward weight")) != ZERO_OK) return rc;
    if ((rc = check_elem_ptr(ids, 8, "zero_embedding_forward ids")) != ZERO_OK) return rc;
    if ((rc = check_elem_ptr(out, size, "zero_embedding_forward out")) != ZERO_OK) return rc;
    Piece piece(d, size);
    piece.add(weight, size, 0);
    piece.add(out, size, 0);
    const int e = piece.elems();
    zk::EmbedArgs a{weight, ids, out, vocab, n, (uint32_t)d, (uint32_t)(d / e), 0, (float)scale};
    while (a.lanes_log2 < 5 && (1u << a.lanes_log2) < a.dv) ++a.lanes_log2;
    const int64_t ctas = ((n << a.lanes_log2) + zk::kThreads - 1) / zk::kThreads;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    ZL_DISPATCH(dtype, e, zk::embed_kernel<T, E><<<capped(ctas), zk::kThreads, 0, s>>>(a));
    return after_launch(what);
}

extern "C" zero_status_t zero_embedding_workspace(int64_t vocab, int64_t d, int64_t n, int64_t* bytes) {
    clear_error();
    const zero_status_t rc = check_embedding("zero_embedding_workspace", vocab, d, n);
    if (rc != ZERO_OK) return rc;
    if (!bytes) return fail(ZERO_ERR_INVALID, "zero_embedding_workspace: NULL bytes");
    *bytes = EmbedWorkspace(d, n).bytes;
    return ZERO_OK;
}

namespace {

template <class F, class O, int E>
zero_status_t launch_embed_grad(const zk::EmbedGradArgs& a, cudaStream_t s) {
    const char* what = "zero_embedding_backward";
    // narrow rows: 8 lanes a piece
    const auto go = [&](auto k, int64_t lanes) {
        const int64_t items = a.pieces * (((int64_t)a.dv + lanes - 1) / lanes);
        return launch_after(k, dim3((unsigned)persistent_grid(k, (items * lanes + zk::kThreads - 1) / zk::kThreads)), zk::kThreads, 0, s, what, a);
    };
    const zero_status_t rc = a.dv > 16 ? go(zk::embed_grad_kernel<F, O, E, 32>, 32) : go(zk::embed_grad_kernel<F, O, E, 8>, 8);
    if (rc != ZERO_OK || a.pieces < 2) return rc;
    // few CTAs find something to add: pieces x column slices
    const dim3 grid((unsigned)capped(std::min<int64_t>((a.pieces + 6) / 8, 65535)),
                    (unsigned)(max_ctas() > 0 ? 1 : std::min<int64_t>((a.dv + 31) / 32, 64)));
    return launch_after(zk::embed_join_kernel<F, O, E>, grid, zk::kThreads, 0, s, what, a);
}

}  // namespace

namespace {

// Clusters of the sort that run at once: a CTA of 1024 threads fills an SM's registers, whatever shared memory it asks for.
int64_t resident_clusters(void (*kern)(zk::SortArgs), cudaLaunchConfig_t cfg, int cluster, bool shared) {
    static std::atomic<int> known[64][9][2];   // by device, size and form; zero-initialised (static storage)
    int dev = 0, n = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    std::atomic<int>& at = known[dev][cluster][shared];
    n = at.load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 2) {
            cudaGetLastError();
            n = 2;
        }
        at.store(n, std::memory_order_relaxed);
    }
    return n;
}

}  // namespace

extern "C" zero_status_t zero_embedding_backward(const void* grad_out, const int64_t* ids, int64_t vocab, int64_t d,
                                                 int64_t n, int32_t dtype, int32_t grad_dtype, double scale,
                                                 int32_t accumulate, void* grad_weight, void* workspace,
                                                 zero_stream_t stream) {
    clear_error();
    const char* what = "zero_embedding_backward";
    zero_status_t rc = check_embedding(what, vocab, d, n);
    if (rc != ZERO_OK) return rc;
    if (!known(dtype)) return fail(ZERO_ERR_INVALID, "zero_embedding_backward: unknown dtype");
    if (grad_dtype != dtype && grad_dtype != ZERO_FP32)
        return fail(ZERO_ERR_INVALID, "zero_embedding_backward: grad_dtype must be dtype or ZERO_FP32");
    if (!std::isfinite((float)scale)) return fail(ZERO_ERR_INVALID, "zero_embedding_backward: scale must be finite in binary32");
    const int size = elem_size(dtype), gsize = elem_size(grad_dtype);
    if ((rc = check_elem_ptr(grad_weight, gsize, "zero_embedding_backward grad_weight")) != ZERO_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (n == 0) {
        if (accumulate) return ZERO_OK;
        const cudaError_t err = cudaMemsetAsync(grad_weight, 0, (size_t)vocab * d * gsize, s);
        return err == cudaSuccess ? ZERO_OK : fail(ZERO_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(err));
    }
    if ((rc = check_elem_ptr(grad_out, size, "zero_embedding_backward grad_out")) != ZERO_OK) return rc;
    if ((rc = check_elem_ptr(ids, 8, "zero_embedding_backward ids")) != ZERO_OK) return rc;
    if ((rc = check_dev_ptr(workspace, "zero_embedding_backward workspace")) != ZERO_OK) return rc;
    const EmbedWorkspace ws(d, n);
    uint8_t* base = static_cast<uint8_t*>(workspace);

    zk::SortArgs sa{};
    sa.ids = ids;
    sa.pairs[0] = reinterpret_cast<uint64_t*>(base + ws.pairs0);
    sa.pairs[1] = reinterpret_cast<uint64_t*>(base + ws.pairs1);
    sa.zero = static_cast<uint8_t*>(grad_weight);
    sa.zero_bytes = accumulate ? 0 : vocab * d * gsize;
    sa.vocab = vocab;
    sa.n = (uint32_t)n;
    sa.passes = 1;
    while (sa.passes < 4 && (vocab >> (8 * sa.passes)) > 0) ++sa.passes;
    const int32_t cap = max_ctas();
    // the cluster that sorts: 8 CTAs, one for what one can sort as fast; under a cap with room for one that zeroes beside it
    const int clusters = sa.zero_bytes > 0 ? 2 : 1;
    int cluster = n <= 2048 ? 1 : 8;
    while (cap > 0 && cluster > 1 && clusters * cluster > cap) cluster /= 2;
    const int64_t warps = (int64_t)cluster * zk::kSortWarps;
    sa.per_warp = (uint32_t)((n + warps * 32 - 1) / (warps * 32) * 32);
    constexpr int64_t kMost = 192 << 10;   // of shared memory for the pairs: 98304 tokens in 8 CTAs
    const int64_t held = 2 * zk::kSortWarps * (int64_t)sa.per_warp * 8;
    const bool shared = held <= kMost;
    const auto kern = shared ? zk::embed_sort_kernel<true> : zk::embed_sort_kernel<false>;
    if (shared && held > (8 << 10)) {
        static std::atomic<uint64_t> allowed{0};   // by device
        int dev = 0;
        cudaGetDevice(&dev);
        const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
        if (!(allowed.load(std::memory_order_relaxed) & bit) || !bit) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost) != cudaSuccess) return after_launch(what);
            allowed.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(zk::kSortThreads);
    cfg.dynamicSmemBytes = shared ? (size_t)held : 0;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    // the clusters that zero: as many as run at once with the one that sorts (clusters of 8 do not fill every GPC: of 19, two
    // began when others had ended, and the launch took twice as long)
    cfg.gridDim = dim3((unsigned)cluster);
    if (sa.zero_bytes > 0) {
        int64_t fill = std::min<int64_t>((sa.zero_bytes / 32768 + cluster) / cluster, resident_clusters(kern, cfg, cluster, shared) - 1);
        if (cap > 0) fill = std::min<int64_t>(fill, cap / cluster - 1);
        cfg.gridDim = dim3((unsigned)(cluster * (1 + std::max<int64_t>(1, fill))));
    }
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, sa);
    if (err != cudaSuccess) {
        cudaGetLastError();
        return fail(ZERO_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(err));
    }
    if ((rc = after_launch(what)) != ZERO_OK) return rc;

    Piece piece(d, size);
    piece.add(grad_out, size, 0);
    piece.add(grad_weight, gsize, 0);
    const int e = piece.elems();
    zk::EmbedGradArgs a{};
    a.grad = grad_out;
    a.pairs = sa.pairs[sa.passes & 1];
    a.out = grad_weight;
    a.parts = reinterpret_cast<float*>(base + ws.parts);
    a.n = (uint32_t)n;
    a.piece = (int32_t)embed_piece(d, n);
    a.pieces = (uint32_t)((n + a.piece - 1) / a.piece);
    a.d = (uint32_t)d;
    a.dv = (uint32_t)(d / e);
    a.vocab = (uint32_t)vocab;
    a.accumulate = accumulate != 0;
    a.scale = (float)scale;
    if (grad_dtype == dtype) ZL_DISPATCH(dtype, e, rc = launch_embed_grad<T, T, E>(a, s));
    else ZL_DISPATCH(dtype, e, rc = launch_embed_grad<T, zk::Fp32, E>(a, s));
    return rc;
}

// ----------------------------------------------------------------------------
// Layer norm
// ----------------------------------------------------------------------------
namespace {

zero_status_t check_norm(const char* what, int64_t rows, int64_t d) {
    if (rows < 0 || rows > kMaxRows) return fail(ZERO_ERR_INVALID, std::string(what) + ": rows must be 0 .. 2^31-1");
    if (d < 1 || d > ZERO_MAX_NORM_DIM) return fail(ZERO_ERR_INVALID, std::string(what) + ": d must be 1 .. ZERO_MAX_NORM_DIM");
    return ZERO_OK;
}

template <class F, int E>
void launch_norm(const zk::NormArgs& a, cudaStream_t s) {
    // a warp keeps up to 64 elements a lane, a CTA's thread 16, or 32 above 8192 columns
    const auto warps = [&](auto kern) { kern<<<persistent_grid(kern, (a.rows + 7) / 8), zk::kThreads, 0, s>>>(a); };
    if constexpr (E >= 4) {
        constexpr int B = 8 / E;   // twice as many pieces of half the elements
        switch ((a.dv + 32 * B - 1) / (32 * B)) {
            case 1: return warps(zk::norm_warp_kernel<F, 1 * B>);
            case 2: return warps(zk::norm_warp_kernel<F, 2 * B>);
            case 3: return warps(zk::norm_warp_kernel<F, 3 * B>);
            case 4: return warps(zk::norm_warp_kernel<F, 4 * B>);
            case 5: return warps(zk::norm_warp_kernel<F, 5 * B>);
            case 6: return warps(zk::norm_warp_kernel<F, 6 * B>);
            case 7: return warps(zk::norm_warp_kernel<F, 7 * B>);
            case 8: return warps(zk::norm_warp_kernel<F, 8 * B>);
            default: break;
        }
    } else {
        constexpr int WIDE = E == 1 ? 32 : 16;
        if (a.dv <= 32u * WIDE) return warps(zk::norm_kernel<F, E, WIDE, true>);
    }
    const auto ctas = [&](auto kern, uint32_t nv) {
        const int threads = (int)((a.dv + nv - 1) / nv + 31) / 32 * 32;
        kern<<<persistent_grid(kern, a.rows, 0, threads), threads, 0, s>>>(a);
    };
    if (E == 1 || a.dv * E <= 512 * 16) return ctas(zk::norm_kernel<F, E, 16 / E, false>, 16 / E);
    if constexpr (E > 1) ctas(zk::norm_kernel<F, E, 32 / E, false>, 32 / E);
}

int64_t norm_rows_per_block(int64_t rows) { return std::max<int64_t>(1, (rows + zk::kNormBlocks - 1) / zk::kNormBlocks); }

template <class F, int E, int NV, int G, int THREADS>
zero_status_t launch_norm_team(const zk::NormGradArgs& a, cudaStream_t s, const char* what) {
    const int smem = THREADS / 32 / G * 2 * (int)a.d * 4;   // 128 KB at most
    auto kern = zk::norm_grad_kernel<F, E, NV, G, THREADS>;
    static std::atomic<uint64_t> allowed{0};   // by device
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (!(allowed.load(std::memory_order_relaxed) & bit) || !bit) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 131072) != cudaSuccess) return after_launch(what);
        allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    kern<<<capped(std::min<int64_t>(a.blocks, std::max(1, sm_count()))), THREADS, smem, s>>>(a);
    return after_launch(what);
}

// 16 columns a thread, 8 of single elements (each takes two registers while it
// is loaded, and 16 left none for the loads of the next row: 32768 x 1600 bf16 at
// an odd place 144 us, now 108), and as many warps a row as that takes; more
// columns a thread above 16 warps.
template <class F, int E>
zero_status_t launch_norm_grad(const zk::NormGradArgs& a, cudaStream_t s, const char* what) {
    constexpr int C = E == 1 ? 8 : 16, B = C / E;
    if (a.dv <= 16u * B) return launch_norm_team<F, E, B / 2, 1, 512>(a, s, what);
    if (a.dv <= 32u * B) return launch_norm_team<F, E, B, 1, 512>(a, s, what);
    if (a.dv <= 64u * B) return launch_norm_team<F, E, B, 2, 512>(a, s, what);
    if (a.dv <= 128u * B) return launch_norm_team<F, E, B, 4, 512>(a, s, what);
    if (a.dv <= 256u * B) return launch_norm_team<F, E, B, 8, 512>(a, s, what);
    if constexpr (C == 8)
        if (a.dv <= 512u * B) return launch_norm_team<F, E, B, 16, 512>(a, s, what);
    if (a.dv * E <= 8192) return launch_norm_team<F, E, 32 / E, 8, 256>(a, s, what);
    return launch_norm_team<F, E, 64 / E, 8, 256>(a, s, what);
}

}  // namespace

extern "C" zero_status_t zero_layer_norm_forward(const void* x, int64_t x_stride, const void* weight, const void* bias,
                                                 int64_t rows, int64_t d, int32_t dtype, double eps, void* y, float* mean,
                                                 float* rstd, zero_stream_t stream) {
    clear_error();
    const char* what = "zero_layer_norm_forward";
    zero_status_t rc = check_norm(what, rows, d);
    if (rc != ZERO_OK) return rc;
    if (!known(dtype)) return fail(ZERO_ERR_INVALID, "zero_layer_norm_forward: unknown dtype");
    if (!(eps >= 0.0) || !std::isfinite(eps)) return fail(ZERO_ERR_INVALID, "zero_layer_norm_forward: eps must be >= 0");
    if (x_stride < d) return fail(ZERO_ERR_INVALID, "zero_layer_norm_forward: rows overlap (x_stride < d)");
    if ((mean == nullptr) != (rstd == nullptr)) return fail(ZERO_ERR_INVALID, "zero_layer_norm_forward: mean and rstd go together");
    if (rows == 0) return ZERO_OK;
    const int size = elem_size(dtype);
    if ((rc = check_elem_ptr(x, size, "zero_layer_norm_forward x")) != ZERO_OK) return rc;
    if ((rc = check_elem_ptr(weight, size, "zero_layer_norm_forward weight")) != ZERO_OK) return rc;
    if (bias && (rc = check_elem_ptr(bias, size, "zero_layer_norm_forward bias")) != ZERO_OK) return rc;
    if ((rc = check_elem_ptr(y, size, "zero_layer_norm_forward y")) != ZERO_OK) return rc;
    if (mean && ((rc = check_elem_ptr(mean, 4, "zero_layer_norm_forward mean")) != ZERO_OK ||
                 (rc = check_elem_ptr(rstd, 4, "zero_layer_norm_forward rstd")) != ZERO_OK)) return rc;
    Piece piece(d, size);
    piece.add(x, size, rows > 1 ? x_stride : 0);
    piece.add(weight, size, 0);
    piece.add(bias, size, 0);
    piece.add(y, size, 0);
    const int e = piece.elems();
    const zk::NormArgs a{x, weight, bias, y, mean, rstd, rows, x_stride, (uint32_t)d, (uint32_t)(d / e), (float)eps};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    ZL_DISPATCH(dtype, e, launch_norm<T, E>(a, s));
    return after_launch(what);
}

extern "C" zero_status_t zero_layer_norm_workspace(int64_t rows, int64_t d, int64_t* bytes) {
    clear_error();
    const zero_status_t rc = check_norm("zero_layer_norm_workspace", rows, d);
    if (rc != ZERO_OK) return rc;
    if (!bytes) return fail(ZERO_ERR_INVALID, "zero_layer_norm_workspace: NULL bytes");
    const int64_t per = norm_rows_per_block(rows);
    *bytes = ((rows + per - 1) / per * 2 * d * 4 + 255) / 256 * 256 + 256;
    return ZERO_OK;
}

extern "C" zero_status_t zero_layer_norm_backward(const void* grad_y, int64_t gy_stride, const void* x, int64_t x_stride,
                                                  const void* weight, const float* mean, const float* rstd, int64_t rows,
                                                  int64_t d, int32_t dtype, int32_t grad_dtype, int32_t accumulate,
                                                  void* grad_x, void* grad_weight, void* grad_bias, void* workspace,
                                                  zero_stream_t stream) {
    clear_error();
    const char* what = "zero_layer_norm_backward";
    zero_status_t rc = check_norm(what, rows, d);
    if (rc != ZERO_OK) return rc;
    if (!known(dtype)) return fail(ZERO_ERR_INVALID, "zero_layer_norm_backward: unknown dtype");
    if (grad_dtype != dtype && grad_dtype != ZERO_FP32)
        return fail(ZERO_ERR_INVALID, "zero_layer_norm_backward: grad_dtype must be dtype or ZERO_FP32");
    if (x_stride < d || gy_stride < d) return fail(ZERO_ERR_INVALID, "zero_layer_norm_backward: rows overlap (a stride < d)");
    const int size = elem_size(dtype), gsize = elem_size(grad_dtype);
    if ((rc = check_elem_ptr(grad_weight, gsize, "zero_layer_norm_backward grad_weight")) != ZERO_OK) return rc;
    if (grad_bias && (rc = check_elem_ptr(grad_bias, gsize, "zero_layer_norm_backward grad_bias")) != ZERO_OK) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (accumulate) return ZERO_OK;
        cudaError_t err = cudaMemsetAsync(grad_weight, 0, (size_t)d * gsize, s);
        if (err == cudaSuccess && grad_bias) err = cudaMemsetAsync(grad_bias, 0, (size_t)d * gsize, s);
        return err == cudaSuccess ? ZERO_OK : fail(ZERO_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(err));
    }
    if ((rc = check_elem_ptr(grad_y, size, "zero_layer_norm_backward grad_y")) != ZERO_OK) return rc;
    if ((rc = check_elem_ptr(x, size, "zero_layer_norm_backward x")) != ZERO_OK) return rc;
    if ((rc = check_elem_ptr(weight, size, "zero_layer_norm_backward weight")) != ZERO_OK) return rc;
    if ((rc = check_elem_ptr(mean, 4, "zero_layer_norm_backward mean")) != ZERO_OK) return rc;
    if ((rc = check_elem_ptr(rstd, 4, "zero_layer_norm_backward rstd")) != ZERO_OK) return rc;
    if ((rc = check_elem_ptr(grad_x, size, "zero_layer_norm_backward grad_x")) != ZERO_OK) return rc;
    if ((rc = check_dev_ptr(workspace, "zero_layer_norm_backward workspace")) != ZERO_OK) return rc;
    Piece piece(d, size);
    piece.add(x, size, rows > 1 ? x_stride : 0);
    piece.add(grad_y, size, rows > 1 ? gy_stride : 0);
    piece.add(weight, size, 0);
    piece.add(grad_x, size, 0);
    const int e = piece.elems();
    zk::NormGradArgs a{};
    a.gy = grad_y;
    a.x = x;
    a.weight = weight;
    a.mean = mean;
    a.rstd = rstd;
    a.gx = grad_x;
    a.gw = grad_weight;
    a.gb = grad_bias;
    a.parts = static_cast<float*>(workspace);
    a.rows = rows;
    a.gy_stride = gy_stride;
    a.x_stride = x_stride;
    a.per_block = norm_rows_per_block(rows);
    a.blocks = (int32_t)((rows + a.per_block - 1) / a.per_block);
    a.d = (uint32_t)d;
    a.dv = (uint32_t)(d / e);
    a.accumulate = accumulate != 0;
    ZL_DISPATCH(dtype, e, rc = (launch_norm_grad<T, E>(a, s, what)));
    if (rc != ZERO_OK) return rc;
    const dim3 join((unsigned)capped(2 * ((d + 31) / 32)));
    if (grad_dtype == ZERO_FP32) return launch_after(zk::norm_join_kernel<zk::Fp32>, join, 1024, 0, s, what, a);
    if (grad_dtype == ZERO_BF16) return launch_after(zk::norm_join_kernel<zk::Bf16>, join, 1024, 0, s, what, a);
    return launch_after(zk::norm_join_kernel<zk::Fp16>, join, 1024, 0, s, what, a);
}
