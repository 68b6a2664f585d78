// AdamW over a list of tensors, with 32-bit or 8-bit states; the global norm
// of such a list; the 8-bit states from and to 32-bit ones.
//
// One launch walks all tensors: the list is cut into chunks of kChunk elements
// that never straddle a tensor, and a table in device memory (written once, by
// zero_multi_bind) says for each chunk which tensor it belongs to and for each
// tensor where its arrays are.
#include <algorithm>
#include <cmath>
#include <new>
#include <type_traits>
#include <vector>

#include "zero_launch.h"

namespace zk {

constexpr int kChunk = 2048;             // elements of one work item, a tile of the updates
constexpr int kBlock8 = 32;              // elements under one scale of an 8-bit state
constexpr int kSlices = 1216;            // fixed split of a list for the norm (8 CTAs on each of 152 SMs)
constexpr int kRowsPerLaunch = 256;      // table rows passed through one launch's parameters

// MultiRow::vec: which arrays begin on a boundary for the widest access.  The
// first four after `shift` elements were put in front of the tensor (the
// gradients' distance for the norm is `gshift`, and always right); the others at
// the tensor's own first element: gradients, parameters and 16-bit copies of the
// 8-bit update and its states (kWhole8), m and v for the codec, the codes.
enum { kVecGrad = 1, kVecMaster = 2, kVecStates = 4, kVecOut = 8, kWhole8 = 16, kCodec = 32, kCodes = 64 };

// What the kernels know of one tensor: 12 words of 8 bytes, which a warp reads
// with 12 lanes.
struct MultiRow {
    const void* grad;
    float* master;
    uint8_t* m8;
    uint8_t* v8;
    uint8_t* ms;
    uint8_t* vs;
    uint16_t* out;
    int64_t numel;
    uint32_t first_chunk;
    uint32_t tensor;  // its own index
    uint8_t vec;
    uint8_t shift;    // elements by which the tiles of the 32-bit update begin before the tensor,
    uint8_t gshift;   // and those of the norm
    uint8_t pad0;
    int32_t group;
    float* m;
    float* v;
};
constexpr int kRowWords = sizeof(MultiRow) / 8;
static_assert(kRowWords == 12 && kRowWords <= 32, "a warp reads a row");

// The device workspace: counters, rows, chunk map, norm partials.  How many chunks
// a list has goes by where its tensors begin, so a bind writes the count there
// too: launches recorded into a graph find what the last bind gave.
struct MultiTable {
    uint32_t* counters;      // CTAs that are done: [0] norm, [1] others; [2] tiles dealt; [3] errors of the codec;
                             // [4] CTAs that have read the state
    const MultiRow* rows;
    const uint32_t* tensor;  // tensor of each chunk
    float2* partials;        // kSlices
    float* grad_scale;       // the loss scale that the gradients of the last norm carried
    const uint32_t* n_chunks;
    uint32_t most_chunks;    // wherever the tensors begin: places of the map
    uint32_t n_tensors;
    uint64_t slack;          // bounds-checked builds: test hook
};

struct MultiHp {
    double lr[ZERO_MAX_GROUPS], eps[ZERO_MAX_GROUPS], wd[ZERO_MAX_GROUPS];
    int32_t n;
};

struct MultiArgs {
    MultiTable t;
    MultiHp hp;
    zero_step_state* st;
    int32_t flags;
    uint32_t seed;
};

// ----------------------------------------------------------------------------
// Binding
// ----------------------------------------------------------------------------
// The kernels of a step are launched so that they may begin while the kernel before them in the stream ends (launch_early);
// what that kernel wrote is read after grid_wait() only.  The rows and the chunk map are read before it (multi_reset_kernel).
struct RowBatch {
    MultiRow rows[kRowsPerLaunch];
};

__global__ void multi_rows_kernel(const __grid_constant__ RowBatch b, MultiRow* rows, int n, uint32_t* count, uint32_t n_chunks) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) rows[i] = b.rows[i];
    if (i == 0) *count = n_chunks;
}

// The last kernel of a bind: whatever begins while it ends finds the rows, the
// count and the map whole, since it began after their kernels' end.
__global__ void multi_reset_kernel(uint32_t* counters, float* grad_scale) {
    if (threadIdx.x < 5) counters[threadIdx.x] = 0;
    if (threadIdx.x == 0 && grad_scale) *grad_scale = 0.0f;
}

// Tensor of every chunk: the last row whose first chunk is not behind it
// (tensors without elements have no chunk and are passed over).
__global__ void multi_map_kernel(const MultiRow* rows, uint32_t n_tensors, uint32_t* tensor, uint32_t n_chunks) {
    for (uint32_t c = blockIdx.x * blockDim.x + threadIdx.x; c < n_chunks; c += gridDim.x * blockDim.x) {
        uint32_t lo = 0, hi = n_tensors;  // rows[lo].first_chunk <= c < rows[hi].first_chunk
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) >> 1;
            if (rows[mid].first_chunk <= c) lo = mid;
            else hi = mid;
        }
        tensor[c] = lo;
    }
}

// 8 values that begin `over` places behind a 16-byte boundary of shared memory.
__device__ __forceinline__ void lds8_over(const float* p, int over, float (&o)[8]) {
    float q[12];
#pragma unroll
    for (int j = 0; j < 3; ++j) {
        const float4 f = reinterpret_cast<const float4*>(p)[j];
        q[4 * j] = f.x, q[4 * j + 1] = f.y, q[4 * j + 2] = f.z, q[4 * j + 3] = f.w;
    }
    if (over & 1)
#pragma unroll
        for (int j = 0; j < 11; ++j) q[j] = q[j + 1];
    if (over & 2)
#pragma unroll
        for (int j = 0; j < 9; ++j) q[j] = q[j + 2];
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = q[e];
}
__device__ __forceinline__ uint4 lds8_over(const uint16_t* p, int over) {
    uint32_t q[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint4 f = reinterpret_cast<const uint4*>(p)[j];
        q[4 * j] = f.x, q[4 * j + 1] = f.y, q[4 * j + 2] = f.z, q[4 * j + 3] = f.w;
    }
    if (over & 2)
#pragma unroll
        for (int j = 0; j < 7; ++j) q[j] = q[j + 1];
    if (over & 4)
#pragma unroll
        for (int j = 0; j < 6; ++j) q[j] = q[j + 2];
    if (over & 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = __funnelshift_r(q[j], q[j + 1], 16);
    return make_uint4(q[0], q[1], q[2], q[3]);
}

// ----------------------------------------------------------------------------
// Loads and stores of 8 consecutive elements of which [e0, e1) exist (`none` is
// read for the others); `vec`: the first is on a boundary for the wide access.
// ----------------------------------------------------------------------------
struct GradBf16 {
    using T = uint16_t;
    static __device__ __forceinline__ float one(uint16_t h) { return Bf16::dec1(h); }
    static __device__ __forceinline__ void eight(const uint16_t* p, float (&o)[8]) { unpack8<Bf16>(ld_stream(p), o); }
    using Raw = uint4;
    static __device__ __forceinline__ Raw raw(const uint16_t* p) {
        Raw r;
        asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
        return r;
    }
    static __device__ __forceinline__ void values(const Raw& r, float (&o)[8]) { unpack8<Bf16>(r, o); }
    static __device__ __forceinline__ void load8(const uint16_t* p, float (&o)[8]) {
        unpack8<Bf16>(*reinterpret_cast<const uint4*>(p), o);
    }
    static __device__ __forceinline__ void load8_over(const uint16_t* p, int over, float (&o)[8]) {
        unpack8<Bf16>(lds8_over(p, over), o);
    }
};
struct GradFp16 {
    using T = uint16_t;
    static __device__ __forceinline__ float one(uint16_t h) { return Fp16::dec1(h); }
    static __device__ __forceinline__ void eight(const uint16_t* p, float (&o)[8]) { unpack8<Fp16>(ld_stream(p), o); }
    using Raw = uint4;
    static __device__ __forceinline__ Raw raw(const uint16_t* p) {
        Raw r;
        asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
        return r;
    }
    static __device__ __forceinline__ void values(const Raw& r, float (&o)[8]) { unpack8<Fp16>(r, o); }
    static __device__ __forceinline__ void load8(const uint16_t* p, float (&o)[8]) {
        unpack8<Fp16>(*reinterpret_cast<const uint4*>(p), o);
    }
    static __device__ __forceinline__ void load8_over(const uint16_t* p, int over, float (&o)[8]) {
        unpack8<Fp16>(lds8_over(p, over), o);
    }
};
struct GradFp32 {
    using T = float;
    static __device__ __forceinline__ float one(float x) { return x; }
    static __device__ __forceinline__ void eight(const float* p, float (&o)[8]) { ld8(p, o); }
    struct Raw {
        float x[8];
    };
    static __device__ __forceinline__ Raw raw(const float* p) {
        Raw r;
        asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(r.x[0]), "=f"(r.x[1]), "=f"(r.x[2]), "=f"(r.x[3]), "=f"(r.x[4]), "=f"(r.x[5]), "=f"(r.x[6]), "=f"(r.x[7])
                     : "l"(p));
        return r;
    }
    static __device__ __forceinline__ void values(const Raw& r, float (&o)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = r.x[e];
    }
    static __device__ __forceinline__ void load8(const float* p, float (&o)[8]) {
        const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
        o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
        o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
    }
    static __device__ __forceinline__ void load8_over(const float* p, int over, float (&o)[8]) { lds8_over(p, over, o); }
};
struct NoOut {
    static constexpr bool kOut = false;
};
struct OutBf16 : Bf16 {
    static constexpr bool kOut = true;
};
struct OutFp16 : Fp16 {
    static constexpr bool kOut = true;
};

// Which of the 8 elements from i on a tensor has; false: none.
__device__ __forceinline__ bool span8(const MultiTable& t, const MultiRow& r, int64_t i, int& e0, int& e1) {
    if (i >= r.numel || i <= -kVec) return false;
    e0 = i < 0 ? (int)-i : 0;
    e1 = r.numel - i < kVec ? (int)(r.numel - i) : kVec;
    const uint64_t lim = (uint64_t)r.numel > t.slack ? (uint64_t)r.numel - t.slack : 0;
    return in_bounds((uint64_t)(i + e1), lim);
}
template <class G>
__device__ __forceinline__ void load_grad(const void* base, int64_t i, int e0, int e1, bool vec, float (&o)[8],
                                          float none = 0.0f) {
    const typename G::T* p = static_cast<const typename G::T*>(base) + i;
    if (vec && e0 <= 0 && e1 >= 8) {
        G::eight(p, o);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = e >= e0 && e < e1 ? G::one(p[e]) : none;
    }
}
__device__ __forceinline__ void load_f32(const float* p, int e0, int e1, bool vec, float (&o)[8], float none = 0.0f) {
    if (vec && e0 <= 0 && e1 >= 8) {
        ld8(p, o);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = e >= e0 && e < e1 ? p[e] : none;
    }
}
__device__ __forceinline__ void store_f32(float* p, int e0, int e1, bool vec, const float (&o)[8]) {
    if (vec && e0 <= 0 && e1 >= 8) {
        st8(p, o);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= e0 && e < e1) p[e] = o[e];
    }
}
template <class O>
__device__ __forceinline__ void store_out(uint16_t* p, int e0, int e1, bool vec, const float (&o)[8]) {
    if constexpr (O::kOut) {
        if (vec && e0 <= 0 && e1 >= 8) {
            st_stream(p, pack8<O>(o));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= e0 && e < e1) p[e] = O::enc1(o[e]);
        }
    }
}

// ----------------------------------------------------------------------------
// 8-bit states: E4M3 (m) and E5M2 (v) codes under one power of two per 32
// elements, which two neighbouring lanes hold, 16 elements each.
// ----------------------------------------------------------------------------
struct E4m3 {
    static constexpr int kTop = 8;      // largest exponent
    static constexpr int kCut = 20;     // binary32 mantissa bits a code does not keep
    static constexpr bool kFloor = false;
    static __device__ __forceinline__ float2 dec2(uint16_t h) {
        uint32_t r;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
        return __half22float2(*reinterpret_cast<const __half2*>(&r));
    }
    static __device__ __forceinline__ uint16_t enc2(float lo, float hi) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
        return r;
    }
};
struct E5m2 {
    static constexpr int kTop = 15;
    static constexpr int kCut = 21;
    static constexpr bool kFloor = true;  // above zero stays above zero: m / sqrt(v) must not meet a lost v
    static __device__ __forceinline__ float2 dec2(uint16_t h) {
        uint32_t r;
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(h));
        return __half22float2(*reinterpret_cast<const __half2*>(&r));
    }
    static __device__ __forceinline__ uint16_t enc2(float lo, float hi) {
        uint16_t r;
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
        return r;
    }
};
constexpr float kSmallestE5m2 = 1.52587890625e-05f;  // 2^-16

// 2^(byte - 127); 2^-127 is a subnormal.
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return __uint_as_float(byte ? byte << 23 : 1u << 22);
}

__device__ __forceinline__ uint32_t mix32(uint32_t x) {
    x ^= x >> 16;
    x *= 0x9E3779B1u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    x ^= x >> 16;
    return x;
}

// ----------------------------------------------------------------------------
// The step's constants of every group
// ----------------------------------------------------------------------------
struct __align__(16) Const8 {
    float b1, omb1, b2, omb2;
    float decay, step_size, eps, isb;  // isb: 1 / sqrt(1 - beta2^t)
};
struct MultiShared {
    AdamConsts k[ZERO_MAX_GROUPS];
    Const8 c8[ZERO_MAX_GROUPS];  // of the 8-bit update
    float unscale;               // 1 / loss scale the gradients carry
    float factor;                // 8-bit update: the last factor of the gradients, and
    int32_t two;                 // whether unscale is another one before it
    uint32_t key;                // of the step's random numbers
    int32_t apply;
};

// ZERO_MULTI_ADVANCE: moves the step on once every CTA has read the state
// (one thread of each calls it, after that).
__device__ __forceinline__ void advance_step(const MultiArgs& a) {
    if (!(a.flags & ZERO_MULTI_ADVANCE)) return;
    __threadfence();
    if (atomicInc(&a.t.counters[4], gridDim.x - 1) != gridDim.x - 1) return;
    zero_step_state* st = a.st;
    st->nonfinite = 0;  // nothing was looked for
    st->overflow = 0;
    st->clip_coef = 1.0f;
    st->apply = 1;
    st->t += 1;
    st->beta1_pow = __dmul_rn(st->beta1_pow, st->beta1);
    st->beta2_pow = __dmul_rn(st->beta2_pow, st->beta2);
    st->good_steps += 1;
}

// All threads of the CTA (at least four warps) call it; false: the step is
// skipped.  Binary64 divisions and square roots are slow here, and a short step
// waits for them: each of four warps has its part of every group.
__device__ __forceinline__ bool multi_constants(const MultiArgs& a, MultiShared& s) {
    const zero_step_state* st = a.st;
    const bool advance = (a.flags & ZERO_MULTI_ADVANCE) != 0;
    static_assert(ZERO_MAX_GROUPS < 32, "a lane for each group, and one for the rest");
    const int g = threadIdx.x & 31, role = threadIdx.x >> 5;
    if (g < a.hp.n && role < 4) {
        AdamConsts& k = s.k[g];
        Const8& q = s.c8[g];
        if (role == 0) {
            const double b1p = advance ? __dmul_rn(st->beta1_pow, st->beta1) : st->beta1_pow;
            k.step_size = q.step_size = __double2float_rn(__ddiv_rn(a.hp.lr[g], __dsub_rn(1.0, b1p)));
        } else if (role == 1) {
            const double b2p = advance ? __dmul_rn(st->beta2_pow, st->beta2) : st->beta2_pow;
            k.sqrt_bc2 = __double2float_rn(__dsqrt_rn(__dsub_rn(1.0, b2p)));
            q.isb = __fdiv_rn(1.0f, k.sqrt_bc2);
        } else if (role == 2) {
            k.b1 = q.b1 = __double2float_rn(st->beta1);
            k.b2 = q.b2 = __double2float_rn(st->beta2);
            k.omb1 = q.omb1 = __double2float_rn(__dsub_rn(1.0, st->beta1));
            k.omb2 = q.omb2 = __double2float_rn(__dsub_rn(1.0, st->beta2));
        } else {  // role 3
            k.decay = q.decay = __double2float_rn(__dsub_rn(1.0, __dmul_rn(a.hp.lr[g], a.hp.wd[g])));
            k.eps = __double2float_rn(a.hp.eps[g]);
            q.eps = fmaxf(k.eps, 1.17549435e-38f);
            k.clip = advance ? 1.0f : st->clip_coef;
        }
    }
    if (threadIdx.x == 2 * 32 + ZERO_MAX_GROUPS) {
        s.apply = advance ? 1 : st->apply;
        const float kept = *a.t.grad_scale;  // zero before the list's first norm
        const float scale = !advance && kept > 0.0f ? kept : st->loss_scale;
        s.unscale = (a.flags & ZERO_MULTI_UNSCALED) ? 1.0f : __fdiv_rn(1.0f, scale);
        const float clip = advance ? 1.0f : st->clip_coef;
        s.two = clip != 1.0f && s.unscale != 1.0f;  // a factor of 1 changes nothing
        s.factor = clip != 1.0f ? clip : s.unscale;
        s.key = mix32(a.seed ^ mix32((uint32_t)(st->t + (advance ? 1 : 0))));
    }
    __syncthreads();
    return s.apply != 0;
}

// ----------------------------------------------------------------------------
// A ring of tiles in shared memory
//
// W warps of a CTA compute and one fetches the inputs of the next tiles by bulk
// copies.  With the loads of a few tiles always under way the memory is busy
// whatever the number of warps, and how near the CTAs are to each other in
// memory decides its rate: with tiles dealt in turns CTAs drift apart.  GB300,
// 1.56e9 elements, us per launch (32-bit / 8-bit update), 16 computing warps on
// an SM: dealt by a counter 6137 / 3561 (7.1 / 7.05 TB/s), 8 warps 6752 / 3846,
// 24 warps 6159 / 3586; dealt in turns 7483 / 3974, 8 warps 6684 / 3664.  The
// plain form of the 32-bit update (8 elements a thread, 32-byte loads, 1024
// threads on an SM) 6605 to 6740.
// ----------------------------------------------------------------------------
template <int S>
struct Ring {
    uint64_t full[S], empty[S];
};

// Up to 4 bytes into shared memory (zeros behind them), counted by an mbarrier.
__device__ __forceinline__ void copy4_async(void* dst_smem, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst_smem)), "l"(src), "r"(min(bytes, 4)) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {  // arrives when the thread's copies so far have landed
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(smem_u32(bar)) : "memory");
}

template <int W, int S>
__device__ __forceinline__ void ring_init(Ring<S>& ring) {
    if (threadIdx.x == 0) {
        for (int k = 0; k < S; ++k) {
            mbar_init(&ring.full[k], 33);  // the fetching warp's lanes' copies, and the bulk copies' bytes
            mbar_init(&ring.empty[k], W);
        }
        fence_mbar_init();
    }
    __syncthreads();
}

// The fetching warp.  Its k-th tile goes into stage k % S: the row by way of
// the lanes, then issue(tile, stage, full) by all lanes, which copies what can
// be copied and arrives at `full` 33 times.  The first S tiles of a CTA are its own; the others are dealt one by one by a
// counter, so that all CTAs work next to each other in memory however long the
// list is (dealt in turns they drift apart, and the memory's rate with them);
// the CTA that ends last puts the counter back.  ready(), which all warps call
// once, says after the first copies whether the tiles are wanted.
template <int S, class Stage, class Issue, class Ready>
__device__ __forceinline__ void ring_fetch(const MultiTable& t, int32_t* error, Stage* stage, Ring<S>& ring, Issue issue,
                                           Ready ready) {
    const int lane = threadIdx.x & 31;
    const uint32_t own = S * gridDim.x;
    // the count and the first tiles' tensors arrive together
    const uint32_t n = *t.n_chunks;
    uint32_t tensor[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
        const uint32_t c = blockIdx.x + j * gridDim.x;
        tensor[j] = c < t.most_chunks ? t.tensor[c] : 0u;  // what an earlier bind has left, behind the count
    }
    auto tensor_of = [&](uint32_t c) { return c < n ? t.tensor[c] : 0u; };
    auto word_of = [&](uint32_t i) {
        return lane < kRowWords ? reinterpret_cast<const unsigned long long*>(t.rows + i)[lane] : 0ull;
    };
    auto put = [&](uint32_t k, uint32_t tile, unsigned long long word) {  // tile >= n: the end
        Stage& x = stage[k % S];
        if (lane < kRowWords) reinterpret_cast<unsigned long long*>(&x.row)[lane] = word;
        if (lane == 0) x.end = tile >= n;
        __syncwarp();
        if (tile < n) {
            issue(tile, x, &ring.full[k % S]);
        } else {
            mbar_arrive(&ring.full[k % S]);
            if (lane == 0) mbar_arrive(&ring.full[k % S]);
        }
    };
    auto deal = [&]() { return lane == 0 ? own + atomicAdd(&t.counters[2], 1u) : 0u; };  // lane 0 has it
    unsigned long long word[S];
#pragma unroll
    for (int j = 0; j < S; ++j) word[j] = word_of(blockIdx.x + j * gridDim.x < n ? tensor[j] : 0u);
    grid_wait();
    uint32_t k = 0;  // tiles put
    bool end = false;
#pragma unroll
    for (int j = 0; j < S; ++j)
        if (!end) {
            const uint32_t tile = blockIdx.x + j * gridDim.x;
            put(k++, tile, word[j]);
            end = tile >= n;
        }
    const bool dealt = n > own;  // a short list is all the CTAs' own: no counter
    if (ready() && !end) {
        // three tiles ahead of the copies: the counter, the tensor, the row
        uint32_t first = n, second = n, third = n;
        if (dealt) {
            first = deal(), second = deal(), third = deal();
            first = __shfl_sync(0xFFFFFFFFu, first, 0), second = __shfl_sync(0xFFFFFFFFu, second, 0);
        }
        unsigned long long first_word = word_of(tensor_of(first));
        uint32_t second_tensor = tensor_of(second);
        while (!end) {
            // every warp is done with the tile that the stage holds
            if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&ring.empty[k % S], (k / S - 1) & 1u))) {
                if (lane == 0) atomicOr(error, ZERO_DEVERR_WAIT_TIMEOUT);
                break;
            }
            put(k++, first, first_word);
            end = first >= n;
            first = second;
            first_word = word_of(second_tensor);
            second = __shfl_sync(0xFFFFFFFFu, third, 0);
            second_tensor = tensor_of(second);
            third = second < n ? deal() : n;
        }
    }
    // the last copies land before the CTA gives up its shared memory (they
    // have, unless the step is skipped or a wait ran out)
    for (uint32_t j = k > S ? k - S : 0u; j < k; ++j) {
        bool landed = false;
        for (int tries = 0; tries < kDrainTries && !landed; ++tries)
            landed = mbar_wait_bounded(&ring.full[j % S], (j / S) & 1u);
        if (!landed) atomicOr(error, ZERO_DEVERR_DRAIN_TIMEOUT);
    }
    if (lane == 0 && dealt) {
        __threadfence();
        if (atomicInc(&t.counters[1], gridDim.x - 1) == gridDim.x - 1) t.counters[2] = 0;
    }
}

// A computing warp: work(stage) for each of the CTA's tiles.
template <int S, class Stage, class Work>
__device__ __forceinline__ void ring_compute(int32_t* error, Stage* stage, Ring<S>& ring, Work work) {
    const int lane = threadIdx.x & 31;
    for (uint32_t k = 0;; ++k) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&ring.full[k % S], (k / S) & 1u))) {
            if (lane == 0) atomicOr(error, ZERO_DEVERR_WAIT_TIMEOUT);
            return;
        }
        if (stage[k % S].end) return;
        work(stage[k % S]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ring.empty[k % S]);
    }
}

// ----------------------------------------------------------------------------
// AdamW, 32-bit states
//
//   g = x / scale * clip,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// with one binary32 rounding per operation (adamw1), so that a tensor gets the
// same bits here as in the flat buffer.  Bound by memory: 14 bytes read and 14
// written per element with 16-bit gradients and copies.  GB300, 1.56e9
// elements in 580 tensors: 6.16 ms, 7.1 TB/s (the copy that the roofline is
// measured with: 6.77).  80K elements in 50 tensors: 3.6 us from a graph, the
// latency of launch, copies, constants, update and stores one after the other.
// ----------------------------------------------------------------------------
// A computing warp takes 256 elements of a tile, 8 consecutive ones per lane.
// The 8 begin on the boundaries that the states' addresses give
// (MultiRow::shift), so that a tensor anywhere in a flat buffer is copied but
// for its first and last few elements, which are read by plain loads.
// Parameters and gradients at other distances are copied from the boundary
// before and taken over by as many elements (GB300, 90e6 elements, one of the
// arrays apart from a gapless buffer: 363 us as aligned; by plain loads 482 to
// 716).
constexpr int kItem32 = 32 * kVec;
constexpr int kWarps32 = kChunk / kItem32;
constexpr int kThreads32 = 32 * (kWarps32 + 1);

template <class G>
struct __align__(128) Stage32 {
    float p[kChunk + 4];  // element e at e + over_p
    float m[kChunk];
    float v[kChunk];
    static constexpr int kPad = 16 / sizeof(typename G::T);
    typename G::T g[kChunk + kPad];  // element e at e + over_g
    MultiRow row;
    int64_t begin;  // the tile's first element in its tensor (below zero: that many do not exist)
    int32_t lo, hi; // elements of the tile that were copied
    int32_t over_p, over_g;
    bool end;       // no tile: the list's end
};
template <class G>
struct Smem32 {
    static constexpr int kStages = 3;
    Stage32<G> stage[kStages];
    float turn[kWarps32][kItem32];
    Ring<kStages> ring;
};

__device__ __forceinline__ void lds8(const float* p, float (&o)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
    o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
}

template <class G, class O>
__global__ void __launch_bounds__(kThreads32, 2) multi_adamw_kernel(const __grid_constant__ MultiArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    Smem32<G>& sh = *reinterpret_cast<Smem32<G>*>(smem);
    __shared__ MultiShared s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ring_init<kWarps32>(sh.ring);
    if (warp == kWarps32) {
        ring_fetch<Smem32<G>::kStages>(a.t, &a.st->error, sh.stage, sh.ring, [&](uint32_t tile, Stage32<G>& x, uint64_t* bar) {
            const MultiRow& r = x.row;
            const int64_t w0 = (int64_t)(tile - r.first_chunk) * kChunk - r.shift;
            int64_t left = r.numel - w0;
            if (kChecked) left -= (int64_t)a.t.slack;
            // parameters and gradients at another distance from a boundary than
            // the states are copied from the boundary before to the one behind,
            // inside the tensor
            constexpr int kPad = Stage32<G>::kPad;
            const typename G::T* const g = static_cast<const typename G::T*>(r.grad) + w0;
            const float* const p = r.master + w0;
            const int over_p = (int)(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(float));
            const int over_g = (int)(reinterpret_cast<uintptr_t>(g) % 16 / sizeof(typename G::T));
            const int more_p = over_p ? 4 - over_p : 0, more_g = over_g ? kPad - over_g : 0;
            int lo = w0 < 0 ? kVec : 0;
            if (w0 + lo < max(over_p, over_g)) lo += kVec;
            left = min(left - max(more_p, more_g), (int64_t)kChunk);
            int hi = left < kVec ? 0 : (int)left / kVec * kVec;
            if (!(r.vec & kVecStates) || hi < lo) hi = lo;
            copies_arrive(bar);
            if (lane == 0) {
                x.begin = w0;
                x.lo = lo;
                x.hi = hi;
                x.over_p = over_p;
                x.over_g = over_g;
                const uint32_t n = (uint32_t)(hi - lo);
                const uint32_t bytes_p = (n + over_p + more_p) * sizeof(float), bytes_g = (n + over_g + more_g) * sizeof(typename G::T);
                mbar_arrive_expect_tx(bar, n > 0 ? bytes_p + n * 2 * sizeof(float) + bytes_g : 0);
                if (n > 0) {
                    bulk_g2s(x.p + lo, p + lo - over_p, bytes_p, bar);
                    bulk_g2s(x.m + lo, r.m + w0 + lo, n * sizeof(float), bar);
                    bulk_g2s(x.v + lo, r.v + w0 + lo, n * sizeof(float), bar);
                    bulk_g2s(x.g + lo, g + lo - over_g, bytes_g, bar);
                }
            }
        }, [&]() {
            const bool apply = multi_constants(a, s);
            if (lane == 0) advance_step(a);
            return apply;
        });
        return;
    }
    grid_wait();
    if (!multi_constants(a, s)) return;
    const float unscale = s.unscale;
    ring_compute<Smem32<G>::kStages>(&a.st->error, sh.stage, sh.ring, [&](Stage32<G>& x) {
        const MultiRow& r = x.row;
        const int at = (warp * 32 + lane) * kVec;  // place in the tile
        const bool fast = at >= x.lo && at + kVec <= x.hi;
        const int64_t i = x.begin + at;
        int e0 = 0, e1 = kVec;
        const uint32_t vec = r.vec;
        // parameters or their copies that are not on the states' boundaries:
        // neighbouring lanes store neighbouring elements
        const bool turned = (vec & (kVecMaster | kVecOut)) != (kVecMaster | kVecOut);
        if (fast || span8(a.t, r, i, e0, e1)) {
            const AdamConsts k = s.k[r.group];
            float g[8], p[8], m[8], v[8];
            if (fast) {
                if (x.over_g) G::load8_over(&x.g[at], x.over_g, g);
                else G::load8(&x.g[at], g);
                if (x.over_p) lds8_over(&x.p[at], x.over_p, p);
                else lds8(&x.p[at], p);
                lds8(&x.m[at], m);
                lds8(&x.v[at], v);
            } else {
                // ones where there is nothing: zeros would take the slow ways of
                // the division and the root
                load_grad<G>(r.grad, i, e0, e1, vec & kVecGrad, g, 1.0f);
                load_f32(r.master + i, e0, e1, vec & kVecMaster, p, 1.0f);
                load_f32(r.m + i, e0, e1, vec & kVecStates, m, 1.0f);
                load_f32(r.v + i, e0, e1, vec & kVecStates, v, 1.0f);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = __fmul_rn(g[e], unscale);
            if (all_zero8x3(g, m, v)) {  // e.g. embedding rows that no batch has held
#pragma unroll
                for (int e = 0; e < 8; ++e) adamw1_zero_state(p[e], m[e], v[e], g[e], k);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) adamw1(p[e], m[e], v[e], g[e], k);
            }
            store_f32(r.m + i, e0, e1, vec & kVecStates, m);
            store_f32(r.v + i, e0, e1, vec & kVecStates, v);
            if (fast && turned) {
                float4* const t = reinterpret_cast<float4*>(&sh.turn[warp][lane * kVec]);
                t[0] = make_float4(p[0], p[1], p[2], p[3]);
                t[1] = make_float4(p[4], p[5], p[6], p[7]);
            } else {
                store_f32(r.master + i, e0, e1, vec & kVecMaster, p);
                if constexpr (O::kOut) store_out<O>(r.out + i, e0, e1, vec & kVecOut, p);
            }
        }
        if (turned) {
            __syncwarp();
            float q[kVec];
#pragma unroll
            for (int j = 0; j < kVec; ++j) q[j] = sh.turn[warp][32 * j + lane];
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const int e = warp * kItem32 + 32 * j + lane;
                if (e >= x.lo && e < x.hi) {
                    r.master[x.begin + e] = q[j];
                    if constexpr (O::kOut) r.out[x.begin + e] = O::enc1(q[j]);
                }
            }
        }
    });
}

// ----------------------------------------------------------------------------
// AdamW, 8-bit states
//
// The same update between decoding and encoding.  16.125 bytes per element, a
// little over half of the 32-bit form's, leave half of its time for more work,
// so the work had to shrink: powers of two as scales make scaling exact and
// need no division, the conversions run in hardware two at a time, stochastic
// rounding is one integer addition to a value's bits, its random integers one
// multiplication each, maxima take three inputs, and root and division are
// approximate.  16 elements a lane halve what is paid per lane and per warp
// (8 a lane, plain loads: 68 instructions an element and 4694 us at 1.56e9
// elements; as it is: 3.56 ms, 7.05 TB/s, bound by memory).
// ----------------------------------------------------------------------------
// A computing warp takes 512 elements of a tile, 16 consecutive ones per lane (a
// block of 32 is two lanes).  The blocks begin where the tensor does, so
// parameters and gradients that are not on a 16-byte boundary cannot be moved
// onto one by a shift of the work, as in the 32-bit update: they are copied
// from the boundary before, taken over by as many elements, and the results
// turned round in shared memory so that neighbouring lanes store neighbouring
// pairs (GB300, 175e6 elements in 158 tensors at odd offsets: 423 us, aligned 408;
// stored one by one 467, read by plain loads as well 588).  A tensor's last few
// elements, and its first 16 if they are not on a boundary, are read by plain
// loads.
constexpr int kLane8 = 16;
constexpr int kItem8 = 32 * kLane8;
constexpr int kWarps8 = kChunk / kItem8;
constexpr int kThreads8 = 32 * (kWarps8 + 1);
static_assert(kChunk / kBlock8 <= 128, "a fetching lane copies 4 scale bytes of a tile");

template <class G>
struct __align__(128) Stage8 {
    static constexpr int kPad = 16 / sizeof(typename G::T);
    float p[kChunk + 4];           // element e at e + over_p
    typename G::T g[kChunk + kPad];
    uint8_t m[kChunk];
    uint8_t v[kChunk];
    uint8_t ms[kChunk / kBlock8];
    uint8_t vs[kChunk / kBlock8];
    MultiRow row;
    int64_t begin;  // the tile's first element in its tensor
    int32_t lo, hi; // elements of the tile that were copied
    int32_t over_p, over_g;
    bool end;       // no tile: the list's end
};
template <class G>
struct Smem8 {
    static constexpr int kStages = 2;
    Stage8<G> stage[kStages];
    float turn[kWarps8][kItem8];
    Ring<kStages> ring;
};

// 16 codes <-> values.
template <class Q>
__device__ __forceinline__ void decode16(uint4 c, float scale, float (&o)[16]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 f = Q::dec2((uint16_t)(w[k >> 1] >> (16 * (k & 1))));
        o[2 * k] = __fmul_rn(f.x, scale);
        o[2 * k + 1] = __fmul_rn(f.y, scale);
    }
}
// Largest magnitude, NaN if one is NaN: three-input maxima.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float top16(const float (&x)[16]) {
    const float a = max3_abs(x[0], x[1], x[2]), b = max3_abs(x[3], x[4], x[5]), c = max3_abs(x[6], x[7], x[8]);
    const float d = max3_abs(x[9], x[10], x[11]), e = max3_abs(x[12], x[13], x[14]);
    return max3_abs(max3_abs(a, b, c), max3_abs(d, e, x[15]), 0.0f);
}
template <class Q>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
    if (top >= 0x7F800000u) return 255u;
    // one more when the mantissa is above 1.75; in binary32's last binade there
    // is no more, and what is above 1.75 * 2^127 saturates
    const int e = (int)min((top + 0x1FFFFFu) >> 23, 254u);
    return (uint32_t)max(1, e - Q::kTop);
}
template <class Q>
__device__ __forceinline__ uint32_t block_scale16(const float (&x)[16]) {
    float t = top16(x);
    t = max3_abs(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1), 0.0f);
    return scale_byte<Q>(__float_as_uint(t));
}
// One stochastically rounded value before its conversion to a code: x on the
// block's scale, a random integer added below the bits that are kept.
template <class Q>
__device__ __forceinline__ float dither(float x, float inv, uint32_t rnd) {
    const float z = __fmul_rn(x, inv);
    float y = __uint_as_float((__float_as_uint(z) + (rnd >> (32 - Q::kCut))) & ~((1u << Q::kCut) - 1u));
    if constexpr (Q::kFloor)
        if (z > 0.0f) y = fmaxf(y, kSmallestE5m2);
    return y;
}
// Codes of a lane's 16 m and v, whose random integers alternate.
__device__ __forceinline__ void encode16(const float (&m)[16], const float (&v)[16], uint32_t bm, uint32_t bv, uint32_t key,
                                         uint32_t group, uint4& cm, uint4& cv) {
    const float im = __uint_as_float((254u - bm) << 23), iv = __uint_as_float((254u - bv) << 23);
    uint32_t wm[4], wv[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t x = mix32(key + 0x9E3779B1u * (group + h));
#pragma unroll
        for (int k = 2 * h; k < 2 * h + 2; ++k) {
            uint32_t qm[2], qv[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float ym[2], yv[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int e = 4 * k + 2 * j + i;
                    x = x * 1664525u + 1013904223u;
                    ym[i] = dither<E4m3>(m[e], im, x);
                    x = x * 1664525u + 1013904223u;
                    yv[i] = dither<E5m2>(v[e], iv, x);
                }
                qm[j] = E4m3::enc2(ym[0], ym[1]);
                qv[j] = E5m2::enc2(yv[0], yv[1]);
            }
            wm[k] = qm[0] | (qm[1] << 16);
            wv[k] = qv[0] | (qv[1] << 16);
        }
    }
    // NaN in both types
    if (bm == 255u) wm[0] = wm[1] = wm[2] = wm[3] = 0x7F7F7F7Fu;
    if (bv == 255u) wv[0] = wv[1] = wv[2] = wv[3] = 0x7F7F7F7Fu;
    cm = make_uint4(wm[0], wm[1], wm[2], wm[3]);
    cv = make_uint4(wv[0], wv[1], wv[2], wv[3]);
}

// A lane's 16 codes, of which nv exist.
__device__ __forceinline__ uint4 load_codes16(const uint8_t* p, int nv, bool vec) {
    if (vec && nv == 16) return __ldcs(reinterpret_cast<const uint4*>(p));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (e < nv) w[e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_codes16(uint8_t* p, int nv, bool vec, uint4 c) {
    if (vec && nv == 16) {
        __stcs(reinterpret_cast<uint4*>(p), c);
        return;
    }
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int e = 0; e < 16; ++e)
        if (e < nv) p[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
}

// The parameter update needs neither the rounded square root nor the rounded
// division: their errors (2^-22 of the update) stay out of the states.  v below
// 2^-126 counts as zero in the root; the constants keep eps at 2^-126 at least.
__device__ __forceinline__ float sqrt_approx(float x) {
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Up to 512 parameters of a tensor from w0 on out of shared memory, and their
// 16-bit copies: neighbouring lanes store neighbouring pairs, which begin one
// element later where the addresses are odd.
template <class O>
__device__ __forceinline__ void store_turned(const MultiRow& r, const float* turn, int64_t w0, int some) {
    const int lane = threadIdx.x & 31;
    float* const p = r.master + w0;
    uint16_t* const o = r.out + w0;
    const int odd = (int)(reinterpret_cast<uintptr_t>(p) / sizeof(float) & 1);
    const bool pairs = !O::kOut || (int)(reinterpret_cast<uintptr_t>(o) / sizeof(uint16_t) & 1) == odd;
    auto one = [&](int e) {
        p[e] = turn[e];
        if constexpr (O::kOut) o[e] = O::enc1(turn[e]);
    };
    if (pairs) {
        float q[kLane8];
#pragma unroll
        for (int j = 0; j < kLane8 / 2; ++j) {
            const int e = 64 * j + 2 * lane + odd;
            q[2 * j] = turn[e];
            q[2 * j + 1] = turn[min(e + 1, kItem8 - 1)];
        }
#pragma unroll
        for (int j = 0; j < kLane8 / 2; ++j) {
            const int e = 64 * j + 2 * lane + odd;
            if (e + 1 < some) {
                __stcs(reinterpret_cast<float2*>(p + e), make_float2(q[2 * j], q[2 * j + 1]));
                if constexpr (O::kOut) __stcs(reinterpret_cast<uint32_t*>(o + e), O::pack(q[2 * j], q[2 * j + 1]));
            }
        }
        // what the pairs leave: the first element where they begin at the second, and the last
        if (lane == 0 && odd && some > 0) one(0);
        if (lane == 1 && some > odd && ((some - odd) & 1)) one(some - 1);
    } else {
#pragma unroll
        for (int j = 0; j < kLane8; ++j)
            if (32 * j + lane < some) one(32 * j + lane);
    }
}

template <class G, class O>
__global__ void __launch_bounds__(kThreads8, 4) multi_adamw8_kernel(const __grid_constant__ MultiArgs a) {
    extern __shared__ __align__(128) unsigned char smem[];
    Smem8<G>& sh = *reinterpret_cast<Smem8<G>*>(smem);
    __shared__ MultiShared s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ring_init<kWarps8>(sh.ring);
    if (warp == kWarps8) {
        ring_fetch<Smem8<G>::kStages>(a.t, &a.st->error, sh.stage, sh.ring, [&](uint32_t tile, Stage8<G>& x, uint64_t* bar) {
            const MultiRow& r = x.row;
            const int64_t w0 = (int64_t)(tile - r.first_chunk) * kChunk;
            int64_t left = r.numel - w0;
            if (kChecked) left -= (int64_t)a.t.slack;
            const typename G::T* const g = static_cast<const typename G::T*>(r.grad) + w0;
            const float* const p = r.master + w0;
            constexpr int kPad = Stage8<G>::kPad;
            const int over_p = (int)(reinterpret_cast<uintptr_t>(p) % 16 / sizeof(float));
            const int over_g = (int)(reinterpret_cast<uintptr_t>(g) % 16 / sizeof(typename G::T));
            // the copies begin on the boundary before and end on the one
            // behind, inside the tensor
            const int lo = w0 == 0 && (over_p | over_g) ? kLane8 : 0;
            const int more_p = over_p ? 4 - over_p : 0, more_g = over_g ? kPad - over_g : 0;
            const int blocks = (int)min((left + kBlock8 - 1) / kBlock8, (int64_t)(kChunk / kBlock8));
            left = min(left - max(more_p, more_g), (int64_t)kChunk);
            int hi = left < kLane8 || !(r.vec & kCodes) ? 0 : (int)left / kLane8 * kLane8;
            if (hi < lo) hi = lo;
            const int n = hi - lo;
            if (n > 0 && lane * 4 < blocks) {
                copy4_async(&x.ms[lane * 4], r.ms + w0 / kBlock8 + lane * 4, blocks - lane * 4);
                copy4_async(&x.vs[lane * 4], r.vs + w0 / kBlock8 + lane * 4, blocks - lane * 4);
            }
            copies_arrive(bar);
            if (lane == 0) {
                x.begin = w0;
                x.lo = lo;
                x.hi = hi;
                x.over_p = over_p;
                x.over_g = over_g;
                const uint32_t bytes_p = (n + over_p + more_p) * sizeof(float), bytes_g = (n + over_g + more_g) * sizeof(typename G::T);
                mbar_arrive_expect_tx(bar, n > 0 ? bytes_p + bytes_g + 2 * n : 0);
                if (n > 0) {
                    bulk_g2s(x.p + lo, p + lo - over_p, bytes_p, bar);
                    bulk_g2s(x.g + lo, g + lo - over_g, bytes_g, bar);
                    bulk_g2s(x.m + lo, r.m8 + w0 + lo, n, bar);
                    bulk_g2s(x.v + lo, r.v8 + w0 + lo, n, bar);
                }
            }
        }, [&]() {
            const bool apply = multi_constants(a, s);
            if (lane == 0) advance_step(a);
            return apply;
        });
        return;
    }
    grid_wait();
    if (!multi_constants(a, s)) return;
    const float factor = s.factor, unscale = s.unscale;
    const bool two = s.two != 0;
    ring_compute<Smem8<G>::kStages>(&a.st->error, sh.stage, sh.ring, [&](Stage8<G>& x) {
        const MultiRow& r = x.row;
        const int at = (warp * 32 + lane) * kLane8;  // place in the tile
        const bool copied = at >= x.lo && at + kLane8 <= x.hi;
        const int64_t w0 = x.begin + warp * kItem8, i = x.begin + at;
        int some = kItem8;  // elements of the item, and of the lane
        if ((warp + 1) * kItem8 > x.hi) {
            const int64_t left = r.numel - w0;
            some = left >= kItem8 ? kItem8 : (left > 0 ? (int)left : 0);
            const uint64_t lim = (uint64_t)r.numel > a.t.slack ? (uint64_t)r.numel - a.t.slack : 0;
            if (some > 0 && !in_bounds((uint64_t)(w0 + some), lim)) some = 0;
        }
        const int nv = min(max(some - lane * kLane8, 0), kLane8);
        if (some > 0) {
            const int64_t blk = i / kBlock8;
            const Const8 c = s.c8[r.group];
            const bool over = (x.over_p | x.over_g) != 0, turned = !(r.vec & kWhole8);
            // a lane has 16 copied elements, fewer at a tensor's ends, or none
            float m[16], v[16];
            if (copied) {
                decode16<E4m3>(*reinterpret_cast<const uint4*>(&x.m[at]), scale_of(x.ms[at / kBlock8]), m);
                decode16<E5m2>(*reinterpret_cast<const uint4*>(&x.v[at]), scale_of(x.vs[at / kBlock8]), v);
            } else if (nv > 0) {
                decode16<E4m3>(load_codes16(r.m8 + i, nv, r.vec & kCodes), scale_of(r.ms[blk]), m);
                decode16<E5m2>(load_codes16(r.v8 + i, nv, r.vec & kCodes), scale_of(r.vs[blk]), v);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) m[e] = v[e] = 0.0f;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int o = 8 * h;
                float g[8], p[8];
                if (copied) {
                    if (over) {
                        G::load8_over(&x.g[at + o], x.over_g, g);
                        lds8_over(&x.p[at + o], x.over_p, p);
                    } else {
                        G::load8(&x.g[at + o], g);
                        lds8(&x.p[at + o], p);
                    }
                } else if (nv > 0) {
                    load_grad<G>(r.grad, i + o, 0, nv - o, false, g);
                    load_f32(r.master + i + o, 0, nv - o, false, p);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] = p[e] = 0.0f;
                }
                if (two) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] = __fmul_rn(g[e], unscale);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float gc = __fmul_rn(g[e], factor);
                    m[o + e] = __fadd_rn(__fmul_rn(c.b1, m[o + e]), __fmul_rn(c.omb1, gc));
                    v[o + e] = __fadd_rn(__fmul_rn(c.b2, v[o + e]), __fmul_rn(c.omb2, __fmul_rn(gc, gc)));
                    const float den = __fmaf_rn(sqrt_approx(v[o + e]), c.isb, c.eps);
                    p[e] = __fmaf_rn(-c.step_size, __fmul_rn(m[o + e], rcp_approx(den)), __fmul_rn(p[e], c.decay));
                }
                if (turned) {
                    float4* const t = reinterpret_cast<float4*>(&sh.turn[warp][lane * kLane8 + o]);
                    t[0] = make_float4(p[0], p[1], p[2], p[3]);
                    t[1] = make_float4(p[4], p[5], p[6], p[7]);
                } else if (copied) {
                    st8(r.master + i + o, p);
                    if constexpr (O::kOut) st_stream(r.out + i + o, pack8<O>(p));
                } else if (nv > 0) {
                    store_f32(r.master + i + o, 0, nv - o, false, p);
                    if constexpr (O::kOut) store_out<O>(r.out + i + o, 0, nv - o, false, p);
                }
            }
            if (turned) {
                __syncwarp();
                store_turned<O>(r, sh.turn[warp], w0, some);
                __syncwarp();
            }
            const uint32_t bm = block_scale16<E4m3>(m), bv = block_scale16<E5m2>(v);
            uint4 cm, cv;
            encode16(m, v, bm, bv, mix32(s.key + r.tensor), (uint32_t)(i >> 3), cm, cv);
            if (nv > 0) {
                store_codes16(r.m8 + i, nv, r.vec & kCodes, cm);
                store_codes16(r.v8 + i, nv, r.vec & kCodes, cv);
                if ((lane & 1) == 0) {
                    r.ms[blk] = (uint8_t)bm;
                    r.vs[blk] = (uint8_t)bv;
                }
            }
        }
    });
}

// ----------------------------------------------------------------------------
// 32-bit states into the 8-bit form and back: 10.06 bytes per element, bound by
// memory.  GB300, 355e6 elements: encode 497 us (7.2 TB/s), decode 510 us (7.0
// TB/s; 621 with all CTAs that fit on an SM, 690 with two).
// ----------------------------------------------------------------------------
// Nearest codes (ties to even) of 16 values.
template <class Q>
__device__ __forceinline__ uint4 nearest16(const float (&x)[16], uint32_t byte) {
    const float inv = __uint_as_float((254u - byte) << 23);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float z = __fmul_rn(x[2 * k + i], inv);
            y[i] = Q::kFloor && z > 0.0f ? fmaxf(z, kSmallestE5m2) : z;
        }
        const uint32_t q = Q::enc2(y[0], y[1]);
        if (k & 1) w[k >> 1] |= q << 16;
        else w[k >> 1] = q;
    }
    if (byte == 255u) w[0] = w[1] = w[2] = w[3] = 0x7F7F7F7Fu;  // NaN in both types
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Tiles and lanes as in the 8-bit update.
struct __align__(128) StageEncode {
    float m[kChunk];
    float v[kChunk];
    MultiRow row;
    int64_t begin, whole;
    bool end;
};
struct __align__(128) StageDecode {
    uint8_t m[kChunk];
    uint8_t v[kChunk];
    uint8_t ms[kChunk / kBlock8];
    uint8_t vs[kChunk / kBlock8];
    MultiRow row;
    int64_t begin, whole;
    bool end;
};
template <class Stage>
struct SmemCodec {
    static constexpr int kStages = 3;
    Stage stage[kStages];
    Ring<kStages> ring;
};

template <bool ENCODE>
__global__ void __launch_bounds__(kThreads8, 4) multi_codec_kernel(const __grid_constant__ MultiTable t) {
    using Stage = std::conditional_t<ENCODE, StageEncode, StageDecode>;
    using Smem = SmemCodec<Stage>;
    extern __shared__ __align__(128) unsigned char smem[];
    Smem& sh = *reinterpret_cast<Smem*>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t* const error = reinterpret_cast<int32_t*>(&t.counters[3]);
    ring_init<kWarps8>(sh.ring);
    if (warp == kWarps8) {
        ring_fetch<Smem::kStages>(t, error, sh.stage, sh.ring, [&](uint32_t tile, Stage& x, uint64_t* bar) {
            const MultiRow& r = x.row;
            const int64_t w0 = (int64_t)(tile - r.first_chunk) * kChunk;
            int64_t left = r.numel - w0;
            if (kChecked) left -= (int64_t)t.slack;
            const bool wide = (r.vec & kCodec) && (r.vec & kCodes);
            const int n = !wide || left < kLane8 ? 0 : (int)min(left, (int64_t)kChunk) / kLane8 * kLane8;
            if constexpr (!ENCODE) {
                const int blocks = (n + kBlock8 - 1) / kBlock8;
                if (lane * 4 < blocks) {
                    copy4_async(&x.ms[lane * 4], r.ms + w0 / kBlock8 + lane * 4, blocks - lane * 4);
                    copy4_async(&x.vs[lane * 4], r.vs + w0 / kBlock8 + lane * 4, blocks - lane * 4);
                }
            }
            copies_arrive(bar);
            if (lane == 0) {
                x.begin = w0;
                x.whole = n;
                mbar_arrive_expect_tx(bar, (uint32_t)n * (ENCODE ? 8 : 2));
                if (n > 0) {
                    if constexpr (ENCODE) {
                        bulk_g2s(x.m, r.m + w0, n * sizeof(float), bar);
                        bulk_g2s(x.v, r.v + w0, n * sizeof(float), bar);
                    } else {
                        bulk_g2s(x.m, r.m8 + w0, n, bar);
                        bulk_g2s(x.v, r.v8 + w0, n, bar);
                    }
                }
            }
        }, []() { return true; });
        return;
    }
    grid_wait();
    ring_compute<Smem::kStages>(error, sh.stage, sh.ring, [&](Stage& x) {
        const MultiRow& r = x.row;
        const int at = (warp * 32 + lane) * kLane8;
        const bool fast = at + kLane8 <= x.whole;
        const int64_t i = x.begin + at;
        int nv = kLane8;
        if ((warp + 1) * kItem8 > x.whole) {
            const int64_t left = r.numel - i;
            nv = left >= kLane8 ? kLane8 : (left > 0 ? (int)left : 0);
            const uint64_t lim = (uint64_t)r.numel > t.slack ? (uint64_t)r.numel - t.slack : 0;
            if (nv > 0 && !in_bounds((uint64_t)(i + nv), lim)) nv = 0;
            if (!__any_sync(0xFFFFFFFFu, nv > 0)) return;
        }
        const bool wide = r.vec & kCodec, codes = r.vec & kCodes;
        const int64_t blk = i / kBlock8;
        float m[16], v[16];
        if constexpr (ENCODE) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float(&mh)[8] = *reinterpret_cast<float(*)[8]>(&m[8 * h]);
                float(&vh)[8] = *reinterpret_cast<float(*)[8]>(&v[8 * h]);
                if (fast) {
                    lds8(&x.m[at + 8 * h], mh);
                    lds8(&x.v[at + 8 * h], vh);
                } else {
                    load_f32(r.m + i + 8 * h, 0, nv - 8 * h, wide && nv == 16, mh);
                    load_f32(r.v + i + 8 * h, 0, nv - 8 * h, wide && nv == 16, vh);
                }
            }
            const uint32_t bm = block_scale16<E4m3>(m), bv = block_scale16<E5m2>(v);
            if (nv > 0) {
                store_codes16(r.m8 + i, nv, codes, nearest16<E4m3>(m, bm));
                store_codes16(r.v8 + i, nv, codes, nearest16<E5m2>(v, bv));
                if ((lane & 1) == 0) {
                    r.ms[blk] = (uint8_t)bm;
                    r.vs[blk] = (uint8_t)bv;
                }
            }
        } else if (nv > 0) {
            if (fast) {
                decode16<E4m3>(*reinterpret_cast<const uint4*>(&x.m[at]), scale_of(x.ms[at / kBlock8]), m);
                decode16<E5m2>(*reinterpret_cast<const uint4*>(&x.v[at]), scale_of(x.vs[at / kBlock8]), v);
            } else {
                decode16<E4m3>(load_codes16(r.m8 + i, nv, codes), scale_of(r.ms[blk]), m);
                decode16<E5m2>(load_codes16(r.v8 + i, nv, codes), scale_of(r.vs[blk]), v);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                store_f32(r.m + i + 8 * h, 0, nv - 8 * h, wide && nv == 16, *reinterpret_cast<const float(*)[8]>(&m[8 * h]));
                store_f32(r.v + i + 8 * h, 0, nv - 8 * h, wide && nv == 16, *reinterpret_cast<const float(*)[8]>(&v[8 * h]));
            }
        }
    });
}

// ----------------------------------------------------------------------------
// Global norm and step decision
//
// sum x^2 over the list.  A thread adds the squares of 8 elements with fused
// multiply-adds and carries the rounding errors of adding those sums up
// (two_sum); pairs (sum, error) are combined by shuffles and, among the CTAs,
// by the one that ends last.  The split into kSlices ranges is fixed, so the
// result does not depend on the grid.  Bound by memory: GB300, 1.56e9 16-bit
// gradients 433 us (7.2 TB/s read); 30.7e6 of them 15.7 us, of which 9 are the
// bytes and the rest launch, first loads and the last CTA's sum.
// ----------------------------------------------------------------------------
// The step decision, as zero_grad_norm makes it: skip on overflow, else the clip
// coefficient, the step counter and beta^t; the loss-scale schedule.  Two
// threads: the clip coefficient, and what does not depend on the norm's value.
__device__ __forceinline__ float clip_of(bool bad, double norm, double max_norm) {
    const double most = __dadd_rn(norm, 1e-6);
    if (bad || !(max_norm > 0.0) || max_norm >= most) return 1.0f;  // a quotient of 1 or more is not needed
    return __double2float_rn(__ddiv_rn(max_norm, most));
}
__device__ __forceinline__ void decide_step(zero_step_state* st, bool bad) {
    st->apply = bad ? 0 : 1;
    if (bad) {
        st->skipped += 1;
        st->good_steps = 0;
        if (st->dynamic_scale) st->loss_scale = fmaxf(1.0f, __fmul_rn(st->loss_scale, 0.5f));
        return;
    }
    st->t += 1;
    st->beta1_pow = __dmul_rn(st->beta1_pow, st->beta1);
    st->beta2_pow = __dmul_rn(st->beta2_pow, st->beta2);
    st->good_steps += 1;
    if (st->dynamic_scale && st->good_steps >= st->growth_interval) {
        st->loss_scale = __fmul_rn(st->loss_scale, 2.0f);
        st->good_steps = 0;
    }
}

// Sum of the CTA's (hi, lo) pairs in a fixed order; thread 0 gets it.
__device__ __forceinline__ float2 sum_pairs(float hi, float lo, float2* sh) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) combine_lanes(hi, lo, m);
    __syncthreads();  // sh: the sum before
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = make_float2(hi, lo);
    __syncthreads();
    if (threadIdx.x < 32) {
        const float2 q = threadIdx.x < kThreads / 32 ? sh[threadIdx.x] : make_float2(0.0f, 0.0f);
        hi = q.x, lo = q.y;
#pragma unroll
        for (int m = 1; m < kThreads / 32; m <<= 1) combine_lanes(hi, lo, m);
    }
    return make_float2(hi, lo);
}

template <class G>
__global__ void __launch_bounds__(kThreads, 8) multi_norm_kernel(const __grid_constant__ MultiTable t, double max_norm,
                                                              zero_step_state* st) {
    __shared__ float2 sh[kThreads / 32];
    __shared__ bool last;
    const uint32_t n_chunks = *t.n_chunks, n_slices = max(1u, min(n_chunks, (uint32_t)kSlices));
    grid_wait();
    for (uint32_t sl = blockIdx.x; sl < n_slices; sl += gridDim.x) {
        // the slice's chunks, tensor by tensor
        const uint32_t c1 = (uint32_t)((uint64_t)(sl + 1) * n_chunks / n_slices);
        uint32_t c = (uint32_t)((uint64_t)sl * n_chunks / n_slices);
        float hi = 0.0f, lo = 0.0f;
        while (c < c1) {
            const uint32_t n = t.tensor[c];
            const MultiRow& r = t.rows[n];
            const int64_t begin = (int64_t)(c - r.first_chunk) * kChunk - r.gshift;
            const uint32_t chunks = (uint32_t)((r.numel + max(r.shift, r.gshift) + kChunk - 1) / kChunk) - (c - r.first_chunk);
            const uint32_t take = min(chunks, c1 - c);
            const int64_t end = min(r.numel, begin + (int64_t)take * kChunk);
            const uint64_t lim = (uint64_t)r.numel > t.slack ? (uint64_t)r.numel - t.slack : 0;
            auto add = [&](const float (&g)[8]) {
                float q = __fmul_rn(g[0], g[0]);
#pragma unroll
                for (int e = 1; e < 8; ++e) q = __fmaf_rn(g[e], g[e], q);
                float sum, err;
                two_sum(hi, q, sum, err);
                hi = sum;
                lo = __fadd_rn(lo, err);
            };
            // kUnroll loads in flight per thread; they may stay in the cache for
            // the update
            constexpr int kUnroll = 64 / sizeof(typename G::Raw), kStep = kThreads * kVec;
            int64_t i = begin + threadIdx.x * kVec;
            auto one = [&]() {
                int e0, e1;
                if (span8(t, r, i, e0, e1)) {
                    float g[8];
                    load_grad<G>(r.grad, i, e0, e1, true, g);  // gshift puts the gradients on a boundary
                    add(g);
                }
                i += kStep;
            };
            if (begin < 0) one();  // the first vector is not whole
            for (; i + (kUnroll - 1) * kStep + kVec <= end; i += kUnroll * kStep) {
                if (!in_bounds((uint64_t)i + (kUnroll - 1) * kStep + kVec, lim)) break;
                typename G::Raw q[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) q[u] = G::raw(static_cast<const typename G::T*>(r.grad) + i + u * kStep);
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    float g[8];
                    G::values(q[u], g);
                    add(g);
                }
            }
            while (i < end) one();
            c += take;
        }
        const float2 sum = sum_pairs(hi, lo, sh);
        if (threadIdx.x == 0) t.partials[sl] = sum;
    }
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicInc(&t.counters[0], gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    float hi = 0.0f, lo = 0.0f;
    // all loads at once (one after the other: 0.3 us more on a list of 1216
    // slices)
    constexpr int kMost = (kSlices + kThreads - 1) / kThreads;
    float2 q[kMost];
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        const uint32_t sl = threadIdx.x + j * kThreads;
        q[j] = sl < n_slices ? __ldcg(&t.partials[sl]) : make_float2(0.0f, 0.0f);
    }
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
        float sum, err;
        two_sum(hi, q[j].x, sum, err);
        hi = sum;
        lo = __fadd_rn(lo, __fadd_rn(err, q[j].y));
    }
    const float scale = st->loss_scale;  // before the decision changes it
    const float2 both = sum_pairs(hi, lo, sh);
    if (threadIdx.x == 0) sh[0] = both;
    __syncthreads();
    if (threadIdx.x != 0 && threadIdx.x != 32) return;
    const double total = __dadd_rn((double)sh[0].x, (double)sh[0].y);
    const bool bad = !isfinite(total);  // an inf or NaN gradient, or a square beyond binary32
    if (threadIdx.x == 32) {
        st->nonfinite = 0;
        st->overflow = bad;
        *t.grad_scale = scale;
        decide_step(st, bad);
        return;
    }
    double norm = bad ? (double)INFINITY : __dsqrt_rn(total);
    if (!bad && scale != 1.0f) norm = __ddiv_rn(norm, (double)scale);
    st->grad_norm = norm;
    st->clip_coef = clip_of(bad, norm, max_norm);
}

}  // namespace zk

using namespace zero_detail;

struct zero_multi {
    std::vector<int64_t> numels;
    std::vector<int32_t> groups;
    int32_t n_groups = 0, grad_dtype = 0, param_dtype = 0;
    int64_t most_chunks = 0;  // wherever the tensors begin
    // the last bind
    int64_t n_chunks = 0;  // for the grid; the kernels go by the count in the workspace
    bool bound = false, grads = false, master = false, states32 = false, states8 = false, param16 = false;
    char* workspace = nullptr;
};

namespace {

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

int64_t chunks_of(int64_t numel, int64_t shift) {
    return numel > 0 ? (numel + shift + zk::kChunk - 1) / zk::kChunk : 0;
}

// Workspace layout: counters and the gradients' scale (256 bytes), rows, chunk map, norm partials, and the count of
// chunks, which every CTA reads first, away from the line that the counters' atomics and the decision write (GB300,
// norm of short lists: 4.5 to 5.4 us, next to the counters 0.1 to 0.2 more).
struct Places {
    int64_t rows, map, partials, count, total;
};
Places places(const zero_multi* M) {
    Places p;
    p.rows = 256;
    p.map = p.rows + up256((int64_t)M->numels.size() * (int64_t)sizeof(zk::MultiRow));
    p.partials = p.map + up256(M->most_chunks * (int64_t)sizeof(uint32_t));
    p.count = p.partials + up256(zk::kSlices * (int64_t)sizeof(float2));
    p.total = p.count + 256;
    return p;
}

zk::MultiTable table_of(const zero_multi* M) {
    const Places p = places(M);
    zk::MultiTable t{};
    t.counters = reinterpret_cast<uint32_t*>(M->workspace);
    t.grad_scale = reinterpret_cast<float*>(M->workspace + 128);
    t.rows = reinterpret_cast<const zk::MultiRow*>(M->workspace + p.rows);
    t.tensor = reinterpret_cast<const uint32_t*>(M->workspace + p.map);
    t.partials = reinterpret_cast<float2*>(M->workspace + p.partials);
    t.n_chunks = reinterpret_cast<const uint32_t*>(M->workspace + p.count);
    t.most_chunks = (uint32_t)M->most_chunks;
    t.n_tensors = (uint32_t)M->numels.size();
    t.slack = (uint64_t)check_slack();
    return t;
}

zero_status_t check_multi_hp(const zero_multi* M, const zero_adamw_hp* hp, const char* what, zk::MultiHp& out) {
    if (!hp) return fail(ZERO_ERR_INVALID, std::string(what) + ": NULL hyperparameters");
    out.n = M->n_groups;
    for (int g = 0; g < M->n_groups; ++g) {
        if (!(hp[g].lr >= 0.0) || !(hp[g].eps > 0.0) || !((float)hp[g].eps > 0.0f) || !(hp[g].weight_decay >= 0.0))
            return fail(ZERO_ERR_INVALID, std::string(what) +
                                              ": need lr >= 0, eps > 0 (also as a binary32), weight_decay >= 0");
        out.lr[g] = hp[g].lr;
        out.eps[g] = hp[g].eps;
        out.wd[g] = hp[g].weight_decay;
    }
    return ZERO_OK;
}

zero_status_t check_bound(const zero_multi* M, const char* what) {
    if (!M) return fail(ZERO_ERR_INVALID, std::string(what) + ": NULL list");
    if (!M->bound) return fail(ZERO_ERR_STATE, std::string(what) + ": the list is not bound");
    return ZERO_OK;
}

zero_status_t missing(const char* what, const char* arrays) {
    return fail(ZERO_ERR_STATE, std::string(what) + ": the list is not bound with " + arrays);
}

// Dynamic shared memory beyond 48 KB is a kernel attribute of each device.
template <class Kernel>
zero_status_t allow_smem(Kernel kern, size_t bytes, const char* what) {
    static std::mutex mu;
    static std::unordered_map<const void*, uint64_t> done;  // a bit per device
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    std::lock_guard<std::mutex> lock(mu);
    uint64_t& mask = done[reinterpret_cast<const void*>(kern)];
    if (!(mask & bit)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
            return after_launch(what);
        mask |= bit;
    }
    return ZERO_OK;
}

// A launch that may begin while the stream's last kernel ends (grid_wait).
template <class... P, class... A>
zero_status_t launch_early(void (*kern)(P...), int grid, int threads, size_t smem, cudaStream_t s, const char* what, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(ZERO_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
    }
    return after_launch(what);
}

// CTAs of a kernel on a ring of tiles: 16 computing warps on an SM.
template <class Kernel>
int ring_grid(Kernel kern, int64_t tiles, size_t smem, int threads) {
    const int64_t sms = sm_count() > 0 ? sm_count() : 1;
    return persistent_grid(kern, std::min<int64_t>(tiles, sms * (16 / (threads / 32 - 1))), smem, threads);
}

template <class G, class O>
zero_status_t launch_update(const zero_multi* M, bool eight, const zk::MultiArgs& a, cudaStream_t s) {
    const char* what = eight ? "zero_multi_adamw8" : "zero_multi_adamw";
    const size_t smem = eight ? sizeof(zk::Smem8<G>) : sizeof(zk::Smem32<G>);
    const int threads = eight ? zk::kThreads8 : zk::kThreads32;
    void (*kern)(zk::MultiArgs) = eight ? zk::multi_adamw8_kernel<G, O> : zk::multi_adamw_kernel<G, O>;
    const zero_status_t rc = allow_smem(kern, smem, what);
    if (rc != ZERO_OK) return rc;
    return launch_early(kern, ring_grid(kern, M->n_chunks, smem, threads), threads, smem, s, what, a);
}

template <class G>
zero_status_t launch_update_out(const zero_multi* M, bool eight, const zk::MultiArgs& a, cudaStream_t s) {
    if (M->param_dtype == ZERO_BF16) return launch_update<G, zk::OutBf16>(M, eight, a, s);
    if (M->param_dtype == ZERO_FP16) return launch_update<G, zk::OutFp16>(M, eight, a, s);
    return launch_update<G, zk::NoOut>(M, eight, a, s);
}

zero_status_t update(const zero_multi* M, const zero_adamw_hp* hp, int32_t flags, uint32_t seed, zero_step_state* st,
                     zero_stream_t stream, bool eight, const char* what) {
    zero_status_t rc;
    if ((rc = check_bound(M, what)) != ZERO_OK) return rc;
    if (flags & ~(ZERO_MULTI_ADVANCE | ZERO_MULTI_UNSCALED)) return fail(ZERO_ERR_INVALID, std::string(what) + ": unknown flags");
    zk::MultiArgs a{};
    if ((rc = check_multi_hp(M, hp, what, a.hp)) != ZERO_OK) return rc;
    if (!M->grads) return missing(what, "grads");
    if (!M->master) return missing(what, "master");
    if (eight && !M->states8) return missing(what, "8-bit states");
    if (!eight && !M->states32) return missing(what, "32-bit states");
    if (M->param_dtype != ZERO_NO_OUT && !M->param16) return missing(what, "param16");
    if ((rc = check_dev_ptr(st, what)) != ZERO_OK) return rc;
    a.t = table_of(M);
    a.st = st;
    a.flags = flags;
    a.seed = seed;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M->grad_dtype == ZERO_BF16) return launch_update_out<zk::GradBf16>(M, eight, a, s);
    if (M->grad_dtype == ZERO_FP16) return launch_update_out<zk::GradFp16>(M, eight, a, s);
    return launch_update_out<zk::GradFp32>(M, eight, a, s);
}

zero_status_t codec(const zero_multi* M, zero_stream_t stream, bool encode, const char* what) {
    zero_status_t rc;
    if ((rc = check_bound(M, what)) != ZERO_OK) return rc;
    if (!M->states32) return missing(what, "32-bit states");
    if (!M->states8) return missing(what, "8-bit states");
    if (M->n_chunks == 0) return ZERO_OK;
    const zk::MultiTable t = table_of(M);
    void (*kern)(zk::MultiTable) = encode ? zk::multi_codec_kernel<true> : zk::multi_codec_kernel<false>;
    const size_t smem = encode ? sizeof(zk::SmemCodec<zk::StageEncode>) : sizeof(zk::SmemCodec<zk::StageDecode>);
    if ((rc = allow_smem(kern, smem, what)) != ZERO_OK) return rc;
    return launch_early(kern, ring_grid(kern, M->n_chunks, smem, zk::kThreads8), zk::kThreads8, smem,
                        reinterpret_cast<cudaStream_t>(stream), what, t);
}

}  // namespace

extern "C" zero_status_t zero_multi_init(const int64_t* numels, int32_t n_tensors, const int32_t* group_of_tensor,
                                         int32_t n_groups, int32_t grad_dtype, int32_t param_dtype, zero_multi** out) {
    clear_error();
    const char* what = "zero_multi_init";
    if (!numels || !out) return fail(ZERO_ERR_INVALID, std::string(what) + ": NULL argument");
    if (n_tensors < 1 || n_tensors > (1 << 29))
        return fail(ZERO_ERR_INVALID, std::string(what) + ": n_tensors must be 1..2^29");
    if (n_groups < 1 || n_groups > ZERO_MAX_GROUPS)
        return fail(ZERO_ERR_INVALID, std::string(what) + ": n_groups must be 1..16");
    if (grad_dtype != ZERO_BF16 && grad_dtype != ZERO_FP16 && grad_dtype != ZERO_FP32)
        return fail(ZERO_ERR_INVALID, std::string(what) + ": unknown gradient dtype");
    if (param_dtype != ZERO_BF16 && param_dtype != ZERO_FP16 && param_dtype != ZERO_NO_OUT)
        return fail(ZERO_ERR_INVALID, std::string(what) + ": unknown parameter dtype");
    int64_t chunks = 0, total = 0;
    for (int32_t i = 0; i < n_tensors; ++i) {
        if (numels[i] < 0 || numels[i] > ((int64_t)1 << 34))
            return fail(ZERO_ERR_INVALID, std::string(what) + ": element counts must be 0..2^34");
        if (group_of_tensor && (group_of_tensor[i] < 0 || group_of_tensor[i] >= n_groups))
            return fail(ZERO_ERR_INVALID, std::string(what) + ": group out of range");
        chunks += chunks_of(numels[i], numels[i] > 0 ? zk::kVec - 1 : 0);
        total += numels[i];
        if (total > ((int64_t)1 << 41) || chunks > ((int64_t)1 << 30))  // tiles are counted in 32 bits
            return fail(ZERO_ERR_INVALID, std::string(what) + ": too many elements");
    }
    try {
        zero_multi* M = new zero_multi;
        try {
            M->numels.assign(numels, numels + n_tensors);
            if (group_of_tensor) M->groups.assign(group_of_tensor, group_of_tensor + n_tensors);
            else M->groups.assign(n_tensors, 0);
        } catch (...) {
            delete M;
            throw;
        }
        M->n_groups = n_groups;
        M->grad_dtype = grad_dtype;
        M->param_dtype = param_dtype;
        M->most_chunks = chunks;
        *out = M;
    } catch (const std::bad_alloc&) {
        return fail(ZERO_ERR_NOMEM, std::string(what) + ": out of host memory");
    }
    return ZERO_OK;
}

extern "C" zero_status_t zero_multi_query(const zero_multi* M, zero_multi_info* out) {
    clear_error();
    if (!M || !out) return fail(ZERO_ERR_INVALID, "zero_multi_query: NULL argument");
    zero_multi_info i{};
    i.n_tensors = (int32_t)M->numels.size();
    i.n_groups = M->n_groups;
    i.grad_dtype = M->grad_dtype;
    i.param_dtype = M->param_dtype;
    i.n_chunks = M->most_chunks;
    for (int64_t n : M->numels) {
        i.numel += n;
        i.state8_bytes += 2 * (n + (n + zk::kBlock8 - 1) / zk::kBlock8);
    }
    i.workspace_bytes = places(M).total;
    *out = i;
    return ZERO_OK;
}

extern "C" void zero_multi_destroy(zero_multi* M) { delete M; }

extern "C" zero_status_t zero_multi_bind(zero_multi* M, const zero_multi_arrays* x, void* workspace,
                                         zero_stream_t stream) {
    clear_error();
    const char* what = "zero_multi_bind";
    if (!M || !x) return fail(ZERO_ERR_INVALID, std::string(what) + ": NULL argument");
    zero_status_t rc;
    if ((rc = check_dev_ptr(workspace, "zero_multi_bind workspace")) != ZERO_OK) return rc;
    if ((x->m == nullptr) != (x->v == nullptr))
        return fail(ZERO_ERR_INVALID, std::string(what) + ": m and v are bound together");
    const int n8 = (x->m8 != nullptr) + (x->m8_scale != nullptr) + (x->v8 != nullptr) + (x->v8_scale != nullptr);
    if (n8 != 0 && n8 != 4)
        return fail(ZERO_ERR_INVALID, std::string(what) + ": m8, m8_scale, v8 and v8_scale are bound together");
    const int n = (int)M->numels.size();
    const uintptr_t gs = M->grad_dtype == ZERO_FP32 ? 4 : 2;
    std::vector<zk::MultiRow> rows;
    try {
        rows.resize(n);
    } catch (const std::bad_alloc&) {
        return fail(ZERO_ERR_NOMEM, std::string(what) + ": out of host memory");
    }
    int64_t chunk = 0;
    for (int i = 0; i < n; ++i) {
        zk::MultiRow& r = rows[i];
        r = zk::MultiRow{};
        r.numel = M->numels[i];
        r.group = M->groups[i];
        r.tensor = (uint32_t)i;
        r.first_chunk = (uint32_t)chunk;
        auto take = [&](const void* const* arr, uintptr_t elem, const char* name) -> uintptr_t {
            if (!arr || r.numel == 0) return 0;
            const uintptr_t p = reinterpret_cast<uintptr_t>(arr[i]);
            if (!p) rc = fail(ZERO_ERR_INVALID, std::string(what) + " " + name + ": NULL device pointer");
            else if (p % elem) rc = fail(ZERO_ERR_ALIGN, std::string(what) + " " + name + ": not aligned to its elements");
            return p;
        };
        const uintptr_t g = take(x->grads, gs, "grads"), p = take((const void* const*)x->master, 4, "master");
        const uintptr_t m = take((const void* const*)x->m, 4, "m"), v = take((const void* const*)x->v, 4, "v");
        const uintptr_t m8 = take((const void* const*)x->m8, 1, "m8"), v8 = take((const void* const*)x->v8, 1, "v8");
        const uintptr_t ms = take((const void* const*)x->m8_scale, 1, "m8_scale");
        const uintptr_t vs = take((const void* const*)x->v8_scale, 1, "v8_scale");
        const uintptr_t o = take((const void* const*)x->param16, 2, "param16");
        if (rc != ZERO_OK) return rc;
        r.grad = reinterpret_cast<const void*>(g);
        r.master = reinterpret_cast<float*>(p);
        r.m = reinterpret_cast<float*>(m);
        r.v = reinterpret_cast<float*>(v);
        r.m8 = reinterpret_cast<uint8_t*>(m8);
        r.v8 = reinterpret_cast<uint8_t*>(v8);
        r.ms = reinterpret_cast<uint8_t*>(ms);
        r.vs = reinterpret_cast<uint8_t*>(vs);
        r.out = reinterpret_cast<uint16_t*>(o);
        // Tensors of a flat buffer have the same distance to a boundary in all
        // arrays.  Where they do not, the states' sets the shift.
        r.shift = (uint8_t)(m / 4 % zk::kVec);
        r.gshift = (uint8_t)(g / gs % zk::kVec);
        auto on = [&](uintptr_t at, uintptr_t elem, uintptr_t vector) {
            return at == 0 || (at - r.shift * elem) % vector == 0;  // an array that is not there is in no one's way
        };
        r.vec = (uint8_t)((on(g, gs, gs * zk::kVec) ? zk::kVecGrad : 0) | (on(p, 4, 32) ? zk::kVecMaster : 0) |
                           (on(m, 4, 32) && on(v, 4, 32) ? zk::kVecStates : 0) | (on(o, 2, 16) ? zk::kVecOut : 0) |
                           (g % 16 == 0 && p % 32 == 0 && (m8 | v8) % 16 == 0 && (ms | vs) % 4 == 0 && o % 16 == 0 ? zk::kWhole8 : 0) |
                           ((m | v) % 32 == 0 ? zk::kCodec : 0) | ((m8 | v8) % 16 == 0 && (ms | vs) % 4 == 0 ? zk::kCodes : 0));
        chunk += chunks_of(r.numel, std::max(r.shift, r.gshift));
    }
    const bool fresh = M->workspace != static_cast<char*>(workspace);  // else a decided step may be under way
    M->bound = false;
    M->workspace = static_cast<char*>(workspace);
    M->n_chunks = chunk;
    const zk::MultiTable t = table_of(M);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    zk::MultiRow* dst = const_cast<zk::MultiRow*>(t.rows);
    uint32_t* count = const_cast<uint32_t*>(t.n_chunks);
    for (int i = 0; i < n; i += zk::kRowsPerLaunch) {
        zk::RowBatch b{};
        const int k = std::min(zk::kRowsPerLaunch, n - i);
        std::copy(rows.begin() + i, rows.begin() + i + k, b.rows);
        zk::multi_rows_kernel<<<1, zk::kRowsPerLaunch, 0, s>>>(b, dst + i, k, count, (uint32_t)chunk);
        if ((rc = after_launch(what)) != ZERO_OK) return rc;
    }
    if (chunk > 0) {
        const uint32_t ctas = (uint32_t)std::min<int64_t>((chunk + 255) / 256, 1024);
        zk::multi_map_kernel<<<ctas, 256, 0, s>>>(t.rows, t.n_tensors, const_cast<uint32_t*>(t.tensor), (uint32_t)chunk);
        if ((rc = after_launch(what)) != ZERO_OK) return rc;
    }
    zk::multi_reset_kernel<<<1, 32, 0, s>>>(t.counters, fresh ? t.grad_scale : nullptr);
    if ((rc = after_launch(what)) != ZERO_OK) return rc;
    M->grads = x->grads != nullptr;
    M->master = x->master != nullptr;
    M->states32 = x->m != nullptr;
    M->states8 = x->m8 != nullptr;
    M->param16 = x->param16 != nullptr;
    M->bound = true;
    return ZERO_OK;
}

extern "C" zero_status_t zero_multi_grad_norm(const zero_multi* M, double max_norm, zero_step_state* st,
                                              zero_stream_t stream) {
    clear_error();
    const char* what = "zero_multi_grad_norm";
    zero_status_t rc;
    if ((rc = check_bound(M, what)) != ZERO_OK) return rc;
    if (std::isnan(max_norm)) return fail(ZERO_ERR_INVALID, std::string(what) + ": max_norm is NaN");
    if (!M->grads) return missing(what, "grads");
    if ((rc = check_dev_ptr(st, "zero_multi_grad_norm state")) != ZERO_OK) return rc;
    const zk::MultiTable t = table_of(M);
    const int64_t slices = std::max<int64_t>(1, std::min<int64_t>(M->n_chunks, zk::kSlices));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto kern) {
        return launch_early(kern, persistent_grid(kern, slices), zk::kThreads, 0, s, what, t, max_norm, st);
    };
    if (M->grad_dtype == ZERO_BF16) return go(zk::multi_norm_kernel<zk::GradBf16>);
    if (M->grad_dtype == ZERO_FP16) return go(zk::multi_norm_kernel<zk::GradFp16>);
    return go(zk::multi_norm_kernel<zk::GradFp32>);
}

extern "C" zero_status_t zero_multi_adamw(const zero_multi* M, const zero_adamw_hp* hp, int32_t flags,
                                          zero_step_state* st, zero_stream_t stream) {
    clear_error();
    return update(M, hp, flags, 0, st, stream, false, "zero_multi_adamw");
}

extern "C" zero_status_t zero_multi_adamw8(const zero_multi* M, const zero_adamw_hp* hp, int32_t flags, uint32_t seed,
                                           zero_step_state* st, zero_stream_t stream) {
    clear_error();
    return update(M, hp, flags, seed, st, stream, true, "zero_multi_adamw8");
}

extern "C" zero_status_t zero_multi_encode8(const zero_multi* M, zero_stream_t stream) {
    clear_error();
    return codec(M, stream, true, "zero_multi_encode8");
}

extern "C" zero_status_t zero_multi_decode8(const zero_multi* M, zero_stream_t stream) {
    clear_error();
    return codec(M, stream, false, "zero_multi_decode8");
}

extern "C" zero_status_t zero_multi_device_error(const zero_multi* M, int32_t* bits) {
    clear_error();
    const char* what = "zero_multi_device_error";
    if (!bits) return fail(ZERO_ERR_INVALID, std::string(what) + ": NULL output");
    zero_status_t rc;
    if ((rc = check_bound(M, what)) != ZERO_OK) return rc;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(bits, &table_of(M).counters[3], sizeof *bits, cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(ZERO_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
    }
    return ZERO_OK;
}
