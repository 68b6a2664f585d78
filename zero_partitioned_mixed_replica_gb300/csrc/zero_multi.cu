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
#include <vector>

#include "zero_launch.h"

namespace zk {

constexpr int kChunk = kThreads * kVec;  // elements of one work item
constexpr int kBlock8 = 32;              // elements under one scale of an 8-bit state
constexpr int kSlices = 1216;            // fixed split of a list for the norm (8 CTAs on each of 152 SMs)
constexpr int kRowsPerLaunch = 256;      // table rows passed through one launch's parameters

enum { kVecGrad = 1, kVec32 = 2, kVec8 = 4, kVecOut = 8, kVecMaster = 16 };  // MultiRow::vec

// What the kernels know of one tensor.
struct MultiRow {
    const void* grad;
    float* master;
    float* m;
    float* v;
    uint8_t* m8;
    uint8_t* ms;
    uint8_t* v8;
    uint8_t* vs;
    uint16_t* out;
    int64_t numel;
    uint32_t first_chunk;
    int32_t group;
    uint32_t vec;  // arrays that begin on a boundary for the widest access
    uint32_t pad0;
};

// The device workspace: counters, rows, chunk map, norm partials.
struct MultiTable {
    uint32_t* counters;      // [0] norm, [1] update: CTAs that are done
    const MultiRow* rows;
    const uint32_t* tensor;  // tensor of each chunk
    float2* partials;        // kSlices
    uint32_t n_chunks;
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
struct RowBatch {
    MultiRow rows[kRowsPerLaunch];
};

__global__ void multi_rows_kernel(const __grid_constant__ RowBatch b, MultiRow* rows, int n, uint32_t* counters) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n) rows[i] = b.rows[i];
    if (i < 2 && counters) counters[i] = 0;
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

// ----------------------------------------------------------------------------
// Loads and stores of up to 8 consecutive elements: nv of them exist; `vec`:
// the array begins on a boundary for the wide access.
// ----------------------------------------------------------------------------
struct GradBf16 {
    using T = uint16_t;
    static __device__ __forceinline__ float one(uint16_t h) { return Bf16::dec1(h); }
    static __device__ __forceinline__ void eight(const uint16_t* p, float (&o)[8]) { unpack8<Bf16>(ld_stream(p), o); }
};
struct GradFp16 {
    using T = uint16_t;
    static __device__ __forceinline__ float one(uint16_t h) { return Fp16::dec1(h); }
    static __device__ __forceinline__ void eight(const uint16_t* p, float (&o)[8]) { unpack8<Fp16>(ld_stream(p), o); }
};
struct GradFp32 {
    using T = float;
    static __device__ __forceinline__ float one(float x) { return x; }
    static __device__ __forceinline__ void eight(const float* p, float (&o)[8]) { ld8(p, o); }
};
struct NoOut {
    static constexpr bool kOut = false;
    static __device__ __forceinline__ uint16_t enc1(float) { return 0; }
    static __device__ __forceinline__ uint32_t pack(float, float) { return 0; }
};
struct OutBf16 : Bf16 {
    static constexpr bool kOut = true;
};
struct OutFp16 : Fp16 {
    static constexpr bool kOut = true;
};

template <class G>
__device__ __forceinline__ void load_grad(const void* base, int64_t i, int nv, bool vec, float (&o)[8]) {
    const typename G::T* p = static_cast<const typename G::T*>(base) + i;
    if (vec && nv == 8) {
        G::eight(p, o);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = e < nv ? G::one(p[e]) : 0.0f;
    }
}
__device__ __forceinline__ void load_f32(const float* p, int nv, bool vec, float (&o)[8]) {
    if (vec && nv == 8) {
        ld8(p, o);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = e < nv ? p[e] : 0.0f;
    }
}
__device__ __forceinline__ void store_f32(float* p, int nv, bool vec, const float (&o)[8]) {
    if (vec && nv == 8) {
        st8(p, o);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < nv) p[e] = o[e];
    }
}
template <class O>
__device__ __forceinline__ void store_out(uint16_t* p, int nv, bool vec, const float (&o)[8]) {
    if constexpr (O::kOut) {
        if (vec && nv == 8) {
            st_stream(p, pack8<O>(o));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < nv) p[e] = O::enc1(o[e]);
        }
    }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int nv, bool vec) {
    if (vec && nv == 8) return __ldcs(reinterpret_cast<const uint2*>(p));
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < nv) w[e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t* p, int nv, bool vec, uint2 c) {
    if (vec && nv == 8) {
        __stcs(reinterpret_cast<uint2*>(p), c);
    } else {
        const uint32_t w[2] = {c.x, c.y};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < nv) p[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
}

// ----------------------------------------------------------------------------
// 8-bit states: E4M3 (m) and E5M2 (v) codes under one power of two per 32
// elements, which 4 neighbouring lanes hold, 8 elements each.
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

template <class Q>
__device__ __forceinline__ void decode8(uint2 c, float scale, float (&o)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 f = Q::dec2((uint16_t)(w[k >> 1] >> (16 * (k & 1))));
        o[2 * k] = __fmul_rn(f.x, scale);
        o[2 * k + 1] = __fmul_rn(f.y, scale);
    }
}

// Scale byte of the block that this lane's 8 values belong to (its 4 lanes get
// the same); values behind the tensor's end are zero.  All lanes call it.
template <class Q>
__device__ __forceinline__ uint32_t block_scale(const float (&x)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    if (top >= 0x7F800000u) return 255u;
    // one more when the mantissa is above 1.75; in binary32's last binade there
    // is no more, and what is above 1.75 * 2^127 saturates
    const int e = (int)min((top + 0x1FFFFFu) >> 23, 254u);
    return (uint32_t)max(1, e - Q::kTop);
}

// Codes of 8 values; rnd: random integers below 2^kCut (stochastic), or null
// (nearest).
template <class Q, bool STOCHASTIC>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], uint32_t byte, const uint32_t (&rnd)[8]) {
    if (byte == 255u) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);  // NaN in both types
    const float inv = __uint_as_float((254u - byte) << 23);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float z = __fmul_rn(x[e], inv);
        y[e] = z;
        if constexpr (STOCHASTIC) y[e] = __uint_as_float((__float_as_uint(z) + rnd[e]) & ~((1u << Q::kCut) - 1u));
        if constexpr (Q::kFloor)
            if (z > 0.0f) y[e] = fmaxf(y[e], kSmallestE5m2);
    }
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = Q::enc2(y[2 * k], y[2 * k + 1]);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
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
struct MultiShared {
    AdamConsts k[ZERO_MAX_GROUPS];
    float isb[ZERO_MAX_GROUPS];  // 1 / sqrt(1 - beta2^t)
    float unscale;               // 1 / loss scale the gradients carry
    uint32_t key;                // of the step's random numbers
    int32_t apply;
};

__device__ __forceinline__ void multi_constants(const MultiArgs& a, MultiShared& s) {
    const zero_step_state* st = a.st;
    const bool advance = (a.flags & ZERO_MULTI_ADVANCE) != 0;
    const int g = threadIdx.x;
    if (g < a.hp.n) {
        const double b1p = advance ? __dmul_rn(st->beta1_pow, st->beta1) : st->beta1_pow;
        const double b2p = advance ? __dmul_rn(st->beta2_pow, st->beta2) : st->beta2_pow;
        s.k[g] = make_consts(st->beta1, st->beta2, b1p, b2p, a.hp.lr[g], a.hp.eps[g], a.hp.wd[g],
                             advance ? 1.0f : st->clip_coef);
        s.isb[g] = __double2float_rn(__ddiv_rn(1.0, __dsqrt_rn(__dsub_rn(1.0, b2p))));
    }
    if (g == 0) {
        s.apply = advance ? 1 : st->apply;
        const float scale = !advance && st->grad_scale > 0.0f ? st->grad_scale : st->loss_scale;
        s.unscale = (a.flags & ZERO_MULTI_UNSCALED) ? 1.0f : __fdiv_rn(1.0f, scale);
        s.key = mix32(a.seed ^ mix32((uint32_t)(st->t + (advance ? 1 : 0))));
    }
    __syncthreads();
}

// ZERO_MULTI_ADVANCE: the CTA that ends last moves the step on; every CTA has
// read the state by then.
__device__ __forceinline__ void multi_advance(const MultiArgs& a) {
    if (!(a.flags & ZERO_MULTI_ADVANCE)) return;
    if (threadIdx.x != 0) return;
    __threadfence();
    if (atomicInc(&a.t.counters[1], gridDim.x - 1) != gridDim.x - 1) return;
    zero_step_state* st = a.st;
    st->clip_coef = 1.0f;
    st->apply = 1;
    st->t += 1;
    st->beta1_pow = __dmul_rn(st->beta1_pow, st->beta1);
    st->beta2_pow = __dmul_rn(st->beta2_pow, st->beta2);
    st->good_steps += 1;
}

// This thread's 8 elements of chunk c.
__device__ __forceinline__ int multi_place(const MultiTable& t, uint32_t c, const MultiRow& r, int64_t& i) {
    i = (int64_t)(c - r.first_chunk) * kChunk + threadIdx.x * kVec;
    const int64_t left = r.numel - i;
    int nv = left >= kVec ? kVec : (left > 0 ? (int)left : 0);
    const uint64_t lim = (uint64_t)r.numel > t.slack ? (uint64_t)r.numel - t.slack : 0;
    if (nv > 0 && !in_bounds((uint64_t)i + nv, lim)) nv = 0;
    return nv;
}

// ----------------------------------------------------------------------------
// AdamW, 32-bit states
// ----------------------------------------------------------------------------
template <class G, class O>
__global__ void __launch_bounds__(kThreads, 4) multi_adamw_kernel(const __grid_constant__ MultiArgs a) {
    __shared__ MultiShared s;
    multi_constants(a, s);
    if (s.apply) {
        const float unscale = s.unscale;
        for (uint32_t c = blockIdx.x; c < a.t.n_chunks; c += gridDim.x) {
            const MultiRow& r = a.t.rows[a.t.tensor[c]];
            int64_t i;
            const int nv = multi_place(a.t, c, r, i);
            if (nv == 0) continue;
            const uint32_t vec = r.vec;
            const AdamConsts k = s.k[r.group];
            float g[8], p[8], m[8], v[8];
            load_grad<G>(r.grad, i, nv, vec & kVecGrad, g);
            load_f32(r.master + i, nv, vec & kVecMaster, p);
            load_f32(r.m + i, nv, vec & kVec32, m);
            load_f32(r.v + i, nv, vec & kVec32, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = __fmul_rn(g[e], unscale);
            if (all_zero8x3(g, m, v)) {  // e.g. embedding rows that no batch has held
#pragma unroll
                for (int e = 0; e < 8; ++e) adamw1_zero_state(p[e], m[e], v[e], g[e], k);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) adamw1(p[e], m[e], v[e], g[e], k);
            }
            store_f32(r.master + i, nv, vec & kVecMaster, p);
            store_f32(r.m + i, nv, vec & kVec32, m);
            store_f32(r.v + i, nv, vec & kVec32, v);
            if constexpr (O::kOut) store_out<O>(r.out + i, nv, vec & kVecOut, p);
        }
    }
    multi_advance(a);
}

// ----------------------------------------------------------------------------
// AdamW, 8-bit states
// ----------------------------------------------------------------------------
__device__ __forceinline__ float sqrt_approx(float x) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <class G, class O>
__global__ void __launch_bounds__(kThreads, 4) multi_adamw8_kernel(const __grid_constant__ MultiArgs a) {
    __shared__ MultiShared s;
    multi_constants(a, s);
    if (s.apply) {
        const float unscale = s.unscale;
        for (uint32_t c = blockIdx.x; c < a.t.n_chunks; c += gridDim.x) {
            const uint32_t n = a.t.tensor[c];
            const MultiRow& r = a.t.rows[n];
            int64_t i;
            const int nv = multi_place(a.t, c, r, i);
            if (!__any_sync(0xFFFFFFFFu, nv > 0)) continue;
            const uint32_t vec = r.vec;
            const AdamConsts k = s.k[r.group];
            const float isb = s.isb[r.group];
            float g[8], p[8], m[8], v[8];
            load_grad<G>(r.grad, i, nv, vec & kVecGrad, g);
            load_f32(r.master + i, nv, vec & kVecMaster, p);
            const int64_t blk = i / kBlock8;
            float sm = 0.0f, sv = 0.0f;
            if (nv > 0) {
                sm = scale_of(r.ms[blk]);
                sv = scale_of(r.vs[blk]);
            }
            decode8<E4m3>(load_codes(r.m8 + i, nv, vec & kVec8), sm, m);
            decode8<E5m2>(load_codes(r.v8 + i, nv, vec & kVec8), sv, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float gc = __fmul_rn(__fmul_rn(g[e], unscale), k.clip);
                m[e] = __fadd_rn(__fmul_rn(k.b1, m[e]), __fmul_rn(k.omb1, gc));
                v[e] = __fadd_rn(__fmul_rn(k.b2, v[e]), __fmul_rn(k.omb2, __fmul_rn(gc, gc)));
                const float den = __fmaf_rn(sqrt_approx(v[e]), isb, k.eps);
                p[e] = __fsub_rn(__fmul_rn(p[e], k.decay), __fmul_rn(k.step_size, __fdividef(m[e], den)));
            }
            store_f32(r.master + i, nv, vec & kVecMaster, p);
            if constexpr (O::kOut) store_out<O>(r.out + i, nv, vec & kVecOut, p);
            uint32_t x = mix32(mix32(s.key + n) + 0x9E3779B1u * (uint32_t)(i >> 3));
            uint32_t rm[8], rv[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x = x * 1664525u + 1013904223u;
                rm[e] = x >> 12;
                x = x * 1664525u + 1013904223u;
                rv[e] = x >> 11;
            }
            const uint32_t bm = block_scale<E4m3>(m), bv = block_scale<E5m2>(v);
            if (nv > 0) {
                store_codes(r.m8 + i, nv, vec & kVec8, encode8<E4m3, true>(m, bm, rm));
                store_codes(r.v8 + i, nv, vec & kVec8, encode8<E5m2, true>(v, bv, rv));
                if ((threadIdx.x & 3) == 0) {
                    r.ms[blk] = (uint8_t)bm;
                    r.vs[blk] = (uint8_t)bv;
                }
            }
        }
    }
    multi_advance(a);
}

// ----------------------------------------------------------------------------
// 32-bit states into the 8-bit form and back
// ----------------------------------------------------------------------------
template <bool ENCODE>
__global__ void __launch_bounds__(kThreads) multi_codec_kernel(const __grid_constant__ MultiTable t) {
    for (uint32_t c = blockIdx.x; c < t.n_chunks; c += gridDim.x) {
        const MultiRow& r = t.rows[t.tensor[c]];
        int64_t i;
        const int nv = multi_place(t, c, r, i);
        if (!__any_sync(0xFFFFFFFFu, nv > 0)) continue;
        const uint32_t vec = r.vec;
        const int64_t blk = i / kBlock8;
        float m[8], v[8];
        if constexpr (ENCODE) {
            const uint32_t none[8] = {};
            load_f32(r.m + i, nv, vec & kVec32, m);
            load_f32(r.v + i, nv, vec & kVec32, v);
            const uint32_t bm = block_scale<E4m3>(m), bv = block_scale<E5m2>(v);
            if (nv > 0) {
                store_codes(r.m8 + i, nv, vec & kVec8, encode8<E4m3, false>(m, bm, none));
                store_codes(r.v8 + i, nv, vec & kVec8, encode8<E5m2, false>(v, bv, none));
                if ((threadIdx.x & 3) == 0) {
                    r.ms[blk] = (uint8_t)bm;
                    r.vs[blk] = (uint8_t)bv;
                }
            }
        } else if (nv > 0) {
            decode8<E4m3>(load_codes(r.m8 + i, nv, vec & kVec8), scale_of(r.ms[blk]), m);
            decode8<E5m2>(load_codes(r.v8 + i, nv, vec & kVec8), scale_of(r.vs[blk]), v);
            store_f32(r.m + i, nv, vec & kVec32, m);
            store_f32(r.v + i, nv, vec & kVec32, v);
        }
    }
}

// ----------------------------------------------------------------------------
// Global norm and step decision
// ----------------------------------------------------------------------------
template <class G>
__global__ void __launch_bounds__(kThreads) multi_norm_kernel(const __grid_constant__ MultiTable t, double max_norm,
                                                              zero_step_state* st, uint32_t n_slices) {
    __shared__ double sh[kThreads];
    __shared__ bool last;
    for (uint32_t sl = blockIdx.x; sl < n_slices; sl += gridDim.x) {
        // the slice's chunks, tensor by tensor
        const uint32_t c1 = (uint32_t)((uint64_t)(sl + 1) * t.n_chunks / n_slices);
        uint32_t c = (uint32_t)((uint64_t)sl * t.n_chunks / n_slices);
        float hi = 0.0f, lo = 0.0f;
        while (c < c1) {
            const uint32_t n = t.tensor[c];
            const MultiRow& r = t.rows[n];
            const int64_t begin = (int64_t)(c - r.first_chunk) * kChunk;
            const uint32_t chunks = (uint32_t)((r.numel + kChunk - 1) / kChunk) - (c - r.first_chunk);
            const uint32_t take = min(chunks, c1 - c);
            const int64_t end = min(r.numel, begin + (int64_t)take * kChunk);
            const bool vec = r.vec & kVecGrad;
            const uint64_t lim = (uint64_t)r.numel > t.slack ? (uint64_t)r.numel - t.slack : 0;
            for (int64_t i = begin + threadIdx.x * kVec; i < end; i += kChunk) {
                const int nv = end - i >= kVec ? kVec : (int)(end - i);
                if (!in_bounds((uint64_t)i + nv, lim)) continue;
                float g[8];
                load_grad<G>(r.grad, i, nv, vec, g);
                float q = __fmul_rn(g[0], g[0]);
#pragma unroll
                for (int e = 1; e < 8; ++e) q = __fmaf_rn(g[e], g[e], q);
                float sum, err;
                two_sum(hi, q, sum, err);
                hi = sum;
                lo = __fadd_rn(lo, err);
            }
            c += take;
        }
        __syncthreads();  // sh: the slice before
        sh[threadIdx.x] = __dadd_rn((double)hi, (double)lo);
        __syncthreads();
        for (int w = kThreads / 2; w > 0; w >>= 1) {
            if ((int)threadIdx.x < w) sh[threadIdx.x] = __dadd_rn(sh[threadIdx.x], sh[threadIdx.x + w]);
            __syncthreads();
        }
        if (threadIdx.x == 0) {
            const float h = __double2float_rn(sh[0]);
            t.partials[sl] = make_float2(h, __double2float_rn(__dsub_rn(sh[0], (double)h)));
        }
    }
    if (threadIdx.x == 0) {
        __threadfence();
        last = atomicInc(&t.counters[0], gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double sum = 0.0;
    for (uint32_t sl = threadIdx.x; sl < n_slices; sl += kThreads) {
        const float2 q = __ldcg(&t.partials[sl]);
        sum = __dadd_rn(sum, __dadd_rn((double)q.x, (double)q.y));
    }
    __syncthreads();
    sh[threadIdx.x] = sum;
    __syncthreads();
    for (int w = kThreads / 2; w > 0; w >>= 1) {
        if ((int)threadIdx.x < w) sh[threadIdx.x] = __dadd_rn(sh[threadIdx.x], sh[threadIdx.x + w]);
        __syncthreads();
    }
    if (threadIdx.x != 0) return;
    const bool bad = !isfinite(sh[0]);  // an inf or NaN gradient, or a square beyond binary32
    const float scale = st->loss_scale;
    const double norm = bad ? (double)INFINITY : __ddiv_rn(__dsqrt_rn(sh[0]), (double)scale);
    st->nonfinite = 0;
    st->overflow = bad;
    st->grad_norm = norm;
    st->grad_scale = scale;
    decide_step(st, bad, norm, max_norm);
}

}  // namespace zk

using namespace zero_detail;

struct zero_multi {
    std::vector<int64_t> numels;
    std::vector<int32_t> groups;
    int32_t n_groups = 0, grad_dtype = 0, param_dtype = 0;
    int64_t n_chunks = 0;
    // the last bind
    bool bound = false, grads = false, master = false, states32 = false, states8 = false, param16 = false;
    char* workspace = nullptr;
};

namespace {

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

// Workspace layout: counters (256 bytes), rows, chunk map, norm partials.
struct Places {
    int64_t rows, map, partials, total;
};
Places places(const zero_multi* M) {
    Places p;
    p.rows = 256;
    p.map = p.rows + up256((int64_t)M->numels.size() * (int64_t)sizeof(zk::MultiRow));
    p.partials = p.map + up256(M->n_chunks * (int64_t)sizeof(uint32_t));
    p.total = p.partials + up256(zk::kSlices * (int64_t)sizeof(float2));
    return p;
}

zk::MultiTable table_of(const zero_multi* M) {
    const Places p = places(M);
    zk::MultiTable t{};
    t.counters = reinterpret_cast<uint32_t*>(M->workspace);
    t.rows = reinterpret_cast<const zk::MultiRow*>(M->workspace + p.rows);
    t.tensor = reinterpret_cast<const uint32_t*>(M->workspace + p.map);
    t.partials = reinterpret_cast<float2*>(M->workspace + p.partials);
    t.n_chunks = (uint32_t)M->n_chunks;
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

template <class G, class O>
zero_status_t launch_update(bool eight, const zk::MultiArgs& a, cudaStream_t s) {
    const int64_t work = a.t.n_chunks;
    if (eight) {
        auto kern = zk::multi_adamw8_kernel<G, O>;
        kern<<<persistent_grid(kern, work), zk::kThreads, 0, s>>>(a);
        return after_launch("zero_multi_adamw8");
    }
    auto kern = zk::multi_adamw_kernel<G, O>;
    kern<<<persistent_grid(kern, work), zk::kThreads, 0, s>>>(a);
    return after_launch("zero_multi_adamw");
}

template <class G>
zero_status_t launch_update_out(bool eight, int32_t param_dtype, const zk::MultiArgs& a, cudaStream_t s) {
    if (param_dtype == ZERO_BF16) return launch_update<G, zk::OutBf16>(eight, a, s);
    if (param_dtype == ZERO_FP16) return launch_update<G, zk::OutFp16>(eight, a, s);
    return launch_update<G, zk::NoOut>(eight, a, s);
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
    if (M->grad_dtype == ZERO_BF16) return launch_update_out<zk::GradBf16>(eight, M->param_dtype, a, s);
    if (M->grad_dtype == ZERO_FP16) return launch_update_out<zk::GradFp16>(eight, M->param_dtype, a, s);
    return launch_update_out<zk::GradFp32>(eight, M->param_dtype, a, s);
}

zero_status_t codec(const zero_multi* M, zero_stream_t stream, bool encode, const char* what) {
    zero_status_t rc;
    if ((rc = check_bound(M, what)) != ZERO_OK) return rc;
    if (!M->states32) return missing(what, "32-bit states");
    if (!M->states8) return missing(what, "8-bit states");
    if (M->n_chunks == 0) return ZERO_OK;
    const zk::MultiTable t = table_of(M);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (encode) {
        auto kern = zk::multi_codec_kernel<true>;
        kern<<<persistent_grid(kern, t.n_chunks), zk::kThreads, 0, s>>>(t);
    } else {
        auto kern = zk::multi_codec_kernel<false>;
        kern<<<persistent_grid(kern, t.n_chunks), zk::kThreads, 0, s>>>(t);
    }
    return after_launch(what);
}

}  // namespace

extern "C" zero_status_t zero_multi_init(const int64_t* numels, int32_t n_tensors, const int32_t* group_of_tensor,
                                         int32_t n_groups, int32_t grad_dtype, int32_t param_dtype, zero_multi** out) {
    clear_error();
    const char* what = "zero_multi_init";
    if (!numels || !out) return fail(ZERO_ERR_INVALID, std::string(what) + ": NULL argument");
    if (n_tensors < 1) return fail(ZERO_ERR_INVALID, std::string(what) + ": need at least one tensor");
    if (n_groups < 1 || n_groups > ZERO_MAX_GROUPS)
        return fail(ZERO_ERR_INVALID, std::string(what) + ": n_groups must be 1..16");
    if (grad_dtype != ZERO_BF16 && grad_dtype != ZERO_FP16 && grad_dtype != ZERO_FP32)
        return fail(ZERO_ERR_INVALID, std::string(what) + ": unknown gradient dtype");
    if (param_dtype != ZERO_BF16 && param_dtype != ZERO_FP16 && param_dtype != ZERO_NO_OUT)
        return fail(ZERO_ERR_INVALID, std::string(what) + ": unknown parameter dtype");
    int64_t chunks = 0;
    for (int32_t i = 0; i < n_tensors; ++i) {
        if (numels[i] < 0 || numels[i] > ((int64_t)1 << 34))
            return fail(ZERO_ERR_INVALID, std::string(what) + ": element counts must be 0..2^34");
        if (group_of_tensor && (group_of_tensor[i] < 0 || group_of_tensor[i] >= n_groups))
            return fail(ZERO_ERR_INVALID, std::string(what) + ": group out of range");
        chunks += (numels[i] + zk::kChunk - 1) / zk::kChunk;
        if (chunks > ((int64_t)1 << 30)) return fail(ZERO_ERR_INVALID, std::string(what) + ": too many elements");
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
        M->n_chunks = chunks;
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
    i.n_chunks = M->n_chunks;
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
    uint32_t chunk = 0;
    for (int i = 0; i < n; ++i) {
        zk::MultiRow& r = rows[i];
        r = zk::MultiRow{};
        r.numel = M->numels[i];
        r.group = M->groups[i];
        r.first_chunk = chunk;
        chunk += (uint32_t)((r.numel + zk::kChunk - 1) / zk::kChunk);
        // address of tensor i in one array; `wide`: every array so far begins on a boundary for the wide access
        auto take = [&](const void* const* arr, uintptr_t elem, uintptr_t vector, const char* name, bool& wide) -> const void* {
            if (!arr) return nullptr;
            const uintptr_t p = reinterpret_cast<uintptr_t>(arr[i]);
            if (r.numel > 0 && !p) rc = fail(ZERO_ERR_INVALID, std::string(what) + " " + name + ": NULL device pointer");
            else if (r.numel > 0 && p % elem)
                rc = fail(ZERO_ERR_ALIGN, std::string(what) + " " + name + ": not aligned to its elements");
            if (p % vector) wide = false;
            return arr[i];
        };
        bool wg = true, wp = true, w32 = true, w8 = true, wo = true, any = true;
        r.grad = take(x->grads, gs, gs * 8, "grads", wg);
        r.master = (float*)take((const void* const*)x->master, 4, 32, "master", wp);
        r.m = (float*)take((const void* const*)x->m, 4, 32, "m", w32);
        r.v = (float*)take((const void* const*)x->v, 4, 32, "v", w32);
        r.m8 = (uint8_t*)take((const void* const*)x->m8, 1, 8, "m8", w8);
        r.v8 = (uint8_t*)take((const void* const*)x->v8, 1, 8, "v8", w8);
        r.ms = (uint8_t*)take((const void* const*)x->m8_scale, 1, 1, "m8_scale", any);
        r.vs = (uint8_t*)take((const void* const*)x->v8_scale, 1, 1, "v8_scale", any);
        r.out = (uint16_t*)take((const void* const*)x->param16, 2, 16, "param16", wo);
        if (rc != ZERO_OK) return rc;
        r.vec = (wg ? zk::kVecGrad : 0) | (wp ? zk::kVecMaster : 0) | (w32 ? zk::kVec32 : 0) | (w8 ? zk::kVec8 : 0) |
                (wo ? zk::kVecOut : 0);
    }
    M->bound = false;
    M->workspace = static_cast<char*>(workspace);
    const zk::MultiTable t = table_of(M);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    zk::MultiRow* dst = const_cast<zk::MultiRow*>(t.rows);
    for (int i = 0; i < n; i += zk::kRowsPerLaunch) {
        zk::RowBatch b{};
        const int k = std::min(zk::kRowsPerLaunch, n - i);
        std::copy(rows.begin() + i, rows.begin() + i + k, b.rows);
        zk::multi_rows_kernel<<<1, zk::kRowsPerLaunch, 0, s>>>(b, dst + i, k, i == 0 ? t.counters : nullptr);
        if ((rc = after_launch(what)) != ZERO_OK) return rc;
    }
    if (t.n_chunks > 0) {
        const uint32_t ctas = std::min<uint32_t>((t.n_chunks + 255) / 256, 1024);
        zk::multi_map_kernel<<<ctas, 256, 0, s>>>(t.rows, t.n_tensors, const_cast<uint32_t*>(t.tensor), t.n_chunks);
        if ((rc = after_launch(what)) != ZERO_OK) return rc;
    }
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
    const uint32_t slices = std::max<uint32_t>(1, std::min<uint32_t>(t.n_chunks, zk::kSlices));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto kern) {
        kern<<<persistent_grid(kern, slices), zk::kThreads, 0, s>>>(t, max_norm, st, slices);
        return after_launch(what);
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
