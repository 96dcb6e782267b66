// seqio.h — element access and gates of the sequence kernels (scan, block norms, distillation), gfx950.
//
// Rows are read and written in vectors of 16 bytes per lane at any element alignment: gfx950 takes unaligned global
// accesses, so rows whose length is no multiple of 16 bytes need no second code path. A row's last vector is moved
// back to end with the row (start min(c, D - V)); the lanes then share a few elements, which they compute alike.
#pragma once

#include "devmath.h"

namespace mdl {

struct bf16 {
    uint16_t u;
};

// V elements of T as they lie in memory, in whole registers (4, 2 or 1 words)
template <typename W, int N>
struct WordsOf {
    typedef W type __attribute__((ext_vector_type(N)));
};
template <typename W>
struct WordsOf<W, 1> {
    typedef W type;
};
template <typename T, int V>
struct Raw;
template <int V>
struct Raw<float, V> {
    typename WordsOf<float, V>::type w;
    __device__ inline void fill(float x) { w = x; }
    __device__ inline float operator[](int i) const {
        if constexpr (V == 1) return w;
        else return w[i];
    }
};
template <int V>
struct Raw<bf16, V> {
    typename WordsOf<uint32_t, (V + 1) / 2>::type w;  // element 2i in the low half of word i
    __device__ inline void fill(float x) {             // x exact in bfloat16
        const uint32_t u = __float_as_uint(x) >> 16;
        w = u | u << 16;
    }
    __device__ inline float operator[](int i) const {
        uint32_t u;
        if constexpr (V <= 2) u = w;
        else u = w[i >> 1];
        return __uint_as_float((i & 1) ? (u & 0xffff0000u) : (u << 16));
    }
};

typedef uint32_t u32x4_e __attribute__((ext_vector_type(4), aligned(2), may_alias));
typedef float f32x4_e __attribute__((ext_vector_type(4), aligned(4), may_alias));

template <int V>
__device__ inline Raw<float, V> load_raw(const float* p) {
    static_assert(V == 1 || V == 4, "16 bytes or one element");
    Raw<float, V> r;
    if constexpr (V == 4) r.w = *reinterpret_cast<const f32x4_e*>(p);
    else r.w = *p;
    return r;
}
template <int V>
__device__ inline Raw<bf16, V> load_raw(const bf16* p) {
    static_assert(V == 1 || V == 8, "16 bytes or one element");
    Raw<bf16, V> r;
    if constexpr (V == 8) r.w = *reinterpret_cast<const u32x4_e*>(p);
    else r.w = p->u;
    return r;
}

// load_raw of data that will not be read again soon
template <int V, typename T>
__device__ inline Raw<T, V> load_once(const T* p) {
    Raw<T, V> r;
    if constexpr (V == 4) r.w = __builtin_nontemporal_load(reinterpret_cast<const f32x4_e*>(p));
    else if constexpr (V == 8) r.w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(p));
    else r = load_raw<V>(p);
    return r;
}

// two fp32 values rounded to nearest even into one word of bfloat16 (v_cvt_pk_bf16_f32)
__device__ inline uint32_t pack_bf16(float lo, float hi) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const b2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// Whole vectors of an output are stored as data that is not read again here (nontemporal): they then leave the inputs in
// the caches. 4096 x 32000 distilled in bfloat16 takes 102 us this way and 119 with plain stores, a scan of 656603 x 32 in
// fp32 both ways 126 and 150, the norms of 20480 x 2048 in bfloat16 both ways 224 and 229 (each with the other in one
// session). Where rows share lines between workgroups it can lose: a scan of 206796 x 1030 in bfloat16 takes 615 us forward
// and 1377 backward, 686 and 1208 with plain stores.
template <int V>
__device__ inline void store_vec(float* p, const float (&v)[V]) {
    if constexpr (V == 4) {
        __builtin_nontemporal_store(f32x4_e{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4_e*>(p));
    } else {
        *p = v[0];
    }
}
template <int V>
__device__ inline void store_vec(bf16* p, const float (&v)[V]) {
    if constexpr (V == 8) {
        const u32x4_e q = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        __builtin_nontemporal_store(q, reinterpret_cast<u32x4_e*>(p));
    } else {
        p->u = (uint16_t)pack_bf16(v[0], 0.f);
    }
}
// V floats at p (any 4-byte alignment)
template <int V>
__device__ inline void load_f32(const float* p, float (&v)[V]) {
    if constexpr (V == 1) {
        v[0] = *p;
    } else {
        for (int i = 0; i < V; i += 4) {
            const f32x4_e q = *reinterpret_cast<const f32x4_e*>(p + i);
            for (int j = 0; j < 4; ++j) v[i + j] = q[j];
        }
    }
}
template <int V>
__device__ inline void store_f32(float* p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = v[0];
    } else {
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<f32x4_e*>(p + i) = f32x4_e{v[i], v[i + 1], v[i + 2], v[i + 3]};
    }
}

template <typename T>
struct Width;  // elements in 16 bytes
template <>
struct Width<float> {
    static constexpr int v = 4;
};
template <>
struct Width<bf16> {
    static constexpr int v = 8;
};

// e^x for x <= 0. For streams of bfloat16 the hardware exp2 of the rounded product x log2 e: its relative error of up to
// |x| 2^-24 is far below half a step of their outputs, and the fp32 states that such streams leave (last states, stepped
// states, gradients of the first ones) carry it in their gates beside the roundings of the recurrence itself. For fp32
// streams the product's rounding error is carried along (its remainder and log2 e's own low part, to first order), which
// leaves about 1.5 ulp at any x. exp2, the reciprocal of the sigmoid and the norms' reciprocal root are the hardware's,
// within 1 ulp where a division or root would be rounded.
template <typename T>
__device__ inline float exp_neg(float x) {
    constexpr float hi = 1.44269502162933349609f, lo = 1.92596299112661746887e-8f;  // log2 e in two floats
    if constexpr (sizeof(T) == 2) {
        return __builtin_amdgcn_exp2f(x * hi);
    } else {
        // x = -inf (and every x below exp2's range) gives 0: the remainder, NaN or infinite there, is not used
        const float t = x * hi;
        const float r = __builtin_fmaf(x, lo, __builtin_fmaf(x, hi, -t));
        const float e = __builtin_amdgcn_exp2f(t);
        return t < -150.f ? e : __builtin_fmaf(e * r, 0.693147180559945309f, e);
    }
}

// sigmoid(z) and 1 - sigmoid(z), each from e^-|z| without cancellation: exact 0 and 1 at infinite z
template <typename T>
__device__ inline void sigm2(float z, float& s, float& c) {
    const float e = exp_neg<T>(-fabsf(z));
    const float r = frcp(1.0f + e);
    const float q = e * r;
    s = z >= 0.f ? r : q;
    c = z >= 0.f ? q : r;
}

// Sum over each group of R neighbouring lanes (R a power of two up to 64), the same bits in every lane of the group:
// rotations inside rows of 16 lanes (v_add with a DPP operand), then exchanges between rows.
template <int CTRL>
__device__ inline float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int R>
__device__ inline float group_sum(float v) {
    constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
    if constexpr (R >= 2) v = dpp_add<kQuadXor1>(v);
    if constexpr (R >= 4) v = dpp_add<kQuadXor2>(v);
    if constexpr (R >= 8) v = dpp_add<kHalfMirror>(v);   // lane i with 7 - i: the other quad, whose sums are equal
    if constexpr (R >= 16) v = dpp_add<kMirror>(v);      // lane i with 15 - i: the other half row
    if constexpr (R >= 32) v += __shfl_xor(v, 16);
    if constexpr (R >= 64) v += __shfl_xor(v, 32);
    return v;
}
template <int CTRL>
__device__ inline float dpp_max(float v) {
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true)));
}
template <int R>
__device__ inline float group_max(float v) {
    constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;
    if constexpr (R >= 2) v = dpp_max<kQuadXor1>(v);
    if constexpr (R >= 4) v = dpp_max<kQuadXor2>(v);
    if constexpr (R >= 8) v = dpp_max<kHalfMirror>(v);
    if constexpr (R >= 16) v = dpp_max<kMirror>(v);
    if constexpr (R >= 32) v = fmaxf(v, __shfl_xor(v, 16));
    if constexpr (R >= 64) v = fmaxf(v, __shfl_xor(v, 32));
    return v;
}

// sigmoid(z) and 1 - sigmoid(z) with both of them in one register, q: the smaller one, with the sign of z
template <typename T>
__device__ inline float sigm_enc(float z, float& s, float& c) {
    const float e = exp_neg<T>(-fabsf(z));
    const float r = frcp(1.0f + e), q = e * r;
    s = z >= 0.f ? r : q;
    c = z >= 0.f ? q : r;
    return __builtin_copysignf(q, z);
}
__device__ inline void sigm_dec(float q, float& s, float& c) {
    const float t = fabsf(q), o = 1.f - t;
    const bool neg = (int)__float_as_uint(q) < 0;
    s = neg ? t : o;
    c = neg ? o : t;
}

// Register economy. forget: what was computed from these values before is computed again when it is needed after.
// settle: the value is formed here, not where it is used. one_at_a_time: the scheduler moves nothing across.
template <int N, int V>
__device__ inline void forget(float (&q)[N][V]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) asm volatile("" : "+v"(q[i][v]));
}
template <typename T, int N, int V>
__device__ inline void forget(Raw<T, V> (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(r[i].w));
}
__device__ inline float settle(float q) {
    asm volatile("" : "+v"(q));
    return q;
}
__device__ inline void one_at_a_time() { __builtin_amdgcn_sched_barrier(0); }

}  // namespace mdl
