// k_distill.hip — distillation from a teacher's top logits: loss and gradient per frame in one pass.
//
// With the teacher's k kept classes id_j and logits t_j, the student's logits z over V classes and a temperature tau:
//   p = softmax_j(t / tau),  q = softmax(z / tau)
//   loss = w tau^2 sum_j p_j (ln p_j - ln q_{id_j}),  dz = w tau (q - sum_j p_j [id_j = .])
// Written with e_j = exp((t_j - max t) / tau), T = sum e, m = max z and L = sum exp((z - m) / tau):
//   loss / (w tau) = (1/T) sum_j e_j ((t_j - max t) - (z_{id_j} - m)) + tau (ln L - ln T),
// in which neither tau^2 nor 1 / tau can leave the range of fp32 before the loss does.
//
// R lanes share a row. A row that fits their registers is read once, kept as it lies in memory, and its gradient is
// formed from there; longer rows are read twice. The maximum and the sum run along with the reading. The few kept classes sit
// in LDS; their gradients are written over the row's after it, by the lanes that own the slots (a class named twice gets
// both slots' p). Statistics are fp32; the gradient is rounded once.
//
// Bound by HBM: 4096 x 32000 in bfloat16 takes 98 us (525 MB, 5.4 TB/s; a copy runs at 4.93), 1000 x 100003 in fp32
// 186 us (800 MB, 4.3 TB/s; 192 if it is read twice), 60000 x 80 in fp32 13 us (38 MB). Each kept class is compared with
// all of them, so that many of them on a short row are bound by that: 50000 x 256 in fp32 takes 23 us with 8 kept classes,
// 71 with 64 and 967 with 256 (102 MB).
#include "kernels.h"
#include "seqio.h"

#include <algorithm>

namespace mdl {

namespace {

constexpr float kLn2 = 0.693147180559945309f;

template <int V_, int R_, int NV_>
struct DistillShape {  // elements a vector, lanes a row, vectors a lane (0: the row is read twice)
    static constexpr int V = V_, R = R_, NV = NV_;
    static constexpr int threads = R_ > 256 ? R_ : 256;
    static constexpr int rows = threads / R_;
};

template <int R>
__device__ inline void row_sync() {
    if constexpr (R > 64) {
        __syncthreads();
    } else {  // the lanes of one wave: order their LDS and global accesses
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    }
}
// maxima (MAX) or sums of K values over a row's lanes, the same in all of them
template <int R, int K, bool MAX>
__device__ inline void row_reduce(float (&s)[K], float* red) {
    constexpr int W = R < 64 ? R : 64;
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = MAX ? group_max<W>(s[k]) : group_sum<W>(s[k]);
    if constexpr (R > 64) {
        const int wave = threadIdx.x >> 6, w0 = threadIdx.x / R * (R / 64);  // the row's first wave
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
            for (int k = 0; k < K; ++k) red[wave * K + k] = s[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            s[k] = red[w0 * K + k];
#pragma unroll 2
            for (int w = w0 + 1; w < w0 + R / 64; ++w) s[k] = MAX ? fmaxf(s[k], red[w * K + k]) : s[k] + red[w * K + k];
        }
    }
}

// element 0 of a vector
template <int V>
__device__ inline void set_first(Raw<float, V>& r, const Raw<float, 1>& x) {
    if constexpr (V == 1) r.w = x.w;
    else r.w[0] = x.w;
}
template <int V>
__device__ inline void set_first(Raw<bf16, V>& r, const Raw<bf16, 1>& x) {
    if constexpr (V == 1) r.w = x.w;
    else r.w[0] = (r.w[0] & 0xffff0000u) | x.w;
}
// the first n elements set to -inf
template <int V>
__device__ inline void hide(Raw<float, V>& r, int n) {
    if constexpr (V == 1) {
        if (n > 0) r.w = -INFINITY;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) r.w[v] = v < n ? -INFINITY : r.w[v];
    }
}
template <int V>
__device__ inline void hide(Raw<bf16, V>& r, int n) {
    if constexpr (V == 1) {
        if (n > 0) r.w = 0xff80u;
    } else {
#pragma unroll
        for (int v = 0; v < V; v += 2) {
            uint32_t w = r.w[v / 2];
            if (v < n) w = (w & 0xffff0000u) | 0xff80u;
            if (v + 1 < n) w = (w & 0xffffu) | 0xff800000u;
            r.w[v / 2] = w;
        }
    }
}
template <int V>
__device__ inline void store_zeros(float* p) {
    const float o[V] = {};
    store_vec<V>(p, o);
}
template <int V>
__device__ inline void store_zeros(bf16* p) {
    const float o[V] = {};
    store_vec<V>(p, o);
}

// a copy that the compiler takes for another value: places formed from it are not kept in registers for later walks
__device__ inline int anew(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

struct DistillArgs {
    int64_t N;
    int V, k;
    const void* z;
    int64_t ldz;
    const int32_t* ids;
    const void* t;
    int t_bf16;
    const float* w;
    float tau, log2e_tau;
    float* loss;
    void* dz;
    int64_t ldd;
};

// exp(d / tau) for d <= 0 (NaN where the row's maximum is not finite), from the product with log2 e / tau: with the
// rounding of d, the argument is off by 3 |d / tau| 2^-24, no more than by way of d / tau
__device__ inline float exp_tau(float d, const DistillArgs& a) { return __builtin_amdgcn_exp2f(d * a.log2e_tau); }

template <typename T, typename S>
__global__ __launch_bounds__(S::threads, 4) void k_distill(DistillArgs a) {
    constexpr int V = S::V, R = S::R, NV = S::NV > 0 ? S::NV : 1;
    constexpr bool kTwice = S::NV == 0;
    static_assert(R >= V, "the elements past a row's whole vectors: one a lane");
    constexpr int kAhead = S::NV == 0 || NV % 4 == 0 ? 4 : NV % 2 == 0 ? 2 : 1;  // vectors walked at a time
    __shared__ float red[S::threads / 64 * 5];
    extern __shared__ float top[];  // [rows][3][k]: class, e_j, z of the class
    const int lane = threadIdx.x % R, group = threadIdx.x / R;
    const int64_t row = (int64_t)blockIdx.x * S::rows + group;
    const bool live = row < a.N;
    const int64_t n = live ? row : a.N - 1;
    const T* z = static_cast<const T*>(a.z) + n * a.ldz;
    int* const cls = reinterpret_cast<int*>(top + (size_t)group * 3 * a.k);
    float* const ej = top + (size_t)group * 3 * a.k + a.k;
    float* const zj = ej + a.k;

    // the row: each lane's running maximum and sum, some vectors at a time, as they arrive
    Raw<T, V> q[NV];
    const int full = a.V / V, tail = full * V, rest = a.V - tail;
    float mx = -INFINITY, run = 0.f;
    auto take = [&](const Raw<T, V>* r) {
        float b = mx, p = 0.f;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) b = fmaxf(b, r[i][v]);
        if (b > mx) run *= exp_tau(mx - b, a);
        mx = b;
        const float c = b == -INFINITY ? 0.f : b;  // nothing but -inf so far: exp(-inf) = 0
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) p += exp_tau(r[i][v] - c, a);
        run += p;
    };
    if constexpr (!kTwice) {
        // a vector past the row's end is moved back to end with it: what it repeats is hidden from the sums
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            one_at_a_time();
            if (i / kAhead * kAhead * R * V < a.V) q[i] = load_raw<V>(z + min((lane + i * R) * V, a.V - V));
        }
#pragma unroll
        for (int i = 0; i < NV; i += kAhead) {
            if (i * R * V >= a.V) continue;  // none of the row's lanes has a part in these
            one_at_a_time();
            const int at = anew(lane);
#pragma unroll
            for (int j = i; j < i + kAhead; ++j)
                if (const int skip = (at + j * R) * V - (a.V - V); skip > 0) hide(q[j], skip);
            take(q + i);
        }
        mx = settle(mx);
        run = settle(run);
        forget(q);
    } else {
        int i = lane;
        for (; i + (kAhead - 1) * R < full; i += kAhead * R) {
            Raw<T, V> r[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) r[j] = load_raw<V>(z + (int64_t)(i + j * R) * V);
            take(r);
        }
        for (; i < full; i += R) {
            Raw<T, V> r[kAhead];
            r[0] = load_raw<V>(z + (int64_t)i * V);
#pragma unroll
            for (int j = 1; j < kAhead; ++j) r[j].fill(-INFINITY);
            take(r);
        }
        if (lane < rest) {
            Raw<T, V> r[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) r[j].fill(-INFINITY);
            set_first(r[0], load_raw<1>(z + tail + lane));
            take(r);
        }
    }
    // the kept classes
    float m2[2] = {mx, -INFINITY};
    float kept = 0.f, bad = 0.f;
    for (int j = lane; j < a.k; j += R) {
        int c = a.ids[n * a.k + j];
        const float t = a.t_bf16 ? load_raw<1>(static_cast<const bf16*>(a.t) + n * a.k + j)[0]
                                 : static_cast<const float*>(a.t)[n * a.k + j];
        const bool ok = c >= 0 && c < a.V;
        kept += ok ? 1.f : 0.f;
        bad += !ok && c != -1 ? 1.f : 0.f;
        cls[j] = ok ? c : -1;
        ej[j] = t;
        zj[j] = ok ? load_raw<1>(z + c)[0] : 0.f;
        if (ok) m2[1] = fmaxf(m2[1], t);
    }
    row_reduce<R, 2, true>(m2, red);
    const float m = m2[0], tm = m2[1];
    // L, T, sum e_j (...), kept classes, classes that do not exist (a lane that has seen only -inf: nothing)
    float s[5] = {mx == m ? run : run * exp_tau(mx - m, a), 0.f, 0.f, kept, bad};
    for (int j = lane; j < a.k; j += R) {
        if (cls[j] < 0) {
            ej[j] = 0.f;
            continue;
        }
        const float d = ej[j] - tm, e = exp_tau(d, a);
        s[1] += e;
        if (e > 0.f || e != e) s[2] += e * (d - (zj[j] - m));
        ej[j] = e;
    }
    row_reduce<R, 5, false>(s, red);
    const float w = a.w ? a.w[n] : 1.f;
    const bool counts = s[3] > 0.f && s[4] == 0.f && w != 0.f;
    const float inv_l = 1.f / s[0], inv_t = 1.f / s[1];
    if (live && lane == 0) {
        const float logs = __builtin_amdgcn_logf(s[0]) * kLn2 - __builtin_amdgcn_logf(s[1]) * kLn2;
        a.loss[n] = s[4] > 0.f && w != 0.f ? NAN : counts ? w * a.tau * (s[2] * inv_t + a.tau * logs) : 0.f;
    }
    if (!a.dz) return;
    const float g = w * a.tau, gl = g * inv_l;
    T* const dz = static_cast<T*>(a.dz) + n * a.ldd;
    auto grad = [&](float x) { return exp_tau(x - m, a) * gl; };
    row_sync<R>();  // the row and its kept classes have been read: dz may be z
    if (!counts) {
        for (int i = lane; i < full && live; i += R) store_zeros<V>(dz + (int64_t)i * V);
        if (lane < rest && live) store_zeros<1>(dz + tail + lane);
    } else if constexpr (!kTwice) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (i * R * V >= a.V) continue;
            const int c = (anew(lane) + i * R) * V, skip = c - (a.V - V);
            float o[V];
            one_at_a_time();
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = grad(q[i][v]);
            if (!live) continue;
            if (skip <= 0) {
                store_vec<V>(dz + c, o);
            } else if (skip < V) {
#pragma unroll
                for (int v = 1; v < V; ++v) {
                    const float x[1] = {o[v]};
                    if (v >= skip) store_vec<1>(dz + (a.V - V) + v, x);
                }
            }
        }
    } else {
        auto put = [&](const Raw<T, V>& r, int i) {
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = grad(r[v]);
            if (live) store_vec<V>(dz + (int64_t)i * V, o);
        };
        int i = lane;
        for (; i + (kAhead - 1) * R < full; i += kAhead * R) {
            Raw<T, V> r[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) r[j] = load_raw<V>(z + (int64_t)(i + j * R) * V);
#pragma unroll
            for (int j = 0; j < kAhead; ++j) put(r[j], i + j * R);
        }
        for (; i < full; i += R) put(load_raw<V>(z + (int64_t)i * V), i);
        if (lane < rest && live) {
            const float o[1] = {grad(load_raw<1>(z + tail + lane)[0])};
            store_vec<1>(dz + tail + lane, o);
        }
    }
    row_sync<R>();  // the row's stores come before those of its kept classes
    if (!live || !counts) return;
    for (int j = lane; j < a.k; j += R) {
        const int c = cls[j];
        if (c < 0) continue;
        float p = 0.f;
        for (int i = 0; i < a.k; ++i) p += cls[i] == c ? ej[i] : 0.f;
        const float o[1] = {grad(zj[j]) - g * (p * inv_t)};
        store_vec<1>(dz + c, o);
    }
}

// Lanes a row: few with several vectors each, which leaves more rows to a workgroup and fewer exchanges between lanes
// (60000 frames x 80 classes in fp32: 8 lanes of 4 vectors 12.9 us, 64 of one 32.9; 26225 x 4046 in bfloat16: 128 lanes of
// 4 vectors 73 us, 256 of 4 112), up to 26 vectors, what 1024 threads' registers hold.
template <typename F>
void with_shape(int64_t V_, int dtype, F&& fn) {
    auto go = [&](auto ty) {
        using T = decltype(ty);
        constexpr int V = Width<T>::v;
        const int64_t nv = (V_ + V - 1) / V;
        if (V_ < V) return fn(ty, DistillShape<1, 8, 1>{});
        if (nv <= 16) return fn(ty, DistillShape<V, 8, 2>{});
        if (nv <= 32) return fn(ty, DistillShape<V, 8, 4>{});
        if (nv <= 64) return fn(ty, DistillShape<V, 16, 4>{});
        if (nv <= 128) return fn(ty, DistillShape<V, 32, 4>{});
        if (nv <= 256) return fn(ty, DistillShape<V, 64, 4>{});
        if (nv <= 512) return fn(ty, DistillShape<V, 128, 4>{});
        if (nv <= 1024) return fn(ty, DistillShape<V, 256, 4>{});
        if (nv <= 2048) return fn(ty, DistillShape<V, 256, 8>{});
        if (nv <= 4096) return fn(ty, DistillShape<V, 256, 16>{});
        if (nv <= 8192) return fn(ty, DistillShape<V, 512, 16>{});
        if (nv <= 16384) return fn(ty, DistillShape<V, 1024, 16>{});
        if (nv <= 26624) return fn(ty, DistillShape<V, 1024, 26>{});
        return fn(ty, DistillShape<V, 1024, 0>{});
    };
    if (dtype == 1) go(bf16{});
    else go(float{});
}

}  // namespace

int distill_max_k() { return 1024; }

hipError_t launch_distill(int64_t N, int V, int k, int dtype, const void* z, int64_t ldz, const int32_t* ids,
                          const void* t, int t_dtype, const float* w, float tau, float* loss, void* dz, int64_t ldd,
                          hipStream_t st) {
    with_shape(V, dtype, [&](auto ty, auto sh) {
        using T = decltype(ty);
        using S = decltype(sh);
        const int64_t most = kMaxLaunchThreads / S::threads * S::rows;  // rows a launch can take
        for (int64_t n = 0; n < N; n += most) {
            const int64_t m = std::min(most, N - n);
            const void* tn = t_dtype == 1 ? static_cast<const void*>(static_cast<const bf16*>(t) + n * k)
                                          : static_cast<const void*>(static_cast<const float*>(t) + n * k);
            const DistillArgs a{m, V, k, static_cast<const T*>(z) + n * ldz, ldz, ids + n * k, tn, t_dtype == 1,
                                w ? w + n : nullptr, tau, (float)(1.4426950408889634 / tau), loss + n,
                                dz ? static_cast<T*>(dz) + n * ldd : nullptr, ldd};
            launch(k_distill<T, S>, dim3((unsigned)((m + S::rows - 1) / S::rows)), dim3(S::threads),
                   sizeof(float) * 3 * k * S::rows, st, a);
        }
    });
    return hipGetLastError();
}

}  // namespace mdl
