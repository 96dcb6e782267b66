// k_norm.hip — the norms before and after a block, fused with the block's gate and the scaled residual.
//
// Row by row, with x the residual stream, z the block's output and u its gate's pre-activation:
//   zh = z / sqrt(mean z^2 + eps);  r = x + scale sigmoid(u) w_post zh
//   rh = r / sqrt(mean r^2 + eps);  v = w_pre rh
// (v feeds the next block). Backward, from dr and dv, with m the mean over a row:
//   d = dr + (t - rh m(t rh)) / rms(r),  t = w_pre dv;  dx = d
//   k = d sigmoid(u);  dz = (p - zh m(p zh)) / rms(z),  p = k scale w_post;  du = d scale w_post zh s (1 - s)
//   dw_post = scale q, dscale = w_post q with q the column sum of k zh;  dw_pre = the column sum of dv rh
// so two column sums give the three weight gradients.
//
// R lanes share a row and keep all of it in registers: each tensor is read once and written once (the backward forms r
// again from x, z and u, so it needs no row statistics of the forward). Row sums are exchanged between the lanes, and
// between waves through LDS where a row takes more than one. r enters the second norm as the fp32 value, before its
// rounding to the output's type. All sums are fp32.
//
// Bound by HBM: 20480 x 2048 in bfloat16 takes 80 us forward (419 MB, 5.2 TB/s) and 145 us backward (671 MB, 4.6 TB/s) and
// 7.5 us for the weight gradients out of the workgroups' column sums; 81920 x 50 in fp32, rows of 200 bytes, 13.0, 23.5
// and 4.8 us (82, 131 and 0.8 MB; the first two above the rate of a large copy, 4.93 TB/s). The backward of rows above
// 8192 elements is bound by its spills: 4096 x 16384 takes 1.13 ms in bfloat16 and 1.33 ms in fp32 (1.07 and 2.15 GB; 4096 x
// 8192: 0.17 and 0.26 ms).
#include "kernels.h"
#include "seqio.h"

#include <algorithm>

namespace mdl {

namespace {

template <int V_, int R_, int NV_>
struct NormShape {  // elements a vector, lanes a row, vectors a lane
    static constexpr int V = V_, R = R_, NV = NV_;
    static constexpr int threads = R_ > 256 ? R_ : 256;
    static constexpr int rows = threads / R_;  // rows a workgroup holds at once
};

// Row sums of K values over the R lanes of a row; every lane of the workgroup takes part where R > 64.
template <int R, int K>
__device__ inline void row_sums(float (&s)[K], float* red) {
#pragma unroll
    for (int k = 0; k < K; ++k) s[k] = group_sum<(R < 64 ? R : 64)>(s[k]);
    if constexpr (R > 64) {
        const int wave = threadIdx.x >> 6;
        __syncthreads();  // the last use of red is over
        if ((threadIdx.x & 63) == 0)
            for (int k = 0; k < K; ++k) red[wave * K + k] = s[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            s[k] = 0.f;
            for (int w = 0; w < R / 64; ++w) s[k] += red[w * K + k];
        }
    }
}

// a lane's vectors of a row: vector i starts at channel c[i], moved back to ch[i] where it would pass the row's end;
// its first skip[i] elements belong to a neighbour (all of them past the end)
template <typename S>
struct Cols {
    int ch[S::NV], skip[S::NV];
    __device__ inline Cols(int D) {
        const int lane = threadIdx.x % S::R;
#pragma unroll
        for (int i = 0; i < S::NV; ++i) {
            const int c = (lane + i * S::R) * S::V;
            ch[i] = min(c, D - S::V);
            skip[i] = c - ch[i];
        }
    }
    __device__ inline bool has(int i) const { return skip[i] < S::V; }
    __device__ inline float own(int i, int v, float x) const { return v >= skip[i] ? x : 0.f; }
};

template <typename T, typename S>
__device__ inline void load_row(Raw<T, S::V> (&q)[S::NV], const void* base, int64_t off, const Cols<S>& c) {
#pragma unroll
    for (int i = 0; i < S::NV; ++i) q[i] = load_raw<S::V>(static_cast<const T*>(base) + off + c.ch[i]);
}
template <typename S>
__device__ inline void load_w(float (&w)[S::NV][S::V], const float* p, const Cols<S>& c) {
#pragma unroll
    for (int i = 0; i < S::NV; ++i) {
        if (p) load_f32<S::V>(p + c.ch[i], w[i]);
        else
            for (int v = 0; v < S::V; ++v) w[i][v] = 1.f;
    }
}

template <typename T, typename S>
__global__ __launch_bounds__(S::threads) void k_norm_fwd(NormArgs a) {
    constexpr int V = S::V, NV = S::NV;
    __shared__ float red[S::threads / 64 * 2];
    const int64_t row = (int64_t)blockIdx.x * S::rows + threadIdx.x / S::R;
    const bool live = row < a.N;
    const int64_t n = live ? row : a.N - 1;
    const Cols<S> c(a.D);
    Raw<T, V> x[NV], z[NV], u[NV];
    load_row<T, S>(x, a.x, n * a.ldx, c);
    float r[NV][V];
    if (a.z) {
        load_row<T, S>(z, a.z, n * a.ldz, c);
        if (a.u) load_row<T, S>(u, a.u, n * a.ldu, c);
        float wp[NV][V], sc[NV][V];
        load_w<S>(wp, a.w_post, c);
        load_w<S>(sc, a.scale, c);
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) s[0] = __builtin_fmaf(c.own(i, v, z[i][v]), z[i][v], s[0]);
        row_sums<S::R>(s, red);
        const float sig = __builtin_amdgcn_rsqf(__builtin_fmaf(s[0], a.inv_d, a.eps));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float g = 1.f, gc;
                if (a.u) sigm2<T>(u[i][v], g, gc);
                r[i][v] = __builtin_fmaf(sc[i][v] * wp[i][v] * g, z[i][v] * sig, x[i][v]);
            }
            if (live && c.has(i)) store_vec<V>(static_cast<T*>(a.r) + n * a.ldr + c.ch[i], r[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) r[i][v] = x[i][v];
    }
    if (!a.v) return;
    float wn[NV][V];
    load_w<S>(wn, a.w_pre, c);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) s[0] = __builtin_fmaf(c.own(i, v, r[i][v]), r[i][v], s[0]);
    row_sums<S::R>(s, red);
    const float rho = __builtin_amdgcn_rsqf(__builtin_fmaf(s[0], a.inv_d, a.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = r[i][v] * rho * wn[i][v];
        if (live && c.has(i)) store_vec<V>(static_cast<T*>(a.v) + n * a.ldr + c.ch[i], o);
    }
}

// Workgroup b takes the rows b rows, b rows + gridDim rows, ... and adds its column sums (q, then dw_pre's) in registers;
// they go to part[b][2][D].
template <typename T, typename S>
__global__ __launch_bounds__(S::threads) void k_norm_bwd(NormArgs a) {
    constexpr int V = S::V, NV = S::NV;
    __shared__ float red[S::threads / 64 * 2];
    extern __shared__ float colsum[];  // [rows][R NV V], where a workgroup holds several rows
    const Cols<S> c(a.D);
    float q[NV][V] = {}, p[NV][V] = {};
    const int group = threadIdx.x / S::R;
    for (int64_t base = (int64_t)blockIdx.x * S::rows; base < a.N; base += (int64_t)gridDim.x * S::rows) {
        const bool live = base + group < a.N;
        const int64_t n = live ? base + group : a.N - 1;
        Raw<T, V> x[NV], z[NV], u[NV], dr[NV], dv[NV];
        load_row<T, S>(x, a.x, n * a.ldx, c);
        if (a.z) load_row<T, S>(z, a.z, n * a.ldz, c);
        if (a.u) load_row<T, S>(u, a.u, n * a.ldu, c);
        if (a.dr) load_row<T, S>(dr, a.dr, n * a.ldr, c);
        if (a.dv) load_row<T, S>(dv, a.dv, n * a.ldr, c);
        float cs[NV][V], wn[NV][V];  // scale w_post, w_pre
        if (a.z) {
            float wp[NV][V];
            load_w<S>(wp, a.w_post, c);
            load_w<S>(cs, a.scale, c);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) cs[i][v] *= wp[i][v];
        }
        if (a.dv) load_w<S>(wn, a.w_pre, c);
        float sig = 0.f;
        if (a.z) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) s[0] = __builtin_fmaf(c.own(i, v, z[i][v]), z[i][v], s[0]);
            row_sums<S::R>(s, red);
            sig = __builtin_amdgcn_rsqf(__builtin_fmaf(s[0], a.inv_d, a.eps));
        }
        // long rows: what was unpacked for one walk over the row is unpacked again for the next
        auto anew = [&] {
            if constexpr (NV >= 4) {
                one_at_a_time();
                if (a.z) forget(z);
                if (a.u) forget(u);
                if (a.dv) forget(dv);
            }
        };
        anew();
        float d[NV][V];
        if (a.dv) {
            float r[NV][V], s[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    r[i][v] = x[i][v];
                    if (a.z) {
                        float g = 1.f, gc;
                        if (a.u) sigm2<T>(u[i][v], g, gc);
                        r[i][v] = __builtin_fmaf(cs[i][v] * g, z[i][v] * sig, r[i][v]);
                    }
                    const float ro = c.own(i, v, r[i][v]);
                    s[0] = __builtin_fmaf(ro, r[i][v], s[0]);
                    s[1] = __builtin_fmaf(ro, dv[i][v] * wn[i][v], s[1]);
                }
            row_sums<S::R>(s, red);
            const float rho = __builtin_amdgcn_rsqf(__builtin_fmaf(s[0], a.inv_d, a.eps));
            const float m = s[1] * rho * a.inv_d;  // m(t rh)
            anew();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float rh = r[i][v] * rho;
                    d[i][v] = rho * __builtin_fmaf(-rh, m, dv[i][v] * wn[i][v]);
                    if (a.dr) d[i][v] += dr[i][v];
                    p[i][v] += live ? dv[i][v] * rh : 0.f;
                }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) d[i][v] = dr[i][v];
        }
        anew();
        float pz[NV][V], du[NV][V];
        float s[1] = {0.f};
        if (a.z) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float g = 1.f, gc = 0.f;
                    if (a.u) sigm2<T>(u[i][v], g, gc);
                    const float zh = z[i][v] * sig, k = d[i][v] * g;
                    q[i][v] += live ? k * zh : 0.f;
                    pz[i][v] = k * cs[i][v];
                    du[i][v] = pz[i][v] * zh * gc;
                    s[0] = __builtin_fmaf(c.own(i, v, pz[i][v]), zh, s[0]);
                }
            row_sums<S::R>(s, red);
        }
        const float m = s[0] * a.inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!(live && c.has(i))) continue;
            const int64_t o = n * a.ldd + c.ch[i];
            store_vec<V>(static_cast<T*>(a.dx) + o, d[i]);
            if (a.z) {
                float dz[V];
#pragma unroll
                for (int v = 0; v < V; ++v) dz[v] = sig * __builtin_fmaf(-(z[i][v] * sig), m, pz[i][v]);
                store_vec<V>(static_cast<T*>(a.dz) + o, dz);
            }
            if (a.u) store_vec<V>(static_cast<T*>(a.du) + o, du[i]);
        }
    }
    // the workgroup's rows' column sums, added in row order
    float* const out = a.part + (int64_t)blockIdx.x * 2 * a.D;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float(&w)[NV][V] = h ? p : q;
        if constexpr (S::rows > 1) {
            constexpr int L = S::R * NV * V;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) colsum[group * L + (i * V + v) * S::R + threadIdx.x % S::R] = w[i][v];
            __syncthreads();
            if (group == 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        for (int k = 1; k < S::rows; ++k) w[i][v] += colsum[k * L + (i * V + v) * S::R + threadIdx.x];
            }
        }
        if (group == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (c.has(i)) store_f32<V>(out + h * a.D + c.ch[i], w[i]);
        }
    }
}

// the weight gradients from the workgroups' column sums: 16 columns by 64 threads a column, thread g adding workgroups
// g, g + 64, ... in order, then the 64 sums pairwise
constexpr int kWredCols = 16, kWredGroups = 64;
__global__ __launch_bounds__(kWredCols * kWredGroups) void k_norm_wreduce(
    const float* __restrict__ part, int nb, int D, const float* __restrict__ w_post, const float* __restrict__ scale,
    float* __restrict__ dw_post, float* __restrict__ dscale, float* __restrict__ dw_pre) {
    __shared__ float red[kWredGroups][kWredCols];
    const int lane = threadIdx.x % kWredCols, g = threadIdx.x / kWredCols;
    const int i = blockIdx.x * kWredCols + lane;
    float s = 0.f;
    if (i < 2 * D) {
#pragma unroll 4
        for (int b = g; b < nb; b += kWredGroups) s += part[(int64_t)b * 2 * D + i];
    }
    red[g][lane] = s;
    for (int h = kWredGroups / 2; h > 0; h >>= 1) {
        __syncthreads();
        if (g < h) red[g][lane] += red[g + h][lane];
    }
    if (g || i >= 2 * D) return;
    s = red[0][lane];
    if (i >= D) {
        if (dw_pre) dw_pre[i - D] = s;
        return;
    }
    if (dw_post) dw_post[i] = scale ? s * scale[i] : s;
    if (dscale) dscale[i] = w_post ? s * w_post[i] : s;
}

// Lanes a row: the fewest that hold it in one vector each up to a wave, two vectors each up to 128 (the row sums then need
// no LDS), and from there as many waves as keep the backward's row in its registers (five tensors, 224 registers at two
// vectors of eight). Rows of more than 8192 elements take 1024 threads of 128 registers each, of which the backward spills
// 144 in bfloat16 (484 bytes a lane) and 195 in fp32 (544 bytes); in fp32 rows of more than 4096 spill 2 (12 bytes).
template <typename F>
void with_shape(int D, int dtype, F&& fn) {
    auto go = [&](auto ty) {
        using T = decltype(ty);
        constexpr int V = Width<T>::v;
        const int nv = (D + V - 1) / V;
        if (D < V) return fn(ty, NormShape<1, 8, 1>{});
        if (nv <= 8) return fn(ty, NormShape<V, 8, 1>{});
        if (nv <= 16) return fn(ty, NormShape<V, 16, 1>{});
        if (nv <= 32) return fn(ty, NormShape<V, 32, 1>{});
        if (nv <= 64) return fn(ty, NormShape<V, 64, 1>{});
        if (nv <= 128) return fn(ty, NormShape<V, 64, 2>{});
        if (nv <= 256) return fn(ty, NormShape<V, 256, 1>{});
        if (nv <= 512) return fn(ty, NormShape<V, 256, 2>{});
        if (nv <= 1024) return fn(ty, NormShape<V, 512, 2>{});
        if constexpr (V == 8) {
            return fn(ty, NormShape<V, 1024, 2>{});
        } else {
            if (nv <= 2048) return fn(ty, NormShape<V, 512, 4>{});
            return fn(ty, NormShape<V, 1024, 4>{});
        }
    };
    if (dtype == 1) go(bf16{});
    else go(float{});
}

// workgroups of the backward: each leaves 8 D bytes of column sums, so at least four turns each where there are rows
// enough to fill the device with a quarter of that many, and no more than fill it a few times
int bwd_blocks(int64_t N, int rows) {
    const int64_t turns = (N + rows - 1) / rows;
    return (int)std::max<int64_t>(1, std::min(turns, std::max<int64_t>(256, std::min<int64_t>(turns / 4, 1024))));
}

}  // namespace

int norm_max_d() { return 16384; }

size_t norm_bwd_ws(int64_t N, int D, int dtype) {
    size_t bytes = 0;
    with_shape(D, dtype, [&](auto, auto sh) { bytes = (size_t)bwd_blocks(N, decltype(sh)::rows) * 2 * D * 4; });
    return bytes;
}

hipError_t launch_norm_fwd(const NormArgs& a, int dtype, hipStream_t st) {
    with_shape(a.D, dtype, [&](auto ty, auto sh) {
        using T = decltype(ty);
        using S = decltype(sh);
        const int64_t most = kMaxLaunchThreads / S::threads * S::rows;  // rows a launch can take
        for (int64_t n = 0; n < a.N; n += most) {
            NormArgs b = a;
            b.N = std::min(most, a.N - n);
            b.x = static_cast<const T*>(a.x) + n * a.ldx;
            if (a.z) b.z = static_cast<const T*>(a.z) + n * a.ldz;
            if (a.u) b.u = static_cast<const T*>(a.u) + n * a.ldu;
            if (a.r) b.r = static_cast<T*>(a.r) + n * a.ldr;
            if (a.v) b.v = static_cast<T*>(a.v) + n * a.ldr;
            launch(k_norm_fwd<T, S>, dim3((unsigned)((b.N + S::rows - 1) / S::rows)), dim3(S::threads), 0, st, b);
        }
    });
    return hipGetLastError();
}

hipError_t launch_norm_bwd(const NormArgs& a, int dtype, float* dw_post, float* dscale, float* dw_pre,
                           hipStream_t st) {
    with_shape(a.D, dtype, [&](auto ty, auto sh) {
        using S = decltype(sh);
        const int nb = bwd_blocks(a.N, S::rows);
        const size_t lds = S::rows > 1 ? sizeof(float) * S::threads * S::NV * S::V : 0;
        launch(k_norm_bwd<decltype(ty), S>, dim3(nb), dim3(S::threads), lds, st, a);
        if (dw_post || dscale || dw_pre)
            launch(k_norm_wreduce, dim3((2 * a.D + kWredCols - 1) / kWredCols), dim3(kWredCols * kWredGroups), 0, st, a.part, nb, a.D, a.w_post, a.scale,
                   dw_post, dscale, dw_pre);
    });
    return hipGetLastError();
}

}  // namespace mdl
