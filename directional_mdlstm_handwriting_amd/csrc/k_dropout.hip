// k_dropout.hip — dropout from a counter-based generator, with the residual it is added to; the mask is never stored.
//
//   y = r + x [u >= c] 65536 / (65536 - c),   c = round(65536 p)
// u: 16 bits of Philox 4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3") for each element: eight
// neighbouring elements of a row share one evaluation, its counter the group's number (row-major over N rows of
// ceil(D / 8) groups) and the call's number, its key the seed. So the mask depends on N, D and the pair (seed, call)
// alone, and the backward, the same kernel on dy, forms it again.
//
// 16 bits an element and not 32: the generator then takes 20 products of 32 x 32 bits for eight elements. The
// probability is a multiple of 2^-16 and the scale is that of the rounded one, so the expectation is exact.
//
// Bound by memory: 20480 x 2048 in bfloat16 with the residual takes 42 us (252 MB, 6.0 TB/s), without it 31 (168 MB, 5.4),
// where a copy of 2 GB runs at 5.1; a thread has its four groups' loads in flight before it draws the first one's numbers.
#include "kernels.h"
#include "seqio.h"

namespace mdl {

namespace {

constexpr int kLanes = 256, kPerThread = 4;  // groups of eight elements a thread

struct Philox {
    uint32_t w[4];
};
__device__ inline Philox philox(uint64_t ctr, uint64_t call, uint64_t seed) {
    uint32_t c0 = (uint32_t)ctr, c1 = (uint32_t)(ctr >> 32), c2 = (uint32_t)call, c3 = (uint32_t)(call >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)p1;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return {{c0, c1, c2, c3}};
}

struct Group {
    float v[8];
};
__device__ inline Group load8(const float* p) {
    const auto a = load_once<4>(p), b = load_once<4>(p + 4);
    return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ inline Group load8(const bf16* p) {
    const auto a = load_once<8>(p);
    return {{a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7]}};
}
__device__ inline void store8(float* p, const Group& g) {
    const float a[4] = {g.v[0], g.v[1], g.v[2], g.v[3]}, b[4] = {g.v[4], g.v[5], g.v[6], g.v[7]};
    store_vec<4>(p, a);
    store_vec<4>(p + 4, b);
}
__device__ inline void store8(bf16* p, const Group& g) { store_vec<8>(p, g.v); }

template <typename T>
__device__ inline Group load_some(const T* p, int n) {
    Group g;
#pragma unroll
    for (int i = 0; i < 8; ++i) g.v[i] = i < n ? load_raw<1>(p + i)[0] : 0.f;
    return g;
}

struct Args {
    int64_t N, groups;              // N times the groups of a row
    int D, per_row;
    uint32_t mul, shift;            // t / per_row = t mul >> (31 + shift) for t < 2^31
    const void *x, *r;
    int64_t ldx, ldr, ldy;
    uint32_t cut;
    float scale;
    const uint64_t* rng;
    void* y;
};

template <typename T, bool RES>
__global__ __launch_bounds__(kLanes) void dropout(const Args a) {
    const int64_t first = (int64_t)blockIdx.x * (kLanes * kPerThread);
    const int64_t row0 = first / a.per_row;
    const uint32_t rem0 = (uint32_t)(first - row0 * a.per_row);
    const uint64_t seed = a.rng[0], call = a.rng[1];
    Group x[kPerThread], r[kPerThread];
    int64_t row[kPerThread];
    int col[kPerThread], n[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const uint32_t t = i * kLanes + threadIdx.x, u = rem0 + t;
        const uint32_t q = (uint32_t)(((uint64_t)u * a.mul) >> (31 + a.shift));
        row[i] = row0 + q;
        col[i] = (int)(u - q * (uint32_t)a.per_row) * 8;
        n[i] = first + t < a.groups ? a.D - col[i] : 0;
        const T* px = static_cast<const T*>(a.x) + row[i] * a.ldx + col[i];
        const T* pr = RES ? static_cast<const T*>(a.r) + row[i] * a.ldr + col[i] : nullptr;
        if (n[i] >= 8) {
            x[i] = load8(px);
            if (RES) r[i] = load8(pr);
        } else if (n[i] > 0) {
            x[i] = load_some(px, n[i]);
            if (RES) r[i] = load_some(pr, n[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        if (n[i] <= 0) continue;
        const Philox p = philox((uint64_t)(first + i * kLanes + threadIdx.x), call, seed);
        Group y;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t u = (j & 1) ? p.w[j >> 1] >> 16 : p.w[j >> 1] & 0xffffu;
            const float v = u >= a.cut ? x[i].v[j] * a.scale : 0.f;
            y.v[j] = RES ? r[i].v[j] + v : v;
        }
        T* py = static_cast<T*>(a.y) + row[i] * a.ldy + col[i];
        if (n[i] >= 8) {
            store8(py, y);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n[i]) {
                    const float one[1] = {y.v[j]};
                    store_vec<1>(py + j, one);
                }
        }
    }
}

template <typename T>
void go(const Args& a, hipStream_t st) {
    const dim3 grid((uint32_t)((a.groups + kLanes * kPerThread - 1) / (kLanes * kPerThread)));
    if (a.r) launch(dropout<T, true>, grid, dim3(kLanes), 0, st, a);
    else launch(dropout<T, false>, grid, dim3(kLanes), 0, st, a);
}

}  // namespace

int64_t dropout_max_groups() { return kMaxLaunchThreads / kLanes * (kLanes * kPerThread); }

hipError_t launch_dropout(int64_t N, int D, int dtype, const void* x, int64_t ldx, const void* r, int64_t ldr, int cut,
                          const uint64_t* rng, void* y, int64_t ldy, hipStream_t st) {
    if (N == 0) return hipSuccess;
    Args a{};
    a.N = N;
    a.D = D;
    a.per_row = (int)(((int64_t)D + 7) / 8);
    a.groups = N * a.per_row;
    int l = 0;
    while ((int64_t(1) << l) < a.per_row) ++l;
    a.mul = (uint32_t)(((uint64_t(1) << (31 + l)) + a.per_row - 1) / a.per_row);
    a.shift = (uint32_t)l;
    a.x = x;
    a.r = r;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldy = ldy;
    a.cut = (uint32_t)cut;
    a.scale = 65536.f / (float)(65536 - cut);
    a.rng = rng;
    a.y = y;
    if (dtype == 1) go<bf16>(a, st);
    else go<float>(a, st);
    return hipGetLastError();
}

}  // namespace mdl
