// k_vocab.hip — softmax cross entropy over a vocabulary from the hidden states and the class weights, with its gradients:
// of all the logits, no more than a block of rows' is ever held (up to 256 MB, or 1024 rows), and for the loss alone none.
//
//   z = h W^T,  loss_n = w_n (ln sum_c exp z_nc - z_n,id),  G = w (softmax z - [c = id]),  dh = G W,  dW = G^T h
//
// A first product, a block of rows at a time, leaves per row and 256 (or 128) classes the maximum and sum of exponentials of
// those that are not the target, and the target's logit; `join` makes the losses of them. With the target t apart, and e_c =
// exp(z_c - top) below the larger of the others' maximum and z_t,
//   loss = w ln(1 + sum e_c) where z_t is the larger, w (top - z_t + ln(e_t + sum e_c)) else,  p_t - 1 = -sum e_c / (e_t + sum e_c)
// in which nothing cancels: a row that is sure of its target has its small loss and gradient, whatever its logits have in
// common (as one float, the logarithm of the whole sum is off by half a step of the largest logit). With gradients it also keeps the block's logits: in fp32 as they
// are, in bfloat16 the exponentials below their tile's maximum, times 2^15, as 16 bits of half precision (a rounding of 2^-11
// of the value, an eighth of the one G is about to get, or of 2^-40 of the maximum). `grad` makes G of them where they lie, and two products take G into dh and dW: 6 N V D operations. Several
// blocks add up dW in fp32, which costs 8 bytes an element and block: at 1024 rows a quarter of the block's products.
// (Forming the logits again, once the statistics are known, is 8 N V D operations and nothing written but G: 4096 x 2048 over
// 32000 classes in bfloat16 took 1985 us that way and takes 1507 to 1553, in fp32 15.6 and 12.1 ms. 16384 x 2048 over 131072
// classes, 16 blocks of 1024 rows, takes 31.0 ms: 0.85 PFLOP/s where one block of 4096 rows over 32000 reaches 1.05.)
//
// Products: tiles of BM x BN by 8 (4) waves, 32 x 32 results of the matrix instructions (32x32x16 bfloat16, 32x32x2 fp32),
// 128 bytes of depth at a time from global memory straight into LDS, one step ahead of the products. An operand whose rows
// run along the depth is laid row by row, its 16-byte chunks turned by every second row, so that the reads of 16 rows meet
// all banks (turned by every row: 3.9 cycles of conflicts a read, now 0.2, and the same time); one whose rows run across it
// is laid as it comes and read by transposing reads (bfloat16) or word by word (fp32).
//
// Measured, 4096 x 2048 over 32000 classes in bfloat16 (537 GFLOP a product): logits and statistics 575 us, of which writing
// 262 MB is some 50 to 100 (the loss alone, all launches, takes 470 to 486), dh 495 + 14, dW 481 (0.93, 1.08 and 1.12 PFLOP/s;
// the matrix units are busy for 51, 55 and 61 % of the cycles; the library's 8192^3 reaches 1.39), G 85 (524 MB at 6.2 TB/s),
// packing and joining 16.
#include "kernels.h"
#include "seqio.h"

#include <algorithm>

namespace mdl {

namespace {

typedef __bf16 bh8 __attribute__((ext_vector_type(8)));
typedef short h4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

#define MDL_LDS __attribute__((address_space(3)))

// ---- operand tiles ----------------------------------------------------------------------------------------------
constexpr uint32_t kOut = 0x80000000u;  // an offset past every buffer's end: the load gives zeros
// ROWS rows (of the result) by 128 bytes of depth in LDS. ALONG: the operand's rows in memory run along the depth.
template <typename T, int ROWS, int THREADS, bool ALONG>
struct Tile {
    static constexpr int E = sizeof(T), BK = 128 / E, per_thread = ROWS * 8 / THREADS, bytes = ROWS * 128;
    static constexpr int row_bytes = ALONG ? 128 : ROWS * E, row_chunks = row_bytes / 16;
    static_assert(ROWS * 8 % THREADS == 0, "whole chunks a thread");
    const char* base;     // ALONG: row 0 at the depth of the next step; else the next step's first row
    int64_t ld;           // bytes
    int edge;             // ALONG: rows of the tile that exist; else: bytes of a row that exist
    int64_t depth;        // ALONG: bytes of depth that are left; else rows
    uint32_t off[per_thread];
    int at;               // ALONG: this thread's chunks' place in the depth, bytes (the same for all of them)

    // row0: the tile's first row of the result, k0: first element of depth, k1: its end
    __device__ inline void init(const void* p, int64_t ld_elems, int64_t row0, int64_t n_rows, int64_t k0, int64_t k1) {
        static_assert(!ALONG || THREADS % 128 == 0, "whole groups of sixteen rows between a thread's chunks");
        ld = ld_elems * E;
        if constexpr (ALONG) {
            base = static_cast<const char*>(p) + row0 * ld + k0 * E;
            edge = (int)(n_rows - row0 < ROWS ? n_rows - row0 : ROWS);
            depth = (k1 - k0) * E;
        } else {
            base = static_cast<const char*>(p) + k0 * ld + row0 * E;
            const int64_t left = (n_rows - row0) * E;
            edge = (int)(left < row_bytes ? left : row_bytes);
            depth = k1 - k0;
        }
        at = 16 * (threadIdx.x % 8 ^ (threadIdx.x / 16 & 7));
#pragma unroll
        for (int i = 0; i < per_thread; ++i) {
            const int q = i * THREADS + threadIdx.x, r = q / row_chunks, c = q % row_chunks;
            if constexpr (ALONG) {
                off[i] = (uint32_t)(r * ld) + at;
            } else {
                const int col = 16 * (c ^ (E == 2 ? (r & 3) << 2 : (r >> 2 & 1) << 3));
                off[i] = col < edge ? (uint32_t)(r * ld) + col : kOut;
            }
        }
    }
    // the next 128 bytes of depth into the LDS tile; zeros past the depth's end and the operand's edge. Chunks are whole:
    // the depth (ALONG) and the row's width (else) count in chunks of 16 bytes, of which the caller keeps the last one
    // readable and finite.
    __device__ inline void load(char* lds) {
        constexpr int64_t most = ALONG ? 128 : BK;
        const int64_t now = depth < most ? (depth > 0 ? depth : 0) : most;
        const int64_t records = ALONG ? (edge - 1) * ld + now : (now - 1) * ld + edge;
        const __amdgpu_buffer_rsrc_t r = rsrc(base, now > 0 ? (records + 15) & ~int64_t(15) : 0);
        const bool in = !ALONG || at < now;
#pragma unroll
        for (int i = 0; i < per_thread; ++i) {
            const int first = (i * THREADS + (int)(threadIdx.x & ~63u)) * 16;  // of the wave
            const int o = (int)(in ? off[i] : kOut);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (MDL_LDS void*)(lds + first), 16, o, 0, 0, 0);
        }
        base += ALONG ? 128 : BK * ld;
        depth -= most;
    }
    // this lane's part of the operand for 32 rows from row0 on, at 32 bytes of depth: 16 bytes of row lane % 32, the lower
    // half of the depth in the lower 32 lanes
    static __device__ inline u32x4 part(const char* lds, int row0, int s) {
        const int lane = threadIdx.x & 63;
        if constexpr (ALONG) {
            const int r = row0 + (lane & 31);
            return *reinterpret_cast<const u32x4*>(lds + r * 128 + 16 * ((2 * s + (lane >> 5)) ^ (r >> 1 & 7)));
        } else if constexpr (E == 2) {
            typedef MDL_LDS h4* P;
            const int q = lane >> 4, i = lane & 15, k = 16 * s + 8 * (q >> 1) + (i >> 2);
            const int col = (row0 + 16 * (q & 1)) * 2 + 8 * (i & 3);
            const char* p = lds + k * row_bytes + (col ^ (i >> 2) << 6);
            const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p)));
            const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + 4 * row_bytes)));
            return u32x4{a[0], a[1], b[0], b[1]};
        } else {
            const int h = lane >> 5, k = 8 * s + 4 * h;
            const char* p = lds + k * row_bytes + ((row0 + (lane & 31)) * 4 ^ h << 7);
            u32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const uint32_t*>(p + e * row_bytes);
            return v;
        }
    }
};

template <typename T>
__device__ inline f32x16 mma(u32x4 x, u32x4 y, f32x16 c) {
    if constexpr (sizeof(T) == 2) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bh8, x), __builtin_bit_cast(bh8, y), c, 0, 0, 0);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(x[e]), __uint_as_float(y[e]), c, 0, 0, 0);
        return c;
    }
}

// (maximum, sum) of two parts of a row; the sum beside a maximum of -inf is 0 or NaN
__device__ inline float2 joined(float2 a, float2 b) {
    const float top = fmaxf(a.x, b.x);
    const float x = a.x == -INFINITY ? a.y : a.y * exp_neg<float>(a.x - top);
    const float y = b.x == -INFINITY ? b.y : b.y * exp_neg<float>(b.x - top);
    return make_float2(top, x + y);
}

// ---- the product ------------------------------------------------------------------------------------------------
template <int WM_, int WN_, int TM_, int TN_>
struct Shape {  // waves down and across, 32 x 32 tiles of a wave down and across
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_, threads = 64 * WM * WN, BM = 32 * WM * TM, BN = 32 * WN * TN;
};
typedef Shape<2, 4, 4, 2> Large;  // 256 x 256
typedef Shape<2, 2, 2, 2> Small;  // 128 x 128
typedef Shape<1, 4, 1, 1> Thin;   // 32 x 128
enum Size { kLarge, kSmall, kThin };

// 128 bytes of depth of a wave's tiles: a quarter's operands are read while the products of the one before run
template <typename S, typename TA, typename TB>
__device__ inline void read_parts(const char* la, const char* lb, int wm, int wn, int s, u32x4 (&x)[S::TM], u32x4 (&y)[S::TN]) {
#pragma unroll
    for (int j = 0; j < S::TN; ++j) y[j] = TB::part(lb, wn + 32 * j, s);
#pragma unroll
    for (int i = 0; i < S::TM; ++i) x[i] = TA::part(la, wm + 32 * i, s);
}
template <typename T, typename S, typename TA, typename TB>
__device__ inline void one_step(const char* la, const char* lb, int wm, int wn, f32x16 (&c)[S::TM][S::TN]) {
    u32x4 x[2][S::TM], y[2][S::TN];
    read_parts<S, TA, TB>(la, lb, wm, wn, 0, x[0], y[0]);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if (s < 3) read_parts<S, TA, TB>(la, lb, wm, wn, s + 1, x[(s + 1) & 1], y[(s + 1) & 1]);
#pragma unroll
        for (int i = 0; i < S::TM; ++i)
#pragma unroll
            for (int j = 0; j < S::TN; ++j) c[i][j] = mma<T>(y[s & 1][j], x[s & 1][i], c[i][j]);
        __builtin_amdgcn_sched_barrier(0);
    }
}

struct Args {
    const void *a, *b;            // result rows and columns' operands
    int64_t lda, ldb, M, N, K;
    int64_t tiles_m, tiles_n, splits;
    // epilogues
    float2* stats;                // [tiles_n][M] maximum and sum
    float* target;                // [M]
    const int32_t* ids;           // [M] -1: none
    void* out;                    // [M] at ldo; kStats: the logits or exponentials, or null
    int64_t ldo, cols;            // cols: columns that are written
    float* slab;                  // [splits][M][N]
    int add;                      // onto what the slab holds
};

enum { kStats, kStore, kSlab };

// two values as 16 bits each, the nearest ones: exponentials of at most 1 times kHalfScale in half precision (1 becomes 2^15,
// half precision's largest power of 2, and what is 2^-29 of it still has all its bits), or bfloat16
constexpr float kHalfScale = 32768.f;
template <bool HALF>
__device__ inline uint32_t pack16(float a, float b) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    if constexpr (HALF) return __builtin_bit_cast(uint32_t, h2{(_Float16)(a * kHalfScale), (_Float16)(b * kHalfScale)});
    else return pack_bf16(a, b);
}

// A wave's tiles as they lie, four neighbours of a row a lane; onto what is there with `add` (fp32 alone).
template <typename S, bool HALF = false, typename E>
__device__ inline void store_direct(const f32x16 (&c)[S::TM][S::TN], E* out, int64_t ldo, int64_t cols, bool add, int64_t M,
                                    int64_t m0, int64_t n0, int wm) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < S::TM; ++i) {
        const int64_t m = m0 + wm + 32 * i + (lane & 31);
        if (m >= M) continue;
#pragma unroll
        for (int j = 0; j < S::TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const int64_t n = n0 + 32 * j + 2 * e + 4 * (lane >> 5);
                E* o = out + m * ldo + n;
                f32x4 v = {c[i][j][e], c[i][j][e + 1], c[i][j][e + 2], c[i][j][e + 3]};
                if constexpr (sizeof(E) == 2) {
                    typedef u32x2 u32x2_e __attribute__((aligned(2), may_alias));
                    const u32x2 q = {pack16<HALF>(v[0], v[1]), pack16<HALF>(v[2], v[3])};
                    if (n + 4 <= cols) *reinterpret_cast<u32x2_e*>(o) = q;
                    else
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (n + r < cols) o[r].u = (uint16_t)(q[r >> 1] >> (16 * (r & 1)));
                } else if (n + 4 <= cols) {
                    if (add) v += *reinterpret_cast<const f32x4_e*>(o);
                    *reinterpret_cast<f32x4_e*>(o) = v;
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (n + r < cols) o[r] = add ? o[r] + v[r] : v[r];
                }
            }
    }
}

// A workgroup's tile as 16 bits each, through LDS (in which no tile is read any more), so that whole lines leave: a quarter
// (half) of the tile's rows in each array, their 16-byte chunks rotated by the row.
template <typename S, bool HALF, typename E>
__device__ inline void store_lines(const f32x16 (&c)[S::TM][S::TN], char* a0, char* b0, char* a1, char* b1, E* out, int64_t ldo,
                                   int64_t cols, int64_t M, int64_t m0, int64_t n0, int wm, int wn) {
    constexpr int chunks = S::BN / 8;
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const auto part = [&](int row) {
        const int k = row >> 6;
        return (k == 0 ? a0 : k == 1 ? b0 : k == 2 ? a1 : b1) + (row & 63) * (S::BN * 2);
    };
#pragma unroll
    for (int i = 0; i < S::TM; ++i) {
        const int row = wm + 32 * i + (lane & 31);
        char* q = part(wm + 32 * i) + (lane & 31) * (S::BN * 2);
#pragma unroll
        for (int j = 0; j < S::TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const int n = wn + 32 * j + 2 * e;  // and 4 h
                const u32x2 v = {pack16<HALF>(c[i][j][e], c[i][j][e + 1]), pack16<HALF>(c[i][j][e + 2], c[i][j][e + 3])};
                *reinterpret_cast<u32x2*>(q + 16 * ((n >> 3) ^ (row & (chunks - 1))) + 8 * h) = v;
            }
    }
    __syncthreads();
#pragma unroll 4
    for (int q = threadIdx.x; q < S::BM * chunks; q += S::threads) {
        const int row = q / chunks, ch = q % chunks;
        const int64_t m = m0 + row, n = n0 + 8 * ch;
        if (m >= M || n >= cols) continue;
        const u32x4 v = *reinterpret_cast<const u32x4*>(part(row) + 16 * (ch ^ (row & (chunks - 1))));
        E* o = out + m * ldo + n;
        if (n + 8 <= cols) {
            *reinterpret_cast<u32x4_e*>(o) = v;
        } else {
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (n + r < cols) o[r].u = (uint16_t)(v[r >> 1] >> (16 * (r & 1)));
        }
    }
}

template <typename T, typename S, bool AA, bool BA, int EPI>
__global__ __launch_bounds__(S::threads, 2) void product(const Args g) {
    typedef Tile<T, S::BM, S::threads, AA> TA;
    typedef Tile<T, S::BN, S::threads, BA> TB;
    // four arrays: the compiler sees that loads into one pair do not meet the reads of the other
    __shared__ alignas(16) char a0[TA::bytes], b0[TB::bytes], a1[TA::bytes], b1[TB::bytes];
    __shared__ float2 part[EPI == kStats ? S::WN : 1][S::BM];  // a wave's (maximum, sum) of a row
    constexpr bool kLines = sizeof(T) == 2 && S::TM * S::TN > 1;
    static_assert(!kLines || (TA::bytes == 64 * S::BN * 2 && TB::bytes == TA::bytes), "64 rows an array");
    // neighbouring workgroups go to the eight dies in turn: each die takes one run of tiles, in groups of 8 rows of tiles
    const int64_t total = (int64_t)gridDim.x;
    int64_t id = blockIdx.x;
    {
        const int64_t per = total / 8, more = total % 8, x = id % 8;
        id = x * per + (x < more ? x : more) + id / 8;
    }
    const int64_t tiles = g.tiles_m * g.tiles_n, split = id / tiles;
    id -= split * tiles;
    const int64_t band = 8 * g.tiles_n, first = id / band * 8;
    const int64_t high = g.tiles_m - first < 8 ? g.tiles_m - first : 8;
    const int64_t tm = first + id % band % high, tn = id % band / high;
    const int64_t m0 = tm * S::BM, n0 = tn * S::BN;
    constexpr int BK = TA::BK;
    const int64_t steps_all = (g.K + BK - 1) / BK;
    const int64_t s0 = steps_all * split / g.splits, s1 = steps_all * (split + 1) / g.splits;
    const int64_t k1 = s1 * BK < g.K ? s1 * BK : g.K;
    TA ta;
    TB tb;
    ta.init(g.a, g.lda, m0, g.M, s0 * BK, k1);
    tb.init(g.b, g.ldb, n0, g.N, s0 * BK, k1);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, h = lane >> 5;
    const int wm = wave / S::WN * (32 * S::TM), wn = wave % S::WN * (32 * S::TN);
    f32x16 c[S::TM][S::TN];
#pragma unroll
    for (int i = 0; i < S::TM; ++i)
#pragma unroll
        for (int j = 0; j < S::TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) c[i][j][e] = 0.f;
    ta.load(a0);
    tb.load(b0);
    __syncthreads();
    // two steps a turn; what is loaded behind the last one are zeros
    for (int64_t t = s0; t < s1; t += 2) {
        ta.load(a1);
        tb.load(b1);
        one_step<T, S, TA, TB>(a0, b0, wm, wn, c);
        __syncthreads();
        if (t + 1 < s1) {
            ta.load(a0);
            tb.load(b0);
            one_step<T, S, TA, TB>(a1, b1, wm, wn, c);
            __syncthreads();
        }
    }
    // A lane holds row lane % 32 of each of its tiles, columns 8 (e / 4) + 4 h + e % 4.
    if constexpr (EPI == kStats) {
        T* kept = static_cast<T*>(g.out);
        if constexpr (sizeof(T) == 4)
            if (kept) store_direct<S>(c, kept, g.ldo, g.N, false, g.M, m0, n0 + wn, wm);
        const int64_t limit = g.N - n0;
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
            const int row = wm + 32 * i + (lane & 31);
            const int64_t m = m0 + row;
            const int64_t id = m < g.M ? (int64_t)g.ids[m] - n0 : -1;
            if (__any(id >= wn && id < wn + 32 * S::TN)) {  // few waves hold a target
#pragma unroll
                for (int j = 0; j < S::TN; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (wn + 32 * j + 8 * (e >> 2) + 4 * h + (e & 3) == id) {
                            g.target[m] = c[i][j][e];
                            c[i][j][e] = -INFINITY;  // the statistics are the other classes'
                        }
            }
            if (limit < S::BN) {
#pragma unroll
                for (int j = 0; j < S::TN; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (wn + 32 * j + 8 * (e >> 2) + 4 * h + (e & 3) >= limit) c[i][j][e] = -INFINITY;
            }
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, c[i][j][e]);
            top = fmaxf(top, __shfl_xor(top, 32));
            if (h == 0) part[wave % S::WN][row].x = top;
        }
        __syncthreads();
        const auto top_of = [&](int row) {
            float t = part[0][row].x;
#pragma unroll
            for (int w = 1; w < S::WN; ++w) t = fmaxf(t, part[w][row].x);
            return t;
        };
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
            const int row = wm + 32 * i + (lane & 31);
            // a row of -inf alone: sum 0, and NaN where one of them is NaN, which the maximum passes over
            const float top = top_of(row), base = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    c[i][j][e] = exp_neg<T>(c[i][j][e] - base);
                    sum += c[i][j][e];
                }
            sum += __shfl_xor(sum, 32);
            if (h == 0) part[wave % S::WN][row].y = sum;
        }
        if constexpr (kLines) {
            if (kept) store_lines<S, true>(c, a0, b0, a1, b1, kept, g.ldo, g.cols, g.M, m0, n0, wm, wn);
            else __syncthreads();
        } else {
            if constexpr (sizeof(T) == 2)
                if (kept) store_direct<S, true>(c, kept, g.ldo, g.cols, false, g.M, m0, n0 + wn, wm);
            __syncthreads();
        }
        for (int row = threadIdx.x; row < S::BM; row += S::threads) {
            if (m0 + row >= g.M) continue;
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < S::WN; ++w) sum += part[w][row].y;
            g.stats[tn * g.M + m0 + row] = make_float2(top_of(row), sum);
        }
    } else if constexpr (EPI == kSlab) {
        store_direct<S>(c, g.slab + split * g.M * g.N, g.N, g.N, g.add != 0, g.M, m0, n0 + wn, wm);
    } else if constexpr (kLines) {
        store_lines<S, false>(c, a0, b0, a1, b1, static_cast<T*>(g.out), g.ldo, g.cols, g.M, m0, n0, wm, wn);
    } else {
        store_direct<S>(c, static_cast<T*>(g.out), g.ldo, g.cols, false, g.M, m0, n0 + wn, wm);
    }
}

template <typename T, typename S, bool AA, bool BA, int EPI>
void go_shape(Args g, int64_t splits, hipStream_t st) {
    g.tiles_m = (g.M + S::BM - 1) / S::BM;
    g.tiles_n = (g.N + S::BN - 1) / S::BN;
    g.splits = splits;
    launch(product<T, S, AA, BA, EPI>, dim3((uint32_t)(g.tiles_m * g.tiles_n * splits)), dim3(S::threads), 0, st, g);
}
template <typename T, bool AA, bool BA, int EPI>
void go(const Args& g, Size size, int64_t splits, hipStream_t st) {
    if (size == kLarge) {
        if constexpr (sizeof(T) == 2) go_shape<T, Large, AA, BA, EPI>(g, splits, st);
    } else if (size == kSmall || !AA) go_shape<T, Small, AA, BA, EPI>(g, splits, st);
    else if constexpr (AA) go_shape<T, Thin, AA, BA, EPI>(g, splits, st);
}

// ---- the rows before and after ------------------------------------------------------------------------------------
// Rows of src as rows of a whole number of 16-byte chunks, zeros past their end; with ids, each row's target and weight,
// and zeros for a row that counts for nothing, so that nothing it holds meets a product.
template <typename T, bool ROWS>
__global__ __launch_bounds__(256) void pack(const T* src, int64_t ld, int64_t n, int D, T* dst, int64_t ldd,
                                            const int32_t* ids, const float* w, int V, int32_t* target, float* coef) {
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (row >= n) return;
    const int lane = threadIdx.x & 63;
    bool live = true;
    if constexpr (ROWS) {
        const int id = ids[row];
        const float c = w ? w[row] : 1.f;
        live = c != 0.f && id >= 0 && id < V;
        if (lane == 0) {
            target[row] = live ? id : (c == 0.f || id == -1 ? -1 : -2);
            coef[row] = live ? c : 0.f;
        }
    }
    constexpr int E = Width<T>::v;
    for (int64_t d = (int64_t)lane * E; d < ldd; d += 64 * E) {
        T* o = dst + row * ldd + d;
        if (live && d + E <= D) {
            *reinterpret_cast<u32x4*>(o) = *reinterpret_cast<const u32x4_e*>(src + row * ld + d);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const float one[1] = {live && d + e < D ? load_raw<1>(src + row * ld + d + e)[0] : 0.f};
                store_vec<1>(o + e, one);
            }
        }
    }
}

// A row's tiles joined, 8 rows by 32 groups of tiles a workgroup: each group's own, then the groups of a wave, then the waves,
// then the target. Leaves the loss and, for `grad`, the row's maximum, the inverse of its sum below it, and the target's p - 1
// (where its logit was).
__global__ __launch_bounds__(256) void join(const float2* stats, int64_t tiles, int64_t N, float* own,
                                            const int32_t* target, const float* coef, float2* norm, float* loss) {
    __shared__ float2 part[4][8];
    const int r = threadIdx.x & 7, grp = threadIdx.x >> 3;
    const int64_t n = (int64_t)blockIdx.x * 8 + r;
    float2 p = make_float2(-INFINITY, 0.f);
    if (n < N) {
        constexpr int U = 4;  // loads at once
        for (int64_t t = grp; t < tiles; t += 32 * U) {
            float2 q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = t + 32 * u < tiles ? stats[(t + 32 * u) * N + n] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int u = 0; u < U; ++u) p = joined(p, q[u]);
        }
    }
#pragma unroll
    for (int m = 8; m < 64; m *= 2) p = joined(p, make_float2(__shfl_xor(p.x, m), __shfl_xor(p.y, m)));
    if ((threadIdx.x & 63) < 8) part[threadIdx.x >> 6][r] = p;
    __syncthreads();
    if (grp != 0 || n >= N) return;
    for (int i = 1; i < 4; ++i) p = joined(p, part[i][r]);
    const int id = target[n];
    if (id < 0) {
        norm[n] = make_float2(0.f, 0.f);
        own[n] = 0.f;
        loss[n] = id == -1 ? 0.f : NAN;
        return;
    }
    // NaN and +inf among the logits, and -inf in all of them, make one of the exponentials NaN, and with it everything
    const float z = own[n], top = fmaxf(p.x, z);
    const float others = p.y * exp_neg<float>(p.x - top), t = exp_neg<float>(z - top), sum = others + t;
    norm[n] = make_float2(top, 1.f / sum);
    own[n] = -others / sum;
    loss[n] = coef[n] * (z >= p.x ? log1pf(others * t) : p.x - z + logf(sum));
}

// G of a block of rows over what is kept of its logits, eight neighbours a thread; zeros past the classes.
struct GradArgs {
    int64_t ld, rows;
    int V, tile;               // classes a tile of the statistics
    const float2* stats;
    const float2* norm;
    const float *coef, *own;
    const int32_t* target;
};
template <typename T>
__global__ __launch_bounds__(256) void grad(const GradArgs a, T* G) {
    const uint32_t per = (uint32_t)(a.ld / 8), i = blockIdx.x * 256u + threadIdx.x, m = i / per;
    if (m >= a.rows) return;
    const int v = (int)(i - m * per) * 8, id = a.target[m];
    const float2 row = a.norm[m];
    const float k = a.coef[m];
    T* p = G + m * a.ld + v;
    float x[8];
    if constexpr (sizeof(T) == 4) {
        load_f32<8>(p, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = exp_neg<T>(x[e] - row.x) * row.y;
    } else {
        typedef _Float16 h8 __attribute__((ext_vector_type(8)));
        const h8 q = __builtin_bit_cast(h8, *reinterpret_cast<const u32x4*>(p));
        const float f = exp_neg<T>(a.stats[v / a.tile * a.rows + m].x - row.x) * row.y * (1.f / kHalfScale);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)q[e] * f;
    }
    const float own = id >= v && id < v + 8 ? a.own[m] : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = k == 0.f || v + e >= a.V ? 0.f : k * (v + e == id ? own : x[e]);
    if constexpr (sizeof(T) == 4) {
        store_f32<8>(p, x);
    } else {
        *reinterpret_cast<u32x4*>(p) = u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    }
}

template <typename T>
__global__ __launch_bounds__(256) void clear(T* p, int64_t n) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const float one[1] = {0.f};
    if (i < n) store_vec<1>(p + i, one);
}

// out = sum of the slabs, in their order
template <typename T, int V>
__global__ __launch_bounds__(256) void sum_slabs(const float* slab, int slabs, int64_t M, int64_t N, T* out, int64_t ldo) {
    const int64_t per = (N + V - 1) / V, i = (int64_t)blockIdx.x * 256 + threadIdx.x, m = i / per, n = i % per * V;
    if (m >= M) return;
    float v[V];
#pragma unroll
    for (int r = 0; r < V; ++r) v[r] = 0.f;
    const float* p = slab + m * N + n;
#pragma unroll 8
    for (int s = 0; s < slabs; ++s) {
        float x[V];
        load_f32<V>(p + s * M * N, x);
#pragma unroll
        for (int r = 0; r < V; ++r) v[r] += x[r];
    }
    if constexpr (V == 1) {
        store_vec<1>(out + m * ldo + n, v);
    } else if constexpr (sizeof(T) == 4) {
        store_vec<4>(out + m * ldo + n, v);
    } else {
        typedef u32x2 u32x2_e __attribute__((aligned(2), may_alias));
        *reinterpret_cast<u32x2_e*>(out + m * ldo + n) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    }
}
template <typename T>
void go_sum(const float* slab, int64_t slabs, int64_t M, int64_t N, T* out, int64_t ldo, hipStream_t st) {
    const int V = N % 4 == 0 ? 4 : 1;
    const dim3 grid((uint32_t)((M * (N / V) + 255) / 256));
    if (V == 4) launch(sum_slabs<T, 4>, grid, dim3(256), 0, st, slab, slabs, M, N, out, ldo);
    else launch(sum_slabs<T, 1>, grid, dim3(256), 0, st, slab, slabs, M, N, out, ldo);
}

// ---- plan ---------------------------------------------------------------------------------------------------------
int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

struct Cut {
    Size size;
    int64_t splits;  // parts of the depth, whose sums are joined afterwards
};
// How a product is cut. Thin tiles for few rows, where those of 128 would spend most of their products on rows that are not
// there, which fp32 feels first, and for few tiles whose depth is not split. Otherwise what an estimate of the time says: a
// compute unit takes one of the larger tiles at a time or two small ones, rounds come out even or not, a part of the depth
// costs its sums' way to memory and back, a round its loads' latency and its results. In fp32 the small tiles are as fast as
// the larger ones (4096 x 2048 over 32000: 12.0 ms both when they were compared) and leave less of the last round idle (19795 x 1664 over 4193: 6.8
// ms, 8.9 in the larger ones), so that the larger ones are bfloat16's alone (dh of 4096 x 2048 over 32000: 495 us in 2 parts
// of larger tiles, 600 in small ones).
Cut cut_of(int64_t M, int64_t N, int64_t K, int e, bool along, bool split) {
    const int64_t steps = (K * e + 127) / 128;
    const auto tiles_of = [&](int64_t b) { return ((M + b - 1) / b) * ((N + b - 1) / b); };
    const int64_t small = tiles_of(128), most = split ? std::max<int64_t>(1, steps / 2) : 1;
    if (along && (M <= (e == 4 ? 64 : 32) || small * most < 128)) {
        const int64_t tiles = ((M + 31) / 32) * ((N + 127) / 128);
        return {kThin, split ? std::max<int64_t>(1, std::min<int64_t>({512 / tiles, most, int64_t(128)})) : 1};
    }
    Cut best{kSmall, 1};
    double least = 1e300;
    const auto look = [&](Size size, int64_t tiles, double rate, double round, int64_t n) {
        const double b = size == kLarge ? 256 : 128;
        const int64_t t = tiles * n, rest = t % 512;
        const double rounds = size == kLarge ? (double)((t + 255) / 256) : (double)(t / 512) * 2 + (rest > 256 ? 2. : rest > 0 ? 1.3 : 0.);
        const double sums = n > 1 ? 5e-6 + 8. * (double)n * (double)M * (double)N / 5e12 : 0.;
        const double cost = rounds * (2. * b * b * (double)K / (double)n / (rate / 256) + round) + sums;
        if (cost < least) {
            least = cost;
            best = {size, n};
        }
    };
    for (const int64_t n : {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 16, 20, 24, 32, 48, 64, 96, 128}) {
        if (n > most) break;
        look(kSmall, small, e == 2 ? 0.85e15 : 1.35e14, 1.5e-6, n);
        if (e == 2 && M > 128 && N > 128 && steps / n > 3) look(kLarge, tiles_of(256), 1.1e15, 3e-6, n);
    }
    return best;
}

}  // namespace

// rows of a tile times a row's bytes stay inside the 31 bits of a buffer's offsets: 256 rows of 2^20 fp32 logits are 2^30
int64_t vocab_max_classes() { return int64_t(1) << 20; }
int vocab_max_d() { return 1 << 16; }

// Workspace: the hidden states as they meet the products, the weights too where their rows are no whole number of chunks,
// the tiles' statistics, a row's numbers, and with gradients G of a block of rows, dh's slabs and dW's.
VocabPlan vocab_plan(int64_t N, int D, int V, int dtype, bool grads) {
    const int e = dtype == 1 ? 2 : 4, chunk = 16 / e;
    constexpr int64_t kMB = int64_t(1) << 20;
    VocabPlan p;
    p.ldh = up(D, chunk);
    p.pack_w = D % chunk != 0;
    p.rows = std::max<int64_t>(N, 1);
    p.ldg = up(V, 8);
    grads = grads && N > 0;
    int64_t blocks = 1;
    if (grads) {  // G of up to 256 MB, or 1024 rows (fp32, whose products are ten times as dear: 128)
        const int64_t fit = std::max<int64_t>(256 * kMB / e / V / 128 * 128, e == 4 ? 128 : 1024);
        blocks = (N + fit - 1) / fit;
        p.rows = std::min(N, up((N + blocks - 1) / blocks, 128));
    }
    p.tiles = (V + 127) / 128;  // at most
    // 256 threads a tile of 128 x 128 logits: the loss alone of very many rows takes several launches
    if (!grads) p.rows = std::min<int64_t>(p.rows, kMaxLaunchThreads / 256 / p.tiles * 128);
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    p.h = take((size_t)N * p.ldh * e);
    p.w = take(p.pack_w ? (size_t)V * p.ldh * e : 0);
    p.stats = take((size_t)p.tiles * p.rows * sizeof(float2));
    p.norm = take((size_t)N * 8);
    p.target_logit = take((size_t)N * 4);
    p.target = take((size_t)N * 4);
    p.coef = take((size_t)N * 4);
    if (grads) {
        const Cut dh = cut_of(p.rows, D, V, e, true, true), dw = cut_of(V, D, p.rows, e, false, true);
        p.dh_size = dh.size;
        p.dh_splits = dh.splits;
        p.dw_size = dw.size;
        p.dw_splits = dw.splits;
        p.g = take((size_t)p.rows * p.ldg * e);
        p.dh = take(p.dh_splits > 1 ? (size_t)p.dh_splits * p.rows * D * 4 : 0);
        p.dw_slab = p.dw_splits > 1 || (e == 2 && blocks > 1);  // (blocks of fp32 add up in dW itself)
        p.dw = take(p.dw_slab ? (size_t)p.dw_splits * V * D * 4 : 0);
    }
    p.total = at;
    return p;
}

namespace {

template <typename T>
struct Vocab {
    const VocabArgs& x;
    const VocabPlan& p;
    char* ws;
    const T* W;  // rows of ldh
    hipStream_t st;

    template <typename U>
    U* at(size_t o, int64_t i = 0) const {
        return reinterpret_cast<U*>(ws + o) + i;
    }
    // losses of rows r0 .., and G of them where there are gradients
    void losses(int64_t r0, int64_t rows, bool grads) const {
        Args a{};
        a.a = at<T>(p.h, r0 * p.ldh);
        a.b = W;
        a.lda = a.ldb = p.ldh;
        a.M = rows;
        a.N = x.V;
        a.K = x.D;
        a.ids = at<int32_t>(p.target, r0);
        a.stats = at<float2>(p.stats);
        a.target = at<float>(p.target_logit, r0);
        if (grads) a.out = at<T>(p.g);
        a.ldo = a.cols = p.ldg;
        const Size s = cut_of(rows, x.V, x.D, sizeof(T), true, false).size;
        go<T, true, true, kStats>(a, s, 1, st);
        const int tile = s == kLarge ? 256 : 128;
        const float* coef = at<float>(p.coef, r0);
        float2* norm = at<float2>(p.norm, r0);
        launch(join, dim3((uint32_t)((rows + 7) / 8)), dim3(256), 0, st, a.stats, (int64_t)((x.V + tile - 1) / tile), rows, a.target,
               a.ids, coef, norm, x.loss + r0);
        if (!grads) return;
        const GradArgs g{p.ldg, rows, x.V, tile, a.stats, norm, coef, a.target, a.ids};
        launch(grad<T>, dim3((uint32_t)((rows * (p.ldg / 8) + 255) / 256)), dim3(256), 0, st, g, at<T>(p.g));
    }
    // G of rows r0 .. into dh, and into dW, which is a sum over the blocks of rows
    void take(int64_t r0, int64_t rows) const {
        Args b{};
        b.a = at<T>(p.g);
        b.b = W;
        b.lda = p.ldg;
        b.ldb = p.ldh;
        b.M = rows;
        b.N = x.D;
        b.K = x.V;
        T* dh = static_cast<T*>(x.dh) + r0 * x.lddh;
        b.out = dh;
        b.ldo = x.lddh;
        b.cols = x.D;
        b.slab = at<float>(p.dh);
        const Size sh = (Size)p.dh_size;
        if (p.dh_splits > 1) {
            go<T, true, false, kSlab>(b, sh, p.dh_splits, st);
            go_sum(b.slab, p.dh_splits, rows, x.D, dh, x.lddh, st);
        } else {
            go<T, true, false, kStore>(b, sh, 1, st);
        }

        const bool first = r0 == 0, last = r0 + rows == x.N;
        Args c{};
        c.a = at<T>(p.g);
        c.b = at<T>(p.h, r0 * p.ldh);
        c.lda = p.ldg;
        c.ldb = p.ldh;
        c.M = x.V;
        c.N = x.D;
        c.K = rows;
        T* dW = static_cast<T*>(x.dW);
        c.out = dW;
        c.ldo = c.cols = x.D;
        c.add = !first;
        const Size sw = (Size)p.dw_size;
        if (p.dw_slab) {
            c.slab = at<float>(p.dw);
            go<T, false, false, kSlab>(c, sw, p.dw_splits, st);
            if (last) go_sum(c.slab, p.dw_splits, x.V, x.D, dW, x.D, st);
        } else if (!(first && last)) {  // fp32: dW is its own slab
            c.slab = reinterpret_cast<float*>(dW);
            go<T, false, false, kSlab>(c, sw, 1, st);
        } else {
            go<T, false, false, kStore>(c, sw, 1, st);
        }
    }

    void run(bool grads) const {
        for (int64_t r0 = 0; r0 < x.N; r0 += p.rows) {
            const int64_t rows = std::min(p.rows, x.N - r0);
            losses(r0, rows, grads);
            if (grads) take(r0, rows);
        }
    }
};

template <typename T>
hipError_t vocab_loss(const VocabArgs& x, int dtype, void* ws, hipStream_t st) {
    const bool grads = x.dW != nullptr;
    if (x.N == 0) {
        const int64_t n = (int64_t)x.V * x.D;
        if (grads) launch(clear<T>, dim3((uint32_t)((n + 255) / 256)), dim3(256), 0, st, static_cast<T*>(x.dW), n);
        return hipGetLastError();
    }
    const VocabPlan p = vocab_plan(x.N, x.D, x.V, dtype, grads);
    Vocab<T> v{x, p, static_cast<char*>(ws), static_cast<const T*>(x.W), st};
    launch(pack<T, true>, dim3((uint32_t)((x.N + 3) / 4)), dim3(256), 0, st, static_cast<const T*>(x.h), x.ldh, x.N, x.D,
           v.template at<T>(p.h), p.ldh, x.ids, x.w, x.V, v.template at<int32_t>(p.target), v.template at<float>(p.coef));
    if (p.pack_w) {
        T* to = v.template at<T>(p.w);
        launch(pack<T, false>, dim3((uint32_t)((x.V + 3) / 4)), dim3(256), 0, st, v.W, (int64_t)x.D, (int64_t)x.V, x.D, to, p.ldh,
               static_cast<const int32_t*>(nullptr), static_cast<const float*>(nullptr), 0, static_cast<int32_t*>(nullptr),
               static_cast<float*>(nullptr));
        v.W = to;
    }
    v.run(grads);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_vocab(const VocabArgs& x, int dtype, void* ws, hipStream_t st) {
    return dtype == 1 ? vocab_loss<bf16>(x, dtype, ws, st) : vocab_loss<float>(x, dtype, ws, st);
}

}  // namespace mdl
