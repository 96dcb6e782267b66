// k_vocab.hip — softmax cross entropy over a vocabulary from the hidden states and the class weights, with its gradients,
// without the logits in memory.
//
//   z = h W^T,  loss_n = w_n (ln sum_c exp z_nc - z_n,id),  G = w (softmax z - [c = id]),  dh = G W,  dW = G^T h
//
// A first product leaves per row and 256 (or 128) classes their maximum and sum of exponentials, and the target's logit;
// `join` makes the losses of them. What the gradients then need of the logits is held for a piece of them at a time, in one of two
// ways. Logits kept: the first product, a block of rows at a time, also writes the block's logits (fp32),
// `grad` makes G of them, and two products take G into dh and dW: 6 N V D operations. Logits formed again: behind the first
// product over all rows, piece of the vocabulary by piece, a second one of the same operands forms G of the piece, and two
// more take it into dh and dW: 8 N V D operations, but nothing is written that is not G. Kept are they where one block takes
// all rows, and for fp32 always, whose products are the dearer half: 4096 x 2048 over 32000 classes in fp32 takes 15.6 ms
// with the logits formed again. Several blocks in bfloat16 would have dW's sums read and written once a block.
//
// Products: tiles of BM x BN by 8 (4) waves, 32 x 32 results of the matrix instructions (32x32x16 bfloat16, 32x32x2 fp32),
// 128 bytes of depth at a time from global memory straight into LDS, one step ahead of the products. An operand whose rows
// run along the depth is laid row by row, its 16-byte chunks rotated by the row so that a wave's reads meet all banks; one
// whose rows run across it is laid as it comes and read by transposing reads (bfloat16) or word by word (fp32).
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
        static_assert(!ALONG || THREADS % 64 == 0, "whole groups of eight rows between a thread's chunks");
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
        at = 16 * (threadIdx.x % 8 ^ (threadIdx.x / 8 & 7));
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
            return *reinterpret_cast<const u32x4*>(lds + r * 128 + 16 * ((2 * s + (lane >> 5)) ^ (r & 7)));
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
    float* logits;                // [M] at ldo, or null
    float *target, *lse;          // [M]
    const int32_t* ids;           // [M] -1: none
    const float* coef;            // [M]
    int64_t n_first;              // class of column 0
    void* out;
    int64_t ldo, cols;            // cols: columns that are written (zeros past N)
    float* slab;                  // [splits][M][N]
    int add;                      // onto what the slab holds
};

enum { kStats, kGrad, kStore, kSlab };

// A wave's tiles as they lie, four neighbours of a row a lane; onto what is there with `add` (fp32 alone).
template <typename S, typename E>
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
                    const u32x2 q = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
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

template <typename T, typename S, bool AA, bool BA, int EPI>
__global__ __launch_bounds__(S::threads, 2) void product(const Args g) {
    typedef Tile<T, S::BM, S::threads, AA> TA;
    typedef Tile<T, S::BN, S::threads, BA> TB;
    // four arrays: the compiler sees that loads into one pair do not meet the reads of the other
    __shared__ alignas(16) char a0[TA::bytes], b0[TB::bytes], a1[TA::bytes], b1[TB::bytes];
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
        if (g.logits) store_direct<S>(c, g.logits, g.ldo, g.N, false, g.M, m0, n0 + wn, wm);
        float2* part = reinterpret_cast<float2*>(a0);  // [WN][BM]; all reads of the tiles are done
        const int64_t limit = g.N - n0;
#pragma unroll
        for (int i = 0; i < S::TM; ++i) {
            const int row = wm + 32 * i + (lane & 31);
            const int64_t m = m0 + row;
            const int64_t id = m < g.M ? (int64_t)g.ids[m] - n0 : -1;
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int n = wn + 32 * j + 8 * (e >> 2) + 4 * h + (e & 3);
                    if (n >= limit) c[i][j][e] = -INFINITY;
                    if (n == id) g.target[m] = c[i][j][e];
                    top = fmaxf(top, c[i][j][e]);
                }
            top = fmaxf(top, __shfl_xor(top, 32));
            // a row of -inf alone: sum 0, and NaN where one of them is NaN, which the maximum passes over
            const float base = top == -INFINITY ? 0.f : top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < S::TN; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e) sum += exp_neg<T>(c[i][j][e] - base);
            sum += __shfl_xor(sum, 32);
            if (h == 0) part[wave % S::WN * S::BM + row] = make_float2(top, sum);
        }
        __syncthreads();
        for (int row = threadIdx.x; row < S::BM; row += S::threads) {
            if (m0 + row >= g.M) continue;
            float2 p = part[row];
#pragma unroll
            for (int w = 1; w < S::WN; ++w) p = joined(p, part[w * S::BM + row]);
            g.stats[tn * g.M + m0 + row] = p;
        }
    } else {
        if constexpr (EPI == kGrad) {
#pragma unroll
            for (int i = 0; i < S::TM; ++i) {
                const int64_t m = m0 + wm + 32 * i + (lane & 31);
                const float lse = m < g.M ? g.lse[m] : 0.f, coef = m < g.M ? g.coef[m] : 0.f;
                const int64_t id = m < g.M ? (int64_t)g.ids[m] - g.n_first - n0 : -1;
#pragma unroll
                for (int j = 0; j < S::TN; ++j)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int n = wn + 32 * j + 8 * (e >> 2) + 4 * h + (e & 3);
                        const float p = exp_neg<T>(c[i][j][e] - lse) - (n == id ? 1.f : 0.f);
                        c[i][j][e] = coef == 0.f || n0 + n >= g.N ? 0.f : coef * p;
                    }
            }
        }
        if constexpr (sizeof(T) == 2 && EPI != kSlab && S::TM * S::TN > 1) {
            // Through LDS, so that whole lines leave: a quarter (half) of the tile's rows in each array, their 16-byte
            // chunks rotated by the row.
            constexpr int chunks = S::BN / 8;
            static_assert(TA::bytes == 64 * S::BN * 2 && TB::bytes == TA::bytes, "64 rows an array");
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
                        const u32x2 v = {pack_bf16(c[i][j][e], c[i][j][e + 1]), pack_bf16(c[i][j][e + 2], c[i][j][e + 3])};
                        *reinterpret_cast<u32x2*>(q + 16 * ((n >> 3) ^ (row & (chunks - 1))) + 8 * h) = v;
                    }
            }
            __syncthreads();
#pragma unroll 4
            for (int q = threadIdx.x; q < S::BM * chunks; q += S::threads) {
                const int row = q / chunks, ch = q % chunks;
                const int64_t m = m0 + row, n = n0 + 8 * ch;
                if (m >= g.M || n >= g.cols) continue;
                const u32x4 v = *reinterpret_cast<const u32x4*>(part(row) + 16 * (ch ^ (row & (chunks - 1))));
                T* o = static_cast<T*>(g.out) + m * g.ldo + n;
                if (n + 8 <= g.cols) {
                    *reinterpret_cast<u32x4_e*>(o) = v;
                } else {
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        if (n + r < g.cols) o[r].u = (uint16_t)(v[r >> 1] >> (16 * (r & 1)));
                }
            }
        } else {
            if constexpr (EPI == kSlab)
                store_direct<S>(c, g.slab + split * g.M * g.N, g.N, g.N, g.add != 0, g.M, m0, n0 + wn, wm);
            else
                store_direct<S>(c, static_cast<T*>(g.out), g.ldo, g.cols, false, g.M, m0, n0 + wn, wm);
        }
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
    if (size == kLarge) go_shape<T, Large, AA, BA, EPI>(g, splits, st);
    else if (size == kSmall || !AA) go_shape<T, Small, AA, BA, EPI>(g, splits, st);
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

// A row's tiles joined, 8 rows by 32 groups of tiles a workgroup.
__global__ __launch_bounds__(256) void join(const float2* stats, int64_t tiles, int64_t N, const float* target_logit,
                                            const int32_t* target, const float* coef, float* lse, float* loss) {
    __shared__ float2 part[32][8];
    const int r = threadIdx.x & 7, grp = threadIdx.x >> 3;
    const int64_t n = (int64_t)blockIdx.x * 8 + r;
    float2 p = make_float2(-INFINITY, 0.f);
    if (n < N)
        for (int64_t t = grp; t < tiles; t += 32) p = joined(p, stats[t * N + n]);
    part[grp][r] = p;
    __syncthreads();
    if (grp != 0 || n >= N) return;
    for (int i = 1; i < 32; ++i) p = joined(p, part[i][r]);
    const float l = p.x + logf(p.y);
    lse[n] = l;
    const int id = target[n];
    loss[n] = id >= 0 ? coef[n] * (l - target_logit[n]) : (id == -1 ? 0.f : NAN);
}

// G of a block of rows from its logits, eight neighbours a thread; zeros past the classes. fp32: over the logits.
template <typename T>
__global__ __launch_bounds__(256) void grad(const float* z, int64_t ld, int64_t rows, int V, const float* lse, const float* coef,
                                            const int32_t* target, T* out) {
    const uint32_t per = (uint32_t)(ld / 8), i = blockIdx.x * 256u + threadIdx.x, m = i / per;
    if (m >= rows) return;
    const int v = (int)(i - m * per) * 8, id = target[m];
    const float l = lse[m], k = coef[m];
    float x[8];
    load_f32<8>(z + m * ld + v, x);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] = k == 0.f || v + e >= V ? 0.f : k * (exp_neg<T>(x[e] - l) - (v + e == id ? 1.f : 0.f));
    T* o = out + m * ld + v;
    if constexpr (sizeof(T) == 4) {
        store_f32<8>(o, x);
    } else {
        *reinterpret_cast<u32x4*>(o) = u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
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

// The larger tiles where they fill the compute units; the thin ones for few rows, where those of 128 would spend most of
// their products on rows that are not there, which fp32 feels first, and for few tiles whose depth is not split.
Size size_of(int64_t M, int64_t N, int64_t K, int e, bool along, bool split) {
    if (along && M <= (e == 4 ? 64 : 32)) return kThin;
    const bool fills = ((M + 255) / 256) * ((N + 255) / 256) >= 192;
    if (fills && M > 128 && N > 128 && K * e > 3 * 128) return kLarge;
    const int64_t small = ((M + 127) / 128) * ((N + 127) / 128) * (split ? std::max<int64_t>(1, K * e / 128 / 2) : 1);
    return along && small < 128 ? kThin : kSmall;
}
// how often the depth is split where there are few tiles: so that some 512 workgroups share the work, none with less than
// two steps of it
int64_t splits_of(int64_t M, int64_t N, int64_t K, int e, bool along) {
    const Size size = size_of(M, N, K, e, along, true);
    if (size == kLarge) return 1;
    const int64_t bm = size == kThin ? 32 : 128, tiles = ((M + bm - 1) / bm) * ((N + 127) / 128), steps = (K * e + 127) / 128;
    return std::max<int64_t>(1, std::min<int64_t>({512 / tiles, steps / 2, int64_t(128)}));
}

}  // namespace

// rows of a tile times a row's bytes stay inside the 31 bits of a buffer's offsets: 256 rows of 2^20 fp32 logits are 2^30
int64_t vocab_max_classes() { return int64_t(1) << 20; }
int vocab_max_d() { return 1 << 16; }

// Workspace: the hidden states as they meet the products, the weights too where their rows are no whole number of chunks,
// the tiles' statistics, a row's numbers, and with gradients a block of logits or a piece of G (or both), dh's slabs and dW's.
VocabPlan vocab_plan(int64_t N, int D, int V, int dtype, bool grads) {
    const int e = dtype == 1 ? 2 : 4, chunk = 16 / e;
    constexpr int64_t kMB = int64_t(1) << 20;
    VocabPlan p;
    p.ldh = up(D, chunk);
    p.pack_w = D % chunk != 0;
    p.rows = std::max<int64_t>(N, 1);
    p.piece = up(V, 256);
    grads = grads && N > 0;
    if (grads) {
        // logits of up to 256 MB; in bfloat16 they cost 8 bytes of traffic each beside G's, and formed again 2 D operations:
        // as much at some 800 channels, unless all of it stays in the caches
        const int64_t fit = std::max<int64_t>(256 * kMB / 4 / V / 128 * 128, 128);
        p.keep = e == 4 || (N <= fit && (D >= 768 || N * V * 4 <= 32 * kMB));
        if (p.keep) {
            const int64_t blocks = (N + fit - 1) / fit;
            p.rows = std::min(N, up((N + blocks - 1) / blocks, 128));
            p.piece = up(V, 8);
        } else {  // at least 2048 classes
            p.piece = std::min(p.piece, std::max<int64_t>(2048, 128 * kMB / (N * e) / 256 * 256));
            const int64_t pieces = (V + p.piece - 1) / p.piece;
            p.piece = up((V + pieces - 1) / pieces, 256);
        }
    }
    p.tiles = (V + 127) / 128;  // at most
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    p.h = take((size_t)N * p.ldh * e);
    p.w = take(p.pack_w ? (size_t)V * p.ldh * e : 0);
    p.stats = take((size_t)p.tiles * p.rows * sizeof(float2));
    p.lse = take((size_t)N * 4);
    p.target_logit = take((size_t)N * 4);
    p.target = take((size_t)N * 4);
    p.coef = take((size_t)N * 4);
    if (grads) {
        const int64_t cols = std::min<int64_t>(p.piece, V);
        p.dh_splits = splits_of(p.rows, D, cols, e, true);
        p.dw_splits = splits_of(cols, D, p.rows, e, false);
        p.logits = take(p.keep ? (size_t)p.rows * p.piece * 4 : 0);
        p.g = p.keep && e == 4 ? p.logits : take((size_t)p.rows * p.piece * e);
        p.dh_slab = p.dh_splits > 1 || cols < V;
        p.dh = take(p.dh_slab ? (size_t)p.dh_splits * p.rows * D * 4 : 0);
        p.dw = take(p.dw_splits > 1 ? (size_t)p.dw_splits * cols * D * 4 : 0);
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
    // the logits of rows r0 .. against classes v0 ..
    Args logits(int64_t r0, int64_t rows, int64_t v0, int64_t cols) const {
        Args a{};
        a.a = at<T>(p.h, r0 * p.ldh);
        a.b = W + v0 * p.ldh;
        a.lda = a.ldb = p.ldh;
        a.M = rows;
        a.N = cols;
        a.K = x.D;
        a.ids = at<int32_t>(p.target, r0);
        a.n_first = v0;
        a.ldo = p.piece;
        return a;
    }
    Size size(const Args& a) const { return size_of(a.M, a.N, a.K, sizeof(T), true, false); }  // of the logits
    // losses of rows r0 .., their logits kept where there is a place for them
    void losses(int64_t r0, int64_t rows, bool keep) const {
        Args a = logits(r0, rows, 0, x.V);
        a.stats = at<float2>(p.stats);
        a.target = at<float>(p.target_logit, r0);
        if (keep) a.logits = at<float>(p.logits);
        const Size s = size(a);
        go<T, true, true, kStats>(a, s, 1, st);
        const int64_t tiles = (x.V + (s == kLarge ? 255 : 127)) / (s == kLarge ? 256 : 128);
        launch(join, dim3((uint32_t)((rows + 7) / 8)), dim3(256), 0, st, a.stats, tiles, rows, a.target, a.ids,
               at<float>(p.coef, r0), at<float>(p.lse, r0), x.loss + r0);
    }
    // G of rows r0 .. and classes v0 .. is at p.g: into dh (first, last: of the pieces) and dW (the same, of the blocks)
    void take(int64_t r0, int64_t rows, int64_t v0, int64_t cols, bool first_piece, bool last_piece, bool first_block,
              bool last_block) const {
        const T* G = at<T>(p.g);
        Args b{};
        b.a = G;
        b.b = W + v0 * p.ldh;
        b.lda = p.piece;
        b.ldb = p.ldh;
        b.M = rows;
        b.N = x.D;
        b.K = cols;
        T* dh = static_cast<T*>(x.dh) + r0 * x.lddh;
        b.out = dh;
        b.ldo = x.lddh;
        b.cols = x.D;
        b.slab = at<float>(p.dh);
        b.add = !first_piece;
        const Size sh = size_of(p.rows, x.D, std::min<int64_t>(p.piece, x.V), sizeof(T), true, true);
        if (p.dh_slab) go<T, true, false, kSlab>(b, sh, p.dh_splits, st);
        else go<T, true, false, kStore>(b, sh, 1, st);
        if (p.dh_slab && last_piece) go_sum(b.slab, p.dh_splits, rows, x.D, dh, x.lddh, st);

        Args c{};
        c.a = G;
        c.b = at<T>(p.h, r0 * p.ldh);
        c.lda = p.piece;
        c.ldb = p.ldh;
        c.M = cols;
        c.N = x.D;
        c.K = rows;
        T* dW = static_cast<T*>(x.dW) + v0 * x.D;
        c.out = dW;
        c.ldo = x.D;
        c.cols = x.D;
        c.add = !first_block;
        const Size sw = size_of(std::min<int64_t>(p.piece, x.V), x.D, p.rows, sizeof(T), false, true);
        if (p.dw_splits > 1) {
            c.slab = at<float>(p.dw);
            go<T, false, false, kSlab>(c, sw, p.dw_splits, st);
            if (last_block) go_sum(c.slab, p.dw_splits, cols, x.D, dW, x.D, st);
        } else if (sizeof(T) == 4 && !(first_block && last_block)) {
            c.slab = reinterpret_cast<float*>(dW);  // blocks are several in fp32 alone: dW is its own slab
            go<T, false, false, kSlab>(c, sw, 1, st);
        } else {
            go<T, false, false, kStore>(c, sw, 1, st);
        }
    }

    void run(bool grads) const {
        if (!p.keep) losses(0, x.N, false);
        if (!grads) return;
        if (p.keep) {
            for (int64_t r0 = 0; r0 < x.N; r0 += p.rows) {
                const int64_t rows = std::min(p.rows, x.N - r0);
                losses(r0, rows, true);
                const int64_t n = rows * (p.piece / 8);
                launch(grad<T>, dim3((uint32_t)((n + 255) / 256)), dim3(256), 0, st, at<float>(p.logits), p.piece, rows, x.V,
                       at<float>(p.lse, r0), at<float>(p.coef, r0), at<int32_t>(p.target, r0), at<T>(p.g));
                take(r0, rows, 0, x.V, true, true, r0 == 0, r0 + rows == x.N);
            }
            return;
        }
        for (int64_t v0 = 0; v0 < x.V; v0 += p.piece) {
            const int64_t cols = std::min<int64_t>(p.piece, x.V - v0);
            Args a = logits(0, x.N, v0, cols);
            a.lse = at<float>(p.lse);
            a.coef = at<float>(p.coef);
            a.out = at<T>(p.g);
            a.cols = up(cols, 16 / (int64_t)sizeof(T));
            go<T, true, true, kGrad>(a, size(a), 1, st);
            take(0, x.N, v0, cols, v0 == 0, v0 + cols == x.V, true, true);
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
