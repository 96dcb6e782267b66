// k_linattn.hip — linear attention with a decay for each head over packed sequences, gfx950.
//
// Per head, with d its decay, and R the state [Da][Dc] (float32):
//     R_t = b_t c_t^T + d R_{t-1},   out_t = a_t^T R_t
// The forward is (a, b, c) = (q, k, v). All gradients are the same recurrence again: dq is (dy, v, k) in the forward's
// order, on the transposed states; dv is (k, q, dy) and dk is (v, dy, q), both against the forward's order, on one state
// (the gradient of the forward's) and its transpose. In blocks of C tokens i, j = 0.. after an entering state E:
//     out_i = sum_{j <= i} d^{i-j} (a_i . b_j) c_j + d^{i+1} a_i^T E,   E' = d^n E + sum_j d^{n-1-j} b_j c_j^T
// (one power less on E and one more on E' where the entering state is that of the token itself: the gradients).
//
// Sequences are cut into tiles of L tokens, each taken by a workgroup a head. Three launches: `states` forms what each tile
// adds to the state (to the slot of its boundary with the next tile in scan order, or to the last states), `chain` walks each
// sequence's boundaries and leaves in each slot the state that enters the tile behind it, `outputs` walks the tiles block by
// block. No tile waits for another. The slots of the forward stand in the workspace for the backward's dq.
//
// Which tile a workgroup has follows from the offsets alone, with nothing summed over the sequences: sequence s owns the
// numbers from off[s] / L + s on, which are at least as many as its tiles (those behind them have nothing to do), and its
// boundaries the slots from off[s] / L on, which are as many as it can need; T / L + S numbers and T / L slots in all.
//
// What bounds it. bfloat16: memory. Both ways over 4 documents (208246 tokens, 8 heads of 128 + 128) move each tensor 18 times
// (426 MB each; states 2, outputs 4, states 2, dv and dk 6, dq 4) where 8 would do, in 1.91 to 1.94 ms: 222 + 402 + 217 + 665 +
// 405 us and two chains of 19, 3.8 to 4.3 TB/s, the matrix units busy for 19 to 30 % of the cycles. fp32 with heads of 50 (656603
// tokens, 1024 sequences): the matrix units, busy for 50 % of them in the outputs (192 + 392 + 196 us of 942 in all; 64 x 64
// padded, products whose depth is a head's channels run 16 steps of 4 where 13 hold values).
//
// Heads are padded to 64 or 128 channels, so narrow ones cost what 64 do: 20597 tokens of 8 heads, both ways, take 119, 108 and
// 115 us for heads of 8, 16 and 32 in bfloat16 (140 for 64) and 301, 252 and 281 in fp32 (305 for 64).
#include "kernels.h"
#include "seqio.h"

#include <algorithm>

namespace mdl {

namespace {

constexpr int kThreads = 256;  // of chain and step, and of the four waves that share a block's products
__device__ inline int thread_id() { return (int)threadIdx.x & (kThreads - 1); }

typedef __bf16 bh8 __attribute__((ext_vector_type(8)));
typedef short h4 __attribute__((ext_vector_type(4)));

// ---- operands of the matrix instructions ------------------------------------------------------------------------
// A Quad holds four values of one row of a 16 x 16 tile, at the columns 4 g + 0..3 of lane group g = lane / 16 for row
// lane % 16: the layout in which the 16 x 16 forms also leave their results (with rows and columns exchanged), so that a
// result tile is an operand of the next product as it lies. mma2 multiplies over two tiles' depth.
template <typename T>
struct Op;
template <>
struct Op<bf16> {
    typedef u32x2 Quad;
    static constexpr int C = 32;  // tokens a block
    static __device__ inline Quad make(f32x4 v) { return Quad{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])}; }
    static __device__ inline f32x4 values(Quad q) {
        return f32x4{__uint_as_float(q[0] << 16), __uint_as_float(q[0] & 0xffff0000u), __uint_as_float(q[1] << 16),
                     __uint_as_float(q[1] & 0xffff0000u)};
    }
    // out[m][n] += sum over the two tiles' depth of x[m][.] y[n][.]
    static __device__ inline f32x4 mma2(f32x4 c, Quad x0, Quad x1, Quad y0, Quad y1) {
        const u32x4 x = {x0[0], x0[1], x1[0], x1[1]}, y = {y0[0], y0[1], y1[0], y1[1]};
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bh8, x), __builtin_bit_cast(bh8, y), c, 0, 0, 0);
    }
};
template <>
struct Op<float> {
    typedef f32x4 Quad;
    static constexpr int C = 32;
    static __device__ inline Quad make(f32x4 v) { return v; }
    static __device__ inline f32x4 values(Quad q) { return q; }
    static __device__ inline f32x4 mma2(f32x4 c, Quad x0, Quad x1, Quad y0, Quad y1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x0[r], y0[r], c, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x1[r], y1[r], c, 0, 0, 0);
        return c;
    }
};

// A head's decay d, as its powers take it: log2 |d| and the sign. The instruction is within 1 ulp of log2 over all of
// [1/4, 1), near 1 too (every float was tried).
struct Decay {
    float l2;
    uint32_t sign;
};
__device__ inline Decay decay_of(float d) { return {__builtin_amdgcn_logf(fabsf(d)), __float_as_uint(d) & 0x80000000u}; }
// d^e for whole e >= 0: d^0 is 1 also for d = 0, and odd powers of a decay below 0 are
__device__ inline float power(Decay d, int e) {
    const float m = e == 0 ? 1.f : __builtin_amdgcn_exp2f((float)e * d.l2);
    return __uint_as_float(__float_as_uint(m) ^ ((uint32_t)e << 31 & d.sign));
}

// a value that all lanes share, in a scalar register
__device__ inline float uniform(float x) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// What a kernel of this file works on.
struct Args {
    const int64_t* off;
    int S, H;
    int64_t T;
    int L;                     // tokens a tile
    double inv_l;              // 1 / L
    int dir;                   // +1: tokens ascending, -1: descending
    int post;                  // 1: the entering state is the previous token's; 0: it is the token's own
    const float* decay;
    float pscale, sscale, oscale;  // of a . b, of b c^T in the state, of the output
    float* slots;              // [T / L][H][size], a tile boundary's state
    const float* init;         // [S][H][size] or null
    float* last;               // [S][H][size] or null
    int64_t size;              // elements of a state
    struct Side {
        const void *a, *b, *c; // [T][H][da or dc] at row strides
        int64_t lda, ldb, ldc;
        int da, dc, trans;     // states are stored [da][dc], or [dc][da]
        void* out;             // [T][H][dc]
        int64_t ldo;
    } side[2];
};

// offsets that leave [0, T] end there: whatever they hold, no tile leaves the tensors or the slots
__device__ inline int64_t offset(const Args& a, int64_t s) {
    const int64_t o = a.off[s];
    return o < 0 ? 0 : (o > a.T ? a.T : o);
}

// floor(x / L) for 0 <= x < 2^40: the product is off by less than one
__device__ inline int64_t over_l(const Args& a, int64_t x) {
    int64_t q = (int64_t)((double)x * a.inv_l);
    const int64_t r = x - q * a.L;
    q -= r < 0;
    q += r >= a.L;
    return q;
}

struct Tile {
    int seq;                   // -1: nothing to do
    int len;
    int64_t from;              // first token in scan order
    int64_t enter, leave;      // slots, or -1 where the sequence begins or ends with the tile
};
// The tile with this number: its sequence is the last one whose numbers begin no later (64 probes at a time, alike in every
// wave).
__device__ inline Tile tile_of(const Args& a, int64_t number) {
    int lo = 0, hi = a.S;
    const int lane = threadIdx.x & 63;
    while (lo < hi) {
        const int step = (int)(((int64_t)(hi - lo) + 63) / 64);
        const int64_t p = lo + (int64_t)lane * step;
        const uint64_t m = __ballot(p < hi && over_l(a, offset(a, p)) + p > number);
        if (m == 0) {
            lo += ((hi - lo - 1) / step) * step + 1;
        } else {
            const int f = __builtin_ctzll(m);
            hi = lo + f * step;
            if (f > 0) lo += (f - 1) * step + 1;
        }
    }
    Tile t;
    t.seq = lo - 1;
    if (t.seq < 0) return t;
    const int64_t o0 = offset(a, t.seq), o1 = offset(a, (int64_t)t.seq + 1), L = a.L;
    const int64_t slot = number - t.seq, begin = o0 + (slot - over_l(a, o0)) * L;
    if (begin >= o1) t.seq = -1;
    const int64_t end = begin + L < o1 ? begin + L : o1;
    const int64_t before = begin > o0 ? slot - 1 : -1, after = end < o1 ? slot : -1;
    t.len = (int)(end - begin);
    t.from = a.dir > 0 ? begin : end - 1;
    t.enter = a.dir > 0 ? before : after;
    t.leave = a.dir > 0 ? after : before;
    return t;
}

// ---- blocks of rows ---------------------------------------------------------------------------------------------
// An LDS tile of C rows of D elements, in whose rows the 16-byte chunks change places with the row, so that reads of 16 rows
// spread over the banks; nothing lies between the rows, as the loads that go straight to LDS need it. fp32 has hardly any
// conflicts left (0 to 0.2 cycles an LDS instruction), bfloat16 2.0 in `states` and 2.6 to 2.8 in `outputs`: an order that
// took these down to 0 and 1.6 left the kernels' times as they were and was not kept.
template <typename T, int D>
struct Plane {
    typedef typename Op<T>::Quad Quad;
    static constexpr int E = sizeof(T), C = Op<T>::C, row_bytes = D * E, bytes = C * row_bytes;
    static __device__ inline int turn(int r) { return row_bytes == 128 ? r >> 1 & 7 : r & 15; }
    // the place of byte c of row r
    static __device__ inline int at(int r, int c) { return r * row_bytes + (((c >> 4) ^ turn(r)) << 4) + (c & 15); }
    // A lane's reads: of row i = lane % 16, columns 4 g .., and of column i, rows 4 g .. (bfloat16: by a transposing read, in
    // which each group of 16 lanes names 4 rows of 16 values), at the tile of 16 x 16 from row0, col0 on: what col0 adds to the
    // place is a change of some of its chunk's bits. The places are found again for each block (the constructor's lane is
    // taken as new): kept, they would take some twenty registers.
    int by_row, by_col;
    __device__ inline Plane() {
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int g = lane >> 4, i = lane & 15;
        by_row = at(i, 4 * g * E);
        by_col = E == 2 ? at(4 * g + (i >> 2), 4 * (i & 3) * E) : at(4 * g, i * E);
    }
    __device__ inline Quad row(const char* t, int row0, int col0) const {
        return *reinterpret_cast<const Quad*>(t + row0 * row_bytes + (by_row ^ (col0 * E)));
    }
    __device__ inline Quad col(const char* t, int row0, int col0) const {
        if constexpr (E == 2) {
            typedef __attribute__((address_space(3))) h4* P;
            const char* p = t + row0 * row_bytes + (by_col ^ (col0 * E));
            return __builtin_bit_cast(Quad, __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p)));
        } else {
            Quad q;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                q[e] = *reinterpret_cast<const float*>(t + (row0 + e) * row_bytes + (by_col ^ (col0 * E) ^ (e << 4)));
            return q;
        }
    }
};

constexpr uint32_t kOut = 0x80000000u;  // an offset past every buffer's end: the load gives zeros

// n rows of d elements from `first` on in scan order to a plane, zero outside: what lies behind a sequence or beside a head
// never meets a product. ld: bytes, below 2^25, so that a block's offsets have 31 bits.
// DIRECT: straight to LDS, 16 bytes a lane; rows start and end at multiples of it.
// Else staged in registers (load) and then laid (lay), any alignment. Every lane loads, without a branch: past the rows the
// last one, which is laid as zeros, past the row its last 16 bytes, which end with it and are laid there again; the columns
// past d stay as `zero_fill` left them. Heads of less than 16 bytes go element by element.
template <typename T, int D, bool DIRECT>
struct Rows {
    typedef Plane<T, D> P;
    static constexpr int C = Op<T>::C, E = sizeof(T), n = P::bytes / (kThreads * 16);
    static_assert(P::bytes % (kThreads * 16) == 0, "whole loads a thread");
    __device__ inline void load(const T* base, int64_t ld, int64_t first, int dir, int rows, int d, char* to) {
        const char* low = reinterpret_cast<const char*>(base) + (dir > 0 ? first : first - (C - 1)) * ld;
        const __amdgpu_buffer_rsrc_t buf = rsrc(low, 0x7fffffff);
        int tid = thread_id();
        if constexpr (n > 2) asm volatile("" : "+v"(tid));  // many loads: their places are found again, not kept
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const int q = (i * kThreads + tid) * 16, r = q / P::row_bytes, at = q % P::row_bytes;
            const int c = ((at >> 4) ^ P::turn(r)) << 4;
            const uint32_t o = (uint32_t)(dir > 0 ? r : C - 1 - r) * (uint32_t)ld + (uint32_t)c;
            const int off = (int)(r < rows && c < d * E ? o : kOut);
            char* l = to + (i * kThreads + (thread_id() & ~63)) * 16;  // of the wave
            typedef __attribute__((address_space(3))) void* L;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (L)l, 16, off, 0, 0, 0);
        }
    }
};
template <typename T, int D>
struct Rows<T, D, false> {
    typedef Plane<T, D> P;
    static constexpr int V = Width<T>::v, per = D / V, C = Op<T>::C, n_vec = C * per / kThreads;
    static_assert(n_vec >= 1 && C * per % kThreads == 0, "whole vectors a thread");
    u32x4 q[n_vec];
    __device__ inline void load(const T* base, int64_t ld, int64_t first, int dir, int n, int d, char*) {
        const char* low = reinterpret_cast<const char*>(base) + (dir > 0 ? first : first - (n - 1)) * ld;
        const int col = thread_id() % per * V, c0 = d < V ? 0 : min(col, d - V);
#pragma unroll
        for (int i = 0; i < n_vec; ++i) {
            const int r = min((i * kThreads + thread_id()) / per, n - 1);
            const uint32_t o = (uint32_t)(dir > 0 ? r : n - 1 - r) * (uint32_t)ld + (uint32_t)(c0 * sizeof(T));
            if (d >= V) {
                q[i] = *reinterpret_cast<const u32x4_e*>(low + o);
            } else {
                q[i] = u32x4{0, 0, 0, 0};
                if (col == 0)
                    for (int e = 0; e < d; ++e) {
                        if constexpr (sizeof(T) == 2) {
                            const uint32_t v = *reinterpret_cast<const uint16_t*>(low + o + 2 * e);
                            q[i][e >> 1] |= v << (16 * (e & 1));
                        } else {
                            q[i][e] = *reinterpret_cast<const uint32_t*>(low + o + 4 * e);
                        }
                    }
            }
        }
    }
    __device__ inline void lay(char* t, int n, int d) const {
        const int col = thread_id() % per * V;
#pragma unroll
        for (int i = 0; i < n_vec; ++i) {
            const int r = (i * kThreads + thread_id()) / per;
            const bool in = r < n;
            const u32x4 v = {in ? q[i][0] : 0, in ? q[i][1] : 0, in ? q[i][2] : 0, in ? q[i][3] : 0};
            if (col + V <= d || (d < V && col == 0)) {
                *reinterpret_cast<u32x4*>(t + P::at(r, col * (int)sizeof(T))) = v;
            } else if (col < d) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    char* p = t + P::at(r, (d - V + e) * (int)sizeof(T));
                    if constexpr (sizeof(T) == 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
                    else *reinterpret_cast<uint32_t*>(p) = v[e];
                }
            }
        }
    }
};
__device__ inline void zero_fill(char* t, int bytes) {
    for (int i = 16 * thread_id(); i < bytes; i += 16 * kThreads) *reinterpret_cast<u32x4*>(t + i) = u32x4{0, 0, 0, 0};
}

// All waves of the workgroup meet here: with what they wrote to LDS done, and (ALL) their loads to LDS, which an ordinary
// barrier would wait for at either place. The waits' counters: 0xC07F lgkmcnt(0), 0x0070 vmcnt(0) and lgkmcnt(0).
template <bool ALL>
__device__ inline void meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(ALL ? 0x0070 : 0xC07F);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A head's sizes: four waves, with a quarter of the state's columns each.
template <typename T, int DA_, int DC_, bool DIRECT_>
struct Head {
    typedef T type;
    typedef Op<T> O;
    static constexpr bool DIRECT = DIRECT_;
    static constexpr int DA = DA_, DC = DC_, C = O::C, CT = C / 16, NT = DC / 64, waves = 4;
    // waves a SIMD that the registers are to allow: of workgroups of four waves, so many a compute unit. (`outputs` with two
    // sides of wide heads has eight waves and 156 registers: one workgroup. fp32 outputs of 128 + 128 channels fill all 256
    // registers and keep 8 more in scratch.)
    static constexpr int occupancy = DA + DC == 128 ? 4 : !DIRECT && (DA + DC > 192 || sizeof(T) == 4) ? 2 : 3;
    typedef Plane<T, DA> PA;
    typedef Plane<T, DC> PC;
    typedef Rows<T, DA, DIRECT> RA;
    typedef Rows<T, DC, DIRECT> RC;
    static constexpr int sp = C * (int)sizeof(T) + 16;  // bytes between the rows of a block's products
};
// ---- states -----------------------------------------------------------------------------------------------------
// A wave's 16 NT columns of the state: result tiles of 16 x 16, rows 16 t + 4 g + r, columns 16 u + lane % 16.
template <int DA, int NT>
struct State {
    static constexpr int AT = DA / 16;
    f32x4 x[AT][NT];
    __device__ inline void clear() {
#pragma unroll
        for (int t = 0; t < AT; ++t)
#pragma unroll
            for (int u = 0; u < NT; ++u) x[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    __device__ inline void scale(float f) {
#pragma unroll
        for (int t = 0; t < AT; ++t)
#pragma unroll
            for (int u = 0; u < NT; ++u) x[t][u] *= f;
    }
    // (the lane is taken as new at each call, or else the elements' places would be kept in registers from the start)
    __device__ inline void load(const Args::Side& a, const float* p) {
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int g = lane >> 4, n0 = (thread_id() >> 6) * (16 * NT) + (lane & 15);
        const bool quads = a.trans && a.da % 4 == 0;  // they lie as they are held
        const int sm = a.trans ? 1 : a.dc, sn = a.trans ? a.da : 1;
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const int n = n0 + 16 * u;
            const bool in = n < a.dc;
            const float* q = p + (uint32_t)(min(n, a.dc - 1) * sn);
            if (quads) {
#pragma unroll
                for (int t = 0; t < AT; ++t) {
                    const int m = 16 * t + 4 * g;
                    const f32x4 v = *reinterpret_cast<const f32x4_e*>(q + min(m, a.da - 4));
                    const bool k = in && m < a.da;
                    x[t][u] = f32x4{k ? v[0] : 0.f, k ? v[1] : 0.f, k ? v[2] : 0.f, k ? v[3] : 0.f};
                }
            } else {
#pragma unroll
                for (int t = 0; t < AT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int m = 16 * t + 4 * g + r;
                        const float v = q[(uint32_t)(min(m, a.da - 1) * sm)];
                        x[t][u][r] = in && m < a.da ? v : 0.f;
                    }
            }
            one_at_a_time();
        }
    }
    __device__ inline void store(const Args::Side& a, float* p) const {
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));
        const int g = lane >> 4, n0 = (thread_id() >> 6) * (16 * NT) + (lane & 15);
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const int n = n0 + 16 * u;
            if (n >= a.dc) continue;
#pragma unroll
            for (int t = 0; t < AT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int m = 16 * t + 4 * g + r;
                    if (m < a.da) p[(uint32_t)(m * a.dc + n)] = x[t][u][r];
                }
        }
    }
};

// x += sum over the block's rows j of b_j f_j c_j^T, f(t) the weights of rows 16 t + 4 g ..; PARTS: how many bfloat16 terms
// f c is taken as (one for fp32)
template <typename Hd, int PARTS, typename F>
__device__ inline void add_block(State<Hd::DA, Hd::NT>& s, const char* B, const char* Cv, F f) {
    typedef typename Hd::O O;
    constexpr int JT = Hd::CT, NT = Hd::NT;
    const int n0 = __builtin_amdgcn_readfirstlane(thread_id() >> 6) * (16 * NT);
    const typename Hd::PA pb;
    const typename Hd::PC pc;
    typename O::Quad w[PARTS][JT][NT];
#pragma unroll
    for (int t = 0; t < JT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            f32x4 v = O::values(pc.col(Cv, 16 * t, n0 + 16 * u)) * f(t);
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                w[p][t][u] = O::make(v);
                if (p + 1 < PARTS) v -= O::values(w[p][t][u]);
            }
        }
#pragma unroll
    for (int m = 0; m < Hd::DA / 16; ++m) {
#pragma unroll
        for (int t = 0; t < JT; t += 2) {
            const auto b0 = pb.col(B, 16 * t, 16 * m), b1 = pb.col(B, 16 * t + 16, 16 * m);
#pragma unroll
            for (int u = 0; u < NT; ++u)
#pragma unroll
                for (int p = 0; p < PARTS; ++p) s.x[m][u] = O::mma2(s.x[m][u], b0, b1, w[p][t][u], w[p][t + 1][u]);
        }
    }
}

// What each tile adds to its sequence's state. bfloat16: f c is split into three terms (24 bits, as fp32 has), so that the
// states are sums of fp32 products.
template <typename T, int DA, int DC, bool DIRECT>
__global__ __launch_bounds__(kThreads, (DIRECT ? 4 : Head<T, DA, DC, DIRECT>::occupancy)) void states(const Args a) {
    typedef Head<T, DA, DC, DIRECT> Hd;
    constexpr int C = Hd::C, PARTS = sizeof(T) == 2 ? 3 : 1, nb = Hd::PA::bytes, nc = Hd::PC::bytes;
    // two sets of planes, of which the compiler sees that loads into one do not meet the reads of the other
    __shared__ alignas(16) char t0[nb + nc], t1[DIRECT ? nb + nc : 16];
    const Tile t = tile_of(a, blockIdx.x / (uint32_t)a.H);
    if (t.seq < 0 || (t.leave < 0 && !a.last)) return;
    const int h = blockIdx.x % (uint32_t)a.H, g = (threadIdx.x & 63) >> 4;
    const Args::Side& side = a.side[0];
    const int da = side.da, dc = side.dc;
    const T* pb = static_cast<const T*>(side.b) + (int64_t)h * da;
    const T* pc = static_cast<const T*>(side.c) + (int64_t)h * dc;
    const int64_t ldb = side.ldb * (int64_t)sizeof(T), ldc = side.ldc * (int64_t)sizeof(T);
    typename Hd::RA rb;
    typename Hd::RC rc;
    const auto load = [&](int k, char* to) {
        const int n = min(C, t.len - k);
        rb.load(pb, ldb, t.from + a.dir * k, a.dir, n, da, to);
        rc.load(pc, ldc, t.from + a.dir * k, a.dir, n, dc, to + nb);
    };
    load(0, t0);
    const Decay d = decay_of(a.decay[h]);
    State<DA, Hd::NT> x;
    x.clear();
    const auto add = [&](int k, const char* p) {
        const int n = min(C, t.len - k);
        if (k > 0) x.scale(power(d, n));
        add_block<Hd, PARTS>(x, p, p + nb, [&](int q) {
            f32x4 f;
#pragma unroll
            for (int r = 0; r < 4; ++r) f[r] = a.sscale * power(d, max(n - a.post - (16 * q + 4 * g + r), 0));
            return f;
        });
    };
    if constexpr (DIRECT) {
        for (int k = 0; k < t.len; k += 2 * C) {
            meet<true>();
            if (k + C < t.len) load(k + C, t1);
            add(k, t0);
            if (k + C < t.len) {
                meet<true>();
                if (k + 2 * C < t.len) load(k + 2 * C, t0);
                add(k + C, t1);
            }
        }
    } else {
        zero_fill(t0, nb + nc);
        for (int k = 0; k < t.len; k += C) {
            const int n = min(C, t.len - k);
            __syncthreads();
            rb.lay(t0, n, da);
            rc.lay(t0 + nb, n, dc);
            if (k + C < t.len) load(k + C, t0);
            __syncthreads();
            add(k, t0);
        }
    }
    x.store(side, t.leave >= 0 ? a.slots + (t.leave * a.H + h) * a.size : a.last + ((int64_t)t.seq * a.H + h) * a.size);
}

// Per sequence, head and V state elements: the boundaries in scan order, eight read ahead.
template <int V>
__global__ __launch_bounds__(kThreads) void chain(const Args a, int blocks_per_head) {
    const int64_t id = blockIdx.x;
    const int eb = (int)(id % blocks_per_head), h = (int)(id / blocks_per_head % a.H);
    const int64_t s = id / blocks_per_head / a.H, e = ((int64_t)eb * kThreads + threadIdx.x) * V;
    if (e >= a.size) return;
    const int64_t o0 = offset(a, s), o1 = offset(a, s + 1), at = (s * a.H + h) * a.size + e;
    float x[V];
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = 0.f;
    if (a.init) load_f32<V>(a.init + at, x);
    if (o0 >= o1) {
        if (a.last) store_f32<V>(a.last + at, x);
        return;
    }
    const int64_t L = a.L, base = over_l(a, o0), end = over_l(a, o1 - o0 - 1);
    const Decay d = decay_of(a.decay[h]);
    const float whole = power(d, (int)L);
    const int64_t hop = a.dir * a.H * a.size;
    // all tiles but the sequence's last one are whole
    const int rest = (int)(o1 - o0 - end * L), lead = end > 0 ? (int)L : rest;
    float* p = a.slots + ((a.dir > 0 ? base : base + end - 1) * a.H + h) * a.size + e;
    float f = power(d, a.dir > 0 ? lead : rest), v[V];
    constexpr int U = 8;
    for (int64_t i = 0; i < end; i += U) {
        float w[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < end) load_f32<V>(p + u * hop, w[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < end) {
#pragma unroll
                for (int j = 0; j < V; ++j) x[j] = __builtin_fmaf(x[j], f, w[u][j]);
                store_f32<V>(p + u * hop, x);
                f = whole;
            }
        p += U * hop;
    }
    if (a.last) {
        load_f32<V>(a.last + at, v);
        f = power(d, a.dir > 0 ? rest : lead);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = __builtin_fmaf(x[j], f, v[j]);
        store_f32<V>(a.last + at, v);
    }
}

template <typename T>
__device__ inline void store_quad(T* p, f32x4 v, int n) {
    if constexpr (sizeof(T) == 2) {
        typedef u32x2 u32x2_e __attribute__((aligned(2), may_alias));
        const u32x2 q = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        if (n >= 4) *reinterpret_cast<u32x2_e*>(p) = q;
        else
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < n) p[r].u = (uint16_t)(q[r >> 1] >> (16 * (r & 1)));
    } else {
        if (n >= 4) *reinterpret_cast<f32x4_e*>(p) = v;
        else
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < n) p[r] = v[r];
    }
}

// The tiles' outputs, block by block. bfloat16 roundings on the way: of (a . b) d^{i-j} before its product with c, of the
// entering state before its product with a, and of f c before it is added to the state that is handed on within the tile
// (two terms there); each is half a step of values that reach the output as a sum with its own half step. Sums and states
// are fp32.
//
// SIDES 2: two outputs of one tile at once, by four waves each, where the second's b is the first's c and its c the first's b
// (dv and dk, whose states are each other's transposes): four tensors are read instead of six.
template <typename T, int DA, int DC, bool DIRECT, int SIDES>
__global__ __launch_bounds__(SIDES * kThreads, (SIDES == 2 && DA > 64 ? 2 : Head<T, DA, DC, DIRECT>::occupancy)) void outputs(const Args a) {
    typedef Head<T, DA, DC, DIRECT> Hd;
    typedef typename Hd::O O;
    typedef typename O::Quad Quad;
    typedef typename Hd::PA PA;
    typedef typename Hd::PC PC;
    static_assert(SIDES == 1 || DA == DC, "one side's c is the other's b");
    constexpr int C = Hd::C, CT = Hd::CT, NT = Hd::NT, PARTS = sizeof(T) == 2 ? 2 : 1, sp = Hd::sp;
    // [a][b] a side, then c (SIDES 2: the other side's b); two sets, of which the compiler sees that loads into one do not
    // meet the reads of the other
    constexpr int na = PA::bytes, per_side = 2 * na, all = SIDES * per_side + (SIDES == 1 ? PC::bytes : 0);
    __shared__ alignas(16) char t0[all], t1[DIRECT ? all : 16], products[SIDES * C * sp];
    const Tile tile = tile_of(a, blockIdx.x / (uint32_t)a.H);
    if (tile.seq < 0) return;
    const int h = blockIdx.x % (uint32_t)a.H;
    const int sd = SIDES == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
    const int wave = __builtin_amdgcn_readfirstlane(thread_id() >> 6);
    const int lane = threadIdx.x & 63, g = lane >> 4, i = lane & 15;
    const Args::Side& side = a.side[sd];
    const int own = sd * per_side, at_c = SIDES == 1 ? per_side : (1 - sd) * per_side + na;
    char* lp = products + sd * C * sp;
    const int da = side.da, dc = side.dc;
    const T* pa = static_cast<const T*>(side.a) + (int64_t)h * da;
    const T* pb = static_cast<const T*>(side.b) + (int64_t)h * da;
    const T* pc = static_cast<const T*>(side.c) + (int64_t)h * dc;
    const int64_t lda = side.lda * (int64_t)sizeof(T), ldb = side.ldb * (int64_t)sizeof(T), ldc = side.ldc * (int64_t)sizeof(T);
    char* po = reinterpret_cast<char*>(static_cast<T*>(side.out) + (int64_t)h * dc);
    const int64_t ldo = side.ldo * (int64_t)sizeof(T);
    const bool whole = dc % 4 == 0;
    typename Hd::RA ra, rb;
    typename Hd::RC rc;
    const auto load = [&](int k, char* to) {
        const int n = min(C, tile.len - k);
        const int64_t f = tile.from + a.dir * k;
        ra.load(pa, lda, f, a.dir, n, da, to + own);
        rb.load(pb, ldb, f, a.dir, n, da, to + own + na);
        if constexpr (SIDES == 1) rc.load(pc, ldc, f, a.dir, n, dc, to + at_c);
    };
    load(0, t0);
    const float* enter = tile.enter >= 0 ? a.slots + (tile.enter * a.H + h) * a.size
                         : a.init ? a.init + ((int64_t)tile.seq * a.H + h) * a.size : nullptr;
    State<DA, NT> x;
    if (enter) x.load(side, enter);
    else x.clear();
    // d^e for the e that occur, in two factors: within 16 (a lane's) and of 16s
    const Decay d = decay_of(a.decay[h]);
    float d16[CT], row_f = power(d, i + a.post), near[4], far[4], left[4];
#pragma unroll
    for (int q = 0; q < CT; ++q) d16[q] = uniform(power(d, 16 * q));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int e = i - (4 * g + r);
        near[r] = e < 0 ? 0.f : a.pscale * power(d, e);
        far[r] = a.pscale * power(d, 16 + e);
        left[r] = a.sscale * power(d, 16 - a.post - (4 * g + r));
    }
    const float d_block = uniform(power(d, C));

    // (a_i . b_j) d^{i-j}: the tiles of 16 x 16 on and below the diagonal, the lowest rows first, dealt out to the waves; row
    // i at lane % 16, j at 4 g + r
    const auto multiply = [&](const char* set) {
        const char *la = set + own, *lb = la + na;
        constexpr int kPairs = CT * (CT + 1) / 2;
        static_assert(kPairs <= Hd::waves, "a tile a wave");
        if (wave >= kPairs) return;
        int it = CT - 1, jt = wave;
#pragma unroll
        for (int q = CT; q > 1; --q)
            if (it == q - 1 && jt >= q) {
                jt -= q;
                --it;
            }
        const PA plane;
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < DA; m += 32)
            v = O::mma2(v, plane.row(lb, 16 * jt, m), plane.row(lb, 16 * jt, m + 16), plane.row(la, 16 * it, m),
                        plane.row(la, 16 * it, m + 16));
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = it == jt && i < 4 * g + r ? 0.f : v[r] * (it == jt ? near[r] : far[r]);
        static_assert(CT == 2, "tiles are on the diagonal or next to it");
        *reinterpret_cast<Quad*>(lp + (16 * it + i) * sp + (16 * jt + 4 * g) * (int)sizeof(T)) = O::make(v);
    };
    const auto product_row = [&](int it, int jt) {
        return *reinterpret_cast<const Quad*>(lp + (16 * it + i) * sp + (16 * jt + 4 * g) * (int)sizeof(T));
    };
    // outputs: row i at lane % 16, columns 4 g + r of the wave's tiles; then the state behind the block
    const auto finish = [&](int k, const char* set) {
        const char *la = set + own, *lb = la + na, *lc = set + at_c;
        const PA plane;
        const PC plane_c;
        f32x4 o[CT][NT];
#pragma unroll
        for (int it = 0; it < CT; ++it)
#pragma unroll
            for (int u = 0; u < NT; ++u) o[it][u] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (k > 0 || enter) {
#pragma unroll
            for (int m = 0; m < DA / 16; m += 2) {
                Quad x0[NT], x1[NT];
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    x0[u] = O::make(x.x[m][u]);
                    x1[u] = O::make(x.x[m + 1][u]);
                }
#pragma unroll
                for (int it = 0; it < CT; ++it) {
                    const Quad a0 = plane.row(la, 16 * it, 16 * m), a1 = plane.row(la, 16 * it, 16 * m + 16);
#pragma unroll
                    for (int u = 0; u < NT; ++u) o[it][u] = O::mma2(o[it][u], x0[u], x1[u], a0, a1);
                }
            }
#pragma unroll
            for (int it = 0; it < CT; ++it)
#pragma unroll
                for (int u = 0; u < NT; ++u) o[it][u] *= row_f * d16[it];
        }
#pragma unroll
        for (int t = 0; t < CT; t += 2) {
            Quad c0[NT], c1[NT];
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                c0[u] = plane_c.col(lc, 16 * t, 16 * (NT * wave + u));
                c1[u] = plane_c.col(lc, 16 * t + 16, 16 * (NT * wave + u));
            }
#pragma unroll
            for (int it = t; it < CT; ++it) {
                const Quad p0 = product_row(it, t);
                // the tile past the diagonal is never written
                const Quad p1 = it > t ? product_row(it, t + 1) : O::make(f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int u = 0; u < NT; ++u) o[it][u] = O::mma2(o[it][u], c0[u], c1[u], p0, p1);
            }
        }
        char* q = po + (tile.from + a.dir * k) * ldo;
#pragma unroll
        for (int it = 0; it < CT; ++it) {
            const int row = 16 * it + i;
            if (row >= tile.len - k) continue;
            char* qr = q + (int64_t)(a.dir * row) * ldo;
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const int col = 16 * (NT * wave + u) + 4 * g;
                if (col < dc) store_quad<T>(reinterpret_cast<T*>(qr) + col, o[it][u] * a.oscale, whole ? 4 : dc - col);
            }
        }
        if (k + C < tile.len) {  // of a whole block
            x.scale(d_block);
            add_block<Hd, PARTS>(x, lb, lc, [&](int q) {
                return f32x4{left[0], left[1], left[2], left[3]} * d16[CT - 1 - q];
            });
        }
    };

    if constexpr (DIRECT) {
        for (int k = 0; k < tile.len; k += 2 * C) {
            meet<true>();
            if (k + C < tile.len) load(k + C, t1);
            multiply(t0);
            meet<false>();
            finish(k, t0);
            if (k + C < tile.len) {
                meet<true>();
                if (k + 2 * C < tile.len) load(k + 2 * C, t0);
                multiply(t1);
                meet<false>();
                finish(k + C, t1);
            }
        }
    } else {
        zero_fill(t0 + own, per_side);
        if constexpr (SIDES == 1) zero_fill(t0 + at_c, PC::bytes);
        for (int k = 0; k < tile.len; k += C) {
            const int n = min(C, tile.len - k);
            __syncthreads();
            ra.lay(t0 + own, n, da);
            rb.lay(t0 + own + na, n, da);
            if constexpr (SIDES == 1) rc.lay(t0 + at_c, n, dc);
            if (k + C < tile.len) load(k + C, t0);
            __syncthreads();
            multiply(t0);
            __syncthreads();
            finish(k, t0);
        }
    }
}

enum { kStates, kOutputs, kBothOutputs };
template <typename T, int DA, int DC, bool DIRECT>
hipError_t go(const Args& a, int what, hipStream_t st) {
    const dim3 grid((uint32_t)((a.T / a.L + a.S) * a.H));  // the heads of a tile side by side
    if (what == kStates) {
        launch(states<T, DA, DC, DIRECT>, grid, dim3(kThreads), 0, st, a);
    } else if (what == kOutputs) {
        launch(outputs<T, DA, DC, DIRECT, 1>, grid, dim3(kThreads), 0, st, a);
    } else {
        if constexpr (DA == DC) launch(outputs<T, DA, DC, DIRECT, 2>, grid, dim3(2 * kThreads), 0, st, a);
        else return hipErrorInvalidValue;
    }
    return hipGetLastError();
}
// Rows that start and end at multiples of 16 bytes go straight to LDS. Others are staged in registers, and so are fp32 heads
// wider than 64: two sets of planes would leave room for one workgroup. (At 656603 x 50 in fp32, heads of 50, 4 bytes a lane
// straight to LDS took longer than the registers' way.)
bool whole_chunks(const Args& a, int what, int e) {
    const auto fits = [&](const void* p, int64_t ld, int d) {
        return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * e % 16 == 0 && (int64_t)d * e % 16 == 0);
    };
    bool all = true;
    for (int i = 0; i < (what == kBothOutputs ? 2 : 1); ++i) {
        const Args::Side& s = a.side[i];
        all = all && (what == kStates || fits(s.a, s.lda, s.da)) && fits(s.b, s.ldb, s.da) && fits(s.c, s.ldc, s.dc);
    }
    return all;
}
template <typename T, int DA, int DC>
hipError_t go_wide(const Args& a, int what, hipStream_t st) {
    const bool chunks = whole_chunks(a, what, sizeof(T));
    if constexpr (sizeof(T) == 2) return chunks ? go<T, DA, DC, true>(a, what, st) : go<T, DA, DC, false>(a, what, st);
    else if constexpr (DA + DC == 128) return chunks ? go<T, DA, DC, true>(a, what, st) : go<T, DA, DC, false>(a, what, st);
    else return go<T, DA, DC, false>(a, what, st);
}
// the padded size of keys or values
constexpr int padded(int d) { return d <= 64 ? 64 : 128; }
template <typename T>
hipError_t go_sizes(const Args& a, int what, hipStream_t st) {
    const int da = padded(a.side[0].da), dc = padded(a.side[0].dc);
    if (da == 64) return dc == 64 ? go_wide<T, 64, 64>(a, what, st) : go_wide<T, 64, 128>(a, what, st);
    return dc == 64 ? go_wide<T, 128, 64>(a, what, st) : go_wide<T, 128, 128>(a, what, st);
}
hipError_t go_any(const Args& a, int dtype, int what, hipStream_t st) {
    return dtype == 1 ? go_sizes<bf16>(a, what, st) : go_sizes<float>(a, what, st);
}

int64_t chain_blocks(int64_t size) {
    const int64_t lanes = size % 4 == 0 ? size / 4 : size;
    return (lanes + kThreads - 1) / kThreads;
}
hipError_t go_chain(const Args& a, hipStream_t st) {
    const int per = (int)chain_blocks(a.size);
    const dim3 grid((uint32_t)((int64_t)a.S * a.H * per));
    if (a.size % 4 == 0) launch(chain<4>, grid, dim3(kThreads), 0, st, a, per);
    else launch(chain<1>, grid, dim3(kThreads), 0, st, a, per);
    return hipGetLastError();
}

// ---- one token of each stream -----------------------------------------------------------------------------------
// A workgroup takes one row's head: lanes along the state's columns (V of them a lane), the rows dealt out to the lane
// groups, each row read, advanced, written and taken into y. Bound by the state's bytes: 1024 streams of 8 x 128 x 128 (537 MB
// read, 537 written) take 206 to 224 us, 4.8 to 5.2 TB/s, a copy's rate. One stream of 8 x 64 x 64 takes 5 us.
struct StepArgs {
    int S, H, Dk, Dv, n_slots;
    const float* decay;
    float scale;
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv, ldy;
    const int32_t* slots;
    const float* h_in;
    float* h_out;
    void* y;
};
template <typename T, int V>
__global__ __launch_bounds__(kThreads) void step(const StepArgs a) {
    constexpr int kMaxD = 128, LC = V == 4 ? 32 : 128, G = kThreads / LC, RU = 8;  // lanes a row, row groups, rows at once
    __shared__ float lq[kMaxD], lk[kMaxD], lv[kMaxD], ly[G][LC * V + 4];
    const int h = blockIdx.x % a.H, row = blockIdx.x / a.H;
    const int slot = a.slots ? a.slots[row] : row;
    if (slot < 0 || slot >= a.n_slots) return;
    const int64_t at = ((int64_t)slot * a.H + h) * a.Dk * a.Dv;
    const float* in = a.h_in + at;
    float* out = a.h_out + at;
    const int t = threadIdx.x, col = t % LC * V, grp = t / LC;
    const auto value = [&](const void* p, int64_t ld, int d, int i) {
        return load_raw<1>(static_cast<const T*>(p) + row * ld + (int64_t)h * d + i)[0];
    };
    if (t < a.Dk) lq[t] = value(a.q, a.ldq, a.Dk, t);
    if (t >= kMaxD && t - kMaxD < a.Dk) lk[t - kMaxD] = value(a.k, a.ldk, a.Dk, t - kMaxD);
    if (t < a.Dv) lv[t] = value(a.v, a.ldv, a.Dv, t);
    const float d = a.decay[h];
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) y[j] = 0.f;
    const bool live = col < a.Dv;
    for (int m0 = 0; m0 < a.Dk; m0 += RU * G) {
        float x[RU][V];
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const int m = m0 + u * G + grp;
            if (live && m < a.Dk) load_f32<V>(in + m * a.Dv + col, x[u]);
        }
        if (m0 == 0) __syncthreads();
#pragma unroll
        for (int u = 0; u < RU; ++u) {
            const int m = m0 + u * G + grp;
            if (!live || m >= a.Dk) continue;
            const float k = lk[m], q = lq[m];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                x[u][j] = __builtin_fmaf(k, lv[col + j], d * x[u][j]);
                y[j] = __builtin_fmaf(q, x[u][j], y[j]);
            }
            store_f32<V>(out + m * a.Dv + col, x[u]);
        }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) ly[grp][col + j] = y[j];
    __syncthreads();
    if (t < a.Dv) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < G; ++i) sum += ly[i][t];
        const float one[1] = {sum * a.scale};
        store_vec<1>(static_cast<T*>(a.y) + row * a.ldy + (int64_t)h * a.Dv + t, one);
    }
}

}  // namespace

int linattn_max_d() { return 128; }

// Tiles: so many that their workgroups fill the chip a whole number of times, as many tiles as sequences at least beside the
// sequences' own (whose last tiles are short): once where there are few sequences, since a tile costs its state's way to
// memory and back, else four times, since tiles of many lengths do not end together. Counted are the workgroups a compute
// unit takes of bfloat16 in whole chunks: three with wide heads, four with narrow ones. All launches of both directions share
// the tiles; wide heads in fp32 or of other rows have two (20597 x 8 x 128 in fp32, both ways: 1026 us, 5 times the matrix
// units' floor; 20597 x 8 x 100 in bfloat16: 391 us, 316 for 128), the launch of dv and dk one. At 656603 x 50 (fp32, 1024 sequences, both ways) tiles of 224 take 941 to 987 us, of 672 1101.
AttnPlan attn_plan(int S, int64_t T, int H, int Dk, int Dv) {
    AttnPlan p;
    const int64_t fill = (std::max(Dk, Dv) > 64 ? 3 : 4) * 256;
    int64_t rounds = std::max<int64_t>(1, (2 * (int64_t)S * H + fill - 1) / fill);
    if (rounds > 1) rounds = std::max<int64_t>(rounds, 4);
    const int64_t tiles = std::max<int64_t>(1, (fill * rounds + H - 1) / H - S);
    p.L = (int)std::min<int64_t>(4096, std::max<int64_t>(64, (T + tiles * 32 - 1) / (tiles * 32) * 32));
    const int64_t size = (int64_t)Dk * Dv;
    p.nslots = T / p.L;
    p.total = 2 * (((size_t)p.nslots * (size_t)(H * size) * sizeof(float) + 15) / 16 * 16);
    p.chain_blocks = H * chain_blocks(size);
    return p;
}

namespace {
Args args_of(const AttnArgs& x, const AttnPlan& p) {
    Args a{};
    a.off = x.off;
    a.S = x.S;
    a.H = x.H;
    a.T = x.T;
    a.L = p.L;
    a.inv_l = 1.0 / p.L;
    a.decay = x.decay;
    a.size = (int64_t)x.Dk * x.Dv;
    return a;
}
struct Rows_ {  // a tensor's rows
    const void* p;
    int64_t ld;
};
Args::Side side_of(Rows_ a, Rows_ b, Rows_ c, int da, int dc, int trans, void* out, int64_t ldo) {
    return Args::Side{a.p, b.p, c.p, a.ld, b.ld, c.ld, da, dc, trans, out, ldo};
}
}  // namespace

hipError_t launch_attn_fwd(const AttnArgs& x, int dtype, void* ws, hipStream_t st) {
    const AttnPlan p = attn_plan(x.S, x.T, x.H, x.Dk, x.Dv);
    Args a = args_of(x, p);
    a.dir = x.reverse ? -1 : 1;
    a.post = 1;
    a.pscale = a.sscale = 1.f;
    a.oscale = x.scale;
    a.slots = static_cast<float*>(ws);
    a.init = x.h0;
    a.last = x.hT;
    a.side[0] = side_of({x.q, x.ldq}, {x.k, x.ldk}, {x.v, x.ldv}, x.Dk, x.Dv, 0, x.y, x.ldy);
    hipError_t e = hipSuccess;
    const bool states = p.nslots > 0 || x.hT;
    if (states && x.T > 0 && (e = go_any(a, dtype, kStates, st)) != hipSuccess) return e;
    if (states && (e = go_chain(a, st)) != hipSuccess) return e;
    return x.T > 0 ? go_any(a, dtype, kOutputs, st) : e;
}

hipError_t launch_attn_bwd(const AttnArgs& x, int dtype, void* ws, hipStream_t st) {
    const AttnPlan p = attn_plan(x.S, x.T, x.H, x.Dk, x.Dv);
    const Rows_ q{x.q, x.ldq}, k{x.k, x.ldk}, v{x.v, x.ldv}, dy{x.dy, x.lddy};
    // the state's gradient, against the forward's order
    Args g = args_of(x, p);
    g.dir = x.reverse ? 1 : -1;
    g.post = 0;
    g.pscale = g.sscale = x.scale;
    g.oscale = 1.f;
    g.slots = reinterpret_cast<float*>(static_cast<char*>(ws) + p.total / 2);
    g.init = x.dhT;
    g.last = x.dh0;
    g.side[0] = side_of(k, q, dy, x.Dk, x.Dv, 0, x.dv, x.lddv);
    g.side[1] = side_of(v, dy, q, x.Dv, x.Dk, 1, x.dk, x.lddk);
    hipError_t e = hipSuccess;
    const bool states = p.nslots > 0 || x.dh0;
    if (states && x.T > 0 && (e = go_any(g, dtype, kStates, st)) != hipSuccess) return e;
    if (states && (e = go_chain(g, st)) != hipSuccess) return e;
    if (x.T == 0) return e;
    if (padded(x.Dk) == padded(x.Dv)) {
        if ((e = go_any(g, dtype, kBothOutputs, st)) != hipSuccess) return e;
    } else {
        if ((e = go_any(g, dtype, kOutputs, st)) != hipSuccess) return e;
        g.side[0] = g.side[1];
        if ((e = go_any(g, dtype, kOutputs, st)) != hipSuccess) return e;
    }
    Args f = args_of(x, p);
    f.dir = x.reverse ? -1 : 1;
    f.post = 1;
    f.pscale = f.sscale = 1.f;
    f.oscale = x.scale;
    f.slots = static_cast<float*>(ws);
    f.init = x.h0;
    f.side[0] = side_of(dy, v, k, x.Dv, x.Dk, 1, x.dq, x.lddq);
    return go_any(f, dtype, kOutputs, st);
}

hipError_t launch_attn_step(const AttnArgs& x, int dtype, const int32_t* slots, int n_slots, const float* h_in,
                            float* h_out, hipStream_t st) {
    const StepArgs a{x.S, x.H, x.Dk, x.Dv, n_slots, x.decay, x.scale, x.q, x.k, x.v, x.ldq, x.ldk, x.ldv, x.ldy,
                     slots, h_in, h_out, x.y};
    const dim3 grid((uint32_t)((int64_t)x.S * x.H));
    const bool wide = x.Dv % 4 == 0;
    if (dtype == 1) {
        if (wide) launch(step<bf16, 4>, grid, dim3(kThreads), 0, st, a);
        else launch(step<bf16, 1>, grid, dim3(kThreads), 0, st, a);
    } else {
        if (wide) launch(step<float, 4>, grid, dim3(kThreads), 0, st, a);
        else launch(step<float, 1>, grid, dim3(kThreads), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace mdl
