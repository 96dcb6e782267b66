// k_scan.hip — the gated linear recurrence over packed sequences: forward, backward and the single-token step.
//
// Per channel, with gates that do not read the state (the Leaky cell's update s = f s + (1 - f) g along one axis):
//   f = sigmoid(zf), o = sigmoid(zo);  h_t = f_t h_{t-1} + (1 - f_t) g_t;  y_t = o_t h_t  (y = h without zo)
// and, with l_t = dL/dh_t,
//   l_t = o_t dy_t + f_{t+1} l_{t+1}  (dhT instead of the second term at a sequence's last token)
//   dg = (1 - f) l;  dzf = f (1 - f) (h_{t-1} - g) l;  dzo = dy h o (1 - o);  dh0 = f_first l_first.
//
// Both recurrences are affine maps x -> A x + B composed along time, so they are cut into tiles of TT tokens by CB
// channels that run at once: the packed token axis is tiled evenly whatever the sequences' lengths, and a sequence
// start inside a tile is a map that ignores its argument, written A = -1 (A is a product of sigmoids otherwise).
// A thread owns V channels (16 bytes of a row) and NT consecutive tokens; the 256 / CL threads of one channel vector
// hold the tile's successive token groups. Thread maps meet in LDS, where one thread per channel chains them.
// The tiles' maps are handed from tile to tile in the same launch (see look_back), so every stream is read and written
// once. All states, maps and sums are fp32; a stream of bfloat16 is rounded once, as it is stored.
//
// Bound by HBM on long inputs: 208246 tokens x 1024 channels in bfloat16 take 352 us forward (1.71 GB, 4.9 TB/s, the rate
// of a copy) and 597 us backward (2.99 GB, 5.0 TB/s), with the vector ALUs, by the count of their instructions, close to
// busy as well (89 and 76 % of the cycles); 656603 tokens x 32 in fp32 without an output gate 52 us (252 MB) and 75 us
// (420 MB). A generation or two of workgroups are bound by their latency, read, chain, write: 20597 tokens x 512 in
// bfloat16 take 24 us (84 MB) and 38 us (148 MB). Rows that are no multiple of 128 bytes cost far more: a tile's 128 bytes
// then straddle two lines of every row, which two workgroups read and write; 206796 x 1030 take 615 and 1377 us.
// (Medians of 10 passes under the profiler; in 60 passes in a row the first case takes 338 and 563 us a pass, with the
// launches that clear the words. The backward for bfloat16 spills 4 registers, 20 bytes a lane.)
// The tile of 128 tokens by 128 bytes of channels, beside others in one session, us forward and backward:
//   tokens by bytes             128 by 128     64 by 128     64 by 256     256 by 64
//   208246 x 1024, bfloat16      352   597     446   697     455   599     457   849
//   656603 x 32, fp32             52    75      62    82      85   114      70   106
//   20597 x 512, bfloat16         24    38      27    41      25    38      33    49
#include "kernels.h"
#include "seqio.h"

#include <algorithm>
#include <type_traits>

namespace mdl {

namespace {

// (min and max of two int64_t go through double)
__device__ inline int64_t lesser(int64_t a, int64_t b) { return a < b ? a : b; }

// vectors of V elements that hold a row of D, any D >= 1
__host__ __device__ constexpr int vectors(int D, int V) { return (D - 1) / V + 1; }

constexpr int SCAN_THREADS = 256;
constexpr float kReset = -1.0f;  // the A of a map that ignores its argument

// the states of a map applied to x
__device__ inline float apply_map(float A, float B, float x) { return A < 0.f ? B : __builtin_fmaf(A, x, B); }

// First index i in [0, n) with off[i] >= v (n if none), off ascending: 64 probes a round, one per lane, every lane of
// the wave in it. Any contents of off keep the probes inside [0, n).
__device__ inline int lower_bound_wave(const int64_t* off, int n, int64_t v) {
    const int lane = threadIdx.x & 63;
    int lo = 0, len = n;
    while (len > 0) {
        const int step = (len + 63) >> 6;
        const int64_t idx = (int64_t)lane * step;
        const bool below = idx < len && off[lo + idx] < v;
        const int cnt = __popcll(__ballot(below));
        if (cnt == 0) break;
        const int used = (cnt - 1) * step + 1;
        lo += used;
        len = min(step - 1, len - used);
    }
    return lo;
}

struct Tile {
    int64_t p0;   // first position (token order of the scan) of the tile
    int c0;       // first channel
};

// the tokens [t0, t1) of a tile that starts at position p0
template <int TT>
__device__ inline void tile_tokens(const ScanArgs& a, int64_t p0, int64_t& t0, int64_t& t1) {
    t1 = a.reverse ? a.T - p0 : lesser(p0 + TT, a.T);
    t0 = a.reverse ? -lesser(p0 + TT - a.T, 0) : p0;
}
// the first sequence that may hold tokens of [t0, ...): the one before the first that starts there
__device__ inline int first_sequence(const ScanArgs& a, int64_t t0) {
    return max(lower_bound_wave(a.off, a.S, t0) - 1, 0);
}
// a thread's sequence of the tile: read before the tile's rows, so that it does not wait for them
struct Seq {
    int64_t s, b, e;
    __device__ inline Seq(const ScanArgs& a, int first) : s(first + (int64_t)threadIdx.x), b(0), e(0) { read(a); }
    __device__ inline void read(const ScanArgs& a) {
        if (s < a.S) {
            b = a.off[s];
            e = a.off[s + 1];
        }
    }
};
// Sequence marks of the tile's positions: start[p] / last[p] hold sequence + 1 where position p0 + p is a sequence's
// first / last in scan order, 0 elsewhere. Sequences without tokens hand `from` to `to` ([S][D], zero if null).
template <int TT, int CB>
__device__ inline void mark_tile(const ScanArgs& a, Tile t, Seq q, int* start, int* last, const float* from,
                                 float* to) {
    for (int i = threadIdx.x; i < TT; i += SCAN_THREADS) start[i] = last[i] = 0;
    int64_t t0, t1;
    tile_tokens<TT>(a, t.p0, t0, t1);
    const bool final_tile = t1 >= a.T;
    __syncthreads();
    // one sequence: false where the tile's sequences have ended
    auto mark = [&]() {
        const int64_t s = q.s, b = q.b, e = q.e;
        if (s >= a.S || (b >= t1 && !final_tile)) return false;
        if (e <= b) {
            // by the tile that holds the offset, the last one for offsets at the end
            const bool mine = b >= t0 && (b < t1 || final_tile);
            if (mine && to) {
                for (int c = t.c0; c < min(t.c0 + CB, a.D); ++c) to[s * a.D + c] = from ? from[s * a.D + c] : 0.f;
            }
            return true;
        }
        const int64_t ps = (a.reverse ? a.T - e : b) - t.p0, pl = (a.reverse ? a.T - 1 - b : e - 1) - t.p0;
        if (ps >= 0 && ps < TT) start[ps] = (int)s + 1;
        if (pl >= 0 && pl < TT) last[pl] = (int)s + 1;
        return true;
    };
    // the first, read before the tile's rows, does not wait for them (loads return in order); more of them are rare
    bool more = mark();
    while (more) {
        q.s += SCAN_THREADS;
        q.read(a);
        more = mark();
    }
    __syncthreads();
}

// a thread's share of the tile
template <int V, int CL, int NT>
struct Share {
    int group;        // its token group
    int ch;           // its first channel (inside the row)
    bool active;      // false: a lane past the row's end, which repeats the last vector and stores nothing
    int64_t tok;      // its first token, moved inside [0, T) if past the end (loads from there go unused)
    int room;         // how many of its next tokens lie inside
    int dir;          // the tokens' order
    unsigned inside;  // bit i: its i-th position is a token of a sequence
    __device__ inline Share(const ScanArgs& a, Tile t) {
        group = threadIdx.x / CL;
        const int c = t.c0 + (threadIdx.x % CL) * V;
        active = c < a.D;
        ch = min(c, a.D - V);
        // the tile's positions that are rows, and those that are tokens of a sequence, counted from its first
        const int rows = (int)lesser(a.T - t.p0, 1 << 20), g0 = group * NT;
        const int64_t lo = a.off[0], hi = a.off[a.S];
        const int64_t b = (a.reverse ? a.T - hi : lo) - t.p0, e = (a.reverse ? a.T - lo : hi) - t.p0;
        const int sb = (int)lesser(b < 0 ? 0 : b, 1 << 20), se = min((int)lesser(e < 0 ? 0 : e, 1 << 20), rows);
        const int p = min(g0, rows - 1);
        room = min(rows - 1 - p, NT - 1);
        dir = a.reverse ? -1 : 1;
        tok = a.reverse ? a.T - 1 - t.p0 - p : t.p0 + p;
        const int ib = max(0, min(sb - g0, NT)), ie = max(0, min(se - g0, NT));
        inside = ((1u << ie) - 1) & ~((1u << ib) - 1);
    }
    // offset of the i-th token's elements in rows of stride ld
    __device__ inline int64_t at(int i, int ld, int64_t base) const { return base + (int64_t)min(i, room) * (dir * ld); }
    __device__ inline int64_t base(int ld) const { return tok * ld + ch; }
};

// Number of a workgroup's tile and channel block, tile ncb + block: the blocks of successive tiles are rotated by one, so
// that a workgroup id's remainder by the 8 dies, whose L2s share the work round-robin, falls on every part of a row. (With
// the plain order a die reads the same eighth of every row: 208246 tokens x 1024 in bfloat16 take 439 us forward and 634
// backward, rotated 352 and 597. Rows of one channel block are the same either way.)
__device__ inline int tile_id(const ScanArgs& a) {
    const int k = blockIdx.x / a.ncb, c = blockIdx.x % a.ncb;
    return k * a.ncb + (c + k) % a.ncb;
}
__device__ inline Tile tile_of(const ScanArgs& a, int linear, int tt, int cb) {
    return {(int64_t)(linear / a.ncb) * tt, linear % a.ncb * cb};
}

// The tiles' maps are handed on through a.words [ntiles][slots], one 64-bit word (A, B) per tile and channel, cleared to
// kEmpty before the launch: a tile first offers its own map, and, once it knows its incoming state, stores the state it
// ends in as a map that ignores its argument. A tile looks at the words of its last kWindow predecessors, one thread per
// channel, until the nearest state and all maps after it are there, and chains from that state on. Words are loaded and
// stored whole by relaxed device-scope atomics and carry all that is handed on: no other memory has to be ordered with
// them.
// No wait depends on the order in which workgroups run: after a.polls looks a thread walks back over the words on its
// own, forms a map that is still missing from the inputs, with the owner's arithmetic, and offers it in the owner's
// place; the walk ends at the nearest state or at the first tile. States are always the same chain of multiply-adds of
// the same maps, so the results do not depend on timing either. (Tickets taken in order, the other way to bound the wait,
// cost 11.5 ns each on one counter: 60 us for the 5130 tiles of 1024 image rows, whose data takes 50 us.)
constexpr uint64_t kEmpty = ~uint64_t(0);
constexpr int kWindow = 8;
__device__ inline uint64_t pack_map(float A, float B) {
    if (A != A) A = __uint_as_float(0x7fc00000u);  // no NaN is taken for an empty word
    return (uint64_t)__float_as_uint(B) << 32 | __float_as_uint(A);
}
__device__ inline void put_word(uint64_t* p, float A, float B) {
    __hip_atomic_store(p, pack_map(A, B), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// A tile's map handed on by other waves than those that look back (a wave's loads wait for its stores before them): the
// state, if it is there already, stays.
__device__ inline void offer_word(uint64_t* p, float A, float B) {
    uint64_t want = kEmpty;
    __hip_atomic_compare_exchange_strong(p, &want, pack_map(A, B), __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline uint64_t get_word(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// x handed through a word
__device__ inline float apply_word(uint64_t m, float x) {
    return apply_map(__uint_as_float((uint32_t)m), __uint_as_float((uint32_t)(m >> 32)), x);
}
// the state (or gradient) that enters tile number `tile` of the chain: word k lies at w + k stride, and map(k, A, B) forms
// the map of tile k from the inputs
template <typename F>
__device__ inline float look_back(uint64_t* w, int tile, int64_t stride, int polls, F&& map) {
    for (int n = 0; n <= polls; ++n) {
        uint64_t m[kWindow];
#pragma unroll
        for (int i = 0; i < kWindow; ++i) {
            const int k = tile - 1 - i;
            m[i] = k >= 0 ? get_word(w + k * stride) : (uint64_t)__float_as_uint(kReset);  // before the first: state 0
        }
        bool known = false;
        float h = 0.f;
#pragma unroll
        for (int i = kWindow - 1; i >= 0; --i) {
            h = apply_word(m[i], h);
            known = m[i] != kEmpty && (__uint_as_float((uint32_t)m[i]) < 0.f || known);
        }
        if (known) return h;
        __builtin_amdgcn_s_sleep(2);
    }
    int k = tile - 1;
    for (; k >= 0; --k) {
        uint64_t m = get_word(w + k * stride);
        if (m == kEmpty) {
            float A, B;
            map(k, A, B);
            m = pack_map(A, B);
            offer_word(w + k * stride, A, B);
        }
        if (__uint_as_float((uint32_t)m) < 0.f) break;
    }
    float h = 0.f;
    for (k = k < 0 ? 0 : k; k < tile; ++k) h = apply_word(get_word(w + k * stride), h);
    return h;
}

// The sequence that holds a token, for one thread that goes through tokens one by one.
struct Walk {
    int64_t b = 0, e = 0;  // the sequence's tokens
    int s = 0;
    // whether the token belongs to a sequence, and is its first or last in scan order
    __device__ inline bool at(const ScanArgs& a, int64_t tok, bool& first, bool& fin) {
        if (tok < b || tok >= e) {
            int lo = 0, n = a.S;  // the last sequence that starts at or before the token
            while (n > 1) {
                const int half = n >> 1;
                if (a.off[lo + half] <= tok) lo += half;
                n -= half;
            }
            s = lo;
            b = a.off[lo];
            e = a.off[lo + 1];
        }
        const bool in = tok >= b && tok < e;
        first = in && tok == (a.reverse ? e - 1 : b);
        fin = in && tok == (a.reverse ? b : e - 1);
        return in;
    }
};
// Channel ch of tile k's map from the inputs by one thread, token group by token group as the tile's own threads do.
template <typename T, int G, int NT>
__device__ inline void forward_map(const ScanArgs& a, int k, int ch, float& ta, float& tb) {
    Walk walk;
    ta = 1.f;
    tb = 0.f;
#pragma unroll 1
    for (int j = 0; j < G; ++j) {
        float A = 1.f, h = 0.f;
        bool reset = false;
#pragma unroll 1
        for (int i = 0; i < NT; ++i) {
            const int64_t p = ((int64_t)k * G + j) * NT + i, tok = a.reverse ? a.T - 1 - p : p;
            bool first = false, fin = false;
            if (p >= a.T || !walk.at(a, tok, first, fin)) continue;
            if (first) {
                reset = true;
                h = a.h0 ? a.h0[(int64_t)walk.s * a.D + ch] : 0.f;
            }
            float f, c;
            sigm_enc<T>(load_raw<1>(static_cast<const T*>(a.zf) + tok * a.ldz + ch)[0], f, c);
            h = __builtin_fmaf(f, h, c * load_raw<1>(static_cast<const T*>(a.g) + tok * a.ldz + ch)[0]);
            A *= f;
        }
        if (reset) A = kReset;
        tb = apply_map(A, h, tb);
        ta = A < 0.f || ta < 0.f ? kReset : ta * A;
    }
}
template <typename T, int G, int NT>
__device__ inline void reverse_map(const ScanArgs& a, int k, int ch, float& ta, float& tb) {
    Walk walk;
    ta = 1.f;
    tb = 0.f;
#pragma unroll 1
    for (int j = G - 1; j >= 0; --j) {
        float A = 1.f, d = 0.f;
        bool ends = false;
#pragma unroll 1
        for (int i = 0; i < NT; ++i) {
            const int64_t p = ((int64_t)k * G + j) * NT + i, tok = a.reverse ? a.T - 1 - p : p;
            bool first = false, fin = false;
            if (p >= a.T || !walk.at(a, tok, first, fin)) continue;
            float f, c, so = 1.f, co;
            sigm_enc<T>(load_raw<1>(static_cast<const T*>(a.zf) + tok * a.ldz + ch)[0], f, c);
            if (a.zo) sigm_enc<T>(load_raw<1>(static_cast<const T*>(a.zo) + tok * a.ldz + ch)[0], so, co);
            A *= f;
            if (!ends) {
                d = __builtin_fmaf(A, so * load_raw<1>(static_cast<const T*>(a.dy) + tok * a.ldy + ch)[0], d);
                if (fin) d = __builtin_fmaf(A, a.dhT ? a.dhT[(int64_t)walk.s * a.D + ch] : 0.f, d);
            }
            ends |= fin;
        }
        if (ends) A = kReset;
        tb = apply_map(A, d, tb);
        ta = A < 0.f || ta < 0.f ? kReset : ta * A;
    }
}
// the channel of slot c of a channel block that starts at c0
template <int V>
__device__ inline int slot_channel(const ScanArgs& a, int c0, int c) {
    return min(c0 + c / V * V, a.D - V) + c % V;
}

// before tiles that hand on their maps: words cleared, and each tile's first sequence found
template <int TT>
__global__ __launch_bounds__(SCAN_THREADS) void k_scan_init(ScanArgs a) {
    const int64_t n = a.ntiles * a.slots, step = (int64_t)gridDim.x * SCAN_THREADS;
    for (int64_t i = (int64_t)blockIdx.x * SCAN_THREADS + threadIdx.x; i < n; i += step) a.words[i] = kEmpty;
    for (int64_t k = ((int64_t)blockIdx.x * SCAN_THREADS + threadIdx.x) >> 6; k < a.ntiles; k += step >> 6) {
        int64_t t0, t1;
        tile_tokens<TT>(a, k * TT, t0, t1);
        const int s = first_sequence(a, t0);
        if ((threadIdx.x & 63) == 0) a.seq[k] = s;
    }
}
template <int TT>
__device__ inline int tile_sequence(const ScanArgs& a, Tile t) {
    if (a.ntiles > 1) return a.seq[t.p0 / TT];
    int64_t t0, t1;
    tile_tokens<TT>(a, t.p0, t0, t1);
    return first_sequence(a, t0);
}

// The registers of a thread's tokens hold the gates encoded (sigm_enc) and the other streams as loaded. Decoded gates are
// not kept from one pass over them to the next (forget), and the scheduler works on half a vector at a time: either would
// double the registers, which other workgroups need to keep loads in flight.
// positions of no sequence: their state and gradient pass through (f = 1), and nothing enters
template <int NT, typename R>
__device__ inline void outside(unsigned inside, R (&r)[NT], float x) {
    if (inside == (1u << NT) - 1) return;
#pragma unroll
    for (int i = 0; i < NT; ++i)
        if (!(inside >> i & 1)) r[i].fill(x);
}
// a sequence's row of p (zeros if null) into x: at its first or last token, so rarely that it is read on the spot
template <int V>
__device__ inline void enter(const float* p, int seq1, int D, int ch, float (&x)[V]) {
    if (p) load_f32<V>(p + (int64_t)(seq1 - 1) * D + ch, x);
    else
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = 0.f;
}

template <typename T, int V, int CL, int NT>
__global__ __launch_bounds__(SCAN_THREADS, 4) void k_scan_fwd(ScanArgs a) {
    constexpr int G = SCAN_THREADS / CL, TT = G * NT, CB = CL * V, HV = V > 4 ? 4 : V;
    // the waves that hold one thread per channel
    constexpr int CW = (CB + 63) / 64 * 64;
    static_assert(2 * CW <= SCAN_THREADS, "two sets of one thread per channel");
    __shared__ int start[TT], last[TT];
    __shared__ f32x2 maps[G][CB];  // of the token groups, and the states that enter them
    __shared__ float into[G][CB];
    const int linear = tile_id(a);
    const Tile tile = tile_of(a, linear, TT, CB);
    Share<V, CL, NT> me(a, tile);
    const Seq seq(a, tile_sequence<TT>(a, tile));
    Raw<T, V> rf[NT], rg[NT], ro[NT];
    const int64_t bz = me.base(a.ldz);
    auto rows = [&](auto&& load) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int64_t t = me.at(i, a.ldz, bz);
            rf[i] = load(static_cast<const T*>(a.zf) + t);
            rg[i] = load(static_cast<const T*>(a.g) + t);
            if (a.zo) ro[i] = load(static_cast<const T*>(a.zo) + t);
        }
    };
    if (a.once) rows([](const T* p) { return load_once<V>(p); });
    else rows([](const T* p) { return load_raw<V>(p); });
    mark_tile<TT, CB>(a, tile, seq, start, last, a.h0, a.hT);
    outside(me.inside, rf, INFINITY);
    outside(me.inside, rg, 0.f);
    const int* const first = start + me.group * NT;
    float qf[NT][V], A[V], h[V] = {};
    unsigned reset = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if (first[i]) {
            reset |= 1u << i;
            enter<V>(a.h0, first[i], a.D, me.ch, h);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f, c;
            qf[i][v] = settle(sigm_enc<T>(rf[i][v], f, c));
            h[v] = __builtin_fmaf(f, h[v], c * rg[i][v]);
            A[v] *= f;
        }
    }
    const int col = (threadIdx.x % CL) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) maps[me.group][col + v] = f32x2{reset ? kReset : A[v], h[v]};
    __syncthreads();
    // the tile's own map of channel c
    auto tile_map = [&](int c, float& ta, float& tb) {
        ta = 1.f;
        tb = 0.f;
#pragma unroll 8
        for (int j = 0; j < G; ++j) {
            const f32x2 m = maps[j][c];
            tb = apply_map(m[0], m[1], tb);
            ta = m[0] < 0.f || ta < 0.f ? kReset : ta * m[0];
        }
    };
    if (const int c = (int)threadIdx.x - (SCAN_THREADS - CW); a.ntiles > 1 && c >= 0 && c < CB) {
        float ta, tb;
        tile_map(c, ta, tb);
        offer_word(a.words + (int64_t)(linear / a.ncb) * a.slots + tile.c0 + c, ta, tb);
    }
    if (threadIdx.x < CB) {
        const int c = threadIdx.x;
        float x = 0.f;
        if (a.ntiles > 1) {
            const int64_t k = linear / a.ncb, slot = tile.c0 + c;
            float ta, tb;
            tile_map(c, ta, tb);
            uint64_t* const w = a.words + slot;
            x = look_back(w, (int)k, a.slots, a.polls, [&](int i, float& A, float& B) {
                forward_map<T, G, NT>(a, i, slot_channel<V>(a, tile.c0, c), A, B);
            });
            if (!(ta < 0.f)) put_word(w + k * a.slots, kReset, __builtin_fmaf(ta, x, tb));
            a.carry[k * a.slots + slot] = x;
        }
#pragma unroll 8
        for (int j = 0; j < G; ++j) {
            const f32x2 m = maps[j][c];
            into[j][c] = x;
            x = apply_map(m[0], m[1], x);
        }
    }
    __syncthreads();
    forget(qf);
    forget(rg);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = into[me.group][col + v];
    const int64_t by = me.base(a.ldy);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if (reset >> i & 1) enter<V>(a.h0, first[i], a.D, me.ch, h);
        float y[V];
#pragma unroll
        for (int v0 = 0; v0 < V; v0 += HV) {
            one_at_a_time();
#pragma unroll
            for (int v = v0; v < v0 + HV; ++v) {
                float f, c, so = 1.f, co;
                sigm_dec(qf[i][v], f, c);
                h[v] = __builtin_fmaf(f, h[v], c * rg[i][v]);
                if (a.zo) sigm2<T>(ro[i][v], so, co);
                y[v] = so * h[v];
            }
        }
        if (me.active && (me.inside >> i & 1)) {
            store_vec<V>(static_cast<T*>(a.y) + me.at(i, a.ldy, by), y);
            const int en = last[me.group * NT + i];
            if (en && a.hT) store_f32<V>(a.hT + (int64_t)(en - 1) * a.D + me.ch, h);
        }
    }
}

// Backward: the tile's states again from its incoming one in a.carry, and the reverse recurrence, whose tiles are
// chained from the last to the first.
template <typename T, int V, int CL, int NT>
__global__ __launch_bounds__(SCAN_THREADS, V == 4 ? 4 : 3) void k_scan_bwd(ScanArgs a) {
    constexpr int G = SCAN_THREADS / CL, TT = G * NT, CB = CL * V, HV = V > 4 ? 4 : V;
    constexpr int CW = (CB + 63) / 64 * 64;
    static_assert(3 * CW <= SCAN_THREADS, "three sets of one thread per channel");
    __shared__ int start[TT], last[TT];
    __shared__ f32x2 maps[G][CB], rmaps[G][CB];  // of the token groups, and what enters them
    __shared__ float into[G][CB], rinto[G][CB];
    // the chain's k-th tile is the k-th from the end
    const int id = tile_id(a), k = id / a.ncb, linear = ((int)a.ntiles - 1 - k) * a.ncb + id % a.ncb;
    const Tile tile = tile_of(a, linear, TT, CB);
    Share<V, CL, NT> me(a, tile);
    const Seq seq(a, tile_sequence<TT>(a, tile));
    Raw<T, V> rf[NT], rg[NT], ro[NT], rd[NT];
    const int64_t bz = me.base(a.ldz), by = me.base(a.ldy);
    auto rows = [&](auto&& load) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int64_t t = me.at(i, a.ldz, bz);
            rf[i] = load(static_cast<const T*>(a.zf) + t);
            rg[i] = load(static_cast<const T*>(a.g) + t);
            if (a.zo) ro[i] = load(static_cast<const T*>(a.zo) + t);
            else ro[i].fill(INFINITY);  // an open gate
            rd[i] = load(static_cast<const T*>(a.dy) + me.at(i, a.ldy, by));
        }
    };
    if (a.once) rows([](const T* p) { return load_once<V>(p); });
    else rows([](const T* p) { return load_raw<V>(p); });
    mark_tile<TT, CB>(a, tile, seq, start, last, a.dhT, a.dh0);
    outside(me.inside, rf, INFINITY);
    outside(me.inside, rg, 0.f);
    outside(me.inside, ro, 0.f);
    outside(me.inside, rd, 0.f);
    const int *const first = start + me.group * NT, *const fin = last + me.group * NT;
    // Both maps in one walk over the tokens: with P_t = f_first ... f_t, the reverse one is x -> P_last x + sum_t P_t e_t
    // for the gradients e_t = o_t dy_t that enter at the tokens, up to the first sequence's end.
    float qf[NT][V], qo[NT][V], A[V], h[V] = {}, d[V] = {};
    unsigned reset = 0, ends = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if (first[i]) {
            reset |= 1u << i;
            enter<V>(a.h0, first[i], a.D, me.ch, h);
        }
#pragma unroll
        for (int v0 = 0; v0 < V; v0 += HV) {
            one_at_a_time();
#pragma unroll
            for (int v = v0; v < v0 + HV; ++v) {
                float f, c, so, co;
                qf[i][v] = settle(sigm_enc<T>(rf[i][v], f, c));
                qo[i][v] = settle(sigm_enc<T>(ro[i][v], so, co));
                h[v] = __builtin_fmaf(f, h[v], c * rg[i][v]);
                A[v] *= f;
                if (!ends) d[v] = __builtin_fmaf(A[v], so * rd[i][v], d[v]);
            }
        }
        if (fin[i]) {
            if (!ends) {
                float x[V];
                enter<V>(a.dhT, fin[i], a.D, me.ch, x);
#pragma unroll
                for (int v = 0; v < V; ++v) d[v] = __builtin_fmaf(A[v], x[v], d[v]);
            }
            ends |= 1u << i;
        }
    }
    const int col = (threadIdx.x % CL) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        maps[me.group][col + v] = f32x2{reset ? kReset : A[v], h[v]};
        rmaps[me.group][col + v] = f32x2{ends ? kReset : A[v], d[v]};
    }
    __syncthreads();
    // Waves in parallel, one thread per channel: the first composes the tile's reverse map, the next chains the forward
    // maps from the incoming state, a third hands on the reverse map.
    uint64_t* const w = a.words + tile.c0;
    const int c1 = threadIdx.x, c2 = c1 - CW, c3 = c2 - CW;
    float ta = 1.f, tb = 0.f;
    if (a.ntiles > 1 && (c1 < CB || (c3 >= 0 && c3 < CB))) {
        const int c = c1 < CB ? c1 : c3;
#pragma unroll 8
        for (int j = G - 1; j >= 0; --j) {
            const f32x2 m = rmaps[j][c];
            tb = apply_map(m[0], m[1], tb);
            ta = m[0] < 0.f || ta < 0.f ? kReset : ta * m[0];
        }
        if (c1 >= CB) offer_word(w + k * a.slots + c, ta, tb);
    }
    if (c2 >= 0 && c2 < CB) {
        float x = a.ntiles > 1 ? a.carry[(int64_t)(linear / a.ncb) * a.slots + tile.c0 + c2] : 0.f;
#pragma unroll 8
        for (int j = 0; j < G; ++j) {
            const f32x2 m = maps[j][c2];
            into[j][c2] = x;
            x = apply_map(m[0], m[1], x);
        }
    }
    __syncthreads();
    // the first wave looks back while the others walk forward
    if (c1 < CB) {
        float x = 0.f;
        if (a.ntiles > 1) {
            x = look_back(w + c1, k, a.slots, a.polls, [&](int i, float& A, float& B) {
                reverse_map<T, G, NT>(a, (int)a.ntiles - 1 - i, slot_channel<V>(a, tile.c0, c1), A, B);
            });
            if (!(ta < 0.f)) put_word(w + k * a.slots + c1, kReset, __builtin_fmaf(ta, x, tb));
        }
#pragma unroll 8
        for (int j = G - 1; j >= 0; --j) {
            const f32x2 m = rmaps[j][c1];
            rinto[j][c1] = x;
            x = apply_map(m[0], m[1], x);
        }
    }
    // Forward: the states, with which the output gates' gradients are done. What is left of the other streams is the
    // entering gradient e = o dy and h_{t-1} - g.
    forget(qf);
    forget(qo);
    forget(rg);
    forget(rd);
    const int64_t bd = me.base(a.ldd);
    float e[NT][V], pg[NT][V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = into[me.group][col + v];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if (reset >> i & 1) enter<V>(a.h0, first[i], a.D, me.ch, h);
        float dzo[V];
#pragma unroll
        for (int v0 = 0; v0 < V; v0 += HV) {
            one_at_a_time();
#pragma unroll
            for (int v = v0; v < v0 + HV; ++v) {
                float f, c, so, co;
                sigm_dec(qf[i][v], f, c);
                sigm_dec(qo[i][v], so, co);
                const float g = rg[i][v];
                pg[i][v] = settle(h[v] - g);
                h[v] = __builtin_fmaf(f, h[v], c * g);
                e[i][v] = settle(so * rd[i][v]);
                dzo[v] = e[i][v] * co * h[v];
            }
        }
        if (a.zo && me.active && (me.inside >> i & 1)) store_vec<V>(static_cast<T*>(a.dzo) + me.at(i, a.ldd, bd), dzo);
    }
    __syncthreads();
    forget(qf);
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = rinto[me.group][col + v];
#pragma unroll
    for (int i = NT - 1; i >= 0; --i) {
        float dzf[V], dg[V];
        if (ends >> i & 1) enter<V>(a.dhT, fin[i], a.D, me.ch, d);
#pragma unroll
        for (int v0 = 0; v0 < V; v0 += HV) {
            one_at_a_time();
#pragma unroll
            for (int v = v0; v < v0 + HV; ++v) {
                float f, c;
                sigm_dec(qf[i][v], f, c);
                const float lam = e[i][v] + d[v];
                dg[v] = c * lam;
                d[v] = f * lam;
                dzf[v] = f * dg[v] * pg[i][v];
            }
        }
        if (me.active && (me.inside >> i & 1)) {
            const int64_t o = me.at(i, a.ldd, bd);
            store_vec<V>(static_cast<T*>(a.dzf) + o, dzf);
            store_vec<V>(static_cast<T*>(a.dg) + o, dg);
            if ((reset >> i & 1) && a.dh0)
                store_f32<V>(a.dh0 + (int64_t)(first[i] - 1) * a.D + me.ch, d);
        }
    }
}

// sequences without tokens, where there is no token at all
__global__ __launch_bounds__(256) void k_scan_copy(const float* __restrict__ from, float* __restrict__ to, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        to[i] = from ? from[i] : 0.f;
}

// one token of each row: state rows h_in[slot] -> h_out[slot]
template <typename T, int V>
__global__ __launch_bounds__(256) void k_scan_step(int S, int D, const T* __restrict__ zf, const T* __restrict__ g,
                                                   const T* __restrict__ zo, int64_t ldz,
                                                   const int32_t* __restrict__ slots, int n_slots, const float* h_in,
                                                   float* h_out, T* __restrict__ y, int64_t ldy) {
    const int per = vectors(D, V);
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)S * per) return;
    const int s = (int)(i / per), c = (int)(i % per) * V;
    const int slot = slots ? slots[s] : s;
    if (slot < 0 || slot >= n_slots) return;
    // the row's last vector, moved back, shares elements with its neighbour: with the state written in place it takes
    // them one at a time instead
    const int n = min(V, D - c);
    auto body = [&](auto vtag, int ch) {
        constexpr int W = decltype(vtag)::value;
        const auto rf = load_raw<W>(zf + (int64_t)s * ldz + ch);
        const auto rg = load_raw<W>(g + (int64_t)s * ldz + ch);
        float h[W], out[W];
        load_f32<W>(h_in + (int64_t)slot * D + ch, h);
#pragma unroll
        for (int v = 0; v < W; ++v) {
            float f, fc;
            sigm2<T>(rf[v], f, fc);
            h[v] = __builtin_fmaf(f, h[v], fc * rg[v]);
            out[v] = h[v];
        }
        if (zo) {
            const auto ro = load_raw<W>(zo + (int64_t)s * ldz + ch);
#pragma unroll
            for (int v = 0; v < W; ++v) {
                float so, co;
                sigm2<T>(ro[v], so, co);
                out[v] *= so;
            }
        }
        store_f32<W>(h_out + (int64_t)slot * D + ch, h);
        store_vec<W>(y + (int64_t)s * ldy + ch, out);
    };
    if (n == V) {
        body(std::integral_constant<int, V>{}, c);
    } else {
        for (int k = 0; k < n; ++k) body(std::integral_constant<int, 1>{}, c + k);
    }
}

// the tile shape for a row: a vector of 16 bytes a thread and as many lanes along the row as it fills, at most 8; rows of
// no more than one vector take one element a lane and more tokens instead; forward and backward have the same
template <typename F>
void with_shape(int D, int dtype, F&& fn) {
    auto go = [&](auto ty) {
        constexpr int V = Width<decltype(ty)>::v;
        if (D <= 4) return fn(ty, ScanShape<1, 4, 16>{});
        if constexpr (V > 4) {
            if (D <= V) return fn(ty, ScanShape<1, 8, 16>{});
        }
        const int lanes = vectors(D, V);
        if (lanes <= 4) return fn(ty, ScanShape<V, 4, 4>{});
        return fn(ty, ScanShape<V, 8, 4>{});
    };
    if (dtype == 1) go(bf16{});
    else go(float{});
}

}  // namespace

ScanPlan scan_plan(int64_t T, int D, int dtype) {
    ScanPlan p;
    with_shape(D, dtype, [&](auto, auto sh) {
        using S = decltype(sh);
        const int64_t cb = S::CL * S::V, tt = (int64_t)(SCAN_THREADS / S::CL) * S::NT;
        p.ncb = (int)((D + cb - 1) / cb);
        p.slots = p.ncb * cb;
        p.ntiles = (T + tt - 1) / tt;
    });
    if (p.ntiles > 1) {
        p.seq = p.ntiles * p.slots * 8;
        p.carry = (p.seq + p.ntiles * 4 + 15) & ~size_t(15);
        p.total = p.carry + p.ntiles * p.slots * 4;
    }
    return p;
}

static hipError_t scan_run(ScanArgs a, int dtype, void* ws, bool backward, hipStream_t st) {
    if (a.T == 0) {
        const int64_t n = (int64_t)a.S * a.D;
        float* to = backward ? a.dh0 : a.hT;
        if (n > 0 && to)
            launch(k_scan_copy, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4096)), dim3(256), 0, st,
                   backward ? a.dhT : a.h0, to, n);
        return hipGetLastError();
    }
    const ScanPlan p = scan_plan(a.T, a.D, dtype);
    a.ncb = p.ncb;
    a.ntiles = p.ntiles;
    a.slots = p.slots;
    if (p.ntiles > 1) {
        uint8_t* w = static_cast<uint8_t*>(ws);
        a.words = reinterpret_cast<uint64_t*>(w);
        a.seq = reinterpret_cast<int32_t*>(w + p.seq);
        a.carry = reinterpret_cast<float*>(w + p.carry);
    }
    // Streams larger than the memory-side cache are read past it: nothing of them would be found there again (both
    // kernels: 208246 x 1024 in bfloat16, 426 MB a stream, 949 us, 1015 otherwise; 656603 x 32 in fp32, 84 MB a stream, 135
    // us, 126 otherwise). Rows that are no multiple of 128 bytes lose by it, since the line that two workgroups share is
    // then read twice: 206796 x 1030 takes 1992 us, 1669 otherwise.
    a.once = a.T * a.D >= (int64_t(256) << 20) / (dtype == 1 ? 2 : 4);
    const dim3 grid((unsigned)(p.ntiles * p.ncb)), block(SCAN_THREADS);
    with_shape(a.D, dtype, [&](auto ty, auto sh) {
        using T = decltype(ty);
        using S = decltype(sh);
        if (p.ntiles > 1) {
            const int64_t n = std::max(p.ntiles * p.slots, p.ntiles * 64);
            launch(k_scan_init<SCAN_THREADS / S::CL * S::NT>,
                   dim3((unsigned)std::min<int64_t>((n + SCAN_THREADS - 1) / SCAN_THREADS, 8192)), block, 0, st, a);
        }
        if (backward) launch(k_scan_bwd<T, S::V, S::CL, S::NT>, grid, block, 0, st, a);
        else launch(k_scan_fwd<T, S::V, S::CL, S::NT>, grid, block, 0, st, a);
    });
    return hipGetLastError();
}

hipError_t launch_scan_fwd(const ScanArgs& a, int dtype, void* ws, hipStream_t st) {
    return scan_run(a, dtype, ws, false, st);
}
hipError_t launch_scan_bwd(const ScanArgs& a, int dtype, void* ws, hipStream_t st) {
    return scan_run(a, dtype, ws, true, st);
}

hipError_t launch_scan_step(int S, int D, int dtype, const void* zf, const void* g, const void* zo, int64_t ldz,
                            const int32_t* slots, int n_slots, const float* h_in, float* h_out, void* y, int64_t ldy,
                            hipStream_t st) {
    auto go = [&](auto ty) {
        using T = decltype(ty);
        constexpr int V = Width<T>::v;
        const int64_t n = (int64_t)S * vectors(D, V);
        launch(k_scan_step<T, V>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, S, D, static_cast<const T*>(zf),
               static_cast<const T*>(g), static_cast<const T*>(zo), ldz, slots, n_slots, h_in, h_out,
               static_cast<T*>(y), ldy);
    };
    if (dtype == 1) go(bf16{});
    else go(float{});
    return hipGetLastError();
}

}  // namespace mdl
