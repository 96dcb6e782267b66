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
#include "kernels.h"
#include "seqio.h"

#include <algorithm>
#include <type_traits>

namespace mdl {

namespace {

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

// Sequence marks of the tile's positions: start[p] / last[p] hold sequence + 1 where position p0 + p is a sequence's
// first / last in scan order, 0 elsewhere. Sequences without tokens hand `from` to `to` ([S][D], zero if null).
template <int TT>
__device__ inline void tile_tokens(const ScanArgs& a, int64_t p0, int64_t& t0, int64_t& t1) {  // tokens [t0, t1)
    t1 = a.reverse ? a.T - p0 : min(p0 + TT, a.T);
    t0 = a.reverse ? max<int64_t>(a.T - p0 - TT, 0) : p0;
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
template <int TT, int CB>
__device__ inline void mark_tile(const ScanArgs& a, Tile t, Seq q, int* start, int* last, const float* from,
                                 float* to) {
    for (int i = threadIdx.x; i < TT; i += SCAN_THREADS) start[i] = last[i] = 0;
    int64_t t0, t1;
    tile_tokens<TT>(a, t.p0, t0, t1);
    const bool final_tile = t1 >= a.T;
    __syncthreads();
    for (; q.s < a.S; q.s += SCAN_THREADS, q.read(a)) {
        const int64_t s = q.s, b = q.b, e = q.e;
        if (b >= t1 && !final_tile) break;
        if (e <= b) {
            // by the tile that holds the offset, the last one for offsets at the end
            const bool mine = b >= t0 && (b < t1 || final_tile);
            if (mine && to) {
                for (int c = t.c0; c < min(t.c0 + CB, a.D); ++c) to[s * a.D + c] = from ? from[s * a.D + c] : 0.f;
            }
            continue;
        }
        const int64_t ps = (a.reverse ? a.T - e : b) - t.p0, pl = (a.reverse ? a.T - 1 - b : e - 1) - t.p0;
        if (ps >= 0 && ps < TT) start[ps] = (int)s + 1;
        if (pl >= 0 && pl < TT) last[pl] = (int)s + 1;
    }
    __syncthreads();
}

// a thread's share of the tile
template <int V, int CL, int NT>
struct Share {
    int64_t p;          // its first position
    int group;          // its token group
    int ch;             // its first channel (inside the row)
    bool active;        // false: a lane past the row's end, which repeats the last vector and stores nothing
    unsigned inside;    // bit i: position p + i is a token of a sequence
    __device__ inline Share(const ScanArgs& a, Tile t) {
        group = threadIdx.x / CL;
        const int c = t.c0 + (threadIdx.x % CL) * V;
        p = t.p0 + group * NT;
        active = c < a.D;
        ch = min(c, a.D - V);
        inside = 0;
    }
    // token of position p + i, moved inside [0, T) for positions past the end (their loads go unused)
    __device__ inline int64_t token(const ScanArgs& a, int i) const {
        const int64_t q = min(p + i, a.T - 1);
        return a.reverse ? a.T - 1 - q : q;
    }
    __device__ inline void bounds(const ScanArgs& a) {
        const int64_t lo = a.off[0], hi = a.off[a.S];
        for (int i = 0; i < NT; ++i) {
            const int64_t q = p + i, tok = a.reverse ? a.T - 1 - q : q;
            if (q < a.T && tok >= lo && tok < hi) inside |= 1u << i;
        }
    }
};

__device__ inline Tile tile_of(const ScanArgs& a, int linear, int tt, int cb) {
    return {(int64_t)(linear / a.ncb) * tt, linear % a.ncb * cb};
}

// The tiles' maps are handed on through a.words [ntiles][slots], one 64-bit word (A, B) per tile and channel, cleared to
// kEmpty before the launch: a tile first stores its own map, and, once it knows its incoming state, the state it ends
// in as a map that ignores its argument. A tile looks at the words of its last kWindow predecessors, one thread per
// channel, until the nearest state and all maps after it are there, and chains from that state on. States are always
// the same chain of multiply-adds, wherever a tile found the nearest one, so the results do not depend on timing. Words
// are loaded and stored whole by relaxed device-scope atomics and carry all that is handed on: no other memory has to
// be ordered with them.
// Every wait ends: tiles are taken in ticket order, in which a tile comes after all that it waits for, so the earliest
// unfinished tile is held by a running workgroup and waits for none.
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
// the state (or gradient) that enters tile number `tile` of the chain: word k lies at w + k stride
__device__ inline float look_back(const uint64_t* w, int64_t tile, int64_t stride) {
    while (true) {
        uint64_t m[kWindow];
#pragma unroll
        for (int i = 0; i < kWindow; ++i) {
            const int64_t k = tile - 1 - i;
            m[i] = k >= 0 ? __hip_atomic_load(w + k * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                          : (uint64_t)__float_as_uint(kReset);  // before the first tile: state 0
        }
        bool known = false;
        float h = 0.f;
#pragma unroll
        for (int i = kWindow - 1; i >= 0; --i) {
            const float A = __uint_as_float((uint32_t)m[i]), B = __uint_as_float((uint32_t)(m[i] >> 32));
            const bool state = A < 0.f;
            h = state ? B : __builtin_fmaf(A, h, B);
            known = m[i] != kEmpty && (state || known);
        }
        if (known) return h;
        __builtin_amdgcn_s_sleep(2);
    }
}
// the workgroup's tile number in the launch: by ticket where tiles wait for each other
__device__ inline int take_tile(const ScanArgs& a, int* shared) {
    if (a.ntiles == 1) return blockIdx.x;
    if (threadIdx.x == 0) *shared = 1 + atomicAdd(a.ticket, 1);  // cleared to -1 like the words
    __syncthreads();
    const int t = __builtin_amdgcn_readfirstlane(*shared);
    __syncthreads();
    return t;
}
// before tiles that hand on their maps: words and ticket cleared, and each tile's first sequence found
template <int TT>
__global__ __launch_bounds__(SCAN_THREADS) void k_scan_init(ScanArgs a) {
    const int64_t n = a.ntiles * a.slots + 1, step = (int64_t)gridDim.x * SCAN_THREADS;
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

template <typename T, int V, int CL, int NT>
__global__ __launch_bounds__(SCAN_THREADS) void k_scan_fwd(ScanArgs a) {
    constexpr int G = SCAN_THREADS / CL, TT = G * NT, CB = CL * V;
    // the waves that hold one thread per channel
    constexpr int CW = (CB + 63) / 64 * 64;
    static_assert(2 * CW <= SCAN_THREADS, "two sets of one thread per channel");
    __shared__ int start[TT], last[TT];
    __shared__ f32x2 maps[G][CB];  // of the token groups, and the states that enter them
    __shared__ float into[G][CB];
    const int linear = take_tile(a, start);
    const Tile tile = tile_of(a, linear, TT, CB);
    Share<V, CL, NT> me(a, tile);
    const Seq seq(a, tile_sequence<TT>(a, tile));
    me.bounds(a);
    Raw<T, V> rf[NT], rg[NT], ro[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int64_t t = me.token(a, i);
        rf[i] = load_raw<V>(static_cast<const T*>(a.zf) + t * a.ldz + me.ch);
        rg[i] = load_raw<V>(static_cast<const T*>(a.g) + t * a.ldz + me.ch);
        if (a.zo) ro[i] = load_raw<V>(static_cast<const T*>(a.zo) + t * a.ldz + me.ch);
    }
    mark_tile<TT, CB>(a, tile, seq, start, last, a.h0, a.hT);
    float f[NT][V], b[NT][V], A[V], B[V];
    unsigned reset = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = 1.f;
        B[v] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const bool in = me.inside >> i & 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s, c;
            sigm2<T>(rf[i][v], s, c);
            f[i][v] = in ? s : 1.f;
            b[i][v] = in ? c * rg[i][v] : 0.f;
        }
        const int st = in ? start[me.group * NT + i] : 0;
        if (st) {
            reset |= 1u << i;
            if (a.h0) {
                float h[V];
                load_f32<V>(a.h0 + (int64_t)(st - 1) * a.D + me.ch, h);
#pragma unroll
                for (int v = 0; v < V; ++v) b[i][v] = __builtin_fmaf(f[i][v], h[v], b[i][v]);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            B[v] = st ? b[i][v] : __builtin_fmaf(f[i][v], B[v], b[i][v]);
            A[v] = A[v] * f[i][v];
        }
    }
    const int col = (threadIdx.x % CL) * V;
#pragma unroll
    for (int v = 0; v < V; ++v) maps[me.group][col + v] = f32x2{reset ? kReset : A[v], B[v]};
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
        float h = 0.f;
        if (a.ntiles > 1) {
            const int64_t k = linear / a.ncb, slot = tile.c0 + c;
            float ta, tb;
            tile_map(c, ta, tb);
            uint64_t* const w = a.words + slot;
            h = look_back(w, k, a.slots);
            if (!(ta < 0.f)) put_word(w + k * a.slots, kReset, __builtin_fmaf(ta, h, tb));
            a.carry[k * a.slots + slot] = h;
        }
#pragma unroll 8
        for (int j = 0; j < G; ++j) {
            const f32x2 m = maps[j][c];
            into[j][c] = h;
            h = apply_map(m[0], m[1], h);
        }
    }
    __syncthreads();
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = into[me.group][col + v];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const bool r = reset >> i & 1;
        float y[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = r ? b[i][v] : __builtin_fmaf(f[i][v], h[v], b[i][v]);
            y[v] = h[v];
            if (a.zo) {
                float s, c;
                sigm2<T>(ro[i][v], s, c);
                y[v] *= s;
            }
        }
        if (me.active && (me.inside >> i & 1)) {
            store_vec<V>(static_cast<T*>(a.y) + me.token(a, i) * a.ldy + me.ch, y);
            const int en = last[me.group * NT + i];
            if (en && a.hT) store_f32<V>(a.hT + (int64_t)(en - 1) * a.D + me.ch, h);
        }
    }
}

// Backward: the tile's states again from its incoming one in a.carry, and the reverse recurrence, whose tiles are
// chained from the last to the first. Gates stay encoded (sigm_enc) between the passes over the registers.
template <typename T, int V, int CL, int NT>
__global__ __launch_bounds__(SCAN_THREADS) void k_scan_bwd(ScanArgs a) {
    constexpr int G = SCAN_THREADS / CL, TT = G * NT, CB = CL * V;
    // the waves that hold one thread per channel
    constexpr int CW = (CB + 63) / 64 * 64;
    static_assert(2 * CW <= SCAN_THREADS, "two sets of one thread per channel");
    __shared__ int start[TT], last[TT];
    __shared__ f32x2 maps[G][CB], rmaps[G][CB];  // of the token groups, and what enters them
    __shared__ float into[G][CB], rinto[G][CB];
    const int ticket = take_tile(a, start);
    // the chain's k-th tile is the k-th from the end
    const int k = ticket / a.ncb, linear = ((int)a.ntiles - 1 - k) * a.ncb + ticket % a.ncb;
    const Tile tile = tile_of(a, linear, TT, CB);
    Share<V, CL, NT> me(a, tile);
    const Seq seq(a, tile_sequence<TT>(a, tile));
    me.bounds(a);
    Raw<T, V> rf[NT], rg[NT], ro[NT], rd[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int64_t t = me.token(a, i);
        rf[i] = load_raw<V>(static_cast<const T*>(a.zf) + t * a.ldz + me.ch);
        rg[i] = load_raw<V>(static_cast<const T*>(a.g) + t * a.ldz + me.ch);
        if (a.zo) ro[i] = load_raw<V>(static_cast<const T*>(a.zo) + t * a.ldz + me.ch);
        rd[i] = load_raw<V>(static_cast<const T*>(a.dy) + t * a.ldy + me.ch);
    }
    mark_tile<TT, CB>(a, tile, seq, start, last, a.dhT, a.dh0);
    unsigned reset = 0, ends = 0;
    float qf[NT][V], qo[NT][V];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const bool in = me.inside >> i & 1;
        if (in && start[me.group * NT + i]) reset |= 1u << i;
        if (in && last[me.group * NT + i]) ends |= 1u << i;
        if (!in) {  // a token of no sequence: state and gradient pass through, nothing enters
            rg[i] = Raw<T, V>{};
            rd[i] = Raw<T, V>{};
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            qf[i][v] = in ? sigm_enc<T>(rf[i][v]) : kSigmOne;
            qo[i][v] = a.zo && in ? sigm_enc<T>(ro[i][v]) : kSigmOne;
        }
    }
    // a sequence's incoming state at its first token, and the gradient of its last state at its last: rare, so read
    // where they are needed
    auto first_state = [&](int i, float(&h)[V]) {
        if ((reset >> i & 1)) {
            if (a.h0) load_f32<V>(a.h0 + (int64_t)(start[me.group * NT + i] - 1) * a.D + me.ch, h);
            else
#pragma unroll
                for (int v = 0; v < V; ++v) h[v] = 0.f;
        }
    };
    auto last_grad = [&](int i, float(&d)[V]) {
        if ((ends >> i & 1)) {
            if (a.dhT) load_f32<V>(a.dhT + (int64_t)(last[me.group * NT + i] - 1) * a.D + me.ch, d);
            else
#pragma unroll
                for (int v = 0; v < V; ++v) d[v] = 0.f;
        }
    };
    // decoded gates are not kept from one pass over the registers to the next (they would double its registers)
    auto forget = [&] {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) asm volatile("" : "+v"(qf[i][v]), "+v"(qo[i][v]));
    };
    const int col = (threadIdx.x % CL) * V;
    float A[V], h[V] = {}, d[V] = {};
#pragma unroll
    for (int v = 0; v < V; ++v) A[v] = 1.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        first_state(i, h);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f, c;
            sigm_dec(qf[i][v], f, c);
            h[v] = __builtin_fmaf(f, h[v], c * rg[i][v]);
            A[v] *= f;
        }
    }
    forget();
#pragma unroll
    for (int i = NT - 1; i >= 0; --i) {
        last_grad(i, d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f, c, so, co;
            sigm_dec(qf[i][v], f, c);
            sigm_dec(qo[i][v], so, co);
            d[v] = f * __builtin_fmaf(so, rd[i][v], d[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        maps[me.group][col + v] = f32x2{reset ? kReset : A[v], h[v]};
        rmaps[me.group][col + v] = f32x2{ends ? kReset : A[v], d[v]};
    }
    __syncthreads();
    // one thread per channel chains the reverse maps, one of other waves the forward ones, and a third, where there are
    // waves left, hands on the tile's own map
    constexpr bool kThird = 3 * CW <= SCAN_THREADS;
    auto tile_map = [&](int c, float& ta, float& tb) {
        ta = 1.f;
        tb = 0.f;
#pragma unroll 8
        for (int j = G - 1; j >= 0; --j) {
            const f32x2 m = rmaps[j][c];
            tb = apply_map(m[0], m[1], tb);
            ta = m[0] < 0.f || ta < 0.f ? kReset : ta * m[0];
        }
    };
    if (threadIdx.x < CB) {
        const int c = threadIdx.x;
        float x = 0.f;
        if (a.ntiles > 1) {
            float ta, tb;
            tile_map(c, ta, tb);
            uint64_t* const w = a.words + tile.c0 + c;
            if (!kThird) put_word(w + k * a.slots, ta, tb);
            x = look_back(w, k, a.slots);
            if (!(ta < 0.f)) put_word(w + k * a.slots, kReset, __builtin_fmaf(ta, x, tb));
        }
#pragma unroll 8
        for (int j = G - 1; j >= 0; --j) {
            const f32x2 m = rmaps[j][c];
            rinto[j][c] = x;
            x = apply_map(m[0], m[1], x);
        }
    }
    if (const int c = (int)threadIdx.x - CW; c >= 0 && c < CB) {
        float x = a.ntiles > 1 ? a.carry[linear / a.ncb * a.slots + tile.c0 + c] : 0.f;
#pragma unroll 8
        for (int j = 0; j < G; ++j) {
            const f32x2 m = maps[j][c];
            into[j][c] = x;
            x = apply_map(m[0], m[1], x);
        }
    }
    if (const int c = (int)threadIdx.x - 2 * CW; kThird && a.ntiles > 1 && c >= 0 && c < CB) {
        float ta, tb;
        tile_map(c, ta, tb);
        offer_word(a.words + k * a.slots + tile.c0 + c, ta, tb);
    }
    __syncthreads();
    forget();
    float prev[NT][V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        h[v] = into[me.group][col + v];
        d[v] = rinto[me.group][col + v];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        first_state(i, h);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f, c;
            sigm_dec(qf[i][v], f, c);
            prev[i][v] = h[v];
            h[v] = __builtin_fmaf(f, h[v], c * rg[i][v]);
        }
    }
    forget();
#pragma unroll
    for (int i = NT - 1; i >= 0; --i) {
        float dzf[V], dg[V], dzo[V];
        last_grad(i, d);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float f, c, so, co;
            sigm_dec(qf[i][v], f, c);
            sigm_dec(qo[i][v], so, co);
            const float g = rg[i][v], own = so * rd[i][v], lam = own + d[v];
            dg[v] = c * lam;
            dzf[v] = f * dg[v] * (prev[i][v] - g);
            dzo[v] = own * co * __builtin_fmaf(f, prev[i][v], c * g);
            d[v] = f * lam;
        }
        if (me.active && (me.inside >> i & 1)) {
            const int64_t o = me.token(a, i) * a.ldd + me.ch;
            store_vec<V>(static_cast<T*>(a.dzf) + o, dzf);
            store_vec<V>(static_cast<T*>(a.dg) + o, dg);
            if (a.zo) store_vec<V>(static_cast<T*>(a.dzo) + o, dzo);
            if ((reset >> i & 1) && a.dh0)
                store_f32<V>(a.dh0 + (int64_t)(start[me.group * NT + i] - 1) * a.D + me.ch, d);
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
    const int per = (D + V - 1) / V;
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

// the tile shape for a row: a vector of 16 bytes a thread (one element where the row is shorter), as many lanes along
// the row as it fills, at most 8; forward and backward have the same
template <typename F>
void with_shape(int D, int dtype, F&& fn) {
    auto go = [&](auto ty) {
        constexpr int V = Width<decltype(ty)>::v;
        if (D < V) return fn(ty, ScanShape<1, 8, 4>{});
        const int lanes = (D + V - 1) / V;
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
        p.seq = p.ntiles * p.slots * 8 + 8;
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
        a.ticket = reinterpret_cast<int32_t*>(w + p.ntiles * p.slots * 8);  // the word after the tiles'
        a.seq = reinterpret_cast<int32_t*>(w + p.seq);
        a.carry = reinterpret_cast<float*>(w + p.carry);
    }
    const dim3 grid((unsigned)(p.ntiles * p.ncb)), block(SCAN_THREADS);
    with_shape(a.D, dtype, [&](auto ty, auto sh) {
        using T = decltype(ty);
        using S = decltype(sh);
        if (p.ntiles > 1) {
            const int64_t n = std::max(p.ntiles * p.slots + 1, p.ntiles * 64);
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
        const int64_t n = (int64_t)S * ((D + V - 1) / V);
        launch(k_scan_step<T, V>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, S, D, static_cast<const T*>(zf),
               static_cast<const T*>(g), static_cast<const T*>(zo), ldz, slots, n_slots, h_in, h_out,
               static_cast<T*>(y), ldy);
    };
    if (dtype == 1) go(bf16{});
    else go(float{});
    return hipGetLastError();
}

}  // namespace mdl
