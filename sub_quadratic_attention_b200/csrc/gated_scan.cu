// gated_scan.cu -- the gated linear recurrence h_t = a_t h_{t-1} + b_t over sequences of
// rows, its backward pass and its single-token step, and their C ABI (gated_scan.h).
//
// Mathematics.  A stretch of rows takes the state h before it to P h + Q, P the product of
// its gates and Q its own result from 0; (P, Q) of two neighbouring stretches join as
// (P2 P1, P2 Q1 + Q2).  So a sequence is cut into chunks of 128 rows that are worked on at
// the same time, and only (P, Q) goes from chunk to chunk.  The backward pass is the same
// recurrence from the other end: E_t = a_t dh_t, dh_t = dy_t + E_{t+1}.
//
// Split.  The work is bound by memory (a few flops a byte), so each tensor is read once
// and written once in a single launch.  A block takes a tile of 128 rows by 64 channels
// (a row's part is 128 bytes of bf16): 16 lanes of 4 channels, 16 groups of 8 rows, each
// thread holding its 8 rows in registers.  A thread walks its rows once for (P, Q); the
// groups' pairs are joined in shared memory; the tile's pair is published to the blocks
// behind it and the state before the tile is found by looking back at the pairs published
// ahead of it; then the thread walks its rows again with the state and writes them.  The
// gates are not kept as (a, b) but as one number each, so that a tile costs few registers.
//
// Looking back.  A tile's pair is one 64-bit word in memory, written whole: readers need
// neither a flag nor a fence.  It is first (P, Q) and, when the state before the tile is
// known, (0, state behind it): a stretch that lets nothing through.  A reader goes back to
// the nearest pair with P = 0 and applies the pairs from there on in order, which is the
// arithmetic that the tiles between do themselves: the result is the same to the bit
// whichever of the two words it meets.  Tiles take their number from a counter, so the
// tiles that a waiting block looks at are held by blocks that run already.  A wait that
// finds nothing for about four seconds ends with NaN in the state and in all rows behind.
#include <new>

#include "gated_scan.h"
#include "rows_io.cuh"

struct gated_scan_s {
    int H, D, C;
    int gate, per;
    int dtype, gate_dtype;
    int device, nsm;
};

namespace gscan {

using namespace rows_io;

constexpr int CHUNK = GATED_SCAN_CHUNK;

struct Gate {
    float a, c;   // h = a h + c v
};

// A gate in one number.  exp: a itself.  sigmoid: the smaller of a = s(g) and 1 - a = s(-g),
// e / (1 + e) with e = exp(-|g|), to its own relative precision, with g's sign to tell which;
// the other is one minus it, exact to half a step since it is at least a half.
template <int FORM> __device__ __forceinline__ float pack_gate(float g) {
    if (FORM == GATED_SCAN_EXP) return expf(g);
    const float e = expf(-fabsf(g));
    return copysignf(e / (1.0f + e), g);
}
template <int FORM> __device__ __forceinline__ Gate open_gate(float k) {
    if (FORM == GATED_SCAN_EXP) return {k, 1.0f};
    const float s = fabsf(k), o = 1.0f - s;
    return signbit(k) ? Gate{s, o} : Gate{o, s};
}
template <int FORM> constexpr float HOLD = FORM == GATED_SCAN_EXP ? 1.0f : 0.0f;   // a = 1

// a * h where a factor of zero takes h out, NaN and infinities included
__device__ __forceinline__ float mul0(float a, float h) { return a == 0.0f ? 0.0f : a * h; }
__device__ __forceinline__ float fma0(float a, float h, float b) { return a == 0.0f ? b : fmaf(a, h, b); }

template <int FORM> __device__ __forceinline__ float input_of(Gate k, float v) {
    return FORM == GATED_SCAN_EXP ? v : mul0(k.c, v);
}
// d(h_t) / d(g_t) from the state before the row
template <int FORM> __device__ __forceinline__ float slope_of(Gate k, float before, float v) {
    return FORM == GATED_SCAN_EXP ? mul0(k.a, before) : mul0(k.a * k.c, before - v);
}


// A tile: CHUNK rows of WIDTH channels.  V channels a thread: 4 where rows and heads allow it,
// else 1 (then a row's part is 32 channels and a thread has 16 rows).
template <int V> struct Tile {
    static constexpr int LANES = V == 4 ? 16 : 32;
    static constexpr int WIDTH = LANES * V;
    static constexpr int ROWS = V == 4 ? 8 : 16;
    static constexpr int GROUPS = CHUNK / ROWS;
    static constexpr int THREADS = LANES * GROUPS;
};

// Workspace: a counter and one word for each tile and channel, all ones before a run.
constexpr size_t COUNTER_BYTES = 256;
constexpr unsigned long long NOTHING = ~0ull;
constexpr int WINDOW = 8;              // pairs that a reader asks for at a time
constexpr unsigned MOST_POLLS = 1u << 22;   // about a microsecond each

struct Args {
    gated_scan_args a;
    int H, D, C;
    int strips;               // tiles beside one another: ceil(C / WIDTH)
    int nchunk;
    long long nseq;           // dense: B
    unsigned *counter;        // null where a sequence has one chunk
    unsigned long long *words;
    float *parts;             // per-head gradients of heads that span strips: [pieces][B L][H]
};

template <typename T> __device__ __forceinline__ T *row(const gated_scan_rows &r, long long b, long long t) {
    return static_cast<T *>(r.data) + b * r.batch_stride + t * r.row_stride;
}

template <typename T, int V> struct alignas(sizeof(T) * V) Pack {
    T v[V];
};
template <typename T, int V> __device__ __forceinline__ Pack<T, V> load(const T *p) {
    return *reinterpret_cast<const Pack<T, V> *>(p);
}
template <typename T, int V> __device__ __forceinline__ void store(T *p, const float *f) {
    Pack<T, V> r;
#pragma unroll
    for (int j = 0; j < V; j++) r.v[j] = from_f<T>(f[j]);
    *reinterpret_cast<Pack<T, V> *>(p) = r;
}

// One 64-bit word is written and read whole, and everything that a reader needs is in it.
__device__ __forceinline__ unsigned long long peek(const unsigned long long *p) {
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void publish(unsigned long long *p, float P, float Q) {
    const unsigned hi = P == P ? __float_as_uint(P) : 0x7fc00000u;   // no NaN is NOTHING
    const unsigned long long v = ((unsigned long long)hi << 32) | __float_as_uint(Q);
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ float word_P(unsigned long long w) { return __uint_as_float((unsigned)(w >> 32)); }
__device__ __forceinline__ float word_Q(unsigned long long w) { return __uint_as_float((unsigned)w); }

// The state in front of tile i (counted in the direction of the walk) of a strip's channel:
// words[j * WIDTH] is tile j's.  Tile 0's word has P = 0.
template <int WIDTH> __device__ float look_back(const unsigned long long *words, int i) {
    int found = -1;
    float state = 0.0f;
    unsigned polls = 0;
    for (int last = i - 1; found < 0;) {
        unsigned long long w[WINDOW];
#pragma unroll
        for (int j = 0; j < WINDOW; j++) w[j] = last - j >= 0 ? peek(words + (long long)(last - j) * WIDTH) : 0;
        int from = -1;      // the nearest tile of this window that lets nothing through
        bool wait = false;
#pragma unroll
        for (int j = 0; j < WINDOW; j++) {
            if (from >= 0 || wait) continue;
            if (w[j] == NOTHING)
                wait = true;
            else if (word_P(w[j]) == 0.0f)
                from = j;
        }
        if (wait) {
            if (++polls > MOST_POLLS) return __uint_as_float(0x7fc00000u);
            continue;
        }
        if (from < 0) {
            last -= WINDOW;
            continue;
        }
#pragma unroll
        for (int j = WINDOW - 1; j >= 0; j--)
            if (j <= from) state = fma0(word_P(w[j]), state, word_Q(w[j]));
        found = last;
    }
    // the tiles behind this window: their words are there, as pairs or already as states
    for (int j = found + 1; j < i; j += WINDOW) {
        unsigned long long w[WINDOW];
#pragma unroll
        for (int k = 0; k < WINDOW; k++) w[k] = j + k < i ? peek(words + (long long)(j + k) * WIDTH) : 0;
#pragma unroll
        for (int k = 0; k < WINDOW; k++)
            if (j + k < i) state = fma0(word_P(w[k]), state, word_Q(w[k]));
    }
    return state;
}

// Where the block's tile lies.  Tiles are numbered chunk by chunk over all batch entries and
// strips, in the direction of the walk, so that every strip advances at the same time.
struct Place {
    int i, strip;        // chunk in walking order
    long long b, tile;   // tile: the strip's first word
};
__device__ __forceinline__ Place place_of(const Args &p, unsigned *shared_ticket) {
    unsigned ticket = blockIdx.x;
    if (p.counter) {
        if (threadIdx.x == 0) *shared_ticket = atomicAdd(p.counter, 1u) + 1u;   // the counter starts at all ones
        __syncthreads();
        ticket = *shared_ticket;
    }
    const unsigned per = (unsigned)(p.a.B * p.strips), i = ticket / per, rest = ticket - i * per;
    Place t;
    t.i = (int)i;
    t.b = rest / p.strips;
    t.strip = (int)(rest - (unsigned)t.b * p.strips);
    t.tile = (t.b * p.strips + t.strip) * p.nchunk;
    return t;
}

// Packed rows: the sequence that starts at, and that ends with, each row of the tile (or -1),
// and the rows that lie in sequences at all.
struct Marks {
    int first[CHUNK], last[CHUNK];
};
__device__ __forceinline__ void mark_sequences(const Args &p, Marks &m, long long t0, long long &lo, long long &hi) {
    const int *cu = p.a.cu_seqlens;
    for (int i = threadIdx.x; i < CHUNK; i += blockDim.x) m.first[i] = m.last[i] = -1;
    __syncthreads();
    for (long long n = threadIdx.x; n < p.nseq; n += blockDim.x) {
        const long long s = cu[n], e = cu[n + 1];
        if (s >= e) continue;
        if (s >= t0 && s < t0 + CHUNK) m.first[s - t0] = (int)n;
        if (e > t0 && e <= t0 + CHUNK) m.last[e - 1 - t0] = (int)n;
    }
    __syncthreads();
    lo = cu[0] > lo ? cu[0] : lo;
    hi = cu[p.nseq] < hi ? cu[p.nseq] : hi;
}

// What an empty sequence's ends are: the state goes through.
__device__ __forceinline__ void pass_empty(const Args &p, const float *from, float *to, int c0, int width) {
    if (!to) return;
    for (long long i = threadIdx.x; i < p.nseq * width; i += blockDim.x) {
        const long long n = i / width;
        const int c = c0 + (int)(i % width);
        if (c < p.C && p.a.cu_seqlens[n] >= p.a.cu_seqlens[n + 1]) to[n * p.C + c] = from ? from[n * p.C + c] : 0.0f;
    }
}
__global__ void pass_all(const float *from, float *to, long long n) {
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (i < n) to[i] = from ? from[i] : 0.0f;
}

template <typename TV, typename TG, int FORM, bool HEAD, int V>
__global__ void __launch_bounds__(Tile<V>::THREADS, 2) scan_forward(Args p) {
    using S = Tile<V>;
    __shared__ float sP[S::GROUPS][S::WIDTH], sQ[S::GROUPS][S::WIDTH], sState[S::WIDTH];
    __shared__ Marks marks;
    __shared__ unsigned ticket;
    const Place at = place_of(p, &ticket);
    const int lane = threadIdx.x % S::LANES, group = threadIdx.x / S::LANES;
    const int c0 = at.strip * S::WIDTH, c = c0 + lane * V;
    const bool mine = c < p.C;
    const bool packed = p.a.cu_seqlens != nullptr;
    const long long tile0 = (long long)at.i * CHUNK, t0 = tile0 + group * S::ROWS;
    long long lo = 0, hi = p.a.L;

    constexpr int GV = HEAD ? 1 : V;
    const int gc = HEAD ? c / p.D : c;
    float k[S::ROWS][GV];
    Pack<TV, V> v[S::ROWS];
    {
        Pack<TG, GV> g[S::ROWS];
#pragma unroll
        for (int r = 0; r < S::ROWS; r++) {
            const bool in = mine && t0 + r < p.a.L;
            if (in) {
                g[r] = load<TG, GV>(row<TG>(p.a.g, at.b, t0 + r) + gc);
                v[r] = load<TV, V>(row<TV>(p.a.v, at.b, t0 + r) + c);
            }
        }
        if (packed) mark_sequences(p, marks, tile0, lo, hi);
#pragma unroll
        for (int r = 0; r < S::ROWS; r++) {
            const bool in = mine && t0 + r >= lo && t0 + r < hi;
#pragma unroll
            for (int j = 0; j < GV; j++) k[r][j] = in ? pack_gate<FORM>(to_f(g[r].v[j])) : HOLD<FORM>;
            if (!in)
#pragma unroll
                for (int j = 0; j < V; j++) v[r].v[j] = from_f<TV>(0.0f);
        }
    }

    float P[V], Q[V];
#pragma unroll
    for (int j = 0; j < V; j++) P[j] = 1.0f, Q[j] = 0.0f;
#pragma unroll
    for (int r = 0; r < S::ROWS; r++) {
        if (packed && mine) {
            const int n = marks.first[group * S::ROWS + r];
            if (n >= 0)
#pragma unroll
                for (int j = 0; j < V; j++) P[j] = 0.0f, Q[j] = p.a.h0 ? p.a.h0[(long long)n * p.C + c + j] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < V; j++) {
            const Gate q = open_gate<FORM>(k[r][HEAD ? 0 : j]);
            Q[j] = fma0(q.a, Q[j], input_of<FORM>(q, to_f(v[r].v[j])));
            P[j] *= q.a;
        }
    }
#pragma unroll
    for (int j = 0; j < V; j++) sP[group][lane * V + j] = P[j], sQ[group][lane * V + j] = Q[j];
    __syncthreads();

    if (threadIdx.x < S::WIDTH) {
        // each group's pair becomes that of all groups ahead of it
        const int x = threadIdx.x, cx = c0 + x;
        float allP = 1.0f, allQ = 0.0f;
#pragma unroll
        for (int i = 0; i < S::GROUPS; i++) {
            const float gP = sP[i][x], gQ = sQ[i][x];
            sP[i][x] = allP;
            sQ[i][x] = allQ;
            allQ = fma0(gP, allQ, gQ);
            allP *= gP;
        }
        float state = 0.0f;
        if (cx < p.C) {
            unsigned long long *words = p.words + at.tile * S::WIDTH + x;
            const bool more = at.i + 1 < p.nchunk;
            if (at.i == 0) {
                if (!packed && p.a.h0) state = p.a.h0[at.b * p.C + cx];
            } else {
                if (more && allP != 0.0f) publish(words + (long long)at.i * S::WIDTH, allP, allQ);
                state = look_back<S::WIDTH>(words, at.i);
            }
            if (more) publish(words + (long long)at.i * S::WIDTH, 0.0f, fma0(allP, state, allQ));
            if (p.a.states) p.a.states[(at.b * p.nchunk + at.i) * p.C + cx] = state;
        }
        sState[x] = state;
    }
    __syncthreads();

    if (mine) {
        float h[V];
#pragma unroll
        for (int j = 0; j < V; j++) h[j] = fma0(sP[group][lane * V + j], sState[lane * V + j], sQ[group][lane * V + j]);
#pragma unroll
        for (int r = 0; r < S::ROWS; r++) {
            const long long t = t0 + r;
            if (t >= p.a.L) break;
            if (packed) {
                const int n = marks.first[group * S::ROWS + r];
                if (n >= 0)
#pragma unroll
                    for (int j = 0; j < V; j++) h[j] = p.a.h0 ? p.a.h0[(long long)n * p.C + c + j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < V; j++) {
                const Gate q = open_gate<FORM>(k[r][HEAD ? 0 : j]);
                h[j] = fma0(q.a, h[j], input_of<FORM>(q, to_f(v[r].v[j])));
            }
            if (t >= lo && t < hi) {
                store<TV, V>(row<TV>(p.a.y, at.b, t) + c, h);
                if (p.a.hT) {
                    const long long n = packed ? marks.last[group * S::ROWS + r] : t == p.a.L - 1 ? at.b : -1;
                    if (n >= 0)
#pragma unroll
                        for (int j = 0; j < V; j++) p.a.hT[n * p.C + c + j] = h[j];
                }
            } else if (p.a.zero_outside) {
                const float zero[V] = {};
                store<TV, V>(row<TV>(p.a.y, at.b, t) + c, zero);
            }
        }
    }
    if (packed && at.i == 0) pass_empty(p, p.a.h0, p.a.hT, c0, S::WIDTH);
}

// The strips that the channels of head h lie in.
__host__ __device__ __forceinline__ int first_strip(int h, int D, int width) { return (int)((long long)h * D / width); }
__host__ __device__ __forceinline__ int last_strip(int h, int D, int width) { return (int)(((long long)h * D + D - 1) / width); }

template <typename TV, typename TG, int FORM, bool HEAD, int V>
__global__ void __launch_bounds__(Tile<V>::THREADS, 2) scan_backward(Args p) {
    using S = Tile<V>;
    // (P, Q) of the states going forward, (R, E) of the gradients going back
    __shared__ float sP[S::GROUPS][S::WIDTH], sQ[S::GROUPS][S::WIDTH];
    __shared__ float sR[S::GROUPS][S::WIDTH], sE[S::GROUPS][S::WIDTH], sGrad[S::WIDTH];
    __shared__ Marks marks;
    __shared__ unsigned ticket;
    const Place at = place_of(p, &ticket);
    const int chunk = p.nchunk - 1 - at.i;
    const int lane = threadIdx.x % S::LANES, group = threadIdx.x / S::LANES;
    const int c0 = at.strip * S::WIDTH, c = c0 + lane * V;
    const bool mine = c < p.C;
    const bool packed = p.a.cu_seqlens != nullptr;
    const long long tile0 = (long long)chunk * CHUNK, t0 = tile0 + group * S::ROWS;
    long long lo = 0, hi = p.a.L;

    constexpr int GV = HEAD ? 1 : V;
    const int gc = HEAD ? c / p.D : c;
    float k[S::ROWS][GV];
    Pack<TV, V> v[S::ROWS], dy[S::ROWS];
    {
        Pack<TG, GV> g[S::ROWS];
#pragma unroll
        for (int r = 0; r < S::ROWS; r++) {
            if (mine && t0 + r < p.a.L) {
                g[r] = load<TG, GV>(row<TG>(p.a.g, at.b, t0 + r) + gc);
                v[r] = load<TV, V>(row<TV>(p.a.v, at.b, t0 + r) + c);
                dy[r] = load<TV, V>(row<TV>(p.a.dy, at.b, t0 + r) + c);
            }
        }
        if (packed) mark_sequences(p, marks, tile0, lo, hi);
#pragma unroll
        for (int r = 0; r < S::ROWS; r++) {
            const bool in = mine && t0 + r >= lo && t0 + r < hi;
#pragma unroll
            for (int j = 0; j < GV; j++) k[r][j] = in ? pack_gate<FORM>(to_f(g[r].v[j])) : HOLD<FORM>;
            if (!in)
#pragma unroll
                for (int j = 0; j < V; j++) v[r].v[j] = dy[r].v[j] = from_f<TV>(0.0f);
        }
    }

    // the sequence that row r starts or ends, or -1
    auto starts = [&](int r) -> long long {
        if (packed) return marks.first[group * S::ROWS + r];
        return t0 + r == 0 ? at.b : -1;
    };
    auto ends = [&](int r) -> long long {
        if (packed) return marks.last[group * S::ROWS + r];
        return t0 + r == p.a.L - 1 ? at.b : -1;
    };

    float P[V], Q[V];
#pragma unroll
    for (int j = 0; j < V; j++) P[j] = 1.0f, Q[j] = 0.0f;
#pragma unroll
    for (int r = 0; r < S::ROWS; r++) {
        const long long n = packed && mine ? starts(r) : -1;
        if (n >= 0)
#pragma unroll
            for (int j = 0; j < V; j++) P[j] = 0.0f, Q[j] = p.a.h0 ? p.a.h0[n * p.C + c + j] : 0.0f;
#pragma unroll
        for (int j = 0; j < V; j++) {
            const Gate q = open_gate<FORM>(k[r][HEAD ? 0 : j]);
            Q[j] = fma0(q.a, Q[j], input_of<FORM>(q, to_f(v[r].v[j])));
            P[j] *= q.a;
        }
    }
#pragma unroll
    for (int j = 0; j < V; j++) sP[group][lane * V + j] = P[j], sQ[group][lane * V + j] = Q[j];
#pragma unroll
    for (int j = 0; j < V; j++) P[j] = 1.0f, Q[j] = 0.0f;
#pragma unroll
    for (int r = S::ROWS - 1; r >= 0; r--) {
        const long long n = mine ? ends(r) : -1;
        if (n >= 0)
#pragma unroll
            for (int j = 0; j < V; j++) P[j] = 0.0f, Q[j] = p.a.dhT ? p.a.dhT[n * p.C + c + j] : 0.0f;
#pragma unroll
        for (int j = 0; j < V; j++) {
            const Gate q = open_gate<FORM>(k[r][HEAD ? 0 : j]);
            Q[j] = mul0(q.a, to_f(dy[r].v[j]) + Q[j]);
            P[j] *= q.a;
        }
    }
#pragma unroll
    for (int j = 0; j < V; j++) sR[group][lane * V + j] = P[j], sE[group][lane * V + j] = Q[j];
    __syncthreads();

    // one warp or two join the gradients and look back; others find the groups' states
    if (threadIdx.x < S::WIDTH) {
        const int x = threadIdx.x, cx = c0 + x;
        float allP = 1.0f, allQ = 0.0f;
#pragma unroll
        for (int i = S::GROUPS - 1; i >= 0; i--) {
            const float gP = sR[i][x], gQ = sE[i][x];
            sR[i][x] = allP;
            sE[i][x] = allQ;
            allQ = fma0(gP, allQ, gQ);
            allP *= gP;
        }
        float grad = 0.0f;
        if (cx < p.C) {
            unsigned long long *words = p.words + at.tile * S::WIDTH + x;
            const bool more = at.i + 1 < p.nchunk;
            if (at.i > 0) {
                if (more && allP != 0.0f) publish(words + (long long)at.i * S::WIDTH, allP, allQ);
                grad = look_back<S::WIDTH>(words, at.i);
            }
            if (more) publish(words + (long long)at.i * S::WIDTH, 0.0f, fma0(allP, grad, allQ));
        }
        sGrad[x] = grad;
    } else if (threadIdx.x < 2 * S::WIDTH) {
        const int x = threadIdx.x - S::WIDTH, cx = c0 + x;
        float h = cx < p.C ? p.a.states[(at.b * p.nchunk + chunk) * p.C + cx] : 0.0f;
#pragma unroll
        for (int i = 0; i < S::GROUPS; i++) {
            const float gP = sP[i][x], gQ = sQ[i][x];
            sQ[i][x] = h;
            h = fma0(gP, h, gQ);
        }
    }
    __syncthreads();

    // forward again for the gate's slope at every row, then back with the gradient
    float slope[S::ROWS][V];
    float h[V], e[V];
#pragma unroll
    for (int j = 0; j < V; j++) {
        h[j] = sQ[group][lane * V + j];
        e[j] = fma0(sR[group][lane * V + j], sGrad[lane * V + j], sE[group][lane * V + j]);
    }
#pragma unroll
    for (int r = 0; r < S::ROWS; r++) {
        const long long n = packed && mine ? starts(r) : -1;
        if (n >= 0)
#pragma unroll
            for (int j = 0; j < V; j++) h[j] = p.a.h0 ? p.a.h0[n * p.C + c + j] : 0.0f;
#pragma unroll
        for (int j = 0; j < V; j++) {
            const Gate q = open_gate<FORM>(k[r][HEAD ? 0 : j]);
            const float vv = to_f(v[r].v[j]);
            slope[r][j] = slope_of<FORM>(q, h[j], vv);
            h[j] = fma0(q.a, h[j], input_of<FORM>(q, vv));
        }
    }
    // lanes of one head: lane + o still in it
    bool same[4];
    int pieces = 1, piece = 0;
    bool leader = true;
    if (HEAD) {
#pragma unroll
        for (int o = 0; o < 4; o++) {
            const int other = c + (V << o);
            same[o] = lane + (1 << o) < S::LANES && other < p.C && other / p.D == gc;
        }
        leader = mine && (lane == 0 || (c - V) / p.D != gc);
        if (mine) piece = at.strip - first_strip(gc, p.D, S::WIDTH);
        pieces = p.parts ? 2 : 1;
    }
    const bool wide5 = HEAD && S::LANES == 32;
    const bool same5 = wide5 && lane + 16 < S::LANES && c + 16 * V < p.C && (c + 16 * V) / p.D == gc;
#pragma unroll
    for (int r = S::ROWS - 1; r >= 0; r--) {
        const long long t = t0 + r;
        const bool in = mine && t >= lo && t < hi;
        const long long n = mine && t < p.a.L ? ends(r) : -1;
        if (n >= 0)
#pragma unroll
            for (int j = 0; j < V; j++) e[j] = p.a.dhT ? p.a.dhT[n * p.C + c + j] : 0.0f;
        float dv[V], dg[V];
#pragma unroll
        for (int j = 0; j < V; j++) {
            const Gate q = open_gate<FORM>(k[r][HEAD ? 0 : j]);
            const float dh = to_f(dy[r].v[j]) + e[j];
            dg[j] = slope[r][j] * dh;
            dv[j] = FORM == GATED_SCAN_EXP ? dh : mul0(q.c, dh);
            e[j] = mul0(q.a, dh);
        }
        if (mine && t < p.a.L && !in && p.a.zero_outside)
#pragma unroll
            for (int j = 0; j < V; j++) dv[j] = dg[j] = 0.0f;
        const bool write = in || (mine && t < p.a.L && p.a.zero_outside);
        if (write) store<TV, V>(row<TV>(p.a.dv, at.b, t) + c, dv);
        if constexpr (!HEAD) {
            if (write) store<TG, V>(row<TG>(p.a.dg, at.b, t) + c, dg);
        } else {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < V; j++) s += write ? dg[j] : 0.0f;
#pragma unroll
            for (int o = 0; o < 4; o++) {
                const float other = __shfl_down_sync(0xffffffffu, s, 1 << o, S::LANES);
                s += same[o] ? other : 0.0f;
            }
            if (wide5) {
                const float other = __shfl_down_sync(0xffffffffu, s, 16, S::LANES);
                s += same5 ? other : 0.0f;
            }
            if (write && leader) {
                if (pieces == 1)
                    row<TG>(p.a.dg, at.b, t)[gc] = from_f<TG>(s);
                else
                    p.parts[(piece * p.a.B * p.a.L + at.b * p.a.L + t) * p.H + gc] = s;
            }
        }
        if (in && p.a.dh0) {
            const long long m = starts(r);
            if (m >= 0)
#pragma unroll
                for (int j = 0; j < V; j++) p.a.dh0[m * p.C + c + j] = e[j];
        }
    }
    if (packed && at.i == 0) pass_empty(p, p.a.dhT, p.a.dh0, c0, S::WIDTH);
}

// The gate's gradient of heads that span strips: their strips' sums, in order.
template <typename TG> __global__ void join_parts(Args p, int width) {
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x, rows = p.a.B * p.a.L;
    if (i >= rows * p.H) return;
    const int h = (int)(i % p.H);
    const long long r = i / p.H, b = r / p.a.L, t = r % p.a.L;
    if (p.a.cu_seqlens && !p.a.zero_outside && (t < p.a.cu_seqlens[0] || t >= p.a.cu_seqlens[p.nseq])) return;
    const int n = last_strip(h, p.D, width) - first_strip(h, p.D, width) + 1;
    float s = 0.0f;
    for (int k = 0; k < n; k++) s += p.parts[(k * rows + r) * p.H + h];
    row<TG>(p.a.dg, b, t)[h] = from_f<TG>(s);
}

// One token: thread (i, c); a slot named by an earlier row is that row's to finish.
template <typename TV, typename TG, int FORM>
__global__ void scan_step(long long B, int C, int D, int per, const TG *g, long long gs, const TV *v,
                          long long vs, const float *state, long long S, const int *slots, TV *y,
                          long long ys, float *next) {
    const int c = blockIdx.y * blockDim.x + threadIdx.x;
    const long long i0 = blockIdx.x;
    const long long slot = slots ? slots[i0] : i0;
    if (slot < 0 || slot >= S) return;
    bool first = true;
    if (slots)
        for (long long j = 0; j < i0; j++) first &= slots[j] != slot;
    if (!first || c >= C) return;
    const int gc = per == GATED_SCAN_PER_HEAD ? c / D : c;
    float h = state[slot * C + c];
    for (long long i = i0; i < B; i++) {
        if (i != i0 && (!slots || slots[i] != slot)) continue;
        const Gate k = open_gate<FORM>(pack_gate<FORM>(to_f(g[i * gs + gc])));
        h = fma0(k.a, h, input_of<FORM>(k, to_f(v[i * vs + c])));
        y[i * ys + c] = from_f<TV>(h);
    }
    next[slot * C + c] = h;
}

// what one output of `width` values a row needs for its rows to lie apart
bool rows_apart(const gated_scan_rows &r, long long B, long long L, long long width) {
    const long long bs = r.batch_stride, rs = r.row_stride;
    if (L > 1 && rs < width) return false;
    if (B > 1 && bs < width) return false;
    if (B > 1 && L > 1) return bs >= (L - 1) * rs + width || rs >= (B - 1) * bs + width;
    return true;
}

bool strides_ok(const gated_scan_rows &r) { return r.batch_stride >= 0 && r.row_stride >= 0; }

size_t elem(int dtype) { return dtype == SPECTRE_F32 ? 4 : 2; }

// The tensors' strips: V = 4 where a head's (or a row's) channels come in fours and every
// access of four is aligned, else 1.
template <int V> int strips_of(int C) { return (C + Tile<V>::WIDTH - 1) / Tile<V>::WIDTH; }
int strips_of(int C, int V) { return V == 4 ? strips_of<4>(C) : strips_of<1>(C); }
int width_of(int V) { return V == 4 ? Tile<4>::WIDTH : Tile<1>::WIDTH; }

// The most strips that a head's channels lie in.
int pieces_of(const gated_scan_s *h, int V) {
    if (h->per != GATED_SCAN_PER_HEAD) return 1;
    const int w = width_of(V);
    if (w % h->D == 0) return 1;
    int most = 1;
    // the first channels of heads within a strip repeat after w heads at the latest
    for (int i = 0; i < h->H && i < w; i++) {
        const int n = last_strip(i, h->D, w) - first_strip(i, h->D, w) + 1;
        most = n > most ? n : most;
    }
    return most;
}

struct Work {
    size_t words, parts, bytes;   // offset of the parts, the whole
};
Work work_of(const gated_scan_s *h, long long B, long long L, bool backward, int V) {
    const size_t nchunk = (L + CHUNK - 1) / CHUNK;
    Work w{};
    if (nchunk > 1) w.words = COUNTER_BYTES + (size_t)B * strips_of(h->C, V) * nchunk * width_of(V) * 8;
    w.words = (w.words + 255) / 256 * 256;
    const int pieces = backward ? pieces_of(h, V) : 1;
    if (pieces > 1) w.parts = (size_t)pieces * B * L * h->H * sizeof(float);
    w.bytes = w.words + w.parts;
    return w;
}

// What a caller provides: enough for either V.
size_t workspace(const gated_scan_s *h, long long B, long long L, bool backward) {
    const size_t four = work_of(h, B, L, backward, 4).bytes, one = work_of(h, B, L, backward, 1).bytes;
    return four > one ? four : one;
}

bool fours(const gated_scan_rows &r, size_t es) {
    return aligned(r.data, 4 * es) && r.batch_stride % 4 == 0 && r.row_stride % 4 == 0;
}
int vector_of(const gated_scan_s *h, const gated_scan_args *a, bool backward) {
    const bool head = h->per == GATED_SCAN_PER_HEAD;
    if ((head ? h->D : h->C) % 4) return 1;
    const size_t ev = elem(h->dtype), eg = elem(h->gate_dtype);
    if (!fours(a->v, ev) || (!head && !fours(a->g, eg))) return 1;
    if (!backward) return fours(a->y, ev) ? 4 : 1;
    return fours(a->dy, ev) && fours(a->dv, ev) && (head || fours(a->dg, eg)) ? 4 : 1;
}

template <typename TV, typename TG, int FORM, bool HEAD, int V>
cudaError_t launch_tiles(Args &p, bool backward, const Work &w, cudaStream_t s) {
    const long long tiles = p.a.B * p.strips * p.nchunk;
    if (w.words) {
        p.counter = static_cast<unsigned *>(p.a.work);
        p.words = reinterpret_cast<unsigned long long *>(static_cast<char *>(p.a.work) + COUNTER_BYTES);
        const cudaError_t e = cudaMemsetAsync(p.a.work, 0xff, w.words, s);
        if (e != cudaSuccess) return e;
    }
    if (w.parts) p.parts = reinterpret_cast<float *>(static_cast<char *>(p.a.work) + w.words);
    if (!backward)
        scan_forward<TV, TG, FORM, HEAD, V><<<(unsigned)tiles, Tile<V>::THREADS, 0, s>>>(p);
    else
        scan_backward<TV, TG, FORM, HEAD, V><<<(unsigned)tiles, Tile<V>::THREADS, 0, s>>>(p);
    if (w.parts) {
        const long long n = p.a.B * p.a.L * p.H;
        join_parts<TG><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p, Tile<V>::WIDTH);
    }
    return cudaGetLastError();
}

template <typename TV, typename TG, int FORM>
cudaError_t launch(Args &p, bool head, int V, bool backward, const Work &w, cudaStream_t s) {
    if (V == 4)
        return head ? launch_tiles<TV, TG, FORM, true, 4>(p, backward, w, s) : launch_tiles<TV, TG, FORM, false, 4>(p, backward, w, s);
    return head ? launch_tiles<TV, TG, FORM, true, 1>(p, backward, w, s) : launch_tiles<TV, TG, FORM, false, 1>(p, backward, w, s);
}

template <int FORM>
cudaError_t launch_types(const gated_scan_s *h, Args &p, int V, bool backward, const Work &w, cudaStream_t s) {
    const bool head = h->per == GATED_SCAN_PER_HEAD;
    if (h->dtype == SPECTRE_F32) return launch<float, float, FORM>(p, head, V, backward, w, s);
    if (h->gate_dtype == SPECTRE_F32) return launch<__nv_bfloat16, float, FORM>(p, head, V, backward, w, s);
    return launch<__nv_bfloat16, __nv_bfloat16, FORM>(p, head, V, backward, w, s);
}

int run(gated_scan_s *h, const gated_scan_args *a, bool backward, void *stream) {
    if (!h || !a || a->B < 0 || a->L < 0) return SPECTRE_ERR_ARG;
    const bool packed = a->cu_seqlens != nullptr;
    if (packed && (a->B != 1 || a->nseq < 0 || a->L > 0x7fffffffLL)) return SPECTRE_ERR_ARG;
    const long long nseq = packed ? a->nseq : a->B;
    if (a->B == 0 || (packed && nseq == 0 && !a->zero_outside)) return SPECTRE_OK;
    const int gw = h->per == GATED_SCAN_PER_HEAD ? h->H : h->C;
    // tiles are counted in 31 bits, and every index stays well inside 63
    if (a->L > (1LL << 40) || a->B > (1LL << 31) || nseq > (1LL << 40) / h->C) return SPECTRE_ERR_ARG;
    const long long nchunk = (a->L + CHUNK - 1) / CHUNK;
    if (nchunk && nchunk * a->B > 0x7fffffffLL / strips_of(h->C, 1)) return SPECTRE_ERR_ARG;
    const int V = vector_of(h, a, backward);
    const Work work = a->L ? work_of(h, a->B, a->L, backward, V) : Work{};
    const size_t ev = elem(h->dtype), eg = elem(h->gate_dtype);
    if (a->L > 0) {
        const gated_scan_rows *in[3] = {&a->g, &a->v, &a->dy};
        for (int i = 0; i < (backward ? 3 : 2); i++) {
            if (!in[i]->data || !strides_ok(*in[i])) return SPECTRE_ERR_ARG;
            if (!aligned(in[i]->data, i ? ev : eg)) return SPECTRE_ERR_ALIGN;
        }
        if (!backward) {
            if (!a->y.data || !rows_apart(a->y, a->B, a->L, h->C)) return SPECTRE_ERR_ARG;
            if (!aligned(a->y.data, ev)) return SPECTRE_ERR_ALIGN;
        } else {
            if (!a->dg.data || !a->dv.data || !a->states || !rows_apart(a->dg, a->B, a->L, gw) ||
                !rows_apart(a->dv, a->B, a->L, h->C))
                return SPECTRE_ERR_ARG;
            if (!aligned(a->dg.data, eg) || !aligned(a->dv.data, ev)) return SPECTRE_ERR_ALIGN;
        }
        const size_t need = workspace(h, a->B, a->L, backward);
        if (need && (!a->work || a->work_bytes < need)) return SPECTRE_ERR_ARG;
        if (need && !aligned(a->work, 256)) return SPECTRE_ERR_ALIGN;
    }
    if (!aligned(a->h0, 4) || !aligned(a->hT, 4) || !aligned(a->dhT, 4) || !aligned(a->dh0, 4) ||
        !aligned(a->states, 4) || !aligned(a->cu_seqlens, 4))
        return SPECTRE_ERR_ALIGN;
    if (!current_device_is(h->device)) return SPECTRE_ERR_DEVICE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->L == 0) {   // no rows: the states go through
        float *to = backward ? a->dh0 : a->hT;
        const long long n = nseq * h->C;
        if (!to || !n) return SPECTRE_OK;
        pass_all<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(backward ? a->dhT : a->h0, to, n);
        return status_of(cudaGetLastError());
    }
    Args p{};
    p.a = *a;
    p.H = h->H;
    p.D = h->D;
    p.C = h->C;
    p.strips = strips_of(h->C, V);
    p.nchunk = (int)nchunk;
    p.nseq = nseq;
    return status_of(h->gate == GATED_SCAN_EXP ? launch_types<GATED_SCAN_EXP>(h, p, V, backward, work, s)
                                               : launch_types<GATED_SCAN_SIGMOID>(h, p, V, backward, work, s));
}

template <typename TV, typename TG, int FORM>
cudaError_t launch_step(const gated_scan_s *h, long long B, const void *g, long long gs, const void *v,
                        long long vs, const float *state, long long S, const int *slots, void *y,
                        long long ys, float *next, cudaStream_t s) {
    const dim3 grid((unsigned)B, (h->C + 127) / 128);
    scan_step<TV, TG, FORM><<<grid, 128, 0, s>>>(B, h->C, h->D, h->per, static_cast<const TG *>(g), gs,
                                                 static_cast<const TV *>(v), vs, state, S, slots,
                                                 static_cast<TV *>(y), ys, next);
    return cudaGetLastError();
}

}  // namespace gscan

extern "C" {

int gated_scan_create(gated_scan_t *out, int H, int D, int gate, int per, int dtype, int gate_dtype) {
    if (!out) return SPECTRE_ERR_ARG;
    *out = nullptr;
    if (H < 1 || D < 1 || (long long)H * D > (1 << 20)) return SPECTRE_ERR_ARG;
    if (gate != GATED_SCAN_SIGMOID && gate != GATED_SCAN_EXP) return SPECTRE_ERR_ARG;
    if (per != GATED_SCAN_PER_CHANNEL && per != GATED_SCAN_PER_HEAD) return SPECTRE_ERR_ARG;
    if (dtype != SPECTRE_F32 && dtype != SPECTRE_BF16) return SPECTRE_ERR_ARG;
    if (gate_dtype != SPECTRE_F32 && (gate_dtype != SPECTRE_BF16 || dtype == SPECTRE_F32)) return SPECTRE_ERR_ARG;
    int dev = -1, nsm = 0;
    const int st = rows_io::usable_device(&dev, &nsm);
    if (st != SPECTRE_OK) return st;
    gated_scan_s *h = new (std::nothrow) gated_scan_s{H, D, H * D, gate, per, dtype, gate_dtype, dev, nsm};
    if (!h) return SPECTRE_ERR_NOMEM;
    *out = h;
    return SPECTRE_OK;
}

size_t gated_scan_workspace_bytes(gated_scan_t h, long long B, long long L, int backward) {
    return !h || B < 1 || L < 1 ? 0 : gscan::workspace(h, B, L, backward != 0);
}

int gated_scan_run(gated_scan_t h, const gated_scan_args *a, void *stream) {
    return gscan::run(h, a, false, stream);
}

int gated_scan_backward(gated_scan_t h, const gated_scan_args *a, void *stream) {
    return gscan::run(h, a, true, stream);
}

int gated_scan_step(gated_scan_t h, long long B, const void *g, long long g_stride, const void *v,
                    long long v_stride, const float *state, long long S, const int *slots, void *y,
                    long long y_stride, float *new_state, void *stream) {
    using namespace gscan;
    if (!h || B < 0 || S < 0) return SPECTRE_ERR_ARG;
    if (B == 0) return SPECTRE_OK;
    if (!g || !v || !state || !y || !new_state || g_stride < 0 || v_stride < 0 || (B > 1 && y_stride < h->C))
        return SPECTRE_ERR_ARG;
    if (B > 0x7fffffffLL || (!slots && S < B)) return SPECTRE_ERR_ARG;
    const size_t ev = elem(h->dtype), eg = elem(h->gate_dtype);
    if (!aligned(g, eg) || !aligned(v, ev) || !aligned(y, ev) || !aligned(state, 4) || !aligned(new_state, 4) ||
        !aligned(slots, 4))
        return SPECTRE_ERR_ALIGN;
    if (!current_device_is(h->device)) return SPECTRE_ERR_DEVICE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    using bf = __nv_bfloat16;
    auto go = [&](auto fn) { return status_of(fn(h, B, g, g_stride, v, v_stride, state, S, slots, y, y_stride, new_state, s)); };
    const bool e = h->gate == GATED_SCAN_EXP;
    if (h->dtype == SPECTRE_F32)
        return e ? go(launch_step<float, float, GATED_SCAN_EXP>) : go(launch_step<float, float, GATED_SCAN_SIGMOID>);
    if (h->gate_dtype == SPECTRE_F32)
        return e ? go(launch_step<bf, float, GATED_SCAN_EXP>) : go(launch_step<bf, float, GATED_SCAN_SIGMOID>);
    return e ? go(launch_step<bf, bf, GATED_SCAN_EXP>) : go(launch_step<bf, bf, GATED_SCAN_SIGMOID>);
}

int gated_scan_destroy(gated_scan_t h) {
    delete h;
    return SPECTRE_OK;
}

}  // extern "C"
