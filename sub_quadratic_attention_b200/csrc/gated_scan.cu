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
// and written once in a single launch.  A block takes a tile of 128 rows by 128 bytes of a
// row (64 bf16 channels): 16 lanes of 4 channels, 16 groups of 8 rows a thread.  Tensor
// copies bring the next tile into shared memory while this one is worked on.  A thread
// walks its rows once and keeps, for each, the product of its gates and the result from 0
// (Q in registers, P where the gates stood); the groups' pairs are joined in shared memory;
// the tile's pair is published to the blocks behind it and the state before the tile is
// found by looking back at the pairs published ahead of it; then a row is one fused
// multiply-add away from its state, and a tensor copy takes the tile out.  The backward
// pass recomputes the states of its tile from the state that the forward pass saved before
// it, keeps the gates as one number each, and goes back through the rows in the same way.
//
// Measured on one B200 (rows of 512 bf16 channels unless said, sigmoid gates a channel):
// forward 2^20 rows 0.83 ms (3.9 TB/s of 3.2 GB), 131,072 rows 115 us, 64 x 1,024 rows 52
// us; 4 x 12,288 rows of 2,048 fp32 channels, a decay a head, 144 us (5.6 TB/s); backward
// 131,072 rows 187 us, 4 x 12,288 x 2,048 fp32 224 us (5.4 TB/s).  The same tiles copied
// without work take 542 us for 2^20 rows (91% of the copy rate), with the work and no look
// back 560: what is left is the way of a pair through the second-level cache, about 2 us
// between publishing and being read with all the others' traffic, and the wait for the
// latest of the tiles ahead.
//
// Looking back.  A tile's pair is one 64-bit word in memory, written whole: readers need
// neither a flag nor a fence.  It is first (P, Q) and, when the state before the tile is
// known, (0, state behind it): a stretch that lets nothing through.  A reader takes the
// nearest pair with P = 0 and applies the pairs from there on in order, which is the
// arithmetic that the tiles between do themselves: the result is the same to the bit
// whichever of the two words it meets.  The blocks are launched together and take the tiles
// in order, so the tiles that a waiting block looks at are done or being worked on.  A wait
// that finds nothing for some seconds ends with NaN in the state and in all rows behind.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <new>
#include <type_traits>

#include "gated_scan.h"
#include "rows_io.cuh"
#include "tc_dft.cuh"

struct gated_scan_s {
    int H, D, C;
    int gate, per;
    int dtype, gate_dtype;
    int device, nsm;
    int test_wait;   // GATED_SCAN_OPT_TEST_WAIT_TIMEOUT
};

namespace gscan {

using namespace rows_io;

constexpr int CHUNK = GATED_SCAN_CHUNK;

template <typename T, int V> __device__ __forceinline__ Pack<T, V> load(const T *p) {
    return *reinterpret_cast<const Pack<T, V> *>(p);
}
template <typename T, int V> __device__ __forceinline__ void store(T *p, const float *f) {
    Pack<T, V> r;
#pragma unroll
    for (int j = 0; j < V; j++) r.v[j] = from_f<T>(f[j]);
    *reinterpret_cast<Pack<T, V> *>(p) = r;
}

struct Gate {
    float a, c;   // h = a h + c v
};

// The smaller of a = s(g) and 1 - a = s(-g) is e / (1 + e) with e = exp(-|g|), to its own
// relative precision; the larger is one minus it, off by at most half a step of one, so that
// a decay close to one stays as exact as its distance from one.  bf16 rows take the hardware's
// exp2 and reciprocal.  The exponent g log2(e) is rounded, and log2(e) itself, so the smaller factor is
// off by up to (1.25 |g| + 10) 2^-24 of itself: 15 units at |g| = 4, 35 at 20, 110 at 80, always far below
// the rows' own rounding of 2^-8; below 2^-126 (|g| > 87) it is zero.  A second word of the product would
// take the growth with |g| away for two more operations a gate; where |g| is large the factor is small and
// its product with it.  A log decay's exp is the accurate one for every type, since its error adds up over
// as many rows as the state lasts.
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float smaller_factor(float g) {
    const float e = expf(-fabsf(g));
    return e / (1.0f + e);
}
template <int FORM> __device__ __forceinline__ Gate gate_of(float g) {
    if (FORM == GATED_SCAN_EXP) return {expf(g), 1.0f};
    const float s = smaller_factor(g), o = 1.0f - s;
    return g >= 0.0f ? Gate{o, s} : Gate{s, o};
}

// Operations on neighbouring values of a thread, two an instruction.
__device__ __forceinline__ Vec<2> two(const float *f) {
    Vec<2> v;
    v.p[0] = pair_of(f[0], f[1]);
    return v;
}
__device__ __forceinline__ void split(float *f, const Vec<2> &v) { f[0] = v[0], f[1] = v[1]; }
template <int N> __device__ __forceinline__ void fma_all(float (&r)[N], const float (&a)[N], const float (&b)[N], const float (&c)[N]) {
#pragma unroll
    for (int j = 0; j + 1 < N; j += 2) split(r + j, fma(two(a + j), two(b + j), two(c + j)));
    if constexpr (N % 2) r[N - 1] = fmaf(a[N - 1], b[N - 1], c[N - 1]);
}
template <int N> __device__ __forceinline__ void mul_all(float (&r)[N], const float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int j = 0; j + 1 < N; j += 2) split(r + j, two(a + j) * two(b + j));
    if constexpr (N % 2) r[N - 1] = a[N - 1] * b[N - 1];
}
template <int N> __device__ __forceinline__ void add_all(float (&r)[N], const float (&a)[N], const float (&b)[N]) {
#pragma unroll
    for (int j = 0; j + 1 < N; j += 2) split(r + j, two(a + j) + two(b + j));
    if constexpr (N % 2) r[N - 1] = a[N - 1] + b[N - 1];
}
template <int V> __device__ __forceinline__ void fill(float (&r)[V], float f) {
#pragma unroll
    for (int j = 0; j < V; j++) r[j] = f;
}
template <int N, typename T, int V> __device__ __forceinline__ void floats(float (&f)[N], const Pack<T, V> &x) {
    static_assert(N == V, "");
#pragma unroll
    for (int j = 0; j < V; j++) f[j] = to_f(x.v[j]);
}

// N gates at once.  For bf16 rows c = 1 / (1 + exp(g)), and a = 1 - c, or exp(g) c where that is the
// smaller: each to the precision of exp (above) relative to itself.
template <int FORM, bool FAST, int N> __device__ __forceinline__ void gates(const float (&g)[N], float (&a)[N], float (&c)[N]) {
    if constexpr (FORM == GATED_SCAN_SIGMOID && FAST) {
        float k[N], e[N], one[N], d[N], small[N];
        fill(k, 1.44269504f);   // log2(e)
        fill(one, 1.0f);
        mul_all(k, g, k);
#pragma unroll
        for (int j = 0; j < N; j++) e[j] = exp2_approx(k[j]);
        add_all(d, e, one);
#pragma unroll
        for (int j = 0; j < N; j++) c[j] = reciprocal_approx(d[j]);
        mul_all(small, e, c);
        fill(d, -1.0f);
        fma_all(a, c, d, one);
#pragma unroll
        for (int j = 0; j < N; j++) a[j] = c[j] <= 0.5f ? a[j] : small[j];
    } else {
#pragma unroll
        for (int j = 0; j < N; j++) {
            const Gate q = gate_of<FORM>(g[j]);
            a[j] = q.a;
            c[j] = q.c;
        }
    }
}
// The same gates, each in one number: a log decay's a, or the smaller factor with g's sign.
template <int FORM, bool FAST, int N> __device__ __forceinline__ void pack_gates(const float (&g)[N], float (&k)[N]) {
    if constexpr (FORM == GATED_SCAN_EXP) {
#pragma unroll
        for (int j = 0; j < N; j++) k[j] = expf(g[j]);
    } else if constexpr (!FAST) {
#pragma unroll
        for (int j = 0; j < N; j++) k[j] = copysignf(smaller_factor(g[j]), g[j]);
    } else {
        float e[N], one[N], d[N];
        fill(d, -1.44269504f);
        fill(one, 1.0f);
#pragma unroll
        for (int j = 0; j < N; j++) e[j] = fabsf(g[j]);
        mul_all(e, e, d);
#pragma unroll
        for (int j = 0; j < N; j++) e[j] = exp2_approx(e[j]);
        add_all(d, e, one);
#pragma unroll
        for (int j = 0; j < N; j++) d[j] = reciprocal_approx(d[j]);
        mul_all(k, e, d);
#pragma unroll
        for (int j = 0; j < N; j++) k[j] = copysignf(k[j], g[j]);
    }
}
template <int FORM, int N> __device__ __forceinline__ void open_gates(const float (&k)[N], float (&a)[N], float (&c)[N]) {
    if constexpr (FORM == GATED_SCAN_EXP) {
#pragma unroll
        for (int j = 0; j < N; j++) a[j] = k[j], c[j] = 1.0f;
    } else {
        float s[N], one[N], o[N];
        fill(one, 1.0f);
#pragma unroll
        for (int j = 0; j < N; j++) s[j] = -fabsf(k[j]);
        add_all(o, s, one);
#pragma unroll
        for (int j = 0; j < N; j++) {
            a[j] = signbit(k[j]) ? -s[j] : o[j];
            c[j] = signbit(k[j]) ? o[j] : -s[j];
        }
    }
}
template <int V, int N> __device__ __forceinline__ void spread(float (&r)[V], const float (&x)[N]) {   // a head's for its channels
#pragma unroll
    for (int j = 0; j < V; j++) r[j] = x[N == 1 ? 0 : j];
}
template <int FORM> constexpr float HOLD = FORM == GATED_SCAN_EXP ? 1.0f : 0.0f;   // packed: a = 1

// a * h where a factor of zero takes h out, NaN and infinities included.  Products of gates are taken so
// too, each gate cutting off those before it: a NaN that meets a product that is zero already has come into
// the rows' own result as well, and the next zero takes out both.
__device__ __forceinline__ float mul0(float a, float h) { return a == 0.0f ? 0.0f : a * h; }
__device__ __forceinline__ float fma0(float a, float h, float b) { return a == 0.0f ? b : fmaf(a, h, b); }
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }

// A tile: CHUNK rows of WIDTH channels, 128 bytes of a row.  V channels a thread: 4 where rows and
// heads allow it, else 1 (then a row's part is 32 channels and a thread has 16 rows).
template <typename TV, int V> struct Tile {
    static constexpr int LANES = V == 4 ? 128 / (4 * (int)sizeof(TV)) : 32;
    static constexpr int WIDTH = LANES * V;
    static constexpr int ROWS = V == 4 ? 8 : 16;
    static constexpr int GROUPS = CHUNK / ROWS;
    static constexpr int THREADS = LANES * GROUPS;
};

// Workspace: one word for each tile and channel, all ones before a run, and as many words ahead of
// the first as a look back may ask for.
constexpr unsigned long long NOTHING = ~0ull;
constexpr unsigned MOST_POLLS = 1u << 22;   // of about a microsecond each

// Set where a bounded wait gave up; gated_scan_device_status reads and clears it.
__device__ unsigned wait_gave_up;

struct Args {
    gated_scan_args a;
    int H, D, C;
    unsigned long long head_of;   // ceil(2^40 / D): c * head_of >> 40 = c / D for c <= 2^20
    int strips;               // tiles beside one another: ceil(C / WIDTH)
    int nchunk;
    int serial;               // a block takes whole strips
    int nsm;
    unsigned copy_polls, look_polls;   // after which a wait gives up
    long long nseq;           // dense: B
    unsigned long long *words;   // null where no tile waits for another
    float *parts;             // per-head gradients of heads that span strips: [pieces][B L][H]
};

__device__ __forceinline__ int head_of(const Args &p, int c) { return (int)((unsigned)c * p.head_of >> 40); }

// Where batch entry b's state stands in h0 and its like, and the state before its chunk in `states`: more
// values than 32 bits count where millions of sequences have a thousand channels.
__device__ __forceinline__ long long end_at(const Args &p, int b) { return (long long)b * p.C; }
__device__ __forceinline__ long long state_at(const Args &p, int b, int chunk) { return ((long long)b * p.nchunk + chunk) * p.C; }

template <typename T> __device__ __forceinline__ T *row(const gated_scan_rows &r, long long b, long long t) {
    return static_cast<T *>(r.data) + b * r.batch_stride + t * r.row_stride;
}

// V neighbouring floats of shared memory, one access
template <int V> __device__ __forceinline__ void get(const float *p, float (&f)[V]) {
    const Pack<float, V> r = *reinterpret_cast<const Pack<float, V> *>(p);
#pragma unroll
    for (int j = 0; j < V; j++) f[j] = r.v[j];
}
template <int V> __device__ __forceinline__ void put(float *p, const float (&f)[V]) { store<float, V>(p, f); }

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

// The state in front of tile i (counted in the direction of the walk) of a strip, for each of its
// channels, found by the whole block: words[j * WIDTH + x] is tile j's word for channel x, and tile
// 0's has P = 0.  Thread (q, x) asks for the REACH words at distances q * REACH + 1 and on.  A
// channel is done when the nearest word with P = 0 is among them and nothing is missing before it;
// tiles ahead that are not done will be, so a block that finds no such word asks again instead of
// going further back.
constexpr int REACH = 8;
constexpr int AHEAD = 64;   // the most tiles that all threads of a block ask for
template <int WIDTH, int QS> struct alignas(16) LookBack {
    float state[WIDTH];
    unsigned char seen[QS][WIDTH];
};
__device__ __forceinline__ float gave_up() {
    atomicExch(&wait_gave_up, 1u);
    return __uint_as_float(0x7fc00000u);
}
// The same for one channel by one thread, where few tiles are in flight.
template <int WIDTH> __device__ __forceinline__ float look_near(const unsigned long long *words, int i, unsigned most) {
    const unsigned long long *from = words + (long long)(i - 1) * WIDTH;
    unsigned long long w[REACH];
    for (unsigned polls = 0; polls < most; polls++) {
#pragma unroll
        for (int j = 0; j < REACH; j++) w[j] = peek(from - j * WIDTH);
        int seen = REACH;
#pragma unroll
        for (int j = REACH - 1; j >= 0; j--) {
            const unsigned P = (unsigned)(w[j] >> 32);
            seen = P == (unsigned)(NOTHING >> 32) ? REACH : P == 0 ? j : seen;
        }
        if (seen == REACH) continue;
        float state = 0.0f;
#pragma unroll
        for (int j = REACH - 1; j >= 0; j--)
            if (j <= seen) state = fma0(word_P(w[j]), state, word_Q(w[j]));
        return state;
    }
    return gave_up();
}
template <int WIDTH, int QS>
__device__ __forceinline__ void look_back(LookBack<WIDTH, QS> &m, const unsigned long long *words, int i, bool mine, unsigned most) {
    const int x = threadIdx.x % WIDTH, q = threadIdx.x / WIDTH;
    // words ahead of tile 0 belong to others, or to nobody: tile 0's comes before them
    const unsigned long long *from = words + (long long)(i - 1 - q * REACH) * WIDTH + x;
    unsigned long long w[REACH];
    unsigned polls = 0;
    for (bool found = false; !found;) {
        // each thread by itself until its words are there, up to one with P = 0
        int seen;
        do {
#pragma unroll
            for (int j = 0; j < REACH; j++) w[j] = peek(from - j * WIDTH);
            seen = REACH;       // how many pairs come before a word with P = 0; one more: a word is missing
#pragma unroll
            for (int j = REACH - 1; j >= 0; j--) {
                const unsigned P = (unsigned)(w[j] >> 32);
                seen = P == (unsigned)(NOTHING >> 32) ? REACH + 1 : P == 0 ? j : seen;
            }
            if (!mine || i - 1 - q * REACH < 0) seen = 0;
        } while (seen > REACH && ++polls < most);
        m.seen[q][x] = (unsigned char)seen;
        __syncthreads();
        int nearest = 0, at = REACH;   // the word with P = 0: thread nearest's number at
        while (nearest < QS && (at = m.seen[nearest][x]) == REACH) nearest++;
        found = !__syncthreads_or(at >= REACH);
        if (!found) {
            if (__syncthreads_or(++polls >= most)) {
                if (q == 0) m.state[x] = gave_up();
                __syncthreads();
                return;
            }
            continue;
        }
        // from the farthest word on, in order
        for (int k = __syncthreads_or(nearest > 0) ? QS - 1 : 0; k >= 0; k--) {
            if (q == k && k <= nearest) {
                float state = k == nearest ? 0.0f : m.state[x];
#pragma unroll
                for (int j = REACH - 1; j >= 0; j--)
                    if (k < nearest || j <= at) state = fma0(word_P(w[j]), state, word_Q(w[j]));
                m.state[x] = mine ? state : 0.0f;
            }
            __syncthreads();
        }
    }
}

// Where the block's tile lies.  Tiles are numbered chunk by chunk over all batch entries and
// strips, in the direction of the walk, so that every strip advances at the same time; a block
// takes every gridDim.x-th, and goes from one to the next without a division.  Where there are
// strips enough, or few chunks, a block takes a strip's chunks one after another instead and
// carries the state itself.
struct Place {
    int i, b, strip;   // i: the chunk in walking order
    __device__ __forceinline__ Place() {}
    __device__ __forceinline__ Place(const Args &p, unsigned ticket) {
        const unsigned strips = p.strips, per = (unsigned)p.a.B * strips, rest = ticket % per;
        i = (int)(ticket / per);
        b = (int)(rest / strips);
        strip = (int)(rest % strips);
    }
    __device__ __forceinline__ void advance(const Args &p, const Place &by) {
        if (p.serial) {   // the strip's next chunk, or another strip
            if (++i < p.nchunk) return;
            i = by.i ? p.nchunk : 0;
        } else {
            i += by.i;
        }
        strip += by.strip;
        b += by.b;
        if (strip >= p.strips) strip -= p.strips, b++;
        if (b >= (int)p.a.B) b -= (int)p.a.B, i = p.serial ? p.nchunk : i + 1;
    }
    __device__ __forceinline__ long long first_word(const Args &p) const { return ((long long)b * p.strips + strip) * p.nchunk; }
};

constexpr int MANY_SEQUENCES = 1024;   // four to a thread

// Packed rows: the sequence that starts at, and that ends with, each row of the tile (or -1),
// and the rows that lie in sequences at all.
struct Marks {
    int first[CHUNK], last[CHUNK];
};
__device__ __forceinline__ void mark_sequences(const Args &p, Marks &m, long long t0, long long &lo, long long &hi) {
    const int *cu = p.a.cu_seqlens;
    __syncthreads();   // the last tile's marks have been read
    for (int i = threadIdx.x; i < CHUNK; i += blockDim.x) m.first[i] = m.last[i] = -1;
    __syncthreads();
    // of many sequences the tile's are found first: every stride-th tells which have ended before it
    const bool many = p.nseq > MANY_SEQUENCES;
    long long n = threadIdx.x;
    if (many) {
        const long long stride = (p.nseq + blockDim.x - 1) / blockDim.x, at = threadIdx.x * stride;
        const int ended = __syncthreads_count(at < p.nseq && cu[at + 1] <= t0);
        n += ended ? (ended - 1) * stride : 0;
    }
    for (; n < p.nseq; n += blockDim.x) {
        const long long s = cu[n], e = cu[n + 1];
        if (many && s >= t0 + CHUNK) break;
        if (s >= e) continue;
        if (s >= t0 && s < t0 + CHUNK) m.first[s - t0] = (int)n;
        if (e > t0 && e <= t0 + CHUNK) m.last[e - 1 - t0] = (int)n;
    }
    __syncthreads();
    lo = cu[0] > lo ? cu[0] : lo;
    hi = cu[p.nseq] < hi ? cu[p.nseq] : hi;
}

// A sequence a warp: the state goes through to the ends of those without rows (cu null: of all).  The scans' blocks do
// this when their tiles are done, each its share, so that nobody waits for it: walked by the blocks of the first tiles
// alone it took them 0.2 us for every four sequences, with the others waiting for their next tiles: 131,072 rows of 512
// bf16 channels in 2,000 sequences took 242 us forward, and take 182 so; 12 million sequences 0.6 s, a seventh of what a
// wait may last.
__device__ __forceinline__ void pass_states(const int *cu, long long nseq, int C, const float *from, float *to) {
    const int warps = blockDim.x / 32;
    for (long long n = blockIdx.x * (long long)warps + threadIdx.x / 32; n < nseq; n += gridDim.x * (long long)warps) {
        if (cu && cu[n] < cu[n + 1]) continue;
        for (int c = threadIdx.x % 32; c < C; c += 32) to[n * C + c] = from ? from[n * C + c] : 0.0f;
    }
}
constexpr int PASS_THREADS = 256, PASS_BLOCKS = 1 << 20;
__global__ void __launch_bounds__(PASS_THREADS) pass_all(long long nseq, int C, const float *from, float *to) { pass_states(nullptr, nseq, C, from, to); }

// The tensors' maps for the tensor copies: boxes of CHUNK rows by WIDTH channels.
struct Maps {
    CUtensorMap g, v, y, dy, dg, dv;
};

// A tile of each input tensor in shared memory, two tiles in turn: one tensor copy brings the next
// tile's while this one is worked on.  Where a thread has read its gates (and values) the products
// of its gates are kept, and at the end the rows of y, which one tensor copy takes out.  Rows that
// cannot be copied so (V = 1) go through registers.
template <typename TV, typename TG, bool HEAD, int V> struct Stage {
    using S = Tile<TV, V>;
    static constexpr bool ON = V == 4;
    static constexpr int G_ROW = S::WIDTH * (int)sizeof(TG), V_ROW = S::WIDTH * (int)sizeof(TV);
    static constexpr int G_BYTES = HEAD ? 0 : CHUNK * G_ROW, V_BYTES = CHUNK * V_ROW;
    static constexpr int INPUT_BYTES = ON ? G_BYTES + V_BYTES : 0;
    __device__ static int at_g(int r) { return (threadIdx.x / S::LANES * S::ROWS + r) * G_ROW + threadIdx.x % S::LANES * 4 * (int)sizeof(TG); }
    __device__ static int at_v(int r) { return (threadIdx.x / S::LANES * S::ROWS + r) * V_ROW + threadIdx.x % S::LANES * 4 * (int)sizeof(TV); }
    // four floats where a row's gates were (two-byte gates leave half of the room, the values the rest)
    __device__ static void keep(char *g, char *v, int r, const float *f) {
        if constexpr (sizeof(TG) == 4) {
            *reinterpret_cast<float4 *>(g + at_g(r)) = make_float4(f[0], f[1], f[2], f[3]);
        } else {
            *reinterpret_cast<float2 *>(g + at_g(r)) = make_float2(f[0], f[1]);
            *reinterpret_cast<float2 *>(v + at_v(r)) = make_float2(f[2], f[3]);
        }
    }
    __device__ static void kept(const char *g, const char *v, int r, float *f) {
        if constexpr (sizeof(TG) == 4) {
            const float4 k = *reinterpret_cast<const float4 *>(g + at_g(r));
            f[0] = k.x, f[1] = k.y, f[2] = k.z, f[3] = k.w;
        } else {
            const float2 a = *reinterpret_cast<const float2 *>(g + at_g(r)), b = *reinterpret_cast<const float2 *>(v + at_v(r));
            f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
        }
    }
};

using spectre::tc::fence_proxy_async;
using spectre::tc::mbar_arrive_expect_tx;
using spectre::tc::mbar_init;
using spectre::tc::mbar_wait;
using spectre::tc::smem_u32;

constexpr unsigned COPY_POLLS = 4000;   // of up to a millisecond's suspension each

__device__ __forceinline__ void tensor_in(char *to, const CUtensorMap *map, int c, int t, int b, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(to)),
                 "l"(map), "r"(c), "r"(t), "r"(b), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tensor_out(const CUtensorMap *map, int c, int t, int b, const char *from) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(c), "r"(t), "r"(b),
                 "r"(smem_u32(from))
                 : "memory");
}
__device__ __forceinline__ void out_close() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void out_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void out_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A thread's rows of a tile: where they are, and which of them exist.
template <typename TV, typename TG, bool HEAD, int V> struct Rows {
    using S = Tile<TV, V>;
    Place at;
    int chunk, c0, c, gc;
    bool mine;
    long long t0;
    int count;   // rows before the tensor's end, 0 to ROWS
    __device__ Rows(const Args &p, const Place &place, bool backward) : at(place) {
        chunk = backward ? p.nchunk - 1 - at.i : at.i;
        c0 = at.strip * S::WIDTH;
        c = c0 + threadIdx.x % S::LANES * V;
        mine = c < p.C;
        gc = HEAD ? head_of(p, c) : c;
        t0 = (long long)chunk * CHUNK + threadIdx.x / S::LANES * S::ROWS;
        const long long left = p.a.L - t0;
        count = mine ? (int)(left < 0 ? 0 : left < S::ROWS ? left : S::ROWS) : 0;
    }
    template <typename T> __device__ T *first(const gated_scan_rows &r, int column) const { return row<T>(r, at.b, t0) + column; }
};

// The strips that the channels of head h lie in.
__host__ __device__ __forceinline__ int first_strip(int h, int D, int width) { return (int)((long long)h * D / width); }
__host__ __device__ __forceinline__ int last_strip(int h, int D, int width) { return (int)(((long long)h * D + D - 1) / width); }

// A head's gradient at a row, or the part of it that a strip has.
template <typename TG> __device__ __forceinline__ void put_gate(const Args &p, int b, long long t, int head, int piece, float sum) {
    if (!p.parts)
        row<TG>(p.a.dg, b, t)[head] = from_f<TG>(sum);
    else
        p.parts[((piece * p.a.B + b) * p.a.L + t) * p.H + head] = sum;
}

// Where a tile's copies do not come in time, the block asks for no more of them and waits for those once again, so
// that none lands in shared memory that is another block's by then.  Here its threads leave NaN in what the tile
// and the block's others behind it would have given.
template <typename TV, typename TG, bool HEAD, int V, bool BACKWARD> __device__ __noinline__ void leave_nan(const Args &p, Place at, Marks &marks) {
    using S = Tile<TV, V>;
    const bool packed = p.a.cu_seqlens != nullptr;
    const float nan = gave_up();
    for (const Place by(p, gridDim.x); at.i < p.nchunk; at.advance(p, by)) {
        const Rows<TV, TG, HEAD, V> rows(p, at, BACKWARD);
        long long lo = 0, hi = p.a.L;
        if (packed) mark_sequences(p, marks, (long long)rows.chunk * CHUNK, lo, hi);
#pragma unroll 1
        for (int r = 0; r < rows.count; r++) {
            const long long t = rows.t0 + r;
            const bool in = t >= lo && t < hi;
            if (!in && !p.a.zero_outside) continue;
            float f[V];
            fill(f, in ? nan : 0.0f);
            store<TV, V>(row<TV>(BACKWARD ? p.a.dv : p.a.y, at.b, t) + rows.c, f);
            if constexpr (BACKWARD && HEAD) put_gate<TG>(p, at.b, t, rows.gc, at.strip - first_strip(rows.gc, p.D, S::WIDTH), f[0]);
            else if constexpr (BACKWARD) store<TG, V>(row<TG>(p.a.dg, at.b, t) + rows.c, f);
        }
        const int x = threadIdx.x, cx = rows.c0 + x;
        float *const ends = BACKWARD ? p.a.dh0 : p.a.hT;
        if (x < S::WIDTH && cx < p.C) {
            if (!p.serial && at.i + 1 < p.nchunk) publish(p.words + (at.first_word(p) + at.i) * S::WIDTH + x, 0.0f, nan);
            if (!BACKWARD && p.a.states) p.a.states[state_at(p, at.b, at.i) + cx] = nan;
            if (ends && !packed && at.i + 1 == p.nchunk) ends[end_at(p, at.b) + cx] = nan;
            for (int r = 0; ends && packed && r < CHUNK; r++) {
                const long long n = BACKWARD ? marks.first[r] : marks.last[r];
                if (n >= 0) ends[n * p.C + cx] = nan;
            }
        }
    }
}

// Blocks an SM: 80 registers a thread leave room for three of 256 threads.  With two and with three, bf16 in
// us: 2^20 rows of 512 channels 930 and 828, 64 x 1,024 rows 58 and 52, 4 x 12,288 rows of 2,048, a decay a
// head, 132 and 112.
template <typename TV, bool HEAD> constexpr int FORWARD_BLOCKS = HEAD && sizeof(TV) == 4 ? 5 : 3;
// Channels one by one, in either direction.  Three blocks spill 100 to 370 bytes a thread going back and are the
// fastest all the same, at one round of tiles and at many; with two, three and four, forward and backward in us, 231
// channels: 5,003 packed rows fp32 a decay a head 20.6 + 45.2, 16.5 + 41.2, 16.5 + 42.5; 20,000 rows of the same
// 31.4 + 93.9, 26.4 + 79.8, 29.1 + 103.6; 65,536 rows, a gate a channel, fp32 90.8 + 249.8, 70.5 + 206.8,
// 74.4 + 276.1, bf16 77.9 + 236.4, 57.1 + 194.2, 60.9 + 231.2.
constexpr int SINGLE_BLOCKS = 3;

template <typename TV, typename TG, int FORM, bool HEAD, int V>
__global__ void __launch_bounds__(Tile<TV, V>::THREADS, V == 1 ? SINGLE_BLOCKS : FORWARD_BLOCKS<TV, HEAD>)
    scan_forward(const __grid_constant__ Args p, const __grid_constant__ Maps maps) {
    using S = Tile<TV, V>;
    using M = Stage<TV, TG, HEAD, V>;
    using R = Rows<TV, TG, HEAD, V>;
    constexpr int GV = HEAD ? 1 : V;
    constexpr bool FAST = sizeof(TV) == 2;
    constexpr bool KEPT = M::ON && !HEAD;   // the gates' products are where the gates were, not in registers
    extern __shared__ __align__(128) char buffers[];
    __shared__ float head_P[HEAD && M::ON ? S::ROWS : 1][S::THREADS];   // a head's: one a row and thread
    __shared__ __align__(16) float sP[S::GROUPS][S::WIDTH], sQ[S::GROUPS][S::WIDTH];
    __shared__ LookBack<S::WIDTH, S::THREADS / S::WIDTH> ahead;
    __shared__ Marks marks;
    __shared__ __align__(8) unsigned long long bars[2];
    const bool packed = p.a.cu_seqlens != nullptr;
    const int lane = threadIdx.x % S::LANES, group = threadIdx.x / S::LANES;
    Place next(p, blockIdx.x);
    const Place by(p, gridDim.x);
    // more tiles of a strip in flight than one thread's REACH: the whole block looks back.  Where
    // few are, one thread a channel is enough and asks for less: 64 x 1,024 bf16 rows of 512 channels
    // 52 against 54 us, back 89 against 94, 4 x 12,288 of 2,048 128 against 136, back 236 against 265
    const bool far = !p.serial && (unsigned)(p.a.B * p.strips) * REACH < gridDim.x;
    float carry = 0.0f;   // serial: a channel's state (or gradient) behind the last tile

    const bool agent = threadIdx.x == S::THREADS - 32;   // issues all copies
    bool lost = false;   // a tile's copies
    auto fetch = [&](const Place &at, int turn) {
        if (!M::ON || !agent || at.i >= p.nchunk) return;
        char *to = buffers + turn * M::INPUT_BYTES;
        const uint32_t bar = smem_u32(&bars[turn]);
        mbar_arrive_expect_tx(bar, M::INPUT_BYTES);
        if (!HEAD) tensor_in(to, &maps.g, at.strip * S::WIDTH, at.i * CHUNK, (int)at.b, bar);
        tensor_in(to + M::G_BYTES, &maps.v, at.strip * S::WIDTH, at.i * CHUNK, (int)at.b, bar);
    };
    // one gate a row is too little for a copy: it waits in a register
    TG g_now[HEAD ? S::ROWS : 1];
    auto fetch_gates = [&](const Place &at) {
        if (!HEAD || !M::ON || at.i >= p.nchunk) return;
        const R rows(p, at, false);
        const TG *g = rows.template first<TG>(p.a.g, rows.gc);
#pragma unroll
        for (int r = 0; r < (HEAD ? S::ROWS : 1); r++) g_now[r] = r < rows.count ? g[r * p.a.g.row_stride] : from_f<TG>(0.0f);
    };
    if (M::ON) {
        if (threadIdx.x == 0) {
            mbar_init(smem_u32(&bars[0]), 1);
            mbar_init(smem_u32(&bars[1]), 1);
        }
        __syncthreads();
        fetch(next, 0);
        fetch_gates(next);
    }
    int turn = 0;
    uint32_t phase = 0;
    while (next.i < p.nchunk) {
        const Place now = next;
        next.advance(p, by);
        char *const pg = buffers + turn * M::INPUT_BYTES, *const pv = pg + M::G_BYTES;
        const R rows(p, now, false);
        const Place &at = rows.at;
        const int c0 = rows.c0, c = rows.c;
        long long lo = 0, hi = p.a.L;
        bool starts = false, ends = at.i == p.nchunk - 1;   // of sequences in this tile
        if (packed) {
            mark_sequences(p, marks, (long long)at.i * CHUNK, lo, hi);
            bool f = false, l = false;
            for (int i = threadIdx.x; i < CHUNK; i += S::THREADS) f |= marks.first[i] >= 0, l |= marks.last[i] >= 0;
            starts = __syncthreads_or(f);
            ends = __syncthreads_or(l);
        }
        // every row that the tensors have is in a sequence, none starts one: rows and channels that
        // do not exist come as zeros from the copies and go nowhere
        const long long tile0 = (long long)at.i * CHUNK;
        const bool whole = !packed || (tile0 >= lo && tile0 + CHUNK <= hi);
        const bool plain = whole && !starts && (M::ON || (tile0 + CHUNK <= p.a.L && rows.mine));

        // row r's state is P[r] h + Q[r], h the state ahead of the thread's rows
        [[maybe_unused]] float P[M::ON ? 1 : S::ROWS][GV];
        float Q[S::ROWS][V], lastP[GV];
        auto walk = [&](auto careful, bool again) {
            constexpr bool CARE = decltype(careful)::value;   // rows that are missing, starts, factors of zero
            float q[V];
#pragma unroll
            for (int j = 0; j < GV; j++) lastP[j] = 1.0f;
#pragma unroll
            for (int j = 0; j < V; j++) q[j] = 0.0f;
            const TG *gp = rows.template first<TG>(p.a.g, rows.gc);
            const TV *vp = rows.template first<TV>(p.a.v, c);
            // all rows first: what is kept goes where they stand.  A careful walk that is a second
            // one reads them from memory again.
            Pack<TG, GV> gs[S::ROWS];
            Pack<TV, V> vs[S::ROWS];
            if constexpr (!CARE) {
#pragma unroll
                for (int r = 0; r < S::ROWS; r++) {
                    if constexpr (!M::ON) gs[r] = load<TG, GV>(gp + r * p.a.g.row_stride);
                    else if constexpr (HEAD) gs[r].v[0] = g_now[r];
                    else gs[r] = load<TG, GV>(reinterpret_cast<const TG *>(pg + M::at_g(r)));
                    if constexpr (!M::ON) vs[r] = load<TV, V>(vp + r * p.a.v.row_stride);
                    else vs[r] = load<TV, V>(reinterpret_cast<const TV *>(pv + M::at_v(r)));
                }
                asm volatile("" ::: "memory");
            }
#pragma unroll
            for (int r = 0; r < S::ROWS; r++) {
                if (CARE && starts) {
                    const int n = rows.mine ? marks.first[group * S::ROWS + r] : -1;
                    if (n >= 0) {
#pragma unroll
                        for (int j = 0; j < GV; j++) lastP[j] = 0.0f;
#pragma unroll
                        for (int j = 0; j < V; j++) q[j] = p.a.h0 ? p.a.h0[(long long)n * p.C + c + j] : 0.0f;
                    }
                }
                if (!CARE || (r < rows.count && rows.t0 + r >= lo && rows.t0 + r < hi)) {
                    if constexpr (CARE) {
                        const bool memory = again || !M::ON;
                        if constexpr (HEAD && M::ON) gs[r].v[0] = g_now[r];
                        else gs[r] = load<TG, GV>(memory ? gp + r * p.a.g.row_stride : reinterpret_cast<const TG *>(pg + M::at_g(r)));
                        vs[r] = load<TV, V>(memory ? vp + r * p.a.v.row_stride : reinterpret_cast<const TV *>(pv + M::at_v(r)));
                        asm volatile("" ::: "memory");
                    }
                    const Pack<TG, GV> &g = gs[r];
                    const Pack<TV, V> &v = vs[r];
                    float gf[GV], vf[V], ka[GV], kc[GV];
                    floats(gf, g);
                    floats(vf, v);
                    gates<FORM, FAST>(gf, ka, kc);
                    if constexpr (CARE) {
#pragma unroll
                        for (int j = 0; j < GV; j++) lastP[j] = mul0(ka[j], lastP[j]);
                    } else {
                        mul_all(lastP, lastP, ka);
                    }
                    float a[V], c[V];
                    spread(a, ka);
                    spread(c, kc);
                    if constexpr (CARE) {
#pragma unroll
                        for (int j = 0; j < V; j++) q[j] = fma0(a[j], q[j], FORM == GATED_SCAN_EXP ? vf[j] : mul0(c[j], vf[j]));
                    } else {
                        if (FORM == GATED_SCAN_SIGMOID) mul_all(vf, c, vf);
                        fma_all(q, a, q, vf);
                    }
                }
                if constexpr (KEPT)
                    M::keep(pg, pv, r, lastP);
                else if constexpr (M::ON)
                    head_P[r][threadIdx.x] = lastP[0];
                else {
#pragma unroll
                    for (int j = 0; j < GV; j++) P[r][j] = lastP[j];
                }
#pragma unroll
                for (int j = 0; j < V; j++) Q[r][j] = q[j];
            }
        };
        bool arrived = true;
        if (M::ON) arrived = mbar_wait(smem_u32(&bars[turn]), phase, p.copy_polls);
        // Without care a NaN or infinity anywhere leaves the last row without a finite value, or the
        // gates' product (an infinite decay of nothing is nothing in Q): then the rows are walked again.
        bool fine = plain;
        if (fine) {
            walk(std::false_type{}, false);
#pragma unroll
            for (int j = 0; j < V; j++) fine &= finite(Q[S::ROWS - 1][j]);
            if (FORM == GATED_SCAN_EXP)
#pragma unroll
                for (int j = 0; j < GV; j++) fine &= finite(lastP[j]);
        }
        if (!fine) walk(std::true_type{}, plain);
        {
            float lp[V], lq[V];
#pragma unroll
            for (int j = 0; j < V; j++) {
                lp[j] = lastP[HEAD ? 0 : j];
                lq[j] = Q[S::ROWS - 1][j];
            }
            put(&sP[group][lane * V], lp);
            put(&sQ[group][lane * V], lq);
        }
        if (!M::ON) {
            __syncthreads();
        } else if (!__syncthreads_and(arrived)) {
            lost = true;
            next = now;
            break;
        }

        if (M::ON && agent) out_read();   // the other buffer's rows of y have left it
        fetch(next, turn ^ 1);
        fetch_gates(next);
        const int x = threadIdx.x, cx = c0 + threadIdx.x % S::WIDTH;
        unsigned long long *const words = p.words + at.first_word(p) * S::WIDTH;
        const bool more = !p.serial && at.i + 1 < p.nchunk;
        float allP = 1.0f, allQ = 0.0f;
        if (x < S::WIDTH) {
            // each group's pair becomes that of all groups ahead of it
#pragma unroll
            for (int i = 0; i < S::GROUPS; i++) {
                const float gP = sP[i][x], gQ = sQ[i][x];
                sP[i][x] = allP;
                sQ[i][x] = allQ;
                allQ = fma0(gP, allQ, gQ);
                allP = mul0(gP, allP);
            }
            if (at.i > 0 && more && cx < p.C) publish(words + (long long)at.i * S::WIDTH + x, allP, allQ);
        }
        if (at.i > 0 && far) {
            look_back(ahead, words, at.i, cx < p.C, p.look_polls);
        } else if (at.i > 0) {
            if (x < S::WIDTH) ahead.state[x] = p.serial ? carry : cx < p.C ? look_near<S::WIDTH>(words + x, at.i, p.look_polls) : 0.0f;
            __syncthreads();
        } else {
            if (x < S::WIDTH) ahead.state[x] = !packed && p.a.h0 && cx < p.C ? p.a.h0[end_at(p, at.b) + cx] : 0.0f;
            __syncthreads();
        }
        if (x < S::WIDTH && cx < p.C) {
            const float state = ahead.state[x];
            carry = fma0(allP, state, allQ);
            if (more) publish(words + (long long)at.i * S::WIDTH + x, 0.0f, carry);
            if (p.a.states) p.a.states[state_at(p, at.b, at.i) + cx] = state;
        }

        float h0[V];
        fine = plain && !(packed && ends);
        {
            float gp[V], gq[V], state[V];
            get(&sP[group][lane * V], gp);
            get(&sQ[group][lane * V], gq);
            get(&ahead.state[lane * V], state);
#pragma unroll
            for (int j = 0; j < V; j++) {
                h0[j] = fma0(gp[j], state[j], gq[j]);
                fine &= finite(h0[j]);
            }
        }
        auto products = [&](int r, float (&pr)[V]) {
            if constexpr (KEPT) M::kept(pg, pv, r, pr);
            else if constexpr (M::ON) fill(pr, head_P[r][threadIdx.x]);
            else spread(pr, P[r]);
        };
        if (!packed && ends && p.a.hT && rows.mine) {
            // the state behind a dense sequence's last row, by the thread that has the row
#pragma unroll
            for (int r = 0; r < S::ROWS; r++)
                if (rows.t0 + r == p.a.L - 1) {
                    float pr[V];
                    products(r, pr);
#pragma unroll
                    for (int j = 0; j < V; j++) p.a.hT[end_at(p, at.b) + c + j] = fma0(pr[j], h0[j], Q[r][j]);
                }
        }
        auto finish = [&](auto careful) {
            constexpr bool CARE = decltype(careful)::value;
            TV *y = rows.template first<TV>(p.a.y, c);
#pragma unroll
            for (int r = 0; r < S::ROWS; r++) {
                if (CARE && r >= rows.count) break;
                float h[V], pr[V];
                products(r, pr);
                if constexpr (CARE) {
#pragma unroll
                    for (int j = 0; j < V; j++) h[j] = fma0(pr[j], h0[j], Q[r][j]);
                } else {
                    fma_all(h, pr, h0, Q[r]);
                }
                const bool in = !CARE || (rows.t0 + r >= lo && rows.t0 + r < hi);
                if (CARE && packed && ends && in && p.a.hT) {
                    const int n = marks.last[group * S::ROWS + r];
                    if (n >= 0)
#pragma unroll
                        for (int j = 0; j < V; j++) p.a.hT[(long long)n * p.C + c + j] = h[j];
                }
                if (M::ON && (!CARE || whole)) {
                    store<TV, V>(reinterpret_cast<TV *>(pv + M::at_v(r)), h);
                    continue;
                }
                if (!in) {
                    if (!p.a.zero_outside) continue;
#pragma unroll
                    for (int j = 0; j < V; j++) h[j] = 0.0f;
                }
                store<TV, V>(y + r * p.a.y.row_stride, h);
            }
        };
        if (fine)
            finish(std::false_type{});
        else
            finish(std::true_type{});
        if (M::ON) {
            fence_proxy_async();
            __syncthreads();
            if (agent && whole) {
                tensor_out(&maps.y, c0, at.i * CHUNK, (int)at.b, pv);
                out_close();
            }
            phase ^= turn;
            turn ^= 1;
        }
    }
    if (M::ON && agent) out_done();
    if (M::ON && lost) {
        if (agent) mbar_wait(smem_u32(&bars[turn]), phase, COPY_POLLS);
        leave_nan<TV, TG, HEAD, V, false>(p, next, marks);
    }
    if (packed && p.a.hT) pass_states(p.a.cu_seqlens, p.nseq, p.C, p.a.h0, p.a.hT);
}

// A thread's rows of a tile without borders, one after another from memory: the state ahead of each is found
// anew, and a factor of zero takes its operand out.  For rows whose states or gradients overflow between a
// thread's first and last, which a gate of zero among them must not turn into NaN: so rare that it may be slow,
// and out of the kernel's way so that it costs few registers there.  Takes the state ahead of the rows and the
// gradient behind them, returns the gradient ahead.
template <int V> struct Ends {
    float h[V], e[V];
};
template <typename TV, typename TG, int FORM, bool HEAD, int V>
__device__ __noinline__ Ends<V> one_by_one(const Args &p, int b, int strip, int chunk, Ends<V> ends, char *pg, char *pv) {
    using S = Tile<TV, V>;
    using M = Stage<TV, TG, HEAD, V>;
    constexpr int GV = HEAD ? 1 : V;
    const int lane = threadIdx.x % S::LANES, c = strip * S::WIDTH + lane * V, gc = HEAD ? head_of(p, c) : c;
    const long long t0 = (long long)chunk * CHUNK + threadIdx.x / S::LANES * S::ROWS;
    const long long count = c < p.C ? p.a.L - t0 : 0;
    const TG *gp = row<TG>(p.a.g, b, t0) + gc;
    const TV *vp = row<TV>(p.a.v, b, t0) + c, *dp = row<TV>(p.a.dy, b, t0) + c;
    auto gate_at = [&](int r, float (&x)[V], float (&y)[V]) {
        float gf[GV], k[GV], ka[GV], kc[GV];
        floats(gf, load<TG, GV>(gp + r * p.a.g.row_stride));
        pack_gates<FORM, sizeof(TV) == 2>(gf, k);
        open_gates<FORM>(k, ka, kc);
        spread(x, ka);
        spread(y, kc);
    };
#pragma unroll 1
    for (int r = S::ROWS - 1; r >= 0; r--) {
        float sum = 0.0f;
        if (r < count) {
            float v[V], x[V], y[V], d[V], dv[V], dg[V], h[V];
#pragma unroll
            for (int j = 0; j < V; j++) h[j] = ends.h[j];
#pragma unroll 1
            for (int q = 0;; q++) {
                gate_at(q, x, y);
                floats(v, load<TV, V>(vp + q * p.a.v.row_stride));
                if (q == r) break;
#pragma unroll
                for (int j = 0; j < V; j++) h[j] = fma0(x[j], h[j], FORM == GATED_SCAN_EXP ? v[j] : mul0(y[j], v[j]));
            }
            floats(d, load<TV, V>(dp + r * p.a.dy.row_stride));
#pragma unroll
            for (int j = 0; j < V; j++) {
                const float w = FORM == GATED_SCAN_EXP ? x[j] : x[j] * y[j];
                d[j] += ends.e[j];
                dg[j] = w == 0.0f ? 0.0f : w * (FORM == GATED_SCAN_EXP ? h[j] : h[j] - v[j]) * d[j];
                dv[j] = FORM == GATED_SCAN_EXP ? d[j] : mul0(y[j], d[j]);
                ends.e[j] = mul0(x[j], d[j]);
                sum += dg[j];
            }
            if constexpr (M::ON) store<TV, V>(reinterpret_cast<TV *>(pv + M::at_v(r)), dv);
            else store<TV, V>(row<TV>(p.a.dv, b, t0 + r) + c, dv);
            if constexpr (!HEAD && M::ON) store<TG, V>(reinterpret_cast<TG *>(pg + M::at_g(r)), dg);
            else if constexpr (!HEAD) store<TG, V>(row<TG>(p.a.dg, b, t0 + r) + c, dg);
        }
        if constexpr (HEAD) {
#pragma unroll
            for (int o = 0; (1 << o) < S::LANES; o++) {
                const float other = __shfl_down_sync(0xffffffffu, sum, 1 << o, S::LANES);
                const int mate = c + (V << o);
                sum += lane + (1 << o) < S::LANES && mate < p.C && head_of(p, mate) == gc ? other : 0.0f;
            }
            if (r < count && (lane == 0 || head_of(p, c - V) != gc)) put_gate<TG>(p, b, t0 + r, gc, strip - first_strip(gc, p.D, S::WIDTH), sum);
        }
    }
    return ends;
}

constexpr int BACKWARD_BLOCKS = 2;   // an SM: two tiles of three tensors each fill its shared memory

template <typename TV, typename TG, int FORM, bool HEAD, int V>
__global__ void __launch_bounds__(Tile<TV, V>::THREADS, V == 1 ? SINGLE_BLOCKS : BACKWARD_BLOCKS)
    scan_backward(const __grid_constant__ Args p, const __grid_constant__ Maps maps) {
    using S = Tile<TV, V>;
    using M = Stage<TV, TG, HEAD, V>;
    using R = Rows<TV, TG, HEAD, V>;
    constexpr int GV = HEAD ? 1 : V;
    constexpr bool FAST = sizeof(TV) == 2;
    constexpr int TILE_BYTES = M::ON ? M::INPUT_BYTES + M::V_BYTES : 0;   // g, v, dy
    constexpr bool IN_PLACE = M::ON && !HEAD;   // the groups' P stand where their gates were
    extern __shared__ __align__(128) char buffers[];
    // (P, Q) of the states going forward, (R, E) of the gradients going back
    __shared__ __align__(16) float sP[IN_PLACE ? 1 : S::GROUPS][S::WIDTH], sQ[S::GROUPS][S::WIDTH];
    __shared__ __align__(16) float sR[S::GROUPS][S::WIDTH], sE[S::GROUPS][S::WIDTH];
    __shared__ LookBack<S::WIDTH, S::THREADS / S::WIDTH> ahead;
    __shared__ Marks marks;
    __shared__ __align__(8) unsigned long long bars[2];
    const bool packed = p.a.cu_seqlens != nullptr;
    const int lane = threadIdx.x % S::LANES, group = threadIdx.x / S::LANES;
    Place next(p, blockIdx.x);
    const Place by(p, gridDim.x);
    const bool far = !p.serial && (unsigned)(p.a.B * p.strips) * REACH < gridDim.x;
    float carry = 0.0f;   // serial: a channel's state (or gradient) behind the last tile

    const bool agent = threadIdx.x == S::THREADS - 32;   // issues all copies
    bool lost = false;   // a tile's copies
    auto fetch = [&](const Place &at, int turn) {
        if (!M::ON || !agent || at.i >= p.nchunk) return;
        char *to = buffers + turn * TILE_BYTES;
        const uint32_t bar = smem_u32(&bars[turn]);
        const int c0 = at.strip * S::WIDTH, t0 = (p.nchunk - 1 - at.i) * CHUNK;
        mbar_arrive_expect_tx(bar, TILE_BYTES);
        if (!HEAD) tensor_in(to, &maps.g, c0, t0, (int)at.b, bar);
        tensor_in(to + M::G_BYTES, &maps.v, c0, t0, (int)at.b, bar);
        tensor_in(to + M::INPUT_BYTES, &maps.dy, c0, t0, (int)at.b, bar);
    };
    TG g_now[HEAD ? S::ROWS : 1];
    auto fetch_gates = [&](const Place &at) {
        if (!HEAD || !M::ON || at.i >= p.nchunk) return;
        const R rows(p, at, true);
        const TG *g = rows.template first<TG>(p.a.g, rows.gc);
#pragma unroll
        for (int r = 0; r < (HEAD ? S::ROWS : 1); r++) g_now[r] = r < rows.count ? g[r * p.a.g.row_stride] : from_f<TG>(0.0f);
    };
    if (M::ON) {
        if (threadIdx.x == 0) {
            mbar_init(smem_u32(&bars[0]), 1);
            mbar_init(smem_u32(&bars[1]), 1);
        }
        __syncthreads();
        fetch(next, 0);
        fetch_gates(next);
    }
    int turn = 0;
    uint32_t phase = 0;
    while (next.i < p.nchunk) {
        const Place now = next;
        next.advance(p, by);
        char *const pg = buffers + turn * TILE_BYTES, *const pv = pg + M::G_BYTES, *const pd = pg + M::INPUT_BYTES;
        const R rows(p, now, true);
        const Place &at = rows.at;
        const int c0 = rows.c0, c = rows.c;
        const long long tile0 = (long long)rows.chunk * CHUNK;
        long long lo = 0, hi = p.a.L;
        bool edges = false;   // packed: a sequence starts or ends in this tile
        if (packed) {
            mark_sequences(p, marks, tile0, lo, hi);
            bool f = false;
            for (int i = threadIdx.x; i < CHUNK; i += S::THREADS) f |= marks.first[i] >= 0 || marks.last[i] >= 0;
            edges = __syncthreads_or(f);
        }
        const bool whole = !packed || (tile0 >= lo && tile0 + CHUNK <= hi);   // the tile's rows are all written, or do not exist
        // rows that do not exist hold the state and the gradient, and have no values
        const bool full = tile0 + CHUNK <= p.a.L, plain = whole && !edges && (M::ON || (full && rows.mine));
        auto in = [&](int r) { return r < rows.count && rows.t0 + r >= lo && rows.t0 + r < hi; };
        // packed: the sequence that row r starts or ends, or -1
        auto starts = [&](int r) { return rows.mine ? marks.first[group * S::ROWS + r] : -1; };
        auto ends = [&](int r) { return rows.mine ? marks.last[group * S::ROWS + r] : -1; };

        bool arrived = true;
        if (M::ON) arrived = mbar_wait(smem_u32(&bars[turn]), phase, p.copy_polls);
        // the rows' gates stay in registers, values and dy where the copies put them (V = 1: in registers)
        float k[S::ROWS][GV];
        Pack<TV, V> own_v[M::ON ? 1 : S::ROWS], own_d[M::ON ? 1 : S::ROWS];
        {
            const TG *gp = rows.template first<TG>(p.a.g, rows.gc);
            const TV *vp = rows.template first<TV>(p.a.v, c), *dp = rows.template first<TV>(p.a.dy, c);
#pragma unroll
            for (int r = 0; r < S::ROWS; r++) {
                Pack<TG, GV> g;
                const bool there = (plain && full) || in(r);
                if constexpr (M::ON) {
                    if constexpr (HEAD) g.v[0] = g_now[r];
                    else g = load<TG, GV>(reinterpret_cast<const TG *>(pg + M::at_g(r)));
                } else {
#pragma unroll
                    for (int j = 0; j < V; j++) own_v[r].v[j] = own_d[r].v[j] = from_f<TV>(0.0f);
                    if (there) {
                        g = load<TG, GV>(gp + r * p.a.g.row_stride);
                        own_v[r] = load<TV, V>(vp + r * p.a.v.row_stride);
                        own_d[r] = load<TV, V>(dp + r * p.a.dy.row_stride);
                    }
                }
                float gf[GV];
                floats(gf, g);
                pack_gates<FORM, FAST>(gf, k[r]);
#pragma unroll
                for (int j = 0; j < GV; j++)
                    if (!there) k[r][j] = HOLD<FORM>;
            }
        }
        // row r of values or dy; rows that are missing or in no sequence are zero
        auto value = [&](auto careful, int r, float (&f)[V]) {
            Pack<TV, V> x;
            if constexpr (M::ON) x = load<TV, V>(reinterpret_cast<const TV *>(pv + M::at_v(r)));
            else x = own_v[r];
            floats(f, x);
            if (decltype(careful)::value && !in(r)) fill(f, 0.0f);
        };
        auto gradient = [&](auto careful, int r, float (&f)[V]) {
            Pack<TV, V> x;
            if constexpr (M::ON) x = load<TV, V>(reinterpret_cast<const TV *>(pd + M::at_v(r)));
            else x = own_d[r];
            floats(f, x);
            if (decltype(careful)::value && !in(r)) fill(f, 0.0f);
        };
        auto opened = [&](int r, float (&a)[V], float (&c)[V]) {
            float ka[GV], kc[GV];
            open_gates<FORM>(k[r], ka, kc);
            spread(a, ka);
            spread(c, kc);
        };

        float P[V], Q[V], T[V], E[V];
        auto walk = [&](auto careful) {
            constexpr bool CARE = decltype(careful)::value;
            fill(P, 1.0f);
            fill(T, 1.0f);
            fill(Q, 0.0f);
            fill(E, 0.0f);
#pragma unroll
            for (int r = 0; r < S::ROWS; r++) {
                if (CARE && edges) {
                    const long long n = starts(r);
                    if (n >= 0)
#pragma unroll
                        for (int j = 0; j < V; j++) P[j] = 0.0f, Q[j] = p.a.h0 ? p.a.h0[n * p.C + c + j] : 0.0f;
                }
                float v[V], a[V], b[V];
                value(careful, r, v);
                opened(r, a, b);
                if constexpr (CARE) {
#pragma unroll
                    for (int j = 0; j < V; j++) P[j] = mul0(a[j], P[j]);
#pragma unroll
                    for (int j = 0; j < V; j++) Q[j] = fma0(a[j], Q[j], FORM == GATED_SCAN_EXP ? v[j] : mul0(b[j], v[j]));
                } else {
                    mul_all(P, P, a);
                    if (FORM == GATED_SCAN_SIGMOID) mul_all(v, b, v);
                    fma_all(Q, a, Q, v);
                }
            }
#pragma unroll
            for (int r = S::ROWS - 1; r >= 0; r--) {
                if (CARE && edges) {
                    const long long n = ends(r);
                    if (n >= 0)
#pragma unroll
                        for (int j = 0; j < V; j++) T[j] = 0.0f, E[j] = p.a.dhT ? p.a.dhT[n * p.C + c + j] : 0.0f;
                }
                float d[V], a[V], b[V];
                gradient(careful, r, d);
                opened(r, a, b);
                add_all(E, d, E);
                if constexpr (CARE) {
#pragma unroll
                    for (int j = 0; j < V; j++) E[j] = mul0(a[j], E[j]), T[j] = mul0(a[j], T[j]);
                } else {
                    mul_all(E, a, E);
                }
            }
            if (!CARE)
#pragma unroll
                for (int j = 0; j < V; j++) T[j] = P[j];   // the same product
        };
        bool fine = plain;
        if (fine) {
            walk(std::false_type{});
#pragma unroll
            for (int j = 0; j < V; j++) fine &= finite(Q[j]) && finite(E[j]) && (FORM == GATED_SCAN_SIGMOID || finite(P[j]));
        }
        if (!fine) walk(std::true_type{});
        put(&sQ[group][lane * V], Q);
        put(&sR[group][lane * V], T);
        put(&sE[group][lane * V], E);
        if constexpr (IN_PLACE) {
            // float4 in the first row's gates, or a half in each of the first two
            float *a = reinterpret_cast<float *>(pg + M::at_g(0)), *b = reinterpret_cast<float *>(pg + M::at_g(1));
            asm volatile("" ::: "memory");   // the gates have been read
            if constexpr (sizeof(TG) == 4) {
                *reinterpret_cast<float4 *>(a) = make_float4(P[0], P[1], P[2], P[3]);
            } else {
                *reinterpret_cast<float2 *>(a) = make_float2(P[0], P[1]);
                *reinterpret_cast<float2 *>(b) = make_float2(P[2], P[3]);
            }
        } else {
            put(&sP[group][lane * V], P);
        }
        if (!M::ON) {
            __syncthreads();
        } else if (!__syncthreads_and(arrived)) {
            lost = true;
            next = now;
            break;
        }

        if (M::ON && agent) out_read();   // the other buffer's gradients have left it
        fetch(next, turn ^ 1);
        fetch_gates(next);
        const int x = threadIdx.x, cx = c0 + threadIdx.x % S::WIDTH;
        unsigned long long *const words = p.words + at.first_word(p) * S::WIDTH;
        const bool more = !p.serial && at.i + 1 < p.nchunk;
        float allT = 1.0f, allE = 0.0f;
        if (x < S::WIDTH) {
            // each group's pair becomes that of all groups ahead of it, going back
#pragma unroll
            for (int i = S::GROUPS - 1; i >= 0; i--) {
                const float gT = sR[i][x], gE = sE[i][x];
                sR[i][x] = allT;
                sE[i][x] = allE;
                allE = fma0(gT, allE, gE);
                allT = mul0(gT, allT);
            }
            if (at.i > 0 && more && cx < p.C) publish(words + (long long)at.i * S::WIDTH + x, allT, allE);
        } else if (x < 2 * S::WIDTH) {
            // each group's result becomes the state ahead of it
            const int y = x - S::WIDTH;
            float h = cx < p.C ? p.a.states[state_at(p, at.b, rows.chunk) + cx] : 0.0f;
#pragma unroll
            for (int i = 0; i < S::GROUPS; i++) {
                float gP;
                if constexpr (IN_PLACE)
                    gP = sizeof(TG) == 4 ? *reinterpret_cast<const float *>(pg + i * S::ROWS * M::G_ROW + y * 4)
                                         : *reinterpret_cast<const float *>(pg + (i * S::ROWS + y % 4 / 2) * M::G_ROW + y / 4 * 8 + y % 2 * 4);
                else
                    gP = sP[i][y];
                const float gQ = sQ[i][y];
                sQ[i][y] = h;
                h = fma0(gP, h, gQ);
            }
        }
        if (at.i > 0 && far) {
            look_back(ahead, words, at.i, cx < p.C, p.look_polls);
        } else if (at.i > 0) {
            if (x < S::WIDTH) ahead.state[x] = p.serial ? carry : cx < p.C ? look_near<S::WIDTH>(words + x, at.i, p.look_polls) : 0.0f;
            __syncthreads();
        } else {
            if (x < S::WIDTH) ahead.state[x] = !packed && p.a.dhT && cx < p.C ? p.a.dhT[end_at(p, at.b) + cx] : 0.0f;
            __syncthreads();
        }
        if (x < S::WIDTH && cx < p.C) {
            carry = fma0(allT, ahead.state[x], allE);
            if (more) publish(words + (long long)at.i * S::WIDTH + x, 0.0f, carry);
        }

        float h[V], e[V];
        auto start = [&]() {
            float gt[V], ge[V], grad[V];
            get(&sQ[group][lane * V], h);
            get(&sR[group][lane * V], gt);
            get(&sE[group][lane * V], ge);
            get(&ahead.state[lane * V], grad);
#pragma unroll
            for (int j = 0; j < V; j++) e[j] = fma0(gt[j], grad[j], ge[j]);
        };
        start();
#pragma unroll
        for (int j = 0; j < V; j++) fine &= finite(h[j]) && finite(e[j]);
        // lanes of one head: lane + 2^o is still in it
        bool same[5], leader = true;
        const bool one_head = HEAD && p.D % S::WIDTH == 0;   // in every strip
        if (HEAD && !one_head) {
#pragma unroll
            for (int o = 0; o < 5; o++) {
                const int other = c + (V << o);
                same[o] = lane + (1 << o) < S::LANES && other < p.C && head_of(p, other) == rows.gc;
            }
            leader = rows.mine && (lane == 0 || head_of(p, c - V) != rows.gc);
        }
        const int piece = HEAD && rows.mine ? at.strip - first_strip(rows.gc, p.D, S::WIDTH) : 0;
        // forward again for the gate's slope at every row, then back with the gradient
        auto finish = [&](auto careful) {
            constexpr bool CARE = decltype(careful)::value;
            float slope[S::ROWS][V];
#pragma unroll
            for (int r = 0; r < S::ROWS; r++) {
                if (CARE && edges) {
                    const long long n = starts(r);
                    if (n >= 0)
#pragma unroll
                        for (int j = 0; j < V; j++) h[j] = p.a.h0 ? p.a.h0[n * p.C + c + j] : 0.0f;
                }
                float v[V], a[V], b[V];
                value(careful, r, v);
                opened(r, a, b);
                if constexpr (CARE) {
#pragma unroll
                    for (int j = 0; j < V; j++) {
                        slope[r][j] = FORM == GATED_SCAN_EXP ? mul0(a[j], h[j]) : mul0(a[j] * b[j], h[j] - v[j]);
                        h[j] = fma0(a[j], h[j], FORM == GATED_SCAN_EXP ? v[j] : mul0(b[j], v[j]));
                    }
                } else if constexpr (FORM == GATED_SCAN_EXP) {
                    mul_all(slope[r], a, h);
                    add_all(h, slope[r], v);
                } else {
                    float ah[V], less[V], minus[V];
                    fill(minus, -1.0f);
                    mul_all(ah, a, b);
                    fma_all(less, v, minus, h);
                    mul_all(slope[r], ah, less);
                    mul_all(v, b, v);
                    fma_all(h, a, h, v);
                }
            }
            // what overflows among the rows stays without a finite value to their end; a held row's distance from
            // its state is in the slopes alone
            constexpr bool IN_SLOPES = !CARE && FORM == GATED_SCAN_SIGMOID;
            if (!CARE)
#pragma unroll
                for (int j = 0; j < V; j++) fine &= finite(h[j]);
            asm volatile("" ::: "memory");   // dv goes where the values were
            TV *dv_row = rows.template first<TV>(p.a.dv, c);
            [[maybe_unused]] float head[HEAD ? S::ROWS : 1];
            [[maybe_unused]] float all[HEAD ? 1 : V];
            fill(all, 0.0f);
            [[maybe_unused]] TG *dg_row = rows.template first<TG>(p.a.dg, rows.gc);
#pragma unroll
            for (int r = S::ROWS - 1; r >= 0; r--) {
                const bool here = !CARE || in(r);
                if (CARE && edges) {
                    const long long n = ends(r);
                    if (n >= 0)
#pragma unroll
                        for (int j = 0; j < V; j++) e[j] = p.a.dhT ? p.a.dhT[n * p.C + c + j] : 0.0f;
                }
                float d[V], dv[V], dg[V], a[V], b[V];
                gradient(careful, r, d);
                opened(r, a, b);
                add_all(d, d, e);
                mul_all(dg, slope[r], d);
                if constexpr (CARE) {
#pragma unroll
                    for (int j = 0; j < V; j++) {
                        dv[j] = !here ? 0.0f : FORM == GATED_SCAN_EXP ? d[j] : mul0(b[j], d[j]);
                        dg[j] = here && (FORM == GATED_SCAN_EXP ? a[j] : a[j] * b[j]) != 0.0f ? dg[j] : 0.0f;
                        e[j] = mul0(a[j], d[j]);
                    }
                } else {
                    if (FORM == GATED_SCAN_EXP) {
#pragma unroll
                        for (int j = 0; j < V; j++) dv[j] = d[j];
                    } else {
                        mul_all(dv, b, d);
                    }
                    mul_all(e, a, d);
                }
                // rows of tiles that are not whole go straight to memory
                const bool write = here || (r < rows.count && p.a.zero_outside);
                if (M::ON && (!CARE || whole))
                    store<TV, V>(reinterpret_cast<TV *>(pv + M::at_v(r)), dv);
                else if (write)
                    store<TV, V>(dv_row + r * p.a.dv.row_stride, dv);
                if constexpr (!HEAD) {
                    if (M::ON && (!CARE || whole))
                        store<TG, V>(reinterpret_cast<TG *>(pg + M::at_g(r)), dg);
                    else if (write)
                        store<TG, V>(dg_row + r * p.a.dg.row_stride, dg);
                    if constexpr (IN_SLOPES) add_all(all, all, dg);
                } else {
                    head[r] = 0.0f;
#pragma unroll
                    for (int j = 0; j < V; j++) head[r] += dg[j];
                    if constexpr (IN_SLOPES) all[0] += head[r];
                }
                if (CARE && edges && here && p.a.dh0) {
                    const long long m = starts(r);
                    if (m >= 0)
#pragma unroll
                        for (int j = 0; j < V; j++) p.a.dh0[m * p.C + c + j] = e[j];
                }
            }
            if constexpr (!CARE)
#pragma unroll
                for (int j = 0; j < V; j++) fine &= finite(e[j]) && (!IN_SLOPES || finite(all[HEAD ? 0 : j]));
            if constexpr (HEAD) {
                // the sums over a head's lanes
                auto write = [&](int r, float sum) {
                    if (r >= rows.count || (CARE && !in(r) && !p.a.zero_outside)) return;
                    put_gate<TG>(p, at.b, rows.t0 + r, rows.gc, piece, sum);
                };
                if (one_head) {
                    // halving: each exchange leaves a lane half of its rows, until it has one (or its share of one)
#pragma unroll
                    for (int o = S::LANES / 2, n = S::ROWS; o > 0; o >>= 1) {
                        if (n > 1) {
                            n >>= 1;
#pragma unroll
                            for (int r = 0; r < n; r++) {
                                const bool up = lane & o;
                                const float give = up ? head[r] : head[r + n], stay = up ? head[r + n] : head[r];
                                head[r] = stay + __shfl_xor_sync(0xffffffffu, give, o, S::LANES);
                            }
                        } else {
                            head[0] += __shfl_xor_sync(0xffffffffu, head[0], o, S::LANES);
                        }
                    }
                    constexpr int SHARE = S::LANES / S::ROWS > 0 ? S::LANES / S::ROWS : 1;   // lanes with the same row
                    if (lane % SHARE == 0)
                        if (rows.mine) write(lane / SHARE, head[0]);
                } else {
#pragma unroll
                    for (int r = 0; r < S::ROWS; r++) {
                        float sum = head[r];
#pragma unroll
                        for (int o = 0; (1 << o) < S::LANES; o++) {
                            const float other = __shfl_down_sync(0xffffffffu, sum, 1 << o, S::LANES);
                            sum += same[o] ? other : 0.0f;
                        }
                        if (leader) write(r, sum);
                    }
                }
            }
        };
        // a warp's lanes sum their heads' gradients together: one way for all of them
        const auto agreed = [&]() { return HEAD ? (bool)__all_sync(0xffffffffu, fine) : fine; };
        if (agreed()) {
            finish(std::false_type{});
            if (!agreed()) {
                // heads' gradients written so far are written over by other lanes; here all of the warp's come
                if constexpr (HEAD) __syncwarp();
                Ends<V> ends;
                start();
#pragma unroll
                for (int j = 0; j < V; j++) ends.h[j] = h[j], ends.e[j] = e[j];
                ends = one_by_one<TV, TG, FORM, HEAD, V>(p, at.b, at.strip, rows.chunk, ends, pg, pv);
#pragma unroll
                for (int j = 0; j < V; j++) e[j] = ends.e[j];
            }
        } else {
            finish(std::true_type{});
        }
        if (!packed && rows.chunk == 0 && group == 0 && rows.mine && p.a.dh0)
#pragma unroll
            for (int j = 0; j < V; j++) p.a.dh0[end_at(p, at.b) + c + j] = e[j];
        if (M::ON) {
            fence_proxy_async();
            __syncthreads();
            if (agent && whole) {
                const int t0 = rows.chunk * CHUNK;
                if (!HEAD) tensor_out(&maps.dg, c0, t0, (int)at.b, pg);
                tensor_out(&maps.dv, c0, t0, (int)at.b, pv);
                out_close();
            }
            phase ^= turn;
            turn ^= 1;
        }
    }
    if (M::ON && agent) out_done();
    if (M::ON && lost) {
        if (agent) mbar_wait(smem_u32(&bars[turn]), phase, COPY_POLLS);
        leave_nan<TV, TG, HEAD, V, true>(p, next, marks);
    }
    if (packed && p.a.dh0) pass_states(p.a.cu_seqlens, p.nseq, p.C, p.a.dhT, p.a.dh0);
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

// One token.  A block has a row and STEP_THREADS * V channels of it; the loads that decide nothing
// come first.  Rows of one slot belong to the first of them, which takes the others in order: every
// block looks through the slots for rows ahead of its own and behind it (B words from the caches).
constexpr int STEP_THREADS = 128;
template <typename TV, typename TG, int FORM, bool HEAD, int V>
__global__ void __launch_bounds__(STEP_THREADS) scan_step(int B, int C, int D, const TG *g, long long gs, const TV *v, long long vs,
                                                          const float *state, long long S, const int *slots, TV *y, long long ys, float *next,
                                                          int zero_skipped) {
    constexpr int GV = HEAD ? 1 : V;
    const int c = (blockIdx.y * STEP_THREADS + threadIdx.x) * V, i0 = blockIdx.x;
    const int gc = HEAD ? c / D : c;
    const long long slot = slots ? slots[i0] : i0;
    const bool there = slot >= 0 && slot < S;
    Pack<float, V> h;
    Pack<TG, GV> gi;
    Pack<TV, V> vi;
    if (there && c < C) {
        h = load<float, V>(state + slot * C + c);
        gi = load<TG, GV>(g + i0 * gs + gc);
        vi = load<TV, V>(v + i0 * vs + c);
    }
    bool behind = false;
    if (slots) {
        bool before = false;
        for (int j = threadIdx.x; j < B; j += STEP_THREADS)
            if (j != i0 && slots[j] == slot) (j < i0 ? before : behind) = true;
        if (__syncthreads_or(before && there)) return;
        behind = __syncthreads_or(behind);
    }
    if (c >= C) return;
    if (!there) {
        const float zero[V] = {};
        if (zero_skipped) store<TV, V>(y + i0 * ys + c, zero);
        return;
    }
    for (int i = i0;;) {
        float f[V];
#pragma unroll
        for (int j = 0; j < V; j++) {
            const Gate k = gate_of<FORM>(to_f(gi.v[HEAD ? 0 : j]));
            h.v[j] = f[j] = fma0(k.a, h.v[j], FORM == GATED_SCAN_EXP ? to_f(vi.v[j]) : mul0(k.c, to_f(vi.v[j])));
        }
        store<TV, V>(y + i * ys + c, f);
        if (!behind) break;
        do i++;
        while (i < B && slots[i] != slot);
        if (i >= B) break;
        gi = load<TG, GV>(g + i * gs + gc);
        vi = load<TV, V>(v + i * vs + c);
    }
    *reinterpret_cast<Pack<float, V> *>(next + slot * C + c) = h;
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
int width_of(const gated_scan_s *h, int V) { return V == 4 ? 128 / (int)elem(h->dtype) : 32; }
int strips_of(const gated_scan_s *h, int V) { return (h->C + width_of(h, V) - 1) / width_of(h, V); }

// The most strips that a head's channels lie in.
int pieces_of(const gated_scan_s *h, int V) {
    if (h->per != GATED_SCAN_PER_HEAD) return 1;
    const int w = width_of(h, V);
    if (w % h->D == 0) return 1;
    int most = 1;
    // the first channels of heads within a strip repeat after w heads at the latest
    for (int i = 0; i < h->H && i < w; i++) {
        const int n = last_strip(i, h->D, w) - first_strip(i, h->D, w) + 1;
        most = n > most ? n : most;
    }
    return most;
}

// Blocks an SM that the kernels are built for.
int blocks_per_sm(const gated_scan_s *h, bool backward, int V) {
    if (V == 1) return SINGLE_BLOCKS;
    if (backward) return BACKWARD_BLOCKS;
    const bool head = h->per == GATED_SCAN_PER_HEAD;
    return h->dtype == SPECTRE_F32 ? (head ? FORWARD_BLOCKS<float, true> : FORWARD_BLOCKS<float, false>)
                                   : (head ? FORWARD_BLOCKS<__nv_bfloat16, true> : FORWARD_BLOCKS<__nv_bfloat16, false>);
}

struct Work {
    bool serial;                  // a block takes whole strips: no words, and an ordinary launch
    size_t words, parts, bytes;   // offset of the parts, the whole
};
Work work_of(const gated_scan_s *h, long long B, long long L, bool backward, int V) {
    const long long nchunk = (L + CHUNK - 1) / CHUNK, strips = B * strips_of(h, V);
    const long long most = (long long)h->nsm * blocks_per_sm(h, backward, V);
    // In tiles that the busiest block takes; looking back costs about a twentieth more and, with the
    // words to clear and the blocks to start together, one tile.  Forward in microseconds, strip by
    // strip against looking back, rows of 512 bf16 channels: 256 rows 8.2 and 10.3, 1,024 rows 20.5
    // and 10.3, 111 x 1,024 rows 67 and 79; 4 x 12,288 rows of 2,048 channels 197 and 127.
    const long long one = (strips + most - 1) / most * nchunk, all = (strips * nchunk + most - 1) / most;
    Work w{};
    w.serial = one * 20 <= all * 21 + 20;
    if (!w.serial) w.words = ((size_t)strips * nchunk + AHEAD) * width_of(h, V) * 8;
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

// Rows that tensor copies can move: 16-byte aligned, with strides that are, and not into one another.
bool sixteens(const gated_scan_rows &r, size_t es, long long width, long long B, long long L) {
    const auto ok = [&](long long n, long long stride) { return n < 2 || (stride >= width && stride * es % 16 == 0 && stride * es < (1ull << 40)); };
    return aligned(r.data, 16) && ok(L, r.row_stride) && ok(B, r.batch_stride);
}
int vector_of(const gated_scan_s *h, const gated_scan_args *a, bool backward) {
    const bool head = h->per == GATED_SCAN_PER_HEAD;
    if ((head ? h->D : h->C) % 4 || a->L > 0x7fffffffLL || a->B > 0x7fffffffLL) return 1;
    const size_t ev = elem(h->dtype), eg = elem(h->gate_dtype);
    const auto ok = [&](const gated_scan_rows &r, size_t es) { return sixteens(r, es, h->C, a->B, a->L); };
    if (!ok(a->v, ev) || (!head && !ok(a->g, eg))) return 1;
    if (!backward) return ok(a->y, ev) ? 4 : 1;
    return ok(a->dy, ev) && ok(a->dv, ev) && (head || ok(a->dg, eg)) ? 4 : 1;
}

PFN_cuTensorMapEncodeTiled_v12000 find_encode() {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

template <typename T> bool encode(CUtensorMap *m, const gated_scan_rows &r, const Args &p, int width) {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = find_encode();
    if (!fn) return false;
    const cuuint64_t es = sizeof(T), line = (p.C * es + 15) / 16 * 16;
    const cuuint64_t dims[3] = {(cuuint64_t)p.C, (cuuint64_t)p.a.L, (cuuint64_t)p.a.B};
    // a stride along one row or one batch entry is never used, but has to be a legal one
    const cuuint64_t strides[2] = {p.a.L > 1 ? (cuuint64_t)r.row_stride * es : line, p.a.B > 1 ? (cuuint64_t)r.batch_stride * es : line};
    const cuuint32_t box[3] = {(cuuint32_t)width, CHUNK, 1}, step[3] = {1, 1, 1};
    return fn(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, r.data, dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Blocks of a kernel that an SM holds at once, 0 where that cannot be told.
template <typename K> int resident(K kernel, int threads, int bytes) {
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, bytes) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

template <typename TV, typename TG, int FORM, bool HEAD, int V>
cudaError_t launch_tiles(Args &p, bool backward, const Work &w, cudaStream_t s) {
    using S = Tile<TV, V>;
    using M = Stage<TV, TG, HEAD, V>;
    const long long tiles = p.a.B * p.strips * p.nchunk;
    Maps maps;
    if (M::ON) {
        bool ok = HEAD || encode<TG>(&maps.g, p.a.g, p, S::WIDTH);
        ok = ok && encode<TV>(&maps.v, p.a.v, p, S::WIDTH);
        if (!backward) {
            ok = ok && encode<TV>(&maps.y, p.a.y, p, S::WIDTH);
        } else {
            ok = ok && encode<TV>(&maps.dy, p.a.dy, p, S::WIDTH) && encode<TV>(&maps.dv, p.a.dv, p, S::WIDTH);
            ok = ok && (HEAD || encode<TG>(&maps.dg, p.a.dg, p, S::WIDTH));
        }
        if (!ok) return cudaErrorInvalidValue;
    }
    if (w.words) {
        p.words = static_cast<unsigned long long *>(p.a.work) + AHEAD * S::WIDTH;
        const cudaError_t e = cudaMemsetAsync(p.a.work, 0xff, w.words, s);
        if (e != cudaSuccess) return e;
    }
    if (w.parts) p.parts = reinterpret_cast<float *>(static_cast<char *>(p.a.work) + w.words);
    const auto kernel = backward ? scan_backward<TV, TG, FORM, HEAD, V> : scan_forward<TV, TG, FORM, HEAD, V>;
    const int bytes = M::ON ? 2 * (M::INPUT_BYTES + (backward ? M::V_BYTES : 0)) : 0;
    // asked for once (every device of this library is of one kind); the attribute is a device's own
    static const int per_sm[2] = {resident(scan_forward<TV, TG, FORM, HEAD, V>, S::THREADS, M::ON ? 2 * M::INPUT_BYTES : 0),
                                  resident(scan_backward<TV, TG, FORM, HEAD, V>, S::THREADS, M::ON ? 2 * (M::INPUT_BYTES + M::V_BYTES) : 0)};
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    const long long most = (long long)p.nsm * per_sm[backward], blocks = w.serial ? p.a.B * p.strips : tiles;
    p.serial = w.serial;
    if (!most) return cudaErrorUnknown;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3((unsigned)(blocks < most ? blocks : most));
    config.blockDim = dim3(S::THREADS);
    config.dynamicSmemBytes = bytes;
    config.stream = s;
    cudaLaunchAttribute together{};
    together.id = cudaLaunchAttributeCooperative;
    together.val.cooperative = 1;
    config.attrs = &together;
    config.numAttrs = p.words ? 1 : 0;   // blocks that wait for one another run at the same time
    e = cudaLaunchKernelEx(&config, kernel, p, maps);
    if (e != cudaSuccess) return e;
    if (w.parts) {
        const long long n = p.a.B * p.a.L * p.H;
        join_parts<TG><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p, S::WIDTH);
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
    if (nchunk > 0x7fffffffLL / strips_of(h, 1) / a->B) return SPECTRE_ERR_ARG;
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
        if (!to || !nseq) return SPECTRE_OK;
        const long long need = (nseq + PASS_THREADS / 32 - 1) / (PASS_THREADS / 32);
        pass_all<<<(unsigned)(need < PASS_BLOCKS ? need : PASS_BLOCKS), PASS_THREADS, 0, s>>>(nseq, h->C, backward ? a->dhT : a->h0, to);
        return status_of(cudaGetLastError());
    }
    Args p{};
    p.a = *a;
    p.H = h->H;
    p.D = h->D;
    p.C = h->C;
    p.head_of = ((1ull << 40) + h->D - 1) / h->D;
    p.strips = strips_of(h, V);
    p.nsm = h->nsm;
    p.copy_polls = h->test_wait == 1 ? 0 : COPY_POLLS;
    p.look_polls = h->test_wait == 2 ? 0 : MOST_POLLS;
    p.nchunk = (int)nchunk;
    p.nseq = nseq;
    return status_of(h->gate == GATED_SCAN_EXP ? launch_types<GATED_SCAN_EXP>(h, p, V, backward, work, s)
                                               : launch_types<GATED_SCAN_SIGMOID>(h, p, V, backward, work, s));
}

template <typename TV, typename TG, int FORM, bool HEAD, int V>
cudaError_t launch_step(const gated_scan_s *h, long long B, const void *g, long long gs, const void *v, long long vs,
                        const float *state, long long S, const int *slots, void *y, long long ys, float *next, int zero_skipped,
                        cudaStream_t s) {
    const dim3 grid((unsigned)B, (h->C + STEP_THREADS * V - 1) / (STEP_THREADS * V));
    scan_step<TV, TG, FORM, HEAD, V><<<grid, STEP_THREADS, 0, s>>>((int)B, h->C, h->D, static_cast<const TG *>(g), gs, static_cast<const TV *>(v), vs,
                                                                   state, S, slots, static_cast<TV *>(y), ys, next, zero_skipped);
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
    gated_scan_s *h = new (std::nothrow) gated_scan_s{H, D, H * D, gate, per, dtype, gate_dtype, dev, nsm, 0};
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
                    long long y_stride, float *new_state, int zero_skipped, void *stream) {
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
    const bool head = h->per == GATED_SCAN_PER_HEAD;
    const auto four = [](const void *p, long long stride, size_t es) { return aligned(p, 4 * es) && stride % 4 == 0; };
    const bool vec = (head ? h->D : h->C) % 4 == 0 && four(v, v_stride, ev) && four(y, y_stride, ev) && (head || four(g, g_stride, eg)) &&
                     aligned(state, 16) && aligned(new_state, 16);
    auto go = [&](auto tv, auto tg, auto form, auto hd, auto four) {
        return status_of(launch_step<decltype(tv), decltype(tg), decltype(form)::value, decltype(hd)::value, decltype(four)::value>(
            h, B, g, g_stride, v, v_stride, state, S, slots, y, y_stride, new_state, zero_skipped, s));
    };
    auto go_shape = [&](auto tv, auto tg, auto form) {
        using one = std::integral_constant<int, 1>;
        using many = std::integral_constant<int, 4>;
        if (head) return vec ? go(tv, tg, form, std::true_type{}, many{}) : go(tv, tg, form, std::true_type{}, one{});
        return vec ? go(tv, tg, form, std::false_type{}, many{}) : go(tv, tg, form, std::false_type{}, one{});
    };
    auto go_types = [&](auto form) {
        if (h->dtype == SPECTRE_F32) return go_shape(0.0f, 0.0f, form);
        if (h->gate_dtype == SPECTRE_F32) return go_shape(bf(), 0.0f, form);
        return go_shape(bf(), bf(), form);
    };
    return h->gate == GATED_SCAN_EXP ? go_types(std::integral_constant<int, GATED_SCAN_EXP>{}) : go_types(std::integral_constant<int, GATED_SCAN_SIGMOID>{});
}

int gated_scan_set_option(gated_scan_t h, int option, int value) {
    if (!h || option != GATED_SCAN_OPT_TEST_WAIT_TIMEOUT || value < 0 || value > 2) return SPECTRE_ERR_ARG;
    h->test_wait = value;
    return SPECTRE_OK;
}

int gated_scan_device_status(gated_scan_t h, void *stream) {
    if (!h) return SPECTRE_ERR_ARG;
    if (!gscan::current_device_is(h->device)) return SPECTRE_ERR_DEVICE;
    unsigned word = 0;
    const unsigned clear = 0;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&word, gscan::wait_gave_up, sizeof word);
    if (e == cudaSuccess && word) e = cudaMemcpyToSymbol(gscan::wait_gave_up, &clear, sizeof clear);
    return e == cudaSuccess && word ? SPECTRE_ERR_TIMEOUT : rows_io::status_of(e);
}

int gated_scan_destroy(gated_scan_t h) {
    delete h;
    return SPECTRE_OK;
}

}  // extern "C"
