// residual_norm.cu -- y = N(out + x) or N(out) + x over rows of C values, N LayerNorm or
// RMSNorm, its backward pass, and their C ABI (residual_norm.h).
//
// TPR threads (a power of two) hold one row in registers, EPT = 8 or 16 values a thread, so a
// row is read once: the sums of a row are shuffles within a warp and, for rows wider than a
// warp's share, one exchange of the warps' sums through shared memory.  Going forward a thread
// loads its part of the next row before it works on this one.  In the backward pass, which has
// no registers for that, rows come by bulk copies into a ring of stages that each row's threads
// have for themselves; rows that cannot be copied so (short, or not 16-byte aligned) are loaded.  The variance is
// taken about the mean in a second sum over the registers (a one-pass sum of squares loses
// it where the mean is large).  The backward pass recomputes the row's statistics from its
// registers instead of reading saved ones, and takes the three sums that need the mean (of
// squares, of dn and of dn (z - mean)) in one exchange.  Each thread keeps the sums of dy n
// and dy of its columns over the rows that its block takes, the block writes them once, and
// a second kernel adds the blocks' rows in their order.
#include <cmath>
#include <new>

#include "residual_norm.h"
#include "rows_io.cuh"
#include "tc_dft.cuh"

struct residual_norm_s {
    int C, dtype, norm;
    float eps;
    int device, nsm;
    int test_wait;   // RESIDUAL_NORM_OPT_TEST_WAIT_TIMEOUT
};

namespace resnorm {

using namespace rows_io;

constexpr int MAX_C = 8192;
constexpr int MAX_EPT = 16;                    // values of a row that a thread holds: 8 or 16
constexpr int MAX_THREADS = MAX_C / MAX_EPT;   // 512
constexpr int MIN_THREADS = 256;

struct Args {
    long long T;
    int C, tpr;
    float eps;
    const void *dy, *out, *x;
    void *y;   // forward: y, backward: dz
    long long dys, outs, xs, ys;
    const float *gamma, *beta;
    float *part_gamma, *part_beta;   // backward: block i's sums at + i * part_stride
    long long part_stride;
    int stages, stage_bytes;   // of the ring
    unsigned polls;            // after which a wait for a copy gives up
};

constexpr int MAX_STAGES = 4;
constexpr int MAX_RINGS = MIN_THREADS / 32;   // rows of a block that have one: a warp's or wider
constexpr unsigned COPY_POLLS = 4000;         // of up to a millisecond's suspension each

// VEC neighbouring values: one 16-byte access where they are 16 bytes, else one value.
// Rows pass through once: they leave the first-level cache to gamma and beta.
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> load(const T *p) {
    Pack<T, VEC> r;
    if constexpr (sizeof(T) * VEC == 16) {
        uint4 u;
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
        *reinterpret_cast<uint4 *>(r.v) = u;
    } else {
        r.v[0] = __ldg(p);
    }
    return r;
}
// VEC values of gamma or beta: from the first-level cache at every row, for registers are dearer.
template <int VEC> __device__ __forceinline__ Vec<VEC> load_vector(const float *p) {
    Vec<VEC> r;
    if constexpr (VEC == 1) {
        r.p = __ldg(p);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 2; i += 2)
            asm volatile("ld.global.nc.v2.u64 {%0, %1}, [%2];" : "=l"(r.p[i]), "=l"(r.p[i + 1]) : "l"(p + 2 * i));
    }
    return r;
}
template <typename T, int VEC> __device__ __forceinline__ void store(T *p, const Vec<VEC> &f) {
    *reinterpret_cast<Pack<T, VEC> *>(p) = packed<T, VEC>(f);
}

// K sums over the row's threads, in every one of them; the same order for every row
template <int K> __device__ __forceinline__ void row_sums(float (&s)[K], int tpr, int &turn) {
    __shared__ float warp_sums[2][K][MAX_THREADS / 32];
    if (tpr >= 32) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < K; k++) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    } else {
        for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < K; k++) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    }
    if (tpr <= 32) {
        __syncwarp();
        return;
    }
    // two buffers in turn: a warp writes a buffer again only after the barrier that follows
    // every warp's reads of it.  Each row of the block has a barrier of its own.
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; k++) warp_sums[turn][k][threadIdx.x >> 5] = s[k];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + threadIdx.x / tpr), "r"(tpr) : "memory");
#pragma unroll
    for (int k = 0; k < K; k++) s[k] = 0.0f;
    // the row's warps, 2 to 16, taken as 16: each of them counts 16 / warps times, which a power of
    // two takes back exactly
    const int first = threadIdx.x / tpr * (tpr / 32), warps = tpr / 32;
    const float share = (float)warps * 0.0625f;
#pragma unroll
    for (int k = 0; k < K; k++) {
        s[k] = warp_sums[turn][k][first + (threadIdx.x & (warps - 1))] * share;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    }
    turn ^= 1;
}

// Set where a bounded wait gave up; residual_norm_device_status reads and clears it.
__device__ unsigned wait_gave_up;

using spectre::tc::bulk_copy_g2s;
using spectre::tc::mbar_arrive_expect_tx;
using spectre::tc::mbar_init;
using spectre::tc::mbar_wait;
using spectre::tc::smem_u32;

// Where a row did not come in time, the thread waits for no more and has NaN for it and those behind it.  The one that
// asks for them asks for no more either, and waits here for those on their way (rows_left counts from the lost one, of
// which the block takes every rows-th), so that none lands in shared memory that is another block's by then.
__device__ __noinline__ void give_up(uint32_t bars, int stage, int stages, uint32_t phase, long long rows_left, long long rows) {
    atomicExch(&wait_gave_up, 1u);
    for (int i = 0; i < stages && rows_left > 0; i++, rows_left -= rows) {
        mbar_wait(bars + 8 * stage, phase, COPY_POLLS);
        if (++stage == stages) stage = 0, phase ^= 1;
    }
}

// A thread's part of a row of N tensors as it stands in memory; columns and rows that do not
// exist are zero.
template <typename T, int VEC, int EPT, int N, bool RING> struct Part {
    static constexpr int NV = EPT / VEC;
    const T *at[N];        // the row to ask for: its first value, or the thread's
    long long step[N];     // to the block's next row
    Pack<T, VEC> v[N][NV];
    char *ring;
    uint32_t bars;
    int stages, stage_bytes, stage, bytes;
    uint32_t phase;
    unsigned polls;
    bool leader, lost;
    __device__ __forceinline__ void begin(int k, const void *p, long long stride, long long r, long long rows, int c) {
        at[k] = static_cast<const T *>(p) + r * stride + (RING ? 0 : c);
        step[k] = rows * stride;
    }
    // the rows' rings, and the first rows on their way
    __device__ __forceinline__ void open(const Args &a, char *buffers, unsigned long long *all, int group, int lane, long long r, long long rows) {
        stages = a.stages;
        if constexpr (RING) {
            polls = a.polls;
            lost = false;
            stage_bytes = a.stage_bytes;
            bytes = a.C * (int)sizeof(T);
            ring = buffers + group * stages * stage_bytes;
            bars = smem_u32(all + group * MAX_STAGES);
            stage = 0;
            phase = 0;
            leader = lane == 0;
            if (leader)
                for (int i = 0; i < stages; i++) mbar_init(bars + 8 * i, 1);
            __syncthreads();
            for (int i = 0; i < stages; i++) {
                send(i, r < a.T);
                r += rows;
            }
        }
    }
    __device__ __forceinline__ void send(int s, bool there) {
        if (there && leader && !lost) {
            mbar_arrive_expect_tx(bars + 8 * s, N * bytes);
#pragma unroll
            for (int k = 0; k < N; k++) bulk_copy_g2s(smem_u32(ring + s * stage_bytes) + k * bytes, at[k], bytes, bars + 8 * s);
        }
#pragma unroll
        for (int k = 0; k < N; k++) at[k] += step[k];
    }
    // the row's values; rows_left: from it to the end, of which the block takes every rows-th
    template <typename M> __device__ __forceinline__ void fetch(long long rows_left, long long rows, const M &mine, int c, int apart) {
        const bool there = rows_left > 0;
        if constexpr (RING)
            if (there && !lost && !mbar_wait(bars + 8 * stage, phase, polls)) {
                lost = true;
                give_up(bars, stage, stages, phase, leader ? rows_left : 0, rows);
            }
#pragma unroll
        for (int k = 0; k < N; k++) {
#pragma unroll
            for (int i = 0; i < NV; i++) {
                if (!there || !mine[i]) {
#pragma unroll
                    for (int j = 0; j < VEC; j++) v[k][i].v[j] = from_f<T>(0.0f);
                    continue;
                }
                if constexpr (RING)
                    v[k][i] = *reinterpret_cast<const Pack<T, VEC> *>(ring + stage * stage_bytes + k * bytes + (c + i * apart) * (int)sizeof(T));
                else
                    v[k][i] = load<T, VEC>(at[k] + i * apart);
            }
            if (!RING) at[k] += step[k];
        }
        if constexpr (RING)
            if (there && lost)
#pragma unroll
                for (int k = 0; k < N; k++)
#pragma unroll
                    for (int i = 0; i < NV; i++)
                        if (mine[i])
#pragma unroll
                            for (int j = 0; j < VEC; j++) v[k][i].v[j] = from_f<T>(__uint_as_float(0x7fc00000u));
    }
    // after every thread of the row has its values: the stage's next row
    __device__ __forceinline__ void pass(bool there) {
        if constexpr (RING) {
            send(stage, there);
            if (++stage == stages) stage = 0, phase ^= 1;
        }
    }
};
// Which of a thread's values exist: all of them where the threads' shares fill the row.
template <int NV, bool FULL> struct Mine {
    bool m[FULL ? 1 : NV];
    __device__ __forceinline__ Mine(int c, int apart, int C) {
        if (!FULL)
#pragma unroll
            for (int i = 0; i < NV; i++) m[FULL ? 0 : i] = c + i * apart < C;
    }
    __device__ __forceinline__ bool operator[](int i) const { return FULL || m[FULL ? 0 : i]; }
};

// Registers a thread: what decides how many rows are in flight.
template <int EPT, bool BACK> constexpr int REGISTERS = BACK ? (EPT == 8 ? 80 : 128) : (EPT == 8 ? 64 : 80);
// The next row is loaded ahead where it has no ring and costs at most 32 bytes a tensor and thread.
template <typename T, int EPT, bool RING> constexpr bool AHEAD = !RING && sizeof(T) * EPT <= 32;

template <typename T, int VEC, int EPT, bool FULL, bool LN, bool POST>
__global__ void __maxnreg__((REGISTERS<EPT, false>)) norm_forward(const __grid_constant__ Args a) {
    constexpr int NV = EPT / VEC;
    const int lane = threadIdx.x % a.tpr, group = threadIdx.x / a.tpr, groups = blockDim.x / a.tpr;
    const int c0 = lane * VEC, apart = a.tpr * VEC;
    const float inv = 1.0f / (float)a.C;
    const long long rows = (long long)gridDim.x * groups;
    long long r = blockIdx.x * (long long)groups + group;
    const Mine<NV, FULL> mine(c0, apart, a.C);
    int turn = 0;
    Part<T, VEC, EPT, 2, false> next;
    next.begin(0, a.out, a.outs, r, rows, c0);
    next.begin(1, a.x, a.xs, r, rows, c0);
    T *y = static_cast<T *>(a.y) + r * a.ys + c0;
    constexpr bool EARLY = AHEAD<T, EPT, false>;
    if (EARLY) next.fetch(a.T - r, rows, mine, c0, apart);
    for (long long r0 = blockIdx.x * (long long)groups; r0 < a.T; r0 += rows, r += rows, y += rows * a.ys) {
        if (!EARLY) next.fetch(a.T - r, rows, mine, c0, apart);
        Vec<VEC> z[NV], sums(0.0f), squares(0.0f);
        Pack<T, VEC> xr[POST ? 1 : NV];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            z[i] = floats(next.v[0][i]);
            if constexpr (POST) z[i] = z[i] + floats(next.v[1][i]);
            else xr[i] = next.v[1][i];
            if (LN) sums = sums + z[i];
        }
        if (EARLY) next.fetch(a.T - r - rows, rows, mine, c0, apart);
        Vec<VEC> minus(0.0f);
        if (LN) {
            float s[1] = {sum_of(sums)};
            row_sums(s, a.tpr, turn);
            minus = Vec<VEC>(-s[0] * inv);
        }
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (mine[i]) {
                if (LN) z[i] = z[i] + minus;
                squares = fma(z[i], z[i], squares);
            }
        float s[1] = {sum_of(squares)};
        row_sums(s, a.tpr, turn);
        const float rstd = rsqrtf(s[0] * inv + a.eps);   // within two units of the last place
        const Vec<VEC> scale(rstd);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (r >= a.T || !mine[i]) continue;
            Vec<VEC> f = fma(z[i] * scale, load_vector<VEC>(a.gamma + c0 + i * apart), load_vector<VEC>(a.beta + c0 + i * apart));
            if constexpr (!POST) f = f + floats(xr[i]);
            store<T, VEC>(y + i * apart, f);
        }
    }
}

template <typename T, int VEC, int EPT, bool RING, bool FULL, bool LN, bool POST>
__global__ void __maxnreg__((REGISTERS<EPT, true>)) norm_backward(const __grid_constant__ Args a) {
    extern __shared__ __align__(128) char buffers[];
    __shared__ __align__(8) unsigned long long bars[RING ? MAX_RINGS * MAX_STAGES : 1];
    constexpr int NV = EPT / VEC;
    const int lane = threadIdx.x % a.tpr, group = threadIdx.x / a.tpr, groups = blockDim.x / a.tpr;
    const int c0 = lane * VEC, apart = a.tpr * VEC;
    const float inv = 1.0f / (float)a.C;
    const long long rows = (long long)gridDim.x * groups;
    long long r = blockIdx.x * (long long)groups + group;
    const Mine<NV, FULL> mine(c0, apart, a.C);
    int turn = 0;
    Vec<VEC> dgamma[NV], dbeta[NV];
#pragma unroll
    for (int i = 0; i < NV; i++) dgamma[i] = dbeta[i] = Vec<VEC>(0.0f);
    Part<T, VEC, EPT, POST ? 3 : 2, RING> next;
    next.begin(0, a.out, a.outs, r, rows, c0);
    next.begin(1, a.dy, a.dys, r, rows, c0);
    if constexpr (POST) next.begin(2, a.x, a.xs, r, rows, c0);
    T *dz = static_cast<T *>(a.y) + r * a.ys + c0;
    next.open(a, buffers, bars, group, lane, r, rows);
    constexpr bool EARLY = AHEAD<T, EPT, RING>;
    if (EARLY) next.fetch(a.T - r, rows, mine, c0, apart);
    for (long long r0 = blockIdx.x * (long long)groups; r0 < a.T; r0 += rows, r += rows, dz += rows * a.ys) {
        if (!EARLY) next.fetch(a.T - r, rows, mine, c0, apart);
        Vec<VEC> z[NV], dy[NV], sums(0.0f), squares(0.0f), along(0.0f), level(0.0f);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            z[i] = floats(next.v[0][i]);
            dy[i] = floats(next.v[1][i]);
            if constexpr (POST) z[i] = z[i] + floats(next.v[2][i]);
            if (LN) sums = sums + z[i];
        }
        if (EARLY) next.fetch(a.T - r - rows, rows, mine, c0, apart);
        Vec<VEC> minus(0.0f);
        if (LN) {
            float s[1] = {sum_of(sums)};
            row_sums(s, a.tpr, turn);
            minus = Vec<VEC>(-s[0] * inv);
        }
#pragma unroll
        for (int i = 0; i < NV; i++)
            if (mine[i]) {
                const Vec<VEC> dn = dy[i] * load_vector<VEC>(a.gamma + c0 + i * apart);
                if (LN) {
                    z[i] = z[i] + minus;
                    level = level + dn;
                }
                squares = fma(z[i], z[i], squares);
                along = fma(dn, z[i], along);
            }
        float s[3] = {sum_of(squares), sum_of(along), LN ? sum_of(level) : 0.0f};
        row_sums(s, a.tpr, turn);
        next.pass(r + next.stages * rows < a.T);
        const float rstd = rsqrtf(s[0] * inv + a.eps);   // within two units of the last place
        // r (dn - mean(dn) - n mean(dn n)), the means' factors taken together
        const Vec<VEC> scale(rstd), toward(-s[1] * rstd * inv * rstd), off(-s[2] * inv * rstd);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            if (r >= a.T || !mine[i]) continue;
            const Vec<VEC> n = z[i] * scale, dn = dy[i] * load_vector<VEC>(a.gamma + c0 + i * apart);
            dbeta[i] = dbeta[i] + dy[i];
            dgamma[i] = fma(dy[i], n, dgamma[i]);
            const Vec<VEC> less = LN ? fma(n, toward, off) : n * toward;
            store<T, VEC>(dz + i * apart, fma(dn, scale, less));
        }
    }
    // the block's row groups add their columns in turn
    __shared__ float all[2][MIN_THREADS * EPT / 2];   // two row groups at least: half of the block's columns
    float *pg = a.part_gamma + blockIdx.x * a.part_stride, *pb = a.part_beta + blockIdx.x * a.part_stride;
    for (int g = 0; g < groups; g++) {
        if (group == g)
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    const int c = c0 + i * apart + j;
                    if (!mine[i]) continue;
                    if (g) {
                        dgamma[i].set(j, dgamma[i][j] + all[0][c]);
                        dbeta[i].set(j, dbeta[i][j] + all[1][c]);
                    }
                    if (g == groups - 1) {
                        pg[c] = dgamma[i][j];
                        pb[c] = dbeta[i][j];
                    } else {
                        all[0][c] = dgamma[i][j];
                        all[1][c] = dbeta[i][j];
                    }
                }
        if (groups > 1) __syncthreads();
    }
}

// column c of the blocks' sums [n][2][C]: the JOIN_ROWS threads of a column take every JOIN_ROWS-th
// block, then their sums are added in order.  A programmatic launch: the kernel ahead gives no signal
// of its own, so this one starts when the last of its blocks has ended, without the gap that a stream
// leaves between two kernels otherwise.  Backward with and without it: 5,003 x 231 fp32 14.5 and 16.5 us,
// 100,000 x 200 bf16 64.6 and 66.8, 65,536 x 512 61.3 and 62.4.
constexpr int JOIN_COLS = 32, JOIN_ROWS = 32;
__global__ void __launch_bounds__(JOIN_COLS *JOIN_ROWS) join_blocks(const float *part, int n, int C, float *dgamma, float *dbeta) {
    __shared__ float sums[JOIN_ROWS][JOIN_COLS];
    const int c = blockIdx.x * JOIN_COLS + threadIdx.x;
    cudaGridDependencySynchronize();
    float s = 0.0f;
    if (c < 2 * C)
#pragma unroll 8
        for (int i = threadIdx.y; i < n; i += JOIN_ROWS) s += part[(long long)i * 2 * C + c];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y || c >= 2 * C) return;
#pragma unroll
    for (int i = 1; i < JOIN_ROWS; i++) s += sums[i][threadIdx.x];
    (c < C ? dgamma[c] : dbeta[c - C]) = s;
}

// The row's threads and the values of each, 8 or 16; the fewest threads that hold the row, and four
// at least.  A block has the rows that fill MIN_THREADS.
int values_per_thread(int C, int dtype, bool backward) {
    if (C <= 32 * 8) return 8;
    if (backward) return 16;
    return dtype == SPECTRE_F32 && C <= MAX_THREADS * 8 ? 8 : 16;
}
int threads_per_row(int C, int dtype, bool backward) {
    int tpr = 4;
    while (tpr * values_per_thread(C, dtype, backward) < C) tpr *= 2;
    return tpr;
}
int block_threads(int tpr) { return tpr > MIN_THREADS ? tpr : MIN_THREADS; }

// Blocks that run at once.
long long resident_blocks(const residual_norm_s *h, bool backward) {
    const bool eight = values_per_thread(h->C, h->dtype, backward) == 8;
    const int registers = backward ? (eight ? REGISTERS<8, true> : REGISTERS<16, true>) : (eight ? REGISTERS<8, false> : REGISTERS<16, false>);
    const int threads = block_threads(threads_per_row(h->C, h->dtype, backward)), n = 65536 / registers / threads;
    return (long long)h->nsm * (n > 0 ? n : 1);
}
long long backward_blocks(const residual_norm_s *h, long long T) {
    const int tpr = threads_per_row(h->C, h->dtype, true), groups = block_threads(tpr) / tpr;
    const long long need = (T + groups - 1) / groups, most = resident_blocks(h, true);
    return need < most ? need : most;
}

// An SM's shared memory for the blocks on it, and what a block needs beside its rings.
constexpr int SM_SHARED_BYTES = 227 * 1024, BLOCK_SHARED_BYTES = 20 * 1024;

template <typename T, int VEC, int EPT, bool RING, bool FULL, bool LN, bool POST>
cudaError_t launch_backward(const Args &a, int grid, cudaStream_t s) {
    const int threads = block_threads(a.tpr), bytes = RING ? threads / a.tpr * a.stages * a.stage_bytes : 0;
    const auto kernel = norm_backward<T, VEC, EPT, RING, FULL, LN, POST>;
    if (RING) {
        // the same for every width: threads with other plans set it at the same time
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM_SHARED_BYTES - BLOCK_SHARED_BYTES);
        if (e != cudaSuccess) return e;
    }
    kernel<<<grid, threads, bytes, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int VEC, int EPT, bool LN, bool POST>
cudaError_t launch_rows(const Args &a, bool backward, int grid, cudaStream_t s) {
    const bool full = VEC > 1 && a.C == a.tpr * EPT;
    if (!backward) {
        if constexpr (VEC > 1)
            if (full) {
                norm_forward<T, VEC, EPT, true, LN, POST><<<grid, block_threads(a.tpr), 0, s>>>(a);
                return cudaGetLastError();
            }
        norm_forward<T, VEC, EPT, false, LN, POST><<<grid, block_threads(a.tpr), 0, s>>>(a);
        return cudaGetLastError();
    }
    if constexpr (VEC > 1)
        if (a.stages)
            return full ? launch_backward<T, VEC, EPT, true, true, LN, POST>(a, grid, s) : launch_backward<T, VEC, EPT, true, false, LN, POST>(a, grid, s);
    // bf16 rows of more than 256 values always have a ring: theirs are 3 * 2 * C bytes a stage at most
    if constexpr (VEC == 8 && EPT == 16) return cudaErrorInvalidConfiguration;
    else return launch_backward<T, VEC, EPT, false, false, LN, POST>(a, grid, s);
}

template <typename T, int VEC, bool LN, bool POST> cudaError_t launch(const Args &a, bool backward, int grid, cudaStream_t s) {
    const bool eight = values_per_thread(a.C, sizeof(T) == 4 ? SPECTRE_F32 : SPECTRE_BF16, backward) == 8;
    return eight ? launch_rows<T, VEC, 8, LN, POST>(a, backward, grid, s) : launch_rows<T, VEC, 16, LN, POST>(a, backward, grid, s);
}

template <typename T, int VEC> cudaError_t launch_norm(int norm, const Args &a, bool backward, int grid, cudaStream_t s) {
    switch (norm) {
    case SPECTRE_NORM_POST_LN: return launch<T, VEC, true, true>(a, backward, grid, s);
    case SPECTRE_NORM_PRE_LN: return launch<T, VEC, true, false>(a, backward, grid, s);
    case SPECTRE_NORM_POST_RMS: return launch<T, VEC, false, true>(a, backward, grid, s);
    default: return launch<T, VEC, false, false>(a, backward, grid, s);
    }
}

bool wide(const void *p, long long stride, size_t es) { return aligned(p, 16) && (stride * es) % 16 == 0; }

int enqueue(const residual_norm_s *h, Args &a, bool backward, int grid, cudaStream_t s) {
    const size_t es = h->dtype == SPECTRE_F32 ? 4 : 2;
    const bool vec = (h->C * es) % 16 == 0 && wide(a.out, a.outs, es) && wide(a.x, a.xs, es) && wide(a.y, a.ys, es) &&
                     wide(a.dy, a.dys, es) && aligned(a.gamma, 16) && aligned(a.beta, 16);
    // The backward pass's rings: rows of a warp or more, each stage one row of every input; four stages
    // where they fit.  Loads instead of rings: 65,536 x 512 bf16 69 against 61 us, 49,152 x 2,048 221
    // against 192.  Going forward it is the other way: 33 against 39 us and 112 against 125, for a
    // thread has registers left for the next row and needs no barrier to take it.
    a.polls = h->test_wait ? 0 : COPY_POLLS;
    a.stages = 0;
    if (backward && vec && a.tpr >= 32) {
        const int inputs = a.x ? 3 : 2, rings = block_threads(a.tpr) / a.tpr;
        a.stage_bytes = inputs * a.C * (int)es;
        const int blocks = (int)(resident_blocks(h, backward) / h->nsm), room = (SM_SHARED_BYTES / blocks - BLOCK_SHARED_BYTES) / rings / a.stage_bytes;
        a.stages = room < MAX_STAGES ? room : MAX_STAGES;
        if (a.stages < 2) a.stages = 0;
    }
    cudaError_t e;
    if (h->dtype == SPECTRE_F32)
        e = vec ? launch_norm<float, 4>(h->norm, a, backward, grid, s) : launch_norm<float, 1>(h->norm, a, backward, grid, s);
    else
        e = vec ? launch_norm<__nv_bfloat16, 8>(h->norm, a, backward, grid, s) : launch_norm<__nv_bfloat16, 1>(h->norm, a, backward, grid, s);
    return status_of(e);
}

size_t partial_bytes(const residual_norm_s *h, long long T) {
    const long long n = backward_blocks(h, T);
    return n > 1 ? (size_t)n * 2 * h->C * sizeof(float) : 0;
}

}  // namespace resnorm

extern "C" {

int residual_norm_create(residual_norm_t *out, int C, int dtype, int norm, float eps) {
    if (!out) return SPECTRE_ERR_ARG;
    *out = nullptr;
    if (C < 1 || C > resnorm::MAX_C || (dtype != SPECTRE_F32 && dtype != SPECTRE_BF16)) return SPECTRE_ERR_ARG;
    if (norm < SPECTRE_NORM_POST_LN || norm > SPECTRE_NORM_PRE_RMS) return SPECTRE_ERR_ARG;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return SPECTRE_ERR_ARG;
    int dev = -1, nsm = 0;
    const int st = rows_io::usable_device(&dev, &nsm);
    if (st != SPECTRE_OK) return st;
    residual_norm_s *h = new (std::nothrow) residual_norm_s{C, dtype, norm, eps, dev, nsm, 0};
    if (!h) return SPECTRE_ERR_NOMEM;
    *out = h;
    return SPECTRE_OK;
}

int residual_norm_run(residual_norm_t h, long long T, const void *out, long long out_stride, const void *x,
                      long long x_stride, const float *gamma, const float *beta, void *y, long long y_stride,
                      void *stream) {
    using namespace resnorm;
    if (!h || T < 0) return SPECTRE_ERR_ARG;
    if (T == 0) return SPECTRE_OK;
    if (!out || !x || !gamma || !beta || !y || out_stride < 0 || x_stride < 0 || (T > 1 && y_stride < h->C))
        return SPECTRE_ERR_ARG;
    const size_t es = h->dtype == SPECTRE_F32 ? 4 : 2;
    if (!aligned(out, es) || !aligned(x, es) || !aligned(y, es) || !aligned(gamma, 4) || !aligned(beta, 4))
        return SPECTRE_ERR_ALIGN;
    if (!current_device_is(h->device)) return SPECTRE_ERR_DEVICE;
    Args a{};
    a.T = T;
    a.C = h->C;
    a.tpr = threads_per_row(h->C, h->dtype, false);
    a.eps = h->eps;
    a.out = out;
    a.outs = out_stride;
    a.x = x;
    a.xs = x_stride;
    a.y = y;
    a.ys = y_stride;
    a.gamma = gamma;
    a.beta = beta;
    const int groups = block_threads(a.tpr) / a.tpr;
    const long long need = (T + groups - 1) / groups, most = resident_blocks(h, false);
    return enqueue(h, a, false, (int)(need < most ? need : most), static_cast<cudaStream_t>(stream));
}

size_t residual_norm_workspace_bytes(residual_norm_t h, long long T) {
    return !h || T < 1 ? 0 : resnorm::partial_bytes(h, T);
}

int residual_norm_backward(residual_norm_t h, long long T, const void *dy, long long dy_stride, const void *out,
                           long long out_stride, const void *x, long long x_stride, const float *gamma, void *dz,
                           long long dz_stride, float *dgamma, float *dbeta, void *work, size_t work_bytes,
                           void *stream) {
    using namespace resnorm;
    if (!h || T < 0 || !dgamma || !dbeta) return SPECTRE_ERR_ARG;
    const bool post = h->norm == SPECTRE_NORM_POST_LN || h->norm == SPECTRE_NORM_POST_RMS;
    const size_t es = h->dtype == SPECTRE_F32 ? 4 : 2, need = T ? partial_bytes(h, T) : 0;
    if (T > 0) {
        if (!dy || !out || (post && !x) || !gamma || !dz || dy_stride < 0 || out_stride < 0 || x_stride < 0 ||
            (T > 1 && dz_stride < h->C))
            return SPECTRE_ERR_ARG;
        if (need && (!work || work_bytes < need)) return SPECTRE_ERR_ARG;
        if (!aligned(dy, es) || !aligned(out, es) || (post && !aligned(x, es)) || !aligned(dz, es) || !aligned(gamma, 4) ||
            (need && !aligned(work, 256)))
            return SPECTRE_ERR_ALIGN;
    }
    if (!aligned(dgamma, 4) || !aligned(dbeta, 4)) return SPECTRE_ERR_ALIGN;
    if (!current_device_is(h->device)) return SPECTRE_ERR_DEVICE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int n = (int)backward_blocks(h, T);
    float *part = static_cast<float *>(work);
    if (T > 0) {
        Args a{};
        a.T = T;
        a.C = h->C;
        a.tpr = threads_per_row(h->C, h->dtype, true);
        a.eps = h->eps;
        a.dy = dy;
        a.dys = dy_stride;
        a.out = out;
        a.outs = out_stride;
        a.x = post ? x : nullptr;
        a.xs = post ? x_stride : 0;
        a.y = dz;
        a.ys = dz_stride;
        a.gamma = gamma;
        // a single block's sums are the gradient
        a.part_gamma = n > 1 ? part : dgamma;
        a.part_beta = n > 1 ? part + h->C : dbeta;
        a.part_stride = 2LL * h->C;
        const int st = enqueue(h, a, true, n, s);
        if (st != SPECTRE_OK || n == 1) return st;
    }
    cudaLaunchConfig_t config{};
    config.gridDim = dim3((2 * h->C + JOIN_COLS - 1) / JOIN_COLS);
    config.blockDim = dim3(JOIN_COLS, JOIN_ROWS);
    config.stream = s;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    config.attrs = &early;
    config.numAttrs = T > 0 ? 1 : 0;
    return status_of(cudaLaunchKernelEx(&config, join_blocks, static_cast<const float *>(part), n, h->C, dgamma, dbeta));
}

int residual_norm_set_option(residual_norm_t h, int option, int value) {
    if (!h || option != RESIDUAL_NORM_OPT_TEST_WAIT_TIMEOUT || value < 0 || value > 1) return SPECTRE_ERR_ARG;
    h->test_wait = value;
    return SPECTRE_OK;
}

int residual_norm_device_status(residual_norm_t h, void *stream) {
    if (!h) return SPECTRE_ERR_ARG;
    if (!resnorm::current_device_is(h->device)) return SPECTRE_ERR_DEVICE;
    unsigned word = 0;
    const unsigned clear = 0;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&word, resnorm::wait_gave_up, sizeof word);
    if (e == cudaSuccess && word) e = cudaMemcpyToSymbol(resnorm::wait_gave_up, &clear, sizeof clear);
    return e == cudaSuccess && word ? SPECTRE_ERR_TIMEOUT : rows_io::status_of(e);
}

int residual_norm_destroy(residual_norm_t h) {
    delete h;
    return SPECTRE_OK;
}

}  // extern "C"
