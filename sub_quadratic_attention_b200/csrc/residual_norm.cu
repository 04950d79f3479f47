// residual_norm.cu -- y = N(out + x) or N(out) + x over rows of C values, N LayerNorm or
// RMSNorm, its backward pass, and their C ABI (residual_norm.h).
//
// TPR threads (a power of two) hold one row in registers, at most 16 values a thread, so a
// row is read once: the sums of a row are shuffles within a warp and, for rows wider than a
// warp's share, one exchange of the warps' sums through shared memory.  The variance is
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

struct residual_norm_s {
    int C, dtype, norm;
    float eps;
    int device, nsm;
};

namespace resnorm {

using namespace rows_io;

constexpr int MAX_C = 8192;
constexpr int EPT = 16;                    // values of a row that a thread holds
constexpr int MAX_THREADS = MAX_C / EPT;   // 512
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
};

// VEC neighbouring values: one 16-byte access where VEC values are 16 bytes, else one value
template <typename T, int VEC> struct Pack {
    T v[VEC];
};
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> load(const T *p) {
    Pack<T, VEC> r;
    if constexpr (sizeof(T) * VEC == 16)
        *reinterpret_cast<uint4 *>(r.v) = *reinterpret_cast<const uint4 *>(p);
    else
        r.v[0] = *p;
    return r;
}
template <typename T, int VEC> __device__ __forceinline__ void store(T *p, const float *f) {
    Pack<T, VEC> r;
#pragma unroll
    for (int j = 0; j < VEC; j++) r.v[j] = from_f<T>(f[j]);
    if constexpr (sizeof(T) * VEC == 16)
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(r.v);
    else
        *p = r.v[0];
}

// K sums over the row's threads, in every one of them; the same order for every row
template <int K> __device__ __forceinline__ void row_sums(float (&s)[K], int tpr, int &turn) {
    __shared__ float warp_sums[2][K][MAX_THREADS / 32];
    for (int o = min(tpr, 32) >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; k++) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
    if (tpr <= 32) return;
    // two buffers in turn: a warp writes a buffer again only after the barrier that follows
    // every warp's reads of it
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; k++) warp_sums[turn][k][threadIdx.x >> 5] = s[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; k++) s[k] = 0.0f;
    const int first = threadIdx.x / tpr * (tpr / 32);   // the row's first warp
    for (int w = first; w < first + tpr / 32; w++)
#pragma unroll
        for (int k = 0; k < K; k++) s[k] += warp_sums[turn][k][w];
    turn ^= 1;
}

template <typename T, int VEC, bool LN, bool POST>
__global__ void __launch_bounds__(MAX_THREADS) norm_forward(Args a) {
    constexpr int NV = EPT / VEC;
    const int lane = threadIdx.x % a.tpr, group = threadIdx.x / a.tpr, groups = blockDim.x / a.tpr;
    const float inv = 1.0f / (float)a.C;
    int turn = 0;
    for (long long r0 = blockIdx.x * (long long)groups; r0 < a.T; r0 += (long long)gridDim.x * groups) {
        const long long r = r0 + group;
        const bool live = r < a.T;
        float z[EPT], xr[POST ? 1 : EPT];
        float s1[1] = {0.0f}, s2[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * a.tpr + lane) * VEC;
            const bool in = live && c < a.C;
            Pack<T, VEC> o, x;
            if (in) {
                o = load<T, VEC>(static_cast<const T *>(a.out) + r * a.outs + c);
                x = load<T, VEC>(static_cast<const T *>(a.x) + r * a.xs + c);
            }
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                const float fo = in ? to_f(o.v[j]) : 0.0f, fx = in ? to_f(x.v[j]) : 0.0f;
                z[i * VEC + j] = POST ? fo + fx : fo;
                if constexpr (!POST) xr[i * VEC + j] = fx;
                s1[0] += z[i * VEC + j];
            }
        }
        float mean = 0.0f;
        if (LN) {
            row_sums(s1, a.tpr, turn);
            mean = s1[0] * inv;
        }
#pragma unroll
        for (int i = 0; i < NV; i++)
            if ((i * a.tpr + lane) * VEC < a.C)
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    z[i * VEC + j] -= mean;
                    s2[0] = fmaf(z[i * VEC + j], z[i * VEC + j], s2[0]);
                }
        row_sums(s2, a.tpr, turn);
        const float rstd = 1.0f / sqrtf(s2[0] * inv + a.eps);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * a.tpr + lane) * VEC;
            if (!live || c >= a.C) continue;
            float f[VEC];
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                f[j] = fmaf(z[i * VEC + j] * rstd, a.gamma[c + j], a.beta[c + j]);
                if constexpr (!POST) f[j] += xr[i * VEC + j];
            }
            store<T, VEC>(static_cast<T *>(a.y) + r * a.ys + c, f);
        }
    }
}

template <typename T, int VEC, bool LN, bool POST>
__global__ void __launch_bounds__(MAX_THREADS) norm_backward(Args a) {
    constexpr int NV = EPT / VEC;
    const int lane = threadIdx.x % a.tpr, group = threadIdx.x / a.tpr, groups = blockDim.x / a.tpr;
    const float inv = 1.0f / (float)a.C;
    int turn = 0;
    float dgamma[EPT], dbeta[EPT];
#pragma unroll
    for (int i = 0; i < EPT; i++) dgamma[i] = dbeta[i] = 0.0f;
    for (long long r0 = blockIdx.x * (long long)groups; r0 < a.T; r0 += (long long)gridDim.x * groups) {
        const long long r = r0 + group;
        const bool live = r < a.T;
        float z[EPT], dy[EPT];
        float s1[1] = {0.0f}, s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * a.tpr + lane) * VEC;
            const bool in = live && c < a.C;
            Pack<T, VEC> o, x, d;
            if (in) {
                o = load<T, VEC>(static_cast<const T *>(a.out) + r * a.outs + c);
                if constexpr (POST) x = load<T, VEC>(static_cast<const T *>(a.x) + r * a.xs + c);
                d = load<T, VEC>(static_cast<const T *>(a.dy) + r * a.dys + c);
            }
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                const int e = i * VEC + j;
                z[e] = in ? to_f(o.v[j]) : 0.0f;
                if constexpr (POST) z[e] += in ? to_f(x.v[j]) : 0.0f;
                dy[e] = in ? to_f(d.v[j]) : 0.0f;
                s1[0] += z[e];
            }
        }
        float mean = 0.0f;
        if (LN) {
            row_sums(s1, a.tpr, turn);
            mean = s1[0] * inv;
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * a.tpr + lane) * VEC;
            if (c >= a.C) continue;
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                const int e = i * VEC + j;
                const float dn = dy[e] * a.gamma[c + j];
                z[e] -= mean;
                s[0] = fmaf(z[e], z[e], s[0]);
                s[1] = fmaf(dn, z[e], s[1]);
                s[2] += dn;
            }
        }
        row_sums(s, a.tpr, turn);
        const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
        const float along = s[1] * rstd * inv, level = LN ? s[2] * inv : 0.0f;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * a.tpr + lane) * VEC;
            if (!live || c >= a.C) continue;
            float f[VEC];
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                const int e = i * VEC + j;
                const float n = z[e] * rstd;
                dgamma[e] = fmaf(dy[e], n, dgamma[e]);
                dbeta[e] += dy[e];
                f[j] = rstd * (fmaf(-n, along, dy[e] * a.gamma[c + j]) - level);
            }
            store<T, VEC>(static_cast<T *>(a.y) + r * a.ys + c, f);
        }
    }
    // the block's row groups add their columns in turn
    __shared__ float sums[2][MIN_THREADS * EPT / 2];
    float *pg = a.part_gamma + blockIdx.x * a.part_stride, *pb = a.part_beta + blockIdx.x * a.part_stride;
    for (int g = 0; g < groups; g++) {
        if (group == g)
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    const int c = (i * a.tpr + lane) * VEC + j, e = i * VEC + j;
                    if (c >= a.C) continue;
                    if (g) {
                        dgamma[e] += sums[0][c];
                        dbeta[e] += sums[1][c];
                    }
                    if (g == groups - 1) {
                        pg[c] = dgamma[e];
                        pb[c] = dbeta[e];
                    } else {
                        sums[0][c] = dgamma[e];
                        sums[1][c] = dbeta[e];
                    }
                }
        if (groups > 1) __syncthreads();
    }
}

// column c of the blocks' sums [n][2][C]: the 16 threads of a column take every 16th block
constexpr int JOIN_COLS = 32, JOIN_ROWS = 16;
__global__ void __launch_bounds__(JOIN_COLS *JOIN_ROWS) join_blocks(const float *part, int n, int C, float *dgamma, float *dbeta) {
    __shared__ float sums[JOIN_ROWS][JOIN_COLS];
    const int c = blockIdx.x * JOIN_COLS + threadIdx.x;
    float s = 0.0f;
    if (c < 2 * C)
        for (int i = threadIdx.y; i < n; i += JOIN_ROWS) s += part[(long long)i * 2 * C + c];
    sums[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y || c >= 2 * C) return;
    for (int i = 1; i < JOIN_ROWS; i++) s += sums[i][threadIdx.x];
    (c < C ? dgamma[c] : dbeta[c - C]) = s;
}

// The row's threads: the fewest that hold it with EPT values each, and four at least; a block
// has the rows that fill MIN_THREADS.
int threads_per_row(int C) {
    int tpr = 4;
    while (tpr * EPT < C) tpr *= 2;
    return tpr;
}
int block_threads(int tpr) { return tpr > MIN_THREADS ? tpr : MIN_THREADS; }

constexpr int BLOCKS_PER_SM = 2;
long long backward_blocks(const residual_norm_s *h, long long T) {
    const int tpr = threads_per_row(h->C), groups = block_threads(tpr) / tpr;
    const long long need = (T + groups - 1) / groups, most = (long long)h->nsm * BLOCKS_PER_SM;
    return need < most ? need : most;
}

template <typename T, int VEC, bool LN, bool POST> void launch(const Args &a, bool backward, int grid, cudaStream_t s) {
    if (backward)
        norm_backward<T, VEC, LN, POST><<<grid, block_threads(a.tpr), 0, s>>>(a);
    else
        norm_forward<T, VEC, LN, POST><<<grid, block_threads(a.tpr), 0, s>>>(a);
}

template <typename T, int VEC> void launch_norm(int norm, const Args &a, bool backward, int grid, cudaStream_t s) {
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
                     wide(a.dy, a.dys, es);
    if (h->dtype == SPECTRE_F32)
        vec ? launch_norm<float, 4>(h->norm, a, backward, grid, s) : launch_norm<float, 1>(h->norm, a, backward, grid, s);
    else
        vec ? launch_norm<__nv_bfloat16, 8>(h->norm, a, backward, grid, s)
            : launch_norm<__nv_bfloat16, 1>(h->norm, a, backward, grid, s);
    return status_of(cudaGetLastError());
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
    residual_norm_s *h = new (std::nothrow) residual_norm_s{C, dtype, norm, eps, dev, nsm};
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
    a.tpr = threads_per_row(h->C);
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
    const long long need = (T + groups - 1) / groups, most = (long long)h->nsm * 8;
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
        a.tpr = threads_per_row(h->C);
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
    join_blocks<<<(2 * h->C + JOIN_COLS - 1) / JOIN_COLS, dim3(JOIN_COLS, JOIN_ROWS), 0, s>>>(part, n, h->C, dgamma, dbeta);
    return status_of(cudaGetLastError());
}

int residual_norm_destroy(residual_norm_t h) {
    delete h;
    return SPECTRE_OK;
}

}  // extern "C"
