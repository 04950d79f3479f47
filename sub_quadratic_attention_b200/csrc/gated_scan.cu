// gated_scan.cu -- the gated linear recurrence h_t = a_t h_{t-1} + b_t over sequences of
// rows, its backward pass and its single-token step, and their C ABI (gated_scan.h).
//
// One thread walks one channel of one sequence, row after row.
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

// a = s(g) and c = 1 - a = s(-g), each to its own relative precision: e = exp(-|g|) never
// overflows, and the smaller of the two is e / (1 + e) instead of a difference.
template <int FORM> __device__ __forceinline__ Gate gate_of(float g) {
    if (FORM == GATED_SCAN_EXP) return {expf(g), 1.0f};
    const float e = expf(-fabsf(g)), r = 1.0f / (1.0f + e), s = e * r;
    return g >= 0.0f ? Gate{r, s} : Gate{s, r};
}

// a * h where a factor of zero takes h out, NaN and infinities included
__device__ __forceinline__ float mul0(float a, float h) { return a == 0.0f ? 0.0f : a * h; }
__device__ __forceinline__ float fma0(float a, float h, float b) { return a == 0.0f ? b : fmaf(a, h, b); }

template <int FORM> __device__ __forceinline__ float input_of(Gate k, float v) {
    return FORM == GATED_SCAN_EXP ? v : mul0(k.c, v);
}

struct Args {
    gated_scan_args a;
    int H, D, C, per;
    long long nchunk, nseq;   // dense: nseq = B
};

__device__ __forceinline__ void span_of(const Args &p, long long n, long long &b, long long &lo, long long &hi) {
    if (!p.a.cu_seqlens) {
        b = n;
        lo = 0;
        hi = p.a.L;
        return;
    }
    b = 0;
    lo = p.a.cu_seqlens[n];
    hi = p.a.cu_seqlens[n + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.a.L ? p.a.L : hi;
}

template <typename T> __device__ __forceinline__ T *row(const gated_scan_rows &r, long long b, long long t) {
    return static_cast<T *>(r.data) + b * r.batch_stride + t * r.row_stride;
}

template <typename TV, typename TG, int FORM>
__global__ void scan_forward(Args p) {
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (i >= p.nseq * p.C) return;
    const int c = (int)(i % p.C), gc = p.per == GATED_SCAN_PER_HEAD ? c / p.D : c;
    const long long n = i / p.C;
    long long b, lo, hi;
    span_of(p, n, b, lo, hi);
    float h = p.a.h0 ? p.a.h0[n * p.C + c] : 0.0f;
    for (long long t = lo; t < hi; t++) {
        if (p.a.states && t % CHUNK == 0) p.a.states[(b * p.nchunk + t / CHUNK) * p.C + c] = h;
        const Gate k = gate_of<FORM>(to_f(row<TG>(p.a.g, b, t)[gc]));
        h = fma0(k.a, h, input_of<FORM>(k, to_f(row<TV>(p.a.v, b, t)[c])));
        row<TV>(p.a.y, b, t)[c] = from_f<TV>(h);
    }
    if (p.a.hT) p.a.hT[n * p.C + c] = h;
}

template <typename TV, typename TG, int FORM>
__global__ void scan_backward(Args p, float *part) {
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (i >= p.nseq * p.C) return;
    const int c = (int)(i % p.C), gc = p.per == GATED_SCAN_PER_HEAD ? c / p.D : c;
    const long long n = i / p.C;
    long long b, lo, hi;
    span_of(p, n, b, lo, hi);
    float carry = p.a.dhT ? p.a.dhT[n * p.C + c] : 0.0f;
    float before[CHUNK];
    for (long long end = hi; end > lo;) {
        long long beg = (end - 1) / CHUNK * CHUNK;
        float h = p.a.states[(b * p.nchunk + beg / CHUNK) * p.C + c];
        if (beg <= lo) {
            beg = lo;
            h = p.a.h0 ? p.a.h0[n * p.C + c] : 0.0f;
        }
        for (long long t = beg; t < end; t++) {
            before[t - beg] = h;
            const Gate k = gate_of<FORM>(to_f(row<TG>(p.a.g, b, t)[gc]));
            h = fma0(k.a, h, input_of<FORM>(k, to_f(row<TV>(p.a.v, b, t)[c])));
        }
        for (long long t = end - 1; t >= beg; t--) {
            const Gate k = gate_of<FORM>(to_f(row<TG>(p.a.g, b, t)[gc]));
            const float v = to_f(row<TV>(p.a.v, b, t)[c]);
            const float dh = to_f(row<TV>(p.a.dy, b, t)[c]) + carry;
            carry = mul0(k.a, dh);
            const float slope = FORM == GATED_SCAN_EXP ? mul0(k.a, before[t - beg])
                                                       : mul0(k.a * k.c, before[t - beg] - v);
            const float dg = slope * dh;
            row<TV>(p.a.dv, b, t)[c] = from_f<TV>(FORM == GATED_SCAN_EXP ? dh : mul0(k.c, dh));
            if (p.per == GATED_SCAN_PER_HEAD)
                part[(b * p.a.L + t) * p.C + c] = dg;
            else
                row<TG>(p.a.dg, b, t)[c] = from_f<TG>(dg);
        }
        end = beg;
    }
    if (p.a.dh0) p.a.dh0[n * p.C + c] = carry;
}

// the head's gate gradient: the sum of its channels' parts
template <typename TG> __global__ void sum_heads(Args p, const float *part) {
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (i >= p.a.B * p.a.L * p.H) return;
    const int h = (int)(i % p.H);
    const long long r = i / p.H, b = r / p.a.L, t = r % p.a.L;
    if (p.a.cu_seqlens && (t < p.a.cu_seqlens[0] || t >= p.a.cu_seqlens[p.nseq])) return;
    float s = 0.0f;
    for (int d = 0; d < p.D; d++) s += part[r * p.C + h * p.D + d];
    row<TG>(p.a.dg, b, t)[h] = from_f<TG>(s);
}

template <typename T> __global__ void zero_rows(Args p, gated_scan_rows r, int width) {
    const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
    if (i >= p.a.L * width) return;
    const long long t = i / width;
    if (t < p.a.cu_seqlens[0] || t >= p.a.cu_seqlens[p.nseq]) row<T>(r, 0, t)[i % width] = from_f<T>(0.0f);
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
        const Gate k = gate_of<FORM>(to_f(g[i * gs + gc]));
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

size_t workspace(const gated_scan_s *h, long long B, long long L, int backward) {
    return backward && h->per == GATED_SCAN_PER_HEAD ? (size_t)B * L * h->C * sizeof(float) : 0;
}

int blocks(long long n, int per) { return (int)((n + per - 1) / per); }

template <typename TV, typename TG, int FORM> cudaError_t launch(const Args &p, bool backward, cudaStream_t s) {
    const int grid = blocks(p.nseq * p.C, 128);
    if (!backward) {
        if (grid) scan_forward<TV, TG, FORM><<<grid, 128, 0, s>>>(p);
        if (p.a.cu_seqlens && p.a.zero_outside && p.a.L) zero_rows<TV><<<blocks(p.a.L * p.C, 256), 256, 0, s>>>(p, p.a.y, p.C);
    } else {
        float *part = static_cast<float *>(p.a.work);
        if (grid) scan_backward<TV, TG, FORM><<<grid, 128, 0, s>>>(p, part);
        if (p.per == GATED_SCAN_PER_HEAD && p.a.L) sum_heads<TG><<<blocks(p.a.B * p.a.L * p.H, 128), 128, 0, s>>>(p, part);
        if (p.a.cu_seqlens && p.a.zero_outside && p.a.L) {
            const int gw = p.per == GATED_SCAN_PER_HEAD ? p.H : p.C;
            zero_rows<TV><<<blocks(p.a.L * p.C, 256), 256, 0, s>>>(p, p.a.dv, p.C);
            zero_rows<TG><<<blocks(p.a.L * gw, 256), 256, 0, s>>>(p, p.a.dg, gw);
        }
    }
    return cudaGetLastError();
}

template <int FORM> cudaError_t launch_types(const gated_scan_s *h, const Args &p, bool backward, cudaStream_t s) {
    if (h->dtype == SPECTRE_F32) return launch<float, float, FORM>(p, backward, s);
    if (h->gate_dtype == SPECTRE_F32) return launch<__nv_bfloat16, float, FORM>(p, backward, s);
    return launch<__nv_bfloat16, __nv_bfloat16, FORM>(p, backward, s);
}

int run(gated_scan_s *h, const gated_scan_args *a, bool backward, void *stream) {
    if (!h || !a || a->B < 0 || a->L < 0) return SPECTRE_ERR_ARG;
    const bool packed = a->cu_seqlens != nullptr;
    if (packed && (a->B != 1 || a->nseq < 0 || a->L > 0x7fffffffLL)) return SPECTRE_ERR_ARG;
    const long long nseq = packed ? a->nseq : a->B;
    if (a->B == 0 || (packed && nseq == 0 && !a->zero_outside)) return SPECTRE_OK;
    const int gw = h->per == GATED_SCAN_PER_HEAD ? h->H : h->C;
    // every count that the kernels index by stays well inside 63 bits, and the grid inside 31
    const long long nchunk = (a->L + CHUNK - 1) / CHUNK;
    if (nchunk > (1LL << 31) / a->B || nchunk * a->B > (1LL << 40) / h->C || nseq > (1LL << 40) / h->C) return SPECTRE_ERR_ARG;
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
    Args p{*a, h->H, h->D, h->C, h->per, nchunk, nseq};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return status_of(h->gate == GATED_SCAN_EXP ? launch_types<GATED_SCAN_EXP>(h, p, backward, s)
                                               : launch_types<GATED_SCAN_SIGMOID>(h, p, backward, s));
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
    return !h || B < 1 || L < 1 ? 0 : gscan::workspace(h, B, L, backward);
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
