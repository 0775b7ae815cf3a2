// Elementwise gated recurrence (include/gla.h, "elementwise gated recurrence"):
//     h_t = a_t h_{t-1} + w_t x_t,   a_t = e^{log a_t},   w_t = 1 or 1 - a_t.
// One state value per channel: the decay of the layer's gated memory (podcast.app episode page,
// summary: a gated memory updated once per token) without its key dimension.
//
// One thread walks one channel of one sequence.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gla_common.cuh"
#include "gla_gate.cuh"
#include "gla_internal.h"

namespace gla {
namespace {

constexpr int kThreads = 128;
constexpr int kSeg = 16;  // rows between the states kept for the backward

struct GateForm {
    bool preact, leak;
    float inv_tau;
};

// a_t and w_t from the gate argument
__device__ __forceinline__ void gate_of(const GateForm& f, float g, float& a, float& w) {
    const float la = f.preact ? logsigmoid_f(g) * f.inv_tau : g;
    a = expf(la);
    w = f.leak ? -expm1f(la) : 1.f;
}

// Rows [lo, hi) of sequence n and the offset of its row 0 of channel tile ch
struct Span {
    int64_t lo, hi, row0, seq;
};
__device__ __forceinline__ Span span_of(const ScanProblem& p, const int32_t* cu, int64_t n, int64_t head) {
    if (!cu) return Span{0, p.L, (n * p.H + head) * p.L, n * p.H + head};
    int64_t lo = cu[n], hi = cu[n + 1];
    lo = lo < 0 ? 0 : lo;
    hi = hi > p.L ? p.L : hi;
    return Span{lo, hi, head * p.L, n * p.H + head};
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_scan_fwd(ScanProblem p, GateForm f, const T* __restrict__ x,
                                                       const float* __restrict__ la, const int32_t* __restrict__ cu,
                                                       const float* __restrict__ h0, T* __restrict__ h,
                                                       float* __restrict__ hT, float* __restrict__ seg) {
    const int64_t tiles = cdiv(p.D, kThreads);
    const int64_t c = (blockIdx.x % tiles) * kThreads + threadIdx.x, nh = blockIdx.x / tiles;
    if (c >= p.D) return;
    const Span sp = span_of(p, cu, nh / p.H, nh % p.H);
    const int64_t nseg = cdiv(p.L, kSeg);
    float y = h0 ? h0[sp.seq * p.D + c] : 0.f;
    for (int64_t t = sp.lo; t < sp.hi; ++t) {
        const int64_t i = (sp.row0 + t) * p.D + c;
        if (seg && t % kSeg == 0) seg[((sp.row0 / p.L) * nseg + t / kSeg) * p.D + c] = y;
        float a, w;
        gate_of(f, la[i], a, w);
        y = fmaf(a, y, w * ldf(x + i));
        if (h) stf(h + i, y);
    }
    if (hT) hT[sp.seq * p.D + c] = y;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_scan_bwd(ScanProblem p, GateForm f, const T* __restrict__ x,
                                                       const float* __restrict__ la, const int32_t* __restrict__ cu,
                                                       const float* __restrict__ h0, const T* __restrict__ dh,
                                                       const float* __restrict__ dhT, T* __restrict__ dx,
                                                       float* __restrict__ dla, float* __restrict__ dh0,
                                                       const float* __restrict__ seg) {
    const int64_t tiles = cdiv(p.D, kThreads);
    const int64_t c = (blockIdx.x % tiles) * kThreads + threadIdx.x, nh = blockIdx.x / tiles;
    if (c >= p.D) return;
    const Span sp = span_of(p, cu, nh / p.H, nh % p.H);
    const int64_t nseg = cdiv(p.L, kSeg);
    float y = dhT ? dhT[sp.seq * p.D + c] : 0.f;
    for (int64_t end = sp.hi; end > sp.lo;) {
        int64_t t0 = (end - 1) / kSeg * kSeg;
        float hp[kSeg];  // state before each row of the segment
        float s;
        if (t0 > sp.lo) s = seg[((sp.row0 / p.L) * nseg + t0 / kSeg) * p.D + c];
        else {
            t0 = sp.lo;
            s = h0 ? h0[sp.seq * p.D + c] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kSeg; ++j) {
            hp[j] = s;
            if (t0 + j < end) {
                const int64_t i = (sp.row0 + t0 + j) * p.D + c;
                float a, w;
                gate_of(f, la[i], a, w);
                s = fmaf(a, s, w * ldf(x + i));
            }
        }
#pragma unroll
        for (int j = kSeg - 1; j >= 0; --j) {
            if (t0 + j < end) {
                const int64_t i = (sp.row0 + t0 + j) * p.D + c;
                float a, w;
                const float z = la[i], xv = ldf(x + i);
                gate_of(f, z, a, w);
                const float g = ldf(dh + i) + y;
                y = a * g;
                float d = y * (f.leak ? hp[j] - xv : hp[j]);
                if (f.preact) d *= sigmoid_neg_f(z) * f.inv_tau;
                dla[i] = d;
                stf(dx + i, w * g);
            }
        }
        end = t0;
    }
    if (dh0) dh0[sp.seq * p.D + c] = y;
}

// Whether an earlier row of the call names the same slot (every thread of the block gets the answer).
__device__ __forceinline__ bool named_before(const int32_t* slots, int64_t b, int32_t slot) {
    int dup = 0;
    for (int64_t i = threadIdx.x; i < b; i += blockDim.x) dup |= slots[i] == slot;
    return __syncthreads_or(dup) != 0;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_scan_step(ScanProblem p, GateForm f, const T* __restrict__ x,
                                                        const float* __restrict__ la,
                                                        const int32_t* __restrict__ slots, int64_t pool,
                                                        float* __restrict__ state, T* __restrict__ h, int* err) {
    const int64_t b = blockIdx.y, n = p.H * p.D;
    int64_t slot = b;
    bool live = true;
    if (slots) {
        const int32_t sl = slots[b];
        slot = sl;
        live = sl >= 0;
        if (live && (sl >= pool || named_before(slots, b, sl))) {  // sl is the same in the whole block
            live = false;
            if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(err, kErrBadRow);
        }
    }
    const int64_t c = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    if (c >= n) return;
    float y = 0.f;
    if (live) {
        float a, w;
        gate_of(f, la[b * n + c], a, w);
        y = fmaf(a, state[slot * n + c], w * ldf(x + b * n + c));
        state[slot * n + c] = y;
    }
    stf(h + b * n + c, y);
}

GateForm form(const ScanProblem& p) { return GateForm{p.preact, p.leak, p.inv_tau}; }

template <typename T>
gla_status fwd_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                     void* h, float* hT, float* seg, cudaStream_t s) {
    const unsigned grid = unsigned(p.B * p.H * cdiv(p.D, kThreads));
    GLA_LAUNCH("scan_fwd", k_scan_fwd<T>, grid, kThreads, 0, s, p, form(p), static_cast<const T*>(x), la, cu, h0,
               static_cast<T*>(h), hT, seg);
    return GLA_OK;
}

template <typename T>
gla_status bwd_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                     const void* dh, const float* dhT, void* dx, float* dla, float* dh0, const float* seg,
                     cudaStream_t s) {
    const unsigned grid = unsigned(p.B * p.H * cdiv(p.D, kThreads));
    GLA_LAUNCH("scan_bwd", k_scan_bwd<T>, grid, kThreads, 0, s, p, form(p), static_cast<const T*>(x), la, cu, h0,
               static_cast<const T*>(dh), dhT, static_cast<T*>(dx), dla, dh0, seg);
    return GLA_OK;
}

template <typename T>
gla_status step_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* slots, int64_t pool,
                      float* state, void* h, cudaStream_t s) {
    const dim3 grid(unsigned(cdiv(p.H * p.D, kThreads)), unsigned(p.B));
    GLA_LAUNCH("scan_step", k_scan_step<T>, grid, kThreads, 0, s, p, form(p), static_cast<const T*>(x), la, slots,
               pool, state, static_cast<T*>(h), device_error_word());
    return GLA_OK;
}

}  // namespace

size_t scan_workspace(const ScanProblem& p, Arena& a) {
    (void)a.take<float>(size_t((p.packed ? p.H : p.B * p.H) * cdiv(p.L, kSeg) * p.D));
    return a.used;
}

gla_status scan_fwd(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0, void* h,
                    float* hT, float* seg, cudaStream_t s) {
    return p.bf16 ? fwd_typed<__nv_bfloat16>(p, x, la, cu, h0, h, hT, seg, s)
                  : fwd_typed<float>(p, x, la, cu, h0, h, hT, seg, s);
}

gla_status scan_bwd(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                    const void* dh, const float* dhT, void* dx, float* dla, float* dh0, float* seg, bool reuse,
                    cudaStream_t s) {
    if (!reuse) {
        const gla_status st = scan_fwd(p, x, la, cu, h0, nullptr, nullptr, seg, s);
        if (st != GLA_OK) return st;
    }
    return p.bf16 ? bwd_typed<__nv_bfloat16>(p, x, la, cu, h0, dh, dhT, dx, dla, dh0, seg, s)
                  : bwd_typed<float>(p, x, la, cu, h0, dh, dhT, dx, dla, dh0, seg, s);
}

gla_status scan_step(const ScanProblem& p, const void* x, const float* la, const int32_t* slots, int64_t pool,
                     float* state, void* h, cudaStream_t s) {
    return p.bf16 ? step_typed<__nv_bfloat16>(p, x, la, slots, pool, state, h, s)
                  : step_typed<float>(p, x, la, slots, pool, state, h, s);
}

}  // namespace gla
