// Elementwise gated recurrence (include/gla.h, "elementwise gated recurrence"):
//     h_t = a_t h_{t-1} + w_t x_t,   a_t = e^{log a_t},   w_t = 1 or 1 - a_t.
// One state value per channel: the decay of the layer's gated memory (podcast.app episode page,
// summary: a gated memory updated once per token) without its key dimension.
//
// A step is the affine map s -> a s + b, and maps compose: (a2, b2) o (a1, b1) = (a1 a2, a2 b1 + b2). So a
// sequence is cut into segments that are reduced to one map each, the maps are joined, and every segment
// then runs its steps from the state that enters it. All of this happens on one read of the inputs:
//   warp     8 rows (steps) x 32 or 64 channels in registers, one or two channels a lane;
//   block    8 warps, 64 rows: the warps' maps are joined in shared memory;
//   cluster  up to 16 blocks, 1024 rows: every block puts its map into the shared memory of all the others
//            (distributed shared memory), one cluster barrier a round, and each joins those in front of it.
// A cluster walks the time axis in rounds and carries the state in registers, so a call needs no workspace,
// no flags in memory and no second launch, and its result does not depend on timing. The kernels are bound by
// memory: 8 (bf16) or 12 (fp32) bytes an element forward, 14 or 20 backward.
//
// A boundary between packed sequences is a step whose map forgets: (forget, a h0 + b). In the backward the same
// steps stop the gradient, which walks the maps the other way: with y_t = a_t g_t, g_t = dh_t + y_{t+1}.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gla_common.cuh"
#include "gla_gate.cuh"
#include "gla_internal.h"

namespace gla {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 8;                 // rows of a warp
constexpr int kTile = kWarps * kRows;    // rows of a block in a round; one state per tile is kept for the backward
constexpr int kMaxCluster = 16;

struct GateForm {
    bool preact, leak;
    float inv_tau;
};

// ---- cluster primitives -----------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// store to the same shared-memory address in block `rank` of the cluster
__device__ __forceinline__ void st_peer(float2* p, uint32_t rank, float2 x) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    asm volatile(
        "{\n\t.reg .b32 r;\n\t"
        "mapa.shared::cluster.u32 r, %0, %1;\n\t"
        "st.shared::cluster.v2.f32 [r], {%2, %3};\n\t}" ::"r"(a),
        "r"(rank), "f"(x.x), "f"(x.y)
        : "memory");
}

// ---- loads and stores of VEC adjacent channels ------------------------------------------
template <int VEC>
__device__ __forceinline__ void ldv(const float* p, float* y) {
    if constexpr (VEC == 2) {
        const float2 t = *reinterpret_cast<const float2*>(p);
        y[0] = t.x;
        y[1] = t.y;
    } else y[0] = *p;
}
template <int VEC>
__device__ __forceinline__ void ldv(const __nv_bfloat16* p, float* y) {
    if constexpr (VEC == 2) {
        const __nv_bfloat162 t = *reinterpret_cast<const __nv_bfloat162*>(p);
        y[0] = __bfloat162float(t.x);
        y[1] = __bfloat162float(t.y);
    } else y[0] = __bfloat162float(*p);
}
template <int VEC>
__device__ __forceinline__ void stv(float* p, const float* y) {
    if constexpr (VEC == 2) *reinterpret_cast<float2*>(p) = make_float2(y[0], y[1]);
    else *p = y[0];
}
template <int VEC>
__device__ __forceinline__ void stv(__nv_bfloat16* p, const float* y) {
    if constexpr (VEC == 2) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(y[0], y[1]);
    else *p = __float2bfloat16_rn(y[0]);
}

// a_t and w_t from the gate argument
__device__ __forceinline__ void gate_of(const GateForm& f, float g, float& a, float& w) {
    const float la = f.preact ? logsigmoid_f(g) * f.inv_tau : g;
    a = expf(la);
    w = f.leak ? -expm1f(la) : 1.f;
}

// Maps of packed rows that hold a sequence's start forget everything in front of it, whatever that is: an infinity
// or a NaN of one sequence must not reach the next through 0 * inf. Such a map has the factor -0, which no product
// of decays gives and which products keep.
constexpr float kForget = -0.f;
template <bool PACKED>
__device__ __forceinline__ bool forgets(float m) { return PACKED && __float_as_uint(m) == 0x80000000u; }
template <bool PACKED>
__device__ __forceinline__ float join(float m, float s, float u) { return forgets<PACKED>(m) ? u : fmaf(m, s, u); }
template <bool PACKED>
__device__ __forceinline__ float join(float m, float f) { return forgets<PACKED>(m) ? m : m * f; }

// What a warp knows of its 8 rows t0 .. t0+7: which belong to a sequence, which start or end one, and (per lane,
// for row t0 + lane) the sequence's number.
struct RowInfo {
    uint32_t valid, start, end;
    int n;
};

// Packed rows: the sequence of row t is the last one with cu[n] <= t. The search reads cu[0 .. B] only, whatever
// the values are.
__device__ __forceinline__ RowInfo rows_packed(const int32_t* __restrict__ cu, int B, int64_t t0, int64_t L, int lane) {
    int lo = 0, hi = B + 1;  // first entry above t lies in [lo, hi]
    const int64_t t = t0 + lane;
    if (lane < kRows && t < L) {
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t) lo = mid + 1;
            else hi = mid;
        }
    }
    RowInfo r;
    r.n = lo - 1;
    const bool ok = r.n >= 0 && r.n < B;
    bool st = false, en = false;
    if (ok) {
        st = cu[r.n] == t;
        en = cu[r.n + 1] == t + 1;
    }
    r.valid = __ballot_sync(0xffffffffu, ok);
    r.start = __ballot_sync(0xffffffffu, st);
    r.end = __ballot_sync(0xffffffffu, en);
    return r;
}

// Empty sequences have no row that could write their end: out[n] = in[n] (or 0), spread over the cluster's warps.
template <int VEC>
__device__ __forceinline__ void copy_empty(const int32_t* __restrict__ cu, int B, int64_t H, int64_t head, int64_t D,
                                           int64_t c, const float* __restrict__ in, float* __restrict__ out, int first,
                                           int stride, int lane) {
    if (!out) return;
    for (int n0 = first * 32; n0 < B; n0 += stride * 32) {
        const int n = n0 + lane;
        uint32_t m = __ballot_sync(0xffffffffu, n < B && cu[n < B ? n : 0] >= cu[n < B ? n + 1 : 0]);
        while (m) {
            const int64_t e = n0 + __ffs(m) - 1;
            m &= m - 1;
            if (c < D) {
                float y[VEC] = {};
                if (in) ldv<VEC>(in + (e * H + head) * D + c, y);
                stv<VEC>(out + (e * H + head) * D + c, y);
            }
        }
    }
}

// ---- forward ------------------------------------------------------------------------------
// Grid: (sequence or head) x channel tile x cluster of `cl` blocks. Rows of round r and block q: (r cl + q) kTile.
template <typename T, int VEC, bool PACKED>
__global__ void __launch_bounds__(kThreads, VEC == 2 ? 3 : 4)
    k_scan_fwd(ScanProblem p, GateForm f, int cl, const T* __restrict__ x, const float* __restrict__ la,
               const int32_t* __restrict__ cu, const float* __restrict__ h0, T* __restrict__ h, float* __restrict__ hT,
               float* __restrict__ seg) {
    constexpr int CW = 32 * VEC;
    __shared__ float2 agg[2][kWarps][CW];
    extern __shared__ float2 peer[];  // [2][cl][CW]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = cl > 1 ? int(cluster_rank()) : 0;
    const int64_t tiles = cdiv(p.D, CW);
    const int64_t id = blockIdx.x / cl, lead = id / tiles, c = (id % tiles) * CW + lane * VEC;
    const bool mine = c < p.D;
    const int64_t head = PACKED ? lead : 0;
    const int64_t row0 = lead * p.L;
    if (cl > 1) cluster_arrive();  // every block of the cluster has started before any puts data into it
    if constexpr (PACKED) copy_empty<VEC>(cu, int(p.B), p.H, head, p.D, c, h0, hT, rank * kWarps + warp, cl * kWarps, lane);
    float carry[VEC] = {};
    if (!PACKED && h0 && mine) ldv<VEC>(h0 + lead * p.D + c, carry);
    if (cl > 1) cluster_wait();
    const int64_t rounds = cdiv(p.L, int64_t(kTile) * cl), nseg = cdiv(p.L, kTile);
    for (int64_t r = 0; r < rounds; ++r) {
        const int par = int(r & 1);
        const int64_t base = (r * cl + rank) * kTile, t0 = base + warp * kRows;
        float a[kRows][VEC], b[kRows][VEC];
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int64_t i = (row0 + t0 + j) * p.D + c;
#pragma unroll
            for (int v = 0; v < VEC; ++v) a[j][v] = b[j][v] = 0.f;
            if (mine && t0 + j < p.L) {
                ldv<VEC>(la + i, a[j]);
                ldv<VEC>(x + i, b[j]);
            }
        }
        RowInfo ri;
        if constexpr (PACKED) ri = rows_packed(cu, int(p.B), t0, p.L, lane);
        float A[VEC], U[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) A[v] = 1.f, U[v] = 0.f;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const bool ok = PACKED ? (ri.valid >> j & 1) : t0 + j < p.L;
            float s0[VEC] = {};
            bool start = false;
            if constexpr (PACKED) {
                start = ri.start >> j & 1;
                if (start) {
                    const int64_t n = __shfl_sync(0xffffffffu, ri.n, j);
                    if (h0 && mine) ldv<VEC>(h0 + (n * p.H + head) * p.D + c, s0);
                }
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                float aa, w;
                gate_of(f, a[j][v], aa, w);
                b[j][v] = ok ? w * b[j][v] : 0.f;
                a[j][v] = ok ? aa : 1.f;
                if (start) {
                    b[j][v] = fmaf(aa, s0[v], b[j][v]);
                    a[j][v] = kForget;
                }
                A[v] = join<PACKED>(a[j][v], A[v]);
                U[v] = join<PACKED>(a[j][v], U[v], b[j][v]);
            }
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) agg[par][warp][v * 32 + lane] = make_float2(A[v], U[v]);
        __syncthreads();
        // the map of the block's rows in front of this warp's
        float pa[VEC], pu[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) pa[v] = 1.f, pu[v] = 0.f;
        for (int w = 0; w < warp; ++w) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float2 m = agg[par][w][v * 32 + lane];
                pa[v] = join<PACKED>(m.x, pa[v]);
                pu[v] = join<PACKED>(m.x, pu[v], m.y);
            }
        }
        float in[VEC];  // state entering the block's rows
        if (cl > 1) {
            if (warp == kWarps - 1) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float2 m = make_float2(join<PACKED>(A[v], pa[v]), join<PACKED>(A[v], pu[v], U[v]));
                    for (int q = 0; q < cl; ++q) st_peer(peer + (par * cl + rank) * CW + v * 32 + lane, q, m);
                }
            }
            cluster_arrive();
            cluster_wait();
            for (int q = 0; q < cl; ++q) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    if (q == rank) in[v] = carry[v];
                    const float2 m = peer[(par * cl + q) * CW + v * 32 + lane];
                    carry[v] = join<PACKED>(m.x, carry[v], m.y);
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                in[v] = carry[v];
                float ta = pa[v], tu = pu[v];
                for (int w = warp; w < kWarps; ++w) {
                    const float2 m = agg[par][w][v * 32 + lane];
                    ta = join<PACKED>(m.x, ta);
                    tu = join<PACKED>(m.x, tu, m.y);
                }
                carry[v] = join<PACKED>(ta, in[v], tu);
            }
        }
        if (seg && warp == 0 && mine && base < p.L) stv<VEC>(seg + (lead * nseg + base / kTile) * p.D + c, in);
        float s[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) s[v] = join<PACKED>(pa[v], in[v], pu[v]);
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) s[v] = join<PACKED>(a[j][v], s[v], b[j][v]);
            const bool ok = PACKED ? (ri.valid >> j & 1) : t0 + j < p.L;
            if (h && ok && mine) stv<VEC>(h + (row0 + t0 + j) * p.D + c, s);
            if constexpr (PACKED) {
                if (ri.end >> j & 1) {
                    const int64_t n = __shfl_sync(0xffffffffu, ri.n, j);
                    if (hT && mine) stv<VEC>(hT + (n * p.H + head) * p.D + c, s);
                }
            }
        }
        // rows behind the last one leave the state as it is, so any warp from there on holds hT
        if (!PACKED && hT && mine && t0 < p.L && t0 + kRows >= p.L) stv<VEC>(hT + lead * p.D + c, s);
    }
}

// ---- backward -----------------------------------------------------------------------------
// Rounds, blocks and warps as in the forward, from the last round to the first. The states inside a block's rows
// are recomputed in fp32 from the state that enters them (seg).
template <typename T, int VEC, bool PACKED>
__global__ void __launch_bounds__(kThreads, 2)
    k_scan_bwd(ScanProblem p, GateForm f, int cl, const T* __restrict__ x, const float* __restrict__ la,
               const int32_t* __restrict__ cu, const float* __restrict__ h0, const T* __restrict__ dh,
               const float* __restrict__ dhT, T* __restrict__ dx, float* __restrict__ dla, float* __restrict__ dh0,
               const float* __restrict__ seg) {
    constexpr int CW = 32 * VEC;
    __shared__ float2 aggu[2][kWarps][CW];
    __shared__ float aggy[2][kWarps][CW];
    extern __shared__ float2 peer[];  // [2][cl][CW]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = cl > 1 ? int(cluster_rank()) : 0;
    const int64_t tiles = cdiv(p.D, CW);
    const int64_t id = blockIdx.x / cl, lead = id / tiles, c = (id % tiles) * CW + lane * VEC;
    const bool mine = c < p.D;
    const int64_t head = PACKED ? lead : 0;
    const int64_t row0 = lead * p.L;
    if (cl > 1) cluster_arrive();
    if constexpr (PACKED) copy_empty<VEC>(cu, int(p.B), p.H, head, p.D, c, dhT, dh0, rank * kWarps + warp, cl * kWarps, lane);
    float carry[VEC] = {};  // y of the row behind the round's last
    if (!PACKED && dhT && mine) ldv<VEC>(dhT + lead * p.D + c, carry);
    if (cl > 1) cluster_wait();
    const int64_t rounds = cdiv(p.L, int64_t(kTile) * cl), nseg = cdiv(p.L, kTile);
    for (int64_t r = rounds - 1; r >= 0; --r) {
        const int par = int(r & 1);
        const int64_t base = (r * cl + rank) * kTile, t0 = base + warp * kRows;
        float a[kRows][VEC], b[kRows][VEC], z[kRows][VEC], xv[kRows][VEC], d[kRows][VEC], w[kRows][VEC];
        float s[VEC] = {};  // state entering the block's rows
        if (mine && base < p.L) ldv<VEC>(seg + (lead * nseg + base / kTile) * p.D + c, s);
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const int64_t i = (row0 + t0 + j) * p.D + c;
#pragma unroll
            for (int v = 0; v < VEC; ++v) z[j][v] = xv[j][v] = d[j][v] = 0.f;
            if (mine && t0 + j < p.L) {
                ldv<VEC>(la + i, z[j]);
                ldv<VEC>(x + i, xv[j]);
                ldv<VEC>(dh + i, d[j]);
            }
        }
        RowInfo ri;
        if constexpr (PACKED) ri = rows_packed(cu, int(p.B), t0, p.L, lane);
        float A[VEC], U[VEC], Y[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) A[v] = 1.f, U[v] = 0.f, Y[v] = 0.f;
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const bool ok = PACKED ? (ri.valid >> j & 1) : t0 + j < p.L;
            float s0[VEC] = {}, e0[VEC] = {};
            bool start = false;
            if constexpr (PACKED) {
                start = ri.start >> j & 1;
                const bool end = ri.end >> j & 1;
                if (start || end) {
                    const int64_t n = __shfl_sync(0xffffffffu, ri.n, j);
                    if (start && h0 && mine) ldv<VEC>(h0 + (n * p.H + head) * p.D + c, s0);
                    if (end && dhT && mine) ldv<VEC>(dhT + (n * p.H + head) * p.D + c, e0);
                }
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                gate_of(f, z[j][v], a[j][v], w[j][v]);
                if (!ok) a[j][v] = 1.f, w[j][v] = 0.f, xv[j][v] = 0.f, d[j][v] = 0.f;
                d[j][v] += e0[v];
                b[j][v] = w[j][v] * xv[j][v];
                if (start) {
                    b[j][v] = fmaf(a[j][v], s0[v], b[j][v]);
                    A[v] = kForget;
                    U[v] = b[j][v];
                } else {
                    A[v] = join<PACKED>(A[v], a[j][v]);  // of both directions: U and Y carry what the other rows hold
                    U[v] = fmaf(a[j][v], U[v], b[j][v]);
                }
            }
        }
#pragma unroll
        for (int j = kRows - 1; j >= 0; --j) {
            const bool start = PACKED ? (ri.start >> j & 1) : false;
#pragma unroll
            for (int v = 0; v < VEC; ++v) Y[v] = start ? 0.f : a[j][v] * (d[j][v] + Y[v]);
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            aggu[par][warp][v * 32 + lane] = make_float2(A[v], U[v]);
            aggy[par][warp][v * 32 + lane] = Y[v];
        }
        __syncthreads();
        for (int q = 0; q < warp; ++q) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float2 m = aggu[par][q][v * 32 + lane];
                s[v] = join<PACKED>(m.x, s[v], m.y);
            }
        }
        // the map (of y) of the block's rows behind this warp's
        float pa[VEC], py[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) pa[v] = 1.f, py[v] = 0.f;
        for (int q = kWarps - 1; q > warp; --q) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float m = aggu[par][q][v * 32 + lane].x;
                pa[v] = join<PACKED>(m, pa[v]);
                py[v] = join<PACKED>(m, py[v], aggy[par][q][v * 32 + lane]);
            }
        }
        float in[VEC];
        if (cl > 1) {
            if (warp == 0) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float2 m = make_float2(join<PACKED>(A[v], pa[v]), join<PACKED>(A[v], py[v], Y[v]));
                    for (int q = 0; q < cl; ++q) st_peer(peer + (par * cl + rank) * CW + v * 32 + lane, q, m);
                }
            }
            cluster_arrive();
            cluster_wait();
            for (int q = cl - 1; q >= 0; --q) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    if (q == rank) in[v] = carry[v];
                    const float2 m = peer[(par * cl + q) * CW + v * 32 + lane];
                    carry[v] = join<PACKED>(m.x, carry[v], m.y);
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                in[v] = carry[v];
                float ta = pa[v], ty = py[v];
                for (int q = warp; q >= 0; --q) {
                    const float m = aggu[par][q][v * 32 + lane].x;
                    ta = join<PACKED>(m, ta);
                    ty = join<PACKED>(m, ty, aggy[par][q][v * 32 + lane]);
                }
                carry[v] = join<PACKED>(ta, in[v], ty);
            }
        }
        float y[VEC], hp[kRows][VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[v] = join<PACKED>(pa[v], in[v], py[v]);
        // states in front of each row
#pragma unroll
        for (int j = 0; j < kRows; ++j) {
            const bool start = PACKED ? (ri.start >> j & 1) : false;
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                hp[j][v] = s[v];
                s[v] = start ? b[j][v] : fmaf(a[j][v], s[v], b[j][v]);
            }
        }
#pragma unroll
        for (int j = kRows - 1; j >= 0; --j) {
            const bool ok = PACKED ? (ri.valid >> j & 1) : t0 + j < p.L;
            float o1[VEC], o2[VEC], s0[VEC] = {};
            bool start = false;
            int64_t n = 0;
            if constexpr (PACKED) {
                start = ri.start >> j & 1;
                if (start) {
                    n = __shfl_sync(0xffffffffu, ri.n, j);
                    if (h0 && mine) ldv<VEC>(h0 + (n * p.H + head) * p.D + c, s0);
                }
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float g = d[j][v] + y[v];
                const float hm = start ? s0[v] : hp[j][v];
                y[v] = a[j][v] * g;
                o1[v] = w[j][v] * g;
                o2[v] = y[v] * (f.leak ? hm - xv[j][v] : hm);
                if (f.preact) o2[v] *= sigmoid_neg_f(z[j][v]) * f.inv_tau;
            }
            if (ok && mine) {
                const int64_t i = (row0 + t0 + j) * p.D + c;
                stv<VEC>(dx + i, o1);
                stv<VEC>(dla + i, o2);
            }
            if (start) {
                if (dh0 && mine) stv<VEC>(dh0 + (n * p.H + head) * p.D + c, y);
#pragma unroll
                for (int v = 0; v < VEC; ++v) y[v] = 0.f;
            }
        }
        if (!PACKED && dh0 && mine && t0 == 0) stv<VEC>(dh0 + lead * p.D + c, y);
    }
}

// ---- one token ----------------------------------------------------------------------------
constexpr int kStepThreads = 128;

// Whether an earlier row of the call names the same slot (every thread of the block gets the answer).
__device__ __forceinline__ bool named_before(const int32_t* slots, int64_t b, int32_t slot) {
    int dup = 0;
    for (int64_t i = threadIdx.x; i < b; i += blockDim.x) dup |= slots[i] == slot;
    return __syncthreads_or(dup) != 0;
}

template <typename T>
__global__ void __launch_bounds__(kStepThreads) k_scan_step(ScanProblem p, GateForm f, const T* __restrict__ x,
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
    const int64_t c = int64_t(blockIdx.x) * kStepThreads + threadIdx.x;
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

// Blocks per cluster: enough to fill the SMs (three blocks of 256 threads on each) where the sequences and channel
// tiles alone do not, but no more than there are row tiles.
int cluster_size(int64_t groups, int64_t L) {
    const int64_t tiles = cdiv(L, kTile);
    int cl = 1;
    while (cl < kMaxCluster && cl < tiles && groups * cl < 148 * 3) cl *= 2;
    return cl;
}

template <typename K, typename... Args>
gla_status launch_clusters(const char* name, K kernel, int64_t groups, int cl, int vec, cudaStream_t s, Args... args) {
    if (groups * cl > (int64_t(1) << 31) - 1) return GLA_ERR_UNSUPPORTED;
    if (cl > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return GLA_ERR_CUDA;
    launch_begin(name, s);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(groups * cl));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = cl > 1 ? size_t(2) * cl * 32 * vec * sizeof(float2) : 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(cl);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    (void)cudaLaunchKernelEx(&cfg, kernel, args...);
    return launch_end(name, s);
}

template <typename T, int VEC, bool PACKED>
gla_status fwd_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                     void* h, float* hT, float* seg, cudaStream_t s) {
    const int64_t groups = (PACKED ? p.H : p.B * p.H) * cdiv(p.D, 32 * VEC);
    const int cl = cluster_size(groups, p.L);
    return launch_clusters("scan_fwd", k_scan_fwd<T, VEC, PACKED>, groups, cl, VEC, s, p, form(p), cl,
                           static_cast<const T*>(x), la, cu, h0, static_cast<T*>(h), hT, seg);
}

template <typename T, int VEC, bool PACKED>
gla_status bwd_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                     const void* dh, const float* dhT, void* dx, float* dla, float* dh0, const float* seg,
                     cudaStream_t s) {
    const int64_t groups = (PACKED ? p.H : p.B * p.H) * cdiv(p.D, 32 * VEC);
    const int cl = cluster_size(groups, p.L);
    return launch_clusters("scan_bwd", k_scan_bwd<T, VEC, PACKED>, groups, cl, VEC, s, p, form(p), cl,
                           static_cast<const T*>(x), la, cu, h0, static_cast<const T*>(dh), dhT, static_cast<T*>(dx),
                           dla, dh0, seg);
}

template <typename T>
gla_status step_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* slots, int64_t pool,
                      float* state, void* h, cudaStream_t s) {
    const dim3 grid(unsigned(cdiv(p.H * p.D, kStepThreads)), unsigned(p.B));
    GLA_LAUNCH("scan_step", k_scan_step<T>, grid, kStepThreads, 0, s, p, form(p), static_cast<const T*>(x), la, slots,
               pool, state, static_cast<T*>(h), device_error_word());
    return GLA_OK;
}

// Two channels a lane where the rows' pairs are aligned (an even width), else one.
#define GLA_SCAN_DISPATCH(fn, ...)                                                                         \
    (p.bf16 ? (p.D % 2 == 0 ? (p.packed ? fn<__nv_bfloat16, 2, true>(__VA_ARGS__)                          \
                                        : fn<__nv_bfloat16, 2, false>(__VA_ARGS__))                        \
                            : (p.packed ? fn<__nv_bfloat16, 1, true>(__VA_ARGS__)                          \
                                        : fn<__nv_bfloat16, 1, false>(__VA_ARGS__)))                       \
            : (p.D % 2 == 0 ? (p.packed ? fn<float, 2, true>(__VA_ARGS__) : fn<float, 2, false>(__VA_ARGS__)) \
                            : (p.packed ? fn<float, 1, true>(__VA_ARGS__) : fn<float, 1, false>(__VA_ARGS__))))

}  // namespace

size_t scan_workspace(const ScanProblem& p, Arena& a) {
    (void)a.take<float>(size_t((p.packed ? p.H : p.B * p.H) * cdiv(p.L, kTile) * p.D));
    return a.used;
}

gla_status scan_fwd(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0, void* h,
                    float* hT, float* seg, cudaStream_t s) {
    return GLA_SCAN_DISPATCH(fwd_typed, p, x, la, cu, h0, h, hT, seg, s);
}

gla_status scan_bwd(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                    const void* dh, const float* dhT, void* dx, float* dla, float* dh0, float* seg, bool reuse,
                    cudaStream_t s) {
    if (!reuse) {
        const gla_status st = scan_fwd(p, x, la, cu, h0, nullptr, nullptr, seg, s);
        if (st != GLA_OK) return st;
    }
    return GLA_SCAN_DISPATCH(bwd_typed, p, x, la, cu, h0, dh, dhT, dx, dla, dh0, seg, s);
}

gla_status scan_step(const ScanProblem& p, const void* x, const float* la, const int32_t* slots, int64_t pool,
                     float* state, void* h, cudaStream_t s) {
    return p.bf16 ? step_typed<__nv_bfloat16>(p, x, la, slots, pool, state, h, s)
                  : step_typed<float>(p, x, la, slots, pool, state, h, s);
}

}  // namespace gla
