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
#include <type_traits>

#include "gla_common.cuh"
#include "gla_gate.cuh"
#include "gla_internal.h"
#include "tc_prims.cuh"

namespace gla {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kSeg = 64;  // rows between the states kept for the backward, which takes a block's rows from one of them
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

// ---- gates --------------------------------------------------------------------------------
// The library's expf / expm1f / log1pf come to about 60 instructions an element, four times what the memory
// bandwidth leaves room for; these take 13 (a and w) and 12 (log alpha from z). Accuracies in units of u = 2^-24.

// a = e^la and 1 - a for la <= 0. Near 0, where a multiplies up over many steps and 1 - a must keep its relative
// precision: 1 - a = -la q(la) with q = (e^x - 1) / x as a polynomial fitted at the Chebyshev nodes of [-1/2, 0]
// (relative error 3e-9), so 1 - a is within 3 u and a = 1 - (1 - a) correctly rounded from it. Below -1/2 (a < 0.61,
// no long products): the ex2 instruction, within (4 + |la|) u.
__device__ __forceinline__ void decay_of(float la, float& a, float& one_minus_a) {
    float q = fmaf(0.00112340425f, la, 0.00818961393f);
    q = fmaf(q, la, 0.0416300744f);
    q = fmaf(q, la, 0.166662425f);
    q = fmaf(q, la, 0.499999821f);
    q = fmaf(q, la, 1.f);
    const float m = -la * q;
    const float e = tc::exp2_ftz(la * tc::kLog2e);
    const bool near = fabsf(la) < 0.5f;
    a = near ? 1.f - m : e;
    one_minus_a = near ? m : 1.f - e;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// logsigmoid(z) = min(z, 0) - log(1 + t), t = e^-|z| in [0, 1], with log(1 + t) = 2 atanh(s), s = t / (2 + t) <= 1/3:
// atanh(s) / s as a polynomial in s^2 fitted at the Chebyshev nodes of [0, 1/9] (relative error 8e-9). Small t
// keeps its relative precision, (8 + |z|) u in all.
__device__ __forceinline__ float logsigmoid_series(float z, float& t) {
    t = tc::exp2_ftz(-fabsf(z) * tc::kLog2e);
    const float s = t * rcp(2.f + t), y = s * s;
    float q = fmaf(0.140788898f, y, 0.139825791f);
    q = fmaf(q, y, 0.200122982f);
    q = fmaf(q, y, 0.333331615f);
    q = fmaf(q, y, 1.f);
    return fmaf(-2.f * s, q, fminf(z, 0.f));
}

// a_t and w_t from the gate argument; for a pre-activation also dlog a / dz = sigmoid(-z) / tau
template <bool PREACT>
__device__ __forceinline__ void gate_of(const GateForm& f, float g, float& a, float& w, float& dz) {
    float la = g;
    if constexpr (PREACT) {
        float t;
        la = logsigmoid_series(g, t) * f.inv_tau;
        const float r = rcp(1.f + t);
        dz = (g < 0.f ? r : t * r) * f.inv_tau;
    }
    decay_of(la, a, w);
    if (!f.leak) w = 1.f;
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

// What a warp knows of its rows t0, t0 + 1, ...: which belong to a sequence, which start or end one, and (per lane,
// for row t0 + lane) the sequence's number.
struct RowInfo {
    uint32_t valid, start, end;
    int n;
};

// Packed rows: the sequence of row t is the last one with cu[n] <= t. The search reads cu[0 .. B] only, whatever
// the values are.
template <int ROWS>
__device__ __forceinline__ RowInfo rows_packed(const int32_t* __restrict__ cu, int B, int64_t t0, int64_t L, int lane) {
    int lo = 0, hi = B + 1;  // first entry above t lies in [lo, hi]
    const int64_t t = t0 + lane;
    if (lane < ROWS && t < L) {
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

// row n of a [B,H,D] state tensor (NULL: zero)
template <int VEC>
__device__ __forceinline__ void state_of(const float* __restrict__ h, int64_t n, const ScanProblem& p, int64_t head,
                                         int64_t c, float* y) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) y[v] = 0.f;
    if (h) ldv<VEC>(h + (n * p.H + head) * p.D + c, y);
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

// A warp's rows of one tensor. Rows behind the last one repeat it, lanes behind the last channel repeat that one, so
// the loads need no predicate; `off` is the row's offset from the warp's first row.
template <int ROWS>
struct RowOffsets {
    uint32_t off[ROWS];
    __device__ __forceinline__ RowOffsets(int64_t rows_left, int64_t D) {
        const int last = int(rows_left < ROWS ? (rows_left < 1 ? 1 : rows_left) : ROWS) - 1;
#pragma unroll
        for (int j = 0; j < ROWS; ++j) off[j] = uint32_t(j < last ? j : last) * uint32_t(D);
    }
};

// ---- staged loads -------------------------------------------------------------------------
// The rows of the next round travel while this one is computed: every lane copies its own channels into its own
// places of shared memory (cp.async, 4 or 8 bytes a row), so that no thread waits for another's copies and two
// rounds' rows cost no registers. Single bf16 channels (an odd width) are too narrow for such a copy and are loaded
// where they are used.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T, int VEC>
constexpr bool kStaged = sizeof(T) * VEC >= 4;

// A lane's rows of one tensor in shared memory: row j at [j][lane].
template <typename T, int VEC, int ROWS>
__device__ __forceinline__ void stage_rows(T* st, const T* src, const RowOffsets<ROWS>& ro) {
    if constexpr (kStaged<T, VEC>) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) copy_async<sizeof(T) * VEC>(st + j * 32 * VEC, src + ro.off[j]);
    }
}
template <typename T, int VEC>
__device__ __forceinline__ void take_row(const T* st, const T* src, uint32_t off, int j, float* y) {
    if constexpr (kStaged<T, VEC>) ldv<VEC>(st + j * 32 * VEC, y);
    else ldv<VEC>(src + off, y);
}

// bytes a warp's stage takes
template <typename T, int VEC, int ROWS>
constexpr int kFwdStage = ROWS * 32 * VEC * int(4 + sizeof(T));
template <typename T, int VEC, int ROWS>
constexpr int kBwdStage = ROWS * 32 * VEC * int(4 + 2 * sizeof(T));

// ---- forward ------------------------------------------------------------------------------
// Grid: (sequence or head) x channel tile x cluster of `cl` blocks. Rows of round r and block q: from (r cl + q) TILE.
template <typename T, int VEC, bool PACKED, bool PREACT, int ROWS>
__global__ void __launch_bounds__(kThreads, ROWS * VEC <= 16 ? 3 : 2)
    k_scan_fwd(ScanProblem p, GateForm f, int cl, const T* __restrict__ x, const float* __restrict__ la,
               const int32_t* __restrict__ cu, const float* __restrict__ h0, T* __restrict__ h, float* __restrict__ hT,
               float* __restrict__ seg) {
    constexpr int CW = 32 * VEC, TILE = kWarps * ROWS;
    __shared__ float2 agg[2][kWarps][CW];
    extern __shared__ float2 peer[];  // [2][cl][CW] the blocks' maps, then the warps' stages
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = cl > 1 ? int(cluster_rank()) : 0;
    const int64_t tiles = cdiv(p.D, CW);
    const int64_t id = blockIdx.x / cl, lead = id / tiles, c = (id % tiles) * CW + lane * VEC;
    const bool mine = c < p.D;
    const int64_t cc = mine ? c : p.D - VEC;
    const int64_t head = PACKED ? lead : 0;
    char* stages = reinterpret_cast<char*>(peer + (cl > 1 ? 2 * cl * CW : 0)) + warp * 2 * kFwdStage<T, VEC, ROWS>;
    const auto row_of = [&](int r) { return (int64_t(r) * cl + rank) * TILE + warp * ROWS; };
    const auto first_of = [&](int64_t t) { return (lead * p.L + (t < p.L ? t : p.L - 1)) * p.D + cc; };
    const auto gates_at = [&](int par) { return reinterpret_cast<float*>(stages + par * kFwdStage<T, VEC, ROWS>) + lane * VEC; };
    const auto x_at = [&](int par) {
        return reinterpret_cast<T*>(stages + par * kFwdStage<T, VEC, ROWS> + ROWS * CW * 4) + lane * VEC;
    };
    const auto stage = [&](int r) {
        const int64_t t = row_of(r), i = first_of(t);
        const RowOffsets<ROWS> ro(p.L - t, p.D);
        stage_rows<float, VEC, ROWS>(gates_at(r & 1), la + i, ro);
        stage_rows<T, VEC, ROWS>(x_at(r & 1), x + i, ro);
    };
    stage(0);
    copies_commit();
    if (cl > 1) cluster_arrive();  // every block of the cluster has started before any puts data into it
    if constexpr (PACKED) copy_empty<VEC>(cu, int(p.B), p.H, head, p.D, c, h0, hT, rank * kWarps + warp, cl * kWarps, lane);
    float carry[VEC] = {};
    if (!PACKED && h0) ldv<VEC>(h0 + lead * p.D + cc, carry);
    if (cl > 1) cluster_wait();
    const int rounds = int(cdiv(p.L, int64_t(TILE) * cl));
    const int64_t nseg = cdiv(p.L, kSeg);
    for (int r = 0; r < rounds; ++r) {
        const int par = r & 1;
        const int64_t t0 = row_of(r), first = first_of(t0);
        const RowOffsets<ROWS> ro(p.L - t0, p.D);
        if (r + 1 < rounds) stage(r + 1);
        copies_commit();
        copies_wait<1>();
        float a[ROWS][VEC], b[ROWS][VEC];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            ldv<VEC>(gates_at(par) + j * CW, a[j]);
            take_row<T, VEC>(x_at(par), x + first, ro.off[j], j, b[j]);
        }
        RowInfo ri{0, 0, 0, 0};
        if constexpr (PACKED) ri = rows_packed<ROWS>(cu, int(p.B), t0, p.L, lane);
        else ri.valid = t0 + ROWS <= p.L ? ~0u : t0 < p.L ? (1u << (p.L - t0)) - 1 : 0u;
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                float w, dz;
                gate_of<PREACT>(f, a[j][v], a[j][v], w, dz);
                b[j][v] *= w;
            }
        }
        constexpr uint32_t kAll = ROWS == 32 ? ~0u : (1u << ROWS) - 1;
        if ((ri.valid & kAll) != kAll) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                if (!(ri.valid >> j & 1)) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) a[j][v] = 1.f, b[j][v] = 0.f;
                }
            }
        }
        float A[VEC], U[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) A[v] = 1.f, U[v] = 0.f;
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (PACKED && (ri.start >> j & 1)) state_of<VEC>(h0, __shfl_sync(0xffffffffu, ri.n, j), p, head, cc, U);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                A[v] *= a[j][v];
                U[v] = fmaf(a[j][v], U[v], b[j][v]);
            }
        }
        if (PACKED && ri.start) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) A[v] = kForget;
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) agg[par][warp][v * 32 + lane] = make_float2(A[v], U[v]);
        __syncthreads();
        // the map of the block's rows in front of this warp's
        float pa[VEC], pu[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) pa[v] = 1.f, pu[v] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w) {
            if (w < warp) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float2 m = agg[par][w][v * 32 + lane];
                    pa[v] = join<PACKED>(m.x, pa[v]);
                    pu[v] = join<PACKED>(m.x, pu[v], m.y);
                }
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
        float s[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) s[v] = join<PACKED>(pa[v], in[v], pu[v]);
        if (seg && mine && t0 < p.L && t0 % kSeg == 0) stv<VEC>(seg + (lead * nseg + t0 / kSeg) * p.D + c, s);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (PACKED && (ri.start >> j & 1)) state_of<VEC>(h0, __shfl_sync(0xffffffffu, ri.n, j), p, head, cc, s);
#pragma unroll
            for (int v = 0; v < VEC; ++v) s[v] = fmaf(a[j][v], s[v], b[j][v]);
            if (h && mine && (ri.valid >> j & 1)) stv<VEC>(h + first + ro.off[j], s);
            if (PACKED && (ri.end >> j & 1)) {
                const int64_t n = __shfl_sync(0xffffffffu, ri.n, j);
                if (hT && mine) stv<VEC>(hT + (n * p.H + head) * p.D + c, s);
            }
        }
        // rows behind the last one leave the state as it is, so the warp with the last row holds hT
        if (!PACKED && hT && mine && t0 < p.L && t0 + ROWS >= p.L) stv<VEC>(hT + lead * p.D + c, s);
    }
}

// ---- backward -----------------------------------------------------------------------------
// Rounds, blocks and warps as in the forward, from the last round to the first. The states inside a block's rows
// are recomputed in fp32 from the state that enters them (seg).
template <typename T, int VEC, bool PACKED, bool PREACT>
__global__ void __launch_bounds__(kThreads, 2)
    k_scan_bwd(ScanProblem p, GateForm f, int cl, const T* __restrict__ x, const float* __restrict__ la,
               const int32_t* __restrict__ cu, const float* __restrict__ h0, const T* __restrict__ dh,
               const float* __restrict__ dhT, T* __restrict__ dx, float* __restrict__ dla, float* __restrict__ dh0,
               const float* __restrict__ seg) {
    constexpr int CW = 32 * VEC, ROWS = kSeg / kWarps;
    __shared__ float2 aggu[2][kWarps][CW];
    __shared__ float aggy[2][kWarps][CW];
    extern __shared__ float2 peer[];  // [2][cl][CW] the blocks' maps, then the warps' stages
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = cl > 1 ? int(cluster_rank()) : 0;
    const int64_t tiles = cdiv(p.D, CW);
    const int64_t id = blockIdx.x / cl, lead = id / tiles, c = (id % tiles) * CW + lane * VEC;
    const bool mine = c < p.D;
    const int64_t cc = mine ? c : p.D - VEC;
    const int64_t head = PACKED ? lead : 0;
    char* stages = reinterpret_cast<char*>(peer + (cl > 1 ? 2 * cl * CW : 0)) + warp * 2 * kBwdStage<T, VEC, ROWS>;
    const auto row_of = [&](int r) { return (int64_t(r) * cl + rank) * kSeg + warp * ROWS; };
    const auto first_of = [&](int64_t t) { return (lead * p.L + (t < p.L ? t : p.L - 1)) * p.D + cc; };
    const auto gates_at = [&](int par) { return reinterpret_cast<float*>(stages + par * kBwdStage<T, VEC, ROWS>) + lane * VEC; };
    const auto x_at = [&](int par) {
        return reinterpret_cast<T*>(stages + par * kBwdStage<T, VEC, ROWS> + ROWS * CW * 4) + lane * VEC;
    };
    const auto dh_at = [&](int par) { return x_at(par) + ROWS * CW; };
    const auto stage = [&](int r) {
        const int64_t t = row_of(r), i = first_of(t);
        const RowOffsets<ROWS> ro(p.L - t, p.D);
        stage_rows<float, VEC, ROWS>(gates_at(r & 1), la + i, ro);
        stage_rows<T, VEC, ROWS>(x_at(r & 1), x + i, ro);
        stage_rows<T, VEC, ROWS>(dh_at(r & 1), dh + i, ro);
    };
    const int rounds = int(cdiv(p.L, int64_t(kSeg) * cl));
    stage(rounds - 1);
    copies_commit();
    if (cl > 1) cluster_arrive();
    if constexpr (PACKED) copy_empty<VEC>(cu, int(p.B), p.H, head, p.D, c, dhT, dh0, rank * kWarps + warp, cl * kWarps, lane);
    float carry[VEC] = {};  // y of the row behind the round's last
    if (!PACKED && dhT) ldv<VEC>(dhT + lead * p.D + cc, carry);
    if (cl > 1) cluster_wait();
    const int64_t nseg = cdiv(p.L, kSeg);
    for (int r = rounds - 1; r >= 0; --r) {
        const int par = r & 1;
        const int64_t tile = int64_t(r) * cl + rank, t0 = row_of(r), first = first_of(t0);
        const RowOffsets<ROWS> ro(p.L - t0, p.D);
        float a[ROWS][VEC], w[ROWS][VEC], xv[ROWS][VEC], d[ROWS][VEC], dz[ROWS][VEC];
        float s[VEC];  // state entering the block's rows
        ldv<VEC>(seg + (lead * nseg + (tile < nseg ? tile : nseg - 1)) * p.D + cc, s);
        if (r > 0) stage(r - 1);
        copies_commit();
        copies_wait<1>();
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            ldv<VEC>(gates_at(par) + j * CW, a[j]);
            take_row<T, VEC>(x_at(par), x + first, ro.off[j], j, xv[j]);
            take_row<T, VEC>(dh_at(par), dh + first, ro.off[j], j, d[j]);
        }
        RowInfo ri{0, 0, 0, 0};
        if constexpr (PACKED) ri = rows_packed<ROWS>(cu, int(p.B), t0, p.L, lane);
        else ri.valid = t0 + ROWS <= p.L ? ~0u : t0 < p.L ? (1u << (p.L - t0)) - 1 : 0u;
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
#pragma unroll
            for (int v = 0; v < VEC; ++v) gate_of<PREACT>(f, a[j][v], a[j][v], w[j][v], dz[j][v]);
        }
        constexpr uint32_t kAll = (1u << ROWS) - 1;
        if ((ri.valid & kAll) != kAll) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                if (!(ri.valid >> j & 1)) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) a[j][v] = 1.f, w[j][v] = 0.f, xv[j][v] = 0.f, d[j][v] = 0.f;
                }
            }
        }
        float A[VEC], U[VEC], Y[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) A[v] = 1.f, U[v] = 0.f, Y[v] = 0.f;
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (PACKED && (ri.start >> j & 1)) state_of<VEC>(h0, __shfl_sync(0xffffffffu, ri.n, j), p, head, cc, U);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                A[v] *= a[j][v];
                U[v] = fmaf(a[j][v], U[v], w[j][v] * xv[j][v]);
            }
        }
#pragma unroll
        for (int j = ROWS - 1; j >= 0; --j) {
            if (PACKED && (ri.end >> j & 1)) {  // the gradient of the last state enters here, in place of the next row's
                float e[VEC];
                state_of<VEC>(dhT, __shfl_sync(0xffffffffu, ri.n, j), p, head, cc, e);
#pragma unroll
                for (int v = 0; v < VEC; ++v) d[j][v] += e[v];
            }
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                Y[v] = a[j][v] * (d[j][v] + Y[v]);
                if (PACKED && (ri.start >> j & 1)) Y[v] = 0.f;
            }
        }
        if (PACKED && ri.start) {  // of both directions: U and Y carry what the warp's other rows hold
#pragma unroll
            for (int v = 0; v < VEC; ++v) A[v] = kForget;
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            aggu[par][warp][v * 32 + lane] = make_float2(A[v], U[v]);
            aggy[par][warp][v * 32 + lane] = Y[v];
        }
        __syncthreads();
        float pa[VEC], py[VEC];  // the map (of y) of the block's rows behind this warp's
#pragma unroll
        for (int v = 0; v < VEC; ++v) pa[v] = 1.f, py[v] = 0.f;
#pragma unroll
        for (int q = 0; q < kWarps; ++q) {
            if (q < warp) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float2 m = aggu[par][q][v * 32 + lane];
                    s[v] = join<PACKED>(m.x, s[v], m.y);
                }
            }
        }
#pragma unroll
        for (int q = kWarps - 1; q > 0; --q) {
            if (q > warp) {
#pragma unroll
                for (int v = 0; v < VEC; ++v) {
                    const float m = aggu[par][q][v * 32 + lane].x;
                    pa[v] = join<PACKED>(m, pa[v]);
                    py[v] = join<PACKED>(m, py[v], aggy[par][q][v * 32 + lane]);
                }
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
        float y[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[v] = join<PACKED>(pa[v], in[v], py[v]);
        // xv becomes what dlog a_t multiplies: h_{t-1}, less x_t where the input's weight is 1 - a
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (PACKED && (ri.start >> j & 1)) state_of<VEC>(h0, __shfl_sync(0xffffffffu, ri.n, j), p, head, cc, s);
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float xj = xv[j][v];
                xv[j][v] = f.leak ? s[v] - xj : s[v];
                s[v] = fmaf(a[j][v], s[v], w[j][v] * xj);
            }
        }
#pragma unroll
        for (int j = ROWS - 1; j >= 0; --j) {
            float o1[VEC], o2[VEC];
#pragma unroll
            for (int v = 0; v < VEC; ++v) {
                const float g = d[j][v] + y[v];
                y[v] = a[j][v] * g;
                o1[v] = w[j][v] * g;
                o2[v] = y[v] * xv[j][v];
                if constexpr (PREACT) o2[v] *= dz[j][v];
            }
            if (mine && (ri.valid >> j & 1)) {
                stv<VEC>(dx + first + ro.off[j], o1);
                stv<VEC>(dla + first + ro.off[j], o2);
            }
            if (PACKED && (ri.start >> j & 1)) {
                const int64_t n = __shfl_sync(0xffffffffu, ri.n, j);
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
        float dz;
        if (f.preact) gate_of<true>(f, la[b * n + c], a, w, dz);
        else gate_of<false>(f, la[b * n + c], a, w, dz);
        y = fmaf(a, state[slot * n + c], w * ldf(x + b * n + c));
        state[slot * n + c] = y;
    }
    stf(h + b * n + c, y);
}

GateForm form(const ScanProblem& p) { return GateForm{p.preact, p.leak, p.inv_tau}; }

// Blocks per cluster: as many as the SMs hold at once (`slots`) where the sequences and channel tiles alone do not
// fill them, but no more than there are row tiles. A grid that just exceeds the slots would run a second, nearly
// empty wave.
int cluster_size(int64_t groups, int64_t L, int tile, int64_t slots) {
    int64_t cl = slots / groups;
    const int64_t tiles = cdiv(L, tile);
    cl = cl < tiles ? cl : tiles;
    return int(cl < 1 ? 1 : cl < kMaxCluster ? cl : kMaxCluster);
}

constexpr int kSms = 148;

template <int VEC>
size_t smem_of(int cl, int stage_bytes) {
    return (cl > 1 ? size_t(2) * cl * 32 * VEC * sizeof(float2) : 0) + size_t(2) * kWarps * stage_bytes;
}

template <typename K, typename... Args>
gla_status launch_clusters(const char* name, K kernel, int64_t groups, int cl, size_t smem, cudaStream_t s, Args... args) {
    if (groups * cl > (int64_t(1) << 31) - 1) return GLA_ERR_UNSUPPORTED;
    if (cl > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return GLA_ERR_CUDA;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
        return GLA_ERR_CUDA;
    launch_begin(name, s);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(groups * cl));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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

constexpr int kFwdRows = 8;
constexpr int kFwdBlocks = 3, kBwdBlocks = 2;  // blocks per SM

template <typename T, int VEC, bool PACKED, bool PREACT>
gla_status fwd_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                     void* h, float* hT, float* seg, cudaStream_t s) {
    const int64_t groups = (PACKED ? p.H : p.B * p.H) * cdiv(p.D, 32 * VEC);
    const int cl = cluster_size(groups, p.L, kWarps * kFwdRows, kSms * kFwdBlocks);
    return launch_clusters("scan_fwd", k_scan_fwd<T, VEC, PACKED, PREACT, kFwdRows>, groups, cl,
                           smem_of<VEC>(cl, kFwdStage<T, VEC, kFwdRows>), s, p, form(p), cl, static_cast<const T*>(x),
                           la, cu, h0, static_cast<T*>(h), hT, seg);
}

template <typename T, int VEC, bool PACKED, bool PREACT>
gla_status bwd_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                     const void* dh, const float* dhT, void* dx, float* dla, float* dh0, const float* seg,
                     cudaStream_t s) {
    const int64_t groups = (PACKED ? p.H : p.B * p.H) * cdiv(p.D, 32 * VEC);
    const int cl = cluster_size(groups, p.L, kSeg, kSms * kBwdBlocks);
    return launch_clusters("scan_bwd", k_scan_bwd<T, VEC, PACKED, PREACT>, groups, cl,
                           smem_of<VEC>(cl, kBwdStage<T, VEC, kSeg / kWarps>), s, p, form(p), cl,
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

// Calls fn(type tag, channels a lane, packed, pre-activation) with compile-time values: two channels a lane where the
// rows' pairs are aligned (an even width), else one.
template <typename F>
gla_status dispatch(const ScanProblem& p, F fn) {
    const auto by_form = [&](auto type, auto vec) {
        if (p.packed) return p.preact ? fn(type, vec, std::true_type{}, std::true_type{})
                                      : fn(type, vec, std::true_type{}, std::false_type{});
        return p.preact ? fn(type, vec, std::false_type{}, std::true_type{})
                        : fn(type, vec, std::false_type{}, std::false_type{});
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    if (p.bf16) return p.D % 2 == 0 ? by_form(__nv_bfloat16{}, Two{}) : by_form(__nv_bfloat16{}, One{});
    return p.D % 2 == 0 ? by_form(float{}, Two{}) : by_form(float{}, One{});
}

}  // namespace

size_t scan_workspace(const ScanProblem& p, Arena& a) {
    (void)a.take<float>(size_t((p.packed ? p.H : p.B * p.H) * cdiv(p.L, kSeg) * p.D));
    return a.used;
}

gla_status scan_fwd(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0, void* h,
                    float* hT, float* seg, cudaStream_t s) {
    return dispatch(p, [&](auto type, auto vec, auto packed, auto preact) {
        return fwd_typed<decltype(type), vec(), packed(), preact()>(p, x, la, cu, h0, h, hT, seg, s);
    });
}

gla_status scan_bwd(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                    const void* dh, const float* dhT, void* dx, float* dla, float* dh0, float* seg, bool reuse,
                    cudaStream_t s) {
    if (!reuse) {
        const gla_status st = scan_fwd(p, x, la, cu, h0, nullptr, nullptr, seg, s);
        if (st != GLA_OK) return st;
    }
    return dispatch(p, [&](auto type, auto vec, auto packed, auto preact) {
        return bwd_typed<decltype(type), vec(), packed(), preact()>(p, x, la, cu, h0, dh, dhT, dx, dla, dh0, seg, s);
    });
}

gla_status scan_step(const ScanProblem& p, const void* x, const float* la, const int32_t* slots, int64_t pool,
                     float* state, void* h, cudaStream_t s) {
    return p.bf16 ? step_typed<__nv_bfloat16>(p, x, la, slots, pool, state, h, s)
                  : step_typed<float>(p, x, la, slots, pool, state, h, s);
}

}  // namespace gla
