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

// ---- cluster primitives -----------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// ---- one or two adjacent channels -------------------------------------------------------
// Two channels are one packed operand: the packed fp32 instructions do both for one issue slot, and issue slots are
// what these kernels run out of first (a wide batch spends about as long issuing as it does on memory).
template <int VEC>
struct VecOf {
    using type = float;
};
template <>
struct VecOf<2> {
    using type = float2;
};
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 vfma(float2 a, float2 b, float2 c) { return fma2(a, b, c); }
__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float2 vmul(float2 a, float2 b) { return mul2(a, b); }
__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ float2 vadd(float2 a, float2 b) { return add2(a, b); }
template <typename V>
__device__ __forceinline__ V vset(float x) {
    if constexpr (sizeof(V) == 8) return make_float2(x, x);
    else return x;
}
// f of each channel
template <typename F>
__device__ __forceinline__ float each(F f, float a) { return f(a); }
template <typename F>
__device__ __forceinline__ float2 each(F f, float2 a) { return make_float2(f(a.x), f(a.y)); }
template <typename F>
__device__ __forceinline__ float each(F f, float a, float b) { return f(a, b); }
template <typename F>
__device__ __forceinline__ float2 each(F f, float2 a, float2 b) { return make_float2(f(a.x, b.x), f(a.y, b.y)); }
template <typename F>
__device__ __forceinline__ float each(F f, float a, float b, float c) { return f(a, b, c); }
template <typename F>
__device__ __forceinline__ float2 each(F f, float2 a, float2 b, float2 c) {
    return make_float2(f(a.x, b.x, c.x), f(a.y, b.y, c.y));
}

template <typename V>
__device__ __forceinline__ V ldv(const float* p) { return *reinterpret_cast<const V*>(p); }
template <typename V>
__device__ __forceinline__ V ldv(const __nv_bfloat16* p) {
    if constexpr (sizeof(V) == 8) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
    else return __bfloat162float(*p);
}
template <typename V>
__device__ __forceinline__ void stv(float* p, V y) { *reinterpret_cast<V*>(p) = y; }
template <typename V>
__device__ __forceinline__ void stv(__nv_bfloat16* p, V y) {
    if constexpr (sizeof(V) == 8) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(y.x, y.y);
    else *p = __float2bfloat16_rn(y);
}

// ---- gates --------------------------------------------------------------------------------
// The library's expf / expm1f / log1pf come to about 60 instructions an element, four times what the memory
// bandwidth leaves room for; these take 13 (a and w) and 12 (log alpha from z). Accuracies in units of u = 2^-24.

// a = e^la and 1 - a for la <= 0. Near 0, where a multiplies up over many steps and 1 - a must keep its relative
// precision: 1 - a = -la q(la) with q = (e^x - 1) / x as a polynomial fitted at the Chebyshev nodes of [-1/2, 0]
// (relative error 3e-9), so 1 - a is within 3 u and a = 1 - (1 - a) correctly rounded from it. Below -1/2 (a < 0.61,
// no long products): the ex2 instruction, within (4 + |la|) u.
template <typename V>
__device__ __forceinline__ void decay_of(V la, V& a, V& one_minus_a) {
    V q = vfma(vset<V>(-0.00112340425f), la, vset<V>(-0.00818961393f));
    q = vfma(q, la, vset<V>(-0.0416300744f));
    q = vfma(q, la, vset<V>(-0.166662425f));
    q = vfma(q, la, vset<V>(-0.499999821f));
    q = vfma(q, la, vset<V>(-1.f));
    const V m = vmul(la, q);
    const V e = each([](float t) { return tc::exp2_ftz(t); }, vmul(la, vset<V>(tc::kLog2e)));
    const V am = vfma(m, vset<V>(-1.f), vset<V>(1.f)), me = vfma(e, vset<V>(-1.f), vset<V>(1.f));
    const auto near = [](float l, float yes, float no) { return fabsf(l) < 0.5f ? yes : no; };
    a = each(near, la, am, e);
    one_minus_a = each(near, la, m, me);
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// logsigmoid(z) = min(z, 0) - log(1 + t), t = e^-|z| in [0, 1], with log(1 + t) = 2 atanh(s), s = t / (2 + t) <= 1/3:
// atanh(s) / s as a polynomial in s^2 fitted at the Chebyshev nodes of [0, 1/9] (relative error 8e-9). Small t
// keeps its relative precision, (8 + |z|) u in all.
template <typename V>
__device__ __forceinline__ V logsigmoid_series(V z, V& t) {
    t = each([](float x) { return tc::exp2_ftz(-fabsf(x) * tc::kLog2e); }, z);
    const V s = vmul(t, each([](float x) { return rcp(x); }, vadd(t, vset<V>(2.f)))), y = vmul(s, s);
    V q = vfma(vset<V>(0.140788898f), y, vset<V>(0.139825791f));
    q = vfma(q, y, vset<V>(0.200122982f));
    q = vfma(q, y, vset<V>(0.333331615f));
    q = vfma(q, y, vset<V>(1.f));
    return vfma(vmul(s, vset<V>(-2.f)), q, each([](float x) { return fminf(x, 0.f); }, z));
}

// a_t and w_t from the gate argument; for a pre-activation also dlog a / dz = sigmoid(-z) / tau
template <bool PREACT, bool LEAK, typename V>
__device__ __forceinline__ void gate_of(float inv_tau, V g, V& a, V& w, V& dz) {
    V la = g;
    if constexpr (PREACT) {
        V t;
        la = vmul(logsigmoid_series(g, t), vset<V>(inv_tau));
        const V r = each([](float x) { return rcp(x); }, vadd(t, vset<V>(1.f)));
        dz = vmul(each([](float x, float yes, float no) { return x < 0.f ? yes : no; }, g, r, vmul(t, r)), vset<V>(inv_tau));
    }
    decay_of(la, a, w);
    if constexpr (!LEAK) w = vset<V>(1.f);
}

// Maps of packed rows that hold a sequence's start forget everything in front of it, whatever that is: an infinity
// or a NaN of one sequence must not reach the next through 0 * inf. Such a map has the factor -0, which no product
// of decays gives and which products keep.
constexpr float kForget = -0.f;
template <bool PACKED>
__device__ __forceinline__ bool forgets(float m) { return PACKED && __float_as_uint(m) == 0x80000000u; }
template <bool PACKED, typename V>
__device__ __forceinline__ V join(V m, V s, V u) {
    const V y = vfma(m, s, u);
    if constexpr (!PACKED) return y;
    else return each([](float f, float yes, float no) { return forgets<true>(f) ? yes : no; }, m, u, y);
}
template <bool PACKED, typename V>
__device__ __forceinline__ V join(V m, V f) {
    const V y = vmul(m, f);
    if constexpr (!PACKED) return y;
    else return each([](float f2, float yes, float no) { return forgets<true>(f2) ? yes : no; }, m, m, y);
}

// The map of a span of rows, for one lane's channels.
template <typename V>
struct alignas(2 * sizeof(V)) Map {
    V a, u;
};

// Put a map into the same place of block `rank`'s shared memory and count it on that block's barrier.
template <typename V>
__device__ __forceinline__ void send(Map<V>* place, uint64_t* bar, uint32_t rank, Map<V> m) {
    if constexpr (sizeof(V) == 8) {
        asm volatile(
            "{\n\t.reg .b32 a, b;\n\t"
            "mapa.shared::cluster.u32 a, %0, %2;\n\t"
            "mapa.shared::cluster.u32 b, %1, %2;\n\t"
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [a], {%3, %4, %5, %6}, [b];\n\t}" ::"r"(
                tc::smem_u32(place)),
            "r"(tc::smem_u32(bar)), "r"(rank), "f"(m.a.x), "f"(m.a.y), "f"(m.u.x), "f"(m.u.y)
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .b32 a, b;\n\t"
            "mapa.shared::cluster.u32 a, %0, %2;\n\t"
            "mapa.shared::cluster.u32 b, %1, %2;\n\t"
            "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [a], {%3, %4}, [b];\n\t}" ::"r"(
                tc::smem_u32(place)),
            "r"(tc::smem_u32(bar)), "r"(rank), "f"(m.a), "f"(m.u)
            : "memory");
    }
}

// The blocks' exchange of one cluster. Each round every block sends its rows' map to all blocks; a block waits for the
// cl maps on its own barrier, of which there are two for alternate rounds. A map of round i + 2 cannot overtake the
// reading of round i's: its sender has waited for this block's map of round i + 1, which left after all of this
// block's warps were done with round i.
template <typename V>
struct Exchange {
    Map<V>* maps;   // [2][cl][32]
    uint64_t* bar;  // [2]
    int* abort;
    int* err;
    int cl, rank, rounds;
    __device__ __forceinline__ uint32_t bytes() const { return uint32_t(cl * 32 * sizeof(Map<V>)); }
    __device__ __forceinline__ void begin() {
        if (cl == 1) return;
        if (threadIdx.x == 0) {
            *abort = 0;
            for (int i = 0; i < 2; ++i) tc::mbar_init(bar + i, 1);
            tc::fence_barrier_init();
            for (int i = 0; i < 2; ++i) tc::mbar_arrive_expect_tx(bar + i, bytes());
        }
        __syncthreads();
        cluster_arrive();  // completed by ready(): every block's barriers exist before any block sends
    }
    __device__ __forceinline__ void ready() const {
        if (cl > 1) cluster_wait();
    }
    // one warp sends its block's map of round `it`
    __device__ __forceinline__ void put(int it, Map<V> m) const {
        const int par = it & 1;
        for (int q = 0; q < cl; ++q) send(maps + (par * cl + rank) * 32 + (threadIdx.x & 31), bar + par, uint32_t(q), m);
    }
    // every thread waits for the maps of round `it`
    __device__ __forceinline__ const Map<V>* get(int it) const {
        const int par = it & 1;
        (void)tc::mbar_wait(bar + par, uint32_t(it >> 1) & 1u, err, abort);
        if (threadIdx.x == 0 && it + 2 < rounds) tc::mbar_arrive_expect_tx(bar + par, bytes());
        return maps + par * cl * 32 + (threadIdx.x & 31);
    }
    // no block leaves while another may still send to it
    __device__ __forceinline__ void end() const {
        if (cl > 1) {
            cluster_arrive();
            cluster_wait();
        }
    }
};

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
template <typename V>
__device__ __forceinline__ V state_of(const float* __restrict__ h, int64_t n, const ScanProblem& p, int64_t head,
                                      int64_t c) {
    return h ? ldv<V>(h + (n * p.H + head) * p.D + c) : vset<V>(0.f);
}

// Empty sequences have no row that could write their end: out[n] = in[n] (or 0), spread over the cluster's warps.
template <typename V>
__device__ __forceinline__ void copy_empty(const int32_t* __restrict__ cu, const ScanProblem& p, int64_t head, int64_t c,
                                           bool mine, const float* __restrict__ in, float* __restrict__ out, int first,
                                           int stride, int lane) {
    if (!out) return;
    const int B = int(p.B);
    for (int n0 = first * 32; n0 < B; n0 += stride * 32) {
        const int n = n0 + lane;
        uint32_t m = __ballot_sync(0xffffffffu, n < B && cu[n < B ? n : 0] >= cu[n < B ? n + 1 : 0]);
        while (m) {
            const int64_t e = n0 + __ffs(m) - 1;
            m &= m - 1;
            if (mine) stv(out + (e * p.H + head) * p.D + c, state_of<V>(in, e, p, head, c));
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
template <typename V, typename T>
__device__ __forceinline__ V take_row(const T* st, const T* src, uint32_t off, int j) {
    constexpr int VEC = int(sizeof(V) / 4);
    if constexpr (kStaged<T, VEC>) return ldv<V>(st + j * 32 * VEC);
    else return ldv<V>(src + off);
}

// bytes a warp's stage takes
template <typename T, int VEC, int ROWS>
constexpr int kFwdStage = ROWS * 32 * VEC * int(4 + sizeof(T));
template <typename T, int VEC, int ROWS>
constexpr int kBwdStage = ROWS * 32 * VEC * int(4 + 2 * sizeof(T));

// What a block is to do and where its lanes' data are.
template <typename T, int VEC, int ROWS, int STAGE>
struct Place {
    int lane, warp, rank, cl;
    int64_t lead, c, cc, L, D;  // sequence or head; channel, and the nearest one that exists
    bool mine;
    char* stages;
    __device__ __forceinline__ Place(const ScanProblem& p, int cl_, char* stages_) : cl(cl_), L(p.L), D(p.D) {
        constexpr int CW = 32 * VEC;
        lane = threadIdx.x & 31;
        warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);
        rank = cl > 1 ? int(cluster_rank()) : 0;
        const int64_t tiles = cdiv(p.D, CW), id = blockIdx.x / cl;
        lead = id / tiles;
        c = (id % tiles) * CW + lane * VEC;
        mine = c < p.D;
        cc = mine ? c : p.D - VEC;
        stages = stages_ + warp * 2 * STAGE;
    }
    __device__ __forceinline__ int64_t row(int r) const { return (int64_t(r) * cl + rank) * (kWarps * ROWS) + warp * ROWS; }
    __device__ __forceinline__ int64_t first(int64_t t) const { return (lead * L + (t < L ? t : L - 1)) * D + cc; }
    __device__ __forceinline__ float* gates(int par) const {
        return reinterpret_cast<float*>(stages + par * STAGE) + lane * VEC;
    }
    // k-th tensor of the element type
    __device__ __forceinline__ T* elems(int par, int k) const {
        return reinterpret_cast<T*>(stages + par * STAGE + ROWS * 32 * VEC * 4) + k * ROWS * 32 * VEC + lane * VEC;
    }
};

// ---- forward ------------------------------------------------------------------------------
// Grid: (sequence or head) x channel tile x cluster of `cl` blocks. Rows of round r and block q: from
// (r cl + q) kWarps ROWS.
template <typename T, int VEC, bool PACKED, bool PREACT, bool LEAK, int ROWS>
__global__ void __launch_bounds__(kThreads, 2)
    k_scan_fwd(ScanProblem p, int cl, const T* __restrict__ x, const float* __restrict__ la,
               const int32_t* __restrict__ cu, const float* __restrict__ h0, T* __restrict__ h, float* __restrict__ hT,
               float* __restrict__ seg, int* err) {
    using V = typename VecOf<VEC>::type;
    constexpr int STAGE = kFwdStage<T, VEC, ROWS>;
    __shared__ Map<V> agg[2][kWarps][32];
    __shared__ uint64_t bar[2];
    __shared__ int abort_flag;
    extern __shared__ __align__(16) char dyn[];  // the cluster's maps, then the warps' stages
    const Place<T, VEC, ROWS, STAGE> at(p, cl, dyn + (cl > 1 ? 2 * cl * 32 * sizeof(Map<V>) : 0));
    const int lane = at.lane, warp = at.warp, rank = at.rank;
    const int64_t lead = at.lead, c = at.c, cc = at.cc, head = PACKED ? lead : 0;
    const bool mine = at.mine;
    const int rounds = int(cdiv(p.L, int64_t(kWarps * ROWS) * cl));
    Exchange<V> ex{reinterpret_cast<Map<V>*>(dyn), bar, &abort_flag, err, cl, rank, rounds};
    const auto stage = [&](int r) {
        const int64_t t = at.row(r), i = at.first(t);
        const RowOffsets<ROWS> ro(p.L - t, p.D);
        stage_rows<float, VEC, ROWS>(at.gates(r & 1), la + i, ro);
        stage_rows<T, VEC, ROWS>(at.elems(r & 1, 0), x + i, ro);
    };
    stage(0);
    copies_commit();
    ex.begin();
    if constexpr (PACKED) copy_empty<V>(cu, p, head, c, mine, h0, hT, rank * kWarps + warp, cl * kWarps, lane);
    V carry = vset<V>(0.f);
    if (!PACKED && h0) carry = ldv<V>(h0 + lead * p.D + cc);
    ex.ready();
    const int64_t nseg = cdiv(p.L, kSeg);
    for (int r = 0; r < rounds; ++r) {
        const int par = r & 1;
        const int64_t t0 = at.row(r), first = at.first(t0);
        const RowOffsets<ROWS> ro(p.L - t0, p.D);
        if (r + 1 < rounds) stage(r + 1);
        copies_commit();
        copies_wait<1>();
        RowInfo ri{0, 0, 0, 0};
        if constexpr (PACKED) ri = rows_packed<ROWS>(cu, int(p.B), t0, p.L, lane);
        else ri.valid = t0 + ROWS <= p.L ? ~0u : t0 < p.L ? (1u << (p.L - t0)) - 1 : 0u;
        V a[ROWS], b[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            V w, dz;
            gate_of<PREACT, LEAK>(p.inv_tau, ldv<V>(at.gates(par) + j * 32 * VEC), a[j], w, dz);
            b[j] = take_row<V>(at.elems(par, 0), x + first, ro.off[j], j);
            if constexpr (LEAK) b[j] = vmul(b[j], w);
        }
        constexpr uint32_t kAll = (1u << ROWS) - 1;
        if ((ri.valid & kAll) != kAll) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j)
                if (!(ri.valid >> j & 1)) a[j] = vset<V>(1.f), b[j] = vset<V>(0.f);
        }
        Map<V> own{vset<V>(1.f), vset<V>(0.f)};
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (PACKED && (ri.start >> j & 1)) own.u = state_of<V>(h0, __shfl_sync(0xffffffffu, ri.n, j), p, head, cc);
            own.a = vmul(own.a, a[j]);
            own.u = vfma(a[j], own.u, b[j]);
        }
        if (PACKED && ri.start) own.a = vset<V>(kForget);
        agg[par][warp][lane] = own;
        __syncthreads();
        Map<V> pre{vset<V>(1.f), vset<V>(0.f)};  // of the block's rows in front of this warp's
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w) {
            if (w < warp) {
                const Map<V> m = agg[par][w][lane];
                pre = Map<V>{join<PACKED>(m.a, pre.a), join<PACKED>(m.a, pre.u, m.u)};
            }
        }
        V in = carry;  // state entering the block's rows
        if (cl > 1) {
            if (warp == kWarps - 1) ex.put(r, Map<V>{join<PACKED>(own.a, pre.a), join<PACKED>(own.a, pre.u, own.u)});
            const Map<V>* m = ex.get(r);
            for (int q = 0; q < cl; ++q) {
                if (q == rank) in = carry;
                carry = join<PACKED>(m[q * 32].a, carry, m[q * 32].u);
            }
        } else {
            Map<V> t = pre;
            for (int w = warp; w < kWarps; ++w) {
                const Map<V> m = agg[par][w][lane];
                t = Map<V>{join<PACKED>(m.a, t.a), join<PACKED>(m.a, t.u, m.u)};
            }
            carry = join<PACKED>(t.a, in, t.u);
        }
        V s = join<PACKED>(pre.a, in, pre.u);
        if (seg && mine && t0 < p.L && t0 % kSeg == 0) stv(seg + (lead * nseg + t0 / kSeg) * p.D + c, s);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (PACKED && (ri.start >> j & 1)) s = state_of<V>(h0, __shfl_sync(0xffffffffu, ri.n, j), p, head, cc);
            s = vfma(a[j], s, b[j]);
            if (h && mine && (ri.valid >> j & 1)) stv(h + first + ro.off[j], s);
            if (PACKED && (ri.end >> j & 1)) {
                const int64_t n = __shfl_sync(0xffffffffu, ri.n, j);
                if (hT && mine) stv(hT + (n * p.H + head) * p.D + c, s);
            }
        }
        // rows behind the last one leave the state as it is, so the warp with the last row holds hT
        if (!PACKED && hT && mine && t0 < p.L && t0 + ROWS >= p.L) stv(hT + lead * p.D + c, s);
    }
    ex.end();
}

// ---- backward -----------------------------------------------------------------------------
// Rounds, blocks and warps as in the forward, from the last round to the first. The states inside a block's rows
// are recomputed in fp32 from the state that enters them (seg).
template <typename T, int VEC, bool PACKED, bool PREACT, bool LEAK>
__global__ void __launch_bounds__(kThreads, 2)
    k_scan_bwd(ScanProblem p, int cl, const T* __restrict__ x, const float* __restrict__ la,
               const int32_t* __restrict__ cu, const float* __restrict__ h0, const T* __restrict__ dh,
               const float* __restrict__ dhT, T* __restrict__ dx, float* __restrict__ dla, float* __restrict__ dh0,
               const float* __restrict__ seg, int* err) {
    using V = typename VecOf<VEC>::type;
    constexpr int ROWS = kSeg / kWarps, STAGE = kBwdStage<T, VEC, ROWS>;
    __shared__ Map<V> agg[2][kWarps][32];
    __shared__ V aggy[2][kWarps][32];
    __shared__ uint64_t bar[2];
    __shared__ int abort_flag;
    extern __shared__ __align__(16) char dyn[];  // the cluster's maps, then the warps' stages
    const Place<T, VEC, ROWS, STAGE> at(p, cl, dyn + (cl > 1 ? 2 * cl * 32 * sizeof(Map<V>) : 0));
    const int lane = at.lane, warp = at.warp, rank = at.rank;
    const int64_t lead = at.lead, c = at.c, cc = at.cc, head = PACKED ? lead : 0;
    const bool mine = at.mine;
    const int rounds = int(cdiv(p.L, int64_t(kSeg) * cl));
    Exchange<V> ex{reinterpret_cast<Map<V>*>(dyn), bar, &abort_flag, err, cl, rank, rounds};
    const auto stage = [&](int r) {
        const int64_t t = at.row(r), i = at.first(t);
        const RowOffsets<ROWS> ro(p.L - t, p.D);
        stage_rows<float, VEC, ROWS>(at.gates(r & 1), la + i, ro);
        stage_rows<T, VEC, ROWS>(at.elems(r & 1, 0), x + i, ro);
        stage_rows<T, VEC, ROWS>(at.elems(r & 1, 1), dh + i, ro);
    };
    stage(rounds - 1);
    copies_commit();
    ex.begin();
    if constexpr (PACKED) copy_empty<V>(cu, p, head, c, mine, dhT, dh0, rank * kWarps + warp, cl * kWarps, lane);
    V carry = vset<V>(0.f);  // y of the row behind the round's last
    if (!PACKED && dhT) carry = ldv<V>(dhT + lead * p.D + cc);
    ex.ready();
    const int64_t nseg = cdiv(p.L, kSeg);
    for (int it = 0; it < rounds; ++it) {
        const int r = rounds - 1 - it, par = r & 1;
        const int64_t t0 = at.row(r), first = at.first(t0), tile = int64_t(r) * cl + rank;
        const RowOffsets<ROWS> ro(p.L - t0, p.D);
        V s = ldv<V>(seg + (lead * nseg + (tile < nseg ? tile : nseg - 1)) * p.D + cc);  // entering the block's rows
        if (r > 0) stage(r - 1);
        copies_commit();
        copies_wait<1>();
        RowInfo ri{0, 0, 0, 0};
        if constexpr (PACKED) ri = rows_packed<ROWS>(cu, int(p.B), t0, p.L, lane);
        else ri.valid = t0 + ROWS <= p.L ? ~0u : t0 < p.L ? (1u << (p.L - t0)) - 1 : 0u;
        V a[ROWS], w[ROWS], xv[ROWS], d[ROWS], dz[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            gate_of<PREACT, LEAK>(p.inv_tau, ldv<V>(at.gates(par) + j * 32 * VEC), a[j], w[j], dz[j]);
            xv[j] = take_row<V>(at.elems(par, 0), x + first, ro.off[j], j);
            d[j] = take_row<V>(at.elems(par, 1), dh + first, ro.off[j], j);
        }
        constexpr uint32_t kAll = (1u << ROWS) - 1;
        if ((ri.valid & kAll) != kAll) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                if (!(ri.valid >> j & 1)) {
                    a[j] = vset<V>(1.f);
                    w[j] = xv[j] = d[j] = vset<V>(0.f);
                }
            }
        }
        Map<V> own{vset<V>(1.f), vset<V>(0.f)};
        V Y = vset<V>(0.f);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (PACKED && (ri.start >> j & 1)) own.u = state_of<V>(h0, __shfl_sync(0xffffffffu, ri.n, j), p, head, cc);
            own.a = vmul(own.a, a[j]);
            own.u = vfma(a[j], own.u, LEAK ? vmul(w[j], xv[j]) : xv[j]);
        }
#pragma unroll
        for (int j = ROWS - 1; j >= 0; --j) {
            if (PACKED && (ri.end >> j & 1))  // the gradient of the last state enters here, in place of the next row's
                d[j] = vadd(d[j], state_of<V>(dhT, __shfl_sync(0xffffffffu, ri.n, j), p, head, cc));
            Y = vmul(a[j], vadd(d[j], Y));
            if (PACKED && (ri.start >> j & 1)) Y = vset<V>(0.f);
        }
        // forgetting holds in both directions: u and Y carry what the warp's other rows hold
        if (PACKED && ri.start) own.a = vset<V>(kForget);
        agg[par][warp][lane] = own;
        aggy[par][warp][lane] = Y;
        __syncthreads();
        Map<V> post{vset<V>(1.f), vset<V>(0.f)};  // the map (of y) of the block's rows behind this warp's
#pragma unroll
        for (int q = 0; q < kWarps - 1; ++q) {
            if (q < warp) {
                const Map<V> m = agg[par][q][lane];
                s = join<PACKED>(m.a, s, m.u);
            }
        }
#pragma unroll
        for (int q = kWarps - 1; q > 0; --q) {
            if (q > warp) {
                const V m = agg[par][q][lane].a;
                post = Map<V>{join<PACKED>(m, post.a), join<PACKED>(m, post.u, aggy[par][q][lane])};
            }
        }
        V in = carry;
        if (cl > 1) {
            if (warp == 0) ex.put(it, Map<V>{join<PACKED>(own.a, post.a), join<PACKED>(own.a, post.u, Y)});
            const Map<V>* m = ex.get(it);
            for (int q = cl - 1; q >= 0; --q) {
                if (q == rank) in = carry;
                carry = join<PACKED>(m[q * 32].a, carry, m[q * 32].u);
            }
        } else {
            Map<V> t = post;
            for (int q = warp; q >= 0; --q) {
                const V m = agg[par][q][lane].a;
                t = Map<V>{join<PACKED>(m, t.a), join<PACKED>(m, t.u, aggy[par][q][lane])};
            }
            carry = join<PACKED>(t.a, in, t.u);
        }
        V y = join<PACKED>(post.a, in, post.u);
        // xv becomes what dlog a_t multiplies: h_{t-1}, less x_t where the input's weight is 1 - a
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if (PACKED && (ri.start >> j & 1)) s = state_of<V>(h0, __shfl_sync(0xffffffffu, ri.n, j), p, head, cc);
            const V xj = xv[j];
            xv[j] = LEAK ? vfma(xj, vset<V>(-1.f), s) : s;
            s = vfma(a[j], s, LEAK ? vmul(w[j], xj) : xj);
        }
#pragma unroll
        for (int j = ROWS - 1; j >= 0; --j) {
            const V g = vadd(d[j], y);
            y = vmul(a[j], g);
            if (mine && (ri.valid >> j & 1)) {
                stv(dx + first + ro.off[j], LEAK ? vmul(w[j], g) : g);
                const V o = vmul(y, xv[j]);
                stv(dla + first + ro.off[j], PREACT ? vmul(o, dz[j]) : o);
            }
            if (PACKED && (ri.start >> j & 1)) {
                const int64_t n = __shfl_sync(0xffffffffu, ri.n, j);
                if (dh0 && mine) stv(dh0 + (n * p.H + head) * p.D + c, y);
                y = vset<V>(0.f);
            }
        }
        if (!PACKED && dh0 && mine && t0 == 0) stv(dh0 + lead * p.D + c, y);
    }
    ex.end();
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
__global__ void __launch_bounds__(kStepThreads) k_scan_step(ScanProblem p, const T* __restrict__ x,
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
        float a, w, dz;
        const float g = la[b * n + c], xv = ldf(x + b * n + c);
        if (p.preact) gate_of<true, true>(p.inv_tau, g, a, w, dz);
        else gate_of<false, true>(p.inv_tau, g, a, w, dz);
        y = fmaf(a, state[slot * n + c], p.leak ? w * xv : xv);
        state[slot * n + c] = y;
    }
    stf(h + b * n + c, y);
}

template <typename V>
size_t smem_of(int cl, int stage_bytes) {
    return (cl > 1 ? size_t(2) * cl * 32 * sizeof(Map<V>) : 0) + size_t(2) * kWarps * stage_bytes;
}

// How many clusters of each size the device holds at once, per kernel: a cluster sits inside one GPC, so large ones
// leave some SMs empty. Asked once per kernel (the answer depends on nothing else).
struct ClusterFit {
    int fit[kMaxCluster + 1] = {};
};
template <typename K>
ClusterFit ask_fit(K kernel, size_t (*smem)(int, int), int stage_bytes) {
    ClusterFit f;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem(kMaxCluster, stage_bytes))) !=
            cudaSuccess)
        return f;
    for (int cl = 1; cl <= kMaxCluster; ++cl) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(cl));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem(cl, stage_bytes);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = unsigned(cl);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) f.fit[cl] = n;
    }
    return f;
}

// Blocks per cluster. A block's time goes by its rounds, and clusters that do not fit at once run in further waves:
// the least waves x rounds, and of those the smallest cluster.
int cluster_size(const ClusterFit& f, int64_t groups, int64_t L, int tile) {
    const int64_t tiles = cdiv(L, tile);
    int best = 1;
    int64_t cost = INT64_MAX;
    for (int cl = 1; cl <= kMaxCluster; ++cl) {
        if (f.fit[cl] < 1 || cl > tiles) continue;
        const int64_t c = cdiv(groups, int64_t(f.fit[cl])) * cdiv(tiles, int64_t(cl));
        if (c < cost) cost = c, best = cl;
    }
    return best;
}

template <typename K, typename... Args>
gla_status launch_clusters(const char* name, K kernel, const ClusterFit& f, int64_t groups, int cl, size_t smem,
                           cudaStream_t s, Args... args) {
    if (f.fit[1] < 1) return GLA_ERR_CUDA;
    if (groups * cl > (int64_t(1) << 31) - 1) return GLA_ERR_UNSUPPORTED;
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

template <typename T, int VEC, bool PACKED, bool PREACT, bool LEAK>
gla_status fwd_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                     void* h, float* hT, float* seg, cudaStream_t s) {
    const int64_t groups = (PACKED ? p.H : p.B * p.H) * cdiv(p.D, 32 * VEC);
    using V = typename VecOf<VEC>::type;
    const auto kernel = k_scan_fwd<T, VEC, PACKED, PREACT, LEAK, kFwdRows>;
    constexpr int stage = kFwdStage<T, VEC, kFwdRows>;
    static const ClusterFit fit = ask_fit(kernel, smem_of<V>, stage);
    const int cl = cluster_size(fit, groups, p.L, kWarps * kFwdRows);
    return launch_clusters("scan_fwd", kernel, fit, groups, cl, smem_of<V>(cl, stage), s, p, cl, static_cast<const T*>(x), la, cu, h0,
                           static_cast<T*>(h), hT, seg, device_error_word());
}

template <typename T, int VEC, bool PACKED, bool PREACT, bool LEAK>
gla_status bwd_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                     const void* dh, const float* dhT, void* dx, float* dla, float* dh0, const float* seg,
                     cudaStream_t s) {
    const int64_t groups = (PACKED ? p.H : p.B * p.H) * cdiv(p.D, 32 * VEC);
    using V = typename VecOf<VEC>::type;
    const auto kernel = k_scan_bwd<T, VEC, PACKED, PREACT, LEAK>;
    constexpr int stage = kBwdStage<T, VEC, kSeg / kWarps>;
    static const ClusterFit fit = ask_fit(kernel, smem_of<V>, stage);
    const int cl = cluster_size(fit, groups, p.L, kSeg);
    return launch_clusters("scan_bwd", kernel, fit, groups, cl, smem_of<V>(cl, stage), s, p, cl, static_cast<const T*>(x),
                           la, cu, h0, static_cast<const T*>(dh), dhT, static_cast<T*>(dx), dla, dh0, seg,
                           device_error_word());
}

template <typename T>
gla_status step_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* slots, int64_t pool,
                      float* state, void* h, cudaStream_t s) {
    const dim3 grid(unsigned(cdiv(p.H * p.D, kStepThreads)), unsigned(p.B));
    GLA_LAUNCH("scan_step", k_scan_step<T>, grid, kStepThreads, 0, s, p, static_cast<const T*>(x), la, slots,
               pool, state, static_cast<T*>(h), device_error_word());
    return GLA_OK;
}

// Calls fn(type tag, channels a lane, packed, pre-activation, leak) with compile-time values: two channels a lane where
// the rows' pairs are aligned (an even width), else one.
template <typename F>
gla_status dispatch(const ScanProblem& p, F fn) {
    const auto flag = [](bool b, auto then) { return b ? then(std::true_type{}) : then(std::false_type{}); };
    const auto by_form = [&](auto type, auto vec) {
        return flag(p.packed, [&](auto packed) {
            return flag(p.preact, [&](auto preact) {
                return flag(p.leak, [&](auto leak) { return fn(type, vec, packed, preact, leak); });
            });
        });
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
    return dispatch(p, [&](auto type, auto vec, auto packed, auto preact, auto leak) {
        return fwd_typed<decltype(type), vec(), packed(), preact(), leak()>(p, x, la, cu, h0, h, hT, seg, s);
    });
}

gla_status scan_bwd(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                    const void* dh, const float* dhT, void* dx, float* dla, float* dh0, float* seg, bool reuse,
                    cudaStream_t s) {
    if (!reuse) {
        const gla_status st = scan_fwd(p, x, la, cu, h0, nullptr, nullptr, seg, s);
        if (st != GLA_OK) return st;
    }
    return dispatch(p, [&](auto type, auto vec, auto packed, auto preact, auto leak) {
        return bwd_typed<decltype(type), vec(), packed(), preact(), leak()>(p, x, la, cu, h0, dh, dhT, dx, dla, dh0, seg, s);
    });
}

gla_status scan_step(const ScanProblem& p, const void* x, const float* la, const int32_t* slots, int64_t pool,
                     float* state, void* h, cudaStream_t s) {
    return p.bf16 ? step_typed<__nv_bfloat16>(p, x, la, slots, pool, state, h, s)
                  : step_typed<float>(p, x, la, slots, pool, state, h, s);
}

}  // namespace gla
