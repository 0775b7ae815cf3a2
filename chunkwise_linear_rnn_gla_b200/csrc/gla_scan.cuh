// Elementwise gated recurrence (include/gla.h, "elementwise gated recurrence"):
//     h_t = a_t h_{t-1} + w_t x_t,   a_t = e^{log a_t},   w_t = 1 or 1 - a_t.
// One state value per channel: the decay of the layer's gated memory (podcast.app episode page,
// summary: a gated memory updated once per token) without its key dimension.
//
// A step is the affine map s -> a s + b, and maps compose: (a2, b2) o (a1, b1) = (a1 a2, a2 b1 + b2). So a
// sequence is cut into segments that are reduced to one map each, the maps are joined, and every segment
// then runs its steps from the state that enters it. All of this happens on one read of the inputs:
//   warp     8 or 16 rows (steps) x 32 or 64 channels in registers, one or two channels a lane;
//   block    4 or 8 warps, 32 to 128 rows: the warps' maps are joined in shared memory;
//   cluster  up to 16 blocks, 512 to 2048 rows: every block sends its map into the shared memory of all the others
//            (asynchronous stores counted on their mbarriers), and each joins those in front of it.
// A cluster walks the time axis in rounds and carries the state in registers, so a call needs no workspace,
// no flags in memory and no second launch, and its result does not depend on timing.
//
// Floor: 8 (bf16) or 12 (fp32) bytes an element forward, 14 or 20 backward, at the copy bandwidth. Measured (device time,
// inputs larger than L2 in turn): forward 33.7 us at 8 sequences of 2048 steps, width 1024 (134 MB, 4.0 TB/s, floor
// 20.5); forward and backward 101 us at 4 x 2048, width 2048, gate from its pre-activation (floor 41 if the inputs were
// read once; 369 MB moved, 57 us, since the backward reads them again). What is left is the chain of a round: gates,
// maps, the exchange, steps, each waiting for the one before. No resource is full: 43% of the issue slots are taken
// forward and 51% backward, DRAM 37%. Without its loads the forward still takes 32 us.
//
// A boundary between packed sequences is a step whose map forgets: (forget, a h0 + b). In the backward the same
// steps stop the gradient, which walks the maps the other way: with y_t = a_t g_t, g_t = dh_t + y_{t+1}.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "gla_common.cuh"
#include "gla_gate.cuh"
#include "gla_internal.h"
#include "tc_prims.cuh"

namespace gla {
namespace {

constexpr int kSeg = 32;  // rows between the states kept for the backward
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
// Two channels are one packed operand: the packed fp32 instructions do both for one issue slot, so a round's chain has
// fewer of them (35 a channel and step forward, 69 backward).
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
//
// A block in which a wait ran out (abort) sends no more maps, so that the waits of the others run out too; a thread whose
// wait ran out arms no barrier and writes no results from then on. Both keep to the block's barriers and the cluster's,
// and the maps that are still on their way to the block land (with a limit) before it ends.
template <typename V>
struct Exchange {
    Map<V>* maps;   // [2][cl][32]
    uint64_t* bar;  // [2]
    int* abort;
    int* err;
    int cl, rank, rounds;
    long long limit;  // of a wait, in cycles
    __device__ __forceinline__ bool gave_up() const { return *static_cast<volatile int*>(abort) != 0; }
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
    // one warp sends its block's map of round `it`, unless the block gave up before
    __device__ __forceinline__ void put(int it, Map<V> m) const {
        const int par = it & 1;
        for (int q = 0; q < cl; ++q) send(maps + (par * cl + rank) * 32 + (threadIdx.x & 31), bar + par, uint32_t(q), m);
    }
    // Every thread waits for the maps of round `it`; `ok` becomes false where the wait ran out. (Thread 0 has a channel, so
    // its `ok` is true until then. Afterwards a wait for the other parity may seem to succeed: it arms nothing more.)
    __device__ __forceinline__ const Map<V>* get(int it, bool& ok) const {
        const int par = it & 1;
        const bool got = tc::mbar_wait(bar + par, uint32_t(it >> 1) & 1u, err, abort, limit);
        ok = ok && got;
        if (ok && threadIdx.x == 0 && it + 2 < rounds) tc::mbar_arrive_expect_tx(bar + par, bytes());
        return maps + par * cl * 32 + (threadIdx.x & 31);
    }
    // no block leaves while another may still send to it
    __device__ __forceinline__ void end() const {
        if (cl > 1) {
            cluster_arrive();
            cluster_wait();
            if (gave_up()) {  // of each barrier one phase is over and the other may not be
                for (int i = 0; i < 4; ++i) tc::mbar_drain(bar + (i & 1), uint32_t(i >> 1), 1000000LL);
            }
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
// rounds' rows cost no registers. Single bf16 channels (an odd width) are too narrow for such a copy and travel in
// registers.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <typename T, int VEC>
constexpr bool kStaged = sizeof(T) * VEC >= 4;

// A lane's rows of one tensor, a round ahead: row j at [j][lane] in shared memory, or in registers where they are too
// narrow for a copy.
template <typename T, int VEC, int ROWS>
struct Ahead {
    T kept[kStaged<T, VEC> ? 1 : ROWS], coming[kStaged<T, VEC> ? 1 : ROWS];
    __device__ __forceinline__ void fetch(T* st, const T* src, const RowOffsets<ROWS>& ro) {
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            if constexpr (kStaged<T, VEC>) copy_async<sizeof(T) * VEC>(st + j * 32 * VEC, src + ro.off[j]);
            else coming[j] = src[ro.off[j]];
        }
    }
    // what was fetched last is this round's now
    __device__ __forceinline__ void turn() {
        if constexpr (!kStaged<T, VEC>) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) kept[j] = coming[j];
        }
    }
    template <typename V>
    __device__ __forceinline__ V row(const T* st, int j) const {
        if constexpr (kStaged<T, VEC>) return ldv<V>(st + j * 32 * VEC);
        else return ldv<V>(&kept[j]);
    }
};

// bytes a warp's stage takes
template <typename T, int VEC, int ROWS>
constexpr int kFwdStage = ROWS * 32 * VEC * int(4 + sizeof(T));
template <typename T, int VEC, int ROWS>
constexpr int kBwdStage = ROWS * 32 * VEC * int(4 + 2 * sizeof(T));

// What a block is to do and where its lanes' data are.
template <typename T, int VEC, int WARPS, int ROWS, int STAGE>
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
    __device__ __forceinline__ int64_t row(int r) const { return (int64_t(r) * cl + rank) * (WARPS * ROWS) + warp * ROWS; }
    __device__ __forceinline__ int64_t first(int64_t t) const { return (lead * L + (t < L ? t : L - 1)) * D + cc; }
    __device__ __forceinline__ float* gates(int par) const {
        return reinterpret_cast<float*>(stages + par * STAGE) + lane * VEC;
    }
    // k-th tensor of the element type
    __device__ __forceinline__ T* elems(int par, int k) const {
        return reinterpret_cast<T*>(stages + par * STAGE + ROWS * 32 * VEC * 4) + k * ROWS * 32 * VEC + lane * VEC;
    }
};

template <typename V>
size_t smem_of(int cl, int stages_bytes) {
    return (cl > 1 ? size_t(2) * cl * 32 * sizeof(Map<V>) : 0) + size_t(2) * stages_bytes;
}

// What a launch with clusters of up to kMaxCluster blocks needs of the kernel, on the current device. The attributes
// belong to the kernel, which other host threads may be about to launch, so `smem` is always what the largest cluster
// takes: no call lowers the limit under another's launch. (How many blocks an SM holds follows the launch's own size.)
template <typename K>
bool allow_clusters(K kernel, size_t smem) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
           cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) == cudaSuccess;
}

// How many clusters of each size the device holds at once, for one kernel: a cluster sits inside one GPC, so large ones
// leave some SMs empty. Asked once (the answer depends on the kernel and the kind of GPU alone); an answer that could
// not be had is asked for again.
struct ClusterFit {
    int fit[kMaxCluster + 1] = {};
};
struct FitOnce {
    std::mutex mu;
    std::atomic<bool> have{false};
    ClusterFit f;
};
template <typename K>
ClusterFit cluster_fit(FitOnce& once, K kernel, int threads, size_t (*smem)(int, int), int stages_bytes) {
    if (once.have.load(std::memory_order_acquire)) return once.f;
    std::lock_guard<std::mutex> lk(once.mu);
    if (once.have.load(std::memory_order_relaxed)) return once.f;
    ClusterFit f;
    if (!allow_clusters(kernel, smem(kMaxCluster, stages_bytes))) return f;
    for (int cl = 1; cl <= kMaxCluster; ++cl) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(cl));
        cfg.blockDim = dim3(unsigned(threads));
        cfg.dynamicSmemBytes = smem(cl, stages_bytes);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = unsigned(cl);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess) f.fit[cl] = n;
        else (void)cudaGetLastError();  // a size that this device does not take is no error of the launch to come
    }
    if (f.fit[1] > 0) {
        once.f = f;
        once.have.store(true, std::memory_order_release);
    }
    return f;
}

// Blocks per cluster. A block's time goes by its rounds, and clusters that do not fit at once run in further waves:
// the least waves x rounds (cost), and of those the smallest cluster.
struct ClusterPlan {
    int size;
    int64_t cost;
};
ClusterPlan cluster_plan(const ClusterFit& f, int64_t groups, int64_t L, int tile) {
    const int64_t tiles = cdiv(L, tile);
    ClusterPlan best{1, INT64_MAX / 8};
    for (int cl = 1; cl <= kMaxCluster; ++cl) {
        if (f.fit[cl] < 1 || cl > tiles) continue;
        const int64_t c = cdiv(groups, int64_t(f.fit[cl])) * cdiv(tiles, int64_t(cl));
        if (c < best.cost) best = ClusterPlan{cl, c};
    }
    return best;
}

// Blocks of four warps where there are channel tiles and sequences for a quarter of the SMs: more blocks that wait at
// different times (forward 33.3 us against 35.6 at 8 sequences of 2048 steps, width 1024). Else of eight, whose rounds
// cover twice the rows (29 us against 43 at one sequence of 16384 steps, width 64, 8 rows a warp).
inline bool many_groups(int64_t groups) { return groups * 4 >= 148; }

template <typename K, typename... Args>
gla_status launch_clusters(const char* name, K kernel, const ClusterFit& f, int64_t groups, int cl, int threads,
                           size_t (*smem)(int, int), int stages_bytes, cudaStream_t s, Args... args) {
    if (f.fit[1] < 1 || !allow_clusters(kernel, smem(kMaxCluster, stages_bytes))) return GLA_ERR_CUDA;
    if (groups * cl > (int64_t(1) << 31) - 1) return GLA_ERR_UNSUPPORTED;
    launch_begin(name, s);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(groups * cl));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem(cl, stages_bytes);
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
}  // namespace gla
