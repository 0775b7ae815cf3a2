// Forward and single-token kernels of the elementwise gated recurrence (gla_scan.cuh).
#include "gla_scan.cuh"

namespace gla {
namespace {

// ---- forward ------------------------------------------------------------------------------
// Grid: (sequence or head) x channel tile x cluster of `cl` blocks. Rows of round r and block q: from
// (r cl + q) WARPS ROWS.
template <typename T, int VEC, bool PACKED, bool PREACT, bool LEAK, int WARPS, int ROWS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS)
    k_scan_fwd(ScanProblem p, int cl, const T* __restrict__ x, const float* __restrict__ la,
               const int32_t* __restrict__ cu, const float* __restrict__ h0, T* __restrict__ h, float* __restrict__ hT,
               float* __restrict__ seg, int* err) {
    using V = typename VecOf<VEC>::type;
    constexpr int STAGE = kFwdStage<T, VEC, ROWS>;
    __shared__ Map<V> agg[2][WARPS][32];
    __shared__ uint64_t bar[2];
    __shared__ int abort_flag;
    extern __shared__ __align__(16) char dyn[];  // the cluster's maps, then the warps' stages
    const Place<T, VEC, WARPS, ROWS, STAGE> at(p, cl, dyn + (cl > 1 ? 2 * cl * 32 * sizeof(Map<V>) : 0));
    const int lane = at.lane, warp = at.warp, rank = at.rank;
    const int64_t lead = at.lead, c = at.c, cc = at.cc, head = PACKED ? lead : 0;
    bool mine = at.mine;
    const int rounds = int(cdiv(p.L, int64_t(WARPS * ROWS) * cl));
    Exchange<V> ex{reinterpret_cast<Map<V>*>(dyn), bar, &abort_flag, err, cl, rank, rounds, p.wait_limit};
    const RowOffsets<ROWS> whole(ROWS, p.D);
    const auto offsets = [&](int64_t t) { return p.L - t >= ROWS ? whole : RowOffsets<ROWS>(p.L - t, p.D); };
    Ahead<float, VEC, ROWS> ga;
    Ahead<T, VEC, ROWS> xa;
    const auto stage = [&](int r) {
        const int64_t t = at.row(r), i = at.first(t);
        const RowOffsets<ROWS> ro = offsets(t);
        ga.fetch(at.gates(r & 1), la + i, ro);
        xa.fetch(at.elems(r & 1, 0), x + i, ro);
    };
    stage(0);
    copies_commit();
    ex.begin();
    if constexpr (PACKED) copy_empty<V>(cu, p, head, c, mine, h0, hT, rank * WARPS + warp, cl * WARPS, lane);
    V carry = vset<V>(0.f);
    if (!PACKED && h0) carry = ldv<V>(h0 + lead * p.D + cc);
    ex.ready();
    const int64_t nseg = cdiv(p.L, kSeg);
    for (int r = 0; r < rounds; ++r) {
        const int par = r & 1;
        const int64_t t0 = at.row(r), first = at.first(t0);
        const RowOffsets<ROWS> ro = offsets(t0);
        xa.turn();
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
            gate_of<PREACT, LEAK>(p.inv_tau, ga.template row<V>(at.gates(par), j), a[j], w, dz);
            b[j] = xa.template row<V>(at.elems(par, 0), j);
            if constexpr (LEAK) b[j] = vmul(b[j], w);
        }
        constexpr uint32_t kAll = (1u << ROWS) - 1;
        const bool all = (ri.valid & kAll) == kAll;
        if (!all) {
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
        const bool sends = cl > 1 && warp == WARPS - 1 && !ex.gave_up();
        __syncthreads();
        Map<V> pre{vset<V>(1.f), vset<V>(0.f)};  // of the block's rows in front of this warp's
#pragma unroll
        for (int w = 0; w < WARPS - 1; ++w) {
            if (w < warp) {
                const Map<V> m = agg[par][w][lane];
                pre = Map<V>{join<PACKED>(m.a, pre.a), join<PACKED>(m.a, pre.u, m.u)};
            }
        }
        V in = carry;  // state entering the block's rows
        if (cl > 1) {
            if (sends) ex.put(r, Map<V>{join<PACKED>(own.a, pre.a), join<PACKED>(own.a, pre.u, own.u)});
            const Map<V>* m = ex.get(r, mine);
            for (int q = 0; q < cl; ++q) {
                if (q == rank) in = carry;
                carry = join<PACKED>(m[q * 32].a, carry, m[q * 32].u);
            }
        } else {
            Map<V> t = pre;
            for (int w = warp; w < WARPS; ++w) {
                const Map<V> m = agg[par][w][lane];
                t = Map<V>{join<PACKED>(m.a, t.a), join<PACKED>(m.a, t.u, m.u)};
            }
            carry = join<PACKED>(t.a, in, t.u);
        }
        V s = join<PACKED>(pre.a, in, pre.u);
        if (seg && mine && t0 < p.L && t0 % kSeg == 0) stv(seg + (lead * nseg + t0 / kSeg) * p.D + c, s);
        T* out = h + first;
        if (!PACKED && all && h) {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                s = vfma(a[j], s, b[j]);
                if (mine) stv(out + ro.off[j], s);
            }
        } else {
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                if (PACKED && (ri.start >> j & 1)) s = state_of<V>(h0, __shfl_sync(0xffffffffu, ri.n, j), p, head, cc);
                s = vfma(a[j], s, b[j]);
                if (h && mine && (ri.valid >> j & 1)) stv(out + ro.off[j], s);
                if (PACKED && (ri.end >> j & 1)) {
                    const int64_t n = __shfl_sync(0xffffffffu, ri.n, j);
                    if (hT && mine) stv(hT + (n * p.H + head) * p.D + c, s);
                }
            }
        }
        // rows behind the last one leave the state as it is, so the warp with the last row holds hT
        if (!PACKED && hT && mine && t0 < p.L && t0 + ROWS >= p.L) stv(hT + lead * p.D + c, s);
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

// One form of the forward kernel and how a call would run on it.
template <typename T, int VEC, bool PACKED, bool PREACT, bool LEAK, int WARPS, int ROWS>
struct FwdForm {
    using V = typename VecOf<VEC>::type;
    static constexpr int threads = WARPS * 32, stages = WARPS * kFwdStage<T, VEC, ROWS>;
    ClusterFit fit;
    int64_t groups;
    ClusterPlan plan;
    static auto kernel() { return k_scan_fwd<T, VEC, PACKED, PREACT, LEAK, WARPS, ROWS>; }
    FwdForm(const ScanProblem& p, int64_t groups_) : groups(groups_) {
        static FitOnce once;
        fit = cluster_fit(once, kernel(), threads, smem_of<V>, stages);
        plan = cluster_plan(fit, groups, p.L, WARPS * ROWS);
    }
    gla_status launch(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0, void* h,
                      float* hT, float* seg, cudaStream_t s) const {
        return launch_clusters("scan_fwd", kernel(), fit, groups, plan.size, threads, smem_of<V>, stages, s, p, plan.size,
                               static_cast<const T*>(x), la, cu, h0, static_cast<T*>(h), hT, seg, device_error_word());
    }
};

// Rows a warp: 8, or 16 where they save rounds. A round of 16 takes 1.6 to 1.75 times as long as one of 8 (its exchange,
// lookups and barriers are paid once), and its stages leave room for fewer blocks, which the plan's waves count. One
// sequence of 16384 steps, width 64: 28.7 us against 35.6; 8000 steps, width 1001: 36.2 against 42.8; but 91 against 64 at
// 16384 steps, width 1024, where half the clusters wait for a second wave, and 4.7 against 3.7 at 256 steps, width 64.
// Two channels a lane in blocks of four warps fill an SM with 8 rows already (33 us against 40 at 8 sequences of 2048
// steps, width 1024).
template <typename T, int VEC, bool PACKED, bool PREACT, bool LEAK, int WARPS>
gla_status fwd_rows(const ScanProblem& p, int64_t groups, const void* x, const float* la, const int32_t* cu,
                    const float* h0, void* h, float* hT, float* seg, cudaStream_t s) {
    const FwdForm<T, VEC, PACKED, PREACT, LEAK, WARPS, 8> few(p, groups);
    if constexpr (VEC == 1 || WARPS == 8) {
        if (few.plan.cost > 1) {
            const FwdForm<T, VEC, PACKED, PREACT, LEAK, WARPS, 16> many(p, groups);
            if (many.plan.cost * 7 <= few.plan.cost * 4) return many.launch(p, x, la, cu, h0, h, hT, seg, s);
        }
    }
    return few.launch(p, x, la, cu, h0, h, hT, seg, s);
}

template <typename T, int VEC, bool PACKED, bool PREACT, bool LEAK>
gla_status fwd_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                     void* h, float* hT, float* seg, cudaStream_t s) {
    const int64_t groups = (PACKED ? p.H : p.B * p.H) * cdiv(p.D, 32 * VEC);
    if (many_groups(groups)) return fwd_rows<T, VEC, PACKED, PREACT, LEAK, 4>(p, groups, x, la, cu, h0, h, hT, seg, s);
    return fwd_rows<T, VEC, PACKED, PREACT, LEAK, 8>(p, groups, x, la, cu, h0, h, hT, seg, s);
}

template <typename T>
gla_status step_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* slots, int64_t pool,
                      float* state, void* h, cudaStream_t s) {
    const dim3 grid(unsigned(cdiv(p.H * p.D, kStepThreads)), unsigned(p.B));
    GLA_LAUNCH("scan_step", k_scan_step<T>, grid, kStepThreads, 0, s, p, static_cast<const T*>(x), la, slots,
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
    return dispatch(p, [&](auto type, auto vec, auto packed, auto preact, auto leak) {
        return fwd_typed<decltype(type), vec(), packed(), preact(), leak()>(p, x, la, cu, h0, h, hT, seg, s);
    });
}

gla_status scan_step(const ScanProblem& p, const void* x, const float* la, const int32_t* slots, int64_t pool,
                     float* state, void* h, cudaStream_t s) {
    return p.bf16 ? step_typed<__nv_bfloat16>(p, x, la, slots, pool, state, h, s)
                  : step_typed<float>(p, x, la, slots, pool, state, h, s);
}

}  // namespace gla
