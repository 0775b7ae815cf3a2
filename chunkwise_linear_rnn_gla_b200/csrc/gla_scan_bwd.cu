// Backward kernel of the elementwise gated recurrence (gla_scan.cuh).
#include "gla_scan.cuh"

namespace gla {
namespace {

constexpr int kBwdRows = 8;  // rows of a warp

// ---- backward -----------------------------------------------------------------------------
// Rounds, blocks and warps as in the forward, from the last round to the first. The states inside a block's rows
// are recomputed in fp32 from the state that enters them (seg).
template <typename T, int VEC, bool PACKED, bool PREACT, bool LEAK, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS)
    k_scan_bwd(ScanProblem p, int cl, const T* __restrict__ x, const float* __restrict__ la,
               const int32_t* __restrict__ cu, const float* __restrict__ h0, const T* __restrict__ dh,
               const float* __restrict__ dhT, T* __restrict__ dx, float* __restrict__ dla, float* __restrict__ dh0,
               const float* __restrict__ seg, int* err) {
    using V = typename VecOf<VEC>::type;
    constexpr int ROWS = kBwdRows, STAGE = kBwdStage<T, VEC, ROWS>;
    __shared__ Map<V> agg[2][WARPS][32];
    __shared__ V aggy[2][WARPS][32];
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
    Ahead<T, VEC, ROWS> xa, da;
    const auto stage = [&](int r) {
        const int64_t t = at.row(r), i = at.first(t);
        const RowOffsets<ROWS> ro = offsets(t);
        ga.fetch(at.gates(r & 1), la + i, ro);
        xa.fetch(at.elems(r & 1, 0), x + i, ro);
        da.fetch(at.elems(r & 1, 1), dh + i, ro);
    };
    stage(rounds - 1);
    copies_commit();
    ex.begin();
    if constexpr (PACKED) copy_empty<V>(cu, p, head, c, mine, dhT, dh0, rank * WARPS + warp, cl * WARPS, lane);
    V carry = vset<V>(0.f);  // y of the row behind the round's last
    if (!PACKED && dhT) carry = ldv<V>(dhT + lead * p.D + cc);
    ex.ready();
    const int64_t nseg = cdiv(p.L, kSeg);
    for (int it = 0; it < rounds; ++it) {
        const int r = rounds - 1 - it, par = r & 1;
        const int64_t t0 = at.row(r), first = at.first(t0);
        const int64_t tile = (int64_t(r) * cl + rank) * (WARPS * ROWS) / kSeg;  // a block's rows begin with a segment
        const RowOffsets<ROWS> ro = offsets(t0);
        V s = ldv<V>(seg + (lead * nseg + (tile < nseg ? tile : nseg - 1)) * p.D + cc);  // entering the block's rows
        xa.turn();
        da.turn();
        if (r > 0) stage(r - 1);
        copies_commit();
        copies_wait<1>();
        RowInfo ri{0, 0, 0, 0};
        if constexpr (PACKED) ri = rows_packed<ROWS>(cu, int(p.B), t0, p.L, lane);
        else ri.valid = t0 + ROWS <= p.L ? ~0u : t0 < p.L ? (1u << (p.L - t0)) - 1 : 0u;
        V a[ROWS], w[ROWS], xv[ROWS], d[ROWS], dz[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            gate_of<PREACT, LEAK>(p.inv_tau, ga.template row<V>(at.gates(par), j), a[j], w[j], dz[j]);
            xv[j] = xa.template row<V>(at.elems(par, 0), j);
            d[j] = da.template row<V>(at.elems(par, 1), j);
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
        const bool sends = cl > 1 && warp == 0 && !ex.gave_up();
        __syncthreads();
        Map<V> post{vset<V>(1.f), vset<V>(0.f)};  // the map (of y) of the block's rows behind this warp's
#pragma unroll
        for (int q = 0; q < WARPS - 1; ++q) {
            if (q < warp) {
                const Map<V> m = agg[par][q][lane];
                s = join<PACKED>(m.a, s, m.u);
            }
        }
#pragma unroll
        for (int q = WARPS - 1; q > 0; --q) {
            if (q > warp) {
                const V m = agg[par][q][lane].a;
                post = Map<V>{join<PACKED>(m, post.a), join<PACKED>(m, post.u, aggy[par][q][lane])};
            }
        }
        V in = carry;
        if (cl > 1) {
            if (sends) ex.put(it, Map<V>{join<PACKED>(own.a, post.a), join<PACKED>(own.a, post.u, Y)});
            const Map<V>* m = ex.get(it, mine);
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

template <typename T, int VEC, bool PACKED, bool PREACT, bool LEAK, int WARPS>
gla_status bwd_launch(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                      const void* dh, const float* dhT, void* dx, float* dla, float* dh0, const float* seg,
                      cudaStream_t s) {
    using V = typename VecOf<VEC>::type;
    constexpr int threads = WARPS * 32, stages = WARPS * kBwdStage<T, VEC, kBwdRows>;
    const int64_t groups = (PACKED ? p.H : p.B * p.H) * cdiv(p.D, 32 * VEC);
    const auto kernel = k_scan_bwd<T, VEC, PACKED, PREACT, LEAK, WARPS>;
    static FitOnce once;
    const ClusterFit fit = cluster_fit(once, kernel, threads, smem_of<V>, stages);
    const int cl = cluster_plan(fit, groups, p.L, WARPS * kBwdRows).size;
    return launch_clusters("scan_bwd", kernel, fit, groups, cl, threads, smem_of<V>, stages, s, p, cl,
                           static_cast<const T*>(x), la, cu, h0, static_cast<const T*>(dh), dhT, static_cast<T*>(dx),
                           dla, dh0, seg, device_error_word());
}

template <typename T, int VEC, bool PACKED, bool PREACT, bool LEAK>
gla_status bwd_typed(const ScanProblem& p, const void* x, const float* la, const int32_t* cu, const float* h0,
                     const void* dh, const float* dhT, void* dx, float* dla, float* dh0, const float* seg,
                     cudaStream_t s) {
    const int64_t groups = (PACKED ? p.H : p.B * p.H) * cdiv(p.D, 32 * VEC);
    if (many_groups(groups)) return bwd_launch<T, VEC, PACKED, PREACT, LEAK, 4>(p, x, la, cu, h0, dh, dhT, dx, dla, dh0, seg, s);
    return bwd_launch<T, VEC, PACKED, PREACT, LEAK, 8>(p, x, la, cu, h0, dh, dhT, dx, dla, dh0, seg, s);
}

}  // namespace

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

}  // namespace gla
