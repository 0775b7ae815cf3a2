// Recurrent-state cache (include/gla.h, "recurrent-state cache"): matrix states held in 8 bits in a pool of slots,
// the last few tokens of each sequence beside them, and the decode step that reads both:
//     S_t = diag(e^G) (scale code) + sum_j (k_j e^{D_j})^T v_j,   o_t = q S_t.
// The decay acts on whole rows, so a scale per row (and 128 columns) carries it exactly; the recurrent form is that
// of the decode step (podcast.app episode page, summary: a gated memory updated once per token).
//
// A step need not form S_t: with w_c = q_c e^{G_c} scale_c and the scores p_j = sum_c q_c k_jc e^{D_jc},
//     o = sum_c w_c code_c + sum_j p_j v_j,
// one multiply-add per 8-bit entry. Only the step that fills a window forms S_t, to round it back.
//
// All kernels give a warp the 128 columns of one group, four to a lane: a row's codes are one 128-byte access of the
// warp, its largest magnitude one warp reduction, a row of fp32 one 512-byte access.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gla_common.cuh"
#include "gla_gate.cuh"
#include "gla_internal.h"
#include "tc_prims.cuh"

namespace gla {
namespace {

constexpr int kG = kCacheGroup;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 8;        // state rows a warp takes at a time
constexpr float kTiny = 1e-30f;  // a group whose largest magnitude is below this is held as zero

struct Pool {
    uint8_t* codes;
    float* scale;
    void* k;
    void* v;
    float* la;
    int64_t slots;
    int W;
    int64_t H;
    int K, V, NG;
};

// ---- 8-bit codes --------------------------------------------------------------------------
// Four codes to fp32, exactly.
template <bool INT8>
__device__ __forceinline__ void decode4(uint32_t x, float* y) {
    if constexpr (INT8) {
        // 2^23 + 128 + code has the biased code in its low byte; the subtraction is exact
        const uint32_t u = x ^ 0x80808080u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440u + e)) - 8388736.f;
    } else {
        const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(x & 0xffffu), __NV_E4M3);
        const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(x >> 16), __NV_E4M3);
        const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
        y[0] = a.x;
        y[1] = a.y;
        y[2] = b.x;
        y[3] = b.y;
    }
}

// scale of a group from the bits of its largest magnitude (NaN and inf order above every finite value)
template <bool INT8>
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    const float m = __uint_as_float(amax_bits);
    if (!(m < INFINITY)) return __uint_as_float(0x7fc00000u);
    return m < kTiny ? 0.f : __fmul_rn(m, INT8 ? float(1.0 / 127) : float(1.0 / 448));
}

template <bool INT8>
__device__ __forceinline__ uint32_t encode4(const float* y, float scale) {
    // the codes of a group held as zero or as NaN are 0
    const float inv = scale > 0.f ? __frcp_rn(scale) : 0.f;
    uint32_t r = 0;
    if (!(scale > 0.f)) return r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float t = __fmul_rn(y[e], inv);
        const uint32_t b = INT8 ? uint32_t(int(fminf(fmaxf(rintf(t), -127.f), 127.f))) & 0xffu
                                : uint32_t(__nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3));
        r |= b << (8 * e);
    }
    return r;
}

// ---- a lane's four columns ------------------------------------------------------------------
// Adjacent (VEC, the width a multiple of 4) or 32 apart; those that do not exist read as 0 and are not written.
template <bool VEC>
struct Cols {
    int col[4];
    bool on[4];
    __device__ __forceinline__ Cols(int grp, int V) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            col[e] = grp * kG + (VEC ? 4 * lane + e : lane + 32 * e);
            on[e] = col[e] < V;
        }
    }
    __device__ __forceinline__ uint32_t codes(const uint8_t* row) const {
        if constexpr (VEC) return on[0] ? __ldcs(reinterpret_cast<const uint32_t*>(row + col[0])) : 0u;
        uint32_t x = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (on[e]) x |= uint32_t(row[col[e]]) << (8 * e);
        return x;
    }
    __device__ __forceinline__ void put_codes(uint8_t* row, uint32_t x) const {
        if constexpr (VEC) {
            if (on[0]) *reinterpret_cast<uint32_t*>(row + col[0]) = x;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (on[e]) row[col[e]] = uint8_t(x >> (8 * e));
        }
    }
    __device__ __forceinline__ void load(const float* row, float* y) const {
        if constexpr (VEC) {
            const float4 t = on[0] ? __ldcs(reinterpret_cast<const float4*>(row + col[0])) : make_float4(0.f, 0.f, 0.f, 0.f);
            y[0] = t.x, y[1] = t.y, y[2] = t.z, y[3] = t.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = on[e] ? row[col[e]] : 0.f;
        }
    }
    __device__ __forceinline__ void store(float* row, const float* y) const {
        if constexpr (VEC) {
            if (on[0]) __stcs(reinterpret_cast<float4*>(row + col[0]), make_float4(y[0], y[1], y[2], y[3]));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (on[e]) row[col[e]] = y[e];
        }
    }
    // place of the lane's e-th column in a [128] shared-memory row
    __device__ __forceinline__ int at(int e) const {
        const int lane = threadIdx.x & 31;
        return VEC ? 4 * lane + e : lane + 32 * e;
    }
};

// Whether an earlier row of the call names the same slot (every thread of the block gets the answer).
__device__ __forceinline__ bool named_before(const int32_t* slots, int64_t b, int32_t slot) {
    int dup = 0;
    for (int64_t i = threadIdx.x; i < b; i += blockDim.x) dup |= slots[i] == slot;
    return __syncthreads_or(dup) != 0;
}

// largest magnitude of the warp's columns, as bits
__device__ __forceinline__ uint32_t warp_amax(const float* y) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max(m, __float_as_uint(y[e]) & 0x7fffffffu);
    return __reduce_max_sync(0xffffffffu, m);
}

// ---- store ----------------------------------------------------------------------------------
// One block per (row of the call, head, group, 64 state rows): 4 bytes read and 1 written an entry.
template <bool INT8, bool VEC>
__global__ void __launch_bounds__(kThreads) k_cache_store(Pool c, int parts, const float* __restrict__ S,
                                                          const int32_t* __restrict__ slots, int* err) {
    const int64_t bhg = blockIdx.x / parts, bh = bhg / c.NG, b = bh / c.H, head = bh % c.H;
    const int part = int(blockIdx.x % parts), grp = int(bhg % c.NG);
    const Cols<VEC> cols(grp, c.V);
    const int r0 = part * kWarps * kBatch + int(threadIdx.x >> 5) * kBatch;
    float y[kBatch][4];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
        if (r0 + i < c.K) cols.load(S + (bh * c.K + r0 + i) * c.V, y[i]);
    const int32_t slot = slots[b];
    if (slot < 0) return;
    if (slot >= c.slots || named_before(slots, b, slot)) {
        if (threadIdx.x == 0) atomicOr(err, kErrBadRow);
        return;
    }
    const int64_t sh = slot * c.H + head;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        if (r0 + i >= c.K) break;
        const float sc = scale_of<INT8>(warp_amax(y[i]));
        cols.put_codes(c.codes + (sh * c.K + r0 + i) * c.V, encode4<INT8>(y[i], sc));
        if ((threadIdx.x & 31) == 0) c.scale[(sh * c.K + r0 + i) * c.NG + grp] = sc;
    }
}

// ---- the window -----------------------------------------------------------------------------
// kt[j][r - r0] = k_jr e^{D_jr} and decay[r - r0] = e^{G_r} for state rows [r0, r1), j < used; place n = used - 1 comes
// from the call in a step (kc, gate) and is put into the window by the blocks of group 0. Sums of log decays run from
// the newest token back, so a zero gate (a huge negative number) hides only what is in front of it.
template <typename T, bool STEP>
__device__ __forceinline__ void window_keys(const Pool& c, int64_t sh, int64_t bh, int n, int r0, int r1, int ld,
                                            const T* __restrict__ kc, const GateArgs& ga, bool put, float* kt,
                                            float* decay) {
    T* wk = static_cast<T*>(c.k) + sh * c.W * c.K;
    float* wl = c.la + sh * c.W * c.K;
    for (int r = r0 + int(threadIdx.x); r < r1; r += kThreads) {
        float D = 0.f;
        if constexpr (STEP) {
            const T k = kc[bh * c.K + r];
            const float la = gate_log_alpha(ga, bh, 0, r, 1, c.K);
            kt[n * ld + r - r0] = ldf(&k);
            if (put) {
                wk[n * c.K + r] = k;
                wl[n * c.K + r] = la;
            }
            D = la;
        }
#pragma unroll 8
        for (int j = n - 1; j >= 0; --j) {
            kt[j * ld + r - r0] = ldf(wk + j * c.K + r) * tc::exp2_ftz(D * tc::kLog2e);
            D += wl[j * c.K + r];
        }
        decay[r - r0] = tc::exp2_ftz(D * tc::kLog2e);
    }
}

// vs[j][0..127]: the group's columns of the window's values, fp32
template <typename T, bool STEP>
__device__ __forceinline__ void window_values(const Pool& c, int64_t sh, int64_t bh, int n, int grp,
                                              const T* __restrict__ vc, float* vs) {
    T* wv = static_cast<T*>(c.v) + sh * c.W * c.V;
    for (int i = threadIdx.x; i < (n + (STEP ? 1 : 0)) * kG; i += kThreads) {
        const int j = i / kG, col = grp * kG + i % kG;
        float x = 0.f;
        if (col < c.V) {
            if (STEP && j == n) {
                const T v = vc[bh * c.V + col];
                wv[n * c.V + col] = v;
                x = ldf(&v);
            } else x = ldf(wv + j * c.V + col);
        }
        vs[i] = x;
    }
}

// Rows r .. r+7 (of those in kt) of the state: code x scale x decay + the window's outer products.
template <bool INT8, bool VEC>
__device__ __forceinline__ void form_rows(const Cols<VEC>& cols, const uint32_t* codes, const float* scale,
                                          const float* decay, const float* kt, int ld, const float* vs, int used,
                                          float (*y)[4]) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        decode4<INT8>(codes[i], y[i]);
        const float f = decay[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] = f * (scale[i] * y[i][e]);
    }
    for (int j = 0; j < used; ++j) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = vs[j * kG + cols.at(e)];
        const float4 ka = *reinterpret_cast<const float4*>(kt + j * ld), kb = *reinterpret_cast<const float4*>(kt + j * ld + 4);
        const float k[kBatch] = {ka.x, ka.y, ka.z, ka.w, kb.x, kb.y, kb.z, kb.w};
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[i][e] = fmaf(k[i], v[e], y[i][e]);
    }
}

// ---- load -----------------------------------------------------------------------------------
// One block per (row of the call, head, group, 64 state rows).
template <typename T, bool INT8, bool VEC>
__global__ void __launch_bounds__(kThreads) k_cache_load(Pool c, int parts, const int32_t* __restrict__ slots,
                                                         const int32_t* __restrict__ lengths, float* __restrict__ S,
                                                         int* err) {
    constexpr int ROWS = kWarps * kBatch;
    extern __shared__ __align__(16) float sm[];
    const int64_t bhg = blockIdx.x / parts, bh = bhg / c.NG, b = bh / c.H, head = bh % c.H;
    const int part = int(blockIdx.x % parts), grp = int(bhg % c.NG);
    const Cols<VEC> cols(grp, c.V);
    const int w0 = int(threadIdx.x >> 5) * kBatch, r0 = part * ROWS + w0;
    const int32_t slot = slots[b];
    const int32_t len = lengths ? lengths[b] : 0;
    bool live = slot >= 0;
    if (live && (slot >= c.slots || len < 0)) {
        live = false;
        if (threadIdx.x == 0) atomicOr(err, kErrBadRow);
    }
    float y[kBatch][4];
    if (live) {
        const int64_t sh = slot * c.H + head;
        const int n = len % c.W;
        uint32_t x[kBatch];
        float sc[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = r0 + i < c.K ? r0 + i : c.K - 1;
            x[i] = cols.codes(c.codes + (sh * c.K + r) * c.V);
            sc[i] = c.scale[(sh * c.K + r) * c.NG + grp];
        }
        float* kt = sm;                   // [W][ROWS]
        float* decay = kt + c.W * ROWS;   // [ROWS]
        float* vs = decay + ROWS;         // [W][128]
        const int first = part * ROWS, last = first + ROWS < c.K ? first + ROWS : c.K;
        window_keys<T, false>(c, sh, bh, n, first, last, ROWS, nullptr, GateArgs{}, false, kt, decay);
        window_values<T, false>(c, sh, bh, n, grp, nullptr, vs);
        __syncthreads();
        form_rows<INT8, VEC>(cols, x, sc, decay + w0, kt + w0, ROWS, vs, n, y);
    } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[i][e] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
        if (r0 + i < c.K) cols.store(S + (bh * c.K + r0 + i) * c.V, y[i]);
}

// ---- step -----------------------------------------------------------------------------------
// One block per (row of the call, head, group).
__host__ __device__ constexpr int round_up(int x, int m) { return (x + m - 1) / m * m; }

template <typename T, bool INT8, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) k_cache_step(Pool c, const T* __restrict__ q, const T* __restrict__ k,
                                                            const T* __restrict__ v, GateArgs ga,
                                                            const int32_t* __restrict__ slots,
                                                            const int32_t* __restrict__ lengths, T* __restrict__ o,
                                                            int* err) {
    constexpr int PASS = 4;  // batches a warp has in flight: 256 rows a block
    extern __shared__ __align__(16) float sm[];
    const int64_t bh = blockIdx.x / c.NG, b = bh / c.H, head = bh % c.H;
    const int grp = int(blockIdx.x % c.NG), tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const Cols<VEC> cols(grp, c.V);
    const int ld = round_up(c.K, kBatch);
    const int32_t slot = slots[b], len = lengths[b];
    bool live = slot >= 0;
    if (live && (slot >= c.slots || len < 0 || named_before(slots, b, slot))) {
        live = false;
        if (tid == 0) atomicOr(err, kErrBadRow);
    }
    if (!live) {
        if (warp == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (cols.on[e]) stf(o + bh * c.V + cols.col[e], 0.f);
        }
        return;
    }
    const int64_t sh = slot * c.H + head;
    const int n = len % c.W, used = n + 1;
    const uint8_t* codes = c.codes + sh * c.K * c.V;
    float* scale = c.scale + sh * c.K * c.NG + grp;
    float* kt = sm;                    // [W][ld]
    float* vs = kt + c.W * ld;         // [W][128]
    float* decay = vs + c.W * kG;      // [ld]
    float* wq = decay + ld;            // [ld] q e^G scale
    float* p = wq + ld;                // [64] scores
    float* red = p + 64;               // [8][128]
    uint32_t x[PASS][kBatch];
    const auto fetch = [&](int r0) {
#pragma unroll
        for (int u = 0; u < PASS; ++u)
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int r = r0 + (u * kWarps + warp) * kBatch + i;
                x[u][i] = r < c.K ? cols.codes(codes + int64_t(r) * c.V) : 0u;
            }
    };
    fetch(0);
    window_keys<T, true>(c, sh, bh, n, 0, c.K, ld, k, ga, grp == 0, kt, decay);
    window_values<T, true>(c, sh, bh, n, grp, v, vs);
    for (int r = tid; r < ld; r += kThreads)
        wq[r] = r < c.K ? ldf(q + bh * c.K + r) * decay[r] * scale[int64_t(r) * c.NG] : 0.f;
    __syncthreads();
    for (int j = warp; j < used; j += kWarps) {
        float s = 0.f;
        for (int r = lane; r < c.K; r += 32) s = fmaf(ldf(q + bh * c.K + r), kt[j * ld + r], s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane == 0) p[j] = s;
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r0 = 0; r0 < c.K; r0 += PASS * kWarps * kBatch) {
        if (r0) fetch(r0);
#pragma unroll
        for (int u = 0; u < PASS; ++u) {
            const int r = r0 + (u * kWarps + warp) * kBatch;
            if (r < c.K) {
                const float4 wa = *reinterpret_cast<const float4*>(wq + r), wb = *reinterpret_cast<const float4*>(wq + r + 4);
                const float w[kBatch] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    float y[4];
                    decode4<INT8>(x[u][i], y);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] = fmaf(w[i], y[e], acc[e]);
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) red[warp * kG + cols.at(e)] = acc[e];
    __syncthreads();
    if (tid < kG && grp * kG + tid < c.V) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += red[w * kG + tid];
        for (int j = 0; j < used; ++j) s = fmaf(p[j], vs[j * kG + tid], s);
        stf(o + bh * c.V + grp * kG + tid, s);
    }
    if (used < c.W) return;
    // the window is full: round the state back
    for (int r = warp * kBatch; r < c.K; r += kWarps * kBatch) {
        uint32_t z[kBatch];
        float sc[kBatch], y[kBatch][4];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int ri = r + i < c.K ? r + i : c.K - 1;
            z[i] = cols.codes(codes + int64_t(ri) * c.V);
            sc[i] = scale[int64_t(ri) * c.NG];
        }
        form_rows<INT8, VEC>(cols, z, sc, decay + r, kt + r, ld, vs, used, y);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (r + i >= c.K) break;
            const float ns = scale_of<INT8>(warp_amax(y[i]));
            cols.put_codes(c.codes + (sh * c.K + r + i) * c.V, encode4<INT8>(y[i], ns));
            if (lane == 0) scale[int64_t(r + i) * c.NG] = ns;
        }
    }
}

Pool pool_of(const CacheProblem& p) {
    return Pool{static_cast<uint8_t*>(p.c.codes), p.c.scale, p.c.k, p.c.v, p.c.log_a, p.c.slots, p.c.window,
                p.H, int(p.K), int(p.V), int(cdiv(p.V, kG))};
}

size_t step_smem(const CacheProblem& p) {
    const size_t ld = size_t(round_up(int(p.K), kBatch));
    return sizeof(float) * (size_t(p.c.window) * (ld + kG) + 2 * ld + 64 + kWarps * kG);
}
size_t load_smem(const CacheProblem& p) {
    constexpr size_t rows = kWarps * kBatch;
    return sizeof(float) * (size_t(p.c.window) * (rows + kG) + rows);
}

template <typename K>
bool allow_smem(K kernel, size_t bytes) {
    return bytes <= 48 * 1024 ||
           cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes)) == cudaSuccess;
}

template <bool INT8, bool VEC>
gla_status store_typed(const CacheProblem& p, const float* S, const int32_t* slots, cudaStream_t s) {
    const Pool c = pool_of(p);
    const int parts = int(cdiv(p.K, kWarps * kBatch));
    GLA_LAUNCH("cache_store", (k_cache_store<INT8, VEC>), unsigned(p.B * p.H * c.NG * parts), kThreads, 0, s, c, parts, S,
               slots, device_error_word());
    return GLA_OK;
}

template <typename T, bool INT8, bool VEC>
gla_status load_typed(const CacheProblem& p, const int32_t* slots, const int32_t* lengths, float* S, cudaStream_t s) {
    const Pool c = pool_of(p);
    const int parts = int(cdiv(p.K, kWarps * kBatch));
    const size_t smem = load_smem(p);
    if (!allow_smem(k_cache_load<T, INT8, VEC>, smem)) return GLA_ERR_CUDA;
    GLA_LAUNCH("cache_load", (k_cache_load<T, INT8, VEC>), unsigned(p.B * p.H * c.NG * parts), kThreads, smem, s, c,
               parts, slots, lengths, S, device_error_word());
    return GLA_OK;
}

template <typename T, bool INT8, bool VEC>
gla_status step_typed(const CacheProblem& p, const void* q, const void* k, const void* v, const float* la,
                      const int32_t* slots, const int32_t* lengths, void* o, cudaStream_t s) {
    const Pool c = pool_of(p);
    const GateArgs ga{la, p.gate, p.inv_tau, p.H};
    const size_t smem = step_smem(p);
    if (!allow_smem(k_cache_step<T, INT8, VEC>, smem)) return GLA_ERR_CUDA;
    GLA_LAUNCH("cache_step", (k_cache_step<T, INT8, VEC>), unsigned(p.B * p.H * c.NG), kThreads, smem, s, c,
               static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), ga, slots, lengths,
               static_cast<T*>(o), device_error_word());
    return GLA_OK;
}

// Four adjacent columns a lane where every row's fours are aligned (a width that is a multiple of 4).
#define GLA_CACHE_DISPATCH(fn, T, ...)                                                                 \
    (p.c.format == GLA_CACHE_INT8 ? (p.V % 4 == 0 ? fn<T true, true>(__VA_ARGS__) : fn<T true, false>(__VA_ARGS__)) \
                                  : (p.V % 4 == 0 ? fn<T false, true>(__VA_ARGS__) : fn<T false, false>(__VA_ARGS__)))
#define GLA_COMMA ,

}  // namespace

bool cache_supported(const CacheProblem& p) {
    if (p.B > (1 << 22) || p.H > 65535 || p.K > 65536 || p.V > 65536) return false;
    if (p.B * p.H * cdiv(p.V, kG) * cdiv(p.K, kWarps * kBatch) > (int64_t(1) << 30)) return false;
    return 4 * size_t(p.c.window) * (p.K + kG) + 16 * p.K + 8192 <= 200 * 1024;
}

gla_status cache_store(const CacheProblem& p, const float* S, const int32_t* slots, cudaStream_t s) {
    return GLA_CACHE_DISPATCH(store_typed, , p, S, slots, s);
}

gla_status cache_load(const CacheProblem& p, const int32_t* slots, const int32_t* lengths, float* S, cudaStream_t s) {
    return p.bf16 ? GLA_CACHE_DISPATCH(load_typed, __nv_bfloat16 GLA_COMMA, p, slots, lengths, S, s)
                  : GLA_CACHE_DISPATCH(load_typed, float GLA_COMMA, p, slots, lengths, S, s);
}

gla_status cache_step(const CacheProblem& p, const void* q, const void* k, const void* v, const float* la,
                      const int32_t* slots, const int32_t* lengths, void* o, cudaStream_t s) {
    return p.bf16 ? GLA_CACHE_DISPATCH(step_typed, __nv_bfloat16 GLA_COMMA, p, q, k, v, la, slots, lengths, o, s)
                  : GLA_CACHE_DISPATCH(step_typed, float GLA_COMMA, p, q, k, v, la, slots, lengths, o, s);
}

}  // namespace gla
