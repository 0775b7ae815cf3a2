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
constexpr int kSms = 148;
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
// Four codes to fp32, exactly. int8: 2^23 + 128 + code has the biased code in its low byte, and the subtraction is
// exact.
template <bool INT8>
__device__ __forceinline__ void decode4(uint32_t x, float2* y) {
    if constexpr (INT8) {
        const uint32_t u = x ^ 0x80808080u;
        const float2 off = make_float2(-8388736.f, -8388736.f);
        y[0] = add2(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440u)),
                                __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441u))), off);
        y[1] = add2(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442u)),
                                __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443u))), off);
    } else {
        y[0] = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(x & 0xffffu), __NV_E4M3)));
        y[1] = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(x >> 16), __NV_E4M3)));
    }
}
// scale of a group from the bits of its largest magnitude (NaN and inf order above every finite value)
template <bool INT8>
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    const float m = __uint_as_float(amax_bits);
    if (!(m < INFINITY)) return __uint_as_float(0x7fc00000u);
    return m < kTiny ? 0.f : __fmul_rn(m, INT8 ? float(1.0 / 127) : float(1.0 / 448));
}

// Four values to codes: round(y inv), ties to even. |y inv| stays below the largest code plus half a step, so nothing
// has to be clamped; the codes of a group held as zero or as NaN are 0 (inv = 0 gives 0, or NaN which is replaced).
template <bool INT8>
__device__ __forceinline__ uint32_t encode4(const float* y, float inv) {
    if (!(inv > 0.f)) return 0u;
    const float t0 = __fmul_rn(y[0], inv), t1 = __fmul_rn(y[1], inv), t2 = __fmul_rn(y[2], inv), t3 = __fmul_rn(y[3], inv);
    if constexpr (INT8) {
        const uint32_t lo = __byte_perm(uint32_t(__float2int_rn(t0)), uint32_t(__float2int_rn(t1)), 0x0040);
        const uint32_t hi = __byte_perm(uint32_t(__float2int_rn(t2)), uint32_t(__float2int_rn(t3)), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    } else {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(t0, t1), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(t2, t3), __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    }
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
    // the lane's columns of a [128] shared-memory row
    __device__ __forceinline__ void pairs(const float* row, float2* t) const {
        const int lane = threadIdx.x & 31;
        if constexpr (VEC) {
            const float4 x = *reinterpret_cast<const float4*>(row + 4 * lane);
            t[0] = make_float2(x.x, x.y);
            t[1] = make_float2(x.z, x.w);
        } else {
            t[0] = make_float2(row[lane], row[lane + 32]);
            t[1] = make_float2(row[lane + 64], row[lane + 96]);
        }
    }
    // place of the lane's e-th column in such a row
    __device__ __forceinline__ int at(int e) const {
        const int lane = threadIdx.x & 31;
        return VEC ? 4 * lane + e : lane + 32 * e;
    }
};

// Two or four adjacent elements as fp32, and four back.
__device__ __forceinline__ float2 ld2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 ld2(const __nv_bfloat16* p) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}
__device__ __forceinline__ void ld4(const float* p, float2* y) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    y[0] = make_float2(x.x, x.y);
    y[1] = make_float2(x.z, x.w);
}
__device__ __forceinline__ void ld4(const __nv_bfloat16* p, float2* y) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    y[0] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x.x));
    y[1] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x.y));
}
__device__ __forceinline__ void st4(float* p, const float2* y) {
    *reinterpret_cast<float4*>(p) = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
}
__device__ __forceinline__ void st4(__nv_bfloat16* p, const float2* y) {
    *reinterpret_cast<uint2*>(p) = make_uint2(tc::pack_bf16x2(y[0].x, y[0].y), tc::pack_bf16x2(y[1].x, y[1].y));
}

// Whether an earlier row of the call names the same slot (every thread of the block gets the answer).
__device__ __forceinline__ bool named_before(const int32_t* slots, int64_t b, int32_t slot) {
    int dup = 0;
    for (int64_t i = threadIdx.x; i < b; i += blockDim.x) dup |= slots[i] == slot;
    return __syncthreads_or(dup) != 0;
}

// Round `rows` <= ROWS rows of a group (four columns a lane) into their codes and scales. Lane i works out row i's scale
// and reciprocal for the whole warp.
template <bool INT8, int ROWS = kBatch, bool VEC>
__device__ __forceinline__ void put_rows(const Cols<VEC>& cols, const float (*y)[4], int rows, uint8_t* codes, int64_t V,
                                         float* scale, int64_t NG) {
    const int lane = threadIdx.x & 31;
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) m = max(m, __float_as_uint(y[i][e]) & 0x7fffffffu);
        m = __reduce_max_sync(0xffffffffu, m);
        if (lane == i) mine = m;
    }
    const float sc = scale_of<INT8>(mine), inv = sc > 0.f ? __frcp_rn(sc) : 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float r = __shfl_sync(0xffffffffu, inv, i);
        if (i < rows) cols.put_codes(codes + i * V, encode4<INT8>(y[i], r));
    }
    if (lane < rows) scale[lane * NG] = sc;
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
    for (int i = 0; i < kBatch; ++i) cols.load(S + (bh * c.K + (r0 + i < c.K ? r0 + i : c.K - 1)) * c.V, y[i]);
    const int32_t slot = slots[b];
    if (slot < 0) return;
    if (slot >= c.slots || named_before(slots, b, slot)) {
        if (threadIdx.x == 0) atomicOr(err, kErrBadRow);
        return;
    }
    const int64_t sh = slot * c.H + head;
    const int rows = c.K - r0 < kBatch ? c.K - r0 : kBatch;
    if (rows <= 0) return;
    put_rows<INT8>(cols, y, rows, c.codes + (sh * c.K + r0) * c.V, c.V, c.scale + (sh * c.K + r0) * c.NG + grp, c.NG);
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
template <typename T, bool STEP, bool VEC>
__device__ __forceinline__ void window_values(const Pool& c, int64_t sh, int64_t bh, int n, int grp,
                                              const T* __restrict__ vc, float* vs) {
    T* wv = static_cast<T*>(c.v) + sh * c.W * c.V;
    constexpr int E = VEC ? 4 : 1;  // columns a thread takes (a width that is a multiple of 4: they are aligned)
    for (int i = threadIdx.x; i < (n + (STEP ? 1 : 0)) * (kG / E); i += kThreads) {
        const int j = i / (kG / E), at = i % (kG / E) * E, col = grp * kG + at;
        const bool in = col < c.V;
        if constexpr (VEC) {
            float2 x[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            if (in) ld4(STEP && j == n ? vc + bh * c.V + col : wv + j * c.V + col, x);
            if (STEP && j == n && in) st4(wv + n * c.V + col, x);
            st4(vs + j * kG + at, x);
        } else {
            float x = 0.f;
            if (in) x = ldf(STEP && j == n ? vc + bh * c.V + col : wv + j * c.V + col);
            if (STEP && j == n && in) stf(wv + n * c.V + col, x);
            vs[j * kG + at] = x;
        }
    }
}

// ROWS rows (4 or 8) of the state: code x scale x decay + the window's outer products. value(j) gives the lane's four columns of
// token j's v, kt + j ld its keys.
template <bool INT8, int ROWS = kBatch, typename F>
__device__ __forceinline__ void form_rows(const uint32_t* codes, const float* scale, const float* decay, const float* kt,
                                          int ld, int used, F value, float (*out)[4]) {
    float2 y[ROWS][2];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        decode4<INT8>(codes[i], y[i]);
        const float2 f = make_float2(decay[i], decay[i]), g = make_float2(scale[i], scale[i]);
        y[i][0] = mul2(f, mul2(g, y[i][0]));
        y[i][1] = mul2(f, mul2(g, y[i][1]));
    }
    for (int j = 0; j < used; ++j) {
        float2 v[2];
        value(j, v);
        float k[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(kt + j * ld + i);
            k[i] = x.x, k[i + 1] = x.y, k[i + 2] = x.z, k[i + 3] = x.w;
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const float2 k2 = make_float2(k[i], k[i]);
            y[i][0] = fma2(k2, v[0], y[i][0]);
            y[i][1] = fma2(k2, v[1], y[i][1]);
        }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) out[i][0] = y[i][0].x, out[i][1] = y[i][0].y, out[i][2] = y[i][1].x, out[i][3] = y[i][1].y;
}

// ---- load -----------------------------------------------------------------------------------
// One block per (row of the call, head, group, kLoadRows state rows); 5 bytes an entry, 4 of them written. The window is
// read once a block, and a warp's codes are on their way before the window is worked out.
constexpr int kLoadRows = 128;

template <typename T, bool INT8, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) k_cache_load(Pool c, int parts, const int32_t* __restrict__ slots,
                                                            const int32_t* __restrict__ lengths, float* __restrict__ S,
                                                            int* err) {
    constexpr int BATCHES = kLoadRows / (kWarps * kBatch);
    extern __shared__ __align__(16) float sm[];
    const int64_t bhg = blockIdx.x / parts, bh = bhg / c.NG, b = bh / c.H, head = bh % c.H;
    const int part = int(blockIdx.x % parts), grp = int(bhg % c.NG);
    const Cols<VEC> cols(grp, c.V);
    const int first = part * kLoadRows, last = first + kLoadRows < c.K ? first + kLoadRows : c.K;
    const int w0 = int(threadIdx.x >> 5) * kBatch;  // this warp's first row of each batch of 64
    const int32_t slot = slots[b];
    const int32_t len = lengths ? lengths[b] : 0;
    bool live = slot >= 0;
    if (live && (slot >= c.slots || len < 0)) {
        live = false;
        if (threadIdx.x == 0) atomicOr(err, kErrBadRow);
    }
    if (!live) {
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        for (int r = first + int(threadIdx.x >> 5); r < last; r += kWarps) cols.store(S + (bh * c.K + r) * c.V, zero);
        return;
    }
    const int64_t sh = slot * c.H + head;
    const int n = len % c.W;
    uint32_t x[BATCHES][kBatch];
#pragma unroll
    for (int u = 0; u < BATCHES; ++u)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int r = first + u * kWarps * kBatch + w0 + i;
            x[u][i] = cols.codes(c.codes + (sh * c.K + (r < c.K ? r : c.K - 1)) * c.V);
        }
    float* kt = sm;                        // [W][kLoadRows]
    float* decay = kt + c.W * kLoadRows;   // [kLoadRows]
    float* scale = decay + kLoadRows;      // [kLoadRows]
    float* vs = scale + kLoadRows;         // [W][128]
    for (int r = threadIdx.x; r < kLoadRows; r += kThreads)
        scale[r] = first + r < last ? c.scale[(sh * c.K + first + r) * c.NG + grp] : 0.f;
    window_keys<T, false>(c, sh, bh, n, first, last, kLoadRows, nullptr, GateArgs{}, false, kt, decay);
    window_values<T, false, VEC>(c, sh, bh, n, grp, nullptr, vs);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < BATCHES; ++u) {
        const int r = u * kWarps * kBatch + w0;
        if (first + r >= last) break;
        float y[kBatch][4];
        form_rows<INT8>(x[u], scale + r, decay + r, kt + r, kLoadRows, n,
                        [&](int j, float2* t) { cols.pairs(vs + j * kG, t); }, y);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (first + r + i < last) cols.store(S + (bh * c.K + first + r + i) * c.V, y[i]);
    }
}

// ---- step -----------------------------------------------------------------------------------
// One block per (row of the call, head, group).
__host__ __device__ constexpr int round_up(int x, int m) { return (x + m - 1) / m * m; }

template <typename T, bool INT8, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) k_cache_step(Pool c, const T* __restrict__ q, const T* __restrict__ k,
                                                            const T* __restrict__ v, GateArgs ga,
                                                            const int32_t* __restrict__ slots,
                                                            const int32_t* __restrict__ lengths, T* __restrict__ o,
                                                            int* err) {
    constexpr int PASS = 2;  // batches a warp has in flight: 128 rows a block
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
    float* sc = wq + ld;               // [ld] scale
    float* p = sc + ld;                // [64] scores
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
    window_values<T, true, VEC>(c, sh, bh, n, grp, v, vs);
    for (int r = tid; r < ld; r += kThreads) {
        const float f = r < c.K ? scale[int64_t(r) * c.NG] : 0.f;
        sc[r] = f;
        wq[r] = r < c.K ? ldf(q + bh * c.K + r) * decay[r] * f : 0.f;
    }
    __syncthreads();
    for (int j = warp; j < used; j += kWarps) {
        float s = 0.f;
        for (int r = lane; r < c.K; r += 32) s = fmaf(ldf(q + bh * c.K + r), kt[j * ld + r], s);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane == 0) p[j] = s;
    }
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
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
                    float2 y[2];
                    decode4<INT8>(x[u][i], y);
                    const float2 w2 = make_float2(w[i], w[i]);
                    acc[0] = fma2(w2, y[0], acc[0]);
                    acc[1] = fma2(w2, y[1], acc[1]);
                }
            }
        }
    }
    red[warp * kG + cols.at(0)] = acc[0].x;
    red[warp * kG + cols.at(1)] = acc[0].y;
    red[warp * kG + cols.at(2)] = acc[1].x;
    red[warp * kG + cols.at(3)] = acc[1].y;
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
        float y[kBatch][4];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) z[i] = cols.codes(codes + int64_t(r + i < c.K ? r + i : c.K - 1) * c.V);
        form_rows<INT8>(z, sc + r, decay + r, kt + r, ld, used, [&](int j, float2* t) { cols.pairs(vs + j * kG, t); }, y);
        put_rows<INT8>(cols, y, c.K - r < kBatch ? c.K - r : kBatch, c.codes + (sh * c.K + r) * c.V, c.V,
                       scale + int64_t(r) * c.NG, c.NG);
    }
}

// ---- step, streamed ---------------------------------------------------------------------------
// For calls with large heads for every SM, of shapes that bulk copies can move (stream_plan below). One
// persistent block per SM takes its share of the heads; its warps have three parts, a head apart in time:
//   3 producers  one thread of the first keeps a head's codes coming, one contiguous stretch fetched in chunks through a
//                ring; the second's fetches its token, keys, log decays and scales ahead of them, the third's its values;
//   8 windows    form the keys k_j e^{D_j}, the scores p_j and the row weights q e^G scale of the next head, then write
//                out the head before: the readers' sums and the window's part;
//  16 readers    multiply the chunks (16 codes a lane) with the row weights.
// So memory does not wait for the window's exponentials or the reductions, and the ring (about 100 KB in flight an SM)
// covers the latency of DRAM. As one sequence of phases in one block the same work took twice the time.
//
// A head whose window is full costs several times the others (every entry takes `window` multiply-adds and is rounded),
// so it is split into its groups of 128 columns, which share nothing but the window: each is an item of its own that
// forms its columns of S_t, reads o from them and rounds them back. The blocks' shares are cut by cost, from the lengths
// that every block reads.
//
// A warp whose wait ran out (abort) neither writes nor announces anything more, so that the waits that depend on it run out
// too, and ends: readers and producers by themselves, window warps together, at their barrier. The producers let the
// copies that they issued land before they end.
constexpr int kReadWarps = 16, kWinWarps = 8;
constexpr int kReadThreads = kReadWarps * 32, kWinThreads = kWinWarps * 32;
constexpr int kStreamThreads = kReadThreads + kWinThreads + 96;
constexpr int kPasses = 4;                    // rows of a chunk that one lane reads
constexpr int kMaxRing = 12;
constexpr int kFoldRows = 4;                  // state rows a warp forms at a time (registers: 25 warps share the SM's)
constexpr int kMaxRows = 1024;                // rows of a call in one launch
constexpr int kDead = 255;
constexpr int kFoldCost = 12;                 // of a folding group, where an ordinary head costs its number of groups
constexpr size_t kStreamSmem = 227 * 1024 - 8192;  // less the static part

struct StreamPlan {
    int ring;         // chunks in flight
    int chunk_rows;   // state rows of a chunk
    int slices;       // rows read at a time
    int off_q, off_k, off_g, off_kw, off_gw, off_sc;   // what the window warps read
    int off_v, off_vw;                                 // what the readers read
    int off_kt, off_dec, off_wq, off_p, win_bytes;     // what the window warps leave (two heads' worth)
    int off_red, off_ring, chunk_bytes;
    size_t smem;      // 0: not for this shape
    long long wait_limit;
};

struct Item {
    int64_t bh, sh;  // row of the call x head; slot x head
    int n;           // tokens in the window
    int grp;         // >= 0: this group alone, and round it back; -1: the whole head
    int live;
};

__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     tc::smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
}

// A wait of a whole warp, which then agrees on its outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err, int* abort) {
    const bool ok = tc::mbar_wait_poll(bar, parity, err, abort);
    return __all_sync(0xffffffffu, ok) != 0;
}
// for waits that are long by design: the warp leaves the issue slots to the others
__device__ __forceinline__ bool warp_sleep(uint64_t* bar, uint32_t parity, int* err, int* abort,
                                           long long limit = tc::kWaitLimit) {
    const bool ok = tc::mbar_wait(bar, parity, err, abort, limit);
    return __all_sync(0xffffffffu, ok) != 0;
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(bar);
}

// acc += weight x 16 codes
template <bool INT8>
__device__ __forceinline__ void add_row(uint4 z, float weight, float2* acc) {
    const uint32_t x[4] = {z.x, z.y, z.z, z.w};
    const float2 w = make_float2(weight, weight);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float2 y[2];
        decode4<INT8>(x[e], y);
        acc[2 * e] = fma2(w, y[0], acc[2 * e]);
        acc[2 * e + 1] = fma2(w, y[1], acc[2 * e + 1]);
    }
}

// A ring position: stage and the parity of its turn.
struct Turn {
    int s = 0;
    uint32_t par = 0;
    __device__ __forceinline__ void next(int stages) {
        if (++s == stages) s = 0, par ^= 1u;
    }
};

// This block's items: of the folding groups (all of them first, then the other heads, in the order of `rows`) those
// whose cost begins in the block's share. A launch has at most kMaxItems groups of heads, all of which may fold, and
// the last share ends less than a unit per block behind the total.
constexpr int kMaxItems = 1 << 24;
static_assert(int64_t(kMaxItems) * kFoldCost + 2 * kSms < INT32_MAX, "Share counts in 32 bits");
struct Share {
    int f0, f1, h0, h1;
    __device__ __forceinline__ Share(int folds, int B, int H, int NG) {
        const int fg = folds * H * NG, hd = (B - folds) * H, total = fg * kFoldCost + hd * NG;
        const int per = (total + int(gridDim.x) - 1) / int(gridDim.x), lo = per * int(blockIdx.x), hi = lo + per;
        const auto first = [](int from, int cost, int most) {
            const int i = from <= 0 ? 0 : (from + cost - 1) / cost;
            return i < most ? i : most;
        };
        f0 = first(lo, kFoldCost, fg);
        f1 = first(hi, kFoldCost, fg);
        h0 = first(lo - fg * kFoldCost, NG, hd);
        h1 = first(hi - fg * kFoldCost, NG, hd);
    }
    __device__ __forceinline__ int count() const { return (f1 - f0) + (h1 - h0); }
};

template <typename T, bool INT8>
__global__ void __launch_bounds__(kStreamThreads, 1)
    k_cache_stream(Pool c, StreamPlan pl, int B, int64_t b0, const T* __restrict__ q, const T* __restrict__ k,
                   const T* __restrict__ v, GateArgs ga, const int32_t* __restrict__ slots,
                   const int32_t* __restrict__ lengths, T* __restrict__ o, int* err) {
    extern __shared__ __align__(128) char dyn[];
    // a: the window warps' inputs; b: the readers' values; w: the window warps' results
    // red: the readers' sums
    __shared__ uint64_t a_full, a_empty, b_full, b_empty, w_full[2], w_empty[2], red_full, red_empty;
    __shared__ uint64_t ring_full[kMaxRing], ring_empty[kMaxRing];
    __shared__ Item a_info, w_info[2];
    __shared__ __align__(16) int32_t row_slot[kMaxRows];
    __shared__ uint16_t rows[kMaxRows];
    __shared__ uint8_t row_n[kMaxRows];
    __shared__ int warp_folds[16], abort_flag;
    const int tid = int(threadIdx.x), lane = tid & 31, warp = tid >> 5;
    const int K = c.K, V = c.V, NG = c.NG;
    const bool gate_rows = ga.kind == kGateChannel || ga.kind == kGatePreact;
    // What every row of the call asks for: its place in the window (kDead: nothing), and the order in which the blocks
    // take the rows: those that fold first.
    int folds = 0;
    {
        static_assert(kMaxRows == 2 * 16 * 32 && kReadWarps == 16, "two rows a reader");
        int fold[2] = {0, 0}, before[2] = {0, 0};
        if (warp < 16) {
            int count = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int b = 64 * warp + 32 * u + lane;
                if (b < B) {
                    const int32_t len = lengths[b0 + b], slot = slots[b0 + b];
                    const bool named = slot >= 0, good = slot < c.slots && len >= 0;
                    if (named && !good && blockIdx.x == 0) atomicOr(err, kErrBadRow);
                    const int n = named && good ? len % c.W : kDead;
                    row_slot[b] = slot;  // a row that is refused names its slot all the same
                    row_n[b] = uint8_t(n);
                    fold[u] = n == c.W - 1;
                } else row_slot[b] = -1;
                const uint32_t m = __ballot_sync(0xffffffffu, fold[u]);
                before[u] = count + __popc(m & ((1u << lane) - 1));
                count += __popc(m);
            }
            if (lane == 0) warp_folds[warp] = count;
        } else if (tid == kReadThreads) {
            abort_flag = 0;
            tc::mbar_init(&a_full, 1), tc::mbar_init(&a_empty, kWinWarps);
            tc::mbar_init(&b_full, 1), tc::mbar_init(&b_empty, kWinWarps);
            tc::mbar_init(&red_full, kReadWarps), tc::mbar_init(&red_empty, kWinWarps);
            for (int i = 0; i < 2; ++i) tc::mbar_init(w_full + i, kWinWarps), tc::mbar_init(w_empty + i, kReadWarps);
            for (int i = 0; i < pl.ring; ++i) tc::mbar_init(ring_full + i, 1), tc::mbar_init(ring_empty + i, kReadWarps);
            tc::fence_barrier_init();
        }
        __syncthreads();
        int first = 0;
        for (int w = 0; w < 16; ++w) {
            if (w < warp) first += warp_folds[w];
            folds += warp_folds[w];
        }
        if (warp < 16) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int b = 64 * warp + 32 * u + lane;
                if (b < B) {
                    const int f = first + before[u];  // folding rows in front of b
                    rows[fold[u] ? f : folds + b - f] = uint16_t(b);
                }
            }
        }
        __syncthreads();
    }
    const Share share(folds, B, int(c.H), NG);
    const int items = share.count();
    const int chunks = (K + pl.chunk_rows - 1) / pl.chunk_rows;
    if (warp >= kReadWarps + kWinWarps) {
        // ---- producers (all lanes look for rows that name a slot twice, lane 0 does the rest)
        const int part = warp - (kReadWarps + kWinWarps);  // 0: codes, 1: keys, 2: values
        Turn rt;
        int checked = -1;       // the row looked at last, and whether it stands
        bool stands = false;
        bool ok = true;
        int sent = 0;           // items whose copies this part has issued (keys: padding rows count too)
        int64_t nch = 0;        // chunks so far
        for (int it = 0; it < items && ok; ++it) {
            Item x;
            int b, head;
            const bool fold = it < share.f1 - share.f0;
            if (fold) {
                const int f = share.f0 + it;
                x.grp = f % NG;
                b = rows[f / NG / int(c.H)];
                head = f / NG % int(c.H);
            } else {
                const int h = share.h0 + it - (share.f1 - share.f0);
                x.grp = -1;
                b = rows[folds + h / int(c.H)];
                head = h % int(c.H);
            }
            if (b != checked) {
                checked = b;
                stands = row_n[b] != kDead;
                if (stands) {
                    const int32_t slot = row_slot[b];
                    bool twice = false;
#pragma unroll 4
                    for (int i = lane; i < b; i += 32) twice |= row_slot[i] == slot;
#pragma unroll 4
                    for (int64_t i = lane; i < b0; i += 32) twice |= slots[i] == slot;
                    stands = !__any_sync(0xffffffffu, twice);
                    if (!stands && lane == 0) atomicOr(err, kErrBadRow);
                }
            }
            x.live = stands;
            x.bh = (b0 + b) * c.H + head;
            x.sh = stands ? row_slot[b] * c.H + head : 0;
            x.n = stands ? row_n[b] : 0;
            const uint32_t n = uint32_t(x.n), kb = uint32_t(K) * sizeof(T), vb = uint32_t(V) * sizeof(T);
            const uint32_t gb = uint32_t(K) * 4u, sb = uint32_t(K) * NG * 4u;
            if (part == 0) {
                if (lane == 0 && stands && !fold) {
                    for (int ch = 0; ch < chunks && ok; ++ch) {
                        if (nch >= pl.ring) ok = tc::mbar_wait_poll(ring_empty + rt.s, rt.par ^ 1u, err, &abort_flag);
                        if (!ok) break;
                        const int r0 = ch * pl.chunk_rows, m = K - r0 < pl.chunk_rows ? K - r0 : pl.chunk_rows;
                        tc::mbar_arrive_expect_tx(ring_full + rt.s, uint32_t(m) * V);
                        bulk_copy(dyn + pl.off_ring + rt.s * pl.chunk_bytes, c.codes + (x.sh * K + r0) * V, uint32_t(m) * V,
                                  ring_full + rt.s);
                        rt.next(pl.ring);
                        ++nch;
                    }
                }
            } else if (part == 1) {
                if (lane == 0) {
                    if (it > 0) ok = tc::mbar_wait_poll(&a_empty, uint32_t(it - 1) & 1u, err, &abort_flag);
                    if (ok) {
                        ++sent;
                        a_info = x;
                        if (!stands) tc::mbar_arrive(&a_full);
                        else {
                            tc::mbar_arrive_expect_tx(&a_full, 2 * kb + (gate_rows ? gb : 0u) + sb + n * (kb + gb));
                            if (n > 0) {
                                bulk_copy(dyn + pl.off_gw, c.la + x.sh * c.W * K, n * gb, &a_full);
                                bulk_copy(dyn + pl.off_kw, static_cast<T*>(c.k) + x.sh * c.W * K, n * kb, &a_full);
                            }
                            bulk_copy(dyn + pl.off_q, q + x.bh * K, kb, &a_full);
                            bulk_copy(dyn + pl.off_k, k + x.bh * K, kb, &a_full);
                            if (gate_rows) bulk_copy(dyn + pl.off_g, ga.g + x.bh * K, gb, &a_full);
                            bulk_copy(dyn + pl.off_sc, c.scale + x.sh * K * NG, sb, &a_full);
                        }
                    }
                }
            } else if (lane == 0 && stands) {
                // the values' stage is free once the head before has been written out
                if (sent > 0) ok = tc::mbar_wait(&b_empty, uint32_t(sent - 1) & 1u, err, &abort_flag);
                if (ok) {
                    ++sent;
                    tc::mbar_arrive_expect_tx(&b_full, (n + 1) * vb);
                    bulk_copy(dyn + pl.off_v, v + x.bh * V, vb, &b_full);
                    if (n > 0) bulk_copy(dyn + pl.off_vw, static_cast<T*>(c.v) + x.sh * c.W * V, n * vb, &b_full);
                }
            }
            ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
        }
        // Warps that gave up do not wait for the copies that were issued: this part does, before the block can end.
        if (lane == 0) {
            for (int i = 0; i < pl.ring && part == 0; ++i)
                if (nch > i) tc::mbar_drain(ring_full + i, uint32_t((nch - 1 - i) / pl.ring) & 1u);
            if (part == 1 && sent > 0) tc::mbar_drain(&a_full, uint32_t(sent - 1) & 1u);
            if (part == 2 && sent > 0) tc::mbar_drain(&b_full, uint32_t(sent - 1) & 1u);
        }
        return;
    }
    const T* vb = reinterpret_cast<const T*>(dyn + pl.off_v);
    const T* vw = reinterpret_cast<const T*>(dyn + pl.off_vw);
    float* red = reinterpret_cast<float*>(dyn + pl.off_red);  // [slices][V], or [warps][128]
    if (warp >= kReadWarps) {
        // ---- window warps
        const int t = tid - kReadThreads, w = warp - kReadWarps;
        const T* qb = reinterpret_cast<const T*>(dyn + pl.off_q);
        const T* kb = reinterpret_cast<const T*>(dyn + pl.off_k);
        const float* gb = reinterpret_cast<const float*>(dyn + pl.off_g);
        const T* kw = reinterpret_cast<const T*>(dyn + pl.off_kw);
        const float* gw = reinterpret_cast<const float*>(dyn + pl.off_gw);
        const float* sc = reinterpret_cast<const float*>(dyn + pl.off_sc);
        const int parts = K / 2 >= kWinThreads ? 1 : kWinThreads / (K / 2), part = parts == 1 ? 0 : t / (K / 2);
        Turn wt;
        Item last{0, 0, 0, -1, 0};
        bool ok = true;
        int lives = 0;
        // the head `last`: what the readers summed and, of an ordinary head, the window's part
        const auto finish = [&](const float* ps, int it) {
            ok = warp_sleep(&red_full, uint32_t(it) & 1u, err, &abort_flag);
            if (last.live) ok = ok && warp_sleep(&b_full, uint32_t(lives++) & 1u, err, &abort_flag);
            if (ok) {
                const int n = last.n, half = t & 1;
                const bool whole = last.grp < 0;
                T* put = static_cast<T*>(c.v) + (last.sh * c.W + n) * V;
                const int v0 = whole ? 0 : last.grp * kG, quads = (whole ? V : kG) / 4;
                const int rows = whole ? pl.slices : kReadWarps, ld = whole ? V : kG;
                // four columns of two lanes, which take every other row of the sums and every other token
                for (int i0 = 0; i0 < quads; i0 += kWinThreads / 2) {
                    const int i = i0 + (t >> 1);
                    const bool mine = i < quads;
                    // first column of the i-th four (the readers' layout)
                    const int at = whole ? i % (V / 16) * 16 + i / (V / 16) * 4 : v0 + 4 * i;
                    float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    if (last.live && mine) {
#pragma unroll 4
                        for (int r = half; r < rows; r += 2) {
                            float2 y[2];
                            ld4(red + r * ld + 4 * i, y);
                            s[0] = add2(s[0], y[0]);
                            s[1] = add2(s[1], y[1]);
                        }
                        if (whole) {
#pragma unroll 4
                            for (int j = half; j <= n; j += 2) {
                                float2 y[2];
                                ld4(j < n ? vw + j * V + at : vb + at, y);
                                const float2 pj = make_float2(ps[j], ps[j]);
                                s[0] = fma2(pj, y[0], s[0]);
                                s[1] = fma2(pj, y[1], s[1]);
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        s[e].x += __shfl_xor_sync(0xffffffffu, s[e].x, 1);
                        s[e].y += __shfl_xor_sync(0xffffffffu, s[e].y, 1);
                    }
                    if (mine && half == 0) st4(o + last.bh * V + at, s);
                    if (mine && half == 1 && last.live) {  // the token's value goes into the window
                        float2 y[2];
                        ld4(vb + at, y);
                        st4(put + at, y);
                    }
                }
            }
            if (ok) warp_arrive(&red_empty);
            if (ok && last.live) warp_arrive(&b_empty);
        };
        for (int it = 0; it < items; ++it) {
            ok = ok && warp_sleep(&a_full, uint32_t(it) & 1u, err, &abort_flag, pl.wait_limit);
            if (it >= 2) ok = ok && warp_sleep(w_empty + wt.s, wt.par ^ 1u, err, &abort_flag);
            Item x{0, 0, 0, -1, 0};
            if (ok) x = a_info;
            char* win = dyn + pl.off_kt + wt.s * pl.win_bytes;
            float* kt = reinterpret_cast<float*>(win);                                // [W][K] k_j e^{D_j}
            float* dec = reinterpret_cast<float*>(win + (pl.off_dec - pl.off_kt));    // [K] e^G
            float* wq = reinterpret_cast<float*>(win + (pl.off_wq - pl.off_kt));      // [groups][K] q e^G scale; folding: q, scale
            float* ps = reinterpret_cast<float*>(win + (pl.off_p - pl.off_kt));       // [64] scores
            const int n = x.n;
            const int64_t place = x.sh * c.W + n;  // of the token in the window; k and log a are put there once a head
            if (x.live) {
                // two channels a thread: all of them at a time, or as many parts of the window as there are threads
                for (int r = 2 * (parts == 1 ? t : t - part * (K / 2)); r < K && part < parts; r += 2 * kWinThreads) {
                    const int lo = n * part / parts, hi = n * (part + 1) / parts;  // this part's tokens
                    float2 la;
                    if (!gate_rows) la.x = la.y = gate_log_alpha(ga, x.bh, 0, r, 1, K);
                    else {
                        la = ld2(gb + r);
                        if (ga.kind == kGatePreact)
                            la = make_float2(logsigmoid_f(la.x) * ga.inv_tau, logsigmoid_f(la.y) * ga.inv_tau);
                    }
                    const auto decay = [](float2 D) {
                        const float2 e = mul2(D, make_float2(tc::kLog2e, tc::kLog2e));
                        return make_float2(tc::exp2_ftz(e.x), tc::exp2_ftz(e.y));
                    };
                    float2 D = la;
#pragma unroll 4
                    for (int j = n - 1; j >= hi; --j) D = add2(D, ld2(gw + j * K + r));
#pragma unroll 4
                    for (int j = hi - 1; j >= lo; --j) {
                        *reinterpret_cast<float2*>(kt + j * K + r) = mul2(ld2(kw + j * K + r), decay(D));
                        D = add2(D, ld2(gw + j * K + r));
                    }
                    if (part == parts - 1) {
                        *reinterpret_cast<float2*>(kt + n * K + r) = ld2(kb + r);
                        if (x.grp <= 0) {
                            T* put = static_cast<T*>(c.k) + place * K + r;
                            put[0] = kb[r];
                            put[1] = kb[r + 1];
                            *reinterpret_cast<float2*>(c.la + place * K + r) = la;
                        }
                    }
                    if (part == 0) {
                        const float2 qr = ld2(qb + r), d = decay(D), qd = mul2(qr, d);
                        *reinterpret_cast<float2*>(dec + r) = d;
                        if (x.grp < 0) {
                            for (int g = 0; g < NG; ++g)
                                *reinterpret_cast<float2*>(wq + g * K + r) =
                                    mul2(qd, make_float2(sc[r * NG + g], sc[(r + 1) * NG + g]));
                        } else {
                            *reinterpret_cast<float2*>(wq + r) = qr;
                            *reinterpret_cast<float2*>(wq + K + r) =
                                make_float2(sc[r * NG + x.grp], sc[(r + 1) * NG + x.grp]);
                        }
                    }
                }
            }
            if (!tc::named_all(2, kWinThreads, ok)) return;
            if (x.live && x.grp < 0) {
                for (int j = w; j <= n; j += kWinWarps) {
                    float s = 0.f;
                    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll 4
                    for (int r = 2 * lane; r < K; r += 64) s2 = fma2(ld2(qb + r), ld2(kt + j * K + r), s2);
                    s = s2.x + s2.y;
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
                    if (lane == 0) ps[j] = s;
                }
            }
            if (t == 0) w_info[wt.s] = x;
            warp_arrive(w_full + wt.s);
            warp_arrive(&a_empty);
            if (it > 0) finish(reinterpret_cast<const float*>(dyn + pl.off_p + (wt.s ^ 1) * pl.win_bytes), it - 1);
            last = x;
            wt.next(2);
        }
        if (!tc::named_all(2, kWinThreads, ok)) return;
        if (items > 0) finish(reinterpret_cast<const float*>(dyn + pl.off_p + (wt.s ^ 1) * pl.win_bytes), items - 1);
        return;
    }
    // ---- readers
    const int unit = tid / (kG / 16), ugrp = unit % NG, slice = unit / NG;  // eight lanes read a group's row
    const int ucol = ugrp * kG + tid % (kG / 16) * 16;
    const bool reads = slice < pl.slices;
    Turn wt, rt;
    int lives = 0;
    // the sums of the head before have been taken (waited for by padding rows too: no part gets two heads ahead)
    const auto last_written = [&](int it) {
        return it == 0 || warp_wait(&red_empty, uint32_t(it - 1) & 1u, err, &abort_flag);
    };
    for (int it = 0; it < items; ++it) {
        if (!warp_wait(w_full + wt.s, wt.par, err, &abort_flag)) return;
        const Item x = w_info[wt.s];
        const char* win = dyn + pl.off_kt + wt.s * pl.win_bytes;
        const float* kt = reinterpret_cast<const float*>(win);
        const float* dec = reinterpret_cast<const float*>(win + (pl.off_dec - pl.off_kt));
        const float* wq = reinterpret_cast<const float*>(win + (pl.off_wq - pl.off_kt));
        if (x.live && x.grp < 0) {
            float2 acc[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = make_float2(0.f, 0.f);
            const float* w = wq + ugrp * K + slice;
            for (int ch = 0; ch < chunks; ++ch, w += pl.chunk_rows) {
                if (!warp_wait(ring_full + rt.s, rt.par, err, &abort_flag)) return;
                const int rn = K - ch * pl.chunk_rows;  // rows from the chunk's first
                const char* src = dyn + pl.off_ring + rt.s * pl.chunk_bytes + ucol;
                if (reads) {
                    // rows behind the state's last one are read as the chunk's first with weight 0
                    uint4 z[kPasses];
                    float u[kPasses];
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) {
                        const int r = slice + i * pl.slices;
                        z[i] = *reinterpret_cast<const uint4*>(src + (r < rn ? r * V : 0));
                        u[i] = r < rn ? w[i * pl.slices] : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < kPasses; ++i) add_row<INT8>(z[i], u[i], acc);
                }
                warp_arrive(ring_empty + rt.s);
                rt.next(pl.ring);
            }
            if (!last_written(it)) return;
            if (reads) {
                // the e-th four columns of all lanes stand together: neighbouring lanes write neighbouring words
                float* d = red + slice * V + ucol / 4;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<float4*>(d + e * (V / 4)) =
                        make_float4(acc[2 * e].x, acc[2 * e].y, acc[2 * e + 1].x, acc[2 * e + 1].y);
            }
        } else if (x.live) {
            // one group of a head whose window is full
            if (!warp_wait(&b_full, uint32_t(lives) & 1u, err, &abort_flag)) return;
            const int n = x.n, used = n + 1;
            uint8_t* codes = c.codes + x.sh * K * V;
            float* scale = c.scale + x.sh * K * NG + x.grp;
            const Cols<true> cols(x.grp, V);
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
            for (int r = warp * kFoldRows; r < K; r += kReadWarps * kFoldRows) {
                uint32_t z[kFoldRows];
                float y[kFoldRows][4];
#pragma unroll
                for (int i = 0; i < kFoldRows; ++i) z[i] = cols.codes(codes + int64_t(r + i) * V);
                const auto value = [&](int j, float2* t) {
                    ld4((j < n ? vw + j * V : vb) + cols.col[0], t);
                };
                form_rows<INT8, kFoldRows>(z, wq + K + r, dec + r, kt + r, K, used, value, y);
#pragma unroll
                for (int i = 0; i < kFoldRows; ++i) {
                    const float qr = wq[r + i];
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[e] = fmaf(qr, y[i][e], acc[e]);
                }
                put_rows<INT8, kFoldRows>(cols, y, kFoldRows, codes + int64_t(r) * V, V, scale + int64_t(r) * NG, NG);
            }
            if (!last_written(it)) return;
            *reinterpret_cast<float4*>(red + warp * kG + 4 * lane) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        } else if (!last_written(it)) return;
        lives += x.live;
        warp_arrive(&red_full);
        warp_arrive(w_empty + wt.s);
        wt.next(2);
    }
}

// The most shared memory that a block of the kernels without a ring takes: cache_supported admits the windows and widths
// whose step (step_smem) stays below it, and a load takes at most 66,560 bytes (64 tokens).
constexpr size_t kHeadSmem = 200 * 1024;

Pool pool_of(const CacheProblem& p) {
    return Pool{static_cast<uint8_t*>(p.c.codes), p.c.scale, p.c.k, p.c.v, p.c.log_a, p.c.slots, p.c.window,
                p.H, int(p.K), int(p.V), int(cdiv(p.V, kG))};
}

size_t step_smem(const CacheProblem& p) {
    const size_t ld = size_t(round_up(int(p.K), kBatch));
    return sizeof(float) * (size_t(p.c.window) * (ld + kG) + 3 * ld + 64 + kWarps * kG);
}
size_t load_smem(const CacheProblem& p) {
    return sizeof(float) * (size_t(p.c.window) * (kLoadRows + kG) + 2 * kLoadRows);
}

// The attribute belongs to the kernel, which other host threads may be about to launch with another window or width: so
// every call above the default of 48 KB asks for `most`, the largest size that any call of the kernel may take, and none
// lowers the limit under another's launch.
template <typename K>
bool allow_smem(K kernel, size_t bytes, size_t most) {
    return bytes <= 48 * 1024 || (bytes <= most && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                        int(most)) == cudaSuccess);
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
    const int parts = int(cdiv(p.K, kLoadRows));
    const size_t smem = load_smem(p);
    if (!allow_smem(k_cache_load<T, INT8, VEC>, smem, kHeadSmem)) return GLA_ERR_CUDA;
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
    if (!allow_smem(k_cache_step<T, INT8, VEC>, smem, kHeadSmem)) return GLA_ERR_CUDA;
    GLA_LAUNCH("cache_step", (k_cache_step<T, INT8, VEC>), unsigned(p.B * p.H * c.NG), kThreads, smem, s, c,
               static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), ga, slots, lengths,
               static_cast<T*>(o), device_error_word());
    return GLA_OK;
}

// Shared memory and tiling of the streamed step, or smem = 0 where it does not apply: bulk copies want every stretch (a
// token's k, v and log a, a window, a row of scales) to be a multiple of 16 bytes, the readers want whole groups, and a
// window must fit beside a ring of at least three chunks. A head costs it about 4 us of phases besides its codes, and a
// call 6 us before the first sums; k_cache_step starts a block for every group and pays those in parallel. So it takes
// the calls with a head of at least 96 K entries for every SM: 1024 heads of 256 x 512 in 42 us against 73, 256 heads in
// 18.6 against 20.6, 148 heads in 11.9 against 11.8, but 1024 heads of 128 x 256 in 33 against 27.
StreamPlan stream_plan(const CacheProblem& p) {
    StreamPlan pl{};
    const int K = int(p.K), V = int(p.V), W = p.c.window, e = p.bf16 ? 2 : 4;
    if (p.B * p.H < kSms || p.K * p.V < 96 * 1024 || p.H * cdiv(p.V, kG) > (1 << 20)) return pl;
    if (K % 8 != 0 || K > 4096 || V % kG != 0 || V > 2048) return pl;
    const int NG = V / kG;
    pl.slices = kReadThreads / (kG / 16) / NG;
    int at = 0;
    const auto take = [&](int bytes) {
        const int here = at;
        at += round_up(bytes, 128);
        return here;
    };
    pl.off_q = take(K * e);
    pl.off_k = take(K * e);
    pl.off_g = take(K * 4);
    pl.off_kw = take((W - 1) * K * e);
    pl.off_gw = take((W - 1) * K * 4);
    pl.off_sc = take(K * NG * 4);
    pl.off_v = take(V * e);
    pl.off_vw = take((W - 1) * V * e);
    pl.off_kt = take(W * K * 4);
    pl.off_dec = take(K * 4);
    pl.off_wq = take(K * (NG > 2 ? NG : 2) * 4);
    pl.off_p = take(64 * 4);
    pl.win_bytes = at - pl.off_kt;
    at += pl.win_bytes;
    const int sums = pl.slices * V > kReadWarps * kG ? pl.slices * V : kReadWarps * kG;
    pl.off_red = take(sums * 4);
    pl.off_ring = at;
    pl.chunk_rows = kPasses * pl.slices;
    pl.chunk_bytes = round_up(pl.chunk_rows * V, 128);
    const int64_t room = int64_t(kStreamSmem) - at, ring = room > 0 ? room / pl.chunk_bytes : 0;
    if (ring < 3) return pl;
    pl.ring = int(ring < kMaxRing ? ring : kMaxRing);
    pl.smem = size_t(at) + size_t(pl.ring) * pl.chunk_bytes;
    pl.wait_limit = wait_limit();
    return pl;
}

template <typename T, bool INT8>
gla_status stream_typed(const CacheProblem& p, const StreamPlan& pl, const void* q, const void* k, const void* v,
                        const float* la, const int32_t* slots, const int32_t* lengths, void* o, cudaStream_t s) {
    const Pool c = pool_of(p);
    const GateArgs ga{la, p.gate, p.inv_tau, p.H};
    if (!allow_smem(k_cache_stream<T, INT8>, pl.smem, kStreamSmem)) return GLA_ERR_CUDA;
    const int64_t fit = kMaxItems / (p.H * c.NG), step = fit < kMaxRows ? fit : kMaxRows;  // rows a launch
    for (int64_t b0 = 0; b0 < p.B; b0 += step) {
        const int n = int(p.B - b0 < step ? p.B - b0 : step);
        GLA_LAUNCH("cache_step", (k_cache_stream<T, INT8>), unsigned(kSms), kStreamThreads, pl.smem, s, c, pl, n, b0,
                   static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), ga, slots, lengths,
                   static_cast<T*>(o), device_error_word());
    }
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
    return 4 * size_t(p.c.window) * (p.K + kG) + 16 * p.K + 8192 <= kHeadSmem;
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
    const StreamPlan pl = stream_plan(p);
    if (pl.smem > 0) {
        const bool i8 = p.c.format == GLA_CACHE_INT8;
        if (p.bf16)
            return i8 ? stream_typed<__nv_bfloat16, true>(p, pl, q, k, v, la, slots, lengths, o, s)
                      : stream_typed<__nv_bfloat16, false>(p, pl, q, k, v, la, slots, lengths, o, s);
        return i8 ? stream_typed<float, true>(p, pl, q, k, v, la, slots, lengths, o, s)
                  : stream_typed<float, false>(p, pl, q, k, v, la, slots, lengths, o, s);
    }
    return p.bf16 ? GLA_CACHE_DISPATCH(step_typed, __nv_bfloat16 GLA_COMMA, p, q, k, v, la, slots, lengths, o, s)
                  : GLA_CACHE_DISPATCH(step_typed, float GLA_COMMA, p, q, k, v, la, slots, lengths, o, s);
}

}  // namespace gla
