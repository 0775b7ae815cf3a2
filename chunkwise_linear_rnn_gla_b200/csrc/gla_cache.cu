// Recurrent-state cache (include/gla.h, "recurrent-state cache"): matrix states held in 8 bits in a pool of slots,
// the last few tokens of each sequence beside them, and the decode step that reads both:
//     S_t = diag(e^G) (scale code) + sum_j (k_j e^{D_j})^T v_j,   o_t = q S_t.
// The decay acts on whole rows, so a scale per row (and 128 columns) carries it exactly; the recurrent form is that
// of the decode step (podcast.app episode page, summary: a gated memory updated once per token).
//
// One block of 128 threads per (row, head, group of 128 columns); a thread has one column and walks the state's rows.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "gla_common.cuh"
#include "gla_gate.cuh"
#include "gla_internal.h"

namespace gla {
namespace {

constexpr int kG = kCacheGroup;
constexpr float kTiny = 1e-30f;  // a group whose largest magnitude is below this is held as zero

__device__ __forceinline__ float decode8(uint8_t b, bool int8) {
    if (int8) return float(int8_t(b));
    __nv_fp8_e4m3 x;
    x.__x = b;
    return float(x);
}

// scale of a group from the bits of its largest magnitude (NaN and inf order above every finite value)
__device__ __forceinline__ float scale_of(uint32_t amax_bits, bool int8) {
    const float m = __uint_as_float(amax_bits);
    if (!(m < INFINITY)) return __uint_as_float(0x7fc00000u);
    return m < kTiny ? 0.f : __fmul_rn(m, int8 ? float(1.0 / 127) : float(1.0 / 448));
}

__device__ __forceinline__ uint8_t encode8(float x, float inv, bool int8) {
    const float y = __fmul_rn(x, inv);
    if (int8) return uint8_t(int8_t(int(fminf(fmaxf(rintf(y), -127.f), 127.f))));
    return uint8_t(__nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3));
}

// 1 / scale, 0 for a group held as zero (its codes are 0 then) and for one held as NaN
__device__ __forceinline__ float inv_of(float scale) { return scale > 0.f ? __frcp_rn(scale) : 0.f; }

// largest magnitude (as bits) over the block's 128 threads
__device__ __forceinline__ uint32_t block_max(uint32_t x, uint32_t* red) {
    x = __reduce_max_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = max(max(red[0], red[1]), max(red[2], red[3]));
    __syncthreads();
    return x;
}

__device__ __forceinline__ bool named_before(const int32_t* slots, int64_t b, int32_t slot) {
    int dup = 0;
    for (int64_t i = threadIdx.x; i < b; i += blockDim.x) dup |= slots[i] == slot;
    return __syncthreads_or(dup) != 0;
}

struct Pool {
    uint8_t* codes;
    float* scale;
    void* k;
    void* v;
    float* la;
    int64_t slots;
    int W;
    bool int8;
    int64_t H;
    int K, V, NG;
};

__global__ void __launch_bounds__(kG) k_cache_store(Pool c, const float* __restrict__ S,
                                                    const int32_t* __restrict__ slots, int* err) {
    __shared__ uint32_t red[4];
    const int64_t bh = blockIdx.x / c.NG, b = bh / c.H, head = bh % c.H;
    const int grp = int(blockIdx.x % c.NG), col = grp * kG + int(threadIdx.x);
    const int32_t slot = slots[b];
    if (slot < 0) return;
    if (slot >= c.slots || named_before(slots, b, slot)) {
        if (threadIdx.x == 0) atomicOr(err, kErrBadRow);
        return;
    }
    const int64_t sh = slot * c.H + head;
    for (int r = 0; r < c.K; ++r) {
        const float x = col < c.V ? S[(bh * c.K + r) * c.V + col] : 0.f;
        const float sc = scale_of(block_max(__float_as_uint(fabsf(x)), red), c.int8);
        if (col < c.V) c.codes[(sh * c.K + r) * c.V + col] = sc > 0.f ? encode8(x, inv_of(sc), c.int8) : uint8_t(0);
        if (threadIdx.x == 0) c.scale[(sh * c.K + r) * c.NG + grp] = sc;
    }
}

// MODE 0: read the states back (S); 1: decode step (o, window, and the slot when the window fills).
template <typename T, int STEP>
__global__ void __launch_bounds__(kG) k_cache_read(Pool c, const T* __restrict__ q, const T* __restrict__ k,
                                                   const T* __restrict__ v, GateArgs ga,
                                                   const int32_t* __restrict__ slots,
                                                   const int32_t* __restrict__ lengths, float* __restrict__ S,
                                                   T* __restrict__ o, int* err) {
    extern __shared__ float sm[];
    __shared__ uint32_t red[4];
    const int64_t bh = blockIdx.x / c.NG, b = bh / c.H, head = bh % c.H;
    const int grp = int(blockIdx.x % c.NG), tid = int(threadIdx.x), col = grp * kG + tid;
    const int32_t slot = slots[b];
    const int32_t len = lengths ? lengths[b] : 0;
    bool live = slot >= 0;
    if (live && (slot >= c.slots || len < 0 || (STEP && named_before(slots, b, slot)))) {
        live = false;
        if (tid == 0) atomicOr(err, kErrBadRow);
    }
    if (!live) {
        if (col < c.V) {
            if (STEP) stf(o + bh * c.V + col, 0.f);
            else
                for (int r = 0; r < c.K; ++r) S[(bh * c.K + r) * c.V + col] = 0.f;
        }
        return;
    }
    const int n = len % c.W, used = n + STEP;  // tokens in the window, with the one of this call
    float* kt = sm;                             // [used][K] k_j e^{D_j}
    float* vw = kt + c.W * c.K;                 // [used][128]
    float* decay = vw + c.W * kG;               // [K] e^G
    const int64_t sh = slot * c.H + head;
    T* wk = static_cast<T*>(c.k) + sh * c.W * c.K;
    T* wv = static_cast<T*>(c.v) + sh * c.W * c.V;
    float* wl = c.la + sh * c.W * c.K;
    for (int r = tid; r < c.K; r += kG) {
        float D = 0.f;
        if (STEP) {
            const float la = gate_log_alpha(ga, bh, 0, r, 1, c.K);
            kt[n * c.K + r] = ldf(k + bh * c.K + r);
            if (grp == 0) {
                wk[n * c.K + r] = k[bh * c.K + r];
                wl[n * c.K + r] = la;
            }
            D = la;
        }
        for (int j = n - 1; j >= 0; --j) {
            kt[j * c.K + r] = ldf(wk + j * c.K + r) * expf(D);
            D += wl[j * c.K + r];
        }
        decay[r] = expf(D);
    }
    for (int j = 0; j < used; ++j) vw[j * kG + tid] = col < c.V ? (j == n ? ldf(v + bh * c.V + col) : ldf(wv + j * c.V + col)) : 0.f;
    if (STEP && col < c.V) wv[n * c.V + col] = v[bh * c.V + col];
    __syncthreads();
    const bool fold = STEP && used == c.W;
    float acc = 0.f;
    for (int r = 0; r < c.K; ++r) {
        const int64_t i = (sh * c.K + r) * c.V + col, si = (sh * c.K + r) * c.NG + grp;
        const float sc = c.scale[si];
        float x = col < c.V ? decay[r] * (sc * decode8(c.codes[i], c.int8)) : 0.f;
        for (int j = 0; j < used; ++j) x = fmaf(kt[j * c.K + r], vw[j * kG + tid], x);
        if (!STEP) {
            if (col < c.V) S[(bh * c.K + r) * c.V + col] = x;
            continue;
        }
        acc = fmaf(ldf(q + bh * c.K + r), x, acc);
        if (fold) {
            const float ns = scale_of(block_max(__float_as_uint(fabsf(x)), red), c.int8);
            if (col < c.V) c.codes[i] = ns > 0.f ? encode8(x, inv_of(ns), c.int8) : uint8_t(0);
            if (tid == 0) c.scale[si] = ns;
        }
    }
    if (STEP && col < c.V) stf(o + bh * c.V + col, acc);
}

Pool pool_of(const CacheProblem& p) {
    return Pool{static_cast<uint8_t*>(p.c.codes), p.c.scale, p.c.k, p.c.v, p.c.log_a, p.c.slots, p.c.window,
                p.c.format == GLA_CACHE_INT8, p.H, int(p.K), int(p.V), int(cdiv(p.V, kG))};
}

size_t smem_of(const CacheProblem& p) { return sizeof(float) * (size_t(p.c.window) * (p.K + kG) + p.K); }

template <typename T, int STEP>
gla_status read_typed(const CacheProblem& p, const void* q, const void* k, const void* v, const float* la,
                      const int32_t* slots, const int32_t* lengths, float* S, void* o, cudaStream_t s) {
    const Pool c = pool_of(p);
    const GateArgs ga{la, p.gate, p.inv_tau, p.H};
    const size_t smem = smem_of(p);
    if (smem > 48 * 1024 && cudaFuncSetAttribute(k_cache_read<T, STEP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 int(smem)) != cudaSuccess)
        return GLA_ERR_CUDA;
    GLA_LAUNCH(STEP ? "cache_step" : "cache_load", (k_cache_read<T, STEP>), unsigned(p.B * p.H * c.NG), kG, smem, s, c,
               static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), ga, slots, lengths, S,
               static_cast<T*>(o), device_error_word());
    return GLA_OK;
}

}  // namespace

bool cache_supported(const CacheProblem& p) {
    if (p.B > (1 << 22) || p.H > 65535 || p.K > 65536 || p.V > 65536) return false;
    if (p.B * p.H * cdiv(p.V, kG) > (int64_t(1) << 30)) return false;
    return 4 * size_t(p.c.window) * (p.K + kG) + 16 * p.K + 8192 <= 200 * 1024;
}

gla_status cache_store(const CacheProblem& p, const float* S, const int32_t* slots, cudaStream_t s) {
    const Pool c = pool_of(p);
    GLA_LAUNCH("cache_store", k_cache_store, unsigned(p.B * p.H * c.NG), kG, 0, s, c, S, slots, device_error_word());
    return GLA_OK;
}

gla_status cache_load(const CacheProblem& p, const int32_t* slots, const int32_t* lengths, float* S, cudaStream_t s) {
    return p.bf16 ? read_typed<__nv_bfloat16, 0>(p, nullptr, nullptr, nullptr, nullptr, slots, lengths, S, nullptr, s)
                  : read_typed<float, 0>(p, nullptr, nullptr, nullptr, nullptr, slots, lengths, S, nullptr, s);
}

gla_status cache_step(const CacheProblem& p, const void* q, const void* k, const void* v, const float* la,
                      const int32_t* slots, const int32_t* lengths, void* o, cudaStream_t s) {
    return p.bf16 ? read_typed<__nv_bfloat16, 1>(p, q, k, v, la, slots, lengths, nullptr, o, s)
                  : read_typed<float, 1>(p, q, k, v, la, slots, lengths, nullptr, o, s);
}

}  // namespace gla
