// qf_adamw.cuh -- sm_100a kernels of the optimizer step: the AdamW update of many tensors
// at once with FP32 or 8-bit states, and the global gradient norm that clips it.
//
// Mathematics (binary32, one rounding per operation; t = step number):
//   g' = s g            m = b1 m + (1 - b1) g'      v = b2 v + (1 - b2) (g' g')
//   root = sqrt(v)      p = p (1 - lr wd) - (m / (root rs2 + eps)) ss
//   ss = lr / (1 - b1^t),  rs2 = 1 / sqrt(1 - b2^t)   (binary64, rounded once)
// 8-bit states keep m and root(!) as E4M3 codes with one FP32 scale per 256 elements.
// root instead of v halves the exponent range, so E4M3's 17 binades of root cover 34 of
// v; the step needs root anyway, so the square root is not an extra one.  A positive root
// never gets code 0: the divisor of a coordinate that has moved stays away from eps.
//
// Bound: HBM.  Per element the kernel must move p twice, g once and the states twice:
// 26 B (FP32 p and states, BF16 g) or 14.06 B (8-bit states) for about 20 operations.
// Layout: a warp takes one 256-element block at a time, two 4-element vectors per lane,
// so every FP32 access is a whole 512-byte warp transaction, a block's scale is one
// warp reduction (redux.sync on the bit patterns) and no shared memory is needed.
#pragma once

#include <cstdint>

namespace qf {

constexpr int kParamBlock = 256;        // elements behind one 8-bit scale
constexpr int kAdamThreads = 256;
constexpr int kSmallP = 8;              // descriptor table sizes; 352 x 88 B = 31 KB of the
constexpr int kLargeP = 352;            // 32 KB of kernel parameters
constexpr int kNormMaxGrid = 2048;

struct DevParam {
    void* p;
    const void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    uint16_t* w;
    double wd;
    int64_t numel;
    int64_t unit_begin;
    int32_t group;
    int32_t pad;
};

// Scalars of one step.  ss and rs2 are the host's when the step number and the learning
// rate came by value; otherwise each CTA forms them from d_step / d_lr, by the same
// function in the same binary64 operations.
struct AdamScalars {
    double lr, beta1, beta2;
    float b1, omb1, b2, omb2, eps;
    float ss, rs2;
    const float* d_lr;
    const int64_t* d_step;
    const float* d_grad_scale;
    int64_t step;
};

template <int MAXT>
struct ParamTable {
    DevParam t[MAXT];
    AdamScalars h;
    int64_t total_units;
    uint32_t* amax;                      // per tie group, FP32 bits; NULL: not wanted
    int n;
};

__host__ __device__ inline double ipow(double b, int64_t n) {
    double r = 1.0;
    for (; n > 0; n >>= 1, b *= b)
        if (n & 1) r *= b;
    return r;
}
__host__ __device__ inline void adam_step_scalars(double lr, double beta1, double beta2,
                                                  int64_t step, float* ss, float* rs2) {
    *ss = (float)(lr / (1.0 - ipow(beta1, step)));
    *rs2 = (float)(1.0 / sqrt(1.0 - ipow(beta2, step)));
}

#ifdef __CUDACC__

// ---- vectors of four elements at element offset e; n = elements left (>= 4: whole)
__device__ __forceinline__ void load4(const float* p, int64_t e, int64_t n, float* x) {
    if (n >= 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + e);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = i < n ? p[e + i] : 0.0f;
    }
}
__device__ __forceinline__ void load4(const uint16_t* p, int64_t e, int64_t n, float* x) {
    if (n >= 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(p + e);
        x[0] = __uint_as_float(v.x << 16); x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16); x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = i < n ? __uint_as_float((uint32_t)p[e + i] << 16) : 0.0f;
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float hi, float lo) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void store4(float* p, int64_t e, int64_t n, const float* x) {
    if (n >= 4) {
        *reinterpret_cast<float4*>(p + e) = make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[e + i] = x[i];
    }
}
__device__ __forceinline__ void store4(uint16_t* p, int64_t e, int64_t n, const float* x) {
    const uint32_t lo = pack_bf16(x[1], x[0]), hi = pack_bf16(x[3], x[2]);
    if (n >= 4) {
        *reinterpret_cast<uint2*>(p + e) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[e + i] = (uint16_t)((i < 2 ? lo : hi) >> (16 * (i & 1)));
    }
}
__device__ __forceinline__ uint32_t load_codes4(const uint8_t* p, int64_t e, int64_t n) {
    if (n >= 4) return *reinterpret_cast<const uint32_t*>(p + e);
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) c |= (uint32_t)p[e + i] << (8 * i);
    return c;
}
__device__ __forceinline__ void store_codes4(uint8_t* p, int64_t e, int64_t n, uint32_t c) {
    if (n >= 4) {
        *reinterpret_cast<uint32_t*>(p + e) = c;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) p[e + i] = (uint8_t)(c >> (8 * i));
}
__device__ __forceinline__ void decode_e4m3x4(uint32_t c, float* x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h2;
        const unsigned short h = (unsigned short)(c >> (16 * i));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(h));
        asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.f32.f16 %0, lo; cvt.f32.f16 %1, hi; }"
            : "=f"(x[2 * i]), "=f"(x[2 * i + 1]) : "r"(h2));
    }
}
__device__ __forceinline__ uint32_t encode_e4m3x4(const float* x) {
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1]), "f"(x[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3]), "f"(x[2]));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
// A block's scale from the bits of its largest magnitude, and the reciprocal its elements
// are multiplied with.  Below 2^-126 the reciprocal would overflow: the block is zero.
__device__ __forceinline__ float state_scale(uint32_t amax_bits, float* inv) {
    float s = __fdiv_rn(__uint_as_float(amax_bits), 448.0f);
    if (s < 0x1p-126f) s = 0.0f;
    *inv = s == 0.0f ? 0.0f : __fdiv_rn(1.0f, s);
    return s;
}

template <int MAXT>
__device__ __forceinline__ int param_of_unit(const ParamTable<MAXT>& P, int64_t u) {
    int lo = 0, hi = P.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (P.t[mid].unit_begin <= u) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// One AdamW step.  PT/GT: float or uint16_t (BF16) parameters and gradients; S8: 8-bit
// states.  A NaN gradient scale leaves every tensor as it was (the amax is still formed).
template <typename PT, typename GT, bool S8, int MAXT>
__global__ void __launch_bounds__(kAdamThreads) k_adamw(const __grid_constant__ ParamTable<MAXT> P) {
    __shared__ float sh[2];
    const int lane = threadIdx.x & 31;
    const AdamScalars& h = P.h;
    float ss = h.ss, rs2 = h.rs2;
    double lr = h.lr;
    if (h.d_lr || h.d_step) {            // uniform: the step's scalars from device memory
        if (h.d_lr) lr = (double)*h.d_lr;
        if (threadIdx.x == 0)
            adam_step_scalars(lr, h.beta1, h.beta2, h.d_step ? *h.d_step : h.step, &sh[0], &sh[1]);
        __syncthreads();
        ss = sh[0];
        rs2 = sh[1];
    }
    const float gs = h.d_grad_scale ? *h.d_grad_scale : 1.0f;
    const bool skip = gs != gs;
    if (skip && !P.amax) return;

    const int64_t stride = (int64_t)gridDim.x * (kAdamThreads / 32);
    int64_t u = (int64_t)blockIdx.x * (kAdamThreads / 32) + (threadIdx.x >> 5);
    int ti = -1;
    int64_t end = 0;
    float keep = 1.0f;
    uint32_t amax = 0;
    int amax_group = -1;
    for (; u < P.total_units; u += stride) {
        if (u >= end) {
            ti = param_of_unit(P, u);
            end = ti + 1 < P.n ? P.t[ti + 1].unit_begin : P.total_units;
            keep = (float)(1.0 - lr * P.t[ti].wd);
            if (P.amax && P.t[ti].group != amax_group) {
                amax = __reduce_max_sync(0xFFFFFFFFu, amax);
                if (lane == 0 && amax) atomicMax(P.amax + amax_group, amax);
                amax = 0;
                amax_group = P.t[ti].group;
            }
        }
        const DevParam& T = P.t[ti];
        const int64_t blk = u - T.unit_begin;
        const int64_t e[2] = {blk * kParamBlock + lane * 4, blk * kParamBlock + 128 + lane * 4};
        PT* const p = static_cast<PT*>(T.p);
        float x[8], g[8], m[8], v[8];
        float sm = 0.0f, sv = 0.0f;
        uint32_t cm[2], cv[2];
        if (S8 && !skip) {
            sm = T.ms[blk];
            sv = T.vs[blk];
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int64_t n = T.numel - e[c];
            load4(p, e[c], n, x + 4 * c);
            if (skip) continue;
            load4(static_cast<const GT*>(T.g), e[c], n, g + 4 * c);
            if (S8) {
                cm[c] = load_codes4(static_cast<const uint8_t*>(T.m), e[c], n);
                cv[c] = load_codes4(static_cast<const uint8_t*>(T.v), e[c], n);
            } else {
                load4(static_cast<const float*>(T.m), e[c], n, m + 4 * c);
                load4(static_cast<const float*>(T.v), e[c], n, v + 4 * c);
            }
        }
        if (!skip) {
            uint32_t am = 0, av = 0;
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (S8) {
                    decode_e4m3x4(cm[c], m + 4 * c);
                    decode_e4m3x4(cv[c], v + 4 * c);
                }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (S8) {
                    m[i] = __fmul_rn(m[i], sm);
                    const float r = __fmul_rn(v[i], sv);
                    v[i] = __fmul_rn(r, r);
                }
                const float gi = __fmul_rn(g[i], gs);
                m[i] = __fadd_rn(__fmul_rn(m[i], h.b1), __fmul_rn(gi, h.omb1));
                v[i] = __fadd_rn(__fmul_rn(v[i], h.b2), __fmul_rn(__fmul_rn(gi, gi), h.omb2));
                const float root = __fsqrt_rn(v[i]);
                const float den = __fadd_rn(__fmul_rn(root, rs2), h.eps);
                x[i] = __fsub_rn(__fmul_rn(x[i], keep), __fmul_rn(__fdiv_rn(m[i], den), ss));
                if (S8) {
                    v[i] = root;
                    am = max(am, __float_as_uint(m[i]) & 0x7FFFFFFFu);
                    av = max(av, __float_as_uint(root));
                }
            }
            if (S8) {
                // elements behind the tensor's end are zero throughout: m = root = 0
                float im, iv;
                sm = state_scale(__reduce_max_sync(0xFFFFFFFFu, am), &im);
                sv = state_scale(__reduce_max_sync(0xFFFFFFFFu, av), &iv);
                if (lane == 0) {
                    T.ms[blk] = sm;
                    T.vs[blk] = sv;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float y[4], z[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[i] = __fmul_rn(m[4 * c + i], im);
                        z[i] = __fmul_rn(v[4 * c + i], iv);
                        // a positive root takes at least the smallest code, 2^-9
                        if (v[4 * c + i] > 0.0f && iv > 0.0f) z[i] = fmaxf(z[i], 0x1p-9f);
                    }
                    cm[c] = encode_e4m3x4(y);
                    cv[c] = encode_e4m3x4(z);
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int64_t n = T.numel - e[c];
                store4(p, e[c], n, x + 4 * c);
                if (S8) {
                    store_codes4(static_cast<uint8_t*>(T.m), e[c], n, cm[c]);
                    store_codes4(static_cast<uint8_t*>(T.v), e[c], n, cv[c]);
                } else {
                    store4(static_cast<float*>(T.m), e[c], n, m + 4 * c);
                    store4(static_cast<float*>(T.v), e[c], n, v + 4 * c);
                }
                if (T.w) store4(T.w, e[c], n, x + 4 * c);
            }
        }
        if (P.amax && amax_group >= 0) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float y = x[4 * c + i];
                    if (sizeof(PT) == 2)     // the amax is that of the weights as they are kept
                        y = __uint_as_float(pack_bf16(0.0f, y) << 16);
                    if (e[c] + i < T.numel) amax = max(amax, __float_as_uint(y) & 0x7FFFFFFFu);
                }
        }
    }
    if (P.amax) {
        amax = __reduce_max_sync(0xFFFFFFFFu, amax);
        if (lane == 0 && amax) atomicMax(P.amax + amax_group, amax);
    }
}

// ---------------------------------------------------------------- global gradient norm
//
// norm = sqrt(sum over every element of every tensor of g^2), the sum in binary64.  The
// binary64 pipe takes one fused multiply-add per element; the conversion to binary64
// would cost the slow conversion pipe instead, so it is done on the bits: shift the
// mantissa, rebias the exponent.  Subnormals come out as if normal, below 2^-126 (their
// squares are below 2^-252, nothing beside any FP32 norm); infinities and NaN come out at
// 2^128 or above, so a gradient that holds one gives norm >= 2^128 = +inf in FP32, which
// is the mark of a step to skip.
// Bound: HBM, one read of g.  Each warp keeps 4 vectors of 16 bytes per lane in flight.
struct NormTask {
    const void* g;
    int64_t numel;
    int64_t unit_begin;
};
struct NormState {                      // workspace: zero before its first use
    uint32_t ticket;
    uint32_t pad;
    double total;
    double partial[kNormMaxGrid];
};
template <int MAXT>
struct NormTable {
    NormTask t[MAXT];
    NormState* ws;
    float* out;
    int64_t* d_step;
    double max_norm;
    int64_t total_units;
    int n;
    int first, last;
};
constexpr int kNormVecs = 4;

__device__ __forceinline__ double widen(uint32_t bits) {       // |x|, see above
    const uint32_t a = bits & 0x7FFFFFFFu;
    return a ? __hiloint2double((int)((a >> 3) + 0x38000000u), (int)(a << 29)) : 0.0;
}

template <typename GT, int MAXT>
__global__ void __launch_bounds__(kAdamThreads) k_grad_norm(const __grid_constant__ NormTable<MAXT> P) {
    constexpr int kVec = 16 / sizeof(GT);
    constexpr int kUnit = 32 * kVec * kNormVecs;
    __shared__ double sh[kAdamThreads / 32];
    __shared__ bool is_last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t stride = (int64_t)gridDim.x * (kAdamThreads / 32);
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
    int64_t end = 0;
    int ti = 0;
    for (int64_t u = (int64_t)blockIdx.x * (kAdamThreads / 32) + warp; u < P.total_units; u += stride) {
        if (u >= end) {
            int lo = ti, hi = P.n - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (P.t[mid].unit_begin <= u) lo = mid; else hi = mid - 1;
            }
            ti = lo;
            end = ti + 1 < P.n ? P.t[ti + 1].unit_begin : P.total_units;
        }
        const NormTask& T = P.t[ti];
        const GT* const g = static_cast<const GT*>(T.g);
        const int64_t e0 = (u - T.unit_begin) * kUnit + lane * kVec;
        uint4 x[kNormVecs];
#pragma unroll
        for (int k = 0; k < kNormVecs; ++k) {
            const int64_t e = e0 + k * 32 * kVec;
            if (e + kVec <= T.numel) {
                x[k] = __ldg(reinterpret_cast<const uint4*>(g + e));
            } else {
                x[k] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    if (e + i < T.numel) {
                        if (sizeof(GT) == 2) {
                            const uint32_t b = (uint32_t)((const uint16_t*)g)[e + i] << (16 * (i & 1));
                            if (i / 2 == 0) x[k].x |= b;
                            if (i / 2 == 1) x[k].y |= b;
                            if (i / 2 == 2) x[k].z |= b;
                            if (i / 2 == 3) x[k].w |= b;
                        } else {
                            const uint32_t b = ((const uint32_t*)g)[e + i];
                            if (i == 0) x[k].x = b;
                            if (i == 1) x[k].y = b;
                            if (i == 2) x[k].z = b;
                            if (i == 3) x[k].w = b;
                        }
                    }
            }
        }
#pragma unroll
        for (int k = 0; k < kNormVecs; ++k) {
            const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (sizeof(GT) == 2) {
                    const double a = widen(w[i] << 16), b = widen(w[i] & 0xFFFF0000u);
                    acc[i] = fma(a, a, acc[i]);
                    acc[i] = fma(b, b, acc[i]);
                } else {
                    const double a = widen(w[i]);
                    acc[i] = fma(a, a, acc[i]);
                }
            }
        }
    }
    double s = (acc[0] + acc[1]) + (acc[2] + acc[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) sh[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0.0;
        for (int i = 0; i < kAdamThreads / 32; ++i) s += sh[i];
        P.ws->partial[blockIdx.x] = s;
        __threadfence();
        // wraps to 0 with the last CTA, so the workspace is ready for the next call
        is_last = atomicInc(&P.ws->ticket, gridDim.x - 1) == gridDim.x - 1;
    }
    __syncthreads();
    if (!is_last) return;
    // the last CTA adds the partial sums in a fixed order
    __threadfence();
    s = 0.0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += kAdamThreads) s += __ldcg(&P.ws->partial[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    __syncthreads();
    if (lane == 0) sh[warp] = s;
    __syncthreads();
    if (threadIdx.x != 0) return;
    s = P.first ? 0.0 : P.ws->total;
    for (int i = 0; i < kAdamThreads / 32; ++i) s += sh[i];
    P.ws->total = s;
    if (!P.last) return;
    const double norm = sqrt(s);
    const float f = (float)norm;
    const bool bad = !(f < __int_as_float(0x7F800000));
    float scale = 1.0f;
    if (P.max_norm > 0.0 && norm > 0.0) scale = (float)fmin(1.0, P.max_norm / norm);
    P.out[0] = f;
    P.out[1] = bad ? __int_as_float(0x7FC00000) : scale;
    if (P.d_step && !bad) *P.d_step += 1;
}

#endif  // __CUDACC__

}  // namespace qf
