// qf_adapters.cuh -- sm_100a kernels of the low-rank adapters of many requests beside a
// shared projection: forward (u = x A^T, y += s u B^T) and backward (v = gy B,
// gx += s v A, gA = s v^T x, gB = s gy^T u), each token with the adapter of its request.
//
// Bound: HBM.  A rank-r product does r operations per byte of x (2 r per 2-byte element),
// where the tensor cores' balance is 247: x, y, gy and gx are streamed once per kernel and
// the factors, a few hundred KB, come from L2.  So the products run on mma.sync straight
// from registers: with the reduction index permuted alike on both operands, the 16 bytes
// a lane loads ARE its fragments, and no tile is staged through shared memory.
#pragma once

#include <cstdint>

namespace qf {

constexpr int kLoraTile = 64;           // tokens of one tile (all of one adapter)
constexpr int kLoraMaxAdapters = 512;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kPlanHead = 4;            // words: tiles, tokens with an adapter, tokens, adapters

struct Adapter {
    const uint16_t* b;                  // [rows, rank]; backward: B^T [rank, rows]
    const uint16_t* a;                  // [rank, cols]; backward: A^T [cols, round16(rank)]
    int rank;
    float scale;
};
template <int MAXA>
struct AdapterTable {
    Adapter t[MAXA];
};

// Device plan, int32 words: head | start[n + 1] | order[tokens] | per tile: adapter (-1:
// empty), begin
struct PlanView {
    const int32_t* w;                   // NULL: every token has adapter 0, in order
    int tokens;
    int n;
};
__host__ __device__ inline int64_t plan_tiles(int64_t tokens, int64_t n) {
    return (tokens + kLoraTile - 1) / kLoraTile + (n < tokens ? n : tokens);
}
__host__ __device__ inline int64_t plan_words(int64_t tokens, int64_t n) {
    return kPlanHead + n + 1 + tokens + 2 * plan_tiles(tokens, n);
}

#ifdef __CUDACC__

__device__ __forceinline__ void wait_previous_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_grid_start() { asm volatile("griddepcontrol.launch_dependents;"); }

// ---------------------------------------------------------------- the plan
//
// Sorts the tokens by adapter (stable) and cuts each adapter's run into tiles.  One CTA
// per adapter: its warps count, over consecutive ranges of tokens, those of smaller
// adapters and their own, note which adapters occur, and place their own by the ballots'
// ranks.  An adapter's first tile is start / 64 + the adapters that occur before it, which
// leaves room for each run's short last tile without knowing the other runs' lengths;
// slots left over are empty tiles.  Latency-bound: every CTA reads the index from L2.
__global__ void __launch_bounds__(kPlanThreads)
k_lora_plan(const int32_t* __restrict__ index, int tokens, int n, int32_t* __restrict__ plan) {
    constexpr int kWarps = kPlanThreads / 32, kAhead = 8;
    __shared__ unsigned char occurs[kLoraMaxAdapters];
    __shared__ int warp_own[kWarps], warp_less[kWarps], warp_seen[kWarps];
    const int a = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < n; i += kPlanThreads) occurs[i] = 0;
    __syncthreads();
    const int per = (tokens + kWarps * 32 - 1) / (kWarps * 32) * 32;
    const int t0 = min(tokens, warp * per), t1 = min(tokens, t0 + per);
    int own = 0, less = 0;
    for (int t = t0; t < t1; t += 32 * kAhead) {
        int k[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) k[i] = t + 32 * i + lane < t1 ? index[t + 32 * i + lane] : -1;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (k[i] >= 0 && k[i] < n) occurs[k[i]] = 1;
            own += k[i] == a;
            less += k[i] >= 0 && k[i] < a;
        }
    }
    own = __reduce_add_sync(0xFFFFFFFFu, own);
    less = __reduce_add_sync(0xFFFFFFFFu, less);
    __syncthreads();
    int seen = 0;
    for (int i = tid; i < a; i += kPlanThreads) seen += occurs[i];
    seen = __reduce_add_sync(0xFFFFFFFFu, seen);
    if (lane == 0) {
        warp_own[warp] = own;
        warp_less[warp] = less;
        warp_seen[warp] = seen;
    }
    __syncthreads();
    int start = 0, count = 0, before = 0, first = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = count;
        count += warp_own[w];
        start += warp_less[w];
        first += warp_seen[w];
    }
    first += start / kLoraTile;
    const int behind = count > 0 ? (start + count) / kLoraTile - start / kLoraTile + 1 : 0;
    int32_t* const starts = plan + kPlanHead;
    int32_t* const order = starts + n + 1;
    int32_t* const tiles = order + tokens;
    if (tid == 0) {
        starts[a] = start;
        if (a == n - 1) {
            starts[n] = start + count;
            plan[0] = first + behind;
            plan[1] = start + count;
            plan[2] = tokens;
            plan[3] = n;
        }
    }
    for (int i = tid; i < behind; i += kPlanThreads) {
        tiles[2 * (first + i)] = i * kLoraTile < count ? a : -1;
        tiles[2 * (first + i) + 1] = start + i * kLoraTile;
    }
    if (own == 0) return;
    int32_t* out = order + start + before;
    for (int t = t0; t < t1; t += 32 * kAhead) {
        int k[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) k[i] = t + 32 * i + lane < t1 ? index[t + 32 * i + lane] : -1;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, k[i] == a);
            if (k[i] == a) out[__popc(hit & ((1u << lane) - 1))] = t + 32 * i + lane;
            out += __popc(hit);
        }
    }
}

struct Tile {
    int adapter, begin, count;          // tokens order[begin] .. order[begin + count - 1]
    const int32_t* order;               // NULL: the tokens themselves
    __device__ __forceinline__ int token(int i) const {
        return order ? order[begin + i] : begin + i;
    }
};
// Tile i of the batch; count 0: there is none.
__device__ __forceinline__ Tile tile_of(const PlanView& P, int i) {
    Tile t{0, 0, 0, nullptr};
    if (P.w == nullptr) {
        t.begin = i * kLoraTile;
        t.count = max(0, min(kLoraTile, P.tokens - t.begin));
        return t;
    }
    if (P.w[2] != P.tokens || P.w[3] != P.n || i >= P.w[0]) return t;   // not this batch's plan
    const int32_t* const start = P.w + kPlanHead;
    t.order = start + P.n + 1;
    const int a = t.order[P.tokens + 2 * i];
    if (a < 0) return t;
    t.adapter = a;
    t.begin = t.order[P.tokens + 2 * i + 1];
    t.count = min(kLoraTile, start[a + 1] - t.begin);
    return t;
}
__device__ __forceinline__ Tile run_of(const PlanView& P, int adapter) {   // an adapter's whole run
    Tile t{adapter, 0, 0, nullptr};
    if (P.w == nullptr) {
        t.count = P.tokens;
        return t;
    }
    if (P.w[2] != P.tokens || P.w[3] != P.n) {
        t.count = -1;
        return t;
    }
    const int32_t* const start = P.w + kPlanHead;
    t.order = start + P.n + 1;
    t.begin = start[adapter];
    t.count = start[adapter + 1] - t.begin;
    return t;
}

__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf16x2(float hi, float lo) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}
// The same four words of the shared memory of every CTA of a cluster, added in rank order.
__device__ __forceinline__ float4 sum_cluster(const float* p, int parts) {
    const uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
    float4 v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        v[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < parts)
            asm volatile("{ .reg .u32 a; mapa.shared::cluster.u32 a, %4, %5;\n\t"
                         "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a]; }"
                         : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                         : "r"(at), "r"(r) : "memory");
    }
#pragma unroll
    for (int r = 1; r < 8; ++r) {
        v[0].x += v[r].x;
        v[0].y += v[r].y;
        v[0].z += v[r].z;
        v[0].w += v[r].w;
    }
    return v[0];
}
// x as the sum of two BF16 values (17 significant bits): the next product's operands.
__device__ __forceinline__ void split_bf16(float4 x, uint2* hi, uint2* lo) {
    hi->x = bf16x2(x.y, x.x);
    hi->y = bf16x2(x.w, x.z);
    lo->x = bf16x2(x.y - __uint_as_float(hi->x & 0xFFFF0000u), x.x - __uint_as_float(hi->x << 16));
    lo->y = bf16x2(x.w - __uint_as_float(hi->y & 0xFFFF0000u), x.z - __uint_as_float(hi->y << 16));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16u : 0u)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

// ---------------------------------------------------------------- down: u = z F^T
//
// z [tokens, depth] (row stride ldz), F the factor with the reduction index contiguous
// ([rank, depth], row stride depth), u [tokens, 2 wide] BF16: the sums as two BF16 values,
// the high parts first, because they are the next products' operands (one BF16 value
// would cost the gradients as much again as their own rounding).
// A CTA takes one tile and a slice of depth; the CTAs of a cluster take the slices of one
// tile and add their sums through distributed shared memory in rank order, so the result
// does not depend on timing.  Within a CTA the warps are split WM over the tile's tokens
// and WK over depth.  z and F stream through a ring of shared memory that belongs to the
// lane: a lane copies (cp.async) exactly the 16 bytes it will read back as fragments, so
// the copies run STAGES - 1 steps ahead without registers and without any barrier.
// NT: 8-wide rank tiles per pass (ranks above 64 take passes of 64).
#ifndef QF_DOWN_STAGES
#define QF_DOWN_STAGES 3
#endif
template <int NT> struct DownShape {
    static constexpr int WM = NT > 4 ? 2 : 1, WK = 8 / WM, MB = 4 / WM, RW = NT * 8 + 4;
    static constexpr int kFrags = 2 * MB + NT;           // 16-byte vectors a lane holds per step
    static constexpr size_t kRing = size_t(8) * QF_DOWN_STAGES * kFrags * 512;
    static constexpr size_t kRed = size_t(WK) * kLoraTile * RW * sizeof(float);
    static constexpr size_t kSmem = kRing > kRed ? kRing : kRed;
};
template <int MAXA, int NT>
__global__ void __launch_bounds__(kLoraThreads)
k_lora_down(const __grid_constant__ AdapterTable<MAXA> A, const PlanView P, const uint16_t* __restrict__ z,
            int64_t ldz, int depth, int backward, int parts, uint16_t* __restrict__ u, int wide_max) {
    using S = DownShape<NT>;
    constexpr int WM = S::WM, WK = S::WK, MB = S::MB, RW = S::RW, ST = QF_DOWN_STAGES;
    extern __shared__ __align__(16) unsigned char smem[];
    float* const red = reinterpret_cast<float*>(smem);   // [WK][64][RW], after the ring's use
    wait_previous_grid();
    let_next_grid_start();
    const Tile tile = tile_of(P, blockIdx.x / parts);     // parts = the cluster size
    if (tile.count <= 0) return;                         // the same for the whole cluster
    const Adapter ad = A.t[tile.adapter];
    const uint16_t* const f = backward ? ad.b : ad.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int wm = warp % WM, wk = warp / WM, row0 = wm * MB * 16;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * ST * S::kFrags * 512 + lane * 16;
    const uint16_t* zr[MB][2];
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = row0 + m * 16 + h * 8 + g;     // rows behind the tile repeat its first
            zr[m][h] = z + (int64_t)tile.token(i < tile.count ? i : 0) * ldz + 8 * q;
        }
    const int steps = (depth + 31) / 32, per = (steps + parts - 1) / parts;
    const int first = (int)(blockIdx.x % parts) * per, last = min(steps, first + per);
    const int wide = (ad.rank + 15) / 16 * 16;           // columns of u this adapter owns
    for (int r0 = 0; r0 < wide; r0 += NT * 8) {
        float acc[MB][NT][4] = {};
        const uint16_t* fr[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int r = r0 + 8 * j + g;
            fr[j] = f + (int64_t)(r < ad.rank ? r : 0) * depth + 8 * q;
        }
        auto fetch = [&](int c, uint32_t at) {
            if (c < last) {
                const bool in = 32 * c + 8 * q < depth;
                const int off = in ? 32 * c : 0;         // (a zero-filled copy reads nothing)
#pragma unroll
                for (int m = 0; m < MB; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (row0 + m * 16 < tile.count) cp_async16(at + (2 * m + h) * 512, zr[m][h] + off, in);
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (r0 + 8 * j < ad.rank)
                        cp_async16(at + (2 * MB + j) * 512, fr[j] + off, in && r0 + 8 * j + g < ad.rank);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int s = 0; s < ST - 1; ++s) fetch(first + wk + s * WK, ring + s * S::kFrags * 512);
        uint32_t read = ring, write = ring + (ST - 1) * S::kFrags * 512;
        for (int c = first + wk; c < last; c += WK) {
            fetch(c + (ST - 1) * WK, write);
            cp_async_wait<ST - 1>();
            uint4 fv[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (r0 + 8 * j < ad.rank) fv[j] = lds16(read + (2 * MB + j) * 512);
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                if (row0 + m * 16 >= tile.count) continue;
                const uint4 z0 = lds16(read + 2 * m * 512), z1 = lds16(read + (2 * m + 1) * 512);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (r0 + 8 * j >= ad.rank) continue;
                    mma_bf16(acc[m][j], z0.x, z1.x, z0.y, z1.y, fv[j].x, fv[j].y);
                    mma_bf16(acc[m][j], z0.z, z1.z, z0.w, z1.w, fv[j].z, fv[j].w);
                }
            }
            write = read;
            read += S::kFrags * 512;
            if (read == ring + ST * S::kFrags * 512) read = ring;
        }
        cp_async_wait<0>();
        __syncthreads();                                 // the ring becomes the reduction's buffer
        float* const mine = red + (int64_t)(wk * kLoraTile) * RW;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if (row0 + m * 16 >= tile.count) continue;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float* const at = mine + (row0 + m * 16 + g) * RW + 8 * j + 2 * q;
                *reinterpret_cast<float2*>(at) = make_float2(acc[m][j][0], acc[m][j][1]);
                *reinterpret_cast<float2*>(at + 8 * RW) = make_float2(acc[m][j][2], acc[m][j][3]);
            }
        }
        __syncthreads();
        const int quads = min(NT * 8, wide - r0) / 4;
        for (int i = threadIdx.x; i < tile.count * quads; i += kLoraThreads) {
            float* const at = red + (i / quads) * RW + i % quads * 4;
            float4 s = *reinterpret_cast<const float4*>(at);
#pragma unroll
            for (int w = 1; w < WK; ++w) {
                const float4 t = *reinterpret_cast<const float4*>(at + w * kLoraTile * RW);
                s.x += t.x;
                s.y += t.y;
                s.z += t.z;
                s.w += t.w;
            }
            *reinterpret_cast<float4*>(at) = s;
        }
        if (parts > 1) cluster_sync(); else __syncthreads();
        const int me = parts > 1 ? (int)cluster_rank() : 0;
        for (int i = me * kLoraThreads + threadIdx.x; i < tile.count * quads; i += parts * kLoraThreads) {
            const int t = i / quads, r = i % quads * 4;
            const float* const at = red + t * RW + r;
            const float4 s = parts > 1 ? sum_cluster(at, parts) : *reinterpret_cast<const float4*>(at);
            uint2 hi, lo;
            split_bf16(s, &hi, &lo);
            uint16_t* const out = u + (int64_t)tile.token(t) * 2 * wide_max + r0 + r;
            *reinterpret_cast<uint2*>(out) = hi;
            *reinterpret_cast<uint2*>(out + wide_max) = lo;
        }
        if (parts > 1) cluster_sync(); else __syncthreads();
    }
}

// ---------------------------------------------------------------- up: y += s u F^T
//
// u [tokens, 2 wide_max] (high and low parts), F [width, ldf] with the rank contiguous
// (forward: B itself, ldf = rank; backward: A^T, padded), y [tokens, width] BF16 (row
// stride ldy), read, added to in FP32 and rounded once.  A warp owns 32 columns and keeps
// their factor rows as fragments; the columns are dealt to the four 8-wide MMA tiles so
// that a lane ends up with 8 neighbouring columns of its rows: y moves in 16-byte vectors,
// 64 bytes per row.  All of the tile's y is on its way (cp.async, each lane what it will
// read itself) before the first product; u comes once per CTA.
// KS: 16-deep rank steps.
template <int KS> struct UpShape {
    static constexpr int kRow = 2 * KS * 16 + 8;          // u's row in shared memory, padded
    static constexpr size_t kSmem = size_t(kLoraTile) * kRow * 2 + size_t(8) * 8 * 512;
};
template <int MAXA, int KS>
__global__ void __launch_bounds__(kLoraThreads)
k_lora_up(const __grid_constant__ AdapterTable<MAXA> A, const PlanView P, const uint16_t* u, int wide_max,
          int width, int backward, uint16_t* __restrict__ y, int64_t ldy) {
    constexpr int UR = UpShape<KS>::kRow;
    extern __shared__ __align__(16) unsigned char smem[];
    wait_previous_grid();
    let_next_grid_start();
    const int across = (width + 255) / 256;
    const Tile tile = tile_of(P, blockIdx.x / across);
    if (tile.count <= 0) return;
    const Adapter ad = A.t[tile.adapter];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int n0 = (int)(blockIdx.x % across) * 256 + warp * 32, col = n0 + 8 * q;
    const int ks = (ad.rank + 15) / 16;
    const uint32_t us = (uint32_t)__cvta_generic_to_shared(smem);
    const uint32_t ys = us + kLoraTile * UR * 2 + warp * 8 * 512 + lane * 16;
    for (int i = threadIdx.x; i < tile.count * ks * 4; i += kLoraThreads) {
        const int t = i / (ks * 4), c = i % (ks * 4) * 8;          // high parts, then low parts
        const int half = c >= ks * 16;
        cp_async16(us + (t * UR + (half ? KS * 16 + c - ks * 16 : c)) * 2,
                   u + (int64_t)tile.token(t) * 2 * wide_max + (half ? wide_max + c - ks * 16 : c), true);
    }
    cp_async_commit();
    uint16_t* at[4][2];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 16 * m + 8 * h + g;
            const bool in = i < tile.count && col < width;
            at[m][h] = in ? y + (int64_t)tile.token(i) * ldy + col : nullptr;
            if (in) cp_async16(ys + (2 * m + h) * 512, at[m][h], true);
        }
        cp_async_commit();
    }
    uint2 fv[KS][4];
    const uint16_t* const f = backward ? ad.a : ad.b;
    const int ldf = backward ? ks * 16 : ad.rank;
    const bool vec = (ldf & 3) == 0 && (reinterpret_cast<uintptr_t>(f) & 7) == 0;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = n0 + 8 * (g >> 1) + 2 * j + (g & 1), r = 16 * k + 4 * q;
            const uint16_t* const p = f + (int64_t)c * ldf + r;
            fv[k][j] = make_uint2(0, 0);
            if (c >= width || r >= ldf) continue;
            if (vec) {
                fv[k][j] = *reinterpret_cast<const uint2*>(p);
            } else {
                fv[k][j].x = p[0] | (r + 1 < ldf ? (uint32_t)p[1] << 16 : 0u);
                if (r + 2 < ldf) fv[k][j].y = p[2] | (r + 3 < ldf ? (uint32_t)p[3] << 16 : 0u);
            }
        }
    cp_async_wait<4>();
    __syncthreads();                                       // u is there for every warp
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        if (16 * m >= tile.count) break;
        float acc[4][4] = {};
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (k >= ks) break;
                // rows behind the tile are stale shared memory: their products are not used
                const uint32_t up = us + ((16 * m + g) * UR + p * KS * 16 + 16 * k + 4 * q) * 2;
                const uint2 u0 = lds8(up), u1 = lds8(up + 8 * UR * 2);
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_bf16(acc[j], u0.x, u1.x, u0.y, u1.y, fv[k][j].x, fv[k][j].y);
            }
        if (m == 0) cp_async_wait<3>();
        if (m == 1) cp_async_wait<2>();
        if (m == 2) cp_async_wait<1>();
        if (m == 3) cp_async_wait<0>();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!at[m][h]) continue;
            const uint4 yv = lds16(ys + (2 * m + h) * 512);
            uint32_t w[4] = {yv.x, yv.y, yv.z, yv.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = bf16x2(__uint_as_float(w[j] & 0xFFFF0000u) + ad.scale * acc[j][2 * h + 1],
                              __uint_as_float(w[j] << 16) + ad.scale * acc[j][2 * h]);
            *reinterpret_cast<uint4*>(at[m][h]) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    cp_async_wait<0>();
}

// ---------------------------------------------------------------- factors turned for the backward pass
//
// A [rank, cols] -> A^T [cols, round16(rank)] (zero-padded), B [rows, rank] -> B^T [rank, rows].
template <int MAXA>
struct TurnTable {
    Adapter t[MAXA];
    uint16_t* at[MAXA];
    uint16_t* bt[MAXA];
};
template <int MAXA>
__global__ void __launch_bounds__(256)
k_lora_turn(const __grid_constant__ TurnTable<MAXA> A, int rows, int cols) {
    let_next_grid_start();
    const Adapter ad = A.t[blockIdx.y];
    const int wide = (ad.rank + 15) / 16 * 16;
    const int na = cols * (wide / 8), nb = rows / 8 * ad.rank;
    for (int i = blockIdx.x * 256 + threadIdx.x; i < na + nb; i += gridDim.x * 256) {
        uint32_t w[4] = {0, 0, 0, 0};
        uint16_t* out;
        if (i < na) {
            const int c = i % cols, r = i / cols * 8;
            out = A.at[blockIdx.y] + (int64_t)c * wide + r;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (r + k < ad.rank) w[k / 2] |= (uint32_t)ad.a[(int64_t)(r + k) * cols + c] << (16 * (k & 1));
        } else {
            const int r = (i - na) % ad.rank, n = (i - na) / ad.rank * 8;
            out = A.bt[blockIdx.y] + (int64_t)r * rows + n;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                w[k / 2] |= (uint32_t)ad.b[(int64_t)(n + k) * ad.rank + r] << (16 * (k & 1));
        }
        *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ---------------------------------------------------------------- the factors' gradients
//
// gA = s v^T x ([rank, cols]) and gB = s gy^T u ([rows, rank]): the reduction runs over an
// adapter's tokens.  One launch for both: blockIdx.x walks 128-column tiles of x, then of
// gy.  A CTA stages 32 tokens at a time (rows gathered by the plan) through four cp.async
// buffers and multiplies with the rank as the MMA's rows, so rank 16 fills it; both operands
// have the token index outermost and come through ldmatrix.trans.  The CTAs of a cluster
// take slices of the tokens and add up through distributed shared memory in rank order.
struct GradOut {
    void* ga;
    void* gb;
};
template <int MAXA>
struct GradTable {
    GradOut t[MAXA];
    float scale[MAXA];
    int rank[MAXA];
};
constexpr int kGradCols = 128, kGradTokens = 32, kGradStages = 4, kGradThreads = 128;

__device__ __forceinline__ void ldmatrix_t(uint32_t* r, const uint16_t* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"((uint32_t)__cvta_generic_to_shared(p)) : "memory");
}
template <int MT> struct GradShape {
    static constexpr int ZS = kGradCols + 8, WS = 2 * MT * 16 + 8, RS = kGradCols + 4;
    static constexpr size_t kPipe = size_t(kGradStages) * kGradTokens * (ZS + WS) * 2;
    static constexpr size_t kRed = size_t(MT) * 16 * RS * sizeof(float);
    static constexpr size_t kSmem = kPipe > kRed ? kPipe : kRed;
};
template <int MAXA, int MT>
__global__ void __launch_bounds__(kGradThreads)
k_lora_grad(const __grid_constant__ GradTable<MAXA> A, const PlanView P, const uint16_t* __restrict__ x,
            int64_t ldx, int cols, const uint16_t* v, const uint16_t* __restrict__ gy, int64_t ldgy, int rows,
            const uint16_t* u, int wide_max) {
    using S = GradShape<MT>;
    constexpr int ZS = S::ZS, WS = S::WS, RS = S::RS;
    extern __shared__ __align__(16) unsigned char smem[];
    uint16_t* const zs = reinterpret_cast<uint16_t*>(smem);
    uint16_t* const ws = zs + kGradStages * kGradTokens * ZS;
    float* const red = reinterpret_cast<float*>(smem);
    wait_previous_grid();
    let_next_grid_start();
    const int parts = gridDim.z, part = blockIdx.z, adapter = blockIdx.y;
    const Tile run = run_of(P, adapter);
    if (run.count < 0) return;                            // not this batch's plan
    const int xt = (cols + kGradCols - 1) / kGradCols;
    const bool of_a = (int)blockIdx.x < xt;
    const uint16_t* const z = of_a ? x : gy;
    const uint16_t* const w = of_a ? v : u;
    const int64_t ldz = of_a ? ldx : ldgy;
    const int depth = of_a ? cols : rows, c0 = (of_a ? (int)blockIdx.x : (int)blockIdx.x - xt) * kGradCols;
    const int rank = A.rank[adapter], wide = (rank + 15) / 16 * 16;
    const int per = ((run.count + parts - 1) / parts + kGradTokens - 1) / kGradTokens * kGradTokens;
    const int first = min(run.count, part * per), last = min(run.count, first + per);
    const int stages = (last - first + kGradTokens - 1) / kGradTokens;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    auto fetch = [&](int s) {
        const uint32_t zd = (uint32_t)__cvta_generic_to_shared(zs + (s % kGradStages) * kGradTokens * ZS);
        const uint32_t wd = (uint32_t)__cvta_generic_to_shared(ws + (s % kGradStages) * kGradTokens * WS);
#pragma unroll
        for (int k = 0; k < kGradTokens * 16 / kGradThreads; ++k) {
            const int id = tid + k * kGradThreads, i = id >> 4, c = (id & 15) * 8;
            const int t = first + s * kGradTokens + i;
            const bool in = t < last && c0 + c < depth;
            cp_async16(zd + (i * ZS + c) * 2, in ? z + (int64_t)run.token(t) * ldz + c0 + c : z, in);
        }
#pragma unroll
        for (int k = 0; k < kGradTokens * MT * 4 / kGradThreads; ++k) {
            const int id = tid + k * kGradThreads, i = id / (MT * 4), c = id % (MT * 4) * 8;
            const int t = first + s * kGradTokens + i, half = c >= MT * 16, r = half ? c - MT * 16 : c;
            const bool in = t < last && r < wide;
            cp_async16(wd + (i * WS + c) * 2,
                       in ? w + (int64_t)run.token(t) * 2 * wide_max + (half ? wide_max + r : r) : w, in);
        }
    };
    float acc[MT][4][4] = {};
    for (int s = 0; s < kGradStages - 1; ++s) {
        if (s < stages) fetch(s);
        cp_async_commit();
    }
    for (int s = 0; s < stages; ++s) {
        cp_async_wait<kGradStages - 2>();
        __syncthreads();
        if (s + kGradStages - 1 < stages) fetch(s + kGradStages - 1);
        cp_async_commit();
        const uint16_t* const zd = zs + (s % kGradStages) * kGradTokens * ZS;
        const uint16_t* const wd = ws + (s % kGradStages) * kGradTokens * WS;
#pragma unroll
        for (int k = 0; k < kGradTokens; k += 16) {
            uint32_t b[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                ldmatrix_t(b[h], zd + (k + (lane & 15)) * ZS + warp * 32 + 16 * h + (lane >> 4) * 8);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (16 * m >= wide) break;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    uint32_t a[4];
                    ldmatrix_t(a, wd + (k + (lane & 7) + ((lane >> 4) & 1) * 8) * WS + (p * MT + m) * 16 +
                                      ((lane >> 3) & 1) * 8);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_bf16(acc[m][j], a[0], a[1], a[2], a[3], b[j / 2][2 * (j & 1)], b[j / 2][2 * (j & 1) + 1]);
                }
            }
        }
    }
    cp_async_wait<0>();
    __syncthreads();
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float* const at = red + (16 * m + g) * RS + warp * 32 + 8 * j + 2 * q;
            *reinterpret_cast<float2*>(at) = make_float2(acc[m][j][0], acc[m][j][1]);
            *reinterpret_cast<float2*>(at + 8 * RS) = make_float2(acc[m][j][2], acc[m][j][3]);
        }
    if (parts > 1) cluster_sync(); else __syncthreads();
    const int me = parts > 1 ? (int)cluster_rank() : 0;
    const int quads = kGradCols / 4 / parts;              // this CTA writes these columns
    const float scale = A.scale[adapter];
    for (int i = tid; i < rank * quads; i += kGradThreads) {
        const int r = of_a ? i / quads : i % rank, c = (me * quads + (of_a ? i % quads : i / rank)) * 4;
        if (c0 + c >= depth) continue;                    // depth is a multiple of 8
        const float* const at = red + r * RS + c;
        const float4 s = parts > 1 ? sum_cluster(at, parts) : *reinterpret_cast<const float4*>(at);
        const uint32_t lo = bf16x2(scale * s.y, scale * s.x), hi = bf16x2(scale * s.w, scale * s.z);
        if (of_a) {
            uint16_t* const out = static_cast<uint16_t*>(A.t[adapter].ga) + (int64_t)r * cols + c0 + c;
            if ((reinterpret_cast<uintptr_t>(out) & 7) == 0) {
                *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
            } else {
                out[0] = (uint16_t)lo;
                out[1] = (uint16_t)(lo >> 16);
                out[2] = (uint16_t)hi;
                out[3] = (uint16_t)(hi >> 16);
            }
        } else {
            uint16_t* const out = static_cast<uint16_t*>(A.t[adapter].gb) + (int64_t)(c0 + c) * rank + r;
            out[0] = (uint16_t)lo;
            out[rank] = (uint16_t)(lo >> 16);
            out[2 * rank] = (uint16_t)hi;
            out[3 * rank] = (uint16_t)(hi >> 16);
        }
    }
    if (parts > 1) cluster_sync();
}

#endif  // __CUDACC__

}  // namespace qf
