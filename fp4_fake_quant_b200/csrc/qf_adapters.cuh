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
constexpr int kPlanThreads = 512;
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

// Device plan, int32 words: head | start[n + 1] | order[tokens] | tile adapter, tile begin
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
// per adapter: each counts all adapters' tokens (for where its own run and tiles begin)
// and places its own.  Latency-bound: every CTA reads the index once from L2.
__global__ void __launch_bounds__(kPlanThreads)
k_lora_plan(const int32_t* __restrict__ index, int tokens, int n, int32_t* __restrict__ plan) {
    __shared__ int count[kLoraMaxAdapters];
    __shared__ int warp_sum[2][kPlanThreads / 32];
    const int a = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < n; i += kPlanThreads) count[i] = 0;
    __syncthreads();
    const int per = (tokens + kPlanThreads - 1) / kPlanThreads;
    const int t0 = min(tokens, tid * per), t1 = min(tokens, t0 + per);
    int mine = 0;
    for (int t = t0; t < t1;) {          // runs of one adapter are counted with one addition
        const int k = index[t];
        int e = t + 1;
        while (e < t1 && index[e] == k) ++e;
        if (k >= 0 && k < n) atomicAdd(&count[k], e - t);
        if (k == a) mine += e - t;
        t = e;
    }
    int scan = mine;                     // inclusive over the threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sum[0][warp] = scan;
    __syncthreads();
    int before = scan - mine;
    for (int w = 0; w < warp; ++w) before += warp_sum[0][w];
    // tokens and tiles of the adapters before this one
    int s = 0, q = 0;
    for (int i = tid; i < a; i += kPlanThreads) {
        s += count[i];
        q += (count[i] + kLoraTile - 1) / kLoraTile;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
    }
    __syncthreads();
    if (lane == 0) {
        warp_sum[0][warp] = s;
        warp_sum[1][warp] = q;
    }
    __syncthreads();
    s = q = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        s += warp_sum[0][w];
        q += warp_sum[1][w];
    }
    int32_t* const start = plan + kPlanHead;
    int32_t* const order = start + n + 1;
    int32_t* const tiles = order + tokens;
    const int own = count[a], own_tiles = (own + kLoraTile - 1) / kLoraTile;
    if (tid == 0) {
        start[a] = s;
        if (a == n - 1) {
            start[n] = s + own;
            plan[0] = q + own_tiles;
            plan[1] = s + own;
            plan[2] = tokens;
            plan[3] = n;
        }
    }
    for (int i = tid; i < own_tiles; i += kPlanThreads) {
        tiles[2 * (q + i)] = a;
        tiles[2 * (q + i) + 1] = s + i * kLoraTile;
    }
    int32_t* const out = order + s + before;
    int k = 0;
    for (int t = t0; t < t1; ++t)
        if (index[t] == a) out[k++] = t;
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
    t.adapter = t.order[P.tokens + 2 * i];
    t.begin = t.order[P.tokens + 2 * i + 1];
    t.count = min(kLoraTile, start[t.adapter + 1] - t.begin);
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
__device__ __forceinline__ float load_cluster(const float* p, uint32_t rank) {   // another CTA's shared word
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint4 load16(const uint16_t* p) {
    return *reinterpret_cast<const uint4*>(p);
}

// ---------------------------------------------------------------- down: u = z F^T
//
// z [tokens, depth] (row stride ldz), F the factor with the reduction index contiguous
// ([rank, depth], row stride depth), u [tokens, ldu] BF16: BF16 because it is the next
// product's operand; the sum itself is FP32.  A CTA takes one tile and a slice of depth;
// the CTAs of a cluster take the slices of one tile and add their sums through
// distributed shared memory, in rank order, so the result does not depend on timing.
// Within a CTA the warps are split WM over the tile's tokens and WK over depth.
// NT: 8-wide rank tiles per pass (ranks above 64 take passes of 64).
template <int MAXA, int NT>
__global__ void __launch_bounds__(kLoraThreads)
k_lora_down(const __grid_constant__ AdapterTable<MAXA> A, const PlanView P, const uint16_t* __restrict__ z,
            int64_t ldz, int depth, int backward, int parts, uint16_t* __restrict__ u, int ldu) {
    constexpr int WM = NT > 4 ? 2 : 1, WK = 8 / WM, MB = 4 / WM, RW = NT * 8 + 4;
    extern __shared__ float red[];                       // [WK][64][RW]
    wait_previous_grid();
    let_next_grid_start();
    const Tile tile = tile_of(P, blockIdx.x / parts);     // parts = the cluster size
    if (tile.count <= 0) return;                         // the same for the whole cluster
    const Adapter ad = A.t[tile.adapter];
    const uint16_t* const f = backward ? ad.b : ad.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int wm = warp % WM, wk = warp / WM, row0 = wm * MB * 16;
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
        for (int c = first + wk; c < last; c += WK) {
            const bool in = 32 * c + 8 * q < depth;
            uint4 zv[MB][2], fv[NT];
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    zv[m][h] = in && row0 + m * 16 < tile.count ? load16(zr[m][h] + 32 * c)
                                                                : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NT; ++j)
                fv[j] = in && r0 + 8 * j + g < ad.rank ? load16(fr[j] + 32 * c) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                if (row0 + m * 16 >= tile.count) continue;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    if (r0 + 8 * j >= ad.rank) continue;
                    mma_bf16(acc[m][j], zv[m][0].x, zv[m][1].x, zv[m][0].y, zv[m][1].y, fv[j].x, fv[j].y);
                    mma_bf16(acc[m][j], zv[m][0].z, zv[m][1].z, zv[m][0].w, zv[m][1].w, fv[j].z, fv[j].w);
                }
            }
        }
        float* const mine = red + (int64_t)(wk * kLoraTile) * RW;
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float* const at = mine + (row0 + m * 16 + g) * RW + 8 * j + 2 * q;
                at[0] = acc[m][j][0];
                at[1] = acc[m][j][1];
                at[8 * RW] = acc[m][j][2];
                at[8 * RW + 1] = acc[m][j][3];
            }
        __syncthreads();
        const int cols = min(NT * 8, wide - r0);
        for (int i = threadIdx.x; i < tile.count * cols; i += kLoraThreads) {
            const int at = (i / cols) * RW + i % cols;
            float s = red[at];
#pragma unroll
            for (int w = 1; w < WK; ++w) s += red[w * kLoraTile * RW + at];
            red[at] = s;
        }
        if (parts > 1) cluster_sync(); else __syncthreads();
        const int me = parts > 1 ? (int)cluster_rank() : 0;
        for (int i = me * kLoraThreads + threadIdx.x; i < tile.count * cols / 2; i += parts * kLoraThreads) {
            const int t = 2 * i / cols, r = 2 * i % cols, at = t * RW + r;
            float s0 = 0.0f, s1 = 0.0f;
            if (parts > 1)
                for (int p = 0; p < parts; ++p) {
                    s0 += load_cluster(red + at, p);
                    s1 += load_cluster(red + at + 1, p);
                }
            else {
                s0 = red[at];
                s1 = red[at + 1];
            }
            *reinterpret_cast<uint32_t*>(u + (int64_t)tile.token(t) * ldu + r0 + r) = bf16x2(s1, s0);
        }
        if (parts > 1) cluster_sync(); else __syncthreads();
    }
}

// ---------------------------------------------------------------- up: y += s u F^T
//
// u [tokens, ldu], F [width, ldf] with the rank contiguous (forward: B itself, ldf = rank;
// backward: A^T, padded), y [tokens, width] BF16 (row stride ldy), read, added to in FP32
// and rounded once.  A warp owns 32 columns and keeps their factor rows as fragments; the
// columns are dealt to the four 8-wide MMA tiles so that a lane ends up with 8
// neighbouring columns of its rows: y moves in 16-byte vectors, 64 bytes per row.
// KS: 16-deep rank steps.
template <int MAXA, int KS>
__global__ void __launch_bounds__(kLoraThreads)
k_lora_up(const __grid_constant__ AdapterTable<MAXA> A, const PlanView P, const uint16_t* u,
          int ldu, int width, int backward, uint16_t* __restrict__ y, int64_t ldy) {
    wait_previous_grid();
    let_next_grid_start();
    const int across = (width + 255) / 256;
    const Tile tile = tile_of(P, blockIdx.x / across);
    if (tile.count <= 0) return;
    const Adapter ad = A.t[tile.adapter];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int n0 = (int)(blockIdx.x % across) * 256 + warp * 32;
    if (n0 >= width) return;
    const int ks = (ad.rank + 15) / 16;
    uint2 fv[KS][4];
    const uint16_t* const f = backward ? ad.a : ad.b;
    const int ldf = backward ? ks * 16 : ad.rank;
    const bool vec = (ldf & 3) == 0 && (reinterpret_cast<uintptr_t>(f) & 7) == 0;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int col = n0 + 8 * (g >> 1) + 2 * j + (g & 1), r = 16 * k + 4 * q;
            const uint16_t* const p = f + (int64_t)col * ldf + r;
            fv[k][j] = make_uint2(0, 0);
            if (col >= width || r >= ldf) continue;
            if (vec) {
                fv[k][j] = *reinterpret_cast<const uint2*>(p);
            } else {
                fv[k][j].x = p[0] | (r + 1 < ldf ? (uint32_t)p[1] << 16 : 0u);
                if (r + 2 < ldf) fv[k][j].y = p[2] | (r + 3 < ldf ? (uint32_t)p[3] << 16 : 0u);
            }
        }
    const int col = n0 + 8 * q;
    for (int m = 0; m < tile.count; m += 16) {
        uint16_t* at[2];
        uint4 yv[2];
        uint2 uv[KS][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = m + 8 * h + g, t = tile.token(i < tile.count ? i : 0);
            at[h] = y + (int64_t)t * ldy + col;
            yv[h] = make_uint4(0, 0, 0, 0);
            if (i < tile.count && col < width) yv[h] = load16(at[h]);
#pragma unroll
            for (int k = 0; k < KS; ++k)
                uv[k][h] = k < ks ? *reinterpret_cast<const uint2*>(u + (int64_t)t * ldu + 16 * k + 4 * q)
                                  : make_uint2(0, 0);
        }
        float acc[4][4] = {};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            if (k >= ks) break;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                mma_bf16(acc[j], uv[k][0].x, uv[k][1].x, uv[k][0].y, uv[k][1].y, fv[k][j].x, fv[k][j].y);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (m + 8 * h + g >= tile.count || col >= width) continue;
            uint32_t w[4] = {yv[h].x, yv[h].y, yv[h].z, yv[h].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = bf16x2(__uint_as_float(w[j] & 0xFFFF0000u) + ad.scale * acc[j][2 * h + 1],
                              __uint_as_float(w[j] << 16) + ad.scale * acc[j][2 * h]);
            *reinterpret_cast<uint4*>(at[h]) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
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

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(in ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void ldmatrix_t(uint32_t* r, const uint16_t* p) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"((uint32_t)__cvta_generic_to_shared(p)) : "memory");
}
template <int MT>
constexpr size_t grad_smem() {
    const size_t pipe = size_t(kGradStages) * kGradTokens * ((kGradCols + 8) + (MT * 16 + 8)) * 2;
    const size_t red = size_t(MT) * 16 * (kGradCols + 4) * 4;
    return pipe > red ? pipe : red;
}

template <int MAXA, int MT>
__global__ void __launch_bounds__(kGradThreads)
k_lora_grad(const __grid_constant__ GradTable<MAXA> A, const PlanView P, const uint16_t* __restrict__ x,
            int64_t ldx, int cols, const uint16_t* v, const uint16_t* __restrict__ gy, int64_t ldgy, int rows,
            const uint16_t* u, int ldu) {
    constexpr int ZS = kGradCols + 8, WS = MT * 16 + 8, RS = kGradCols + 4;
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
        uint16_t* const zd = zs + (s % kGradStages) * kGradTokens * ZS;
        uint16_t* const wd = ws + (s % kGradStages) * kGradTokens * WS;
#pragma unroll
        for (int k = 0; k < kGradTokens * 16 / kGradThreads; ++k) {
            const int id = tid + k * kGradThreads, i = id >> 4, c = (id & 15) * 8;
            const int t = first + s * kGradTokens + i;
            const bool in = t < last && c0 + c < depth;
            cp_async16(zd + i * ZS + c, in ? z + (int64_t)run.token(t) * ldz + c0 + c : z, in);
        }
        for (int id = tid; id < kGradTokens * MT * 2; id += kGradThreads) {
            const int i = id / (MT * 2), c = id % (MT * 2) * 8;
            const int t = first + s * kGradTokens + i;
            const bool in = t < last && c < wide;
            cp_async16(wd + i * WS + c, in ? w + (int64_t)run.token(t) * ldu + c : w, in);
        }
    };
    float acc[MT][4][4] = {};
    for (int s = 0; s < kGradStages - 1; ++s) {
        if (s < stages) fetch(s);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    for (int s = 0; s < stages; ++s) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kGradStages - 2) : "memory");
        __syncthreads();
        if (s + kGradStages - 1 < stages) fetch(s + kGradStages - 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
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
                uint32_t a[4];
                ldmatrix_t(a, wd + (k + (lane & 7) + ((lane >> 4) & 1) * 8) * WS + 16 * m + ((lane >> 3) & 1) * 8);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    mma_bf16(acc[m][j], a[0], a[1], a[2], a[3], b[j / 2][2 * (j & 1)], b[j / 2][2 * (j & 1) + 1]);
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float* const at = red + (16 * m + g) * RS + warp * 32 + 8 * j + 2 * q;
            at[0] = acc[m][j][0];
            at[1] = acc[m][j][1];
            at[8 * RS] = acc[m][j][2];
            at[8 * RS + 1] = acc[m][j][3];
        }
    if (parts > 1) cluster_sync(); else __syncthreads();
    const int me = parts > 1 ? (int)cluster_rank() : 0;
    const int span = kGradCols / parts;                  // this CTA writes these columns
    const float scale = A.scale[adapter];
    for (int i = tid; i < rank * span; i += kGradThreads) {
        const int r = of_a ? i / span : i % rank, c = me * span + (of_a ? i % span : i / rank);
        if (c0 + c >= depth) continue;
        float s = 0.0f;
        if (parts > 1)
            for (int p = 0; p < parts; ++p) s += load_cluster(red + r * RS + c, p);
        else
            s = red[r * RS + c];
        const uint16_t h = (uint16_t)(bf16x2(0.0f, scale * s) & 0xFFFFu);
        if (of_a) static_cast<uint16_t*>(A.t[adapter].ga)[(int64_t)r * cols + c0 + c] = h;
        else static_cast<uint16_t*>(A.t[adapter].gb)[(int64_t)(c0 + c) * rank + r] = h;
    }
    if (parts > 1) cluster_sync();
}

#endif  // __CUDACC__

}  // namespace qf
