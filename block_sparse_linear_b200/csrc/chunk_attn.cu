// Exact causal attention of a chunk of new tokens over the paged cache. With L_b tokens
// held by sequence b, the chunk's n_b among them, query t of the chunk stands at
// position L_b - n_b + t and sees the tokens up to its own:
//   o_t = sum_{s <= pos_t} p_ts v_s / sum p_ts,   p_ts = exp(scale q_t . k_s),
//   lse_t = log sum_{s <= pos_t} p_ts
// in one pass over the tokens with a running maximum (softmax attention as in the Baidu
// article's section 1; the paged pools are the decode path's own).
#include "common.cuh"

namespace spla {

// The chunk of sequence b: false (and a status bit) where its count or length is out of range.
__device__ __forceinline__ bool chunk_of(const CacheView& c, const ChunkArgs& a, int b,
                                         int32_t* L, int32_t* n, bool flag) {
    *L = c.lens[b];
    *n = a.n_new[b];
    int32_t bad = 0;
    if (*n < 0 || *n > a.max_new) bad = SPLA_DEV_BAD_COUNT;
    else if (*L < 0 || *L > (int64_t)c.mbp * c.bs) bad = SPLA_DEV_CAPACITY;
    else if (*n > *L) bad = SPLA_DEV_BAD_COUNT;
    if (bad && flag) set_status(a.status, bad);
    return bad == 0;
}

constexpr int kSimtWarps = 4;

// One warp per (sequence, new token, query head): lanes over 32 tokens for the logits,
// over dimensions for the values.
template <int D, typename T>
__global__ void __launch_bounds__(kSimtWarps * 32)
chunk_simt_kernel(CacheView c, ChunkArgs a) {
    __shared__ float qs[kSimtWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    const int64_t row = (int64_t)blockIdx.x * kSimtWarps + warp;
    if (row >= (int64_t)c.batch * a.max_new * c.hq) return;
    const int hq = (int)(row % c.hq);
    const int64_t bt = row / c.hq;
    const int b = (int)(bt / a.max_new), t = (int)(bt - (int64_t)b * a.max_new);
    int32_t L, n;
    if (!chunk_of(c, a, b, &L, &n, t == 0 && hq == 0 && lane == 0) || t >= n) return;
    const int h = hq / c.group;
    const T* q = (const T*)a.q + row * D;
    for (int i = lane; i < D; i += 32) qs[warp][i] = to_f<T>(q[i]) * a.sl2;
    __syncwarp();
    const int pos = L - n + t;
    float m = -SPLA_INF, l = 0.f;
    constexpr int CPL = D / 32;
    float acc[CPL] = {};
    for (int s0 = 0; s0 <= pos; s0 += 32) {
        const int s = s0 + lane;
        const int lb = s0 / c.bs;                 // 32 divides the block size
        const int32_t phys = c.table[(int64_t)b * c.mbp + lb];
        const bool good = phys >= 0 && phys < c.num_phys;
        if (!good && lane == 0) set_status(a.status, SPLA_DEV_BAD_BLOCK_TABLE);
        const int64_t base = (((int64_t)(good ? phys : 0) * c.hkv + h) * c.bs + (s0 - lb * c.bs)) * D;
        float x = -SPLA_INF;
        if (s <= pos) {
            x = 0.f;
            const T* k = (const T*)c.k_pool + base + (int64_t)lane * D;
            if (good)
                for (int i = 0; i < D; ++i) x = fmaf(qs[warp][i], to_f<T>(k[i]), x);
        }
        const float mn = fmaxf(m, warp_max(x));
        const float mu = mn == -SPLA_INF ? 0.f : mn;
        const float f = exp2f(m - mu);
        const float p = exp2f(x - mu);
        l = l * f + warp_sum(p);
        m = mn;
#pragma unroll
        for (int i = 0; i < CPL; ++i) acc[i] *= f;
        const int cnt = min(32, pos - s0 + 1);
        const T* v = (const T*)c.v_pool + base + lane * CPL;
        for (int j = 0; j < cnt; ++j) {
            const float pj = __shfl_sync(0xffffffffu, p, j);
            if (good)
#pragma unroll
                for (int i = 0; i < CPL; ++i)
                    acc[i] = fmaf(pj, to_f<T>(v[(int64_t)j * D + i]), acc[i]);
        }
    }
    T* o = (T*)a.out + row * D + lane * CPL;
#pragma unroll
    for (int i = 0; i < CPL; ++i) o[i] = from_f<T>(acc[i] / l);
    if (a.lse && lane == 0) a.lse[row] = (m + log2f(l)) * 0.69314718055994531f;
}

size_t chunk_tc_workspace_bytes(int d);

size_t chunk_workspace_bytes(int d, int dtype) {
    return dtype == SPLA_BF16 ? chunk_tc_workspace_bytes(d) : 256;
}

cudaError_t launch_chunk_simt(const CacheView& c, int dtype, const ChunkArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)c.batch * a.max_new * c.hq;
    const dim3 grid((unsigned)((rows + kSimtWarps - 1) / kSimtWarps)), block(kSimtWarps * 32);
    using B16 = __nv_bfloat16;
    if (c.d == 128)
        return dtype == SPLA_BF16 ? launch_pdl(chunk_simt_kernel<128, B16>, grid, block, 0, s, c, a)
                                  : launch_pdl(chunk_simt_kernel<128, float>, grid, block, 0, s, c, a);
    return dtype == SPLA_BF16 ? launch_pdl(chunk_simt_kernel<64, B16>, grid, block, 0, s, c, a)
                              : launch_pdl(chunk_simt_kernel<64, float>, grid, block, 0, s, c, a);
}

}  // namespace spla
