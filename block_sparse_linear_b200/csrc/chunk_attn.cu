// Chunk attention, fp32, and the join of both types' partials. chunk_attn.cuh states the
// mathematics and the split over the GPU.
//
// The products run on the tensor cores in three parts: x = hi + lo with hi the tf32 part
// of x (its upper 11 significant bits) and lo the exact rest, rounded to tf32, and
// a b = hi hi + hi lo + lo hi. What is dropped, lo lo, and the rounding of lo are 2^-22 of
// a product, as fp32's own rounding is 2^-24 of a sum: the results are fp32 attention's
// (tensor cores take tf32 at most, and fp32 FMAs have a quarter of this rate). mma.sync
// m16n8k8 with the operands split in registers: the split parts of a tile would take twice
// the shared memory. What that costs: every warp splits the whole K and V tile again, between
// MMAs that wait for the parts. 512 tokens over 3584 (4/1 heads of 64) take 57 us with the tensor
// pipe busy 47 % of the time and issue slots 37 %, warps waiting for one another's MMAs and for
// the split; one token over each of 4 x 32768 (32/8 heads of 128) reads K and V at 2.9 TB/s, with
// a two-stage ring and barriers of the whole CTA around each step.
//
// A CTA of 8 warps: WM of them side by side over rows (16 each), the others over the
// tokens of a 64-token step, chosen so that few rows (decode) still use every warp; their
// sums meet in shared memory at the end of a segment. K and V tiles come through cp.async into a
// two-stage ring, rows padded by 16 bytes (every fragment load is free of bank conflicts).
// The probabilities' accumulator layout is the next product's A layout once the tokens of
// a group of 8 are taken in the order 0 2 4 6 1 3 5 7, which the V loads follow.
//
// Infinities and NaN in V: a probability of zero does not cancel them and the split turns
// an infinity into NaN, so they are taken out of each tile and noted (first token per
// dimension and kind), and the epilogue adds them to the rows that see that token.
#include <algorithm>

#include "chunk_attn.cuh"

namespace spla {

template <int WM> using FWalk = Walk<kFKT, FCost, (WM < 8)>;   // (WM < 8: one unit holds the chunk)

template <int D, int WM>
struct FShape {
    // 8 warps of 255 registers: 16 of 128 spill the fragments, 83 us against 61 for 512
    // tokens over 3584 (4/1 heads of 64).
    static constexpr int kWarps = 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kWN = kWarps / WM;         // warps over the tokens
    static constexpr int kNT = kFKT / 8 / kWN;      // token groups of 8 per warp and step
    static constexpr int kLd = D + 4;               // floats between tile rows
    static constexpr int kTile = kFKT * kLd;
    static constexpr int kSums = 16 * kWarps * (kLd + 2);   // the warps' sums, where the tiles were
    static constexpr size_t kSmem = sizeof(float) * (kSums > 4 * kTile ? kSums : 4 * kTile);
};

__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) + 0x1000u;    // rounded where the MMA cuts it
}
// D += A (16x8, row) * B (8x8, col), tf32.
__device__ __forceinline__ void mma_tf32(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// N products with one A. The small parts have an accumulator of their own: the tensor core
// cuts an accumulator's low bits at every addition, always towards zero, and so loses the
// fewer the fewer large parts are added (the sums over many groups are fp32 additions).
template <int N>
__device__ __forceinline__ void mma_3tf32(float (*hi)[4], float (*lo)[4], const float* a,
                                          const float* b0, const float* b1) {
    uint32_t ah[4], al[4], h0[N], l0[N], h1[N], l1[N];
#pragma unroll
    for (int e = 0; e < 4; ++e) split_tf32(a[e], ah[e], al[e]);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        split_tf32(b0[n], h0[n], l0[n]);
        split_tf32(b1[n], h1[n], l1[n]);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) mma_tf32(lo[n], al, h0[n], h1[n]);
#pragma unroll
    for (int n = 0; n < N; ++n) mma_tf32(hi[n], ah, h0[n], h1[n]);
#pragma unroll
    for (int n = 0; n < N; ++n) mma_tf32(lo[n], ah, l0[n], l1[n]);
}
constexpr int kFChain = 4;                          // products of 8 in one accumulator

template <int D, int WM>
__global__ void __launch_bounds__(FShape<D, WM>::kThreads, 1)
chunk_f32_kernel(const CacheView c, const ChunkArgs a) {
    using S = FShape<D, WM>;
    constexpr int WN = S::kWN, NT = S::kNT, kFThreads = S::kThreads;
    constexpr int kRows = 16 * WM, kGrp = NT < 4 ? NT : 4;
    extern __shared__ __align__(16) float f_smem[];
    __shared__ int64_t scan[kFThreads / 32], run;
    __shared__ FWalk<WM> start;
    __shared__ int32_t first[3][D], noted;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wm = warp % WM, wn = warp / WM, g = lane >> 2, t = lane & 3;
    const int G = c.group, lgG = G >> 1, U = kRows >> lgG;
    if (tid == 0) {
        start.j = 0;
        start.F = start.end = 0;
    }
    pdl_trigger();
    pdl_wait();
    find_run<kFThreads>(c, a, U, U, scan, first[0], &start, &run);
    FWalk<WM> wk = start;
    ChunkCut cut = {};
    auto ktile = [&](int s) { return f_smem + s * 2 * S::kTile; };
    auto vtile = [&](int s) { return f_smem + s * 2 * S::kTile + S::kTile; };

    while (wk.next(c, a, U, U)) {
        const int tok0 = wk.qb * U;
        const int base_pos = wk.L - wk.n;
        // this lane's two rows
        const int row_a = wm * 16 + g, row_b = row_a + 8;
        const int tok_a = tok0 + (row_a >> lgG), tok_b = tok0 + (row_b >> lgG);
        const int pos_a = base_pos + tok_a, pos_b = base_pos + tok_b;
        const bool warp_live = tok0 + (wm * 16 >> lgG) < wk.n;
        float o[D / 8][4] = {};
        float m_a = -SPLA_INF, m_b = -SPLA_INF, l_a = 0.f, l_b = 0.f;
        __syncthreads();                            // the last segment's sums have been read
#pragma unroll 1
        for (int i = tid; i < 3 * D; i += kFThreads) first[i / D][i % D] = 0x7fffffff;
        if (tid == 0) noted = 0;

        const int32_t* table = c.table + (int64_t)wk.b * c.mbp;
        const int lg_steps = c.bs >> 7;             // steps of a page: 1 or 2
        auto page_of = [&](int j) { return table[j >> lg_steps]; };
        auto load = [&](int j, int s, int32_t phys) {   // a step's tiles; slots past the end are zeros
            const bool good = phys >= 0 && phys < c.num_phys;
            if (!good && tid == 0) set_status(a.status, SPLA_DEV_BAD_BLOCK_TABLE);
            const int64_t at = (((int64_t)(good ? phys : 0) * c.hkv + wk.h) * c.bs +
                                ((j * kFKT) & (c.bs - 1))) * D;
            const int held = good ? min(kFKT, wk.L - j * kFKT) : 0;
#pragma unroll 4
            for (int i = tid; i < kFKT * (D / 4); i += kFThreads) {
                const int r = i / (D / 4), x = (i - r * (D / 4)) * 4;
                const int64_t src = at + (r < held ? (int64_t)r * D + x : 0);
                cp_async16(ktile(s) + r * S::kLd + x, (const float*)c.k_pool + src, r < held);
                cp_async16(vtile(s) + r * S::kLd + x, (const float*)c.v_pool + src, r < held);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int32_t page = page_of(wk.j0);
        __syncthreads();
        load(wk.j0, 0, page);
        if (wk.j0 + 1 < wk.j1) page = page_of(wk.j0 + 1);
        float q[D / 8][4];
        {
            const float* qp = (const float*)a.q + ((int64_t)wk.b * a.max_new * c.hq + wk.h * G) * D;
            const float* qa = qp + ((int64_t)tok_a * c.hq + (row_a & (G - 1))) * D + t;
            const float* qb = qp + ((int64_t)tok_b * c.hq + (row_b & (G - 1))) * D + t;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
                q[k][0] = tok_a < wk.n ? qa[8 * k] : 0.f;
                q[k][1] = tok_b < wk.n ? qb[8 * k] : 0.f;
                q[k][2] = tok_a < wk.n ? qa[8 * k + 4] : 0.f;
                q[k][3] = tok_b < wk.n ? qb[8 * k + 4] : 0.f;
            }
        }
#pragma unroll 1
        for (int j = wk.j0; j < wk.j1; ++j) {
            const int s = (j - wk.j0) & 1;
            if (j + 1 < wk.j1) {
                load(j + 1, s ^ 1, page);
                if (j + 2 < wk.j1) page = page_of(j + 2);   // a step ahead of its use
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            // the chunks of V this thread fetched
#pragma unroll 4
            for (int i = tid; i < kFKT * (D / 4); i += kFThreads) {
                const int r = i / (D / 4), x = (i - r * (D / 4)) * 4;
                float* p = vtile(s) + r * S::kLd + x;
                const float4 v = *reinterpret_cast<const float4*>(p);
                const float big = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
                // (a maximum passes over NaN: the sum of zero products does not)
                if (!(big < SPLA_INF) || !((v.x * 0.f + v.y * 0.f) + (v.z * 0.f + v.w * 0.f) == 0.f)) {
#pragma unroll 1
                    for (int e = 0; e < 4; ++e)
                        if (!(fabsf(p[e]) < SPLA_INF)) {
                            const int kind = p[e] != p[e] ? 2 : p[e] < 0.f;
                            atomicMin(&first[kind][x + e], j * kFKT + r);
                            p[e] = 0.f;
                            noted = 1;
                        }
                }
            }
            __syncthreads();
            if (warp_live) {
                const float* kt = ktile(s) + (wn * NT * 8) * S::kLd;
                const float* vt = vtile(s) + (wn * NT * 8) * S::kLd;
                float x[NT][4] = {};
#pragma unroll
                for (int n = 0; n < NT; n += kGrp) {
#pragma unroll
                    for (int k0 = 0; k0 < D / 8; k0 += kFChain) {
                        float hi[kGrp][4] = {}, lo[kGrp][4] = {};
#pragma unroll
                        for (int k = k0; k < k0 + kFChain; ++k) {
                            float b0[kGrp], b1[kGrp];
#pragma unroll
                            for (int e = 0; e < kGrp; ++e) {
                                const float* kp = kt + ((n + e) * 8 + g) * S::kLd + 8 * k + t;
                                b0[e] = kp[0];
                                b1[e] = kp[4];
                            }
                            mma_3tf32<kGrp>(hi, lo, q[k], b0, b1);
                        }
#pragma unroll
                        for (int e = 0; e < kGrp; ++e)
#pragma unroll
                            for (int z = 0; z < 4; ++z) x[n + e][z] += hi[e][z] + lo[e][z];
                    }
                }
                const int s0 = j * kFKT + wn * NT * 8 + 2 * t;      // token of x[0][0]
                if ((j + 1) * kFKT > base_pos + tok0 + 1) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (s0 + 8 * n + (e & 1) > (e < 2 ? pos_a : pos_b)) x[n][e] = -SPLA_INF;
                }
                float ta = -SPLA_INF, tb = -SPLA_INF;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    ta = fmaxf(ta, fmaxf(x[n][0], x[n][1]));
                    tb = fmaxf(tb, fmaxf(x[n][2], x[n][3]));
                }
                for (int d = 1; d < 4; d <<= 1) {
                    ta = fmaxf(ta, __shfl_xor_sync(0xffffffffu, ta, d));
                    tb = fmaxf(tb, __shfl_xor_sync(0xffffffffu, tb, d));
                }
                // log2 units from here on; sums are scaled by the running maximum
                ta = fmaxf(m_a, ta * a.sl2);
                tb = fmaxf(m_b, tb * a.sl2);
                if (__any_sync(0xffffffffu, ta > m_a || tb > m_b)) {
                    const float fa = m_a == -SPLA_INF ? 0.f : ex2(m_a - ta);
                    const float fb = m_b == -SPLA_INF ? 0.f : ex2(m_b - tb);
                    l_a *= fa;
                    l_b *= fb;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][0] *= fa;
                        o[n][1] *= fa;
                        o[n][2] *= fb;
                        o[n][3] *= fb;
                    }
                    m_a = ta;
                    m_b = tb;
                }
                const float za = m_a == -SPLA_INF ? 0.f : m_a, zb = m_b == -SPLA_INF ? 0.f : m_b;
                float sa = 0.f, sb = 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    x[n][0] = ex2(fmaf(x[n][0], a.sl2, -za));
                    x[n][1] = ex2(fmaf(x[n][1], a.sl2, -za));
                    x[n][2] = ex2(fmaf(x[n][2], a.sl2, -zb));
                    x[n][3] = ex2(fmaf(x[n][3], a.sl2, -zb));
                    sa += x[n][0] + x[n][1];
                    sb += x[n][2] + x[n][3];
                }
                l_a += sa;
                l_b += sb;
#pragma unroll
                for (int n = 0; n < D / 8; n += 4) {
#pragma unroll
                    for (int k0 = 0; k0 < NT; k0 += kGrp) {
                        float hi[4][4] = {}, lo[4][4] = {};
#pragma unroll
                        for (int k = k0; k < k0 + kGrp; ++k) {
                            // A's columns t and t + 4 are tokens 2t and 2t + 1
                            const float p[4] = {x[k][0], x[k][2], x[k][1], x[k][3]};
                            const float* vp = vt + (k * 8 + 2 * t) * S::kLd + g + 8 * n;
                            float b0[4], b1[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                b0[e] = vp[8 * e];
                                b1[e] = vp[8 * e + S::kLd];
                            }
                            mma_3tf32<4>(hi, lo, p, b0, b1);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int z = 0; z < 4; ++z) o[n + e][z] += hi[e][z] + lo[e][z];
                    }
                }
            }
            __syncthreads();
        }

        // ---- the warps' sums meet where the tiles were
        for (int d = 1; d < 4; d <<= 1) {
            l_a += __shfl_xor_sync(0xffffffffu, l_a, d);
            l_b += __shfl_xor_sync(0xffffffffu, l_b, d);
        }
        float* sum = f_smem;                        // [16 kWarps][kLd]: row wn * kRows + row
        float* sm = f_smem + 16 * S::kWarps * S::kLd;
        float* sl = sm + 16 * S::kWarps;
        const int ra = wn * kRows + row_a, rb = wn * kRows + row_b;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            *reinterpret_cast<float2*>(sum + ra * S::kLd + 8 * n + 2 * t) = make_float2(o[n][0], o[n][1]);
            *reinterpret_cast<float2*>(sum + rb * S::kLd + 8 * n + 2 * t) = make_float2(o[n][2], o[n][3]);
        }
        if (t == 0) {
            sm[ra] = m_a;
            sm[rb] = m_b;
            sl[ra] = l_a;
            sl[rb] = l_b;
        }
        __syncthreads();
        const bool whole = wk.j0 == 0 && wk.j1 == wk.T;
        float* part = reinterpret_cast<float*>(a.ws + kCutBytes) +
                      ((int64_t)blockIdx.x * 2 + (wk.j0 == 0 ? 1 : 0)) * part_floats(D);
#pragma unroll 1
        for (int i = tid; i < kRows * (D / 4); i += kFThreads) {
            const int row = i / (D / 4), x = (i - row * (D / 4)) * 4;
            const int tok = tok0 + (row >> lgG);
            if (tok >= wk.n) break;                 // rows ascend with i
            float M = -SPLA_INF, l = 0.f;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < WN; ++w) M = fmaxf(M, sm[w * kRows + row]);
#pragma unroll
            for (int w = 0; w < WN; ++w) {
                const float mw = sm[w * kRows + row], lw = sl[w * kRows + row];
                // no tokens: no part; nothing but NaN logits: NaN
                if (!has_part(mw, lw)) continue;
                const float f = mw == -SPLA_INF ? lw : ex2(mw - M);
                const float4 v = *reinterpret_cast<const float4*>(sum + (w * kRows + row) * S::kLd + x);
                l = fmaf(lw, f, l);
                y.x = fmaf(v.x, f, y.x);
                y.y = fmaf(v.y, f, y.y);
                y.z = fmaf(v.z, f, y.z);
                y.w = fmaf(v.w, f, y.w);
            }
            if (noted) {
                const int pos = base_pos + tok;
                y.x += note_term(first[0][x], first[1][x], first[2][x], pos);
                y.y += note_term(first[0][x + 1], first[1][x + 1], first[2][x + 1], pos);
                y.z += note_term(first[0][x + 2], first[1][x + 2], first[2][x + 2], pos);
                y.w += note_term(first[0][x + 3], first[1][x + 3], first[2][x + 3], pos);
            }
            if (whole) {
                const float inv = 1.f / l;
                const int64_t orow = ((int64_t)wk.b * a.max_new + tok) * c.hq + wk.h * G + (row & (G - 1));
                *reinterpret_cast<float4*>((float*)a.out + orow * D + x) =
                    make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
                if (x == 0 && a.lse) a.lse[orow] = (M + log2f(l)) * 0.69314718055994531f;
            } else {
                *reinterpret_cast<float4*>(part + (int64_t)row * D + x) = y;
                if (x == 0) {
                    part[256 * D + row] = M;
                    part[256 * D + 256 + row] = l;
                }
            }
        }
        wk.note_cut(cut, blockIdx.x, U, G, run);
    }
    if (tid == 0) reinterpret_cast<ChunkCut*>(a.ws)[blockIdx.x] = cut;
}

// ------------------------------------------------------------------ the join
// One warp per row of a unit that was cut: log-sum-exp merge of its partials in run
// order (the result does not depend on timing), lanes over the dimensions.
constexpr int kJoinWarps = 8;

template <int D, typename T>
__global__ void __launch_bounds__(kJoinWarps * 32)
chunk_combine_kernel(const CacheView c, const ChunkArgs a) {
    constexpr int CPL = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int run = blockIdx.y, row = blockIdx.x * kJoinWarps + warp;
    pdl_trigger();
    pdl_wait();
    const ChunkCut cut = reinterpret_cast<const ChunkCut*>(a.ws)[run];
    if (row >= cut.rows || cut.parts == 0) return;
    const float* base = reinterpret_cast<const float*>(a.ws + kCutBytes) +
                        (int64_t)run * 2 * part_floats(D);
    // partial p is run + p's, slot 1 for the first of them and slot 0 after it
    auto part = [&](int p) { return base + ((int64_t)p * 2 + (p == 0 ? 1 : 0)) * part_floats(D); };
    // the first partials' sums are on their way with the maxima that weigh them
    constexpr int kBatch = 8;                       // partial rows in flight
    float x[kBatch][CPL];
    auto fetch = [&](int p) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (p + u >= cut.parts) break;
            const float* q = part(p + u) + (int64_t)row * D + lane * CPL;
            if constexpr (CPL == 4) *reinterpret_cast<float4*>(x[u]) = *reinterpret_cast<const float4*>(q);
            else *reinterpret_cast<float2*>(x[u]) = *reinterpret_cast<const float2*>(q);
        }
    };
    float m = -SPLA_INF, lp = 0.f;
    auto weigh = [&](int p) {
        m = p < cut.parts ? part(p)[256 * D + row] : -SPLA_INF;
        lp = p < cut.parts ? part(p)[256 * D + 256 + row] : 0.f;
    };
    weigh(lane);
    fetch(0);
    float M = m;
#pragma unroll 1
    for (int p = lane + 32; p < cut.parts; p += 32) M = fmaxf(M, part(p)[256 * D + row]);
    M = warp_max(M);
    float l = 0.f, acc[CPL] = {};
#pragma unroll 1
    for (int p0 = 0; p0 < cut.parts; p0 += 32) {
        if (p0 > 0) weigh(p0 + lane);
        // no tokens: no part (-1); nothing but NaN logits: NaN; else a part whatever the
        // weight: zero times an infinity or NaN among the sums is NaN
        const float w = !has_part(m, lp) ? -1.f : m == -SPLA_INF ? lp : ex2(m - M);
        if (!(w < 0.f)) l += w * lp;
        const int cnt = min(32, cut.parts - p0);
#pragma unroll 1
        for (int i = 0; i < cnt; i += kBatch) {
            if (p0 + i > 0) fetch(p0 + i);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const float f = __shfl_sync(0xffffffffu, w, (i + u) & 31);
                if (i + u < cnt && !(f < 0.f))
#pragma unroll
                    for (int e = 0; e < CPL; ++e) acc[e] = fmaf(x[u][e], f, acc[e]);
            }
        }
    }
    l = warp_sum(l);
    const int lgG = c.group >> 1;
    const int64_t orow = ((int64_t)cut.b * a.max_new + cut.t0 + (row >> lgG)) * c.hq +
                         cut.h * c.group + (row & (c.group - 1));
    const float inv = 1.f / l;
    T* o = (T*)a.out + orow * D + lane * CPL;
    if constexpr (sizeof(T) == 4) {
        if constexpr (CPL == 4)
            *reinterpret_cast<float4*>(o) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv,
                                                        acc[3] * inv);
        else
            *reinterpret_cast<float2*>(o) = make_float2(acc[0] * inv, acc[1] * inv);
    } else if constexpr (CPL == 4) {
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv),
                                                  pack_bf16(acc[2] * inv, acc[3] * inv));
    } else {
        *reinterpret_cast<uint32_t*>(o) = pack_bf16(acc[0] * inv, acc[1] * inv);
    }
    if (a.lse && lane == 0) a.lse[orow] = (M + log2f(l)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ host launchers
cudaError_t launch_chunk_combine(const CacheView& c, int dtype, const ChunkArgs& a, int rows,
                                 cudaStream_t s) {
    const dim3 grid((rows + kJoinWarps - 1) / kJoinWarps, kMaxRuns), block(kJoinWarps * 32);
    using B16 = __nv_bfloat16;
    if (c.d == 128)
        return dtype == SPLA_BF16 ? launch_pdl(chunk_combine_kernel<128, B16>, grid, block, 0, s, c, a)
                                  : launch_pdl(chunk_combine_kernel<128, float>, grid, block, 0, s, c, a);
    return dtype == SPLA_BF16 ? launch_pdl(chunk_combine_kernel<64, B16>, grid, block, 0, s, c, a)
                              : launch_pdl(chunk_combine_kernel<64, float>, grid, block, 0, s, c, a);
}

size_t chunk_workspace_bytes(int d) {
    return kCutBytes + (size_t)kMaxRuns * 2 * part_floats(d) * sizeof(float);
}

template <int D, int WM>
static cudaError_t launch_f32(const CacheView& c, const ChunkArgs& a, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(chunk_f32_kernel<D, WM>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)FShape<D, WM>::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(chunk_f32_kernel<D, WM>, dim3(kMaxRuns), dim3(FShape<D, WM>::kThreads),
                   FShape<D, WM>::kSmem, s, c, a);
    if (e != cudaSuccess) return e;
    const int rows = (int)std::min<int64_t>(16 * WM, (int64_t)a.max_new * c.group);
    return launch_chunk_combine(c, SPLA_F32, a, rows, s);
}

// As few warps over the rows as hold the chunk, the others over the tokens.
template <int D>
static cudaError_t launch_f32_rows(const CacheView& c, const ChunkArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)a.max_new * c.group;
    if (rows <= 16) return launch_f32<D, 1>(c, a, s);
    if (rows <= 32) return launch_f32<D, 2>(c, a, s);
    if (rows <= 64) return launch_f32<D, 4>(c, a, s);
    return launch_f32<D, 8>(c, a, s);
}

cudaError_t launch_chunk_f32(const CacheView& c, const ChunkArgs& a, cudaStream_t s) {
    return c.d == 128 ? launch_f32_rows<128>(c, a, s) : launch_f32_rows<64>(c, a, s);
}

}  // namespace spla
