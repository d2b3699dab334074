// RMSNorm of every query and key head and the rotary position in one pass, between a
// fused QKV projection and the cache. For a head x of a token at position p:
//   y_i = x_i * gamma_i / sqrt(mean(x^2) + eps)
//   (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = p * inv_freq_i,
// over the pairs (i, i + rot/2) or (2i, 2i+1) of the first rot dimensions; the rest of
// the head and the values pass through. Queries go out as rows; keys and values either
// as rows (the append call's input) or straight into their pages by slot.
//
// Each element is read once and written once, so HBM bounds it, with the latency of a row's
// loads behind it (16 warps of 128 registers an SM; their issue slots are busy 37 % of the
// time, and warps mostly wait for loads): a group of d/16 lanes holds one head, 16 elements
// a lane, as two 16-byte (bf16) loads whose positions are chosen so that every rotated pair
// lies within one lane, and the group's lanes still cover whole 128-byte lines. A warp takes rows one
// after another with two heads a lane in flight and no barrier wider than itself; scales,
// cosines and sines are folded into four factors per pair once a row, and the arithmetic is
// on pairs of fp32 (two to an instruction). 65536 bf16 rows of 32 + 8 + 8 heads of 128, keys
// and values into pages: 307 us (5.25 TB/s); with the arithmetic left out the same accesses
// take 277 us. One head in flight 379 us, four 362 us (spills); 12 warps an SM 342 us, 20
// 356 us (spills).
// The angle is taken in 64 bits (a position near a million times a frequency near one
// has lost five digits in 32) and reduced in turns, where the reduction is exact; a row's
// sines and cosines are made once, by all lanes of its warp. Norms and rotations are fp32;
// the one rounding is the store to the tensors' type.
#include "common.cuh"

namespace spla {

constexpr int kRopeThreads = 128;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeCtas = 4;                     // per SM

// Two fp32 values in one 64-bit register.
typedef unsigned long long f2;
__device__ __forceinline__ f2 f2_of(float x, float y) {
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 f2_to(f2 a) {
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(a));
    return d;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// 8 consecutive elements, as fp32 or back.
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
    uint4 u;
    __device__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    __device__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
    __device__ void get(float* f) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(w[i]);
            f[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    __device__ void set(const float* f) {
        u = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                       pack_bf16(f[6], f[7]));
    }
};
template <> struct Vec8<float> {
    float4 a, b;
    __device__ void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    __device__ void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
    __device__ void get(float* f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ void set(const float* f) {
        a = make_float4(f[0], f[1], f[2], f[3]);
        b = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// A lane's 16 elements as the 8 pairs they rotate in, two pairs to a register.
template <bool kInter>
__device__ __forceinline__ void to_pairs(const float* f, f2* a, f2* b) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        a[e] = kInter ? f2_of(f[4 * e], f[4 * e + 2]) : f2_of(f[2 * e], f[2 * e + 1]);
        b[e] = kInter ? f2_of(f[4 * e + 1], f[4 * e + 3]) : f2_of(f[8 + 2 * e], f[8 + 2 * e + 1]);
    }
}
template <bool kInter>
__device__ __forceinline__ void from_pairs(const f2* a, const f2* b, float* f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 x = f2_to(a[e]), y = f2_to(b[e]);
        f[kInter ? 4 * e : 2 * e] = x.x;
        f[kInter ? 4 * e + 2 : 2 * e + 1] = x.y;
        f[kInter ? 4 * e + 1 : 8 + 2 * e] = y.x;
        f[kInter ? 4 * e + 3 : 8 + 2 * e + 1] = y.y;
    }
}

// What turns a lane's pairs (p, q) into the result, rstd apart: (p A - q B, q C + p E) with
// the scales within: A = ga cos, -B = -gb sin, C = gb cos, E = ga sin.
struct Turn {
    f2 A[4], nB[4], C[4], E[4];
};

// One warp, heads h0, h0 + step, ... (HPT at a time) of one row: nothing, norm, rotation
// or both. src, dst: head h at + h * the stride; dst null: a skipped row.
template <int D, typename T, bool kInter>
__device__ __forceinline__ void rope_heads(const T* src, T* dst, int heads, int64_t dst_head,
                                           int h0, int step, const Turn* w, bool norm, bool turn,
                                           bool scale, float eps, int c0, int c1, unsigned group) {
    constexpr int LPH = D / 16;
    constexpr int kAhead = sizeof(T) == 2 ? 2 : 1;      // heads a lane has in flight
    for (int h = h0; __any_sync(0xffffffffu, h < heads); h += kAhead * step) {
        Vec8<T> x[kAhead][2];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (h + u * step < heads) {
                const T* p = src + (int64_t)(h + u * step) * D;
                x[u][0].load(p + c0);
                x[u][1].load(p + c1);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (h + u * step >= heads) break;
            if (w && (norm || turn || scale)) {
                float f[16];
                f2 p[4], q[4];
                x[u][0].get(f);
                x[u][1].get(f + 8);
                to_pairs<kInter>(f, p, q);
                if (norm) {
                    f2 ss = f2_mul(p[0], p[0]);
                    ss = f2_fma(q[0], q[0], ss);
#pragma unroll
                    for (int e = 1; e < 4; ++e) ss = f2_fma(q[e], q[e], f2_fma(p[e], p[e], ss));
                    const float2 s2 = f2_to(ss);
                    float sum = s2.x + s2.y;
#pragma unroll
                    for (int o = LPH / 2; o; o >>= 1) sum += __shfl_xor_sync(group, sum, o);
                    const float rs = rsqrtf(sum * (1.f / D) + eps);
                    const f2 r2 = f2_of(rs, rs);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = f2_mul(p[e], r2);
                        q[e] = f2_mul(q[e], r2);
                    }
                }
                if (turn) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const f2 y = f2_mul(q[e], w->nB[e]), z = f2_mul(p[e], w->E[e]);
                        p[e] = f2_fma(p[e], w->A[e], y);
                        q[e] = f2_fma(q[e], w->C[e], z);
                    }
                } else if (scale) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        p[e] = f2_mul(p[e], w->A[e]);
                        q[e] = f2_mul(q[e], w->C[e]);
                    }
                }
                from_pairs<kInter>(p, q, f);
                x[u][0].set(f);
                x[u][1].set(f + 8);
            }
            if (dst) {
                T* o = dst + (int64_t)(h + u * step) * dst_head;
                x[u][0].store(o + c0);
                x[u][1].store(o + c1);
            }
        }
    }
}

// Warp v of the grid takes rows v / split, + warps / split, ...; within a row, every
// split-th group of 32 / LPH heads from v % split, queries, then keys, then values.
template <int D, typename T, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
norm_rope_kernel(const RopeArgs a, int split) {
    constexpr int LPH = D / 16;                  // lanes of one head
    constexpr int HPT = 32 / LPH;                // heads side by side
    constexpr int kAng = D / 64;                 // angles per lane
    __shared__ __align__(16) float2 cs_all[kRopeWarps][D / 2];
    __shared__ __align__(16) float gam[2][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float2* cs = cs_all[warp];
    const int half = a.rot / 2;
    const int lane_h = lane % LPH;
    // element offsets of this lane's two chunks of 8 within a head
    const bool turn = 16 * lane_h < a.rot;
    const int c0 = kInter || !turn ? 16 * lane_h : 8 * lane_h;
    const int c1 = kInter || !turn ? c0 + 8 : c0 + half;
    const unsigned group = (LPH == 8 ? 0xffu : 0xfu) << (lane / LPH * LPH);
    pdl_trigger();
    pdl_wait();
    for (int i = threadIdx.x; i < D; i += kRopeThreads) {
        gam[0][i] = a.q_gamma ? a.q_gamma[i] : 1.f;
        gam[1][i] = a.k_gamma ? a.k_gamma[i] : 1.f;
    }
    double freq[kAng];                           // turns per position
#pragma unroll
    for (int u = 0; u < kAng; ++u)
        freq[u] = lane + 32 * u < half ? a.inv_freq[lane + 32 * u] * 0.15915494309189535 : 0.0;
    __syncthreads();

    const int64_t vw = (int64_t)blockIdx.x * kRopeWarps + warp;
    const int64_t rows_step = (int64_t)gridDim.x * kRopeWarps / split;
    if (vw / split >= rows_step) return;         // (warps left over by the split)
    const int h0 = (int)(vw % split) * HPT + lane / LPH, step = split * HPT;
    for (int64_t row = vw / split; row < a.rows; row += rows_step) {
        const int32_t pos = a.positions[row];
        if (pos < 0) continue;
        int64_t kv_at = row * a.hkv * D, kv_head = D;
        if (a.slots) {
            const int64_t slot = a.slots[row];
            kv_at = -1;
            kv_head = (int64_t)D << a.lg_bs;
            if (slot >= a.num_slots) {
                if (lane == 0) set_status(a.status, SPLA_DEV_BAD_BLOCK_TABLE);
            } else if (slot >= 0) {
                kv_at = (((slot >> a.lg_bs) * a.hkv << a.lg_bs) + (slot & ((1 << a.lg_bs) - 1))) * D;
            }
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < kAng; ++e)
            if (lane + 32 * e < half) {
                const double turns = (double)pos * freq[e];
                float sn, cn;
                sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cn);
                cs[lane + 32 * e] = make_float2(cn, sn);
            }
        __syncwarp();
        Turn w;
        auto tables = [&](const float* g) {
            float t[16];
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                *reinterpret_cast<float4*>(t + e) = *reinterpret_cast<const float4*>(g + c0 + e);
                *reinterpret_cast<float4*>(t + 8 + e) = *reinterpret_cast<const float4*>(g + c1 + e);
            }
            to_pairs<kInter>(t, w.A, w.C);
            if (!turn) return;
            const float4* c4 = reinterpret_cast<const float4*>(cs + (kInter ? c0 / 2 : c0));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 v = c4[e];
                const f2 co = f2_of(v.x, v.z), si = f2_of(v.y, v.w), ns = f2_of(-v.y, -v.w);
                w.nB[e] = f2_mul(w.C[e], ns);
                w.E[e] = f2_mul(w.A[e], si);
                w.A[e] = f2_mul(w.A[e], co);
                w.C[e] = f2_mul(w.C[e], co);
            }
        };
        tables(gam[0]);
        rope_heads<D, T, kInter>((const T*)a.q + row * a.q_stride, (T*)a.q_out + row * a.hq * D, a.hq,
                                 D, h0, step, &w, a.q_gamma != nullptr, turn,
                                 a.q_gamma != nullptr, a.eps, c0, c1, group);
        tables(gam[1]);
        rope_heads<D, T, kInter>((const T*)a.k + row * a.k_stride,
                                 kv_at >= 0 ? (T*)a.k_out + kv_at : nullptr, a.hkv, kv_head, h0,
                                 step, &w, a.k_gamma != nullptr, turn, a.k_gamma != nullptr, a.eps,
                                 c0, c1, group);
        if (a.v && kv_at >= 0)
            rope_heads<D, T, kInter>((const T*)a.v + row * a.v_stride, (T*)a.v_out + kv_at, a.hkv,
                                     kv_head, h0, step, nullptr, false, false, false, a.eps, c0, c1,
                                     group);
    }
}

// ------------------------------------------------------------------ host launcher
template <int D, typename T>
static cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
    const int hpt = 32 / (D / 16), trips = (a.hq + hpt - 1) / hpt;
    // a row to a warp; with fewer rows than resident warps, several warps to a row
    const int64_t warps = (int64_t)kNumSms * kRopeCtas * kRopeWarps;
    int split = (int)(warps / (a.rows < warps ? a.rows : warps));
    if (split > trips) split = trips;
    int64_t ctas = (a.rows * split + kRopeWarps - 1) / kRopeWarps;
    if (ctas > kNumSms * kRopeCtas) ctas = kNumSms * kRopeCtas;
    const dim3 grid((unsigned)ctas), block(kRopeThreads);
    return a.interleaved ? launch_pdl(norm_rope_kernel<D, T, true>, grid, block, 0, s, a, split)
                         : launch_pdl(norm_rope_kernel<D, T, false>, grid, block, 0, s, a, split);
}

cudaError_t launch_norm_rope(const RopeArgs& a, int d, int dtype, cudaStream_t s) {
    if (d == 128)
        return dtype == SPLA_BF16 ? launch_rope<128, __nv_bfloat16>(a, s) : launch_rope<128, float>(a, s);
    return dtype == SPLA_BF16 ? launch_rope<64, __nv_bfloat16>(a, s) : launch_rope<64, float>(a, s);
}

}  // namespace spla
