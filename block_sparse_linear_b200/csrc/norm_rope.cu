// RMSNorm of every query and key head and the rotary position in one pass, between a
// fused QKV projection and the cache. For a head x of a token at position p:
//   y_i = x_i * gamma_i / sqrt(mean(x^2) + eps)
//   (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = p * inv_freq_i,
// over the pairs (i, i + rot/2) or (2i, 2i+1) of the first rot dimensions; the rest of
// the head and the values pass through. Queries go out as rows; keys and values either
// as rows (the append call's input) or straight into their pages by slot.
//
// Each element is read once and written once, so HBM bounds it: a group of d/16 lanes
// holds one head, 16 elements a lane, as two 16-byte (bf16) loads whose positions are
// chosen so that every rotated pair lies within one lane: no shared memory and no second
// read for the partner, and the group's lanes still cover whole 128-byte lines.
// The angle is taken in 64 bits (a position near a million times a frequency near one
// has lost five digits in 32) and reduced in turns, where the reduction is exact; its
// sine and cosine, shared by the token's q and k heads, are made once per CTA and row
// while the first heads' loads are in flight. Norms and rotations are fp32; the one
// rounding is the store to the tensors' type.
#include "common.cuh"

namespace spla {

constexpr int kRopeThreads = 256;

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

// Grid: ceil(rows / rows_per_cta). Dynamic shared memory: rows_per_cta * rot/2 float2.
template <int D, typename T>
__global__ void __launch_bounds__(kRopeThreads)
norm_rope_kernel(const RopeArgs a, int rows_per_cta) {
    extern __shared__ float2 cs[];               // [row][rot/2] (cos, sin)
    constexpr int LPH = D / 16;                  // lanes of one head
    const int64_t row0 = (int64_t)blockIdx.x * rows_per_cta;
    const int nrow = (int)min((int64_t)rows_per_cta, a.rows - row0);
    const int heads = a.hq + a.hkv + (a.v ? a.hkv : 0);
    const int items = nrow * heads * LPH;
    const int half = a.rot / 2;
    const int lane_h = threadIdx.x % LPH;
    // element offsets of this lane's two chunks of 8 within a head
    int c0, c1;
    const bool turn = 16 * lane_h < a.rot;
    if (a.interleaved || !turn) {
        c0 = 16 * lane_h;
        c1 = c0 + 8;
    } else {
        c0 = 8 * lane_h;
        c1 = c0 + half;
    }
    pdl_trigger();
    pdl_wait();

    auto src_of = [&](int item, int* hd, int* r) {
        const int hi = item / LPH;
        *r = hi / heads;
        *hd = hi - *r * heads;
        const int64_t row = row0 + *r;
        const T* p;
        if (*hd < a.hq) p = (const T*)a.q + row * a.q_stride + (int64_t)*hd * D;
        else if (*hd < a.hq + a.hkv)
            p = (const T*)a.k + row * a.k_stride + (int64_t)(*hd - a.hq) * D;
        else p = (const T*)a.v + row * a.v_stride + (int64_t)(*hd - a.hq - a.hkv) * D;
        return p;
    };

    Vec8<T> x0, x1;
    int hd = 0, r = 0;
    int item = threadIdx.x;
    if (item < items) {
        const T* p = src_of(item, &hd, &r);
        x0.load(p + c0);
        x1.load(p + c1);
    }
    for (int i = threadIdx.x; i < nrow * half; i += kRopeThreads) {
        const int ri = i / half;
        const double turns = (double)a.positions[row0 + ri] * a.inv_freq[i - ri * half] *
                             0.15915494309189535;           // 1 / 2 pi
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[i] = make_float2(c, s);
    }
    __syncthreads();

    // every lane of a head's group runs the same trips (items is a multiple of LPH)
    const unsigned group = (LPH == 8 ? 0xffu : 0xfu) << ((threadIdx.x & 31) / LPH * LPH);
    while (item < items) {
        const int64_t row = row0 + r;
        const int32_t pos = a.positions[row];
        T* dst = nullptr;
        if (pos >= 0) {
            if (hd < a.hq) {
                dst = (T*)a.q_out + (row * a.hq + hd) * D;
            } else {
                const bool is_v = hd >= a.hq + a.hkv;
                const int h = hd - a.hq - (is_v ? a.hkv : 0);
                T* base = (T*)(is_v ? a.v_out : a.k_out);
                if (a.slots) {
                    const int64_t slot = a.slots[row];
                    if (slot >= a.num_slots) {
                        if (lane_h == 0) set_status(a.status, SPLA_DEV_BAD_BLOCK_TABLE);
                    } else if (slot >= 0) {
                        const int64_t page = slot / a.bs;
                        dst = base + ((page * a.hkv + h) * a.bs + (slot - page * a.bs)) * D;
                    }
                } else {
                    dst = base + (row * a.hkv + h) * D;
                }
            }
        }
        if (hd < a.hq + a.hkv) {
            float f[16];
            x0.get(f);
            x1.get(f + 8);
            const float* gamma = hd < a.hq ? a.q_gamma : a.k_gamma;
            if (gamma) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
                for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
                const float rstd = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    f[e] *= rstd * gamma[c0 + e];
                    f[8 + e] *= rstd * gamma[c1 + e];
                }
            }
            if (turn) {
                const float2* t = cs + r * half;
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 w = t[c0 / 2 + e / 2];
                        const float u = f[e], z = f[e + 1];
                        f[e] = u * w.x - z * w.y;
                        f[e + 1] = z * w.x + u * w.y;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 w = t[c0 + e];
                        const float u = f[e], z = f[8 + e];
                        f[e] = u * w.x - z * w.y;
                        f[8 + e] = z * w.x + u * w.y;
                    }
                }
            }
            x0.set(f);
            x1.set(f + 8);
        }
        if (dst) {
            x0.store(dst + c0);
            x1.store(dst + c1);
        }
        item += kRopeThreads;
        if (item < items) {
            const T* p = src_of(item, &hd, &r);
            x0.load(p + c0);
            x1.load(p + c1);
        }
    }
}

// ------------------------------------------------------------------ host launcher
cudaError_t launch_norm_rope(const RopeArgs& a, int d, int dtype, cudaStream_t s) {
    if (a.rows == 0) return cudaSuccess;
    // rows per CTA: the sines of a row serve all of its heads whatever this is; a few
    // rows keep every thread busy where a row has few heads
    const int heads = a.hq + a.hkv + (a.v ? a.hkv : 0);
    const int lanes = heads * (d / 16);
    int per = (4 * kRopeThreads + lanes - 1) / lanes;
    const int64_t fill = a.rows / (4 * kNumSms);      // small calls: spread over the SMs first
    if (per > fill) per = (int)(fill < 1 ? 1 : fill);
    if (per > 16) per = 16;
    const int64_t ctas = (a.rows + per - 1) / per;
    const size_t smem = (size_t)per * (a.rot / 2) * sizeof(float2);
    const dim3 grid((unsigned)ctas), block(kRopeThreads);
    using B16 = __nv_bfloat16;
    if (d == 128)
        return dtype == SPLA_BF16 ? launch_pdl(norm_rope_kernel<128, B16>, grid, block, smem, s, a, per)
                                  : launch_pdl(norm_rope_kernel<128, float>, grid, block, smem, s, a, per);
    return dtype == SPLA_BF16 ? launch_pdl(norm_rope_kernel<64, B16>, grid, block, smem, s, a, per)
                              : launch_pdl(norm_rope_kernel<64, float>, grid, block, smem, s, a, per);
}

}  // namespace spla
