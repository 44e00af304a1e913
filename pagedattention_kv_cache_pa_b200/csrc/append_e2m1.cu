// Append into a 4-bit (E2M1) paged cache, with the position rotation on the way, and the rows
// read back.
//
// The format and the group quantization are in pa_e2m1.cuh.  A new token's K row may first be
// turned by RoPE (rotate-half pairing, as in rope.cu) at its position; the turned row is rounded
// to bf16 and that row is quantized.  Everything is one pass: q, k and v are read once, the turned
// q and 9 D / 16 bytes a K or V row are written.  It is bound by those bytes.
//
// Work: a thread takes one group of 16 values (32 bytes) of a V row, or of a K row without
// rotation; with rotation a thread takes the two groups of a K row that turn into one another
// (dims 16 g .. and D/2 + 16 g ..), or 8 pairs of a q row.  A CTA runs over a few tokens at a
// time, whose D/2 cosines and sines it first forms in double (once for all heads).
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"
#include "pa_e2m1.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kThreads = 256;

struct E2m1Args {
    const uint16_t* q;
    uint16_t* q_out;
    const uint16_t* k;
    const uint16_t* v;
    const int32_t* positions;
    const int64_t* slots;
    int32_t T, Hq, Hkv, Bs;
    int64_t num_slots;
    float theta, k_inv, v_inv;
    uint8_t* k_cache;
    uint8_t* v_cache;
};

template <int D>
__device__ __forceinline__ uint8_t* page_of(uint8_t* cache, int64_t slot, int h, int Hkv, int Bs, int& off) {
    const int32_t blk = (int32_t)slot / Bs;          // slots fit in 32 bits (checked on the host)
    off = (int32_t)slot - blk * Bs;
    return cache + ((size_t)blk * Hkv + h) * e2m1_page_bytes(Bs, D);
}

// One group of a bf16 row into its page.
template <int D>
__device__ __forceinline__ void store_group(uint8_t* page, int Bs, int off, int g, const float (&x)[16], float inv) {
    uint32_t s;
    const uint2 c = e2m1_quantize16(x, inv, s);
    *e2m1_codes<D>(page, off, g) = c;
    *e2m1_scale<D>(page, Bs, off, g) = (uint8_t)s;
}

// K and V as they come: item i = (token, kv head, group), one group of K and one of V.
template <int D>
__global__ void __launch_bounds__(kThreads) append_e2m1_kernel(const E2m1Args a, int tokens_per_cta) {
    allow_dependents();
    constexpr int kGroups = D / 16;
    const int per_token = a.Hkv * kGroups;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens_per_cta; t0 < a.T; t0 += (int64_t)gridDim.x * tokens_per_cta) {
        const int n = (int)min((int64_t)tokens_per_cta, a.T - t0) * per_token;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int tl = i / per_token, w = i - tl * per_token, h = w / kGroups, g = w % kGroups;
            const int64_t t = t0 + tl, slot = a.slots[t];
            if (slot < 0 || slot >= a.num_slots) continue;
            const size_t src = ((size_t)t * a.Hkv + h) * D + g * 16;
            const uint4* ks = reinterpret_cast<const uint4*>(a.k + src);
            const uint4* vs = reinterpret_cast<const uint4*>(a.v + src);
            const uint4 k0 = __ldg(ks), k1 = __ldg(ks + 1), v0 = __ldg(vs), v1 = __ldg(vs + 1);
            int off;
            uint8_t* kp = page_of<D>(a.k_cache, slot, h, a.Hkv, a.Bs, off);
            uint8_t* vp = a.v_cache + (kp - a.k_cache);
            float x[16];
            bf16x16_to_f32(k0, k1, x);
            store_group<D>(kp, a.Bs, off, g, x, a.k_inv);
            bf16x16_to_f32(v0, v1, x);
            store_group<D>(vp, a.Bs, off, g, x, a.v_inv);
        }
    }
}

// q, K and V of a few tokens, q and K turned by RoPE.  kAtEnd: the newest token of each sequence
// (position context_lens[b] - 1, through its table row); else positions and slots.
constexpr int kMaxTokens = 8;

template <int D, bool kAtEnd>
__global__ void __launch_bounds__(kThreads) rope_append_e2m1_kernel(const E2m1Args a, const DecodeParams p,
                                                                    int tokens_per_cta) {
    allow_dependents();
    constexpr int kHalf = D / 2, kQItems = D / 16, kKItems = D / 32, kVItems = D / 16;
    __shared__ double s_inv[kHalf];
    __shared__ double s_c[kMaxTokens][kHalf], s_s[kMaxTokens][kHalf];
    __shared__ float s_cf[kMaxTokens][kHalf], s_sf[kMaxTokens][kHalf];
    __shared__ int64_t s_slot[kMaxTokens];
    if (a.theta > 0.f)
        for (int i = threadIdx.x; i < kHalf; i += kThreads) s_inv[i] = rope_inv_freq64(i, D, a.theta);
    const int qn = a.q_out ? a.Hq * kQItems : 0, kn = a.Hkv * kKItems, per_token = qn + kn + a.Hkv * kVItems;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens_per_cta; t0 < a.T; t0 += (int64_t)gridDim.x * tokens_per_cta) {
        const int nt = (int)min((int64_t)tokens_per_cta, a.T - t0);
        __syncthreads();   // s_inv is written; the previous tokens' cosines are no longer read
        for (int i = threadIdx.x; i < nt * kHalf; i += kThreads) {
            const int tl = i / kHalf, j = i % kHalf;
            const int32_t t = (int32_t)(t0 + tl);
            int32_t pos;
            if (kAtEnd) {
                const int32_t L = clipped_length(p, t);
                pos = L > 0 ? L - 1 : 0;
                if (j == 0) {
                    int64_t slot = -1;
                    if (L > 0) {
                        const int32_t blk = p.block_tables[(size_t)t * p.max_blocks_per_seq + pos / a.Bs];
                        if (blk >= 0 && blk < p.num_blocks) slot = (int64_t)blk * a.Bs + pos % a.Bs;
                    }
                    s_slot[tl] = slot;
                }
            } else {
                pos = a.positions[t];
                if (j == 0) {
                    const int64_t slot = a.slots[t];
                    s_slot[tl] = slot < a.num_slots ? slot : -1;
                }
            }
            double c = 1.0, s = 0.0;
            if (a.theta > 0.f) rope_cos_sin64(pos, s_inv[j], &c, &s);
            s_c[tl][j] = c;
            s_s[tl][j] = s;
            s_cf[tl][j] = (float)c;
            s_sf[tl][j] = (float)s;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < nt * per_token; i += kThreads) {
            const int tl = i / per_token;
            int w = i - tl * per_token;
            const size_t t = (size_t)(t0 + tl);
            if (w < qn) {
                const int h = w / kQItems, c = w % kQItems;
                const size_t src = (t * a.Hq + h) * D + c * 8;
                uint4 x1 = *reinterpret_cast<const uint4*>(a.q + src);
                uint4 x2 = *reinterpret_cast<const uint4*>(a.q + src + kHalf);
                rope_rotate8(x1, x2, s_cf[tl] + c * 8, s_sf[tl] + c * 8);
                *reinterpret_cast<uint4*>(a.q_out + src) = x1;
                *reinterpret_cast<uint4*>(a.q_out + src + kHalf) = x2;
                continue;
            }
            const int64_t slot = s_slot[tl];
            if (slot < 0) continue;
            w -= qn;
            int off;
            if (w < kn) {
                const int h = w / kKItems, g = w % kKItems;
                const uint4* s1 = reinterpret_cast<const uint4*>(a.k + (t * a.Hkv + h) * D + g * 16);
                const uint4* s2 = reinterpret_cast<const uint4*>(a.k + (t * a.Hkv + h) * D + kHalf + g * 16);
                float x1[16], x2[16];
                bf16x16_to_f32(__ldg(s1), __ldg(s1 + 1), x1);
                bf16x16_to_f32(__ldg(s2), __ldg(s2 + 1), x2);
                if (a.theta > 0.f) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const double c = s_c[tl][g * 16 + e], s = s_s[tl][g * 16 + e];
                        const double u = (double)x1[e], z = (double)x2[e];
                        x1[e] = __uint_as_float((uint32_t)rope_round(u * c - z * s) << 16);
                        x2[e] = __uint_as_float((uint32_t)rope_round(u * s + z * c) << 16);
                    }
                }
                uint8_t* page = page_of<D>(a.k_cache, slot, h, a.Hkv, a.Bs, off);
                store_group<D>(page, a.Bs, off, g, x1, a.k_inv);
                store_group<D>(page, a.Bs, off, g + D / 32, x2, a.k_inv);
            } else {
                w -= kn;
                const int h = w / kVItems, g = w % kVItems;
                const uint4* s1 = reinterpret_cast<const uint4*>(a.v + (t * a.Hkv + h) * D + g * 16);
                float x[16];
                bf16x16_to_f32(__ldg(s1), __ldg(s1 + 1), x);
                uint8_t* page = page_of<D>(a.v_cache, slot, h, a.Hkv, a.Bs, off);
                store_group<D>(page, a.Bs, off, g, x, a.v_inv);
            }
        }
    }
}

// The rows of the given slots as bf16: code * scale is exact in f16, times gs in float, rounded once.
template <int D>
__global__ void __launch_bounds__(kThreads) gather_e2m1_kernel(const E2m1Args a, uint16_t* k_out, uint16_t* v_out,
                                                               int tokens_per_cta) {
    allow_dependents();
    constexpr int kGroups = D / 16;
    const int per_token = a.Hkv * kGroups;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens_per_cta; t0 < a.T; t0 += (int64_t)gridDim.x * tokens_per_cta) {
        const int n = (int)min((int64_t)tokens_per_cta, a.T - t0) * per_token;
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const int tl = i / per_token, w = i - tl * per_token, h = w / kGroups, g = w % kGroups;
            const int64_t t = t0 + tl, slot = a.slots[t];
            const size_t dst = ((size_t)t * a.Hkv + h) * D + g * 16;
            const bool live = slot >= 0 && slot < a.num_slots;
            int off = 0;
            uint8_t* kp = live ? page_of<D>(a.k_cache, slot, h, a.Hkv, a.Bs, off) : nullptr;
            uint2 c[2] = {make_uint2(0, 0), make_uint2(0, 0)};
            uint32_t s[2] = {0, 0};
            if (live) {
                uint8_t* vp = a.v_cache + (kp - a.k_cache);
                c[0] = *e2m1_codes<D>(kp, off, g);
                c[1] = *e2m1_codes<D>(vp, off, g);
                s[0] = *e2m1_scale<D>(kp, a.Bs, off, g);
                s[1] = *e2m1_scale<D>(vp, a.Bs, off, g);
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint32_t sc = e4m3x2_to_f16x2(s[m] | (s[m] << 8));
                const float gs = m ? a.v_inv : a.k_inv;      // here: the scales themselves
                uint32_t h4[4], o[8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    e2m1x8_to_f16x2x4(u ? c[m].y : c[m].x, h4);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = f16x2_to_f32x2(mul_f16x2(h4[j], sc));
                        o[4 * u + j] = pack_bf16x2(__fmul_rn(f.x, gs), __fmul_rn(f.y, gs));
                    }
                }
                uint4* d4 = reinterpret_cast<uint4*>((m ? v_out : k_out) + dst);
                d4[0] = make_uint4(o[0], o[1], o[2], o[3]);
                d4[1] = make_uint4(o[4], o[5], o[6], o[7]);
            }
        }
    }
}

// Tokens a CTA takes at a time: enough items to fill its threads, few enough that a small call
// spreads over the SMs.
int tokens_per_cta(int32_t T, int items_per_token, int most) {
    int n = (2 * kThreads + items_per_token - 1) / items_per_token;
    const int spread = T / (148 * 2);
    if (n > spread) n = spread;
    if (n > most) n = most;
    return n < 1 ? 1 : n;
}
unsigned grid_for(int32_t T, int tpc) {
    const int64_t g = ((int64_t)T + tpc - 1) / tpc;
    return (unsigned)(g < 148 * 8 ? g : 148 * 8);
}

}  // namespace

cudaError_t launch_append_e2m1(const pa_bf16* q, pa_bf16* q_out, const pa_bf16* k, const pa_bf16* v,
                               const int32_t* positions, const int64_t* slots, int32_t T, float theta, float k_inv,
                               float v_inv, uint8_t* k_cache, uint8_t* v_cache, const pa_cache_desc& d,
                               cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    E2m1Args a{q, q_out, k, v, positions, slots, T, d.num_q_heads, d.num_kv_heads, d.block_size,
               (int64_t)d.num_blocks * d.block_size, theta, k_inv, v_inv, k_cache, v_cache};
    const int D = d.head_dim;
    if (theta > 0.f) {
        const int items = (d.num_q_heads + d.num_kv_heads) * D / 16 + d.num_kv_heads * D / 32;
        const int tpc = tokens_per_cta(T, items, kMaxTokens);
        const DecodeParams none{};
        if (D == 64)
            rope_append_e2m1_kernel<64, false><<<grid_for(T, tpc), kThreads, 0, stream>>>(a, none, tpc);
        else
            rope_append_e2m1_kernel<128, false><<<grid_for(T, tpc), kThreads, 0, stream>>>(a, none, tpc);
    } else {
        const int tpc = tokens_per_cta(T, d.num_kv_heads * D / 16, 64);
        if (D == 64)
            append_e2m1_kernel<64><<<grid_for(T, tpc), kThreads, 0, stream>>>(a, tpc);
        else
            append_e2m1_kernel<128><<<grid_for(T, tpc), kThreads, 0, stream>>>(a, tpc);
    }
    return cudaGetLastError();
}

cudaError_t launch_append_e2m1_at_end(const DecodeParams& p, uint16_t* q_out, cudaStream_t stream) {
    if (p.num_seqs == 0) return cudaSuccess;
    E2m1Args a{p.q, p.rope_theta > 0.f ? q_out : nullptr, p.k_new, p.v_new, nullptr, nullptr, p.num_seqs,
               p.num_q_heads, p.num_kv_heads, p.block_size, (int64_t)p.num_blocks * p.block_size, p.rope_theta,
               p.k_inv_scale, p.v_inv_scale,
               // the caches are the caller's writable buffers (pa_append_decode)
               reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(p.k_cache)),
               reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(p.v_cache))};
    const int D = p.head_dim;
    const int items = (p.num_q_heads + p.num_kv_heads) * D / 16 + p.num_kv_heads * D / 32;
    const int tpc = tokens_per_cta(p.num_seqs, items, kMaxTokens);
    if (D == 64)
        rope_append_e2m1_kernel<64, true><<<grid_for(p.num_seqs, tpc), kThreads, 0, stream>>>(a, p, tpc);
    else
        rope_append_e2m1_kernel<128, true><<<grid_for(p.num_seqs, tpc), kThreads, 0, stream>>>(a, p, tpc);
    return cudaGetLastError();
}

cudaError_t launch_gather_e2m1(const uint8_t* k_cache, const uint8_t* v_cache, const int64_t* slots, int32_t T,
                               float k_scale, float v_scale, pa_bf16* k, pa_bf16* v, const pa_cache_desc& d,
                               cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    E2m1Args a{nullptr, nullptr, nullptr, nullptr, nullptr, slots, T, d.num_q_heads, d.num_kv_heads, d.block_size,
               (int64_t)d.num_blocks * d.block_size, 0.f, k_scale, v_scale, const_cast<uint8_t*>(k_cache),
               const_cast<uint8_t*>(v_cache)};
    const int tpc = tokens_per_cta(T, d.num_kv_heads * d.head_dim / 16, 64);
    if (d.head_dim == 64)
        gather_e2m1_kernel<64><<<grid_for(T, tpc), kThreads, 0, stream>>>(a, k, v, tpc);
    else
        gather_e2m1_kernel<128><<<grid_for(T, tpc), kThreads, 0, stream>>>(a, k, v, tpc);
    return cudaGetLastError();
}

}  // namespace pa
