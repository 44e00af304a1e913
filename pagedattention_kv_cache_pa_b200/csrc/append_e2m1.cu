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
// time, whose D/2 cosines and sines are formed in double, once for all heads.
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

// q, K and V of a few tokens at a time, q and K turned by RoPE.  kAtEnd: the newest token of each
// sequence (position context_lens[b] - 1, through its table row); else positions and slots.
//
// The cosines and sines (in double) take some hundred dependent instructions a pair, and a tile of
// tokens has few pairs beside its rows.  So the rows' threads form them for the first tile only,
// with their first loads of q already under way; from then on a ninth warp forms the next tile's
// while the others work on this one.  (Formed between two barriers by all, they were a third of the
// time.)  Bound by the loads' latency and DRAM: 16384 tokens of 64 + 2 x 8 heads of 128 take, with their
// read-back, 141 us (690 MB, 76 % of the copy rate) with three CTAs an SM of two rows in flight a thread (which
// spill 20 bytes a thread), 144 with two CTAs of four, 154 with three of four or four of two (which spill more),
// 168 with the next tile's rows requested into L2 ahead.
constexpr int kMaxTokens = 8;
constexpr int kRopeThreads = kThreads + 32, kRopeCtas = 3;   // CTAs an SM

template <int D, bool kAtEnd>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    rope_append_e2m1_kernel(const E2m1Args a, const DecodeParams p, int tokens_per_cta) {
    allow_dependents();
    constexpr int kHalf = D / 2, kQItems = D / 16, kKItems = D / 32, kVItems = D / 16;
    __shared__ double s_inv[kHalf];
    __shared__ double s_c[2][kMaxTokens][kHalf], s_s[2][kMaxTokens][kHalf];
    __shared__ float s_cf[2][kMaxTokens][kHalf], s_sf[2][kMaxTokens][kHalf];
    __shared__ int64_t s_slot[2][kMaxTokens];
    const int tid = threadIdx.x;
    const int64_t step = (int64_t)gridDim.x * tokens_per_cta;
    // angles and slots of the tile at t0, by n threads of which this is number `who`
    auto angles = [&](int buf, int64_t t0, int who, int n) {
        const int nt = (int)min((int64_t)tokens_per_cta, a.T - t0);
        for (int i = who; i < nt * kHalf; i += n) {
            const int tl = i / kHalf, j = i % kHalf;
            const int32_t t = (int32_t)(t0 + tl);
            int32_t pos;
            if (kAtEnd) {
                const int32_t given = p.context_lens[t], L = clip_length(p, given);
                pos = L > 0 ? L - 1 : 0;
                if (j == 0) {
                    int64_t slot = -1;
                    if (L > 0 && L == given) {               // where a clipped length ends another token stands
                        const int32_t blk = p.block_tables[(size_t)t * p.max_blocks_per_seq + pos / a.Bs];
                        if (blk >= 0 && blk < p.num_blocks) slot = (int64_t)blk * a.Bs + pos % a.Bs;
                    }
                    s_slot[buf][tl] = slot;
                }
            } else {
                pos = a.positions[t];
                if (j == 0) {
                    const int64_t slot = a.slots[t];
                    s_slot[buf][tl] = slot < a.num_slots ? slot : -1;
                }
            }
            if (a.theta > 0.f) {
                double c, s;
                rope_cos_sin64(pos, s_inv[j], &c, &s);
                s_c[buf][tl][j] = c;
                s_s[buf][tl][j] = s;
                s_cf[buf][tl][j] = (float)c;
                s_sf[buf][tl][j] = (float)s;
            }
        }
    };
    // q rows (token, head) are contiguous: kQItems threads a row, kAhead rows in flight a thread
    constexpr int kRowStep = kThreads / kQItems, kAhead = 2;
    const int c8 = (tid % kQItems) * 8;
    uint4 x1[kAhead], x2[kAhead];
    auto load_q = [&](int64_t t0, int row, int rows) {
        const uint16_t* q = a.q + (size_t)t0 * a.Hq * D + c8;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int rr = row + u * kRowStep;
            if (rr < rows) {
                x1[u] = *reinterpret_cast<const uint4*>(q + (size_t)rr * D);
                x2[u] = *reinterpret_cast<const uint4*>(q + (size_t)rr * D + kHalf);
            }
        }
    };
    int64_t t0 = (int64_t)blockIdx.x * tokens_per_cta;
    const bool worker = tid < kThreads, turn_q = a.q_out != nullptr;
    int nt = (int)min((int64_t)tokens_per_cta, a.T - t0);
    if (worker && turn_q) load_q(t0, tid / kQItems, nt * a.Hq);
    if (a.theta > 0.f)
        for (int i = tid; i < kHalf; i += kRopeThreads) s_inv[i] = rope_inv_freq(i, D, a.theta);
    __syncthreads();
    angles(0, t0, tid, kRopeThreads);
    const int kn = a.Hkv * kKItems, per_token = kn + a.Hkv * kVItems;
    for (int buf = 0; t0 < a.T; buf ^= 1, t0 += step) {
        __syncthreads();   // this tile's angles are there; the last tile's are no longer read
        if (!worker) {
            if (t0 + step < a.T) angles(buf ^ 1, t0 + step, tid - kThreads, 32);
            continue;
        }
        nt = (int)min((int64_t)tokens_per_cta, a.T - t0);
        if (turn_q) {
            uint16_t* qo = a.q_out + (size_t)t0 * a.Hq * D + c8;
            const int rows = nt * a.Hq;
            for (int row = tid / kQItems; row < rows; row += kRowStep * kAhead) {
                if (row >= kRowStep || t0 != (int64_t)blockIdx.x * tokens_per_cta) load_q(t0, row, rows);
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int rr = row + u * kRowStep;
                    if (rr < rows) {
                        const int tl = rr / a.Hq;
                        rope_rotate8(x1[u], x2[u], s_cf[buf][tl] + c8, s_sf[buf][tl] + c8);
                        *reinterpret_cast<uint4*>(qo + (size_t)rr * D) = x1[u];
                        *reinterpret_cast<uint4*>(qo + (size_t)rr * D + kHalf) = x2[u];
                    }
                }
            }
        }
        for (int i = tid; i < nt * per_token; i += kThreads) {
            const int tl = i / per_token;
            int w = i - tl * per_token;
            const size_t t = (size_t)(t0 + tl);
            const int64_t slot = s_slot[buf][tl];
            if (slot < 0) continue;
            int off;
            if (w < kn) {
                const int h = w / kKItems, g = w % kKItems;
                const uint4* s1 = reinterpret_cast<const uint4*>(a.k + (t * a.Hkv + h) * D + g * 16);
                const uint4* s2 = reinterpret_cast<const uint4*>(a.k + (t * a.Hkv + h) * D + kHalf + g * 16);
                float y1[16], y2[16];
                bf16x16_to_f32(__ldg(s1), __ldg(s1 + 1), y1);
                bf16x16_to_f32(__ldg(s2), __ldg(s2 + 1), y2);
                if (a.theta > 0.f) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const double c = s_c[buf][tl][g * 16 + e], s = s_s[buf][tl][g * 16 + e];
                        const double u = (double)y1[e], z = (double)y2[e];
                        y1[e] = __uint_as_float((uint32_t)rope_round(u * c - z * s) << 16);
                        y2[e] = __uint_as_float((uint32_t)rope_round(u * s + z * c) << 16);
                    }
                }
                uint8_t* page = page_of<D>(a.k_cache, slot, h, a.Hkv, a.Bs, off);
                store_group<D>(page, a.Bs, off, g, y1, a.k_inv);
                store_group<D>(page, a.Bs, off, g + D / 32, y2, a.k_inv);
            } else {
                w -= kn;
                const int h = w / kVItems, g = w % kVItems;
                const uint4* s1 = reinterpret_cast<const uint4*>(a.v + (t * a.Hkv + h) * D + g * 16);
                float y[16];
                bf16x16_to_f32(__ldg(s1), __ldg(s1 + 1), y);
                uint8_t* page = page_of<D>(a.v_cache, slot, h, a.Hkv, a.Bs, off);
                store_group<D>(page, a.Bs, off, g, y, a.v_inv);
            }
        }
    }
}

// The rows of the given slots as bf16: code * scale is exact in f16, times gs in float, rounded once.
// A thread takes 8 dims of K and of V (a word of codes, a 16-byte store: whole sectors a warp), several
// of them in flight.
template <int D>
__global__ void __launch_bounds__(kThreads) gather_e2m1_kernel(const E2m1Args a, uint16_t* k_out, uint16_t* v_out,
                                                               int tokens_per_cta) {
    allow_dependents();
    constexpr int kWords = D / 8, kAhead = 4;
    const int per_token = a.Hkv * kWords;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens_per_cta; t0 < a.T; t0 += (int64_t)gridDim.x * tokens_per_cta) {
        const int n = (int)min((int64_t)tokens_per_cta, a.T - t0) * per_token;
        for (int i0 = threadIdx.x; i0 < n; i0 += kThreads * kAhead) {
            uint32_t c[kAhead][2], s[kAhead][2];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * kThreads;
                c[u][0] = c[u][1] = s[u][0] = s[u][1] = 0;
                if (i < n) {
                    const int tl = i / per_token, w = i - tl * per_token, h = w / kWords, word = w % kWords;
                    const int64_t slot = a.slots[t0 + tl];
                    if (slot >= 0 && slot < a.num_slots) {
                        int off;
                        uint8_t* kp = page_of<D>(a.k_cache, slot, h, a.Hkv, a.Bs, off);
                        uint8_t* vp = a.v_cache + (kp - a.k_cache);
                        c[u][0] = reinterpret_cast<const uint32_t*>(kp + off * (D / 2))[word];
                        c[u][1] = reinterpret_cast<const uint32_t*>(vp + off * (D / 2))[word];
                        s[u][0] = *e2m1_scale<D>(kp, a.Bs, off, word >> 1);
                        s[u][1] = *e2m1_scale<D>(vp, a.Bs, off, word >> 1);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int i = i0 + u * kThreads;
                if (i >= n) break;
                const size_t dst = ((size_t)t0 * per_token + i) * 8;   // words are contiguous in the output
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t sc = e4m3x2_to_f16x2(s[u][m] | (s[u][m] << 8));
                    const float gs = m ? a.v_inv : a.k_inv;      // here: the scales themselves
                    uint32_t h4[4], o[4];
                    e2m1x8_to_f16x2x4(c[u][m], h4);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = f16x2_to_f32x2(mul_f16x2(h4[j], sc));
                        o[j] = pack_bf16x2(__fmul_rn(f.x, gs), __fmul_rn(f.y, gs));
                    }
                    *reinterpret_cast<uint4*>((m ? v_out : k_out) + dst) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
}

// Tokens a CTA takes at a time: up to `most`, few enough that a small call spreads over `ctas` CTAs.
int tokens_per_cta(int32_t T, int most, int ctas) {
    const int spread = (T + ctas - 1) / ctas;
    return spread < most ? (spread < 1 ? 1 : spread) : most;
}
// CTAs for tiles of tpc tokens, at most `most`.  The rotating kernel's are all resident at once: a CTA's later
// tiles have their angles ready.
unsigned grid_for(int32_t T, int tpc, int most) {
    const int64_t g = ((int64_t)T + tpc - 1) / tpc;
    return (unsigned)(g < most ? g : most);
}
constexpr int kPlainCtas = 8, kPlainSpread = 2;   // CTAs an SM at most without rotation; those a small call spreads over

}  // namespace

cudaError_t launch_append_e2m1(const pa_bf16* q, pa_bf16* q_out, const pa_bf16* k, const pa_bf16* v,
                               const int32_t* positions, const int64_t* slots, int32_t T, float theta, float k_inv,
                               float v_inv, uint8_t* k_cache, uint8_t* v_cache, const pa_cache_desc& d,
                               cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    int sms = 0;
    if (num_sms_current_device(&sms) != PA_OK) return cudaErrorInvalidDevice;
    E2m1Args a{q, q_out, k, v, positions, slots, T, d.num_q_heads, d.num_kv_heads, d.block_size,
               (int64_t)d.num_blocks * d.block_size, theta, k_inv, v_inv, k_cache, v_cache};
    const int D = d.head_dim;
    if (theta > 0.f) {
        const int tpc = tokens_per_cta(T, kMaxTokens, sms * kRopeCtas);
        const DecodeParams none{};
        if (D == 64)
            rope_append_e2m1_kernel<64, false><<<grid_for(T, tpc, sms * kRopeCtas), kRopeThreads, 0, stream>>>(a, none, tpc);
        else
            rope_append_e2m1_kernel<128, false><<<grid_for(T, tpc, sms * kRopeCtas), kRopeThreads, 0, stream>>>(a, none, tpc);
    } else {
        const int tpc = tokens_per_cta(T, 8, sms * kPlainSpread);
        if (D == 64)
            append_e2m1_kernel<64><<<grid_for(T, tpc, sms * kPlainCtas), kThreads, 0, stream>>>(a, tpc);
        else
            append_e2m1_kernel<128><<<grid_for(T, tpc, sms * kPlainCtas), kThreads, 0, stream>>>(a, tpc);
    }
    return cudaGetLastError();
}

cudaError_t launch_append_e2m1_at_end(const DecodeParams& p, uint16_t* q_out, cudaStream_t stream) {
    if (p.num_seqs == 0) return cudaSuccess;
    int sms = 0;
    if (num_sms_current_device(&sms) != PA_OK) return cudaErrorInvalidDevice;
    E2m1Args a{p.q, p.rope_theta > 0.f ? q_out : nullptr, p.k_new, p.v_new, nullptr, nullptr, p.num_seqs,
               p.num_q_heads, p.num_kv_heads, p.block_size, (int64_t)p.num_blocks * p.block_size, p.rope_theta,
               p.k_inv_scale, p.v_inv_scale,
               // the caches are the caller's writable buffers (pa_append_decode)
               reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(p.k_cache)),
               reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(p.v_cache))};
    const int D = p.head_dim;
    const int tpc = tokens_per_cta(p.num_seqs, kMaxTokens, sms * kRopeCtas);
    if (D == 64)
        rope_append_e2m1_kernel<64, true><<<grid_for(p.num_seqs, tpc, sms * kRopeCtas), kRopeThreads, 0, stream>>>(a, p, tpc);
    else
        rope_append_e2m1_kernel<128, true><<<grid_for(p.num_seqs, tpc, sms * kRopeCtas), kRopeThreads, 0, stream>>>(a, p, tpc);
    return cudaGetLastError();
}

cudaError_t launch_gather_e2m1(const uint8_t* k_cache, const uint8_t* v_cache, const int64_t* slots, int32_t T,
                               float k_scale, float v_scale, pa_bf16* k, pa_bf16* v, const pa_cache_desc& d,
                               cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    int sms = 0;
    if (num_sms_current_device(&sms) != PA_OK) return cudaErrorInvalidDevice;
    E2m1Args a{nullptr, nullptr, nullptr, nullptr, nullptr, slots, T, d.num_q_heads, d.num_kv_heads, d.block_size,
               (int64_t)d.num_blocks * d.block_size, 0.f, k_scale, v_scale, const_cast<uint8_t*>(k_cache),
               const_cast<uint8_t*>(v_cache)};
    const int tpc = tokens_per_cta(T, 8, sms * kPlainSpread);
    if (d.head_dim == 64)
        gather_e2m1_kernel<64><<<grid_for(T, tpc, sms * kPlainCtas), kThreads, 0, stream>>>(a, k, v, tpc);
    else
        gather_e2m1_kernel<128><<<grid_for(T, tpc, sms * kPlainCtas), kThreads, 0, stream>>>(a, k, v, tpc);
    return cudaGetLastError();
}

}  // namespace pa
