// Single-token attention over a 4-bit (E2M1) paged cache.
//
// The format (pa_e2m1.cuh) holds a K or V row of D values in 9 D / 16 bytes, 3.6 times fewer than
// bf16.  At that size a decode is no longer bound by its bytes alone: every code has to be widened
// and scaled before a tensor core can take it, so the kernel is built around that work.
//
//  * A warp owns one kv head of a run of tokens and keeps everything in registers: the codes of 16
//    tokens come straight from global memory in the shape of the MMA operands (no shared memory,
//    no barrier, nothing to wait for but the loads themselves), a few slabs ahead of their use.
//  * S = K q^T (16 tokens x 8 heads) takes K as the row operand: lane (r, c) holds, of tokens
//    tau(r) and tau(r) + 2, the c-th quarter of the head dimension, which is one load of whole
//    scale groups; the order of the dims inside the product is free, so q is laid out to match.
//  * O^T += V^T P takes V as the row operand: lane (r, c) holds the r-th eighth of the head
//    dimension of tokens 4c .. 4c+3.  A product needs pairs of tokens side by side: nibbles of two
//    tokens' words are merged into bytes (two shifts and two selects give eight of them), and one
//    conversion makes an f16 pair of each.
//  * tau(r) = 4 (r / 2) + r % 2 makes S come out in exactly the token order V wants, and the four
//    tokens of a lane are one word of scales for either operand (the page keeps the scales of a
//    group token by token for that).
//  * Codes and scales multiply in f16, exactly: 2 x 4 significant bits, 2^-10 <= |code scale| <=
//    2688.  q is brought to f16 by a power of two per row (its largest value near 2^8), undone on
//    the scores; P is rounded to f16 (relative 2^-11), sums and outputs are fp32.
//
// The work is the concatenation, over groups of HG kv heads (HG = 8, 4, 2 or 1, the largest that
// divides Hkv) and sequences, of slabs of tokens (an empty sequence counts one).  8 / HG teams of
// HG warps a CTA take equal slices of it; a team's warps read the same tokens, one kv head each, so
// that the team reads a page's heads together.  A sequence that lies in one slice is written out;
// one cut between slices leaves fp32 partial states, two a slice at most, which the merge kernel
// (merge.cu) joins.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "pa_device.cuh"
#include "pa_e2m1.cuh"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kLazyLog2 = 8.f;      // a slab rescales O only when a score passes the max by this

template <int D, int NT>
struct ECfg {
    static constexpr int kTiles = D == 64 ? 2 : 1;          // 16-token tiles a slab
    static constexpr int kSlab = 16 * kTiles;
    static constexpr int kBufs = D == 64 ? 2 : 3;           // slabs in registers
    static constexpr int kW = D / 64;                       // words of 8 codes a lane and token (V); half of K's
    static constexpr int kSteps = D / 16;                   // k steps of S, m tiles of O
    static constexpr int kMinBlocks = NT == 1 ? 2 : 1;
};

// What a lane holds of a slab, and what the slab is.
template <int D, int NT>
struct ESlab {
    using C = ECfg<D, NT>;
    uint32_t kc[C::kTiles][2][2 * C::kW];   // K codes of tokens tau(r), tau(r) + 2
    uint32_t ks[C::kTiles][C::kW];          // their group scales, four tokens a word
    uint32_t vc[C::kTiles][4][C::kW];       // V codes of tokens 4c .. 4c+3
    uint32_t vs[C::kTiles];                 // their scales
    int32_t b, valid;                       // sequence; tokens of the slab (0: an empty sequence)
    int32_t kvh;
    int32_t flags;                          // kFirst, kLast; nsplit << 8; slot << 7
};
enum : int32_t { kFirst = 1, kLast = 2, kSlot1 = 128 };

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// CTA-slice arithmetic: slice i of G takes slabs [i S / G, (i + 1) S / G); in 32 bits where they hold it.
__device__ __forceinline__ int64_t slice_lo(int64_t i, int64_t S, int64_t G, bool small) {
    return small ? (int64_t)((uint32_t)i * (uint32_t)S / (uint32_t)G) : i * S / G;
}
__device__ __forceinline__ int32_t slice_of(int64_t s, int64_t S, int64_t G, bool small) {
    return small ? (int32_t)((((uint32_t)s + 1u) * (uint32_t)G - 1u) / (uint32_t)S)
                 : (int32_t)(((s + 1) * G - 1) / S);
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, (ECfg<D, NT>::kMinBlocks))
    decode_e2m1_kernel(const DecodeParams p, const int HG) {
    using C = ECfg<D, NT>;
    constexpr int SL = C::kSlab, TS = C::kTiles, W = C::kW;
    allow_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    const int G = p.group, Hkv = p.num_kv_heads, B = p.num_seqs, Bs = p.block_size;
    const int bs_shift = 31 - __clz(Bs);                    // block sizes are powers of two
    const int hl = warp % HG, groups = Hkv / HG;
    const int64_t slice = (int64_t)blockIdx.x * (kWarps / HG) + warp / HG;
    const int64_t slices = (int64_t)gridDim.x * (kWarps / HG);
    const size_t page_bytes = e2m1_page_bytes(Bs, D);

    // ---- the slice: lane i sums the slabs of sequences [i cs, (i + 1) cs), one scan joins them ----
    const int cs = (B + 31) / 32;
    const int c_lo = min(B, lane * cs), c_hi = min(B, c_lo + cs);
    auto slabs_of = [&](int32_t L) { return L == 0 ? 1 : (L + SL - 1) / SL; };
    int64_t lane_sum = 0;
#pragma unroll 4
    for (int b = c_lo; b < c_hi; ++b) lane_sum += slabs_of(clipped_length(p, b));
    int64_t incl = lane_sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    const int64_t S_seq = __shfl_sync(0xffffffffu, incl, 31), S = S_seq * groups;
    const int64_t Gc = S < slices ? S : slices;             // never more slices than slabs
    const bool small = (S + 1) * (Gc + 1) < (1ll << 32);
    if (slice >= Gc) return;
    const int64_t lo = slice_lo(slice, S, Gc, small), hi = slice_lo(slice + 1, S, Gc, small);

    // ---- where slab lo is: group gi, sequence b, slab j of it; P = stream index of b's slab 0 ----
    int32_t gi = small ? (int32_t)((uint32_t)lo / (uint32_t)S_seq) : (int32_t)(lo / S_seq);
    int32_t b = 0, j = 0;
    int64_t P = 0;
    {
        const int64_t rem = lo - (int64_t)gi * S_seq, excl = incl - lane_sum;
        const int k = __ffs(__ballot_sync(0xffffffffu, rem >= excl && rem < incl)) - 1;
        if (lane == k) {
            int64_t acc = excl;
            for (int bb = c_lo; bb < c_hi; ++bb) {
                const int n = slabs_of(clipped_length(p, bb));
                if (rem < acc + n) {
                    b = bb;
                    j = (int32_t)(rem - acc);
                    P = (int64_t)gi * S_seq + acc;
                    break;
                }
                acc += n;
            }
        }
        b = __shfl_sync(0xffffffffu, b, k);
        j = __shfl_sync(0xffffffffu, j, k);
        P = __shfl_sync(0xffffffffu, P, k);
    }

    // ---- load cursor: the next slab to request, with its sequence's table window ----
    int32_t L = clipped_length(p, b), nb = slabs_of(L);
    auto entry = [&](int32_t bb, int32_t idx) -> int32_t {
        return idx < p.max_blocks_per_seq ? __ldg(p.block_tables + (size_t)bb * p.max_blocks_per_seq + idx) : -1;
    };
    int32_t win_base = (j * SL) >> bs_shift;
    int32_t win = entry(b, win_base + lane), win2 = entry(b, win_base + 32 + lane);
    int32_t nx_len = 0, nx_win = -1;                        // the next sequence's length and first window
    int64_t s = lo;
    int32_t seg = 0;                                        // nsplit << 8 | slot << 7 of the current segment

    const int tau = 4 * (r >> 1) + (r & 1);                 // K token of row r (the other is tau + 2)
    const int k_quad = 4 * (r >> 1), v_quad = 4 * c;        // first token of the scale words
    const uint32_t v_group = D == 64 ? r >> 1 : r;
    uint8_t* const kc_base = reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(p.k_cache));
    uint8_t* const vc_base = reinterpret_cast<uint8_t*>(const_cast<uint16_t*>(p.v_cache));

    auto fetch = [&](ESlab<D, NT>& x) {
        const bool first = s == lo || j == 0, last = s == hi - 1 || j == nb - 1;
        if (first) {
            const int32_t i_first = slice_of(P, S, Gc, small), i_last = slice_of(P + nb - 1, S, Gc, small);
            const int32_t fslot = P < slice_lo(i_first, S, Gc, small) ? 0 : 1;
            seg = ((i_last - i_first + 1) << 8) | (P < lo ? 0 : kSlot1);
            if (P >= lo && hl == 0 && lane == 0)            // this slice holds the sequence's first slab
                reinterpret_cast<int4*>(p.seq_desc)[(size_t)gi * B + b] =
                    make_int4(i_last - i_first + 1, i_first, fslot, 0);
            if (s != lo) {
                win_base = 0;
                win = nx_win;
                win2 = entry(b, 32 + lane);
            }
            if (s + (nb - j) < hi) {                        // the slice reaches the next sequence
                const int32_t bn = b + 1 == B ? 0 : b + 1;
                nx_len = __ldg(p.context_lens + bn);
                nx_win = entry(bn, lane);
            }
        }
        const int32_t t0 = j * SL;
        x.b = b;
        x.kvh = gi * HG + hl;
        x.valid = L == 0 ? 0 : min(SL, L - t0);
        x.flags = (first ? kFirst : 0) | (last ? kLast : 0) | seg;
        if (((t0 >> bs_shift) - win_base) >= 32) {          // a slab's blocks never straddle windows
            win_base += 32;
            win = win2;
            win2 = entry(b, win_base + 32 + lane);
        }
#pragma unroll
        for (int u = 0; u < TS; ++u) {
            const int tk = t0 + 16 * u + k_quad, tv = t0 + 16 * u + v_quad;
            const int32_t bk = __shfl_sync(0xffffffffu, win, ((tk >> bs_shift) - win_base) & 31);
            const int32_t bv = __shfl_sync(0xffffffffu, win, ((tv >> bs_shift) - win_base) & 31);
            bool ok = tk < L, ov = tv < L;
            if ((ok && (bk < 0 || bk >= p.num_blocks)) || (ov && (bv < 0 || bv >= p.num_blocks)))
                raise_status(p.status, kStatusBadBlock);
            ok = ok && bk >= 0 && bk < p.num_blocks;        // a block outside the pool reads as zeros
            ov = ov && bv >= 0 && bv < p.num_blocks;
#pragma unroll
            for (int i = 0; i < W; ++i) x.ks[u][i] = 0u;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 2 * W; ++i) x.kc[u][h][i] = 0u;
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < W; ++i) x.vc[u][t][i] = 0u;
            x.vs[u] = 0u;
            if (ok) {
                const uint8_t* page = kc_base + ((size_t)bk * Hkv + x.kvh) * page_bytes;
                const int off = tk & (Bs - 1);
                const uint8_t* row = page + (off + (r & 1)) * (D / 2) + c * (D / 8);
                if constexpr (D == 64) {
                    const uint2 a0 = __ldcg(reinterpret_cast<const uint2*>(row));
                    const uint2 a1 = __ldcg(reinterpret_cast<const uint2*>(row + 2 * (D / 2)));
                    x.kc[u][0][0] = a0.x; x.kc[u][0][1] = a0.y;
                    x.kc[u][1][0] = a1.x; x.kc[u][1][1] = a1.y;
                } else {
                    const uint4 a0 = __ldcg(reinterpret_cast<const uint4*>(row));
                    const uint4 a1 = __ldcg(reinterpret_cast<const uint4*>(row + 2 * (D / 2)));
                    x.kc[u][0][0] = a0.x; x.kc[u][0][1] = a0.y; x.kc[u][0][2] = a0.z; x.kc[u][0][3] = a0.w;
                    x.kc[u][1][0] = a1.x; x.kc[u][1][1] = a1.y; x.kc[u][1][2] = a1.z; x.kc[u][1][3] = a1.w;
                }
                const uint8_t* sc = page + Bs * (D / 2) + off;
#pragma unroll
                for (int i = 0; i < W; ++i)
                    x.ks[u][i] = __ldcg(reinterpret_cast<const uint32_t*>(sc + (c * W + i) * Bs));
            }
            if (ov) {
                const uint8_t* page = vc_base + ((size_t)bv * Hkv + x.kvh) * page_bytes;
                const int off = tv & (Bs - 1);
                const uint8_t* row = page + off * (D / 2) + r * (D / 16);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if constexpr (D == 64) {
                        x.vc[u][t][0] = __ldcg(reinterpret_cast<const uint32_t*>(row + t * (D / 2)));
                    } else {
                        const uint2 a = __ldcg(reinterpret_cast<const uint2*>(row + t * (D / 2)));
                        x.vc[u][t][0] = a.x; x.vc[u][t][1] = a.y;
                    }
                }
                uint32_t w = __ldcg(reinterpret_cast<const uint32_t*>(page + Bs * (D / 2) + v_group * Bs + off));
                x.vs[u] = w;
            }
        }
        // the next slab of the stream
        ++s;
        if (++j == nb) {
            j = 0;
            P += nb;
            if (++b == B) {
                b = 0;
                ++gi;
            }
            if (s < hi) {
                L = clip_length(p, nx_len);
                nb = slabs_of(L);
            }
        }
    };

    // ---- state of the current segment ----
    uint32_t qf[NT][C::kSteps][2];
    float sl2[NT][2], m_run[NT][2], l_run[NT][2];
    float o_acc[NT][C::kSteps][4];
    const uint32_t sel = (r & 1) ? 0x3311u : 0x2200u;       // scales of tokens tau, tau + 2, each twice

    auto start = [&](const ESlab<D, NT>& x) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = nt * 8 + r;
            uint4 qv[D / 32];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) qv[i] = make_uint4(0, 0, 0, 0);
            if (h < G) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    p.q + ((size_t)x.b * p.num_q_heads + (size_t)x.kvh * G + h) * D + c * (D / 4));
#pragma unroll
                for (int i = 0; i < D / 32; ++i) qv[i] = __ldcg(src + i);
            }
            // the row's power of two: its largest value between 2^8 and 2^9 in f16
            float big = 0.f;
            const uint32_t* w = reinterpret_cast<const uint32_t*>(qv);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) big = fmax3(big, fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i])));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            const uint32_t e = __float_as_uint(big) >> 23;                    // biased exponent
            const uint32_t up = e < 9u ? 253u : 262u - e;                     // 2^(8 - (e - 127)), biased
            const float f = __uint_as_float(up << 23);
            const float back = p.scale_log2 * __uint_as_float((254u - up) << 23);   // 2^-(up - 127)
#pragma unroll
            for (int ks = 0; ks < C::kSteps; ++ks) {
                qf[nt][ks][0] = pack_f16x2(bf16_lo(w[2 * ks]) * f, bf16_hi(w[2 * ks]) * f);
                qf[nt][ks][1] = pack_f16x2(bf16_lo(w[2 * ks + 1]) * f, bf16_hi(w[2 * ks + 1]) * f);
            }
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                sl2[nt][jj] = __shfl_sync(0xffffffffu, back, (2 * c + jj) * 4);
                m_run[nt][jj] = -INFINITY;
                l_run[nt][jj] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < C::kSteps; ++mt)
#pragma unroll
                for (int e4 = 0; e4 < 4; ++e4) o_acc[nt][mt][e4] = 0.f;
        }
    };

    auto process = [&](ESlab<D, NT>& x) {
        if (x.valid == 0) {                                 // an empty sequence: zeros
            store_zero_group(p, x.b, x.kvh, lane, 32);
            return;
        }
        if (x.flags & kFirst) start(x);
        // ---- S = K q^T ----
        float sv[TS][NT][4];
#pragma unroll
        for (int u = 0; u < TS; ++u) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sv[u][nt][e] = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) {                   // one scale group: 16 dims, 4 k steps
                const uint32_t ss = __byte_perm(x.ks[u][i], 0u, sel);
                const uint32_t s0 = e4m3x2_to_f16x2(ss), s1 = e4m3x2_to_f16x2(ss >> 16);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t lo4[4], hi4[4];
                    e2m1x8_to_f16x2x4(x.kc[u][0][2 * i + half], lo4);
                    e2m1x8_to_f16x2x4(x.kc[u][1][2 * i + half], hi4);
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        const uint32_t a[4] = {mul_f16x2(lo4[2 * k2], s0), mul_f16x2(hi4[2 * k2], s1),
                                               mul_f16x2(lo4[2 * k2 + 1], s0), mul_f16x2(hi4[2 * k2 + 1], s1)};
                        const int ks = 4 * i + 2 * half + k2;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(sv[u][nt], a, qf[nt][ks][0], qf[nt][ks][1]);
                    }
                }
            }
        }
        // ---- online softmax in the log2 domain, the running max kept lazily ----
        float mx[NT][2];
        bool need = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
        for (int u = 0; u < TS; ++u) {
            const bool v_lo = 16 * u + tau < x.valid, v_hi = 16 * u + tau + 2 < x.valid;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    sv[u][nt][e] = (e < 2 ? v_lo : v_hi) ? sv[u][nt][e] * sl2[nt][e & 1] : -INFINITY;
                mx[nt][0] = fmax3(mx[nt][0], sv[u][nt][0], sv[u][nt][2]);
                mx[nt][1] = fmax3(mx[nt][1], sv[u][nt][1], sv[u][nt][3]);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            need |= mx[nt][0] > m_run[nt][0] + kLazyLog2 || mx[nt][1] > m_run[nt][1] + kLazyLog2;
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    float v = mx[nt][jj];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                    const float mn = fmaxf(m_run[nt][jj], v), al = fast_exp2(m_run[nt][jj] - mn);
                    m_run[nt][jj] = mn;
                    l_run[nt][jj] *= al;
#pragma unroll
                    for (int mt = 0; mt < C::kSteps; ++mt) {
                        o_acc[nt][mt][jj] *= al;
                        o_acc[nt][mt][jj + 2] *= al;
                    }
                }
        }
        uint32_t pb[TS][NT][2];
#pragma unroll
        for (int u = 0; u < TS; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float p0 = fast_exp2(sv[u][nt][0] - m_run[nt][0]), p1 = fast_exp2(sv[u][nt][1] - m_run[nt][1]);
                const float p2 = fast_exp2(sv[u][nt][2] - m_run[nt][0]), p3 = fast_exp2(sv[u][nt][3] - m_run[nt][1]);
                l_run[nt][0] += p0 + p2;
                l_run[nt][1] += p1 + p3;
                pb[u][nt][0] = movmatrix_trans(pack_f16x2(p0, p1));   // tokens 4c, 4c+1
                pb[u][nt][1] = movmatrix_trans(pack_f16x2(p2, p3));   // tokens 4c+2, 4c+3
            }
        // ---- O^T += V^T P ----
#pragma unroll
        for (int u = 0; u < TS; ++u) {
            // tokens past the sequence may hold any bytes, NaN scales among them: scale 0
            const int left = x.valid - 16 * u - v_quad;
            uint32_t vs = x.vs[u];
            if (left < 4) vs = left <= 0 ? 0u : vs & (0xFFFFFFFFu >> (32 - 8 * left));
            const uint32_t s01 = e4m3x2_to_f16x2(vs), s23 = e4m3x2_to_f16x2(vs >> 16);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const uint32_t M = 0x0F0F0F0Fu;
                const uint32_t w0 = x.vc[u][0][i], w1 = x.vc[u][1][i], w2 = x.vc[u][2][i], w3 = x.vc[u][3][i];
                uint32_t e01[4], d01[4], e23[4], d23[4];    // even and odd dims of token pairs
                e2m1x8_to_f16x2x4((w0 & M) | ((w1 << 4) & ~M), e01);
                e2m1x8_to_f16x2x4(((w0 >> 4) & M) | (w1 & ~M), d01);
                e2m1x8_to_f16x2x4((w2 & M) | ((w3 << 4) & ~M), e23);
                e2m1x8_to_f16x2x4(((w2 >> 4) & M) | (w3 & ~M), d23);
#pragma unroll
                for (int k = 0; k < 4; ++k) {               // m tile 4 i + k: dims base + 2k (row r), + 1 (row r + 8)
                    const uint32_t a[4] = {mul_f16x2(e01[k], s01), mul_f16x2(d01[k], s01), mul_f16x2(e23[k], s23),
                                           mul_f16x2(d23[k], s23)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16_16816(o_acc[nt][4 * i + k], a, pb[u][nt][0], pb[u][nt][1]);
                }
            }
        }
        if (!(x.flags & kLast)) return;
        // ---- end of the segment: write out, or leave a partial state ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int jj = 0; jj < 2; ++jj)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l_run[nt][jj] += __shfl_xor_sync(0xffffffffu, l_run[nt][jj], off);
        const bool whole = (x.flags >> 8) == 1;
        const size_t prow = (((size_t)slice * 2 + ((x.flags & kSlot1) ? 1 : 0)) * Hkv + x.kvh) * G;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int h = nt * 8 + 2 * c + jj;
                if (h >= G) continue;
                const float inv = p.out_scale / l_run[nt][jj];
                // the lane's D / 8 dims r D / 8 ..: consecutive pairs
                if (whole) {
                    uint4* out = reinterpret_cast<uint4*>(
                        p.out + ((size_t)x.b * p.num_q_heads + (size_t)x.kvh * G + h) * D + r * (D / 8));
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        out[i] = make_uint4(
                            pack_bf16x2(o_acc[nt][4 * i][jj] * inv, o_acc[nt][4 * i][jj + 2] * inv),
                            pack_bf16x2(o_acc[nt][4 * i + 1][jj] * inv, o_acc[nt][4 * i + 1][jj + 2] * inv),
                            pack_bf16x2(o_acc[nt][4 * i + 2][jj] * inv, o_acc[nt][4 * i + 2][jj + 2] * inv),
                            pack_bf16x2(o_acc[nt][4 * i + 3][jj] * inv, o_acc[nt][4 * i + 3][jj + 2] * inv));
                } else {
                    float4* po = reinterpret_cast<float4*>(p.part_o + (prow + h) * D + r * (D / 8));
#pragma unroll
                    for (int i = 0; i < 2 * W; ++i)
                        po[i] = make_float4(o_acc[nt][2 * i][jj] * inv, o_acc[nt][2 * i][jj + 2] * inv,
                                            o_acc[nt][2 * i + 1][jj] * inv, o_acc[nt][2 * i + 1][jj + 2] * inv);
                    if (r == 0) p.part_lse[prow + h] = m_run[nt][jj] + __log2f(l_run[nt][jj]);
                }
            }
    };

    // everything below reads or writes what the previous kernel on the stream may touch
    wait_prerequisite();
    ESlab<D, NT> buf[C::kBufs];
    const int64_t total = hi - lo;
#pragma unroll
    for (int i = 0; i < C::kBufs; ++i)
        if (i < total) fetch(buf[i]);
    for (int64_t done = 0; done < total; done += C::kBufs) {
#pragma unroll
        for (int i = 0; i < C::kBufs; ++i) {
            if (done + i >= total) break;
            process(buf[i]);
            if (s < hi) fetch(buf[i]);
        }
    }
}

template <int D, int NT>
int occupancy() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int occ = cache[dev].load(std::memory_order_acquire);
    if (occ > 0) return occ;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, decode_e2m1_kernel<D, NT>, kThreads, 0) != cudaSuccess)
        return 0;
    cache[dev].store(occ, std::memory_order_release);
    return occ;
}

template <int D, int NT>
cudaError_t launch_e(const DecodeParams& p, int grid, bool pdl, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, decode_e2m1_kernel<D, NT>, p, p.desc_heads);
}

}  // namespace

int e2m1_head_group(int num_kv_heads) {
    for (int g = kWarps; g > 1; g >>= 1)
        if (num_kv_heads % g == 0) return g;
    return 1;
}
int e2m1_slab_tokens(int head_dim) { return head_dim == 64 ? ECfg<64, 1>::kSlab : ECfg<128, 1>::kSlab; }

int e2m1_kernel_grid(const pa_cache_desc& d, int max_ctas) {
    int sms = 0;
    if (num_sms_current_device(&sms) != PA_OK) return 0;
    const bool two = d.num_q_heads / d.num_kv_heads > 8;
    const int occ = d.head_dim == 64 ? (two ? occupancy<64, 2>() : occupancy<64, 1>())
                                     : (two ? occupancy<128, 2>() : occupancy<128, 1>());
    if (occ <= 0) return 0;
    const int grid = sms * occ;
    return max_ctas > 0 && max_ctas < grid ? max_ctas : grid;
}

cudaError_t launch_decode_e2m1(const DecodeParams& p, int grid, bool pdl, cudaStream_t stream) {
    const bool two = p.group > 8;
    if (p.head_dim == 64)
        return two ? launch_e<64, 2>(p, grid, pdl, stream) : launch_e<64, 1>(p, grid, pdl, stream);
    if (p.head_dim == 128)
        return two ? launch_e<128, 2>(p, grid, pdl, stream) : launch_e<128, 1>(p, grid, pdl, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pa
