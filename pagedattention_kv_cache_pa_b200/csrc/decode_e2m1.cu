// Single-token attention over a 4-bit (E2M1) paged cache.
//
// The format (pa_e2m1.cuh) holds a K or V row of D values in 9 D / 16 bytes, 3.6 times fewer than
// bf16.  At that size a decode is no longer bound by its bytes alone: every code has to be widened
// and scaled before a tensor core can take it, so the kernel is built around that work.
//
//  * A warp owns one kv head of a run of tokens, copies its pages into a ring of its own in shared
//    memory (16-byte asynchronous copies, a few slabs ahead) and takes the codes from there in the
//    shape of the MMA operands: no barrier, no other warp to wait for.  Held in registers instead,
//    the slabs ahead were one at most, and the loads' latency half of the time.
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
//    the scores; P is rounded to f16 (see kHeadLog2), sums and outputs are fp32.
//
// The work is the concatenation, over groups of HG kv heads (HG = 8, 4, 2 or 1, the largest that
// divides Hkv) and sequences, of slabs of tokens (an empty sequence counts one).  8 / HG teams of
// HG warps a TSA take equal slices of it; a team's warps read the same tokens, one kv head each, so
// that the team reads a page's heads together.  A sequence that lies in one slice is written out;
// one cut between slices leaves fp32 partial states, two a slice at most, which the merge kernel
// (merge.cu) joins.
//
// Measured (a call inside a CUDA graph, merge included): 32 and 8 heads of 64, 64 sequences up to 2048 tokens
// 22.5 us, 32 sequences on pages of 256 33 us (2.7 TB/s of 4-bit rows), one of 777 tokens 8.8 us; 64 and 8 heads
// of 128, 4 sequences up to 131072 87 us (4.1 TB/s).  Bound by instruction issue (63 % of the slots on the
// last, 368 warp instructions per 16 keys), and by about 8 us of start, plan and merge.
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <atomic>

#include "pa_device.cuh"
#include "pa_e2m1.cuh"
#include "pa_ptx.cuh"

namespace pa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// P is rounded to f16, whose steps below 2^-14 no longer shrink with the value: a long context's many small
// weights, which the sum keeps in fp32, would be lost from the products.  So the running max is kept 2^11
// below the largest score (weights reach 2^11, and 2^15 before a rescale): a weight is rounded by 2^-12 of
// itself down to 2^-25 of the largest, and by 2^-36 of the largest below that.
constexpr float kHeadLog2 = 11.f;
constexpr float kLazyLog2 = 4.f;      // a slab rescales O only when a score passes the largest by this
static_assert(kHeadLog2 + kLazyLog2 < 16.f, "P in f16's range");

template <int D, int NT>
struct ECfg {
    // 16-token tiles a slab, all of them in one turn of the softmax: with turns of half a slab the longest
    // case took 90.3 us for 88.1
    static constexpr int kTiles = D == 64 ? 4 : 2;
    static constexpr int kSlab = 16 * kTiles;
    static constexpr int kStages = 3;                       // slabs of a warp's ring: two CTAs fill shared memory
    static constexpr int kW = D / 64;                       // words of 8 codes a lane and token (V); half of K's
    static constexpr int kSteps = D / 16;                   // k steps of S, m tiles of O
    static constexpr int kMinBlocks = NT == 1 ? 2 : 1;
    // a stage: K codes, V codes, then per tile the scales of K and of V
    static constexpr int kCodeBytes = kSlab * D / 2, kTileScales = D;
    static constexpr int kStageBytes = 2 * kCodeBytes + 2 * kTiles * kTileScales;
    static constexpr size_t kSmem = (size_t)kWarps * kStages * kStageBytes;
};

// What a slab is (kept beside its bytes).
struct ESlab {
    int32_t b, kvh;
    int32_t valid;                          // tokens of the sequence from the slab's first on (0: it is empty)
    int32_t flags;                          // kFirst, kLast
    int64_t P;                              // stream index of the sequence's slab 0
    int32_t nb;                             // its slabs
};
enum : int32_t { kFirst = 1, kLast = 2 };

// 16-byte copies to shared memory, zeros instead where !live.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live = true) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t r;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}

// Where 16-byte chunk i of a tile's codes lies: chunks are permuted inside their 128-byte line so
// that a warp's reads of either operand's shape touch every bank once.  D = 64 (4 tokens a line):
// by 0, 4, 2, 6 from line to line; D = 128 (2 tokens a line): by 0, 0, 2, 2, 4, 4, 6, 6.
template <int D>
__device__ __forceinline__ uint32_t code_chunk(uint32_t i) {
    const uint32_t line = i >> 3;
    return D == 64 ? i ^ (((line & 1) << 2) | (line & 2)) : i ^ (line & 6);
}

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

// Slice i of G takes slabs [i S / G, (i + 1) S / G).  small (from the call's bounds): 32 bits hold S G.
__device__ __forceinline__ int64_t slice_lo(int64_t i, int64_t S, int64_t G, bool small) {
    return small ? (int64_t)((uint32_t)i * (uint32_t)S / (uint32_t)G) : i * S / G;
}
__device__ __forceinline__ int32_t slice_of(int64_t s, int64_t S, int64_t G, bool small) {
    return small ? (int32_t)((((uint32_t)s + 1u) * (uint32_t)G - 1u) / (uint32_t)S)
                 : (int32_t)(((s + 1) * G - 1) / S);
}

// kSmall: pages of 8 tokens (a 16-token tile spans two).
// kRows: causal prefill of few rows.  The columns of the products are (token, query head) pairs of up
// to p.q_tokens rows of a sequence, whose remaining rows are further "sequences" of the stream; a
// column sees the tokens up to its row's own.
template <int D, int NT, bool kSmall, bool kRows>
__global__ void __launch_bounds__(kThreads, (ECfg<D, NT>::kMinBlocks))
    decode_e2m1_kernel(const DecodeParams p, const int HG, const bool small) {
    using C = ECfg<D, NT>;
    constexpr int SL = C::kSlab, TS = C::kTiles, W = C::kW;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ ESlab s_slab[kWarps][C::kStages];
    allow_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, c = lane & 3;
    const int G = p.group, Hkv = p.num_kv_heads, B = p.num_seqs, Bs = p.block_size, cols = p.cols;
    const int bs_shift = 31 - __clz(Bs);                    // block sizes are powers of two
    const int hl = warp % HG, groups = Hkv / HG;
    const int64_t slice = (int64_t)blockIdx.x * (kWarps / HG) + warp / HG;
    const int64_t slices = (int64_t)gridDim.x * (kWarps / HG);

    // ---- the slice: lane i sums the slabs of sequences [i cs, (i + 1) cs), one scan joins them ----
    const int cs = (B + 31) / 32;
    const int c_lo = min(B, lane * cs), c_hi = min(B, c_lo + cs);
    // tokens that sequence b's last column sees: its length, or with kRows that of its last row
    auto length = [&](int32_t bb) -> int32_t {
        if constexpr (kRows) {
            int32_t row0, n;
            return rows_length(p, bb, row0, n);
        } else {
            return clipped_length(p, bb);
        }
    };
    auto table_row = [&](int32_t bb) { return (size_t)(kRows ? bb / p.q_chunks : bb) * p.max_blocks_per_seq; };
    auto slabs_of = [&](int32_t L) { return L == 0 ? 1 : (L + SL - 1) / SL; };
    int64_t lane_sum = 0, incl;
    if (small) {
        uint32_t sum = 0;
#pragma unroll 4
        for (int b = c_lo; b < c_hi; ++b) sum += slabs_of(length(b));
        uint32_t acc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, acc, off);
            if (lane >= off) acc += v;
        }
        lane_sum = sum;
        incl = acc;
    } else {
        for (int b = c_lo; b < c_hi; ++b) lane_sum += slabs_of(length(b));
        incl = lane_sum;
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
    }
    const int64_t S_seq = small ? (int64_t)__shfl_sync(0xffffffffu, (uint32_t)incl, 31) : __shfl_sync(0xffffffffu, incl, 31);
    const int64_t S = S_seq * groups, Gc = S < slices ? S : slices;   // never more slices than slabs
    if (slice >= Gc) return;
    const int64_t lo = slice_lo(slice, S, Gc, small), hi = slice_lo(slice + 1, S, Gc, small);

    // ---- where slab lo is: group gi, sequence b, slab j of it; P = stream index of b's slab 0 ----
    int32_t gi = groups == 1 ? 0 : small ? (int32_t)((uint32_t)lo / (uint32_t)S_seq) : (int32_t)(lo / S_seq);
    int32_t b = 0, j = 0;
    int64_t P = 0;
    {
        const int64_t rem = lo - (int64_t)gi * S_seq, excl = incl - lane_sum;
        const int k = __ffs(__ballot_sync(0xffffffffu, rem >= excl && rem < incl)) - 1;
        b = c_lo;
        int64_t acc = excl;
        if (lane == k) {
            for (int n; rem >= acc + (n = slabs_of(length(b))); ++b) acc += n;
            j = (int32_t)(rem - acc);
            P = (int64_t)gi * S_seq + acc;
        }
        b = __shfl_sync(0xffffffffu, b, k);
        j = __shfl_sync(0xffffffffu, j, k);
        P = __shfl_sync(0xffffffffu, P, k);
    }

    // ---- load cursor: the next slab to request, with its sequence's table window ----
    int32_t L = length(b), nb = slabs_of(L);
    auto entry = [&](int32_t bb, int32_t idx) -> int32_t {
        return idx < p.max_blocks_per_seq ? __ldg(p.block_tables + table_row(bb) + idx) : -1;
    };
    int32_t win_base = (j * SL) >> bs_shift;
    int32_t win = entry(b, win_base + lane), win2 = entry(b, win_base + 32 + lane);
    int32_t nx_len = 0, nx_win = -1;                        // the next sequence's length and first window
    int32_t left = (int32_t)(hi - lo);                      // slabs to request (fits: checked on the host)
    bool at_start = true;

    const uint32_t page_bytes = (uint32_t)e2m1_page_bytes(Bs, D);
    const uint8_t* const kc = reinterpret_cast<const uint8_t*>(p.k_cache);
    const uint8_t* const vc = reinterpret_cast<const uint8_t*>(p.v_cache);
    const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
    ESlab* const slabs = s_slab[warp];
    // this lane's scale copies: tile, cache, chunk of the tile's scales
    constexpr int kScaleChunks = D / 16;
    const int sc_u = lane / (2 * kScaleChunks), sc_v = (lane / kScaleChunks) & 1, sc_i = lane % kScaleChunks;
    const int sc_tok = kSmall ? 8 * (sc_i / (kScaleChunks / 2)) : 0;                     // first token it covers
    const uint32_t sc_off = Bs * (D / 2) + (kSmall ? (sc_i % (kScaleChunks / 2)) * 16 : sc_i * Bs);
    constexpr int kScaleTiles = 32 / (2 * kScaleChunks), kScaleCopies = TS / kScaleTiles;   // tiles a copy, copies
    static_assert(kScaleCopies * kScaleTiles == TS, "whole copies of scales");
    const uint8_t* const sc_src = (sc_v ? vc : kc) + sc_off;
    const uint32_t sc_dst = 2 * C::kCodeBytes + lane * 16;
    constexpr int kTileCodes = 16 * D / 2;
    const uint8_t *const kc_lane = kc + lane * 16, *const vc_lane = vc + lane * 16;
    uint32_t code_at[D / 64];
#pragma unroll
    for (int i = 0; i < D / 64; ++i) code_at[i] = code_chunk<D>(32 * i + lane) * 16;

    auto fetch = [&](int st) {
        const bool first = at_start || j == 0;
        if (first) {
            if (!at_start) {
                win_base = 0;
                win = nx_win;
                win2 = entry(b, 32 + lane);
            }
            at_start = false;
            if (!kRows && lane < (G * D + 63) / 64)         // its query rows, needed when it is processed
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + ((size_t)b * p.num_q_heads +
                                                                     (size_t)(gi * HG + hl) * G) * D + lane * 64));
            if (nb - j < left) {                            // the slice reaches the next sequence
                const int32_t bn = b + 1 == B ? 0 : b + 1;
                nx_len = kRows ? length(bn) : __ldg(p.context_lens + bn);
                nx_win = entry(bn, lane);
            }
        }
        const int32_t t0 = j * SL, kvh = gi * HG + hl;
        if (lane == 0) {
            const bool last = left == 1 || j == nb - 1;
            slabs[st] = ESlab{b, kvh, L - t0, (first ? kFirst : 0) | (last ? kLast : 0), P, nb};
        }
        if (((t0 >> bs_shift) - win_base) >= 32) {          // a slab's blocks never straddle windows
            win_base += 32;
            win = win2;
            win2 = entry(b, win_base + 32 + lane);
        }
        // Every lane copies, whatever the slab holds: tokens past the sequence are masked later; a
        // block outside the pool is read as block 0, with zeros for its scales.
        const uint32_t dst = ring + st * C::kStageBytes;
        bool bad = false;
#pragma unroll
        for (int u = 0; u < TS; ++u) {
            if (kSmall) {                                   // pages of 8 tokens: two a tile
                constexpr int kPageChunks = D / 4;          // chunks of codes of a page
                const int32_t tok = t0 + 16 * u + (D == 64 ? 8 * (lane / kPageChunks) : 0);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const int32_t blk = __shfl_sync(0xffffffffu, win, ((tok >> 3) + i - win_base) & 31);
                    const bool out = (uint32_t)blk >= (uint32_t)p.num_blocks;
                    bad |= out && tok + 8 * i < L;
                    const uint64_t off = (uint64_t)(uint32_t)((out ? 0 : blk) * Hkv + kvh) * page_bytes;
                    const uint32_t at = dst + u * kTileCodes + code_at[i];
                    copy16(at, kc + off + (lane % kPageChunks) * 16);
                    copy16(at + C::kCodeBytes, vc + off + (lane % kPageChunks) * 16);
                }
            } else {
                const int32_t tok = t0 + 16 * u;
                const int32_t blk = __shfl_sync(0xffffffffu, win, ((tok >> bs_shift) - win_base) & 31);
                const bool out = (uint32_t)blk >= (uint32_t)p.num_blocks;
                bad |= out && tok < L;
                const uint64_t off = (uint64_t)(uint32_t)((out ? 0 : blk) * Hkv + kvh) * page_bytes +
                                     (uint32_t)(tok & (Bs - 1)) * (D / 2);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {          // 32 chunks of codes, of K and of V
                    const uint32_t at = dst + u * kTileCodes + code_at[i];
                    copy16(at, kc_lane + off + 512 * i);
                    copy16(at + C::kCodeBytes, vc_lane + off + 512 * i);
                }
            }
        }
#pragma unroll
        for (int w = 0; w < kScaleCopies; ++w) {
            const int32_t tok = t0 + 16 * (sc_u + w * kScaleTiles) + sc_tok;
            const int32_t blk = __shfl_sync(0xffffffffu, win, ((tok >> bs_shift) - win_base) & 31);
            const bool in = (uint32_t)blk < (uint32_t)p.num_blocks;
            copy16(dst + sc_dst + 512 * w,
                   sc_src + (uint64_t)(uint32_t)((in ? blk : 0) * Hkv + kvh) * page_bytes + (kSmall ? 0 : tok & (Bs - 1)), in);
        }
        if (bad) raise_status(p.status, kStatusBadBlock);
        // the next slab of the stream
        --left;
        if (++j == nb) {
            j = 0;
            P += nb;
            if (++b == B) {
                b = 0;
                ++gi;
            }
            if (left > 0) {
                L = kRows ? nx_len : clip_length(p, nx_len);
                nb = slabs_of(L);
            }
        }
    };

    // ---- state of the current segment ----
    int32_t seg_split = 1, seg_slot = 0;
    uint32_t qf[NT][C::kSteps][2];
    float sl2[NT][2], m_run[NT][2], l_run[NT][2];
    float o_acc[NT][C::kSteps][4];
    const uint32_t sel = (r & 1) ? 0x3311u : 0x2200u;       // scales of tokens tau, tau + 2, each twice

    int32_t fewer[NT][2], fewer_most = 0, row0 = 0, ntok = 1;   // kRows: tokens that a column sees fewer than the last

    auto start = [&](const ESlab& x) {
        if constexpr (kRows) {
            rows_length(p, x.b, row0, ntok);
            fewer_most = ntok - 1;
        } else {
            row0 = x.b;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = nt * 8 + r, tok = kRows ? col / G : 0, h = col - tok * G;
            uint4 qv[D / 32];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) qv[i] = make_uint4(0, 0, 0, 0);
            if (kRows ? tok < ntok : h < G) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    p.q + ((size_t)(row0 + tok) * p.num_q_heads + (size_t)x.kvh * G + h) * D + c * (D / 4));
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
            // the scale's sign goes with q, so that a larger product is a larger score
            const float f = copysignf(__uint_as_float(up << 23), p.scale_log2);
            // (never 0, which would turn a masked -inf into a NaN)
            const float back = fmaxf(fabsf(p.scale_log2) * __uint_as_float((254u - up) << 23), 1e-37f);
#pragma unroll
            for (int ks = 0; ks < C::kSteps; ++ks) {
                qf[nt][ks][0] = pack_f16x2(bf16_lo(w[2 * ks]) * f, bf16_hi(w[2 * ks]) * f);
                qf[nt][ks][1] = pack_f16x2(bf16_lo(w[2 * ks + 1]) * f, bf16_hi(w[2 * ks + 1]) * f);
            }
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                sl2[nt][jj] = __shfl_sync(0xffffffffu, back, (2 * c + jj) * 4);
                // finite, so that a slab with nothing for a column weighs nothing (and is no NaN)
                m_run[nt][jj] = -FLT_MAX;
                if (kRows) fewer[nt][jj] = max(0, ntok - 1 - (nt * 8 + 2 * c + jj) / G);
                l_run[nt][jj] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < C::kSteps; ++mt)
#pragma unroll
                for (int e4 = 0; e4 < 4; ++e4) o_acc[nt][mt][e4] = 0.f;
        }
    };

    // this lane's places in a stage
    const int tau = 4 * (r >> 1) + (r & 1);                 // K token of row r (the other is tau + 2)
    const int k_quad = 4 * (r >> 1), v_quad = 4 * c;        // first token of the scale words
    uint32_t k_at[2], v_at[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)   // (D = 128: two tokens on is the next line, under the same permutation)
        k_at[i] = D == 64 ? code_chunk<D>((tau + 2 * i) * 2 + (c >> 1)) * 16 + (c & 1) * 8
                          : code_chunk<D>(tau * 4 + c) * 16 + 128 * i;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v_at[i] = C::kCodeBytes + (D == 64 ? code_chunk<D>((v_quad + i) * 2 + (r >> 2)) * 16 + (r & 3) * 4
                                           : code_chunk<D>((v_quad + (i & 1)) * 4 + (r >> 1)) * 16 + (r & 1) * 8 + 128 * (i >> 1));
    // scales of group g, four tokens from `quad`: [g][16 tokens], or [page][g][8 tokens]
    auto scale_at = [&](int g, int quad) {
        return 2 * C::kCodeBytes + (kSmall ? (quad >> 3) * (D / 2) + g * 8 + (quad & 7) : g * 16 + quad);
    };
    const uint32_t ks_at = scale_at(c * W, k_quad), vs_at = scale_at(D == 64 ? r >> 1 : r, v_quad) + C::kTileScales;

    auto process = [&](const ESlab& x, int st) {
        const uint32_t stage = ring + st * C::kStageBytes;
        const int valid = x.valid;

        if (x.valid == 0) {                                 // an empty sequence: zeros, nothing to join
            if (!kRows) store_zero_group(p, x.b, x.kvh, lane, 32);   // kRows: there are no rows
            if (hl == 0 && lane == 0)
                reinterpret_cast<int4*>(p.seq_desc)[(size_t)(x.kvh / HG) * B + x.b] = make_int4(1, 0, 0, 0);
            return;
        }
        if (x.flags & kFirst) {
            start(x);
            // the segment: how many slices share its sequence, and this one's partial slot
            const int32_t i_first = slice_of(x.P, S, Gc, small), i_last = slice_of(x.P + x.nb - 1, S, Gc, small);
            seg_split = i_last - i_first + 1;
            seg_slot = x.P < lo ? 0 : 1;
            if (x.P >= lo && hl == 0 && lane == 0)          // this slice holds the sequence's first slab
                reinterpret_cast<int4*>(p.seq_desc)[(size_t)(x.kvh / HG) * B + x.b] =
                    make_int4(seg_split, i_first, x.P < slice_lo(i_first, S, Gc, small) ? 0 : 1, 0);
        }
        // ---- S = K q^T ----
        float sv[TS][NT][4];
#pragma unroll
        for (int u = 0; u < TS; ++u) {
            uint32_t kw[2][2 * W];                          // codes of tokens tau, tau + 2
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (D == 64) {
                    const uint2 a = lds64(stage + k_at[h] + u * kTileCodes);
                    kw[h][0] = a.x; kw[h][1] = a.y;
                } else {
                    const uint4 a = lds128(stage + k_at[h] + u * kTileCodes);
                    kw[h][0] = a.x; kw[h][1] = a.y; kw[h][2] = a.z; kw[h][3] = a.w;
                }
            }
#pragma unroll
            for (int i = 0; i < W; ++i) {                   // one scale group: 16 dims, 4 k steps
                const uint32_t ss = __byte_perm(lds32(stage + ks_at + 2 * u * C::kTileScales + i * (kSmall ? 8 : 16)), 0u, sel);
                const uint32_t s0 = e4m3x2_to_f16x2(ss), s1 = e4m3x2_to_f16x2(ss >> 16);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t lo4[4], hi4[4];
                    e2m1x8_to_f16x2x4(kw[0][2 * i + half], lo4);
                    e2m1x8_to_f16x2x4(kw[1][2 * i + half], hi4);
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        const uint32_t a[4] = {mul_f16x2(lo4[2 * k2], s0), mul_f16x2(hi4[2 * k2], s1),
                                               mul_f16x2(lo4[2 * k2 + 1], s0), mul_f16x2(hi4[2 * k2 + 1], s1)};
                        const int ks = 4 * i + 2 * half + k2;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            if (ks == 0) mma_f16_16816_zero(sv[u][nt], a, qf[nt][ks][0], qf[nt][ks][1]);
                            else mma_f16_16816(sv[u][nt], a, qf[nt][ks][0], qf[nt][ks][1]);
                    }
                }
            }
        }
        // ---- online softmax in the log2 domain, the running max kept lazily ----
        uint32_t vs4[TS];
#pragma unroll
        for (int u = 0; u < TS; ++u) vs4[u] = lds32(stage + vs_at + 2 * u * C::kTileScales);
        if (valid - (kRows ? fewer_most : 0) < 16 * TS) {
            // tokens past the sequence: no weight; their V may hold any bytes, NaN scales among them
#pragma unroll
            for (int u = 0; u < TS; ++u) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (16 * u + tau + (e < 2 ? 0 : 2) >= valid - (kRows ? fewer[nt][e & 1] : 0))
                            sv[u][nt][e] = -INFINITY;
                const int in = valid - 16 * u - v_quad;
                if (in < 4) vs4[u] = in <= 0 ? 0u : vs4[u] & (0xFFFFFFFFu >> (32 - 8 * in));
            }
        }
        float mx[NT][2];
        bool need = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mx[nt][0] = fmaxf(sv[0][nt][0], sv[0][nt][2]);
            mx[nt][1] = fmaxf(sv[0][nt][1], sv[0][nt][3]);
#pragma unroll
            for (int u = 1; u < TS; ++u) {
                mx[nt][0] = fmax3(mx[nt][0], sv[u][nt][0], sv[u][nt][2]);
                mx[nt][1] = fmax3(mx[nt][1], sv[u][nt][1], sv[u][nt][3]);
            }
            mx[nt][0] *= sl2[nt][0];                        // sl2 > 0
            mx[nt][1] *= sl2[nt][1];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            need |= mx[nt][0] > m_run[nt][0] + (kHeadLog2 + kLazyLog2) || mx[nt][1] > m_run[nt][1] + (kHeadLog2 + kLazyLog2);
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    float v = mx[nt][jj];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                    const float mn = fmaxf(m_run[nt][jj], v - kHeadLog2), al = fast_exp2(m_run[nt][jj] - mn);
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
                const float p0 = fast_exp2(fmaf(sv[u][nt][0], sl2[nt][0], -m_run[nt][0]));
                const float p1 = fast_exp2(fmaf(sv[u][nt][1], sl2[nt][1], -m_run[nt][1]));
                const float p2 = fast_exp2(fmaf(sv[u][nt][2], sl2[nt][0], -m_run[nt][0]));
                const float p3 = fast_exp2(fmaf(sv[u][nt][3], sl2[nt][1], -m_run[nt][1]));
                l_run[nt][0] += p0 + p2;
                l_run[nt][1] += p1 + p3;
                pb[u][nt][0] = movmatrix_trans(pack_f16x2(p0, p1));   // tokens 4c, 4c+1
                pb[u][nt][1] = movmatrix_trans(pack_f16x2(p2, p3));   // tokens 4c+2, 4c+3
            }
        // ---- O^T += V^T P ----
#pragma unroll
        for (int u = 0; u < TS; ++u) {
            const uint32_t vs = vs4[u];
            uint32_t vw[4][W];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if constexpr (D == 64) {
                    vw[t][0] = lds32(stage + v_at[t] + u * kTileCodes);
                } else {
                    const uint2 a = lds64(stage + v_at[t] + u * kTileCodes);
                    vw[t][0] = a.x; vw[t][1] = a.y;
                }
            }
            const uint32_t s01 = e4m3x2_to_f16x2(vs), s23 = e4m3x2_to_f16x2(vs >> 16);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const uint32_t M = 0x0F0F0F0Fu;
                const uint32_t w0 = vw[0][i], w1 = vw[1][i], w2 = vw[2][i], w3 = vw[3][i];
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
        const bool whole = seg_split == 1;
        const size_t prow = (((size_t)slice * 2 + seg_slot) * Hkv + x.kvh) * cols;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int col = nt * 8 + 2 * c + jj, tok = kRows ? col / G : 0, h = col - tok * G;
                if (kRows ? tok >= ntok : h >= G) continue;
                // the scale only after the division: a small one over a long context's sum is no float
                const float inv = l_run[nt][jj] == 0.f ? 0.f : 1.f / l_run[nt][jj], os = p.out_scale;
                // the lane's D / 8 dims r D / 8 ..: consecutive pairs
                if (whole) {
                    uint4* out = reinterpret_cast<uint4*>(
                        p.out + ((size_t)(row0 + tok) * p.num_q_heads + (size_t)x.kvh * G + h) * D + r * (D / 8));
#pragma unroll
                    for (int i = 0; i < W; ++i)
                        out[i] = make_uint4(
                            pack_bf16x2(o_acc[nt][4 * i][jj] * inv * os, o_acc[nt][4 * i][jj + 2] * inv * os),
                            pack_bf16x2(o_acc[nt][4 * i + 1][jj] * inv * os, o_acc[nt][4 * i + 1][jj + 2] * inv * os),
                            pack_bf16x2(o_acc[nt][4 * i + 2][jj] * inv * os, o_acc[nt][4 * i + 2][jj + 2] * inv * os),
                            pack_bf16x2(o_acc[nt][4 * i + 3][jj] * inv * os, o_acc[nt][4 * i + 3][jj + 2] * inv * os));
                } else {
                    float4* po = reinterpret_cast<float4*>(p.part_o + (prow + col) * D + r * (D / 8));
#pragma unroll
                    for (int i = 0; i < 2 * W; ++i)
                        po[i] = make_float4(o_acc[nt][2 * i][jj] * inv * os, o_acc[nt][2 * i][jj + 2] * inv * os,
                                            o_acc[nt][2 * i + 1][jj] * inv * os, o_acc[nt][2 * i + 1][jj + 2] * inv * os);
                    if (r == 0)
                        p.part_lse[prow + col] = l_run[nt][jj] == 0.f ? -FLT_MAX : m_run[nt][jj] + __log2f(l_run[nt][jj]);
                }
            }
    };

    // everything below reads or writes what the previous kernel on the stream may touch
    wait_prerequisite();
    // slab i is requested kStages - 1 turns before it is processed (one copy of the code for both)
    const int32_t todo = left;
    for (int32_t i = 1 - C::kStages, st = 1, ahead = 0; i < todo; ++i) {
        if (i >= 0) {
            asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
            __syncwarp();                                   // every lane's copies of slab i; slab i - 1 read by all
        }
        if (left > 0) fetch(ahead);
        asm volatile("cp.async.commit_group;" ::: "memory");
        ahead = ahead + 1 == C::kStages ? 0 : ahead + 1;
        if (i >= 0) {
            const ESlab x = slabs[st];
            process(x, st);
        }
        st = st + 1 == C::kStages ? 0 : st + 1;
    }
}

template <int D, int NT, bool kSmall, bool kRows>
bool ensure_smem() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    const uint64_t bit = 1ull << dev;
    if (done.load(std::memory_order_acquire) & bit) return true;
    if (cudaFuncSetAttribute(decode_e2m1_kernel<D, NT, kSmall, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)ECfg<D, NT>::kSmem) != cudaSuccess)
        return false;
    done.fetch_or(bit, std::memory_order_acq_rel);
    return true;
}

template <int D, int NT>
int occupancy() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int occ = cache[dev].load(std::memory_order_acquire);
    if (occ > 0) return occ;
    if (!ensure_smem<D, NT, false, false>() ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, decode_e2m1_kernel<D, NT, false, false>, kThreads,
                                                      ECfg<D, NT>::kSmem) != cudaSuccess)
        return 0;
    cache[dev].store(occ, std::memory_order_release);
    return occ;
}

template <int D, int NT, bool kSmall, bool kRows>
cudaError_t launch_k(const DecodeParams& p, int grid, bool pdl, cudaStream_t stream) {
    if (!ensure_smem<D, NT, kSmall, kRows>()) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = ECfg<D, NT>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    // slabs of the whole call at most, times its slices: where that fits, the plan is made in 32 bits
    const uint64_t slabs = (uint64_t)p.num_seqs * (p.num_kv_heads / p.desc_heads) *
                           ((uint64_t)p.max_context_len / ECfg<D, NT>::kSlab + 1);
    const bool fits = (slabs + 1) * ((uint64_t)p.grid + 1) < (1ull << 32);
    return cudaLaunchKernelEx(&cfg, decode_e2m1_kernel<D, NT, kSmall, kRows>, p, p.desc_heads, fits);
}

template <int D, int NT>
cudaError_t launch_e(const DecodeParams& p, int grid, bool pdl, cudaStream_t stream) {
    const bool small = p.block_size < 16;
    if (p.cu_q) return small ? launch_k<D, NT, true, true>(p, grid, pdl, stream)
                             : launch_k<D, NT, false, true>(p, grid, pdl, stream);
    return small ? launch_k<D, NT, true, false>(p, grid, pdl, stream)
                 : launch_k<D, NT, false, false>(p, grid, pdl, stream);
}

}  // namespace

int e2m1_head_group(int num_kv_heads) {
    for (int g = kWarps; g > 1; g >>= 1)
        if (num_kv_heads % g == 0) return g;
    return 1;
}
int e2m1_slab_tokens(int head_dim) { return head_dim == 64 ? ECfg<64, 1>::kSlab : ECfg<128, 1>::kSlab; }

int e2m1_kernel_grid(const pa_cache_desc& d, int cols, int max_ctas) {
    int sms = 0;
    if (num_sms_current_device(&sms) != PA_OK) return 0;
    const bool two = cols > 8;
    const int occ = d.head_dim == 64 ? (two ? occupancy<64, 2>() : occupancy<64, 1>())
                                     : (two ? occupancy<128, 2>() : occupancy<128, 1>());
    if (occ <= 0) return 0;
    const int grid = sms * occ;
    return max_ctas > 0 && max_ctas < grid ? max_ctas : grid;
}

cudaError_t launch_decode_e2m1(const DecodeParams& p, int grid, bool pdl, cudaStream_t stream) {
    const bool two = p.cols > 8;
    if (p.head_dim == 64)
        return two ? launch_e<64, 2>(p, grid, pdl, stream) : launch_e<64, 1>(p, grid, pdl, stream);
    if (p.head_dim == 128)
        return two ? launch_e<128, 2>(p, grid, pdl, stream) : launch_e<128, 1>(p, grid, pdl, stream);
    return cudaErrorInvalidValue;
}

}  // namespace pa
