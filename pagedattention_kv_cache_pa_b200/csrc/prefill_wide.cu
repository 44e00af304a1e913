// Attention of many query rows over a paged cache, two row tiles a CTA, on the fifth-generation
// tensor cores: causal (chunked) prefill over a 4-bit cache, and cross attention over a bf16 one with
// 128 dims.
//
// Prefill: sequence b's last Tq tokens attend causally to its L cached tokens, held in 4 bits
// (format: pa_e2m1.cuh).  Cross attention: a sequence's rows attend to all L tokens of its encoder.
//
// Three measurements on the B200 shaped the kernel.
//  * An MMA of 128 x 64 x 16 takes as long as one of 128 x 128 x 16: the A operand is read from
//    shared memory either way (16 of the first: 1013 cycles, of the second: 1139).  So tiles hold 128
//    keys.  For S and P of 128 keys and O of 128 dims, of two row tiles, tensor memory is exactly
//    enough when P takes the place of S (with 64 dims P has columns of its own).
//  * Issued by one thread of a divergent warp, whose descriptors go through vector registers, the
//    MMAs of a 64-dim head cost 80 cycles each; issued by an elected lane of a warp that runs as a
//    whole, 43 (ideal 32).  So the MMA warp runs as a whole.
//  * Widening 4-bit keys costs about as many instructions as half the softmax of 128 rows, so one
//    widened tile serves 256 query rows.
//
// Persistent CTAs, one per SM; items (256 query rows, kv head, sequence) are ordered by size and
// taken in zigzag as in prefill_ws.cu.  Warps with one job each meet through mbarriers only:
//   warps 0-3, 4-7  softmax of row tile 0 and 1: thread = row.  S out of tensor memory (64 keys at a
//                   time; those of the first half twice, to hold no more), the mask, the running max
//                   with lazy rescale of O in tensor memory, P back.
//   warps 8-11      K and V tiles.  4-bit: thread = key; codes and scales of the next tile are in
//                   flight in registers while this one is widened, V to f16 (one conversion and one
//                   product a pair, exact), K to bf16, q's type (the f16 pattern of a code shifted
//                   into bf16's fields is the code times 2^-112, which the scale's factor undoes,
//                   exact too).  bf16: warp 8 requests TMA boxes of 64 dims x min(Bs, 64) tokens.
//                   Rows of V past the sequence are zero, so P = 0 never meets a NaN there.
//   warp 12         (of a fourth warpgroup) MMA issue: O += P(t) V(t) of a row tile, then its
//                   S(t + 1), which with 128 dims overwrites P(t) and so waits for those products: the
//                   order of two MMAs is given for one accumulator and shape, and these have two.
//                   While one row tile's products run, the other's softmax has the exponential
//                   unit to itself; so that it is so from an item's start, the second row tile's
//                   first scores follow the first's second (153 -> 147 us with 64 dims below).
// K and V tiles have rings of their own.
//
// Long prefills of few items: the items of the last, unfilled round are cut (Walk, wide_split_ctas).
//
// Measured (a call inside a CUDA graph): 4-bit, 32 and 8 heads of 64, 4 x 2048 rows 149 us (463 TFLOP/s); 64 and
// 8 heads of 128, the last 1021 rows of 15000 623 us (833 TFLOP/s, the exponentials alone 226 us); cross
// attention, 32 and 8 heads of 128, 4 x 1024 rows over 4096 tokens 298 us (922 TFLOP/s).  Bound by a row tile's
// chain of scores, softmax and products (with 128 dims the wait before the next scores too: without it, on the
// order of issue alone, 613 and 274 us): without the softmax's arithmetic an earlier form of the first two took
// 125 and 513 us.
//
// Every wait is bounded (2 s, then the timeout status bit); the tensor memory is freed and no
// asynchronous operation is left when a CTA exits.
#include <cuda.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_e2m1.cuh"
#include "pa_internal.h"
#include "pa_ptx.cuh"
#include "pa_umma.cuh"

namespace pa {
namespace {

constexpr int kRows = 128;                 // query rows per softmax group (tensor-memory lanes)
constexpr int kItemRows = 2 * kRows;
constexpr int kKeys = 128;
constexpr int kLoad0 = 8, kMmaWarp = 12;   // first K/V warp, the MMA warp
constexpr int kThreads = 512;              // four warpgroups: softmax 0, softmax 1, K/V, MMA
// Registers a thread: 128 at launch, moved from the last two warpgroups to the softmax ones.  The
// shares add up to the launch's: 2 x 168 + 120 + 56 = 4 x 128.
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 168, kLoadRegs = 120, kMmaRegs = 56;
static_assert(2 * kSoftmaxRegs + kLoadRegs + kMmaRegs == 4 * kLaunchRegs, "register shares");
// The running max stays kHeadLog2 below a row's largest score, and O is rescaled when a score passes that by
// kRescaleLog2.  P in f16 (4-bit pools): weights up to 2^15, so that a long context's small ones are not lost (the
// reason is in decode_e2m1.cu): rounded by 2^-12 of themselves down to 2^-21 of the row's largest, and by 2^-32
// of the largest below that.  (11 and 4, as there, cost 10 to 20 % in rescales.)  In bf16 the range is fp32's.
constexpr float kRescaleLog2 = 8.f;
template <bool kE2m1>
constexpr float kHeadLog2 = kE2m1 ? 7.f : 0.f;
static_assert(kHeadLog2<true> + kRescaleLog2 < 16.f, "P in f16's range");

template <int D>
struct PCfg {
    static constexpr int kQBufs = D == 64 ? 2 : 1;                 // of each row tile
    static constexpr int kStages = D == 64 ? 4 : 2;                // of K, and of V
    static constexpr int kQBytes = kRows * D * 2;
    static constexpr int kTileBytes = kKeys * D * 2;
    static constexpr int kOffQ = 0;                                // [buffer][group]
    static constexpr int kOffK = kOffQ + 2 * kQBufs * kQBytes;
    static constexpr int kOffV = kOffK + kStages * kTileBytes;
    static constexpr int kOffBar = kOffV + kStages * kTileBytes;
    // s_full[2], p_full[2], o_done[2], o_free[2], q_full[2][2], drain, v_tail, then per stage k_full,
    // k_empty, v_full, v_empty
    static constexpr int kBars = 14 + 4 * kStages;
    static constexpr int kSmem = kOffBar + kBars * 8 + 16;
    // S: 128 columns a group; P: over the second half of S where O leaves no room for columns of its own
    static constexpr bool kOverS = D == 128;
    static constexpr int kColS = 0, kColP = kOverS ? 64 : 256, kStepP = kOverS ? 128 : 64, kColO = kOverS ? 256 : 384;
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kColO + 2 * D <= 512 && kSmem <= 227 * 1024, "tensor and shared memory of one CTA");
};

template <int ROWS>
__device__ __forceinline__ uint32_t sw128(int row, int c) {        // 16-byte chunk c of a row
    return (uint32_t)((c >> 3) * (ROWS * 128) + row * 128 + ((((c & 7) ^ (row & 7))) << 4));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// P in V's type
template <bool kE2m1>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
    uint32_t r;
    if constexpr (kE2m1) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void tmem_scale32(uint32_t taddr, float a) {
    uint32_t r[32];
    tmem_ld32(taddr, r);
#pragma unroll
    for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * a);
    tmem_st32(taddr, r);
}

// The item a CTA takes in its round r: rounds of grid items in order, CTAs in zigzag.
__device__ __forceinline__ long long item_index(long long r) {
    return r * gridDim.x + ((r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

// One work item: up to 256 query rows of one kv head of one sequence.
struct Item {
    int b, kvh, q0, Tq, L, rows, r0;
    int nt[2];                             // key tiles of either row tile (0: no rows, or none in this piece)
    int t0;                                // first key tile: not 0 for a piece that continues an item
    bool piece;                            // not all of the item's tiles
};

// Item i, as in prefill_ws.cu: the last row tiles of every chunk first.  1: an item to run; 0: none;
// -1: a sequence whose lengths cannot hold its queries; 2 (cross attention): rows with no token.
template <bool kCausal>
__device__ __forceinline__ int get_item(const PrefillParams& p, long long i, Item& it, bool& tile0) {
    const long long nsh = (long long)p.num_seqs * p.num_kv_heads;
    int t_rev, rem;
    if (i <= 0x7fffffffLL && nsh <= 0x7fffffffLL) {
        t_rev = (int)((unsigned)i / (unsigned)nsh);
        rem = (int)((unsigned)i - (unsigned)t_rev * (unsigned)nsh);
    } else {
        t_rev = (int)(i / nsh);
        rem = (int)(i - (long long)t_rev * nsh);
    }
    it.b = rem / p.num_kv_heads;
    it.kvh = rem - it.b * p.num_kv_heads;
    tile0 = t_rev == 0 && it.kvh == 0;
    it.q0 = p.cu_q[it.b];
    it.Tq = p.cu_q[it.b + 1] - it.q0;
    it.L = p.context_lens[it.b];
    if (it.Tq <= 0) return 0;
    // (len_cap says both; with the table's own bound before it, as it stood here, the 128-dim prefill is compiled
    // to 623 us for 1021 rows of 15000, alone to 640)
    if ((kCausal ? it.L < it.Tq : it.L < 0) || (long long)it.L > (long long)p.max_blocks_per_seq * p.block_size ||
        it.L > p.len_cap || it.Tq > p.max_q_len)
        return -1;
    it.rows = it.Tq * p.group;
    const int tile = (it.rows + kItemRows - 1) / kItemRows - 1 - t_rev;
    if (tile < 0) return 0;
    it.r0 = tile * kItemRows;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const int first = it.r0 + g * kRows;
        const int last_tok = min(it.rows - 1, first + kRows - 1) / p.group;
        const int seen = kCausal ? it.L - it.Tq + last_tok + 1 : it.L;
        it.nt[g] = first < it.rows ? (seen + kKeys - 1) / kKeys : 0;
    }
    it.t0 = 0;
    it.piece = false;
    return it.L > 0 ? 1 : 2;
}

// Partial states of 128 rows lie four dims of all rows after the next four: dims 4 i .. 4 i + 3 of state row
// `part` are [i kRows] from here on.
template <int D>
__device__ __forceinline__ float4* part_dims(float* part_o, size_t part) {
    return reinterpret_cast<float4*>(part_o) + part / kRows * kRows * (D / 4) + part % kRows;
}

// The walk of one role's warps over its CTA's items.  next() returns 1 for an item to run, 2 (cross
// attention) for rows with no token, 3 for nothing here, 0 at the end.
//
// kSplit: whole items only as long as there is one for every CTA.  The items of the last, unfilled round
// (fewer than CTAs) are cut: their key tiles stand in one row, of which CTA i of Gc takes tiles
// [i S / Gc, (i + 1) S / Gc).  An item cut between CTAs leaves a partial state (normalised fp32 O, log2-domain
// lse) a piece, joined by wide_merge_kernel; p.cuts says which.
constexpr int kMinSlice = 2;               // tiles a CTA at least

template <bool kCausal, bool kSplit>
struct Walk {
    std::conditional_t<kSplit, int, long long> r = -1;   // round (32 bits with kSplit: wide_split_ctas)
    uint32_t left = 0;                     // tiles of the slice to come
    int idx = 0, t = 0;                    // item of the last round, tile of it
    __device__ __forceinline__ Walk(const PrefillParams& p, long long n_items, bool report) {
        if (kSplit) cut(p, n_items, report);
    }
    static __device__ __forceinline__ long long base(long long n_items) {   // the first item of the last round
        return n_items - n_items % gridDim.x;
    }
    static __device__ __forceinline__ int get(const PrefillParams& p, long long i, Item& it, bool report) {
        bool tile0;
        const int st = get_item<kCausal>(p, i, it, tile0);
        if (report && st < 0 && tile0) raise_status(p.status, kStatusBadLength);
        return st > 0 ? st : 3;
    }
    static __device__ __forceinline__ int tiles(int st, const Item& it) {
        return st == 1 ? max(it.nt[0], it.nt[1]) : st == 2 ? 1 : 0;
    }
    // by a whole warp, once and before its work (beside it, the registers are not to be had): this CTA's
    // slice of the last round
    __device__ __forceinline__ void cut(const PrefillParams& p, long long n_items, bool report) {
        const long long base = Walk::base(n_items);
        const int R = (int)(n_items - base), lane = threadIdx.x & 31, per = (R + 31) / 32;
        const int first = min(R, lane * per), end = min(R, first + per);
        Item it;
        uint32_t sum = 0;                  // fewer items than CTAs, each of at most 2^24 tiles: 32 bits hold them
        for (int j = first; j < end; ++j) sum += tiles(get(p, base + j, it, report), it);
        uint32_t incl = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        const unsigned long long S = __shfl_sync(0xffffffffu, incl, 31);
        const unsigned long long Gc = min((unsigned long long)gridDim.x, max(1ull, S / kMinSlice)), me = blockIdx.x;
        const bool told = report && lane == 0;
        if (told) p.cuts[me] = make_int4(0, 0, 0, 0);
        if (me >= Gc || S == 0) return;
        const uint32_t lo = (uint32_t)(me * S / Gc), lo_before = me ? (uint32_t)((me - 1) * S / Gc) : 0;
        left = (uint32_t)((me + 1) * S / Gc) - lo;
        const int k = __ffs(__ballot_sync(0xffffffffu, lo >= incl - sum && lo < incl)) - 1;
        int nt = 0;
        idx = first;
        if (lane == k) {
            uint32_t rem = lo - (incl - sum);
            while (rem >= (uint32_t)(nt = tiles(get(p, base + idx, it, false), it))) rem -= nt, ++idx;
            t = (int)rem;
        }
        idx = __shfl_sync(0xffffffffu, idx, k);
        t = __shfl_sync(0xffffffffu, t, k);
        nt = __shfl_sync(0xffffffffu, nt, k);
        // the slice begins inside an item, and is the second to hold some of it: what there is to join
        if (told && t > 0 && lo - t >= lo_before) {
            get(p, base + idx, it, false);
            const unsigned long long last = ((lo - t + (unsigned long long)nt) * Gc - 1) / S;
            p.cuts[me] = make_int4((int)(last - me) + 2, it.b, it.kvh, it.r0);
        }
    }
    __device__ __forceinline__ int next(const PrefillParams& p, long long n_items, Item& it, bool report) {
        if (!kSplit) {
            const long long i = item_index(++r);
            return i < n_items ? get(p, i, it, report) : 0;
        }
        const long long base = Walk::base(n_items);
        if ((r + 1LL) * gridDim.x < base) return get(p, item_index(++r), it, report);
        if (left == 0) return 0;
        const int st = get(p, base + idx, it, false), nt = tiles(st, it);
        if (nt == 0) {
            ++idx;
            return 3;
        }
        const int n = (int)min(left, (uint32_t)(nt - t));
        it.t0 = t;
        it.piece = n < nt;
#pragma unroll
        for (int g = 0; g < 2; ++g) it.nt[g] = max(0, min(it.nt[g] - t, n));
        left -= n;
        t += n;
        if (t == nt) {
            t = 0;
            ++idx;
        }
        return st;
    }
};

template <int D, bool kE2m1, bool kCausal, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_wide_kernel(const PrefillParams p, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap) {
    using C = PCfg<D>;
    constexpr int kCh = D / 8, ST = C::kStages, QB = C::kQBufs;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t s_base = smem_u32(smem);
    const uint32_t s_q = s_base + C::kOffQ, s_k = s_base + C::kOffK, s_v = s_base + C::kOffV;
    const uint32_t bars = s_base + C::kOffBar;
    auto bar_s = [&](int g) { return bars + 8 * g; };
    auto bar_p = [&](int g) { return bars + 16 + 8 * g; };
    auto bar_o = [&](int g) { return bars + 32 + 8 * g; };
    auto bar_of = [&](int g) { return bars + 48 + 8 * g; };
    auto bar_q = [&](int buf, int g) { return bars + 64 + 16 * buf + 8 * g; };
    const uint32_t bar_drain = bars + 96, bar_tail = bars + 104;
    const uint32_t bar_kf = bars + 112, bar_ke = bar_kf + 8 * ST, bar_vf = bar_ke + 8 * ST, bar_ve = bar_vf + 8 * ST;
    const uint32_t s_tmem = bars + C::kBars * 8;
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int G = p.group, Hq = p.num_q_heads, Hkv = p.num_kv_heads, Bs = p.block_size;
    const long long n_items =
        (long long)p.num_seqs * Hkv * ((p.max_q_len * (long long)G + kItemRows - 1) / kItemRows);

    if (kSplit) allow_dependents();                          // the merge kernel waits for this grid's end
    if (s_base & 1023u) {                                    // the swizzle needs 1024-byte-aligned tiles
        if (tid == 0) raise_status(p.status, kStatusSmemAlign);
        return;
    }
    if (warp == 0) {
        tmem_alloc(s_tmem, C::kTmemCols);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int g = 0; g < 2; ++g) {
            mbar_init(bar_s(g), 1);
            mbar_init(bar_p(g), 4);                          // one arrival per softmax warp of the group
            mbar_init(bar_o(g), 1);
            mbar_init(bar_of(g), 4);
            mbar_init(bar_q(0, g), 4);
            mbar_init(bar_q(1, g), 4);
        }
        mbar_init(bar_drain, 1);
        mbar_init(bar_tail, 1);
        for (int i = 0; i < ST; ++i) {
            mbar_init(bar_kf + 8 * i, kE2m1 ? 4 : 1);        // 4-bit: one arrival per K/V warp; bf16: the requester's
            mbar_init(bar_vf + 8 * i, kE2m1 ? 4 : 1);
            mbar_init(bar_ke + 8 * i, 1);
            mbar_init(bar_ve + 8 * i, 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    uint32_t tmem;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(s_tmem) : "memory");
    tmem = __shfl_sync(0xffffffffu, tmem, 0);
    using W = Walk<kCausal, kSplit>;

    if (warp >= kLoad0 && warp < kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
        // ============================== K and V ==============================
        if constexpr (kE2m1) {
            constexpr int kBlk = D / 32;                     // 16-byte blocks of codes a row
            const int key = tid - kLoad0 * 32;
            const size_t page_bytes = e2m1_page_bytes(Bs, D);
            const int bs_shift = 31 - __clz(Bs);
            const uint8_t* kc = reinterpret_cast<const uint8_t*>(p.k_cache);
            const uint8_t* vc = reinterpret_cast<const uint8_t*>(p.v_cache);
            struct Cur {                                     // a key tile, and the block of this thread's key
                Item it;
                int t, id;
                bool has;
            };
            struct Raw {
                uint4 k[kBlk], v[kBlk];
                uint32_t ks[kBlk], vs[kBlk];                 // two scale bytes a block, one per half word
            };
            W walk(p, n_items, warp == kLoad0);
            auto lookup = [&](Cur& c) {
                const int kp = (c.it.t0 + c.t) * kKeys + key;
                c.id = -1;
                if (c.has && kp < c.it.L)
                    c.id = __ldg(p.block_tables + (size_t)c.it.b * p.max_blocks_per_seq + (kp >> bs_shift));
            };
            auto next = [&](const Cur& c, Cur& n) {
                n = c;
                if (c.has && ++n.t < max(c.it.nt[0], c.it.nt[1])) {
                    lookup(n);
                    return;
                }
                n.has = false;
                n.t = 0;
                for (int st; (st = walk.next(p, n_items, n.it, warp == kLoad0));)
                    if (st == 1) {
                        n.has = true;
                        break;
                    }
                lookup(n);
            };
            auto load = [&](const Cur& c, Raw& x) {
                const int kp = (c.it.t0 + c.t) * kKeys + key;
                bool ok = c.has && kp < c.it.L;
                if (ok && (c.id < 0 || c.id >= p.num_blocks)) {
                    raise_status(p.status, kStatusBadBlock);
                    ok = false;
                }
#pragma unroll
                for (int i = 0; i < kBlk; ++i) {
                    x.k[i] = x.v[i] = make_uint4(0, 0, 0, 0);
                    x.ks[i] = x.vs[i] = 0u;
                }
                if (!ok) return;
                const int off = kp & (Bs - 1);
                const size_t page = ((size_t)c.id * Hkv + c.it.kvh) * page_bytes;
                const size_t row = page + off * (D / 2), sc = page + Bs * (D / 2) + off;
#pragma unroll
                for (int i = 0; i < kBlk; ++i) {
                    x.k[i] = __ldg(reinterpret_cast<const uint4*>(kc + row + 16 * i));
                    x.v[i] = __ldg(reinterpret_cast<const uint4*>(vc + row + 16 * i));
                    x.ks[i] = (uint32_t)__ldg(kc + sc + (2 * i) * Bs) | ((uint32_t)__ldg(kc + sc + (2 * i + 1) * Bs) << 16);
                    x.vs[i] = (uint32_t)__ldg(vc + sc + (2 * i) * Bs) | ((uint32_t)__ldg(vc + sc + (2 * i + 1) * Bs) << 16);
                }
            };
            int g = 0;                                       // tiles so far (ring counter)
            auto put = [&](uint32_t dst, const uint32_t (&h)[4]) {
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                             : "memory");
            };
            auto publish = [&](uint32_t bar) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            };
            auto widen = [&](const Raw& x) -> bool {
                const int st = g % ST;
                if (g >= ST && !warp_wait(bar_ke + 8 * st, (uint32_t)((g / ST - 1) & 1), p.status)) return false;
#pragma unroll
                for (int i = 0; i < kBlk; ++i) {
                    const uint32_t w[4] = {x.k[i].x, x.k[i].y, x.k[i].z, x.k[i].w};
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr) {         // one scale group: two words
                        const float s = f16x2_to_f32x2(e4m3x2_to_f16x2((x.ks[i] >> (16 * gr)) & 0xFFu)).x;
                        const uint32_t sb = pack_bf16x2(s * 0x1p112f, s * 0x1p112f);
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            uint32_t h[4];
                            e2m1x8_to_f16x2x4(w[2 * gr + u], h);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                h[j] = mul_bf16x2(((h[j] >> 3) & 0x0FFF0FFFu) | (h[j] & 0x80008000u), sb);
                            put(s_k + st * C::kTileBytes + sw128<kKeys>(key, 4 * i + 2 * gr + u), h);
                        }
                    }
                }
                publish(bar_kf + 8 * st);
                if (g >= ST && !warp_wait(bar_ve + 8 * st, (uint32_t)((g / ST - 1) & 1), p.status)) return false;
#pragma unroll
                for (int i = 0; i < kBlk; ++i) {
                    const uint32_t w[4] = {x.v[i].x, x.v[i].y, x.v[i].z, x.v[i].w};
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr) {
                        const uint32_t b = (x.vs[i] >> (16 * gr)) & 0xFFu, s = e4m3x2_to_f16x2(b | (b << 8));
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            uint32_t h[4];
                            e2m1x8_to_f16x2x4(w[2 * gr + u], h);
#pragma unroll
                            for (int j = 0; j < 4; ++j) h[j] = mul_f16x2(h[j], s);
                            put(s_v + st * C::kTileBytes + sw128<kKeys>(key, 4 * i + 2 * gr + u), h);
                        }
                    }
                }
                publish(bar_vf + 8 * st);
                ++g;
                return true;
            };
            Cur a, b;
            Raw xa, xb;
            a.has = false;
            next(a, a);
            load(a, xa);
            next(a, b);
            while (a.has) {                                  // a: loaded; b: its block is known
                load(b, xb);
                next(b, a);
                if (!widen(xa)) break;
                if (!b.has) break;
                load(a, xa);
                next(a, b);
                if (!widen(xb)) break;
            }
        } else if (warp == kLoad0) {
            const int rb = Bs < 64 ? Bs : 64, nslot = kKeys / rb;   // rows a box, boxes a tile (at most 16)
            int g = 0, tails = 0;
            int k_last[ST], v_last[ST];                      // the tile last requested into a stage (V: not a tail)
#pragma unroll
            for (int u = 0; u < ST; ++u) k_last[u] = v_last[u] = -1;
            Item it;
            bool ok = true, tail_out = false;
            W walk(p, n_items, true);
            for (int kind; ok && (kind = walk.next(p, n_items, it, true));) {
                if (kind != 1) continue;
                const int* table = p.block_tables + (size_t)it.b * p.max_blocks_per_seq;
                const int nt = max(it.nt[0], it.nt[1]);
                for (int t = 0; t < nt && ok; ++t, ++g) {
                    const int st = g % ST, kp = (it.t0 + t) * kKeys + lane * rb;
                    bool valid = lane < nslot && kp < it.L;
                    const int id = valid ? __ldg(table + kp / Bs) : 0;
                    if (valid && (id < 0 || id >= p.num_blocks)) {
                        raise_status(p.status, kStatusBadBlock);
                        valid = false;
                    }
                    const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, valid)) * rb * 128 * (D / 64));
                    const int z = id * Hkv + it.kvh, y = kp % Bs;
                    const uint32_t par = (uint32_t)((g / ST - 1) & 1);
                    if (g >= ST && !(ok = warp_wait(bar_ke + 8 * st, par, p.status))) break;
                    if (lane == 0) mbar_arrive_expect_tx(bar_kf + 8 * st, bytes);
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < ST; ++u) k_last[u] = u == st ? g : k_last[u];
                    if (valid)
#pragma unroll
                        for (int a = 0; a < D / 64; ++a)
                            tma_load_3d(s_k + st * C::kTileBytes + a * (kKeys * 128) + lane * rb * 128, &kmap, a * 64, y, z,
                                        bar_kf + 8 * st);
                    if (g >= ST && !(ok = warp_wait(bar_ve + 8 * st, par, p.status))) break;
                    // rows of V past the sequence are zeroed once the tile has landed, before it is published
                    const int in = it.L - (it.t0 + t) * kKeys;
                    const uint32_t vbar = in < kKeys ? bar_tail : bar_vf + 8 * st;
                    if (lane == 0) mbar_arrive_expect_tx(vbar, bytes);
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < ST; ++u) v_last[u] = u != st ? v_last[u] : in >= kKeys ? g : -1;
                    tail_out = in < kKeys;
                    if (valid)
#pragma unroll
                        for (int a = 0; a < D / 64; ++a)
                            tma_load_3d(s_v + st * C::kTileBytes + a * (kKeys * 128) + lane * rb * 128, &vmap, a * 64, y, z, vbar);
                    if (in < kKeys) {
                        if (!(ok = warp_wait(bar_tail, (uint32_t)(tails & 1), p.status))) break;
                        ++tails;
                        tail_out = false;
                        for (int c = lane; c < (kKeys - in) * kCh; c += 32)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             s_v + st * C::kTileBytes + sw128<kKeys>(in + c / kCh, c % kCh)),
                                         "r"(0u)
                                         : "memory");
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar_vf + 8 * st);
                    }
                }
            }
            // in a call that ends as it should, every copy has been waited for; after a wait that ran out,
            // those still out end (or have their own time) before the CTA does
            if (!ok) {
#pragma unroll
                for (int u = 0; u < ST; ++u) {
                    if (k_last[u] >= 0) warp_wait(bar_kf + 8 * u, (uint32_t)((k_last[u] / ST) & 1), p.status);
                    if (v_last[u] >= 0) warp_wait(bar_vf + 8 * u, (uint32_t)((v_last[u] / ST) & 1), p.status);
                }
                if (tail_out) warp_wait(bar_tail, (uint32_t)(tails & 1), p.status);
            }
        }
    } else if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
        // ================================ MMA ================================
        if (warp == kMmaWarp) {
            constexpr uint32_t kIdescS = umma_idesc_bf16(kRows, kKeys, false);
            constexpr uint32_t kIdescO = kE2m1 ? umma_idesc_f16(kRows, D, true) : umma_idesc_bf16(kRows, D, true);
            const bool leader = elect_one();
            // ring positions (stage, phase) and counters of either row tile, all warp-uniform
            int ks = 0, kph = 0, vs = 0, vph = 0;
            int tiles[2] = {0, 0}, items[2] = {0, 0};
            bool ok = true;
            auto issue_s = [&](int gr, int buf, int stage) { // S of row tile gr = Q K^T
                const uint32_t q = s_q + (2 * buf + gr) * C::kQBytes, kt = s_k + stage * C::kTileBytes;
                if (leader) {
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        umma_bf16_ss(tmem + C::kColS + gr * kKeys,
                                     umma_desc_sw128(q + (k >> 2) * (kRows * 128) + (k & 3) * 32, 16, 1024),
                                     umma_desc_sw128(kt + (k >> 2) * (kKeys * 128) + (k & 3) * 32, 16, 1024), kIdescS, k > 0);
                    umma_commit(bar_s(gr));
                }
            };
            auto issue_o = [&](int gr, int stage, bool first) {   // O of row tile gr (+)= P V
                const uint32_t vt = s_v + stage * C::kTileBytes;
                if (leader) {
#pragma unroll
                    for (int k = 0; k < kKeys / 16; ++k)
                        umma_bf16_ts(tmem + C::kColO + gr * D, tmem + C::kColP + gr * C::kStepP + k * 8,
                                     umma_desc_sw128(vt + k * 16 * 128, kKeys * 128, 1024), kIdescO,
                                     (!first || k > 0) ? 1u : 0u);
                    umma_commit(bar_o(gr));
                }
            };
            Item it;
            W walk(p, n_items, false);
            for (int kind; ok && (kind = walk.next(p, n_items, it, false));) {
                if (__shfl_sync(0xffffffffu, kind, 0) != 1) continue;
                const int n0 = __shfl_sync(0xffffffffu, it.nt[0], 0), n1 = __shfl_sync(0xffffffffu, it.nt[1], 0);
                const int nt = max(n0, n1);
                // the first scores of either row tile; the second's follow the first's second
                const bool late = n0 > 0 && n1 > 0;
                const int ks0 = ks;
                if (!(ok = warp_wait(bar_kf + 8 * ks, (uint32_t)kph, p.status))) break;
#pragma unroll
                for (int gr = 0; gr < 2; ++gr) {
                    if ((gr ? n1 : n0) == 0 || (gr && late)) continue;
                    const int buf = items[gr] % QB;
                    if (!(ok = ok && warp_wait(bar_q(buf, gr), (uint32_t)((items[gr] / QB) & 1), p.status))) break;
                    tc_fence_after_sync();
                    issue_s(gr, buf, ks);
                }
                if (!ok) break;
                if (leader && !late) umma_commit(bar_ke + 8 * ks);
                if (++ks == ST) ks = 0, kph ^= 1;
                for (int t = 0; t < nt && ok; ++t) {
                    const bool more = t + 1 < nt;
                    if (more && !(ok = warp_wait(bar_kf + 8 * ks, (uint32_t)kph, p.status))) break;
                    if (!(ok = warp_wait(bar_vf + 8 * vs, (uint32_t)vph, p.status))) break;
#pragma unroll
                    for (int gr = 0; gr < 2; ++gr) {
                        const int n = gr ? n1 : n0;
                        if (t >= n) continue;
                        ok = ok && warp_wait(bar_p(gr), (uint32_t)((tiles[gr] + t) & 1), p.status);
                        // an item's first product overwrites O: not before the last item's was read
                        if (t == 0 && items[gr] > 0)
                            ok = ok && warp_wait(bar_of(gr), (uint32_t)((items[gr] - 1) & 1), p.status);
                        if (!ok) break;
                        tc_fence_after_sync();
                        issue_o(gr, vs, t == 0);
                        if (t + 1 < n) {
                            // P(t) lies in S(t + 1)'s columns: not before its products are done.  (An item's
                            // first scores wait for its Q, published after the last item's products.)
                            if (C::kOverS) {
                                if (!(ok = warp_wait(bar_o(gr), (uint32_t)((tiles[gr] + t) & 1), p.status))) break;
                                tc_fence_after_sync();
                            }
                            issue_s(gr, items[gr] % QB, ks);
                        }
                        if (gr == 0 && t == 0 && late) {
                            const int buf = items[1] % QB;
                            if (!(ok = warp_wait(bar_q(buf, 1), (uint32_t)((items[1] / QB) & 1), p.status))) break;
                            tc_fence_after_sync();
                            issue_s(1, buf, ks0);
                            if (leader) umma_commit(bar_ke + 8 * ks0);
                        }
                    }
                    if (!ok) break;
                    if (leader) {
                        umma_commit(bar_ve + 8 * vs);
                        if (more) umma_commit(bar_ke + 8 * ks);
                    }
                    if (++vs == ST) vs = 0, vph ^= 1;
                    if (more && ++ks == ST) ks = 0, kph ^= 1;
                }
#pragma unroll
                for (int gr = 0; gr < 2; ++gr) {
                    const int n = gr ? n1 : n0;
                    tiles[gr] += n;
                    items[gr] += n > 0 ? 1 : 0;
                }
            }
            // after the last item, or a wait that ran out: this warp's own MMAs
            if (leader) umma_commit(bar_drain);
            warp_wait(bar_drain, 0u, p.status);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        // ============================== softmax ==============================
        const int gr = warp >> 2, tr = tid & (kRows - 1);    // row tile, row in it
        const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_s = t_lane + C::kColS + gr * kKeys, t_p = t_lane + C::kColP + gr * C::kStepP, t_o = t_lane + C::kColO + gr * D;
        const float sl2 = p.scale_log2;
        auto wait_o = [&](int tt) { return warp_wait(bar_o(gr), (uint32_t)(tt & 1), p.status); };
        // a piece's state: in the CTA's first place if it continues an item, in the second if it begins one
        auto part_row = [&](const Item& w) {
            return ((size_t)blockIdx.x * 2 + (w.t0 == 0 ? 1 : 0)) * kItemRows + gr * kRows + tr;
        };
        constexpr int kRowStep = kRows / kCh;
        auto load_q = [&](const Item& w, int buf) {
            const uint32_t qbuf = s_q + (2 * buf + gr) * C::kQBytes;
            const int tok_step = kRowStep / G, g_step = kRowStep - tok_step * G;
            const int ch = tr % kCh;
            int row = tr / kCh, R = w.r0 + gr * kRows + row, tok = R / G, gq = R - tok * G;
#pragma unroll 4
            for (int j = 0; j < kRows / kRowStep; ++j) {
                const bool live = R < w.rows;
                const uint16_t* src =
                    p.q + (((size_t)(w.q0 + (live ? tok : 0)) * Hq + (size_t)w.kvh * G + (live ? gq : 0)) * D + ch * 8);
                cp_async16(qbuf + sw128<kRows>(row, ch), src, live);
                row += kRowStep;
                R += kRowStep;
                tok += tok_step;
                gq += g_step;
                if (gq >= G) {
                    gq -= G;
                    ++tok;
                }
            }
        };
        auto publish_q = [&](int buf) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_q(buf, gr));
        };
        W walk(p, n_items, false);
        auto next_item = [&](Item& w) {                      // the CTA's next item with rows for this group
            for (int st; (st = walk.next(p, n_items, w, false));) {
                if (st == 1 && (gr ? w.nt[1] : w.nt[0]) > 0) return true;
                const int R = w.r0 + gr * kRows + tr;
                if (kSplit && st == 1 && w.piece)            // only tiles behind this row tile's last
                    p.part_lse[part_row(w)] = -FLT_MAX;
                if (!kCausal && st == 2 && R < w.rows) {     // nothing to attend to: a zero row
                    const int tok = R / G;
                    uint4* o = reinterpret_cast<uint4*>(
                        p.out + ((size_t)(w.q0 + tok) * Hq + (size_t)w.kvh * G + (R - tok * G)) * D);
#pragma unroll
                    for (int c = 0; c < kCh; ++c) o[c] = make_uint4(0, 0, 0, 0);
                }
            }
            return false;
        };
        Item it, nx;
        bool has = next_item(it), failed = false;
        if (has) {
            load_q(it, 0);
            publish_q(0);
        }
        int tt = 0, k = 0;                                   // tiles and items so far
        while (has && !failed) {
            const bool has_nx = next_item(nx);
            if (QB == 2 && has_nx) load_q(nx, (k + 1) & 1);
            const int R = it.r0 + gr * kRows + tr, L = it.L, nt = gr ? it.nt[1] : it.nt[0];
            const int pos = kCausal && R < it.rows ? L - it.Tq + R / G : L - 1;   // padded rows: computed, not written
            const int pos_first = kCausal ? L - it.Tq + (it.r0 + gr * kRows) / G : L - 1;
            // finite from the start: a piece may begin behind a row's last key (weights 2^-inf = 0, not NaN)
            float m_run = kSplit ? -FLT_MAX : -INFINITY, l_run = 0.f;
            for (int t = 0; t < nt; ++t, ++tt) {
                if (!warp_wait(bar_s(gr), (uint32_t)(tt & 1), p.status)) {
                    failed = true;
                    break;
                }
                tc_fence_after_sync();
                // one Q buffer: the item's last scores are there, so the next item's rows may come
                if (QB == 1 && has_nx && t == nt - 1) load_q(nx, 0);
                const int k0 = (it.t0 + t) * kKeys;
                const bool diag = k0 + kKeys - 1 > pos_first;   // a tile on the diagonal, or the last: mask
                uint32_t sr[64];
                auto mask = [&](int from) {
                    if (diag) {
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (k0 + from + j > pos) sr[j] = __float_as_uint(-INFINITY);
                    }
                };
                // the row max over four independent chains of three-input maxima
                float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    tmem_ld64(t_s + half * 64, sr);
                    mask(half * 64);
#pragma unroll
                    for (int j = 0; j < 64; j += 2)
                        mq[(j >> 1) & 3] = fmax3(mq[(j >> 1) & 3], __uint_as_float(sr[j]), __uint_as_float(sr[j + 1]));
                }
                const float mx = fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3]));
                // finite: key 0 is in every row's range (pieces: above)
                const float m_new = fmaxf(m_run, fmaf(mx, sl2, -kHeadLog2<kE2m1>));
                if (t == 0) {
                    m_run = m_new;
                } else {
                    const bool need = m_new > m_run + kRescaleLog2;
                    if (__any_sync(0xffffffffu, need)) {
                        if (!wait_o(tt - 1)) {               // O holds the previous tile in full
                            failed = true;
                            break;
                        }
                        tc_fence_after_sync();
                        const float a = need ? fast_exp2(m_run - m_new) : 1.f;
#pragma unroll
                        for (int h = 0; h < D / 32; ++h) tmem_scale32(t_o + h * 32, a);
                        if (need) {
                            l_run *= a;
                            m_run = m_new;
                        }
                    }
                }
                // p = 2^(s sl2 - m), the second half of the keys first (it is in registers, and its
                // P lies over its own S); then the first half again, whose P lies over the second's S
                const uint64_t sc2 = f2(sl2, sl2), nm2 = f2(-m_run, -m_run);
                uint64_t rs2[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
                for (int half = 1; half >= 0; --half) {
                    if (half == 0) {
                        tmem_ld64(t_s, sr);
                        mask(0);
                    }
                    uint32_t pk[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        float x0, x1;
                        f2_split(f2_fma(f2(__uint_as_float(sr[2 * j]), __uint_as_float(sr[2 * j + 1])), sc2, nm2), x0, x1);
                        const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                        rs2[j & 1] = f2_add(rs2[j & 1], f2(p0, p1));
                        pk[j] = pack_p<kE2m1>(p0, p1);
                    }
                    // P's own columns: once the products of the previous tile have read them
                    if (!C::kOverS && half == 1 && t > 0 && !wait_o(tt - 1)) {
                        failed = true;
                        break;
                    }
                    tmem_st32(t_p + half * 32, pk);
                }
                if (failed) break;
                float r0a, r0b, r1a, r1b;
                f2_split(rs2[0], r0a, r0b);
                f2_split(rs2[1], r1a, r1b);
                l_run += (r0a + r1a) + (r0b + r1b);
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_p(gr));
            }
            if (failed || !wait_o(tt - 1)) {
                failed = true;
                break;
            }
            tc_fence_after_sync();
            const int tok = R / G, gq = R - tok * G;
            const float inv = kSplit && l_run == 0.f ? 0.f : 1.f / l_run;
            const size_t part = part_row(it);
            if (kSplit && it.piece) p.part_lse[part] = l_run == 0.f ? -FLT_MAX : m_run + __log2f(l_run);
            uint16_t* out = p.out + ((size_t)(it.q0 + tok) * Hq + (size_t)it.kvh * G + gq) * D;
#pragma unroll
            for (int h = 0; h < D / 32; ++h) {
                uint32_t o[32];
                tmem_ld32(t_o + h * 32, o);                  // warp-wide: padded rows join the load
                // V's scale only after the division: a small one over a long context's sum is no float
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    uint64_t y = f2_mul(f2(__uint_as_float(o[j]), __uint_as_float(o[j + 1])), f2(inv, inv));
                    if (kE2m1) y = f2_mul(y, f2(p.out_scale, p.out_scale));
                    float lo, hi;
                    f2_split(y, lo, hi);
                    o[j] = __float_as_uint(lo), o[j + 1] = __float_as_uint(hi);
                }
                if (kSplit && it.piece) {
                    float4* po = part_dims<D>(p.part_o, part) + h * 8 * kRows;   // a warp's rows side by side
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        po[c * kRows] = make_float4(__uint_as_float(o[4 * c]), __uint_as_float(o[4 * c + 1]),
                                                    __uint_as_float(o[4 * c + 2]), __uint_as_float(o[4 * c + 3]));
                } else if (R < it.rows) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint4 w;
                        w.x = pack_bf16x2(__uint_as_float(o[8 * c + 0]), __uint_as_float(o[8 * c + 1]));
                        w.y = pack_bf16x2(__uint_as_float(o[8 * c + 2]), __uint_as_float(o[8 * c + 3]));
                        w.z = pack_bf16x2(__uint_as_float(o[8 * c + 4]), __uint_as_float(o[8 * c + 5]));
                        w.w = pack_bf16x2(__uint_as_float(o[8 * c + 6]), __uint_as_float(o[8 * c + 7]));
                        *reinterpret_cast<uint4*>(out + h * 32 + 8 * c) = w;
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_of(gr));
            if (has_nx) publish_q((k + 1) % QB);
            ++k;
            it = nx;
            has = has_nx;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");     // nothing left in flight at exit
    }
    // every role is done
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// The pieces of a cut item, joined: M = max lse, w = 2^(lse - M), out = sum w o / sum w.  CTA (x, y): some
// rows of the item that CTA x + 1 was the second to hold some of, if there is one; a warp: 8 rows, 16 dims.
constexpr int kMergeThreads = 512;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) wide_merge_kernel(const PrefillParams p) {
    constexpr int kLanes = D / 4, kMergeRows = kMergeThreads / kLanes;
    wait_prerequisite();
    const int i = blockIdx.x + 1;
    const int4 cut = p.cuts[i];
    const int pieces = cut.x, b = cut.y, kvh = cut.z;
    if (pieces < 2) return;
    constexpr int kQuads = D / 16;                           // 16-dim columns of warps
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.y * kMergeRows + warp / kQuads * 8 + (lane >> 2), d4 = warp % kQuads * 4 + (lane & 3);
    const int R = cut.w + row, q0 = p.cu_q[b], Tq = p.cu_q[b + 1] - q0;
    if (R >= Tq * p.group) return;
    float M = -FLT_MAX, W = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < pieces; ++k) {
        const size_t part = (size_t)(k == 0 ? 2 * i - 1 : 2 * (i - 1 + k)) * kItemRows + row;
        const float lse = p.part_lse[part];
        if (lse == -FLT_MAX) continue;                       // nothing of it for this row
        const float4 o = part_dims<D>(p.part_o, part)[d4 * kRows];
        const float mn = fmaxf(M, lse), a = fast_exp2(M - mn), w = fast_exp2(lse - mn);
        M = mn;
        W = W * a + w;
        acc.x = acc.x * a + w * o.x;
        acc.y = acc.y * a + w * o.y;
        acc.z = acc.z * a + w * o.z;
        acc.w = acc.w * a + w * o.w;
    }
    const float inv = 1.f / W;
    const int tok = R / p.group;
    *reinterpret_cast<uint2*>(p.out + ((size_t)(q0 + tok) * p.num_q_heads + (size_t)kvh * p.group + (R - tok * p.group)) * D + d4 * 4) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn wide_encode_tiled() {
    static std::atomic<EncodeTiledFn> fn{nullptr};
    EncodeTiledFn f = fn.load(std::memory_order_acquire);
    if (!f) {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            f = reinterpret_cast<EncodeTiledFn>(ptr);
            fn.store(f, std::memory_order_release);
        }
    }
    return f;
}

// The pool as a 3-D bf16 tensor [blocks * Hkv][block_size][head_dim]; box = 64 dims x
// min(block_size, 64) tokens x 1, in 128-byte-swizzled rows.
bool wide_pool_map(CUtensorMap* map, const void* base, const PrefillParams& p) {
    EncodeTiledFn fn = wide_encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)p.head_dim, (cuuint64_t)p.block_size,
                                (cuuint64_t)p.num_blocks * p.num_kv_heads};
    const cuuint64_t strides[2] = {(cuuint64_t)p.head_dim * 2, (cuuint64_t)p.block_size * p.head_dim * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)(p.block_size < 64 ? p.block_size : 64), 1u};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kE2m1, bool kCausal, bool kSplit>
cudaError_t launch_wide(const PrefillParams& p, int max_q_len, cudaStream_t stream) {
    constexpr size_t smem = PCfg<D>::kSmem;
    const auto kernel = prefill_wide_kernel<D, kE2m1, kCausal, kSplit>;
    static std::atomic<uint64_t> attr_set{0};               // one bit per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!(attr_set.load(std::memory_order_acquire) & (1ull << dev))) {
        cudaFuncAttributes fa;                              // the register shares count on the launch's number
        if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || fa.numRegs != kLaunchRegs)
            return cudaErrorInvalidConfiguration;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        attr_set.fetch_or(1ull << dev, std::memory_order_acq_rel);
    }
    int sms = 0;
    if (num_sms_current_device(&sms) != PA_OK || sms <= 0) return cudaErrorInvalidDevice;
    const long long tiles = ((long long)max_q_len * p.group + kItemRows - 1) / kItemRows;
    const long long items = (long long)p.num_seqs * p.num_kv_heads * tiles;
    if (items <= 0) return cudaSuccess;
    CUtensorMap km, vm;
    memset(&km, 0, sizeof km);
    memset(&vm, 0, sizeof vm);
    if (!kE2m1 && (!wide_pool_map(&km, p.k_cache, p) || !wide_pool_map(&vm, p.v_cache, p))) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(kSplit ? sms : std::min<long long>(items, sms));
    kernel<<<grid, kThreads, smem, stream>>>(p, km, vm);
    const cudaError_t e = cudaGetLastError();
    if constexpr (!kSplit) {
        return e;
    } else {
        if (e != cudaSuccess || grid < 2) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(grid - 1, kItemRows * (D / 4) / kMergeThreads);
        cfg.blockDim = dim3(kMergeThreads);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, wide_merge_kernel<D>, p);
    }
}

}  // namespace

// Whether the last round's items of a 4-bit prefill are cut, as far as the call's bounds tell: the tiles that
// it would take whole, less those of an even share, against the pieces' way through memory and the merge.
// Measured (us, cut | whole; tiles saved), the last rows of contexts of the given length: 32 and 8 heads of 64,
// 300 of 20000 tokens 111 | 300 (115), 512 of 3000 48 | 53 (14), 4 x 256 of 4000 92 | 68 (4), 4000 of 4000
// 155 | 125 (2); 64 and 8 heads of 128, where the cut's registers are taken from the softmax's, 300 of 20000
// 286 | 373 (72), 1021 of 15000 575 | 585 (32), 4 x 256 of 4000 202 | 175 (9).
int wide_split_ctas(int32_t num_seqs, int32_t num_kv_heads, int32_t group, int32_t head_dim, int32_t max_q_len,
                    int64_t max_len) {
    int sms = 0;
    if (num_sms_current_device(&sms) != PA_OK || sms < 2 || num_seqs < 1 || max_q_len < 1) return 0;
    const int64_t nsh = (int64_t)num_seqs * num_kv_heads, rows = (int64_t)max_q_len * group;
    const int64_t items = nsh * ((rows + kItemRows - 1) / kItemRows), last = items % sms;
    // row tiles of a sequence that come before those of the last round end behind them
    const int64_t seen = max_len - (items - last) / nsh * kItemRows / group;
    const int64_t nt = seen > 0 ? (seen + kKeys - 1) / kKeys : 0;
    const bool cut = last > 0 && items / sms < INT32_MAX && nt * (sms - last) >= wide_split_tiles(head_dim) * sms;
    return cut ? sms : 0;
}
size_t wide_split_rows(int ctas) { return (size_t)ctas * 2 * kItemRows; }

cudaError_t launch_prefill_e2m1(const PrefillParams& p, int max_q_len, cudaStream_t stream) {
    if (p.head_dim == 64)
        return p.cuts ? launch_wide<64, true, true, true>(p, max_q_len, stream)
                      : launch_wide<64, true, true, false>(p, max_q_len, stream);
    if (p.head_dim == 128)
        return p.cuts ? launch_wide<128, true, true, true>(p, max_q_len, stream)
                      : launch_wide<128, true, true, false>(p, max_q_len, stream);
    return cudaErrorInvalidValue;
}

// Cross attention.  With 128 dims these tiles; with 64 dims those of prefill_ws.cu, two CTAs an SM of
// 128 rows each.  Measured (us, these | prefill_ws.cu), 16 heads: 8 x 448 rows over 1500 tokens, 128
// dims 71 | 122, 64 dims 59 | 55; 32 x 100 over 500, 128 dims 50 | 52, 64 dims 42 | 25; 32 and 8 heads,
// 4 x 1024 over 4096, 128 dims 298 (922 TFLOP/s) | 505, 64 dims 264 | 241.  A call of few items
// (p.cuts) goes to the stream of key tiles there.
cudaError_t launch_cross(const PrefillParams& p, int max_q_len, cudaStream_t stream) {
    if (p.head_dim == 128 && !p.cuts) return launch_wide<128, false, false, false>(p, max_q_len, stream);
    return launch_cross_ws(p, max_q_len, stream);
}

}  // namespace pa
