// Prefill over the block-scaled 8-bit pool (dattn_prefill with DATTN_KV_FP8_BLOCK): a chunk of Tq
// new query tokens per request attends the paged cache, causally or block-sparsely, exactly as over
// the bf16 pool (prefill.cu holds the method's sources and the block rules).
//
// Arithmetic. An E4M3 code is an fp16 number, so the codes are widened to fp16 in shared memory
// (one conversion for two codes) and both products run in fp16 with fp32 accumulation. The query
// row is scaled by a power of two 2^a that brings its largest element to [2^14, 2^15) and rounded
// to fp16: exact for every element within 2^28 of the largest. The K scale of a 16-key tile
// multiplies its scores; the V scale, a power of two, goes into the exponent of its weights,
// w = 2^(s - m + log2(scale) - x). The reference m + x is the row's own: it follows the largest
// s + log2(scale) of the keys that the row sees and whose V is not all zeros (w = 2^9 when it is set;
// raised, and the row's accumulator rescaled, when a key exceeds 2^15), so that a V scale which the
// row does not see, or whose keys weigh nothing in it, takes no bits from the others. w enters the
// product as two fp16 terms: 22 bits together, and to 2^-33 of the largest w where it is small.
// The tensor cores add into their fp32 accumulators rounding towards zero, which over a long
// context shrinks the result (5.6e-5 after 4096 products of a 32K context), so a row's accumulator is
// emptied into its output row every kPbWindow key blocks, by fp32 additions.
//
// What bounds it: the tensor cores, then the softmax's latency. A 64-key block of 128 query rows
// takes one product S = Q K^T and two products O += P V, 3 x 2 x 128 x 64 x d operations for the
// 2 x 2 x 128 x 64 x d that count: 2/3 of the dense 16-bit rate at most. Measured: a causal prompt of
// 32K tokens, 32 query and 8 KV heads of 128, 9.45 ms (933 TFLOP/s counted, 0.48 of the bf16 rate);
// without the softmax's arithmetic 6.94 ms. A key block is widened once for 256 query rows: one CTA
// per SM holds two tiles of 128 rows, which work past each other.
//
// A CTA: 256 rows as four quarters of 64 tokens: one query block of four heads of a KV head (g a
// multiple of 4), two query blocks of two heads (even g), or four query blocks of one head. A tile
// (two quarters) takes part in a key block only if one of its quarters keeps it. Where the last
// wave of CTAs would fill less than half of the SMs, its tiles get a CTA each. A chunk of few tiles
// (its blocks run one after another, 0.8-1.1 us each) gives each tile a cluster of up to eight CTAs,
// which share its key blocks and join their sums through shared memory: 64 tokens of 32 heads over 8
// KV heads of 128 after 32K tokens 562 -> 143 us (clusters of 4), 64 of 8 heads over one KV head after
// 100K tokens 1593 -> 211 us (8), 39 of 16 heads after 1284 21.6 -> 17.2 us. 15 warps:
//   0-3, 4-7  one query row per thread of tile 0, 1: the softmax. (Two threads per row took 11% longer:
//             the second's share of the fixed work costs more than its latency saves.)
//   8-11      load codes, widen them and write the K and V stages in the 128-byte-swizzled layout
//             of the MMA operands;
//   12, 13    one thread each issues the products of tile 0, 1: S of the next key block, then P V of
//             this one. (One issuing warp for both tiles made them wait for each other: 12.4 ms.)
//   14        walks the key blocks, eight at a time, one lane per 16-key tile, and leaves each
//             block's place, lengths and scales in a ring in shared memory for the others.
// Tensor memory: O of the two tiles, then two score buffers for each, all 512 columns.
#include <atomic>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "prefill.cuh"

namespace dattn {

namespace {

constexpr int kPbRows = 256;                // query rows of a CTA: two tiles of 128
constexpr int kPbConvWarp = 8;              // warps 8-11 widen the codes
constexpr int kPbConvThreads = 128;
constexpr int kPbMmaWarp = 12;              // warps 12, 13 issue the products of tile 0, 1
constexpr int kPbPlaceWarp = 14;            // the places of the key blocks
constexpr int kPbThreads = 15 * 32;
constexpr int kPbStages = 3;                // K stages, and V stages
constexpr int kPbGroup = 8;                 // key blocks that warp 14 resolves at once
constexpr int kPbRing = 2 * kPbGroup;       // the blocks' ring
// Key blocks between two emptyings of an accumulator: 256 products that each lose up to 2^-24 of the
// sum, 4.3e-6 of the result measured after 28K tokens. (16: 2.2e-6 for 11% more time on a 32K prompt.)
constexpr int kPbWindow = 32;
// Key blocks of a CTA at least, where a cluster shares a tile. With 2, 3 and 4: 17.6, 14.3 and 14.2 us
// for 4 x 75 tokens after 90-700 (d = 64), 17.2, 17.2 and 19.5 for 39 after 1284, 10.9, 12.6 and 12.6
// for 9 after 882.
constexpr int kPbSplitBlocks = 3;
// A row's reference m + x (log2 units): its largest weight is 2^kPbTop when the reference is set, and a
// weight above 2^kPbMost sets it anew (both terms are fp16: below 2^16). With 12 more keys set it anew:
// 4096 tokens after 28K took 2580 us, 2405 with 9.
constexpr float kPbTop = 9.f, kPbMost = 15.f;
constexpr uint32_t kPbCols = 512;           // O: [0, 128), [128, 256); S: 256 + 128 tile + 64 buffer

// mbarriers
constexpr int kBarKFull = 0, kBarKEmpty = 3, kBarVFull = 6, kBarVEmpty = 9;
constexpr int kBarS = 12, kBarP = 16;       // + 2 tile + buffer
constexpr int kBarPv = 20;                  // + tile
constexpr int kBarRingFull = 22, kBarRingEmpty = 24, kBarDrain = 26, kPbBars = 28;
constexpr int kRingReaders = 14;            // warps 0-13

// A key block in the ring: its 16-key tiles as the widening reads them (place in the pool, in tiles,
// and tokens) and as the softmax does (K scale, -, log2 of the V scale, 1 / V scale; kPbNoScale and 1
// for a scale of 0), its index, the quarters of rows that keep it (bits 0-3; bit 4: all its keys are
// written), and the smallest and largest log2 of a V scale of its written tiles.
struct __align__(16) PbBlock {
    int2 rows[kPfTiles];
    float4 scale[kPfTiles];
    int32_t kb, act;
    float low, high;
};
constexpr float kPbNoScale = -1000.f;
constexpr int32_t kPbFull = 16;
// the tiles (bits) of the quarters that keep a block
__device__ __forceinline__ uint32_t tiles_of(uint32_t act) {
    return ((act & 3u) ? 1u : 0u) | ((act & 12u) ? 2u : 0u);
}

struct PbSmem {
    uint32_t q, blk_bytes, kst, vst, bm, ring, bars, taddr, abort, qscale, total;
};

__host__ __device__ inline PbSmem pb_smem_layout(int D, int nq, int nwords) {
    PbSmem s;
    uint32_t o = 0;
    s.q = o;           o += (uint32_t)kPbRows * D * 2u;
    s.blk_bytes = 64u * D * 2u;
    s.kst = o;         o += kPbStages * s.blk_bytes;
    s.vst = o;         o += kPbStages * s.blk_bytes;
    s.ring = o;        o += kPbRing * (uint32_t)sizeof(PbBlock);
    s.bars = o;        o += (kPbBars + 1) * 8u;
    s.taddr = o;       o += 16u;
    s.abort = o;       o += 16u;
    s.qscale = o;      o += kPbRows * 4u;
    s.bm = o;          o += (uint32_t)(nq * nwords) * 4u;
    s.total = o;
    return s;
}

struct PbParams {
    PfParams f;
    int32_t hp, nq;    // heads and query blocks of a CTA: hp * nq = 4
    int32_t whole;     // CTAs of two tiles; the others hold one tile each
    int32_t split;     // CTAs of a cluster, which share a tile's key blocks (1: no cluster)
    const uint8_t* k_pool;
    const uint8_t* v_pool;
    const float2* scale;  // [num_pages][Hkv][P/16] (K, V)
};

// The quarters z that keep the key blocks of word w: the bitmaps of the CTA's query blocks are
// bm[i][nwords]; a quarter outside the tiles that the CTA holds (tmask) keeps none.
__device__ __forceinline__ uint32_t quarter_word(const uint32_t* bm, int nq, int nwords,
                                                 uint32_t tmask, int z, int w) {
    const int i = nq == 4 ? z : nq == 2 ? z >> 1 : 0;
    return ((tmask >> (z >> 1)) & 1u) ? bm[i * nwords + w] : 0u;
}
__device__ __forceinline__ uint32_t held_word(const uint32_t* bm, int nq, int nwords, uint32_t tmask,
                                              int w, uint32_t (&q)[4]) {
#pragma unroll
    for (int z = 0; z < 4; ++z) q[z] = quarter_word(bm, nq, nwords, tmask, z, w);
    return q[0] | q[1] | q[2] | q[3];
}

// kind::f16 with fp16 operands (tc_idesc's type fields cleared) and an fp32 accumulator
__host__ __device__ constexpr uint32_t pb_idesc(uint32_t M, uint32_t N, uint32_t b_mn) {
    return tc_idesc(M, N, b_mn) & ~((7u << 7) | (7u << 10));
}

// out[0..3] += v, at L2; the row belongs to this thread alone
__device__ __forceinline__ void red_add4(float* out, float a, float b, float c, float d) {
    asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(out), "f"(a), "f"(b), "f"(c),
                 "f"(d)
                 : "memory");
}

__device__ __forceinline__ float max16(const float* x) {
    const float a = fmax3(x[0], x[1], x[2]), b = fmax3(x[3], x[4], x[5]);
    const float c = fmax3(x[6], x[7], x[8]), d = fmax3(x[9], x[10], x[11]);
    const float e = fmax3(x[12], x[13], x[14]);
    return fmaxf(fmax3(a, b, x[15]), fmax3(c, d, e));
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }

// SPLIT: a cluster of pp.split CTAs holds one tile, each CTA a run of its key blocks; their sums and
// maxima meet in shared memory.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kPbThreads, 1)
prefill_block_kernel(const __grid_constant__ PbParams pp, int32_t nwords) {
    constexpr uint32_t kHalf = 64u * 128u;  // a 128-byte half of a key block's rows
    const PfParams& p = pp.f;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw;
    const PbSmem L = pb_smem_layout(D, pp.nq, nwords);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the 128-byte swizzle of the MMA operands needs 1024-byte alignment
    if ((smem_u32(base) & 1023u) != 0u) {
        if (tid == 0) set_err(p.dev_err, DATTN_DEVERR_SMEM_ALIGN);
        return;
    }
    // CTA -> (request b, group of kv_group KV heads, tile pair J, KV head of the group, head slot):
    // a group's pairs run together, its last (longest) first. CTAs from `whole` on hold one tile.
    const int hp = pp.hp, nq = pp.nq;
    const int32_t spk = p.g / hp;
    const int32_t ngrp = p.Hkv / p.kv_group;
    const int32_t cta = SPLIT ? (int32_t)blockIdx.x / pp.split : (int32_t)blockIdx.x;
    const int32_t rank = SPLIT ? (int32_t)cluster_rank() : 0;
    const int32_t extra = max(cta - pp.whole, 0);
    const uint32_t tmask = cta < pp.whole ? 3u : 1u << (extra & 1);
    int32_t c = cta < pp.whole ? cta : pp.whole + (extra >> 1);
    const int32_t sk = c % spk;
    c /= spk;
    const int32_t hg = c % p.kv_group;
    c /= p.kv_group;
    const int32_t J = p.nqb - 1 - c % p.nqb;
    c /= p.nqb;
    const int32_t kvh = (c % ngrp) * p.kv_group + hg;
    const int32_t b = c / ngrp;
    const int32_t h0 = kvh * p.g + sk * hp;  // the CTA's first query head
    const uint32_t bars = smem_u32(base + L.bars);
    auto bar = [&](int i) { return bars + 8u * i; };
    PbBlock* ring = reinterpret_cast<PbBlock*>(base + L.ring);
    uint32_t* bm = reinterpret_cast<uint32_t*>(base + L.bm);
    // SPLIT: the tile's sums (rows of D + 4 floats, for the banks) and (m_used, xref, l, m_true) of its
    // rows, where the K and V stages were
    float* part = reinterpret_cast<float*>(base + L.kst);
    float4* stat = reinterpret_cast<float4*>(part + 128 * (D + 4));
    static_assert(128 * (D + 4) * 4 + 128 * 16 <= 2 * kPbStages * 64 * D * 2, "the parts' place");
    float* qscale = reinterpret_cast<float*>(base + L.qscale);
    volatile int* abort_p = reinterpret_cast<volatile int*>(base + L.abort);
    if (tid == 0) {
        for (int s = 0; s < kPbStages; ++s) {
            mbar_init(bar(kBarKFull + s), kPbConvThreads);
            mbar_init(bar(kBarKEmpty + s), 2);
            mbar_init(bar(kBarVFull + s), kPbConvThreads);
            mbar_init(bar(kBarVEmpty + s), 2);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(kBarS + i), 1);
            mbar_init(bar(kBarP + i), 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kBarPv + i), 1);
            mbar_init(bar(kBarRingFull + i), 1);
            mbar_init(bar(kBarRingEmpty + i), kRingReaders);
        }
        mbar_init(bar(kBarDrain), 1);
        mbar_init(bar(kBarDrain + 1), 1);
        *abort_p = 0;
        fence_mbar_init();
    }
    __syncwarp();  // (tcgen05 and cluster-barrier instructions take whole, converged warps)
    if (warp == 0) {  // the whole warp allocates the CTA's tensor memory
        tc_alloc(smem_u32(base + L.taddr), kPbCols);
        tc_relinquish();
    }
    tc_fence_before();
    grid_dependency_wait();  // the lengths and the pool may come from the previous kernel
    grid_launch_dependents();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(base + L.taddr);

    // ---- the CTA's query rows and key blocks (uniform over the CTA) ---------------------------
    const int32_t Ln = p.seq_lens[b];
    bool active = Ln >= p.Tq && Ln <= p.max_pages * p.P;
    if (!active && tid == 0 && h0 == 0 && J == 0 && rank == 0) set_err(p.dev_err, DATTN_DEVERR_LEN_OOB);
    const int32_t c0 = Ln - p.Tq;
    const int32_t qa = (active ? c0 : 0) / kPfBlock + J * nq;  // the first query block
    int kind = p.head_kind ? p.head_kind[kvh] : DATTN_HEAD_DENSE;
    if (kind < 0 || kind > 2) kind = DATTN_HEAD_DENSE;
    // bit i: query block qa + i has rows of the chunk (and, for a retrieval head, a list)
    uint32_t has = 0u;
    for (int i = 0; i < nq && active; ++i) {
        const int32_t q0 = (qa + i) * kPfBlock;
        if (max(c0, q0) >= min(Ln, q0 + kPfBlock)) continue;
        if (kind == DATTN_HEAD_RETRIEVAL && qa + i >= p.qblock_stride) {
            if (tid == 0) set_err(p.dev_err, DATTN_DEVERR_LEN_OOB);
            continue;
        }
        has |= 1u << i;
    }
    active = active && has != 0u;
    const int32_t p_hi = min(Ln, (qa + nq) * kPfBlock);  // no row sees a later key
    const int32_t nw = active ? (qa + nq + 31) / 32 : 0;
    // quarter z (rows 64 z ..): its query block's place and its head
    auto q_block = [&](int z) { return nq == 4 ? z : nq == 2 ? z >> 1 : 0; };
    auto q_head = [&](int z) { return nq == 4 ? 0 : nq == 2 ? z & 1 : z; };
    if (active) {
        for (int32_t x = tid; x < nq * nw; x += kPbThreads) {
            const int i = x / nw, w = x - i * nw;
            const int32_t qb = qa + i;
            uint32_t a = 0u;
            if (kind != DATTN_HEAD_RETRIEVAL && ((has >> i) & 1u)) {
                for (int bit = 0; bit < 32; ++bit) {
                    const int32_t kb = 32 * w + bit;
                    const bool keep = kb <= qb && (kind == DATTN_HEAD_DENSE || kb < p.sink_blocks ||
                                                   kb > qb - p.local_blocks);
                    a |= (keep ? 1u : 0u) << bit;
                }
            }
            bm[i * nwords + w] = a;
        }
        if (kind == DATTN_HEAD_RETRIEVAL) {
            __syncthreads();
            for (int i = 0; i < nq; ++i) {
                if (!((has >> i) & 1u)) continue;
                const int32_t* row = p.block_lists +
                    (((int64_t)b * p.Hkv + kvh) * p.qblock_stride + qa + i) * p.max_sel;
                for (int32_t x = tid; x < p.max_sel; x += kPbThreads) {
                    const int32_t kb = __ldg(row + x);
                    if (kb >= 0 && kb <= qa + i) atomicOr(bm + i * nwords + (kb >> 5), 1u << (kb & 31));
                }
            }
        }
        // The query rows as fp16, [half][256 rows][128 B] swizzled, each scaled by its 2^a; with a
        // negative scale they are negated (exact), so that the scores scale by |scale|. A row's
        // D/8 threads are neighbours, and the loop's last round is whole warps.
        constexpr int TPR = D / 8;
        const uint32_t qneg = p.sl2 < 0.f ? 0x80008000u : 0u;
        for (int idx = tid; idx < kPbRows * TPR; idx += kPbThreads) {
            const int r = idx / TPR, ch = idx - r * TPR, z = r >> 6;
            const int32_t pos = (qa + q_block(z)) * kPfBlock + (r & 63);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (((has >> q_block(z)) & 1u) && pos >= c0 && pos < Ln)
                v = __ldg(reinterpret_cast<const uint4*>(
                    p.q + (((int64_t)b * p.Tq + (pos - c0)) * p.Hq + h0 + q_head(z)) * D) + ch);
            float mx = absmax8(v);
#pragma unroll
            for (int off = 1; off < TPR; off <<= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            int a = 0;
            if (mx > 0.f) a = min(127, max(-113, 14 - ((__float_as_int(mx) >> 23) - 127)));
            const float up = __int_as_float((127 + a) << 23);
            uint32_t w[4] = {v.x ^ qneg, v.y ^ qneg, v.z ^ qneg, v.w ^ qneg};
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_f16(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up);
            *reinterpret_cast<uint4*>(base + L.q + (ch >> 3) * (kPbRows * 128u) +
                                      swz128((uint32_t)r, (uint32_t)(ch & 7))) =
                make_uint4(w[0], w[1], w[2], w[3]);
            // 2^-a |scale| log2(e)
            if (ch == 0)
                qscale[r] = fabsf(p.sl2) *
                            (a < 127 ? __int_as_float((127 - a) << 23) : 5.877471754e-39f);
        }
        fence_proxy_async_smem();  // the tensor cores read these rows through the async proxy
    }
    __syncthreads();
    int32_t n = 0;  // key blocks that some row of the CTA keeps
    for (int32_t w = 0; w < nw; ++w) {
        uint32_t q[4];
        n += __popc(held_word(bm, nq, nwords, tmask, w, q));
    }
    // the CTA's run of them: [first, first + n)
    int32_t first_block = 0, use = 1;
    if constexpr (SPLIT) {
        use = max(1, min(pp.split, n / kPbSplitBlocks));
        const int32_t all = n;
        first_block = rank < use ? all * rank / use : all;
        n = rank < use ? all * (rank + 1) / use - first_block : 0;
    }
    // The ring: block i in slot i % 16, ready with its group of eight; a reader's warp gives a group
    // back after its last block.
    auto wait = [&](uint32_t bar_addr, uint32_t parity) {  // by a whole warp, one answer
        return __all_sync(0xffffffffu, mbar_wait(bar_addr, parity, abort_p, p.dev_err)) != 0;
    };
    auto ring_ready = [&](int32_t i) {
        return (i & (kPbGroup - 1)) != 0 ||
               wait(bar(kBarRingFull) + 8u * ((i / kPbGroup) & 1), (i / kPbRing) & 1);
    };
    auto ring_release = [&](int32_t i) {
        __syncwarp();
        if ((i & (kPbGroup - 1)) == kPbGroup - 1 && lane == 0)
            mbar_arrive(bar(kBarRingEmpty) + 8u * ((i / kPbGroup) & 1));
    };

    if (active && warp == kPbPlaceWarp) {
        // ---------------------------------------------------------------- places of the key blocks
        const int blk = lane >> 2, u = lane & 3;  // this lane: tile u of the group's block blk
        int32_t w = 0;
        uint32_t q[4], word = held_word(bm, nq, nwords, tmask, 0, q);
        if constexpr (SPLIT) {  // past the blocks of the CTAs before
            int32_t skip = first_block;
            while (n > 0 && skip >= __popc(word)) {  // (n > 0: more than skip blocks in all)
                skip -= __popc(word);
                word = held_word(bm, nq, nwords, tmask, ++w, q);
            }
            for (; n > 0 && skip > 0; --skip) word &= word - 1u;
        }
        bool ok = true;
        for (int32_t i = 0; i < n && ok; i += kPbGroup) {
            const int32_t cnt = min(kPbGroup, n - i);
            int32_t kb = 0, act = 0;
            for (int x = 0; x < cnt; ++x) {
                while (word == 0u && w + 1 < nw) word = held_word(bm, nq, nwords, tmask, ++w, q);
                const int bit = __ffs(word) - 1;
                if (x == blk) {
                    kb = 32 * w + bit;
                    act = ((q[0] >> bit) & 1u) | (((q[1] >> bit) & 1u) << 1) |
                          (((q[2] >> bit) & 1u) << 2) | (((q[3] >> bit) & 1u) << 3);
                }
                word &= word - 1u;
            }
            const int32_t t0 = kb * kPfBlock + 16 * u;
            int32_t y = 0, hi = 0;
            float2 sc = make_float2(0.f, 0.f);
            if (blk < cnt && t0 < p_hi) {
                const int32_t lp = t0 / p.P;
                const int32_t page = __ldg(p.block_table + (int64_t)b * p.max_pages + lp);
                if (page < 0) {
                    set_err(p.dev_err, DATTN_DEVERR_UNMAPPED_PAGE);
                } else if (page >= p.num_pages) {
                    set_err(p.dev_err, DATTN_DEVERR_PAGE_OOB);
                } else {
                    y = (page * p.Hkv + kvh) * p.P + (t0 - lp * p.P);
                    hi = min(16, Ln - t0);
                    sc = __ldg(pp.scale + (y >> 4));
                }
            }
            const int ve = (__float_as_int(sc.y) >> 23) - 127;
            float high = sc.y > 0.f ? (float)ve : kPbNoScale;
            float low = hi > 0 ? high : -kPbNoScale;
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, 1));
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, 2));
            high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, 1));
            high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, 2));
            int full = hi == 16 ? 1 : 0;
            full &= __shfl_xor_sync(0xffffffffu, full, 1);
            full &= __shfl_xor_sync(0xffffffffu, full, 2);
            if (i >= kPbRing)
                ok = wait(bar(kBarRingEmpty) + 8u * ((i / kPbGroup) & 1), ((i / kPbRing) - 1) & 1);
            if (ok && blk < cnt) {
                PbBlock& to = ring[(i + blk) & (kPbRing - 1)];
                to.rows[u] = make_int2(y >> 4, hi);
                to.scale[u] = sc.y > 0.f ? make_float4(sc.x, 0.f, (float)ve, pow2i(-ve))
                                         : make_float4(sc.x, 0.f, kPbNoScale, 1.f);
                if (u == 0) {
                    to.kb = kb;
                    to.act = act | (full ? kPbFull : 0);
                    to.low = low;
                    to.high = high;
                }
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(bar(kBarRingFull) + 8u * ((i / kPbGroup) & 1));
        }
    } else if (active && warp >= kPbConvWarp && warp < kPbMmaWarp) {
        // ------------------------------------------------------ widening: codes -> K and V stages
        // A row of D codes is D/16 threads of 16 codes; a pass takes RP rows, NP passes a block.
        // Eight neighbours store to two rows of one half: all banks.
        constexpr int CPR = D / 16, RP = kPbConvThreads / CPR, NP = 64 / RP;
        const int ct = tid - kPbConvWarp * 32;
        const int c16 = D == 64 ? ct & 3 : (ct & 3) | ((ct >> 1) & 4);
        const int rr = D == 64 ? ct >> 2 : ((ct >> 2) & 1) | ((ct >> 4) << 1);
        uint4 kv[NP], vv[NP];
        // 16 codes a row of block x; rows that hold no token of the request are zeros. A thread's rows
        // have one place in their tiles, (rr & 15).
        const int64_t mine = (rr & 15) * D + 16 * c16;
        auto load = [&](const uint8_t* pool, int32_t x, uint4 (&v)[NP]) {
            const PbBlock& blk = ring[x & (kPbRing - 1)];
            const uint8_t* from = pool + mine;
            if (blk.act & kPbFull) {
#pragma unroll
                for (int k = 0; k < NP; ++k)
                    v[k] = __ldg(reinterpret_cast<const uint4*>(
                        from + (int64_t)blk.rows[(rr + RP * k) >> 4].x * (16 * D)));
                return;
            }
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int2 at = blk.rows[(rr + RP * k) >> 4];
                v[k] = make_uint4(0u, 0u, 0u, 0u);
                if ((rr & 15) < at.y)
                    v[k] = __ldg(reinterpret_cast<const uint4*>(from + (int64_t)at.x * (16 * D)));
            }
        };
        const uint32_t half = (c16 >> 2) * kHalf, ch = 2u * (c16 & 3);
        auto store = [&](uint8_t* st, const uint4 (&v)[NP]) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const uint32_t row = (uint32_t)(rr + RP * k);
                uint4 a, c2;
                e4m3x4_to_f16(v[k].x, a.x, a.y);
                e4m3x4_to_f16(v[k].y, a.z, a.w);
                e4m3x4_to_f16(v[k].z, c2.x, c2.y);
                e4m3x4_to_f16(v[k].w, c2.z, c2.w);
                *reinterpret_cast<uint4*>(st + half + swz128(row, ch)) = a;
                *reinterpret_cast<uint4*>(st + half + swz128(row, ch + 1u)) = c2;
            }
        };
        bool ok = n > 0 && ring_ready(0);
        if (ok) {
            load(pp.k_pool, 0, kv);
            load(pp.v_pool, 0, vv);
        }
        for (int32_t i = 0; i < n && ok; ++i) {
            const int s = i % kPbStages, ph = (i / kPbStages) & 1;
            const bool more = i + 1 < n;
            if (i >= kPbStages) ok = wait(bar(kBarKEmpty + s), ph ^ 1);
            if (!ok) break;
            store(base + L.kst + (uint32_t)s * L.blk_bytes, kv);
            fence_proxy_async_smem();
            mbar_arrive(bar(kBarKFull + s));
            ring_release(i);  // (its V is in registers, or on its way)
            // the next block's K is on its way while this block's V is widened
            if (more) {
                ok = ring_ready(i + 1);
                if (!ok) break;
                load(pp.k_pool, i + 1, kv);
            }
            if (i >= kPbStages) ok = wait(bar(kBarVEmpty + s), ph ^ 1);
            if (!ok) break;
            store(base + L.vst + (uint32_t)s * L.blk_bytes, vv);
            fence_proxy_async_smem();
            mbar_arrive(bar(kBarVFull + s));
            if (more) load(pp.v_pool, i + 1, vv);
        }
    } else if (active && (warp == kPbMmaWarp || warp == kPbMmaWarp + 1)) {
        // ---------------------------------------------------------------- MMA issuers
        // A warp for each tile, so that neither tile's products wait for the other's softmax. The
        // whole warp walks the blocks and waits; one lane issues. What the products depend on comes
        // out of warp reductions: the compiler then knows it to be uniform.
        if (n > 0) {
            const uint32_t lead = elect_lane();
            constexpr uint32_t idesc_s = pb_idesc(128, 64, 0);
            constexpr uint32_t idesc_o = pb_idesc(128, D, 1);
            const uint32_t t = __reduce_or_sync(0xffffffffu, (uint32_t)(warp - kPbMmaWarp));
            const uint32_t qd = desc_lo(smem_u32(base + L.q), 16u) + t * (128u * 128u >> 4);
            const uint32_t kd = desc_lo(smem_u32(base + L.kst), 16u);
            const uint32_t vd = desc_lo(smem_u32(base + L.vst), kHalf);
            const uint32_t tb = __reduce_or_sync(0xffffffffu, tbase);
            const uint32_t oc = tb + 128u * t, sc = tb + 256u + 128u * t;
            bool ok = true;
            uint32_t j = 0u;  // the tile's blocks so far
            uint32_t act = 0u, prev = 0u;
            for (int32_t i = 0; i <= n && ok; ++i) {
                prev = act;
                act = 0u;
                if (i < n) {
                    ok = ring_ready(i);
                    if (!ok) break;
                    act = (tiles_of(__reduce_or_sync(0xffffffffu,
                                                     (uint32_t)ring[i & (kPbRing - 1)].act)) >> t) & 1u;
                    ring_release(i);
                    const int s = i % kPbStages;
                    ok = wait(bar(kBarKFull + s), (i / kPbStages) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (act) {
                        // S: the tile's j'th scores into its buffer j % 2 (whose P V, of its block
                        // j - 2, was issued before: products run in order)
                        const uint32_t k_lo = kd + (uint32_t)s * (64u * D * 2u >> 4);
                        const uint32_t to = sc + 64u * (j & 1u);
                        pb_mma_ss<false>(lead, to, qd, k_lo, idesc_s);
#pragma unroll
                        for (int kk = 1; kk < D / 16; ++kk)
                            pb_mma_ss<true>(lead, to,
                                            qd + (((kk >> 2) * (kPbRows * 128u) + (kk & 3) * 32u) >> 4),
                                            k_lo + (((kk >> 2) * kHalf + (kk & 3) * 32u) >> 4), idesc_s);
                        pb_commit(lead, bar(kBarS) + 16u * t + 8u * (j & 1u));
                    }
                    pb_commit(lead, bar(kBarKEmpty + s));
                }
                if (i > 0) {
                    const int sv = (i - 1) % kPbStages;
                    ok = wait(bar(kBarVFull + sv), ((i - 1) / kPbStages) & 1);
                    if (!ok) break;
                    if (prev) {
                        // O += P V of its block before: P from tensor memory (hi terms, then lo);
                        // every kPbWindow'th block begins a new sum
                        const uint32_t jp = j - 1u;
                        ok = wait(bar(kBarP) + 16u * t + 8u * (jp & 1u), (jp >> 1) & 1u);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t v_lo = vd + (uint32_t)sv * (64u * D * 2u >> 4);
                        const uint32_t from = sc + 64u * (jp & 1u);
#pragma unroll
                        for (int part = 0; part < 2; ++part) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                pb_mma_ts(lead, oc, from + 32u * part + 8u * kk, v_lo + (kk * 2048u >> 4),
                                          idesc_o, (part > 0 || kk > 0) ? 1u : jp & (kPbWindow - 1u));
                        }
                        pb_commit(lead, bar(kBarPv) + 8u * t);
                    }
                    pb_commit(lead, bar(kBarVEmpty + sv));
                }
                j += act;
            }
            // every product is done: the epilogue's signal, and nothing of this warp's may still run
            // on the tensor cores when it exits
            pb_commit(lead, bar(kBarDrain) + 8u * t);
            mbar_wait(bar(kBarDrain) + 8u * t, 0, abort_p, p.dev_err);
        }
    } else if (active && warp < 8) {
        // ---------------------------------------------------------------- softmax threads
        const int t = warp >> 2, r = tid, z = r >> 6;  // tile, row and quarter
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ocol = tbase + lanes + 128u * t;
        const uint32_t ecol = tbase + lanes + 128u * (t ^ 1);  // SPLIT: the sums of earlier windows
        const int qi = q_block(z);
        const int32_t pos = (qa + qi) * kPfBlock + (r & 63);
        const bool rowok = ((has >> qi) & 1u) && ((tmask >> t) & 1u) && pos >= c0 && pos < Ln;
        const float frow = qscale[r];
        const int64_t row = ((int64_t)b * p.Tq + (rowok ? pos - c0 : 0)) * p.Hq + h0 + q_head(z);
        float* orow = p.out + row * D;
        float m_used = kPfNegInf, m_true = kPfNegInf, l = 0.f;  // l is relative to m_used
        // O is relative to 2^mref, mref = m_used + xref; xfac is 2^xref
        float xref = -126.f, xfac = pow2i(-126), mref = kPfNegInf;
        // what the output row holds of earlier windows is relative to 2^(ref_m + ref_x) (-inf: nothing)
        float ref_m = kPfNegInf, ref_x = 0.f;
        int32_t j = 0;  // this tile's blocks
        bool ok = true;
        for (int32_t i = 0; i < n; ++i) {
            ok = ring_ready(i);
            if (!ok) break;
            const PbBlock& blk = ring[i & (kPbRing - 1)];
            const int32_t act = blk.act, kb = blk.kb;
            if (!(act & (3 << (2 * t)))) {
                ring_release(i);
                continue;
            }
            // the tiles' score factors (at least 1e-30, so that a masked key, -inf, never meets a
            // zero factor)
            float fu[kPfTiles];
#pragma unroll
            for (int u = 0; u < kPfTiles; ++u) fu[u] = fmaxf(frow * blk.scale[u].x, 1e-30f);
            // The row's query block keeps kb; all keys pass for every row of the warp if they are
            // written and kb is an earlier block (rows without a query compute on zeros).
            const bool keep = (act >> z) & 1;
            const bool all = keep && (act & kPbFull) && kb < qa + qi;
            int32_t lim[kPfTiles];
            if (!all) {
                const int32_t cut = keep && rowok ? pos - kb * kPfBlock + 1 : 0;
#pragma unroll
                for (int u = 0; u < kPfTiles; ++u) lim[u] = min(16 * u + blk.rows[u].y, cut);
            }
            const int buf = j & 1;
            ok = wait(bar(kBarS + 2 * t + buf), (j >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (j > 0 && (j & (kPbWindow - 1)) == 0) {
                // A window is over: its sum goes to the output row, the next one begins at zero.
                // (P V of block j - 2 ended before these scores were made, so the barrier is at most
                // one phase behind, which its parity can tell.)
                ok = wait(bar(kBarPv + t), (j - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                // log2 of the present reference over that of the earlier windows
                const float rise = (m_used - ref_m) + (xref - ref_x);
                if constexpr (SPLIT) {
                    // (to the other tile's columns, which this CTA does not use: the output row is
                    // the cluster's)
                    const float down = ref_m == kPfNegInf ? 0.f : exp2f(-rise);
                    ref_m = m_used;
                    ref_x = xref;
#pragma unroll 1
                    for (int cc = 0; cc < D / 16; ++cc) {
                        float v[16];
                        tc_ld16(ocol + 16u * cc, v);
                        tc_wait_ld();
                        uint32_t o[16];
                        if (j > kPbWindow) {
                            float e16[16];
                            tc_ld16(ecol + 16u * cc, e16);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] = __float_as_uint(fmaf(e16[e], down, v[e]));
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(v[e]);
                        }
                        tc_st16(ecol + 16u * cc, o);
                    }
                    tc_wait_st();
                    tc_fence_before();
                } else {
                    const bool some = rowok && m_used != kPfNegInf;
                    const bool first = some && ref_m == kPfNegInf;
                    // far above the row's reference, what it holds moves to the new one first
                    const bool move = some && !first && rise > 60.f;
                    const float down = move ? exp2f(-rise) : 1.f;
                    const float f = some && !first && !move ? exp2f(rise) : 1.f;
                    if (first || move) {
                        ref_m = m_used;
                        ref_x = xref;
                    }
#pragma unroll 1
                    for (int cc = 0; cc < D / 16; ++cc) {
                        __syncwarp();
                        float v[16];
                        tc_ld16(ocol + 16u * cc, v);
                        tc_wait_ld();
                        float* to = orow + 16 * cc;
                        if (move) {
                            __threadfence();
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const float4 o = __ldcg(reinterpret_cast<const float4*>(to + e));
                                *reinterpret_cast<float4*>(to + e) =
                                    make_float4(fmaf(o.x, down, v[e]), fmaf(o.y, down, v[e + 1]),
                                                fmaf(o.z, down, v[e + 2]), fmaf(o.w, down, v[e + 3]));
                            }
                        } else if (first) {
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<float4*>(to + e) =
                                    make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                        } else if (some) {
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                red_add4(to + e, v[e] * f, v[e + 1] * f, v[e + 2] * f, v[e + 3] * f);
                        }
                    }
                    __syncwarp();
                    tc_fence_before();
                }
            }
            const uint32_t sbuf = tbase + lanes + 256u + 128u * t + 64u * buf;
            float x[64];
            {
                float v[32];
                tc_ld32(sbuf, v);
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = v[e];
                tc_ld32(sbuf + 32u, v);
#pragma unroll
                for (int e = 0; e < 32; ++e) x[32 + e] = v[e];
            }
            tc_wait_ld();
            // Key e of tile u is kept iff e < lim[u].
            if (!all) {
#pragma unroll
                for (int e = 0; e < 64; ++e) x[e] = e < lim[e >> 4] ? x[e] : kPfNegInf;
            }
            // the row maximum of the scores (log2 units); -inf stays -inf
            const float mx = fmaxf(fmaxf(max16(x) * fu[0], max16(x + 16) * fu[1]),
                                   fmaxf(max16(x + 32) * fu[2], max16(x + 48) * fu[3]));
            m_true = fmaxf(m_true, mx);
            // Lazy rescale of l when the row maximum grows by more than 2^8, and of O then and when a
            // weight may exceed 2^kPbMost. The tensor-memory traffic is warp-collective, so a warp
            // rescales when any of its rows must. A tile far below the reference comes here too.
            if (__any_sync(0xffffffffu, mx > m_used + kTcRescale || mx + blk.high > mref + kPbMost ||
                                            blk.low < xref - 64.f)) {
                // Keys whose V is all zeros count in the sum, but not for O's reference (a token of the
                // same tile, whose scale it is, may be one that the row does not see): a lane looks at
                // two rows of the V stage. P V of this block, and so the stage's next use, waits for the
                // weights made below.
                ok = wait(bar(kBarVFull + i % kPbStages), (i / kPbStages) & 1);
                if (!ok) break;
                uint32_t z0 = 0xffffffffu, z1 = 0xffffffffu;
                const uint8_t* vst = base + L.vst + (uint32_t)(i % kPbStages) * L.blk_bytes;
#pragma unroll 1
                for (uint32_t ch = 0; ch < D / 8 && (z0 | z1) != 0u; ++ch) {  // (most often once)
                    const uint8_t* at = vst + (ch >> 3) * kHalf;
                    const uint4 a = *reinterpret_cast<const uint4*>(at + swz128(lane, ch & 7u));
                    const uint4 c = *reinterpret_cast<const uint4*>(at + swz128(lane + 32u, ch & 7u));
                    z0 &= __ballot_sync(0xffffffffu, ((a.x | a.y | a.z | a.w) & 0x7fff7fffu) == 0u);
                    z1 &= __ballot_sync(0xffffffffu, ((c.x | c.y | c.z | c.w) & 0x7fff7fffu) == 0u);
                }
                // the row's largest weight times V scale
                float top = kPfNegInf;
#pragma unroll
                for (int u = 0; u < kPfTiles; ++u) {
                    const uint32_t z = (u < 2 ? z0 : z1) >> (16 * (u & 1));
                    float t;
                    if ((z & 0xffffu) == 0u) {
                        t = max16(x + 16 * u);
                    } else {
                        float y[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) y[e] = (z >> e) & 1u ? kPfNegInf : x[16 * u + e];
                        t = max16(y);
                    }
                    top = fmaxf(top, fmaf(t, fu[u], blk.scale[u].z));
                }
                float fo = 1.f;
                if (mx > m_used + kTcRescale || top > mref + kPbMost) {
                    const float m_new = fmaxf(m_used, mx);
                    const bool none = m_used == kPfNegInf;  // O and l are zeros
                    // (an integer, so that 2^-xref is exact; the reference moves down by less than 1)
                    float x_new = ceilf(top - m_new) - kPbTop;
                    if (!none) x_new = fmaxf(x_new, floorf((m_used - m_new) + xref));
                    x_new = fminf(fmaxf(x_new, -126.f), 127.f);
                    if (!none) {
                        l *= exp2f(m_used - m_new);
                        fo = exp2f((m_used - m_new) + (xref - x_new));
                    }
                    m_used = m_new;
                    xref = x_new;
                    xfac = pow2i((int)x_new);
                    mref = m_new + x_new;
                }
                if ((j & (kPbWindow - 1)) != 0 && __any_sync(0xffffffffu, fo != 1.f)) {
                    // O holds the window's blocks before this one: wait for them, then scale it
                    ok = wait(bar(kBarPv + t), (j - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < D / 16; ++cc) {  // (16 columns: the scores stay in registers)
                        float v[16];
                        tc_ld16(ocol + 16u * cc, v);
                        tc_wait_ld();
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(v[e] * fo);
                        tc_st16(ocol + 16u * cc, o);
                    }
                    tc_wait_st();
                }
                // Keys with a V of zeros, whose weight for O may be of any size, and the tiles 2^64
                // below the reference, whose weights may vanish, enter the sum here and weigh 0 in O.
                const float mu = m_used == kPfNegInf ? 0.f : m_used;
#pragma unroll
                for (int u = 0; u < kPfTiles; ++u) {
                    uint32_t z = ((u < 2 ? z0 : z1) >> (16 * (u & 1))) & 0xffffu;
                    if (blk.scale[u].z < xref - 64.f) z = 0xffffu;
                    if (z != 0u) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const bool out = (z >> e) & 1u;
                            l += out ? ex2_approx(fmaf(x[16 * u + e], fu[u], -mu)) : 0.f;
                            x[16 * u + e] = out ? kPfNegInf : x[16 * u + e];
                        }
                    }
                }
                __syncwarp();
            }
            // w = 2^(x f - mref + log2(V scale)) in pairs; a masked key (-inf) gives +0. w goes to the
            // score buffer as two fp16 terms: hi (rounded) into columns [0, 32), lo (the exact rest,
            // rounded) into [32, 64). hi comes back from fp16 by a conversion, on the FMA pipe:
            // masking its word would load the ALU pipe, which is the fuller one. The sum takes w
            // times 2^xref over its tile's V scale.
            const float base2 = m_used == kPfNegInf ? 0.f : mref;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t ph[16], pl[16];
#pragma unroll
                for (int uu = 0; uu < 2; ++uu) {
                    const int u = 2 * hf + uu;
                    const uint64_t f2 = pack_f32x2(fu[u], fu[u]);
                    const float2 vs = *reinterpret_cast<const float2*>(&blk.scale[u].z);
                    const float nm = vs.x - base2;
                    const float undo = fminf(vs.y * xfac, 1.8446744e19f);  // (at most 2^64 where w counts)
                    const uint64_t n2 = pack_f32x2(nm, nm);
                    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
                    for (int cc = 0; cc < 8; ++cc) {
                        float p0, p1;
                        fma_f32x2(x[16 * u + 2 * cc], x[16 * u + 2 * cc + 1], f2, n2, p0, p1);
                        p0 = ex2_approx(p0);
                        p1 = ex2_approx(p1);
                        if (cc & 1) add_f32x2(s2, s3, p0, p1);
                        else        add_f32x2(s0, s1, p0, p1);
                        const uint32_t g = pack_f16(p0, p1);
                        ph[8 * uu + cc] = g;
                        float r0, r1;
                        sub_f32x2(p0, p1, f16_lo(g), f16_hi(g), r0, r1);
                        pl[8 * uu + cc] = pack_f16(r0, r1);
                    }
                    l = fmaf((s0 + s1) + (s2 + s3), undo, l);
                }
                tc_st16(sbuf + 16u * hf, ph);
                tc_st16(sbuf + 32u + 16u * hf, pl);
            }
            ring_release(i);
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(bar(kBarP + 2 * t + buf));
            ++j;
        }
        // ---- epilogue: this row's O, maximum and sum ------------------------------------------
        if (ok && n > 0) {
            ok = mbar_wait(bar(kBarDrain + t), 0, abort_p, p.dev_err);
            tc_fence_after();
        }
        ok = __all_sync(0xffffffffu, ok);
        const bool any = j > 0 && ok;
        if (SPLIT && use > 1) {
            // the row's sum, relative to 2^(m_used + xref), and what it is relative to
            if ((tmask >> t) & 1u) {
                const bool more = j > kPbWindow;  // (at a multiple of it the last window is still in O)
                const float down =
                    more && ref_m != kPfNegInf ? exp2f((ref_m - m_used) + (ref_x - xref)) : 0.f;
                float* to = part + (r & 127) * (D + 4);
#pragma unroll 1
                for (int cc = 0; cc < D / 16; ++cc) {
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = 0.f;
                    if (any) {
                        tc_ld16(ocol + 16u * cc, v);
                        tc_wait_ld();
                        if (more) {
                            float e16[16];
                            tc_ld16(ecol + 16u * cc, e16);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] = fmaf(e16[e], down, v[e]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<float4*>(to + 16 * cc + e) =
                            make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
                stat[r & 127] = make_float4(m_used, xref, l, m_true);
            }
        } else if (!SPLIT || rank == 0) {
            // out = (O + earlier windows) 2^xref / l, the exponent and 1 / l multiplied in turn (either
            // may be far from 1)
            const float inv = l > 0.f ? 1.f / l : 0.f;
            const float up = xfac;
            // (SPLIT: fewer blocks than a window)
            const bool more = !SPLIT && ref_m != kPfNegInf && ok;
            const float down = more ? exp2f((ref_m - m_used) + (ref_x - xref)) : 0.f;
            if (more) __threadfence();  // the row's earlier additions
#pragma unroll 1
            for (int cc = 0; cc < D / 16; ++cc) {
                __syncwarp();
                float v[16];
                if (any) {
                    tc_ld16(ocol + 16u * cc, v);
                    tc_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = 0.f;
                }
                if (rowok) {
                    float* to = orow + 16 * cc;
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        float4 o = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                        if (more) {
                            const float4 a = __ldcg(reinterpret_cast<const float4*>(to + e));
                            o.x = fmaf(a.x, down, o.x);
                            o.y = fmaf(a.y, down, o.y);
                            o.z = fmaf(a.z, down, o.z);
                            o.w = fmaf(a.w, down, o.w);
                        }
                        *reinterpret_cast<float4*>(to + e) =
                            make_float4(o.x * inv * up, o.y * inv * up, o.z * inv * up, o.w * inv * up);
                    }
                }
            }
            if (rowok) {
                // report the true row max and the sum relative to it
                if (p.m_out) p.m_out[row] = m_true == kPfNegInf ? kPfNegInf : m_true * kLn2;
                if (p.e_out) p.e_out[row] = m_true == kPfNegInf ? 0.f : l * exp2f(m_used - m_true);
            }
        }
    }
    if constexpr (SPLIT) {
        if (use > 1) {  // (one answer in the whole cluster)
            // ---- the rows' parts meet: each CTA of the cluster joins its share of the 128 rows ----
            __syncthreads();
            cluster_arrive();
            cluster_wait();
            const int t = tmask >> 1;  // the CTA's tile
            const int rows = 128 / pp.split;
            for (int x = tid; x < rows * (D / 4); x += kPbThreads) {
                const int rl = rank * rows + x / (D / 4), c4 = x % (D / 4);
                const int r = 128 * t + rl, z = r >> 6, qi = q_block(z);
                const int32_t pos = (qa + qi) * kPfBlock + (r & 63);
                if (!(((has >> qi) & 1u) && pos >= c0 && pos < Ln)) continue;
                // the row's maximum; the parts' largest reference, 2^(top_m + top_x)
                float m = kPfNegInf, top_m = kPfNegInf, top_x = 0.f;
                for (int y = 0; y < use; ++y) {
                    const float4 st = ld_cluster4(smem_u32(stat + rl), y);
                    m = fmaxf(m, st.w);
                    if (st.x != kPfNegInf && (st.x - top_m) + (st.y - top_x) > 0.f) {
                        top_m = st.x;
                        top_x = st.y;
                    }
                }
                float l = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int y = 0; y < use && m != kPfNegInf; ++y) {
                    const float4 st = ld_cluster4(smem_u32(stat + rl), y);
                    if (st.x == kPfNegInf) continue;
                    const float4 v = ld_cluster4(smem_u32(part + rl * (D + 4) + 4 * c4), y);
                    const float f = exp2f((st.x - top_m) + (st.y - top_x));
                    l = fmaf(st.z, exp2f(st.x - m), l);
                    o.x = fmaf(v.x, f, o.x);
                    o.y = fmaf(v.y, f, o.y);
                    o.z = fmaf(v.z, f, o.z);
                    o.w = fmaf(v.w, f, o.w);
                }
                // out = sum 2^(top_m - m) 2^top_x / l, whole powers of two multiplied in turn as above
                float inv = l > 0.f ? 1.f / l : 0.f, up = 0.f, up2 = 0.f;
                if (m != kPfNegInf) {
                    const float whole = fmaxf(rintf(top_m - m), -126.f);
                    inv *= exp2f((top_m - m) - whole);
                    up = pow2i((int)top_x);
                    up2 = pow2i((int)whole);
                }
                const int64_t row = ((int64_t)b * p.Tq + (pos - c0)) * p.Hq + h0 + q_head(z);
                *reinterpret_cast<float4*>(p.out + row * D + 4 * c4) =
                    make_float4(o.x * inv * up * up2, o.y * inv * up * up2, o.z * inv * up * up2,
                                o.w * inv * up * up2);
                if (c4 == 0) {
                    if (p.m_out) p.m_out[row] = m == kPfNegInf ? kPfNegInf : m * kLn2;
                    if (p.e_out) p.e_out[row] = l;
                }
            }
            __syncwarp();
            cluster_arrive();  // no CTA leaves while another reads its parts
            cluster_wait();
        }
    }
    // ---- teardown: the allocating warp frees the tensor memory --------------------------------
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tc_dealloc(tbase, kPbCols);
    }
}

std::mutex g_pb_mutex;

template <int D, bool SPLIT>
dattn_status_t ensure_smem(uint32_t bytes) {
    static int set[kMaxDevices] = {};  // a function attribute belongs to a device
    std::lock_guard<std::mutex> lock(g_pb_mutex);
    int& mine = set[device_index()];
    if ((int)bytes > mine) {
        if (cudaFuncSetAttribute(prefill_block_kernel<D, SPLIT>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)bytes) != cudaSuccess)
            return DATTN_ERR_CUDA;
        mine = (int)bytes;
    }
    return DATTN_OK;
}

// Clusters of s CTAs that the device holds at once (15 of 8, 36 of 4 and 76 of 2 on 152 SMs, one CTA
// per SM whatever its shared memory); asked once per device and size.
template <int D>
int32_t clusters_at_once(int32_t s, uint32_t bytes) {
    static std::atomic<int32_t> known[kMaxDevices][9] = {};
    std::atomic<int32_t>& mine = known[device_index()][s];
    int32_t n = mine.load(std::memory_order_relaxed);
    if (n > 0) return n - 1;
    if (ensure_smem<D, true>(bytes) != DATTN_OK) return 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)s);
    cfg.blockDim = dim3(kPbThreads);
    cfg.dynamicSmemBytes = bytes;
    cudaLaunchAttribute attr[1]{};
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)s, 1u, 1u};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int at_once = 0;
    if (cudaOccupancyMaxActiveClusters(&at_once, prefill_block_kernel<D, true>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        at_once = 0;
    }
    mine.store(at_once + 1, std::memory_order_relaxed);
    return at_once;
}

}  // namespace

template <int D>
static dattn_status_t launch_d(const PfParams& p0, const void* k_pool, const void* v_pool,
                               const float* kv_scale, cudaStream_t stream) {
    PbParams pp{};
    pp.f = p0;
    PfParams& p = pp.f;
    pp.hp = p.g % 4 == 0 ? 4 : p.g % 2 == 0 ? 2 : 1;
    pp.nq = 4 / pp.hp;
    pp.k_pool = static_cast<const uint8_t*>(k_pool);
    pp.v_pool = static_cast<const uint8_t*>(v_pool);
    pp.scale = reinterpret_cast<const float2*>(kv_scale);
    const int32_t nwords = (p.max_pages * p.P / kPfBlock + 1 + 4 + 31) / 32;
    const PbSmem L = pb_smem_layout(D, pp.nq, nwords);
    if (L.total > 227u * 1024u) return DATTN_ERR_UNSUPPORTED;
    const int32_t blocks = (p.Tq + kPfBlock - 1) / kPfBlock + 1;  // query blocks a chunk can touch
    p.nqb = (blocks + pp.nq - 1) / pp.nq;
    const int64_t per_head = (int64_t)p.nqb * (p.g / pp.hp);
    const int64_t pairs = (int64_t)p.B * p.Hkv * per_head;
    const int32_t sms = sm_count_current();
    // a last wave of tile pairs for at most half of the SMs: a CTA for each tile instead
    const int64_t rest = pairs % sms;
    pp.whole = (int32_t)(2 * rest <= sms ? pairs - rest : pairs);
    // Few tiles with rows (of a chunk that begins on a block): the largest cluster for each with which
    // all run at once, where the block table has room for blocks to share.
    const int64_t tiles = (int64_t)p.B * p.Hkv * (p.g / pp.hp) * (((blocks - 1) * pp.hp + 1) / 2);
    pp.split = 1;
    for (int32_t s = 8; s > 1 && pp.split == 1; s /= 2)
        if (tiles * s <= sms &&
            (int64_t)p.max_pages * p.P >= (int64_t)s * kPbSplitBlocks * kPfBlock &&
            tiles <= clusters_at_once<D>(s, L.total)) {
            pp.split = s;
            pp.whole = 0;
        }
    const int64_t ctas = (pp.whole + 2 * (pairs - pp.whole)) * pp.split;
    if (pairs >= (1ll << 31) - sms) return DATTN_ERR_UNSUPPORTED;
    // as in prefill.cu: the smallest group of KV heads whose CTAs fill three waves
    p.kv_group = p.Hkv;
    for (int32_t G = 1; G < p.Hkv; ++G)
        if (p.Hkv % G == 0 && G * per_head >= 3ll * sms) {
            p.kv_group = G;
            break;
        }
    auto kern = pp.split > 1 ? prefill_block_kernel<D, true> : prefill_block_kernel<D, false>;
    const dattn_status_t st =
        pp.split > 1 ? ensure_smem<D, true>(L.total) : ensure_smem<D, false>(L.total);
    if (st != DATTN_OK) return st;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kPbThreads);
    cfg.dynamicSmemBytes = L.total;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)pp.split, 1u, 1u};
    cfg.attrs = attr;
    cfg.numAttrs = pp.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, pp, nwords) == cudaSuccess ? DATTN_OK : DATTN_ERR_CUDA;
}

dattn_status_t launch_prefill_block(const PfParams& p, const void* k_pool, const void* v_pool,
                                    const float* kv_scale, int D, cudaStream_t stream) {
    return D == 64 ? launch_d<64>(p, k_pool, v_pool, kv_scale, stream)
                   : launch_d<128>(p, k_pool, v_pool, kv_scale, stream);
}

}  // namespace dattn
