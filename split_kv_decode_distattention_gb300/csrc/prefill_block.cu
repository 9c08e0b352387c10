// Prefill over the block-scaled 8-bit pool (dattn_prefill with DATTN_KV_FP8_BLOCK): a chunk of Tq
// new query tokens per request attends the paged cache, causally or block-sparsely, exactly as over
// the bf16 pool (prefill.cu holds the method's sources and the block rules).
//
// Arithmetic. An E4M3 code is an fp16 number, so the codes are widened to fp16 in shared memory
// (one conversion for two codes) and both products run in fp16 with fp32 accumulation. The query
// row is scaled by a power of two 2^a that brings its largest element to [2^14, 2^15) and rounded
// to fp16: exact for every element within 2^28 of the largest. The K scale of a 16-key tile
// multiplies its scores; the V scale, a power of two, goes into the exponent of its weights,
// w = 2^(s - m + log2(scale / r)), where 2^r is a power of two that the scales seen so far exceed
// by 2^7 at most (raised, and the accumulators rescaled, when a larger one comes), so that w stays
// below 2^15. w enters the product as two fp16 terms, 22 bits together.
// The tensor cores add into their fp32 accumulators rounding towards zero, which over a long
// context shrinks the result (5.6e-5 after 4096 products of a 32K context), so a row's accumulator is
// emptied into its output row every kPbWindow key blocks, by fp32 additions.
//
// What bounds it: the tensor cores. A step takes two key blocks, 128 keys. For 128 query rows it
// needs one product S = Q K^T and two products O += P V, 3 x 2 x 128 x 128 x d operations for the
// 2 x 2 x 128 x 128 x d that count: 2/3 of the dense 16-bit rate at most. The keys of a step are
// widened once for 256 query rows: one CTA per SM holds two tiles of 128 rows, and while one tile is
// in its softmax the tensor cores work on the other. (One key block to a step, with two score
// buffers for each tile, lost as much again to the waits and the products of half the size.)
//
// A CTA: 256 rows as four quarters of 64 tokens: one query block of four heads of a KV head (g a
// multiple of 4), two query blocks of two heads (even g), or four query blocks of one head. A tile
// (two quarters) takes part in a step only if one of its quarters keeps one of its blocks. Where the
// last wave of CTAs would fill less than half of the SMs, its tiles get a CTA each. 22 warps:
//   0-15   the softmax: a query row is two threads, one for each key block of a step (so that the
//          two tiles' softmaxes fit beside each other's products); they exchange the row's maximum
//          through shared memory, and each rescales and writes half of the row's output;
//   16-19  load codes, widen them and write the K and V stages in the 128-byte-swizzled layout of
//          the MMA operands;
//   20     one thread issues the products: for each tile P V of the last step, then S of this one;
//   21     walks the key blocks, eight at a time, one lane per 16-key tile, and leaves each block's
//          place, lengths and scales in a ring in shared memory for the others.
// Tensor memory: O of the two tiles, then their scores, over which P is written: all 512 columns.
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "prefill.cuh"

namespace dattn {

namespace {

constexpr int kPbRows = 256;                // query rows of a CTA: two tiles of 128
constexpr int kPbSoftWarps = 16;            // a row's softmax takes two threads
constexpr int kPbConvWarp = 16;             // warps 16-19 widen the codes
constexpr int kPbConvThreads = 128;
constexpr int kPbMmaWarp = 20;
constexpr int kPbPlaceWarp = 21;            // the places of the key blocks
constexpr int kPbThreads = 22 * 32;
constexpr int kPbStages = 2;                // K stages, and V stages, of a step (two key blocks)
constexpr int kPbGroup = 8;                 // key blocks that warp 21 resolves at once
constexpr int kPbRing = 2 * kPbGroup;       // the blocks' ring
constexpr int kPbWindow = 8;                // steps between two emptyings of an accumulator
constexpr uint32_t kPbCols = 512;           // O: [0, 128), [128, 256); S and P: 256 + 128 tile

// mbarriers
constexpr int kBarKFull = 0, kBarKEmpty = 2, kBarVFull = 4, kBarVEmpty = 6;  // + stage
constexpr int kBarS = 8, kBarP = 10;        // + tile
constexpr int kBarRingFull = 12, kBarRingEmpty = 14, kBarDrain = 16;
constexpr int kBarPair = 17, kPbBars = 25;  // + warp & 7: the two warps of the same rows
constexpr int kRingReaders = 21;            // warps 0-20

// A key block in the ring: its 16-key tiles as the widening reads them (first row over all heads,
// tokens) and as the softmax does (K scale, -, log2 of the V scale over 2^r, 2 to minus that), its
// index, the quarters of rows that keep it (bits 0-3; bit 4: all its keys are written) and its
// step's r.
struct PbBlock {
    int2 rows[kPfTiles];
    float4 scale[kPfTiles];
    int32_t kb, act, r, pad;
};
constexpr int32_t kPbFull = 16;
// the tiles (bits) of the quarters that keep a block
__device__ __forceinline__ uint32_t tiles_of(uint32_t act) {
    return ((act & 3u) ? 1u : 0u) | ((act & 12u) ? 2u : 0u);
}

struct PbSmem {
    uint32_t q, step_bytes, kst, vst, bm, ring, bars, taddr, abort, qscale, rowx, total;
};

__host__ __device__ inline PbSmem pb_smem_layout(int D, int nq, int nwords) {
    PbSmem s;
    uint32_t o = 0;
    s.q = o;           o += (uint32_t)kPbRows * D * 2u;
    s.step_bytes = 128u * D * 2u;
    s.kst = o;         o += kPbStages * s.step_bytes;
    s.vst = o;         o += kPbStages * s.step_bytes;
    s.ring = o;        o += kPbRing * (uint32_t)sizeof(PbBlock);
    s.bars = o;        o += (kPbBars + 1) * 8u;
    s.taddr = o;       o += 16u;
    s.abort = o;       o += 16u;
    s.qscale = o;      o += kPbRows * 4u;
    s.rowx = o;        o += 2u * 2u * kPbRows * 4u;  // [buffer][half][row]
    s.bm = o;          o += (uint32_t)(nq * nwords) * 4u;
    s.total = o;
    return s;
}

struct PbParams {
    PfParams f;
    int32_t hp, nq;    // heads and query blocks of a CTA: hp * nq = 4
    int32_t whole;     // CTAs of two tiles; the others hold one tile each
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

// Matrix descriptors as their lower words: the upper word (stride 1024 bytes, the descriptor version
// and the 128-byte swizzle, see tc_sdesc) is the same for every operand here, and a step along an
// operand adds its bytes / 16 to the lower word.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
    return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}
// The products are predicated on the issuing lane instead of branched around: the code around them
// stays convergent, so that their operands can live in uniform registers, where tcgen05.mma takes
// them from.
template <bool ACC>
__device__ __forceinline__ void pb_mma_ss(uint32_t lead, uint32_t d_tmem, uint32_t a_lo,
                                          uint32_t b_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\tmov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "n"(kDescHi), "n"(ACC ? 1 : 0), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void pb_mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem,
                                          uint32_t b_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "setp.ne.b32 q, %6, 0;\n\tmov.b64 b, {%2, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "n"(kDescHi), "r"(acc), "r"(lead)
        : "memory");
}
// tc_commit by the issuing lane
__device__ __forceinline__ void pb_commit(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            bar),
        "r"(lead)
        : "memory");
}
// 1 in one lane of the (convergent) warp
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
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

template <int D>
__global__ void __launch_bounds__(kPbThreads, 1)
prefill_block_kernel(const __grid_constant__ PbParams pp, int32_t nwords) {
    constexpr uint32_t kHalf = 128u * 128u;  // a 128-byte half of a step's rows
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
    const int32_t extra = max((int32_t)blockIdx.x - pp.whole, 0);
    const uint32_t tmask = (int32_t)blockIdx.x < pp.whole ? 3u : 1u << (extra & 1);
    int32_t c = (int32_t)blockIdx.x < pp.whole ? (int32_t)blockIdx.x : pp.whole + (extra >> 1);
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
    float* qscale = reinterpret_cast<float*>(base + L.qscale);
    volatile int* abort_p = reinterpret_cast<volatile int*>(base + L.abort);
    if (tid == 0) {
        for (int s = 0; s < kPbStages; ++s) {
            mbar_init(bar(kBarKFull + s), kPbConvThreads);
            mbar_init(bar(kBarKEmpty + s), 1);
            mbar_init(bar(kBarVFull + s), kPbConvThreads);
            mbar_init(bar(kBarVEmpty + s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kBarS + i), 1);
            mbar_init(bar(kBarP + i), 256);
            mbar_init(bar(kBarRingFull + i), 1);
            mbar_init(bar(kBarRingEmpty + i), kRingReaders);
        }
        mbar_init(bar(kBarDrain), 1);
        for (int i = 0; i < 8; ++i) mbar_init(bar(kBarPair + i), 2);
        *abort_p = 0;
        fence_mbar_init();
    }
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
    if (!active && tid == 0 && h0 == 0 && J == 0) set_err(p.dev_err, DATTN_DEVERR_LEN_OOB);
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
    const int32_t ns = (n + 1) >> 1;  // steps of two key blocks; the last may miss its second
    // The ring: block x in slot x % 16, ready with its group of eight (four steps); a reader's warp
    // gives a group back after its last step.
    auto wait = [&](uint32_t bar_addr, uint32_t parity) {  // by a whole warp, one answer
        return __all_sync(0xffffffffu, mbar_wait(bar_addr, parity, abort_p, p.dev_err)) != 0;
    };
    auto ring_ready = [&](int32_t i) {
        return (i & 3) != 0 || wait(bar(kBarRingFull) + 8u * ((i >> 2) & 1), (i >> 3) & 1);
    };
    auto ring_release = [&](int32_t i) {
        __syncwarp();
        if ((i & 3) == 3 && lane == 0) mbar_arrive(bar(kBarRingEmpty) + 8u * ((i >> 2) & 1));
    };

    if (active && warp == kPbPlaceWarp) {
        // ---------------------------------------------------------------- places of the key blocks
        const int blk = lane >> 2, u = lane & 3;  // this lane: tile u of the group's block blk
        int32_t w = 0;
        uint32_t q[4], word = held_word(bm, nq, nwords, tmask, 0, q);
        int r = -126;
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
            // 2^r: what the V scales up to each step exceed by 2^7 at most
            const int ve = sc.y > 0.f ? (__float_as_int(sc.y) >> 23) - 127 : -1000;
            int vm = max(ve, __shfl_xor_sync(0xffffffffu, ve, 1));
            vm = max(vm, __shfl_xor_sync(0xffffffffu, vm, 2));
            int mine = r;
            for (int x = 0; x < kPbGroup / 2; ++x) {
                const int v = max(__shfl_sync(0xffffffffu, vm, 8 * x),
                                  __shfl_sync(0xffffffffu, vm, 8 * x + 4));
                if (v > r + 7) r = v;
                if (x == blk >> 1) mine = r;
            }
            // (far below 2^r a scale counts as 2^(r - 64): nothing beside the others; codes with
            // scale 0 are zeros)
            const int lv = sc.y > 0.f ? max(ve - mine, -64) : 0;
            int full = hi == 16 ? 1 : 0;
            full &= __shfl_xor_sync(0xffffffffu, full, 1);
            full &= __shfl_xor_sync(0xffffffffu, full, 2);
            if (i >= kPbRing)
                ok = wait(bar(kBarRingEmpty) + 8u * ((i / kPbGroup) & 1), ((i / kPbRing) - 1) & 1);
            if (ok && blk < ((cnt + 1) & ~1)) {  // (an empty block completes the last step)
                PbBlock& to = ring[(i + blk) & (kPbRing - 1)];
                to.rows[u] = make_int2(y, hi);
                to.scale[u] = make_float4(sc.x, 0.f, (float)lv, pow2i(-lv));
                if (u == 0) {
                    to.kb = kb;
                    to.act = act | (full ? kPbFull : 0);
                    to.r = mine;
                }
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(bar(kBarRingFull) + 8u * ((i / kPbGroup) & 1));
        }
    } else if (active && warp >= kPbConvWarp && warp < kPbMmaWarp) {
        // ------------------------------------------------------ widening: codes -> K and V stages
        // A row of D codes is D/16 threads of 16 codes; a pass takes RP rows, NP passes a block.
        // Eight neighbours store to two rows of one half: all banks. The loads run two blocks ahead
        // of the stores: K, K, V, V of a step in turn.
        constexpr int CPR = D / 16, RP = kPbConvThreads / CPR, NP = 64 / RP;
        const int ct = tid - kPbConvWarp * 32;
        const int c16 = D == 64 ? ct & 3 : (ct & 3) | ((ct >> 1) & 4);
        const int rr = D == 64 ? ct >> 2 : ((ct >> 2) & 1) | ((ct >> 4) << 1);
        uint4 va[NP], vb[NP];  // the two blocks of a step
        // 16 codes a row of block x; rows that hold no token of the request are zeros
        auto load = [&](const uint8_t* pool, int32_t x, uint4 (&v)[NP]) {
            const PbBlock& blk = ring[x & (kPbRing - 1)];
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int2 at = blk.rows[(rr + RP * k) >> 4];
                const int r = (rr + RP * k) & 15;
                v[k] = make_uint4(0u, 0u, 0u, 0u);
                if (r < at.y)
                    v[k] = __ldg(reinterpret_cast<const uint4*>(pool + (int64_t)(at.x + r) * D +
                                                                16 * c16));
            }
        };
        const uint32_t half = (c16 >> 2) * kHalf, ch = 2u * (c16 & 3);
        auto store = [&](uint8_t* st, int row0, const uint4 (&v)[NP]) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const uint32_t row = (uint32_t)(row0 + rr + RP * k);
                uint4 a, c2;
                e4m3x4_to_f16(v[k].x, a.x, a.y);
                e4m3x4_to_f16(v[k].y, a.z, a.w);
                e4m3x4_to_f16(v[k].z, c2.x, c2.y);
                e4m3x4_to_f16(v[k].w, c2.z, c2.w);
                *reinterpret_cast<uint4*>(st + half + swz128(row, ch)) = a;
                *reinterpret_cast<uint4*>(st + half + swz128(row, ch + 1u)) = c2;
            }
        };
        bool ok = ns > 0 && ring_ready(0);
        if (ok) {
            load(pp.k_pool, 0, va);
            load(pp.k_pool, 1, vb);
        }
        for (int32_t i = 0; i < ns && ok; ++i) {
            const int s = i % kPbStages, ph = (i / kPbStages) & 1;
            if (i >= kPbStages) ok = wait(bar(kBarKEmpty + s), ph ^ 1);
            if (!ok) break;
            uint8_t* st = base + L.kst + (uint32_t)s * L.step_bytes;
            store(st, 0, va);
            load(pp.v_pool, 2 * i, va);
            store(st, 64, vb);
            load(pp.v_pool, 2 * i + 1, vb);
            fence_proxy_async_smem();
            mbar_arrive(bar(kBarKFull + s));
            ring_release(i);
            if (i >= kPbStages) ok = wait(bar(kBarVEmpty + s), ph ^ 1);
            if (!ok) break;
            const bool more = i + 1 < ns;
            if (more) ok = ring_ready(i + 1);
            if (!ok) break;
            st = base + L.vst + (uint32_t)s * L.step_bytes;
            store(st, 0, va);
            if (more) load(pp.k_pool, 2 * i + 2, va);
            store(st, 64, vb);
            if (more) load(pp.k_pool, 2 * i + 3, vb);
            fence_proxy_async_smem();
            mbar_arrive(bar(kBarVFull + s));
        }
    } else if (active && warp == kPbMmaWarp) {
        // ---------------------------------------------------------------- MMA issuer
        // The whole warp walks the blocks and waits; one lane issues. What the products depend on
        // comes out of warp reductions: the compiler then knows it to be uniform.
        if (ns > 0) {
            const uint32_t lead = elect_lane();
            constexpr uint32_t idesc_s = pb_idesc(128, 128, 0);
            constexpr uint32_t idesc_o = pb_idesc(128, D, 1);
            const uint32_t qd = desc_lo(smem_u32(base + L.q), 16u);
            const uint32_t kd = desc_lo(smem_u32(base + L.kst), 16u);
            const uint32_t vd = desc_lo(smem_u32(base + L.vst), kHalf);
            const uint32_t tb = __reduce_or_sync(0xffffffffu, tbase);
            bool ok = true;
            uint32_t j0 = 0u, j1 = 0u;  // each tile's steps so far
            uint32_t act = 0u, prev = 0u;
            // S of a tile, over its P of the step before (whose P V was issued before: products run
            // in order)
            auto issue_s = [&](int t, uint32_t k_lo) {
                const uint32_t to = tb + 256u + 128u * t;
                const uint32_t a_lo = qd + t * (128u * 128u >> 4);
                pb_mma_ss<false>(lead, to, a_lo, k_lo, idesc_s);
#pragma unroll
                for (int kk = 1; kk < D / 16; ++kk)
                    pb_mma_ss<true>(lead, to,
                                    a_lo + (((kk >> 2) * (kPbRows * 128u) + (kk & 3) * 32u) >> 4),
                                    k_lo + (((kk >> 2) * kHalf + (kk & 3) * 32u) >> 4), idesc_s);
                pb_commit(lead, bar(kBarS + t));
            };
            // O += P V of a tile's j'th step; every kPbWindow'th step begins a new sum. P of 32 keys is
            // 16 columns of hi terms, then 16 of lo terms (see the softmax).
            auto issue_pv = [&](int t, uint32_t j, uint32_t v_lo) {
                const uint32_t from = tb + 256u + 128u * t;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
#pragma unroll
                    for (int part = 0; part < 2; ++part)
                        pb_mma_ts(lead, tb + 128u * t,
                                  from + 32u * (kk >> 1) + 16u * part + 8u * (kk & 1),
                                  v_lo + (kk * 2048u >> 4), idesc_o,
                                  (part > 0 || kk > 0) ? 1u : j & (kPbWindow - 1u));
                }
            };
            for (int32_t i = 0; i <= ns && ok; ++i) {
                prev = act;
                act = 0u;
                uint32_t k_lo = 0u, v_lo = 0u;
                if (i < ns) {
                    ok = ring_ready(i);
                    if (!ok) break;
                    const PbBlock* blk = ring + ((2 * i) & (kPbRing - 1));
                    act = tiles_of(__reduce_or_sync(0xffffffffu, (uint32_t)(blk[0].act | blk[1].act)));
                    ring_release(i);
                    const int s = i % kPbStages;
                    ok = wait(bar(kBarKFull + s), (i / kPbStages) & 1);
                    if (!ok) break;
                    k_lo = kd + (uint32_t)s * (128u * D * 2u >> 4);
                }
                if (i > 0) {
                    const int sv = (i - 1) % kPbStages;
                    ok = wait(bar(kBarVFull + sv), ((i - 1) / kPbStages) & 1);
                    if (!ok) break;
                    v_lo = vd + (uint32_t)sv * (128u * D * 2u >> 4);
                }
                if (prev & 1u) {
                    ok = wait(bar(kBarP), (j0 - 1u) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv(0, j0 - 1u, v_lo);
                }
                if (act & 1u) {
                    tc_fence_after();
                    issue_s(0, k_lo);
                }
                if (prev & 2u) {
                    ok = wait(bar(kBarP + 1), (j1 - 1u) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    issue_pv(1, j1 - 1u, v_lo);
                }
                if (i > 0) pb_commit(lead, bar(kBarVEmpty + (i - 1) % kPbStages));
                if (act & 2u) {
                    tc_fence_after();
                    issue_s(1, k_lo);
                }
                if (i < ns) pb_commit(lead, bar(kBarKEmpty + i % kPbStages));
                j0 += act & 1u;
                j1 += act >> 1;
            }
            // every product is done: the epilogue's signal, and nothing of this CTA's may still run
            // on the tensor cores when it exits
            pb_commit(lead, bar(kBarDrain));
            mbar_wait(bar(kBarDrain), 0, abort_p, p.dev_err);
        }
    } else if (active && warp < kPbSoftWarps) {
        // ---------------------------------------------------------------- softmax threads
        constexpr int HC = D / 2;  // output columns of a thread
        const int t = (warp >> 2) & 1, hk = warp >> 3;  // tile; key block of a step, half of the columns
        const int r = 128 * t + 32 * (warp & 3) + lane, z = r >> 6;  // row and quarter
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ocol = tbase + lanes + 128u * t + HC * hk;
        const uint32_t scol = tbase + lanes + 256u + 128u * t + 64u * hk;
        const int qi = q_block(z);
        const int32_t pos = (qa + qi) * kPfBlock + (r & 63);
        const bool rowok = ((has >> qi) & 1u) && ((tmask >> t) & 1u) && pos >= c0 && pos < Ln;
        const float frow = qscale[r];
        float* rowx = reinterpret_cast<float*>(base + L.rowx) + r;
        // Meets the warp of the other half of these rows: the e'th value goes into buffer e % 2, whose
        // reader of two meetings ago has since come to the last one. (An mbarrier, whose wait is
        // bounded, and not a named barrier: after a failed wait the two may part.)
        auto meet = [&](float v, int32_t e, bool& good) {
            float* x2 = rowx + (2 * (e & 1)) * kPbRows;
            x2[hk * kPbRows] = v;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBarPair + (warp & 7)));
            good = wait(bar(kBarPair + (warp & 7)), e & 1);
            return x2[(hk ^ 1) * kPbRows];
        };
        float m_used = kPfNegInf, m_true = kPfNegInf, l = 0.f;  // l (of these keys): to m_used
        int rexp = -126;  // O is relative to m_used and to 2^rexp
        // what the output row holds of earlier windows is relative to 2^ref (-inf: nothing)
        float ref = kPfNegInf;
        int32_t j = 0;  // this tile's steps
        bool ok = true;
        for (int32_t i = 0; i < ns; ++i) {
            ok = ring_ready(i);
            if (!ok) break;
            const PbBlock* step = ring + ((2 * i) & (kPbRing - 1));
            if (!((step[0].act | step[1].act) & (3 << (2 * t)))) {
                ring_release(i);
                continue;
            }
            const PbBlock& blk = step[hk];
            const int32_t act = blk.act, kb = blk.kb, rnew = step[1].r;
            // The row's query block keeps kb; all keys pass for every row of the warp if they are
            // written and kb is an earlier block (rows without a query compute on zeros).
            const bool keep = (act >> z) & 1;
            const bool all = keep && (act & kPbFull) && kb < qa + qi;
            const int32_t cut = keep && rowok ? pos - kb * kPfBlock + 1 : 0;
            ok = wait(bar(kBarS + t), j & 1);
            if (!ok) break;
            tc_fence_after();
            // (these scores were made after P V of the step before: O is complete up to it)
            if (j > 0 && (j & (kPbWindow - 1)) == 0) {
                // a window is over: its sum goes to the output row, the next one begins at zero
                const bool some = rowok && m_used != kPfNegInf;
                const float at = m_used + (float)rexp;
                const bool first = some && ref == kPfNegInf;
                // far above the row's reference, what it holds moves to the new one first
                const bool move = some && !first && at > ref + 60.f;
                const float down = move ? exp2f(ref - at) : 1.f;
                if (first || move) ref = at;
                const float f = some ? exp2f(at - ref) : 0.f;
                float* orow = p.out + (((int64_t)b * p.Tq + (rowok ? pos - c0 : 0)) * p.Hq + h0 +
                                       q_head(z)) * D + HC * hk;
#pragma unroll 1
                for (int cc = 0; cc < HC / 16; ++cc) {
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
                    __syncwarp();
                }
            }
            // The row maximum of the scores (log2 units; -inf stays -inf), 32 at a time: they are
            // loaded again below. A tile's score factor is at least 1e-30, so that a masked key, -inf,
            // never meets a zero factor. Key e of tile u is kept iff e < min(16 u + its tokens, cut).
            auto scores = [&](int hf, float (&x)[32]) {
                tc_ld32(scol + 32u * hf, x);
                tc_wait_ld();
                if (!all) {
                    const int32_t l0 = min(32 * hf + blk.rows[2 * hf].y, cut) - 32 * hf;
                    const int32_t l1 = min(32 * hf + 16 + blk.rows[2 * hf + 1].y, cut) - 32 * hf;
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = e < (e < 16 ? l0 : l1) ? x[e] : kPfNegInf;
                }
            };
            auto factor = [&](int u) { return fmaxf(frow * blk.scale[u].x, 1e-30f); };
            float mx = kPfNegInf;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float x[32];
                scores(hf, x);
                mx = fmax3(mx, max16(x) * factor(2 * hf), max16(x + 16) * factor(2 * hf + 1));
            }
            mx = fmaxf(mx, meet(mx, j, ok));
            if (!ok) break;
            m_true = fmaxf(m_true, mx);
            // lazy rescale of O and l when the row maximum grows by more than 2^8, and of O when r is
            // raised; the tensor-memory traffic is warp-collective, so a warp rescales when any of its
            // rows must
            const bool need = mx > m_used + kTcRescale || (m_used == kPfNegInf && mx != kPfNegInf);
            if (__any_sync(0xffffffffu, need) || rnew != rexp) {
                const float f = need && m_used != kPfNegInf ? exp2f(m_used - mx) : 1.f;
                const float fo = f * (rexp - rnew < -126 ? 0.f : pow2i(rexp - rnew));
                rexp = rnew;
                l *= f;
                if ((j & (kPbWindow - 1)) != 0 && __any_sync(0xffffffffu, fo != 1.f)) {
#pragma unroll 1
                    for (int cc = 0; cc < HC / 16; ++cc) {
                        float v[16];
                        tc_ld16(ocol + 16u * cc, v);
                        tc_wait_ld();
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(v[e] * fo);
                        tc_st16(ocol + 16u * cc, o);
                    }
                }
                if (need) m_used = mx;
            }
            const float mu = m_used == kPfNegInf ? 0.f : m_used;
            // w = 2^(x f - mu + lv) in pairs; a masked key (-inf) gives +0. w goes over the scores as
            // two fp16 terms: of 32 keys, hi (the upper 11 bits) into the first 16 columns, lo (the
            // exact rest, rounded) into the others. The sum takes w without its tile's 2^lv.
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float x[32];
                scores(hf, x);
                uint32_t ph[16], pl[16];
#pragma unroll
                for (int uu = 0; uu < 2; ++uu) {
                    const int u = 2 * hf + uu;
                    const float fu = factor(u);
                    const float2 lv = *reinterpret_cast<const float2*>(&blk.scale[u].z);
                    const uint64_t f2 = pack_f32x2(fu, fu);
                    const float nm = lv.x - mu;
                    const uint64_t n2 = pack_f32x2(nm, nm);
                    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
                    for (int cc = 0; cc < 8; ++cc) {
                        float p0, p1;
                        fma_f32x2(x[16 * uu + 2 * cc], x[16 * uu + 2 * cc + 1], f2, n2, p0, p1);
                        p0 = ex2_approx(p0);
                        p1 = ex2_approx(p1);
                        if (cc & 1) add_f32x2(s2, s3, p0, p1);
                        else        add_f32x2(s0, s1, p0, p1);
                        const float g0 = __uint_as_float(__float_as_uint(p0) & 0xffffe000u);
                        const float g1 = __uint_as_float(__float_as_uint(p1) & 0xffffe000u);
                        ph[8 * uu + cc] = pack_f16(g0, g1);
                        float r0, r1;
                        sub_f32x2(p0, p1, g0, g1, r0, r1);
                        pl[8 * uu + cc] = pack_f16(r0, r1);
                    }
                    l = fmaf((s0 + s1) + (s2 + s3), lv.y, l);
                }
                tc_st16(scol + 32u * hf, ph);
                tc_st16(scol + 32u * hf + 16u, pl);
            }
            ring_release(i);
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(bar(kBarP + t));
            ++j;
        }
        // ---- epilogue: this thread's half of the row's O, its maximum and sum -------------------
        if (ok && ns > 0) {
            ok = mbar_wait(bar(kBarDrain), 0, abort_p, p.dev_err);
            tc_fence_after();
        }
        ok = __all_sync(0xffffffffu, ok);
        if (ok) l += meet(l, j, ok);  // the other half's sum
        const bool any = j > 0 && ok;
        // out = (O + earlier windows) 2^rexp / l, the exponent and 1 / l multiplied in turn (either
        // may be far from 1)
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const float up = pow2i(rexp);
        const bool more = ref != kPfNegInf && ok;
        const float down = more ? exp2f(ref - (m_used + (float)rexp)) : 0.f;
        const int64_t row = ((int64_t)b * p.Tq + (rowok ? pos - c0 : 0)) * p.Hq + h0 + q_head(z);
        float* orow = p.out + row * D + HC * hk;
        if (more) __threadfence();  // the row's earlier additions
#pragma unroll 1
        for (int cc = 0; cc < HC / 16; ++cc) {
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
            __syncwarp();
        }
        if (rowok && hk == 0) {
            // report the true row max and the sum relative to it
            if (p.m_out) p.m_out[row] = m_true == kPfNegInf ? kPfNegInf : m_true * kLn2;
            if (p.e_out) p.e_out[row] = m_true == kPfNegInf ? 0.f : l * exp2f(m_used - m_true);
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
int g_pb_smem_set[2] = {0, 0};

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
    const int32_t blocks = (p.Tq + kPfBlock - 1) / kPfBlock + 1;  // query blocks a chunk can touch
    p.nqb = (blocks + pp.nq - 1) / pp.nq;
    const int64_t per_head = (int64_t)p.nqb * (p.g / pp.hp);
    const int64_t pairs = (int64_t)p.B * p.Hkv * per_head;
    const int32_t sms = sm_count_current();
    // a last wave of tile pairs for at most half of the SMs: a CTA for each tile instead
    const int64_t rest = pairs % sms;
    pp.whole = (int32_t)(2 * rest <= sms ? pairs - rest : pairs);
    const int64_t ctas = pp.whole + 2 * (pairs - pp.whole);
    if (pairs >= (1ll << 31) - sms) return DATTN_ERR_UNSUPPORTED;
    // as in prefill.cu: the smallest group of KV heads whose CTAs fill three waves
    p.kv_group = p.Hkv;
    for (int32_t G = 1; G < p.Hkv; ++G)
        if (p.Hkv % G == 0 && G * per_head >= 3ll * sms) {
            p.kv_group = G;
            break;
        }
    const int32_t nwords = (p.max_pages * p.P / kPfBlock + 1 + 4 + 31) / 32;
    const PbSmem L = pb_smem_layout(D, pp.nq, nwords);
    if (L.total > 227u * 1024u) return DATTN_ERR_UNSUPPORTED;
    {
        std::lock_guard<std::mutex> lock(g_pb_mutex);
        int& set = g_pb_smem_set[D == 128 ? 1 : 0];
        if ((int)L.total > set) {
            if (cudaFuncSetAttribute(prefill_block_kernel<D>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)L.total) != cudaSuccess)
                return DATTN_ERR_CUDA;
            set = (int)L.total;
        }
    }
    return launch_pdl(prefill_block_kernel<D>, dim3((unsigned)ctas), dim3(kPbThreads), L.total,
                      stream, pp, nwords) == cudaSuccess
               ? DATTN_OK
               : DATTN_ERR_CUDA;
}

dattn_status_t launch_prefill_block(const PfParams& p, const void* k_pool, const void* v_pool,
                                    const float* kv_scale, int D, cudaStream_t stream) {
    return D == 64 ? launch_d<64>(p, k_pool, v_pool, kv_scale, stream)
                   : launch_d<128>(p, k_pool, v_pool, kv_scale, stream);
}

}  // namespace dattn
