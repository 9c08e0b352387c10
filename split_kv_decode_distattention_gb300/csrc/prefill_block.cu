// Prefill over the block-scaled 8-bit pool (dattn_prefill with DATTN_KV_FP8_BLOCK): a chunk of Tq
// new query tokens per request attends the paged cache, causally or block-sparsely, exactly as over
// the bf16 pool (prefill.cu holds the method's sources and the block rules).
//
// A block scale is a power of two, so a stored value, code * scale, is a bf16 number: the codes
// are widened to bf16 in shared memory, scale included, and the products and the softmax see
// exactly the pool's values.
//
// What bounds it: the tensor cores. A 64-key block of 128 query rows takes one product S = Q K^T
// and two products O += P V (P as two bf16 terms, hi rounded to nearest and lo the rounded rest, so
// the weights keep 17 bits; one term alone would leave 2^-9 in a result that is fp32), 3 x 2 x 128
// x 64 x d operations for the 2 x 2 x 128 x 64 x d that count: 2/3 of the dense bf16 rate at most.
// The widening costs five integer and bf16 instructions for two codes, so a key block is widened
// once for 256 query rows: one CTA per SM holds two tiles of 128 rows, and while one tile is in its
// softmax the tensor cores work on the other.
//
// A CTA: 256 rows as four quarters of 64 tokens: one query block of four heads of a KV head (g a
// multiple of 4), two query blocks of two heads (even g), or four query blocks of one head. A tile
// (two quarters) takes part in a key block only if one of its quarters keeps it. Warps 0-3 and 4-7
// hold one query row per thread (softmax, as in prefill.cu), warps 8-11 load codes, widen them and
// write K and V stages in the 128-byte-swizzled layout of the MMA operands, one thread of warp 12
// issues the products: S of the next key block for both tiles, then P V of this one.
// Tensor memory: O of the two tiles, then two score buffers for each, all 512 columns.
//
// The key blocks of a CTA can be cut over a cluster of 2, 4 or 8 CTAs (launch_prefill_block chooses:
// few tiles, or a last wave that would be nearly empty). Each leaves its rows' O, maximum and sum
// in its shared memory, and each merges a part of the rows from all of them through distributed
// shared memory, with dattn_merge's equations: no workspace.
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "prefill.cuh"

namespace dattn {

namespace {

constexpr int kPbRows = 256;                // query rows of a CTA: two tiles of 128
constexpr int kPbConvWarp = 8;              // warps 8-11 widen the codes
constexpr int kPbConvThreads = 128;
constexpr int kPbMmaWarp = 12;
constexpr int kPbThreads = 13 * 32;
constexpr int kPbStages = 3;                // K stages, and V stages
constexpr int kPbMetaSlots = 8;             // tile lengths of block i in slot i % 8
constexpr uint32_t kPbCols = 512;           // O: [0, 128), [128, 256); S: 256 + 128 tile + 64 buffer

// mbarriers
constexpr int kBarKFull = 0, kBarKEmpty = 3, kBarVFull = 6, kBarVEmpty = 9;
constexpr int kBarS = 12, kBarP = 16;       // + 2 tile + buffer
constexpr int kBarPv = 20;                  // + tile
constexpr int kBarMeta = 22, kBarDrain = 30, kPbBars = 31;

struct PbSmem {
    uint32_t q, blk_bytes, kst, vst, bm, bars, meta, taddr, abort, mrow, trow, lrow, total;
};

__host__ __device__ inline PbSmem pb_smem_layout(int D, int nq, int nwords) {
    PbSmem s;
    uint32_t o = 0;
    s.q = o;           o += (uint32_t)kPbRows * D * 2u;
    s.blk_bytes = 64u * D * 2u;
    s.kst = o;         o += kPbStages * s.blk_bytes;
    s.vst = o;         o += kPbStages * s.blk_bytes;
    s.bm = o;          o += (uint32_t)(nq * nwords) * 4u;
    o = (o + 15u) & ~15u;
    s.bars = o;        o += (kPbBars + 1) * 8u;
    s.meta = o;        o += kPbMetaSlots * 16u;
    s.taddr = o;       o += 16u;
    s.abort = o;       o += 16u;
    s.mrow = o;        o += kPbRows * 4u;  // a split's row references, maxima and sums
    s.trow = o;        o += kPbRows * 4u;
    s.lrow = o;        o += kPbRows * 4u;
    s.total = o;
    return s;
}

struct PbParams {
    PfParams f;
    int32_t hp, nq;  // heads and query blocks of a CTA: hp * nq = 4
    int32_t split;   // CTAs of a cluster that share a CTA's key blocks
    const uint8_t* k_pool;
    const uint8_t* v_pool;
    const float2* scale;  // [num_pages][Hkv][P/16] (K, V)
};

// The key blocks that the two tiles keep: the bitmaps of the CTA's query blocks are bm[i][nwords].
__device__ __forceinline__ uint32_t tile_word(const uint32_t* bm, int nq, int nwords, int t, int w) {
    if (nq == 1) return bm[w];
    if (nq == 2) return bm[t * nwords + w];
    return bm[2 * t * nwords + w] | bm[(2 * t + 1) * nwords + w];
}

// The walk over the key blocks that any tile keeps, in order, from the skip'th on.
struct Walk {
    const uint32_t* bm;
    int nq, nwords, nw, w;
    uint32_t w0, w1, word;
    __device__ __forceinline__ void fetch() {
        w0 = w1 = 0u;
        if (w < nw) {
            w0 = tile_word(bm, nq, nwords, 0, w);
            w1 = tile_word(bm, nq, nwords, 1, w);
        }
        word = w0 | w1;
    }
    __device__ __forceinline__ Walk(const uint32_t* bm_, int nq_, int nwords_, int nw_, int skip)
        : bm(bm_), nq(nq_), nwords(nwords_), nw(nw_), w(0) {
        fetch();
        while (w < nw && __popc(word) <= skip) {
            skip -= __popc(word);
            ++w;
            fetch();
        }
        for (; skip > 0; --skip) word &= word - 1u;
    }
    // The next key block and which tiles keep it (bit t); the caller counts the blocks.
    __device__ __forceinline__ void next(int32_t& kb, uint32_t& act) {
        while (word == 0u && w < nw) {
            ++w;
            fetch();
        }
        const int bit = __ffs(word) - 1;
        kb = 32 * w + bit;
        act = ((w0 >> bit) & 1u) | (((w1 >> bit) & 1u) << 1);
        word &= word - 1u;
    }
};

// Two E4M3 codes (the bytes at 16-bit places 0 and 1 of y's upper bytes) as bf16: sign, exponent and
// mantissa moved into place make code * 2^-120 (subnormal codes too, as subnormal bf16 numbers),
// and m = 2^120 * scale restores them exactly. A NaN code becomes 480 * scale.
__device__ __forceinline__ uint32_t widen2(uint32_t y, __nv_bfloat162 m) {
    const uint32_t v = (y & 0x80008000u) | ((y >> 4) & 0x07f007f0u);
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v), m);
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint4 widen8(uint32_t a, uint32_t b, __nv_bfloat162 m) {
    return make_uint4(widen2(__byte_perm(a, 0u, 0x1404), m), widen2(__byte_perm(a, 0u, 0x3424), m),
                      widen2(__byte_perm(b, 0u, 0x1404), m), widen2(__byte_perm(b, 0u, 0x3424), m));
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

template <int D>
__global__ void __launch_bounds__(kPbThreads, 1)
prefill_block_kernel(const __grid_constant__ PbParams pp, int32_t nwords) {
    constexpr int KH = D / 64;  // 128-byte halves of a bf16 row
    constexpr uint32_t kHalf = 64u * 128u;
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
    // CTA -> (request b, group of kv_group KV heads, tile J, KV head of the group, head slot, rank
    // of its cluster): a group's tiles run together, its last (longest) first
    const int hp = pp.hp, nq = pp.nq;
    const int32_t spk = p.g / hp;
    const int32_t ngrp = p.Hkv / p.kv_group;
    int32_t c = blockIdx.x / pp.split;
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
    int32_t* meta = reinterpret_cast<int32_t*>(base + L.meta);
    uint32_t* bm = reinterpret_cast<uint32_t*>(base + L.bm);
    volatile int* abort_p = reinterpret_cast<volatile int*>(base + L.abort);
    if (tid == 0) {
        for (int s = 0; s < kPbStages; ++s) {
            mbar_init(bar(kBarKFull + s), kPbConvThreads);
            mbar_init(bar(kBarKEmpty + s), 1);
            mbar_init(bar(kBarVFull + s), kPbConvThreads);
            mbar_init(bar(kBarVEmpty + s), 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(kBarS + i), 1);
            mbar_init(bar(kBarP + i), 128);
        }
        mbar_init(bar(kBarPv), 1);
        mbar_init(bar(kBarPv + 1), 1);
        for (int i = 0; i < kPbMetaSlots; ++i) mbar_init(bar(kBarMeta + i), D == 128 ? 1 : 2);
        mbar_init(bar(kBarDrain), 1);
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

    // ---- the CTA's query rows and key blocks (uniform over the cluster) -----------------------
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
        // the query rows, [half][256 rows][128 B] swizzled; with a negative scale they are negated
        // (exact), so that the scores scale by |scale|
        const uint32_t qneg = p.sl2 < 0.f ? 0x80008000u : 0u;
        for (int idx = tid; idx < kPbRows * (D / 8); idx += kPbThreads) {
            const int r = idx / (D / 8), ch = idx - r * (D / 8), z = r >> 6;
            const int32_t pos = (qa + q_block(z)) * kPfBlock + (r & 63);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (((has >> q_block(z)) & 1u) && pos >= c0 && pos < Ln) {
                v = __ldg(reinterpret_cast<const uint4*>(
                    p.q + (((int64_t)b * p.Tq + (pos - c0)) * p.Hq + h0 + q_head(z)) * D) + ch);
                v = make_uint4(v.x ^ qneg, v.y ^ qneg, v.z ^ qneg, v.w ^ qneg);
            }
            *reinterpret_cast<uint4*>(base + L.q + (ch >> 3) * (kPbRows * 128u) +
                                      swz128((uint32_t)r, (uint32_t)(ch & 7))) = v;
        }
        fence_proxy_async_smem();  // the tensor cores read these rows through the async proxy
    }
    __syncthreads();
    // This CTA's share of the key blocks that some row keeps: n blocks from the i0'th on.
    int32_t nall = 0;
    for (int32_t w = 0; w < nw; ++w)
        nall += __popc(tile_word(bm, nq, nwords, 0, w) | tile_word(bm, nq, nwords, 1, w));
    const int32_t rank = pp.split > 1 ? (int32_t)cluster_rank() : 0;
    const int32_t i0 = (int32_t)((int64_t)nall * rank / pp.split);
    const int32_t n = (int32_t)((int64_t)nall * (rank + 1) / pp.split) - i0;

    if (active && warp >= kPbConvWarp && warp < kPbMmaWarp) {
        // ------------------------------------------------------ widening: codes -> K and V stages
        // A row of D codes is D/16 threads of 16 codes; a pass takes RP rows, NP passes a block.
        constexpr int CPR = D / 16, RP = kPbConvThreads / CPR, NP = 64 / RP;
        const int ct = tid - kPbConvWarp * 32, c16 = ct % CPR, rr = ct / CPR;
        const bool teller = (ct & 63) == 0 && (D == 64 || ct == 0);  // publishes its tiles' lengths
        // the upper row half's threads write their two 16-byte chunks in the other order, so that
        // eight neighbours hit all banks
        const bool odd = D == 128 && c16 >= 4;
        Walk walk(bm, nq, nwords, nw, i0);
        auto first_row = [&](int k) { return rr + RP * k; };
        // the pages of this thread's tiles in key block kb, one block ahead of its codes
        auto read_pages = [&](int32_t kb, int32_t (&pg)[NP]) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int32_t t0 = kb * kPfBlock + (first_row(k) & ~15);
                pg[k] = t0 < p_hi ? __ldg(p.block_table + (int64_t)b * p.max_pages + t0 / p.P) : 0;
            }
        };
        int32_t y[NP], hi[NP];  // the tile's first row over all heads (below 2^31), its tokens
        auto resolve = [&](int32_t kb, const int32_t (&pg)[NP]) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int32_t t0 = kb * kPfBlock + (first_row(k) & ~15);
                y[k] = hi[k] = 0;
                if (t0 >= p_hi) continue;
                if (pg[k] < 0 || pg[k] >= p.num_pages) {
                    if (teller)
                        set_err(p.dev_err, pg[k] < 0 ? DATTN_DEVERR_UNMAPPED_PAGE
                                                     : DATTN_DEVERR_PAGE_OOB);
                    continue;
                }
                y[k] = (pg[k] * p.Hkv + kvh) * p.P + (t0 - (t0 / p.P) * p.P);
                hi[k] = min(16, Ln - t0);
            }
        };
        // 16 codes a row; rows that hold no token of the request are zeros
        auto load = [&](const uint8_t* pool, uint4 (&v)[NP]) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int r = first_row(k) & 15;
                v[k] = make_uint4(0u, 0u, 0u, 0u);
                if (r < hi[k])
                    v[k] = __ldg(reinterpret_cast<const uint4*>(pool + (int64_t)(y[k] + r) * D + 16 * c16));
            }
        };
        auto load_scales = [&](float (&ks)[NP], float (&vs)[NP]) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const float2 s = hi[k] > 0 ? __ldg(pp.scale + (y[k] >> 4)) : make_float2(0.f, 0.f);
                ks[k] = s.x;
                vs[k] = s.y;
            }
        };
        auto store = [&](uint8_t* st, const uint4 (&v)[NP], const float (&sc)[NP]) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                // 2^120 * scale, in two steps above 2^7 (2^127 is bf16's largest power)
                const __nv_bfloat162 m =
                    __float2bfloat162_rn(fminf(sc[k], 128.f) * 1.329227995784916e36f);
                uint4 a = odd ? widen8(v[k].z, v[k].w, m) : widen8(v[k].x, v[k].y, m);
                uint4 c2 = odd ? widen8(v[k].x, v[k].y, m) : widen8(v[k].z, v[k].w, m);
                if (sc[k] > 128.f) {
                    const __nv_bfloat162 m2 = __float2bfloat162_rn(sc[k] * 0.0078125f);
                    uint32_t* w = reinterpret_cast<uint32_t*>(&a);
                    uint32_t* w2 = reinterpret_cast<uint32_t*>(&c2);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        __nv_bfloat162 t = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&w[i]), m2);
                        w[i] = *reinterpret_cast<uint32_t*>(&t);
                        t = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&w2[i]), m2);
                        w2[i] = *reinterpret_cast<uint32_t*>(&t);
                    }
                }
                const uint32_t row = (uint32_t)first_row(k), ch = 2u * (c16 & 3) + (odd ? 1u : 0u);
                uint8_t* half = st + (c16 >> 2) * kHalf;
                *reinterpret_cast<uint4*>(half + swz128(row, ch)) = a;
                *reinterpret_cast<uint4*>(half + swz128(row, ch ^ 1u)) = c2;
            }
        };
        int32_t kb = 0, kb2 = 0, pg[NP];
        uint32_t act;
        uint4 kv[NP], vv[NP];
        float ks[NP], vs[NP], vs2[NP];
        if (n > 0) {
            walk.next(kb, act);
            read_pages(kb, pg);
            resolve(kb, pg);
            load_scales(ks, vs);
            load(pp.k_pool, kv);
            load(pp.v_pool, vv);
            if (n > 1) {
                walk.next(kb2, act);
                read_pages(kb2, pg);
            }
        }
        bool ok = true;
        for (int32_t i = 0; i < n && ok; ++i) {
            const int s = i % kPbStages, ph = (i / kPbStages) & 1;
            if (i >= kPbStages) ok = mbar_wait(bar(kBarKEmpty + s), ph ^ 1, abort_p, p.dev_err);
            if (!ok) break;
            if (teller) {  // (the readers of block i - 8's lengths are done: P V of block i - 4 is)
#pragma unroll
                for (int k = 0; k < NP; ++k)
                    meta[4 * (i & (kPbMetaSlots - 1)) + (first_row(k) >> 4)] = hi[k];
                mbar_arrive(bar(kBarMeta + (i & (kPbMetaSlots - 1))));
            }
            store(base + L.kst + (uint32_t)s * L.blk_bytes, kv, ks);
            fence_proxy_async_smem();
            mbar_arrive(bar(kBarKFull + s));
            // the next block: its places, and its K on the way while this block's V is widened
            const bool more = i + 1 < n;
            if (more) {
                resolve(kb2, pg);
                load_scales(ks, vs2);
                load(pp.k_pool, kv);
            }
            if (i >= kPbStages) ok = mbar_wait(bar(kBarVEmpty + s), ph ^ 1, abort_p, p.dev_err);
            if (!ok) break;
            store(base + L.vst + (uint32_t)s * L.blk_bytes, vv, vs);
            fence_proxy_async_smem();
            mbar_arrive(bar(kBarVFull + s));
            if (more) {
                load(pp.v_pool, vv);
#pragma unroll
                for (int k = 0; k < NP; ++k) vs[k] = vs2[k];
                if (i + 2 < n) {
                    walk.next(kb2, act);
                    read_pages(kb2, pg);
                }
            }
        }
    } else if (active && warp == kPbMmaWarp) {
        // ---------------------------------------------------------------- MMA issuer
        if (lane == 0 && n > 0) {
            constexpr uint32_t idesc_s = tc_idesc(128, 64, 0);
            constexpr uint32_t idesc_o = tc_idesc(128, D, 1);
            const uint32_t qs = smem_u32(base + L.q);
            const uint32_t kst0 = smem_u32(base + L.kst), vst0 = smem_u32(base + L.vst);
            bool ok = true;
            int32_t j[2] = {0, 0};  // each tile's blocks so far
            uint32_t act = 0u, prev = 0u;
            int32_t kb;
            Walk walk(bm, nq, nwords, nw, i0);
            for (int32_t i = 0; i <= n && ok; ++i) {
                // S of block i: tile t's j'th scores into its buffer j % 2 (whose P V, of its block
                // j - 2, was issued before: products run in order)
                prev = act;
                act = 0u;
                if (i < n) {
                    walk.next(kb, act);
                    const int s = i % kPbStages;
                    ok = mbar_wait(bar(kBarKFull + s), (i / kPbStages) & 1, abort_p, p.dev_err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t kst = kst0 + (uint32_t)s * L.blk_bytes;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!((act >> t) & 1u)) continue;
                        const int buf = j[t] & 1;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t ad = tc_sdesc(qs + (kk >> 2) * (kPbRows * 128u) +
                                                             t * (128u * 128u) + (kk & 3) * 32u,
                                                         16u, 1024u);
                            const uint64_t bd =
                                tc_sdesc(kst + (kk >> 2) * kHalf + (kk & 3) * 32u, 16u, 1024u);
                            tc_mma_ss(tbase + 256u + 128u * t + 64u * buf, ad, bd, idesc_s,
                                      kk > 0 ? 1u : 0u);
                        }
                        tc_commit(bar(kBarS + 2 * t + buf));
                        ++j[t];
                    }
                    tc_commit(bar(kBarKEmpty + s));
                }
                if (i == 0) continue;
                // O += P V of block i - 1: P from tensor memory (hi terms, then lo), V from shared
                const int sv = (i - 1) % kPbStages;
                ok = mbar_wait(bar(kBarVFull + sv), ((i - 1) / kPbStages) & 1, abort_p, p.dev_err);
                const uint32_t vst = vst0 + (uint32_t)sv * L.blk_bytes;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (!((prev >> t) & 1u) || !ok) continue;
                    const int32_t jt = j[t] - 1 - (int32_t)((act >> t) & 1u);  // its number
                    const int buf = jt & 1;
                    ok = mbar_wait(bar(kBarP + 2 * t + buf), (jt >> 1) & 1, abort_p, p.dev_err);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint64_t bd = tc_sdesc(vst + kk * 2048u, kHalf, 1024u);
                            tc_mma_ts(tbase + 128u * t,
                                      tbase + 256u + 128u * t + 64u * buf + 32u * part + 8u * kk, bd,
                                      idesc_o, (jt > 0 || part > 0 || kk > 0) ? 1u : 0u);
                        }
                    }
                    tc_commit(bar(kBarPv + t));
                }
                tc_commit(bar(kBarVEmpty + sv));
            }
            // every product is done: the epilogue's signal, and nothing of this CTA's may still run
            // on the tensor cores when it exits
            tc_commit(bar(kBarDrain));
            mbar_wait(bar(kBarDrain), 0, abort_p, p.dev_err);
        }
    } else if (active && warp < 8) {
        // ---------------------------------------------------------------- softmax threads
        const int t = warp >> 2, r = tid, z = r >> 6;  // tile, row and quarter
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int qi = q_block(z);
        const int32_t pos = (qa + qi) * kPfBlock + (r & 63);
        const bool rowok = ((has >> qi) & 1u) && pos >= c0 && pos < Ln;
        const uint32_t* mine = bm + qi * nwords;
        // |scale| log2(e), at least 1e-30 so that a masked key (-inf) never meets a zero factor
        const float sl2a = fmaxf(fabsf(p.sl2), 1e-30f);
        float m_used = kPfNegInf, m_true = kPfNegInf, l = 0.f;  // l is relative to m_used
        int32_t j = 0;  // this tile's blocks
        bool ok = true;
        Walk walk(bm, nq, nwords, nw, i0);
        for (int32_t i = 0; i < n; ++i) {
            int32_t kb;
            uint32_t act;
            walk.next(kb, act);
            if (!((act >> t) & 1u)) continue;
            const int buf = j & 1, ms = i & (kPbMetaSlots - 1);
            ok = mbar_wait(bar(kBarMeta + ms), (i / kPbMetaSlots) & 1, abort_p, p.dev_err) &&
                 mbar_wait(bar(kBarS + 2 * t + buf), (j >> 1) & 1, abort_p, p.dev_err);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int4 his = *reinterpret_cast<const int4*>(meta + 4 * ms);
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
                tc_wait_ld();
            }
            // mask: the row's query block keeps kb, the key is written and at or before the query.
            // Key e of tile u is kept iff e < lim[u]; a block whose keys all pass for every row of
            // the warp skips the selects.
            const bool keep = rowok && ((mine[kb >> 5] >> (kb & 31)) & 1u);
            const int32_t cut = keep ? pos - kb * kPfBlock + 1 : 0;
            float mxr;  // the row maximum of the raw scores
            if (__all_sync(0xffffffffu, cut >= kPfBlock &&
                                            (his.x + his.y + his.z + his.w) == kPfBlock)) {
                mxr = row_max64(x);
            } else {
                const int32_t lim[4] = {min(his.x, cut), min(16 + his.y, cut), min(32 + his.z, cut),
                                        min(48 + his.w, cut)};
#pragma unroll
                for (int e = 0; e < 64; ++e) x[e] = e < lim[e >> 4] ? x[e] : kPfNegInf;
                mxr = row_max64(x);
            }
            const float mx = mxr * sl2a;  // scaled (log2 units); -inf stays -inf
            m_true = fmaxf(m_true, mx);
            // lazy rescale of O and l when the row maximum grows by more than 2^8; the tensor-memory
            // traffic is warp-collective, so a warp rescales when any of its rows must
            const bool need = mx > m_used + kTcRescale || (m_used == kPfNegInf && mx != kPfNegInf);
            const float f = need && m_used != kPfNegInf ? exp2f(m_used - mx) : 1.f;
            if (__any_sync(0xffffffffu, f != 1.f) && j > 0) {
                // O holds the blocks before this one: wait for them, then scale it
                mbar_wait(bar(kBarPv + t), (j - 1) & 1, abort_p, p.dev_err);
                tc_fence_after();
#pragma unroll 1
                for (int cc = 0; cc < D / 16; ++cc) {  // (16 columns: the scores stay in registers)
                    float v[16];
                    tc_ld16(tbase + lanes + 128u * t + 16u * cc, v);
                    tc_wait_ld();
                    uint32_t u[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(v[e] * f);
                    tc_st16(tbase + lanes + 128u * t + 16u * cc, u);
                }
                tc_wait_st();
            }
            if (need) m_used = mx;
            const float mu = m_used == kPfNegInf ? 0.f : m_used;
            // p = 2^(x |scale| log2(e) - mu) in pairs; a masked key (-inf) gives +0. P goes to the
            // score buffer as two bf16 terms: hi (rounded) into columns [0, 32), lo (the rest,
            // rounded) into [32, 64).
            const uint64_t s2 = pack_f32x2(sl2a, sl2a), nmu2 = pack_f32x2(-mu, -mu);
            float ls[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t ph[16], pl[16];
#pragma unroll
                for (int cc = 0; cc < 16; ++cc) {
                    float p0, p1;
                    fma_f32x2(x[32 * hf + 2 * cc], x[32 * hf + 2 * cc + 1], s2, nmu2, p0, p1);
                    p0 = ex2_approx(p0);
                    p1 = ex2_approx(p1);
                    add_f32x2(ls[2 * (cc & 3)], ls[2 * (cc & 3) + 1], p0, p1);
                    ph[cc] = pack_bf16(p0, p1);
                    float r0, r1;
                    sub_f32x2(p0, p1, bf16_lo(ph[cc]), bf16_hi(ph[cc]), r0, r1);
                    pl[cc] = pack_bf16(r0, r1);
                }
                tc_st16(sbuf + 16u * hf, ph);
                tc_st16(sbuf + 32u + 16u * hf, pl);
            }
            l = l * f + (((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7])));
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(bar(kBarP + 2 * t + buf));
            ++j;
        }
        // ---- epilogue: this row's O, maximum and sum ------------------------------------------
        if (ok && n > 0) {
            ok = mbar_wait(bar(kBarDrain), 0, abort_p, p.dev_err);
            tc_fence_after();
        }
        ok = __all_sync(0xffffffffu, ok);
        const bool any = j > 0 && ok;
        const int64_t row = ((int64_t)b * p.Tq + (rowok ? pos - c0 : 0)) * p.Hq + h0 + q_head(z);
        float* orow = p.out + row * D;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        // a split leaves its unnormalised rows in shared memory (every stage and the query rows are
        // done with), padded so that the rows of a quarter warp lie in different banks
        float* srow = reinterpret_cast<float*>(base) + r * (D + 4);
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
            float v[32];
            if (any) {
                tc_ld32(tbase + lanes + 128u * t + 32u * cc, v);
                tc_wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = 0.f;
            }
            if (pp.split > 1) {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4*>(srow + 32 * cc + e) =
                        make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            } else if (rowok) {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<float4*>(orow + 32 * cc + e) =
                        make_float4(v[e] * inv, v[e + 1] * inv, v[e + 2] * inv, v[e + 3] * inv);
            }
        }
        if (pp.split > 1) {
            // the sum and O are relative to m_used
            reinterpret_cast<float*>(base + L.mrow)[r] = l > 0.f ? m_used : kPfNegInf;
            reinterpret_cast<float*>(base + L.trow)[r] = m_true;
            reinterpret_cast<float*>(base + L.lrow)[r] = l;
        } else if (rowok) {
            // report the true row max and the sum relative to it
            if (p.m_out) p.m_out[row] = m_true == kPfNegInf ? kPfNegInf : m_true * kLn2;
            if (p.e_out) p.e_out[row] = m_true == kPfNegInf ? 0.f : l * exp2f(m_used - m_true);
        }
    }
    if (pp.split > 1) {
        // ---- merge the cluster's parts: rank k takes every split'th row from the k'th on -------
        // (an inactive CTA's cluster is inactive as a whole; all pass the barriers)
        cluster_sync();
        if (active) {
            const uint32_t o0 = smem_u32(base), m0 = smem_u32(base + L.mrow);
            const uint32_t t0 = smem_u32(base + L.trow), l0 = smem_u32(base + L.lrow);
            constexpr int TPR = D / 4;  // threads of a row, a float4 each
            for (int x = tid; x < kPbRows / pp.split * TPR; x += kPbThreads) {
                const int r = x / TPR * pp.split + rank, d4 = x % TPR, z = r >> 6;
                const int qi = q_block(z);
                const int32_t pos = (qa + qi) * kPfBlock + (r & 63);
                if (!((has >> qi) & 1u) || pos < c0 || pos >= Ln) continue;
                float mg = kPfNegInf;
                for (int k = 0; k < pp.split; ++k)
                    mg = fmaxf(mg, ld_cluster(map_rank(m0 + 4u * r, k)));
                float e = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < pp.split && mg != kPfNegInf; ++k) {
                    const float mk = ld_cluster(map_rank(m0 + 4u * r, k));
                    if (mk == kPfNegInf) continue;
                    const float w = exp2f(mk - mg);
                    e += w * ld_cluster(map_rank(l0 + 4u * r, k));
                    const float4 v = ld_cluster4(map_rank(o0 + 4u * (r * (D + 4) + 4 * d4), k));
                    o.x += w * v.x;
                    o.y += w * v.y;
                    o.z += w * v.z;
                    o.w += w * v.w;
                }
                const float inv = e > 0.f ? 1.f / e : 0.f;
                const int64_t row = ((int64_t)b * p.Tq + (pos - c0)) * p.Hq + h0 + q_head(z);
                *reinterpret_cast<float4*>(p.out + row * D + 4 * d4) =
                    make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                if (d4 == 0 && (p.m_out || p.e_out)) {
                    float mt = kPfNegInf;  // the true row max; e moves to it
                    for (int k = 0; k < pp.split; ++k)
                        mt = fmaxf(mt, ld_cluster(map_rank(t0 + 4u * r, k)));
                    if (p.m_out) p.m_out[row] = mt == kPfNegInf ? kPfNegInf : mt * kLn2;
                    if (p.e_out) p.e_out[row] = mt == kPfNegInf ? 0.f : e * exp2f(mg - mt);
                }
            }
        }
        cluster_sync();  // no CTA's shared memory goes away while another reads it
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
    const int64_t tiles = (int64_t)p.B * p.Hkv * per_head;
    const int32_t sms = sm_count_current();
    pp.split = 1;
    if (tiles * pp.split >= (1ll << 31)) return DATTN_ERR_UNSUPPORTED;
    // as in prefill.cu: the smallest group of KV heads whose CTAs fill three waves
    p.kv_group = p.Hkv;
    for (int32_t G = 1; G < p.Hkv; ++G)
        if (p.Hkv % G == 0 && G * per_head * pp.split >= 3ll * sms) {
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * pp.split));
    cfg.blockDim = dim3(kPbThreads);
    cfg.dynamicSmemBytes = L.total;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)pp.split, 1u, 1u};
    cfg.attrs = attr;
    cfg.numAttrs = pp.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, prefill_block_kernel<D>, pp, nwords) == cudaSuccess
               ? DATTN_OK
               : DATTN_ERR_CUDA;
}

dattn_status_t launch_prefill_block(const PfParams& p, const void* k_pool, const void* v_pool,
                                    const float* kv_scale, int D, cudaStream_t stream) {
    return D == 64 ? launch_d<64>(p, k_pool, v_pool, kv_scale, stream)
                   : launch_d<128>(p, k_pool, v_pool, kv_scale, stream);
}

}  // namespace dattn
