// Attention of many query rows over the paged cache on the 5th-generation tensor cores, as a persistent
// kernel: what the windowed prefill (window_prefill.cu) and the shared prefixes (shared.cu) have in common.
//
// A tile is up to 128 rows: kTok = 128 / g consecutive query tokens times the g query heads of a KV head
// (row = token * g + head), so that a key block is read once for all heads of its KV head. A CTA per SM
// holds two tiles, which work past each other: while the softmax of one runs, the tensor cores compute the
// other's products. An item is a pair of tiles over a run of 64-key blocks, or one tile, of which the CTA's
// two tiles take every other block each (`alt`) and join their sums in tensor memory at the end. A CTA
// walks its items without a barrier between them: the copies of the next item's queries and keys run
// during this one's softmax and epilogue. 16 warps:
//   0-3, 4-7  one row per thread of tile 0, 1: scores out of tensor memory, masks, the online softmax in
//             base 2 on packed fp32 pairs, and the weights back as two bf16 terms (p cut to its upper 16
//             bits, and the exact rest, rounded), which the second product reads; the accumulator is
//             rescaled only when a row's maximum rises by more than 2^8;
//   8-11      bf16 pool: warps 8 and 10 copy K, 9 and 11 V by TMA. Block-scaled pool: all four widen the
//             codes that warp 15 copied to code * scale, which is a bf16 number: both formats compute alike;
//   12, 13    tile 0, 1: S = Q K^T of the next block, then O += P V of this one, issued by one lane;
//   14        the queries, by TMA.
// Tensor memory: O of the two tiles, then two score buffers for each, all 512 columns.
//
// A job says which items a CTA has (next), which blocks of a pair's a tile keeps (keeps), what a row sees
// (row) and what becomes of its sum (begin_row, write16, finish_row).
#pragma once

#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "prefill.cuh"

namespace dattn {

namespace {

constexpr int kTaThreads = 16 * 32;
constexpr int kTaConvWarp = 8;       // warps 8-11
constexpr int kTaConvThreads = 128;
constexpr int kTaMmaWarp = 12;       // warps 12, 13
constexpr int kTaQWarp = 14;
constexpr int kTaCodeWarp = 15;
constexpr int kTaMeta = 16;          // blocks' metadata slots

// Stages of a key block's K and of its V (bf16 rows), and of its codes (block-scaled pool). A wait tells
// the phase at hand from the one before, so whoever fills (or reads) a stage has to have waited for its
// use before. Two warps fill the bf16 stages in turn, and an alt item's tiles read every other block: the
// numbers of bf16 stages are even, so that a stage has one of the warps, and within an item one of the
// tiles, to itself.
__host__ __device__ constexpr int ta_kstages(int fmt) { return fmt == DATTN_KV_BF16 ? 4 : 2; }
__host__ __device__ constexpr int ta_vstages(int fmt) { return fmt == DATTN_KV_BF16 ? 4 : 3; }
__host__ __device__ constexpr int ta_cstages(int fmt) { return fmt == DATTN_KV_BF16 ? 0 : 4; }

struct TaSmem {
    uint32_t q, kst, vst, cst, blk_bytes, code_bytes, scales, bars, meta, ml, taddr, abort, job, total;
};

__host__ __device__ inline TaSmem ta_smem_layout(int D, int fmt, uint32_t job_bytes) {
    TaSmem s;
    uint32_t o = 0;
    s.q = o;        o += 256u * D * 2u;  // [half][256 rows][128 B]
    s.blk_bytes = 64u * D * 2u;
    s.code_bytes = 64u * D;
    s.kst = o;      o += ta_kstages(fmt) * s.blk_bytes;
    s.vst = o;      o += ta_vstages(fmt) * s.blk_bytes;
    s.cst = o;      o += ta_cstages(fmt) * 2u * s.code_bytes;
    s.scales = o;   o += ta_cstages(fmt) * 48u;  // four (K, V) scales, then the tiles' tokens
    s.bars = o;     o += 96u * 8u;
    s.meta = o;     o += kTaMeta * 8u;
    s.ml = o;       o += 2u * 128u * 16u;
    s.taddr = o;    o += 16u;
    s.abort = o;    o += 16u;
    s.job = o;      o += job_bytes;
    s.total = o;
    return s;
}

// mbarriers
constexpr int kTaKFull = 0, kTaKEmpty = 5, kTaVFull = 10, kTaVEmpty = 15, kTaCFull = 20, kTaCEmpty = 25;
constexpr int kTaS = 30, kTaP = 34;  // + 2 tile + buffer
constexpr int kTaPv = 38, kTaQFull = 40, kTaQEmpty = 41, kTaDrain = 42;  // Pv, Drain: + tile
constexpr int kTaMetaFull = 44, kTaMetaEmpty = kTaMetaFull + kTaMeta;
static_assert(kTaMetaEmpty + kTaMeta <= 96, "the barriers' place");

struct TaParams {
    int32_t num_pages, Hkv, P, max_pages;
    const int32_t* block_table;
    int32_t Hq, g, tok;   // tok: query tokens of a tile
    int32_t box;          // rows of a copy: 16, 32 or 64, a divisor of P
    float sl2;            // scale * log2(e)
    const float2* scale;  // block-scaled pool: [num_pages][Hkv][P/16] (K, V)
    int32_t* dev_err;
};

struct TaItem {
    int32_t n0;                  // its first query token (row of q: request * T + token)
    int32_t tok[2];              // query tokens of tile 0, 1 (alt: of tile 0, and none)
    int32_t kvh, trow;           // KV head; row of the block table
    int32_t first, from, count;  // its key blocks: [0, first), then from `from` on, `count` in all
    int32_t kmax;                // keys from kmax on do not exist
    int32_t low, sinks;          // its rows see no key below `low` but those below `sinks`
    int32_t alt;
    int32_t last[2];             // the last of its blocks (by number) that tile 0, 1 keeps; -1: none
    __device__ int32_t block(int32_t j) const { return j < first ? j : from + (j - first); }
};

// What a row sees: the keys below lim that are at least `low` or below `sinks`.
struct TaRow {
    bool ok;
    int32_t lim, low, sinks;
};

// Bits 0 .. n - 1 (n of any sign and size).
__device__ __forceinline__ uint64_t below64(int32_t n) {
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// Two fp16 values times a packed pair of factors, as bf16 values (exact for codes and powers of two).
__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t h, uint64_t f) {
    float a, b;
    asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%2, %3};\n\tmul.rn.f32x2 x, x, %4;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(a), "=f"(b)
        : "f"(f16_lo(h)), "f"(f16_hi(h)), "l"(f));
    return pack_bf16(a, b);
}

template <class Job, int D, int FMT>
__global__ void __launch_bounds__(kTaThreads, 1)
tile_attention_kernel(const __grid_constant__ TaParams p, const __grid_constant__ typename Job::Params jp,
                      const __grid_constant__ CUtensorMap tmap_q,
                      const __grid_constant__ CUtensorMap tmap_k,
                      const __grid_constant__ CUtensorMap tmap_v) {
    constexpr int KH = D / 64;
    constexpr bool BLK = FMT == DATTN_KV_FP8_BLOCK;
    constexpr int NK = ta_kstages(FMT), NV = ta_vstages(FMT), NC = BLK ? ta_cstages(FMT) : 1;
    static_assert(NK <= 5 && NV <= 5 && NC <= 5, "the barriers' place");
    static_assert(BLK || (NK % 2 == 0 && NV % 2 == 0), "a stage belongs to one of two warps");
    static_assert(NK % 2 == 0 && kTaMeta % 2 == 0, "within an alt item, to one tile");
    constexpr uint32_t kHalf = 64u * 128u;  // a 128-byte half of a key block's rows
    constexpr int32_t kFull = 16 | (16 << 5) | (16 << 10) | (16 << 15);  // tokens of a whole block's tiles
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw;
    const TaSmem L = ta_smem_layout(D, FMT, 0u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the 128-byte swizzle of the TMA copies and the MMA operands needs 1024-byte alignment
    if ((smem_u32(base) & 1023u) != 0u) {
        if (tid == 0) set_err(p.dev_err, DATTN_DEVERR_SMEM_ALIGN);
        Job::skip();
        return;
    }
    const uint32_t bars = smem_u32(base + L.bars);
    auto bar = [&](int i) { return bars + 8u * i; };
    int2* meta = reinterpret_cast<int2*>(base + L.meta);  // (block, its tiles' tokens, 5 bits each)
    volatile int* abort_p = reinterpret_cast<volatile int*>(base + L.abort);
    if (tid == 0) {
        for (int s = 0; s < NK; ++s) {
            mbar_init(bar(kTaKFull + s), BLK ? kTaConvThreads : 1);
            mbar_init(bar(kTaKEmpty + s), 2);
        }
        for (int s = 0; s < NV; ++s) {
            mbar_init(bar(kTaVFull + s), BLK ? kTaConvThreads : 1);
            mbar_init(bar(kTaVEmpty + s), 2);
        }
        for (int s = 0; s < NC; ++s) {
            mbar_init(bar(kTaCFull + s), 1);
            mbar_init(bar(kTaCEmpty + s), kTaConvThreads / 32);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(kTaS + i), 1);
            mbar_init(bar(kTaP + i), 128);
        }
        mbar_init(bar(kTaPv), 1);
        mbar_init(bar(kTaPv + 1), 1);
        mbar_init(bar(kTaDrain), 1);
        mbar_init(bar(kTaDrain + 1), 1);
        mbar_init(bar(kTaQFull), 1);
        mbar_init(bar(kTaQEmpty), 2);
        for (int i = 0; i < kTaMeta; ++i) {
            mbar_init(bar(kTaMetaFull + i), 1);
            mbar_init(bar(kTaMetaEmpty + i), 8);
        }
        *abort_p = 0;
        fence_mbar_init();
    }
    if (warp == kTaQWarp && lane == 0) {
        prefetch_tmap(&tmap_q);
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    __syncwarp();  // (tcgen05 instructions take whole, converged warps)
    if (warp == 0) {  // the whole warp allocates the CTA's tensor memory
        tc_alloc(smem_u32(base + L.taddr), 512u);
        tc_relinquish();
    }
    // Rows of the queries that no copy fills (128 is no multiple of g) compute, on zeros.
    if (128 % p.g != 0)
        for (uint32_t i = tid; i < 256u * D * 2u / 16u; i += kTaThreads)
            reinterpret_cast<uint4*>(base + L.q)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    tc_fence_before();
    Job job(p, jp, base + L.job);  // (waits for the previous kernel where the job reads its results)
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(base + L.taddr);
    auto wait = [&](uint32_t bar_addr, uint32_t parity) {  // by a whole warp, one answer
        return __all_sync(0xffffffffu, mbar_wait(bar_addr, parity, abort_p, p.dev_err)) != 0;
    };

    TaItem it;
    bool ok = true;
    uint32_t done = 0u;  // key blocks of earlier items: block i is in K stage i % NK
    if (warp < 8) {
        // -------------------------------------------------------------------- softmax threads
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ocol = tbase + lanes + 128u * t, xcol = tbase + lanes + 128u * (t ^ 1);
        float4* ml = reinterpret_cast<float4*>(base + L.ml);
        // |scale| log2(e), at least 1e-30 so that a masked key (-inf) never meets a zero factor
        const float sl2a = fmaxf(fabsf(p.sl2), 1e-30f);
        uint32_t j = 0u, held = 0u;  // blocks that the tile kept; items of which it kept some
        // (after an abort a warp still walks the items: all meet at the barriers of the alt ones)
        while (job.next(it)) {
            TaRow row;
            job.row(it, t, r, row);
            const int32_t lim = row.lim, low = row.low, sinks = row.sinks;
            float m_used = kPfNegInf, m_true = kPfNegInf, l = 0.f;  // l and O are relative to m_used
            uint32_t n = 0u;  // the item's blocks so far
            for (int32_t b = it.alt ? t : 0; b < it.count && ok; b += it.alt ? 2 : 1) {
                const uint32_t i = done + b, ms = i % kTaMeta;
                ok = wait(bar(kTaMetaFull + ms), (i / kTaMeta) & 1);
                if (!ok) break;
                const int2 mt = meta[ms];
                __syncwarp();
                if (lane < (it.alt ? 2 : 1)) mbar_arrive(bar(kTaMetaEmpty + ms));
                if (!it.alt && !job.keeps(it, t, mt.x)) continue;
                ok = wait(bar(kTaS + 2 * t) + 8u * (j & 1u), (j >> 1) & 1u);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sbuf = tbase + lanes + 256u + 128u * t + 64u * (j & 1u);
                float xs[64];
                {
                    float v[32];
                    tc_ld32(sbuf, v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) xs[e] = v[e];
                    tc_ld32(sbuf + 32u, v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) xs[32 + e] = v[e];
                    tc_wait_ld();
                }
                // Key e of the block is seen if it exists, e < cut, and e >= from or e < sk. A block
                // whose 64 keys all are by every row of the warp skips the selects.
                const int32_t k0 = mt.x * kPfBlock, cut = lim - k0, from = low - k0, sk = sinks - k0;
                if (!__all_sync(0xffffffffu, cut >= kPfBlock && mt.y == kFull &&
                                                 (from <= 0 || sk >= kPfBlock))) {
                    uint64_t see = below64(cut) & (~below64(from) | below64(sk));
                    if (mt.y != kFull) {
                        uint64_t held = 0ull;
#pragma unroll
                        for (int u = 0; u < kPfTiles; ++u)
                            held |= below64((mt.y >> (5 * u)) & 31) << (16 * u);
                        see &= held;
                    }
                    const uint32_t s0 = (uint32_t)see, s1 = (uint32_t)(see >> 32);
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        xs[e] = ((e < 32 ? s0 : s1) >> (e & 31)) & 1u ? xs[e] : kPfNegInf;
                }
                const float mx = row_max64(xs) * sl2a;  // log2 units; -inf stays -inf
                m_true = fmaxf(m_true, mx);
                const bool need =
                    mx > m_used + kTcRescale || (m_used == kPfNegInf && mx != kPfNegInf);
                const float f = need && m_used != kPfNegInf ? exp2f(m_used - mx) : 1.f;
                if (__any_sync(0xffffffffu, f != 1.f) && n > 0u) {
                    // O holds the item's blocks before this one: wait for them, then scale it. (P V of
                    // the tile's block j - 2 ended before these scores were made, so that the barrier is
                    // at most one phase behind, which its parity can tell.)
                    ok = wait(bar(kTaPv) + 8u * t, (j - 1u) & 1u);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < D / 16; ++cc) {
                        float v[16];
                        tc_ld16(ocol + 16u * cc, v);
                        tc_wait_ld();
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(v[e] * f);
                        tc_st16(ocol + 16u * cc, o);
                    }
                    tc_wait_st();
                }
                if (need) m_used = mx;
                const float mu = m_used == kPfNegInf ? 0.f : m_used;
                // p = 2^(x |scale| log2(e) - mu) in pairs; a masked key gives +0
                const uint64_t s2 = pack_f32x2(sl2a, sl2a), nmu2 = pack_f32x2(-mu, -mu);
                float ls[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t ph[16], pl[16];
#pragma unroll
                    for (int cc = 0; cc < 16; ++cc) {
                        float p0, p1;
                        fma_f32x2(xs[32 * hf + 2 * cc], xs[32 * hf + 2 * cc + 1], s2, nmu2, p0, p1);
                        p0 = ex2_approx(p0);
                        p1 = ex2_approx(p1);
                        add_f32x2(ls[2 * (cc & 3)], ls[2 * (cc & 3) + 1], p0, p1);
                        const uint32_t b0 = __float_as_uint(p0), b1 = __float_as_uint(p1);
                        ph[cc] = __byte_perm(b0, b1, 0x7632);
                        float r0, r1;
                        sub_f32x2(p0, p1, __uint_as_float(b0 & 0xffff0000u),
                                  __uint_as_float(b1 & 0xffff0000u), r0, r1);
                        pl[cc] = pack_bf16(r0, r1);
                    }
                    tc_st16(sbuf + 16u * hf, ph);
                    tc_st16(sbuf + 32u + 16u * hf, pl);
                }
                l = l * f + (((ls[0] + ls[1]) + (ls[2] + ls[3])) + ((ls[4] + ls[5]) + (ls[6] + ls[7])));
                tc_wait_st();
                if (!BLK) {
                    // V rows of keys that do not exist hold other tokens or nothing: zeros, so that a zero
                    // weight cannot meet a NaN (P V of this block waits for this warp, and the stage's
                    // next use for P V)
                    if (mt.y != kFull && wait(bar(kTaVFull + i % NV), (i / NV) & 1)) {
                        uint8_t* vst = base + L.vst + (i % NV) * L.blk_bytes;
                        for (int idx = r; idx < 64 * KH * 8; idx += 128) {
                            const int kr = idx / (KH * 8), rem = idx - kr * (KH * 8);
                            const int hh = rem >> 3, ch = rem & 7;
                            if ((kr & 15) >= ((mt.y >> (5 * (kr >> 4))) & 31))
                                *reinterpret_cast<uint4*>(vst + hh * kHalf + kr * 128 + ch * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                }
                __syncwarp();
                tc_fence_before();
                mbar_arrive(bar(kTaP + 2 * t) + 8u * (j & 1u));
                ++j;
                ++n;
            }
            done += it.count;
            // ---- the rows' results, when the item's products are done: a phase for each item of which
            // the tile keeps a block, so that none ends before this warp gave the item's last weights.
            // (P V's own barrier may have gone on by one phase or by two, which its parity cannot tell.)
            if (n > 0u) {
                if (ok) ok = wait(bar(kTaDrain) + 8u * t, held & 1u);
                ++held;
            }
            tc_fence_after();
            float M = m_true, fa = m_true == kPfNegInf ? 0.f : exp2f(m_used - m_true), fb = 0.f;
            float sum = l * fa;
            const bool mine = n > 0u && ok;
            bool theirs = false;
            int c0 = 0, c1 = D;  // the columns that this thread writes
            if (it.alt) {
                // the other tile's sums are in tensor memory, in the same lanes
                ml[t * 128 + r] = make_float4(m_used, m_true, l, mine ? 1.f : 0.f);
                tc_fence_before();
                named_bar_sync(1, 256);
                tc_fence_after();
                const float4 o = ml[(t ^ 1) * 128 + r];
                theirs = __all_sync(0xffffffffu, o.w != 0.f) != 0;
                M = fmaxf(m_true, o.y);
                fa = m_used == kPfNegInf ? 0.f : exp2f(m_used - M);
                fb = o.x == kPfNegInf ? 0.f : exp2f(o.x - M);
                sum = l * fa + o.z * fb;
                c0 = t * (D / 2);
                c1 = c0 + D / 2;
            }
            job.begin_row(row.ok, M, sum);
#pragma unroll 1
            for (int c = c0; c < c1; c += 16) {
                __syncwarp();
                float v[16];
                if (mine) {
                    tc_ld16(ocol + c, v);
                    tc_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = mine ? v[e] * fa : 0.f;
                if (theirs) {
                    float w[16];
                    tc_ld16(xcol + c, w);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = fmaf(w[e], fb, v[e]);
                }
                if (row.ok) job.write16(c, v);
            }
            if (it.alt) {  // both tiles' sums are read
                tc_fence_before();
                named_bar_sync(1, 256);
                tc_fence_after();
            }
            if (row.ok && (!it.alt || t == 0)) job.finish_row();
            __syncwarp();
        }
    } else if (warp == kTaMmaWarp || warp == kTaMmaWarp + 1) {
        // -------------------------------------------------------------------- MMA issuers
        // The whole warp walks the tile's blocks and waits, one lane issues. What the products depend on
        // comes out of warp reductions: the compiler then knows it to be uniform.
        const uint32_t lead = elect_lane();
        // a negative scale: the queries are negated in the product, so that scores scale by |scale|
        const uint32_t idesc_s = tc_idesc(128, 64, 0) | (p.sl2 < 0.f ? 1u << 13 : 0u);
        constexpr uint32_t idesc_o = tc_idesc(128, D, 1);
        const uint32_t t = __reduce_or_sync(0xffffffffu, (uint32_t)(warp - kTaMmaWarp));
        const uint32_t q0 = desc_lo(smem_u32(base + L.q), 16u);
        const uint32_t kd = desc_lo(smem_u32(base + L.kst), 16u);
        const uint32_t vd = desc_lo(smem_u32(base + L.vst), kHalf);
        const uint32_t tb = __reduce_or_sync(0xffffffffu, tbase);
        const uint32_t oc = tb + 128u * t, sc = tb + 256u + 128u * t;
        uint32_t j = 0u;      // blocks that the tile kept
        uint32_t items = 0u;
        while (ok && job.next(it)) {
            const bool alt = it.alt != 0;
            const uint32_t qd = q0 + (alt ? 0u : t * (128u * 128u >> 4));
            ok = wait(bar(kTaQFull), items & 1u);
            if (!ok) break;
            tc_fence_after();
            if (it.last[t] < 0) pb_commit(lead, bar(kTaQEmpty));
            // O += P V of the tile's block jj, block i of all; `more`: into the sum of the item's earlier
            // ones. A stage is given back by both warps, or twice by the one that read it.
            auto second = [&](uint32_t i, uint32_t jj, uint32_t more) -> bool {
                const uint32_t s = i % NV;
                // The weights first: with them, every product of earlier items is done, by both tiles, and
                // so the stage's earlier uses are over. (Within an alt item the use before was this tile's
                // own, or, of three stages, one whose V was written before this block's K. K's stages need
                // no such care: an item's queries come when both tiles have read all K of the one before.)
                if (!wait(bar(kTaP) + 16u * t + 8u * (jj & 1u), (jj >> 1) & 1u)) return false;
                if (!wait(bar(kTaVFull + s), (i / NV) & 1)) return false;
                tc_fence_after();
                const uint32_t v_lo = vd + s * (64u * D * 2u >> 4), from = sc + 64u * (jj & 1u);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        pb_mma_ts(lead, oc, from + 32u * part + 8u * kk, v_lo + (kk * 2048u >> 4),
                                  idesc_o, (part > 0 || kk > 0) ? 1u : more);
                }
                pb_commit(lead, bar(kTaPv) + 8u * t);
                pb_commit(lead, bar(kTaVEmpty + s));
                if (alt) pb_commit(lead, bar(kTaVEmpty + s));
                return true;
            };
            uint32_t pend = 0u, n = 0u;  // the block whose P V is to come; the item's P V so far
            bool has = false;
            for (int32_t b = alt ? (int32_t)t : 0; b < it.count; b += alt ? 2 : 1) {
                const uint32_t i = done + b, s = i % NK;
                const bool keep = alt || job.keeps(it, t, it.block(b));
                ok = wait(bar(kTaKFull + s), (i / NK) & 1);
                if (!ok) break;
                if (keep) {
                    tc_fence_after();
                    // into buffer j % 2, whose P V (of the tile's block j - 2) was issued before
                    const uint32_t to = sc + 64u * (j & 1u);
                    const uint32_t k_lo = kd + s * (64u * D * 2u >> 4);
                    pb_mma_ss<false>(lead, to, qd, k_lo, idesc_s);
#pragma unroll
                    for (int kk = 1; kk < D / 16; ++kk)
                        pb_mma_ss<true>(lead, to, qd + (((kk >> 2) * (256u * 128u) + (kk & 3) * 32u) >> 4),
                                        k_lo + (((kk >> 2) * kHalf + (kk & 3) * 32u) >> 4), idesc_s);
                    pb_commit(lead, bar(kTaS) + 16u * t + 8u * (j & 1u));
                    if (b == it.last[t]) pb_commit(lead, bar(kTaQEmpty));
                    ++j;
                }
                pb_commit(lead, bar(kTaKEmpty + s));
                if (alt) pb_commit(lead, bar(kTaKEmpty + s));
                if (has) {
                    ok = second(pend, keep ? j - 2u : j - 1u, n > 0u ? 1u : 0u);
                    if (!ok) break;
                    ++n;
                }
                has = keep;
                pend = i;
                if (!keep) {
                    ok = wait(bar(kTaVFull + i % NV), (i / NV) & 1);
                    if (!ok) break;
                    pb_commit(lead, bar(kTaVEmpty + i % NV));
                }
            }
            if (ok && has) ok = second(pend, j - 1u, n > 0u ? 1u : 0u);
            if (it.last[t] >= 0) pb_commit(lead, bar(kTaDrain) + 8u * t);
            done += it.count;
            ++items;
        }
        // Nothing of this warp's may still run on the tensor cores when the CTA exits: the softmax threads
        // have waited for the last product; after an abort, a millisecond is far more than one takes.
        if (*abort_p) {
            const unsigned long long t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 1000000ull) {
            }
        }
    } else if (warp == kTaQWarp) {
        // -------------------------------------------------------------------- the queries
        const uint64_t pol = policy_evict_first();
        const uint32_t qs = smem_u32(base + L.q);
        uint32_t items = 0u;
        while (ok && job.next(it)) {
            if (items > 0u) ok = wait(bar(kTaQEmpty), (items - 1u) & 1u);
            if (!ok) break;
            if (lane == 0) {
                const int tiles = it.tok[1] > 0 ? 2 : 1;
                mbar_arrive_expect_tx(bar(kTaQFull), (uint32_t)(tiles * KH * p.tok * p.g) * 128u);
                for (int t = 0; t < tiles; ++t)
                    for (int hh = 0; hh < KH; ++hh)
                        tma_load_4d(qs + hh * (256u * 128u) + t * (128u * 128u), &tmap_q, 0,
                                    it.kvh * p.g, it.n0 + t * p.tok, hh, bar(kTaQFull), pol);
            }
            __syncwarp();
            ++items;
        }
        if (lane == 0 && *abort_p && items > 0u) {  // (bounded) a copy in flight
            const unsigned long long t0 = global_timer_ns();
            while (!mbar_try_wait(bar(kTaQFull), (items - 1u) & 1u) &&
                   global_timer_ns() - t0 < kWaitLimitNs) {
            }
        }
        __syncwarp();
    } else if (BLK ? warp == kTaCodeWarp : warp >= kTaConvWarp && warp < kTaConvWarp + 4) {
        // -------------------------------------------------------------------- the key blocks
        // bf16: warps 8 and 10 copy K and leave the blocks' metadata, warps 9 and 11 copy V, each every
        // other block (a warp issues the copies of a block of four pages in about a microsecond); block-
        // scaled pool: warp 15 copies the codes of both. Lane (grp, u) resolves tile u of block grp of
        // eight, and copies p.box rows, one or two or all of the block's tiles.
        const int grp = lane >> 2, u = lane & 3;
        const bool isv = !BLK && (warp & 1) != 0;
        const uint32_t turn = BLK ? 0u : (uint32_t)(warp - kTaConvWarp) >> 1;
        const int32_t box = p.box;
        const bool copies = (u * 16) % box == 0;
        const uint64_t pol = policy_evict_normal();
        const uint32_t NS = BLK ? NC : isv ? NV : NK;
        const int full0 = BLK ? kTaCFull : isv ? kTaVFull : kTaKFull;
        const int empty0 = BLK ? kTaCEmpty : isv ? kTaVEmpty : kTaKEmpty;
        const uint32_t st0 = smem_u32(base + (BLK ? L.cst : isv ? L.vst : L.kst));
        uint32_t issued = 0u;
        while (ok && job.next(it)) {
            const int32_t* trow = p.block_table + (int64_t)it.trow * p.max_pages;
            // this lane's tile of the item's block b: its row in the pool and its tokens (0: none)
            auto place = [&](int32_t b, int32_t& y, int32_t& hi, float2& s) {
                y = hi = 0;
                s = make_float2(0.f, 0.f);
                if (b >= it.count) return;
                const int32_t t0 = it.block(b) * kPfBlock + 16 * u;
                if (t0 >= it.kmax) return;
                // a page of which no row sees a token may be gone (it counts as keys that do not exist)
                const int32_t lp = t0 / p.P;
                if (lp * p.P >= it.sinks && (lp + 1) * p.P <= it.low) return;
                const int32_t page = __ldcg(trow + lp);
                if (page < 0) {
                    if (!isv) set_err(p.dev_err, DATTN_DEVERR_UNMAPPED_PAGE);
                } else if (page >= p.num_pages) {
                    if (!isv) set_err(p.dev_err, DATTN_DEVERR_PAGE_OOB);
                } else {
                    y = (page * p.Hkv + it.kvh) * p.P + (t0 - lp * p.P);
                    hi = min(16, it.kmax - t0);
                    if (BLK) s = __ldcg(p.scale + (y >> 4));
                }
            };
            int32_t y, hi, ny, nhi;
            float2 sc, nsc;
            place(grp, y, hi, sc);
            for (int32_t b0 = 0; b0 < it.count && ok; b0 += 8) {
                place(b0 + 8 + grp, ny, nhi, nsc);  // (on its way behind this group's copies)
                int32_t his = hi << (5 * u), valid = hi > 0 && copies ? 1 : 0;
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    his |= __shfl_xor_sync(0xffffffffu, his, o);
                    valid += __shfl_xor_sync(0xffffffffu, valid, o);
                }
                for (int k = 0; k < 8 && b0 + k < it.count; ++k) {
                    const uint32_t i = done + b0 + k, ms = i % kTaMeta, s = i % NS;
                    if (!BLK && (i & 1u) != turn) continue;
                    if (!isv && i >= (uint32_t)kTaMeta)
                        ok = wait(bar(kTaMetaEmpty + ms), ((i / kTaMeta) & 1) ^ 1);
                    if (ok && i >= NS) ok = wait(bar(empty0 + s), ((i / NS) & 1) ^ 1);
                    if (!ok) break;
                    const uint32_t full = bar(full0 + s);
                    if (BLK && grp == k)
                        *reinterpret_cast<float2*>(base + L.scales + 48 * s + 8 * u) = sc;
                    if (grp == k && u == 0 && !isv) {
                        meta[ms] = make_int2(it.block(b0 + k), his);
                        if (BLK) *reinterpret_cast<int32_t*>(base + L.scales + 48 * s + 32) = his;
                        mbar_arrive(bar(kTaMetaFull + ms));
                    }
                    __syncwarp();
                    if (grp == k && u == 0)
                        mbar_arrive_expect_tx(full, (uint32_t)(valid * box) * (BLK ? 2u * D : KH * 128u));
                    __syncwarp();
                    if (grp == k && hi > 0 && copies) {
                        if constexpr (BLK) {
                            const uint32_t dst = st0 + s * 2u * L.code_bytes + u * 16u * D;
                            tma_load_2d(dst, &tmap_k, 0, y, full, pol);
                            tma_load_2d(dst + L.code_bytes, &tmap_v, 0, y, full, pol);
                        } else {
                            const uint32_t dst = st0 + s * L.blk_bytes + u * 2048u;
#pragma unroll
                            for (int hh = 0; hh < KH; ++hh)
                                tma_load_3d(dst + hh * kHalf, isv ? &tmap_v : &tmap_k, 0, y, hh, full,
                                            pol);
                        }
                    }
                    issued = i + 1u;
                }
                y = ny;
                hi = nhi;
                sc = nsc;
            }
            done += it.count;
        }
        // after an abort, wait (bounded in total) for copies still in flight
        if (lane == 0 && *abort_p) {
            const unsigned long long t0 = global_timer_ns();
            for (uint32_t i = issued > NS ? issued - NS : 0u; i < issued; ++i)
                while (!mbar_try_wait(bar(full0 + i % NS), (i / NS) & 1) &&
                       global_timer_ns() - t0 < kWaitLimitNs) {
                }
        }
        __syncwarp();
    } else if (BLK && warp >= kTaConvWarp && warp < kTaConvWarp + 4) {
        // -------------------------------------------------------------------- codes -> K and V stages
        // A row of D codes is D/16 threads of 16 codes; a pass takes RP rows, NP passes a block. Eight
        // neighbours store to two rows of one half: all banks.
        constexpr int CPR = D / 16, RP = kTaConvThreads / CPR, NP = 64 / RP;
        const int ct = tid - kTaConvWarp * 32;
        const int c16 = D == 64 ? ct & 3 : (ct & 3) | ((ct >> 1) & 4);
        const int rr = D == 64 ? ct >> 2 : ((ct >> 2) & 1) | ((ct >> 4) << 1);
        const uint32_t half = (c16 >> 2) * kHalf, ch = 2u * (c16 & 3);
        // A block's K or V; rows without a token become zeros. All codes are read before the first row is
        // written: the compiler cannot tell the stages apart, and read them one after another (a 4K chunk
        // through a window of 4096: 427 us, 386 so). Shifting the codes' bits to a bf16's places and two
        // bf16 products instead of the conversions by fp16 and fp32 load the pipe that the softmax fills
        // (533 us).
        auto widen = [&](const uint8_t* from, uint8_t* to, const float* sc, int32_t his) {
            uint4 c[NP];
#pragma unroll
            for (int a = 0; a < NP; ++a)
                c[a] = *reinterpret_cast<const uint4*>(from + swz_rows<D>((uint32_t)(rr + RP * a), c16));
            if (his != kFull) {  // codes of +0 for rows without a token
#pragma unroll
                for (int a = 0; a < NP; ++a) {
                    const uint32_t r = (uint32_t)(rr + RP * a);
                    if ((int32_t)(r & 15u) >= ((his >> (5 * (r >> 4))) & 31))
                        c[a] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
#pragma unroll
            for (int a = 0; a < NP; ++a) {
                const uint32_t r = (uint32_t)(rr + RP * a);
                const float f = sc[2 * (r >> 4)];
                const uint64_t f2 = pack_f32x2(f, f);
                const uint32_t w[4] = {c[a].x, c[a].y, c[a].z, c[a].w};
                uint32_t o[8];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t lo, hi;
                    e4m3x4_to_f16(w[x], lo, hi);
                    o[2 * x] = scaled_bf16x2(lo, f2);
                    o[2 * x + 1] = scaled_bf16x2(hi, f2);
                }
                *reinterpret_cast<uint4*>(to + half + swz128(r, ch)) = make_uint4(o[0], o[1], o[2], o[3]);
                *reinterpret_cast<uint4*>(to + half + swz128(r, ch + 1u)) =
                    make_uint4(o[4], o[5], o[6], o[7]);
            }
        };
        while (ok && job.next(it)) {
            for (int32_t b = 0; b < it.count; ++b) {
                const uint32_t i = done + b;
                const uint32_t c = i % NC, sk = i % NK, sv = i % NV;
                ok = wait(bar(kTaCFull + c), (i / NC) & 1);
                if (ok && i >= (uint32_t)NK) ok = wait(bar(kTaKEmpty + sk), ((i / NK) & 1) ^ 1);
                if (!ok) break;
                const uint8_t* from = base + L.cst + c * 2u * L.code_bytes;
                const float* sc = reinterpret_cast<const float*>(base + L.scales + 48 * c);
                const int32_t his = *reinterpret_cast<const int32_t*>(base + L.scales + 48 * c + 32);
                widen(from, base + L.kst + sk * L.blk_bytes, sc, his);
                fence_proxy_async_smem();
                mbar_arrive(bar(kTaKFull + sk));
                if (i >= (uint32_t)NV) ok = wait(bar(kTaVEmpty + sv), ((i / NV) & 1) ^ 1);
                if (!ok) break;
                widen(from + L.code_bytes, base + L.vst + sv * L.blk_bytes, sc + 1, his);
                fence_proxy_async_smem();
                mbar_arrive(bar(kTaVFull + sv));
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kTaCEmpty + c));
            }
            done += it.count;
        }
    }
    // ---- teardown: the allocating warp frees the tensor memory --------------------------------
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tc_dealloc(tbase, 512u);
    }
    job.end();
}

// The queries [tokens][Hq][D] as boxes of `tok` tokens of one KV head's g query heads, one 128-byte half
// each: {64, g, tok, 1} values, landing as rows token * g + head of 128 bytes, swizzled.
inline dattn_status_t make_q_tensor_map(void* tmap_out, const void* q, int64_t tokens, int32_t Hq,
                                        int32_t g, int32_t tok, int D) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = tc_encode_fn();
    if (fn == nullptr) return DATTN_ERR_CUDA;
    cuuint64_t dims[4] = {64, (cuuint64_t)Hq, (cuuint64_t)tokens, (cuuint64_t)(D / 64)};
    cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)Hq * D * 2, 128};
    cuuint32_t box[4] = {64, (cuuint32_t)g, (cuuint32_t)tok, 1};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    CUresult r = fn(static_cast<CUtensorMap*>(tmap_out), CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                    const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? DATTN_OK : DATTN_ERR_CUDA;
}

template <class Job, int D, int FMT>
dattn_status_t launch_tiles(const TaParams& p0, const typename Job::Params& jp, const void* q,
                            int64_t tokens, const void* k_pool, const void* v_pool, int32_t grid,
                            uint32_t job_bytes, cudaStream_t stream) {
    const TaSmem L = ta_smem_layout(D, FMT, job_bytes);
    if (L.total > 227u * 1024u) return DATTN_ERR_UNSUPPORTED;
    {
        static std::mutex mutex;
        static int set[kMaxDevices] = {};  // a function attribute belongs to a device
        std::lock_guard<std::mutex> lock(mutex);
        int& mine = set[device_index()];
        if ((int)L.total > mine) {
            if (cudaFuncSetAttribute(tile_attention_kernel<Job, D, FMT>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)L.total) != cudaSuccess)
                return DATTN_ERR_CUDA;
            mine = (int)L.total;
        }
    }
    TaParams p = p0;
    p.box = p.P % 64 == 0 ? 64 : p.P % 32 == 0 ? 32 : 16;
    alignas(64) CUtensorMap tq;
    alignas(64) CUtensorMap tk;
    alignas(64) CUtensorMap tv;
    const int64_t rows = (int64_t)p.num_pages * p.Hkv * p.P;
    dattn_status_t st;
    if ((st = make_q_tensor_map(&tq, q, tokens, p.Hq, p.g, p.tok, D)) != DATTN_OK) return st;
    if (FMT == DATTN_KV_BF16) {
        if ((st = make_half_tensor_map(&tk, k_pool, rows, D, p.box)) != DATTN_OK) return st;
        if ((st = make_half_tensor_map(&tv, v_pool, rows, D, p.box)) != DATTN_OK) return st;
    } else {
        if ((st = make_kv_tensor_map_u8(&tk, k_pool, rows, D, p.box)) != DATTN_OK) return st;
        if ((st = make_kv_tensor_map_u8(&tv, v_pool, rows, D, p.box)) != DATTN_OK) return st;
    }
    return launch_pdl(tile_attention_kernel<Job, D, FMT>, dim3((unsigned)grid), dim3(kTaThreads),
                      L.total, stream, p, jp, tq, tk, tv) == cudaSuccess
               ? DATTN_OK
               : DATTN_ERR_CUDA;
}

}  // namespace
}  // namespace dattn
