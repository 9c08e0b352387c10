// dattn_decode_shared: the decode of a batch whose requests share long prefixes, each prefix read and
// computed once for all the requests of its group.
//
// Mathematics: "Infinite-LLM: Efficient LLM Service for Long Context with DistAttention and
// Distributed KVCache", "DistAttention 的等价数学变换": the keys of a query are cut into parts, each part
// gives (m, e, MA), and the parts' triples aggregate to the attention over all of them. Here the first
// part of every query is its group's prefix, the same keys for all of the group's rows (request, query
// token, query head), so that it is a matrix product S = Q K^T with the rows of all requests; the second
// part is the request's own tokens. Three launches:
//   1. the split-KV engine in its windowed mode (attention_window.cu) over the own tokens, as partials;
//   2. shared_prefix_kernel over the prefixes, which needs nothing of 1 and starts as its CTAs leave;
//   3. shared_merge_kernel, which joins the pieces.
//
// shared_prefix_kernel. A CTA per SM takes 256 rows of one (group, KV head), as two tiles of 128 rows, or
// up to 128 rows, which its two tiles then both hold, each for every other key block. The 64-key blocks
// of all (group, KV head, 256 rows) are laid end to end and cut into equal runs, one per CTA; a CTA leaves
// the unnormalised sum, maximum and weight of its rows for every piece of a segment in its run. 14 warps:
//   0-3, 4-7  one row per thread of tile 0, 1: the softmax (as in prefill.cu: weights as two bf16
//             terms, the accumulator rescaled only when a maximum rises by 2^8);
//   8-11      the key blocks: bf16, warps 8 and 9 copy K and V by TMA; block-scaled pool, all four load
//             the codes and write code * scale, which is a bf16 number, so that both formats compute alike;
//   12, 13    one thread each issues the tcgen05 products of tile 0, 1.
// What bounds it: with up to 128 rows the memory; from there on the tensor cores (three products of
// 128 x 64 x d for two that count) and the softmax.
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "prefill.cuh"
#include "shared.cuh"

namespace dattn {

namespace {

constexpr int kShRows = 256;
constexpr int kShStages = 4;         // K blocks, and V blocks, in flight
constexpr int kShLoadWarp = 8;       // warps 8-11
constexpr int kShLoadThreads = 128;
constexpr int kShMmaWarp = 12;       // warps 12, 13
constexpr int kShThreads = 14 * 32;
constexpr int kShMeta = 16;          // blocks' metadata slots
// Key blocks between two emptyings of a row's accumulator, to which the tensor cores add rounding
// towards zero: 8 products a block, each losing up to 2^-24 of the sum.
constexpr int kShEmpty = 64;
constexpr int32_t kShSegCost = 4;    // a piece's fixed cost in blocks
constexpr int32_t kShMinCost = 6;    // blocks (and fixed costs) of a CTA at least
constexpr int kShMaxGroups = 1024;

// mbarriers
constexpr int kShKFull = 0, kShKEmpty = 4, kShVFull = 8, kShVEmpty = 12;
constexpr int kShS = 16, kShP = 20;  // + 2 tile + buffer
constexpr int kShPv = 24, kShDrain = 26;
constexpr int kShMetaFull = 28, kShBars = kShMetaFull + kShMeta;

struct ShParams {
    int32_t num_pages, Hkv, P, max_pages;
    const int32_t* block_table;
    const uint16_t* q;
    int32_t B, T, Hq, g;
    float sl2;
    const int32_t* seq_lens;
    int32_t groups;
    const int32_t* group_indptr;
    const int32_t* prefix_lens;
    const uint8_t* k_pool;  // the block-scaled pool
    const uint8_t* v_pool;
    const float2* scale;
    // the workspace: the pieces' rows, and (m in log2 units, e) of each; the plan: W, CTAs with work, then
    // per group its first cost unit (groups + 1 of them) and its prefix
    float* slots;
    float2* slot_me;
    int32_t* plan;
    int32_t* dev_err;
};

// The rows of pieces in the workspace: a piece of segment s in CTA c begins at 2 rowbase(s) + 256 c, where
// rowbase counts the rows of earlier segments, and has up to 256 rows, or twice its up to 128 rows: the
// pieces of a CTA, and of a segment, are apart.
__host__ __device__ inline int64_t shared_slot_rows(int64_t rows, int32_t ctas) {
    return 2 * rows + (int64_t)kShRows * ctas;
}

struct ShSmem {
    uint32_t q, kst, vst, blk_bytes, bars, meta, taddr, abort, key, start, scan, total;
};

__host__ __device__ inline ShSmem sh_smem_layout(int D, int groups) {
    ShSmem s;
    uint32_t o = 0;
    s.q = o;        o += (uint32_t)kShRows * D * 2u;
    s.blk_bytes = 64u * D * 2u;
    s.kst = o;      o += kShStages * s.blk_bytes;
    s.vst = o;      o += kShStages * s.blk_bytes;
    s.bars = o;     o += kShBars * 8u;
    s.meta = o;     o += kShMeta * 8u;
    s.taddr = o;    o += 16u;
    s.abort = o;    o += 16u;
    s.key = o;      o += (uint32_t)groups * 8u;  // (length, ~request) of a group's longest, then (prefix, request)
    s.start = o;    o += (uint32_t)(groups + 1) * 4u;
    s.scan = o;     o += 16u * 4u;
    s.total = o;
    return s;
}

// The group's geometry: rows of a KV head, segments of a KV head (256 rows each) and cost of a segment.
struct ShGroup {
    int32_t first, rows, pairs, prefix, blocks, cost;
    __device__ ShGroup(const ShParams& p, int32_t i, int32_t prefix_len) {
        first = __ldcg(p.group_indptr + i);
        rows = (__ldcg(p.group_indptr + i + 1) - first) * p.T * p.g;
        pairs = (rows + kShRows - 1) / kShRows;
        prefix = prefix_len;
        blocks = (prefix + kPfBlock - 1) / kPfBlock;
        cost = blocks > 0 ? blocks + kShSegCost : 0;
    }
};

// The plan of all groups, by all threads, into shared memory. Returns the whole cost; 0 where the groups'
// bounds are out of order (the engine then attends everything).
__device__ int32_t sh_make_plan(const ShParams& p, uint8_t* base, const ShSmem& L, int tid) {
    unsigned long long* key = reinterpret_cast<unsigned long long*>(base + L.key);
    int2* info = reinterpret_cast<int2*>(base + L.key);
    int32_t* start = reinterpret_cast<int32_t*>(base + L.start);
    int32_t* scan = reinterpret_cast<int32_t*>(base + L.scan);
    const int32_t cap = p.max_pages * p.P;
    for (int32_t g = tid; g < p.groups; g += kShThreads) key[g] = 0ull;
    if (!shared_groups_ok(p.group_indptr, p.groups, p.B, tid, kShThreads)) return 0;
    // the longest request of a group has all pages of its prefix; the first of several
    for (int32_t i = tid; i < p.B; i += kShThreads) {
        const int32_t g = shared_group(p.group_indptr, p.groups, i);
        const int32_t len = min(max(__ldcg(p.seq_lens + i), 0), cap);
        if (g >= 0) atomicMax(key + g, ((unsigned long long)len << 32) | (uint32_t)~i);
    }
    __syncthreads();
    const int32_t per = (p.groups + kShThreads - 1) / kShThreads;
    const int32_t g0 = min(p.groups, tid * per), g1 = min(p.groups, g0 + per);
    int32_t sum = 0;
    for (int32_t g = g0; g < g1; ++g) {
        const unsigned long long k = key[g];
        const int32_t prefix = min(max(__ldcg(p.prefix_lens + g), 0), (int32_t)(k >> 32));
        info[g] = make_int2(prefix, (int32_t)~(uint32_t)k);
        const ShGroup G(p, g, prefix);
        start[g] = p.Hkv * G.pairs * G.cost;
        sum += start[g];
    }
    int32_t incl = sum;
    const int warp = tid >> 5, lane = tid & 31;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int32_t v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int32_t run = incl - sum, all = 0;
    for (int w = 0; w < kShThreads / 32; ++w) {
        if (w < warp) run += scan[w];
        all += scan[w];
    }
    for (int32_t g = g0; g < g1; ++g) {
        const int32_t c = start[g];
        start[g] = run;
        run += c;
    }
    if (tid == 0) start[p.groups] = all;
    __syncthreads();
    return all;
}

__device__ __forceinline__ int32_t sh_ctas(int32_t W, int32_t grid) {
    return min(grid, max(W / kShMinCost, 1));
}

// A piece: key blocks [j0, j1) of a segment (rows `row0` .. of KV head kvh of group i).
struct ShPiece {
    int32_t i, kvh, row0, rows, j0, j1;
    int64_t slot;  // its first row in the workspace
};

template <int D, int FMT>
__global__ void __launch_bounds__(kShThreads, 1)
shared_prefix_kernel(const __grid_constant__ ShParams p, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v) {
    constexpr int KH = D / 64;
    constexpr bool BLK = FMT == DATTN_KV_FP8_BLOCK;
    constexpr uint32_t kHalf = 64u * 128u;  // a 128-byte half of a key block's rows
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* base = smem_raw;
    const ShSmem L = sh_smem_layout(D, p.groups);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the 128-byte swizzle of the TMA copies and the MMA operands needs 1024-byte alignment
    if ((smem_u32(base) & 1023u) != 0u) {
        if (tid == 0) set_err(p.dev_err, DATTN_DEVERR_SMEM_ALIGN);
        grid_launch_dependents();
        grid_dependency_wait();
        return;
    }
    const uint32_t bars = smem_u32(base + L.bars);
    auto bar = [&](int i) { return bars + 8u * i; };
    int2* meta = reinterpret_cast<int2*>(base + L.meta);  // (block, its tiles' tokens, 5 bits each)
    volatile int* abort_p = reinterpret_cast<volatile int*>(base + L.abort);
    if (tid == 0) {
        for (int s = 0; s < kShStages; ++s) {
            mbar_init(bar(kShKFull + s), BLK ? kShLoadThreads : 1);
            mbar_init(bar(kShKEmpty + s), 2);
            mbar_init(bar(kShVFull + s), BLK ? kShLoadThreads : 1);
            mbar_init(bar(kShVEmpty + s), 2);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(bar(kShS + i), 1);
            mbar_init(bar(kShP + i), 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kShPv + i), 1);
            mbar_init(bar(kShDrain + i), 1);
        }
        for (int i = 0; i < kShMeta; ++i) mbar_init(bar(kShMetaFull + i), 1);
        *abort_p = 0;
        fence_mbar_init();
    }
    if (!BLK && warp == kShLoadWarp && lane == 0) {
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    __syncwarp();  // (tcgen05 instructions take whole, converged warps)
    if (warp == 0) {  // the whole warp allocates the CTA's tensor memory
        tc_alloc(smem_u32(base + L.taddr), 512u);
        tc_relinquish();
    }
    if constexpr (!BLK) {
        // V rows that the MMA reads with weight 0 (tiles that are never loaded) must hold finite data
        for (uint32_t i = tid; i < kShStages * L.blk_bytes / 16u; i += kShThreads)
            reinterpret_cast<uint4*>(base + L.vst)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    tc_fence_before();
    // No dependency wait here: the kernel before on the stream is the engine's launch of the same call,
    // whose results this one does not read, and whose CTAs let this kernel start only after their own
    // wait: what this call reads is there, in L2, and is read from L2 (an SM's L1 may be older).
    grid_launch_dependents();
    const int32_t W = sh_make_plan(p, base, L, tid);
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(base + L.taddr);
    const int2* info = reinterpret_cast<const int2*>(base + L.key);
    const int32_t* start = reinterpret_cast<const int32_t*>(base + L.start);
    const int32_t cta = blockIdx.x, Gw = sh_ctas(W, gridDim.x);
    if (cta == 0) {  // for the merge
        for (int32_t g = tid; g < p.groups; g += kShThreads) {
            p.plan[2 + g] = W > 0 ? start[g] : 0;
            p.plan[3 + p.groups + g] = W > 0 ? info[g].x : 0;
        }
        if (tid == 0) {
            p.plan[0] = W;
            p.plan[1] = Gw;
        }
    }
    int32_t x = 0, X1 = 0;
    if (cta < Gw && W > 0) {
        x = (int32_t)split_begin(W, Gw, cta);
        X1 = (int32_t)split_begin(W, Gw, cta + 1);
    }
    // the next piece at or after cost unit x, one answer for all threads; x moves past it
    auto next_piece = [&](ShPiece& pc) -> bool {
        while (x < X1) {
            int32_t lo = 0, hi = p.groups - 1;  // the last group with start <= x
            while (lo < hi) {
                const int32_t mid = (lo + hi + 1) >> 1;
                if (start[mid] <= x) lo = mid; else hi = mid - 1;
            }
            const ShGroup G(p, lo, info[lo].x);
            const int32_t seg = (x - start[lo]) / G.cost, cs = start[lo] + seg * G.cost;
            pc.i = lo;
            pc.kvh = seg / G.pairs;
            pc.row0 = (seg - pc.kvh * G.pairs) * kShRows;
            pc.rows = min(kShRows, G.rows - pc.row0);
            pc.j0 = x - cs;
            pc.j1 = min(X1 - cs, G.blocks);
            pc.slot = 2 * ((int64_t)G.first * p.T * p.Hq + (int64_t)pc.kvh * G.rows + pc.row0) +
                      (int64_t)kShRows * cta;
            x = cs + G.cost;
            if (pc.j0 < pc.j1) return true;
        }
        return false;
    };
    auto wait = [&](uint32_t bar_addr, uint32_t parity) {  // by a whole warp, one answer
        return __all_sync(0xffffffffu, mbar_wait(bar_addr, parity, abort_p, p.dev_err)) != 0;
    };

    uint32_t done = 0u;                   // blocks of earlier pieces: block i is in stage i % 4
    uint32_t tdone0 = 0u, tdone1 = 0u;    // those of tile 0, 1
    ShPiece pc;
    for (int32_t piece = 0; next_piece(pc); ++piece) {
        const int32_t n = pc.j1 - pc.j0, prefix = info[pc.i].x, leader = info[pc.i].y;
        const int32_t first = __ldcg(p.group_indptr + pc.i), tg = p.T * p.g;
        // both tiles hold the same rows, and take every other block
        const bool alt = pc.rows <= 128;
        {   // the query rows, [half][256 rows][128 B] swizzled; with a negative scale they are negated
            // (exact), so that the scores scale by |scale|
            const uint32_t qneg = p.sl2 < 0.f ? 0x80008000u : 0u;
            const int nr = alt ? 128 : kShRows;
            for (int idx = tid; idx < nr * (D / 8); idx += kShThreads) {
                const int r = idx / (D / 8), ch = idx - r * (D / 8);
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (r < pc.rows) {
                    const int32_t rr = pc.row0 + r, b = first + rr / tg, c = rr % tg;
                    const int32_t t = c / p.g, j = c - t * p.g;
                    v = __ldcg(reinterpret_cast<const uint4*>(
                        p.q + (((int64_t)b * p.T + t) * p.Hq + pc.kvh * p.g + j) * D) + ch);
                    v = make_uint4(v.x ^ qneg, v.y ^ qneg, v.z ^ qneg, v.w ^ qneg);
                }
                *reinterpret_cast<uint4*>(base + L.q + (ch >> 3) * (kShRows * 128u) +
                                          swz128((uint32_t)r, (uint32_t)(ch & 7))) = v;
            }
            fence_proxy_async_smem();  // the tensor cores read these rows through the async proxy
        }
        __syncthreads();
        if (warp >= kShLoadWarp && warp < kShMmaWarp && (BLK || warp < kShLoadWarp + 2)) {
            // ------------------------------------------------------------ the key blocks
            const int grp = lane >> 2, u = lane & 3;  // lane (grp, u): tile u of the eight blocks' grp
            const int32_t* row = p.block_table + (int64_t)leader * p.max_pages;
            // this lane's tile of block j: its row in the pool and its tokens (0: none)
            auto place = [&](int32_t j, int32_t& y, int32_t& hi) {
                const int32_t t0 = j * kPfBlock + 16 * u;
                y = hi = 0;
                if (j >= pc.j1 || t0 >= prefix) return;
                const int32_t lp = t0 / p.P, page = __ldcg(row + lp);
                if (page < 0) {
                    set_err(p.dev_err, DATTN_DEVERR_UNMAPPED_PAGE);
                } else if (page >= p.num_pages) {
                    set_err(p.dev_err, DATTN_DEVERR_PAGE_OOB);
                } else {
                    y = (page * p.Hkv + pc.kvh) * p.P + (t0 - lp * p.P);
                    hi = min(16, prefix - t0);
                }
            };
            auto tokens = [&](int32_t hi) {  // of the four tiles of this lane's block
                int32_t h = hi << (5 * u);
                h |= __shfl_xor_sync(0xffffffffu, h, 1);
                return h | __shfl_xor_sync(0xffffffffu, h, 2);
            };
            bool ok = true;
            if constexpr (!BLK) {
                const bool isv = warp == kShLoadWarp + 1;
                const CUtensorMap* tmap = isv ? &tmap_v : &tmap_k;
                const uint64_t pol = policy_evict_first();
                const uint32_t st0 = smem_u32(base + (isv ? L.vst : L.kst));
                int32_t y, hi, ny, nhi;
                place(pc.j0 + grp, y, hi);
                for (int32_t j = 0; j < n && ok; j += 8) {
                    place(pc.j0 + j + 8 + grp, ny, nhi);  // (on its way behind this group's copies)
                    const int32_t his = tokens(hi);
                    int32_t valid = hi > 0 ? 1 : 0;
                    valid += __shfl_xor_sync(0xffffffffu, valid, 1);
                    valid += __shfl_xor_sync(0xffffffffu, valid, 2);
                    for (int k = 0; k < 8 && j + k < n; ++k) {
                        const uint32_t i = done + j + k;
                        const int s = i % kShStages;
                        if (i >= kShStages)
                            ok = wait(bar((isv ? kShVEmpty : kShKEmpty) + s),
                                      ((i / kShStages) & 1) ^ 1);
                        if (!ok) break;
                        const uint32_t full = bar((isv ? kShVFull : kShKFull) + s);
                        if (grp == k && u == 0) {
                            if (!isv) {
                                meta[i % kShMeta] = make_int2(pc.j0 + j + k, his);
                                mbar_arrive(bar(kShMetaFull + i % kShMeta));
                            }
                            mbar_arrive_expect_tx(full, (uint32_t)valid * KH * 2048u);
                        }
                        __syncwarp();
                        if (grp == k && hi > 0) {
                            const uint32_t dst = st0 + (uint32_t)s * L.blk_bytes + u * 2048u;
#pragma unroll
                            for (int hh = 0; hh < KH; ++hh)
                                tma_load_3d(dst + hh * kHalf, tmap, 0, y, hh, full, pol);
                        }
                    }
                    y = ny;
                    hi = nhi;
                }
                // after an abort, wait (bounded in total) for copies still in flight
                if (lane == 0 && *abort_p) {
                    const unsigned long long t0 = global_timer_ns();
                    for (uint32_t i = done; i < done + n; ++i)
                        while (!mbar_try_wait(bar((isv ? kShVFull : kShKFull) + i % kShStages),
                                              (i / kShStages) & 1) &&
                               global_timer_ns() - t0 < kWaitLimitNs) {
                        }
                }
                __syncwarp();
            } else {
                // A row of D codes is D/16 threads of 16 codes; a pass takes RP rows, NP passes a block.
                // Eight neighbours store to two rows of one half: all banks.
                constexpr int CPR = D / 16, RP = kShLoadThreads / CPR, NP = 64 / RP;
                const int ct = tid - kShLoadWarp * 32;
                const int c16 = D == 64 ? ct & 3 : (ct & 3) | ((ct >> 1) & 4);
                const int rr = D == 64 ? ct >> 2 : ((ct >> 2) & 1) | ((ct >> 4) << 1);
                const uint32_t half = (c16 >> 2) * kHalf, ch = 2u * (c16 & 3);
                int32_t y, hi, ny = 0, nhi = 0;   // of the eight blocks in hand, and of the next
                uint4 kv[NP], vv[NP];
                float ks[NP], vs[NP];  // scales of the rows in kv, vv
                // block k of the eight: the codes of this thread's rows (rows without a token: zeros)
                auto load = [&](const uint8_t* pool, bool isv, int k, uint4 (&v)[NP], float (&sc)[NP]) {
#pragma unroll
                    for (int a = 0; a < NP; ++a) {
                        const int r = rr + RP * a;
                        const int32_t at = __shfl_sync(0xffffffffu, y, 4 * k + (r >> 4));
                        const int32_t have = __shfl_sync(0xffffffffu, hi, 4 * k + (r >> 4));
                        v[a] = make_uint4(0u, 0u, 0u, 0u);
                        sc[a] = 0.f;
                        if ((r & 15) < have) {
                            v[a] = __ldcg(reinterpret_cast<const uint4*>(
                                pool + (int64_t)(at + (r & 15)) * D + 16 * c16));
                            const float2 s = __ldcg(p.scale + (at >> 4));
                            sc[a] = isv ? s.y : s.x;
                        }
                    }
                };
                auto store = [&](uint8_t* st, const uint4 (&v)[NP], const float (&sc)[NP]) {
#pragma unroll
                    for (int a = 0; a < NP; ++a) {
                        const uint32_t r = (uint32_t)(rr + RP * a);
                        const uint32_t w[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
                        uint32_t o[8];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t lo, hi2;
                            e4m3x4_to_f16(w[c], lo, hi2);
                            o[2 * c] = pack_bf16(f16_lo(lo) * sc[a], f16_hi(lo) * sc[a]);
                            o[2 * c + 1] = pack_bf16(f16_lo(hi2) * sc[a], f16_hi(hi2) * sc[a]);
                        }
                        *reinterpret_cast<uint4*>(st + half + swz128(r, ch)) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4*>(st + half + swz128(r, ch + 1u)) =
                            make_uint4(o[4], o[5], o[6], o[7]);
                    }
                };
                place(pc.j0 + grp, y, hi);
                int32_t his = tokens(hi);
                load(p.k_pool, false, 0, kv, ks);
                load(p.v_pool, true, 0, vv, vs);
                for (int32_t j = 0; j < n && ok; ++j) {
                    const uint32_t i = done + j;
                    const int s = i % kShStages, k = j & 7;
                    const bool more = j + 1 < n;
                    if (k == 0) place(pc.j0 + j + 8 + grp, ny, nhi);
                    if (i >= kShStages) ok = wait(bar(kShKEmpty + s), ((i / kShStages) & 1) ^ 1);
                    if (!ok) break;
                    store(base + L.kst + (uint32_t)s * L.blk_bytes, kv, ks);
                    fence_proxy_async_smem();
                    mbar_arrive(bar(kShKFull + s));
                    if (warp == kShLoadWarp && lane == 4 * k) {
                        meta[i % kShMeta] = make_int2(pc.j0 + j, his);
                        mbar_arrive(bar(kShMetaFull + i % kShMeta));
                    }
                    __syncwarp();
                    if (k == 7) {
                        y = ny;
                        hi = nhi;
                        his = tokens(hi);
                    }
                    // the next block's K is on its way while this block's V is widened
                    if (more) load(p.k_pool, false, (k + 1) & 7, kv, ks);
                    if (i >= kShStages) ok = wait(bar(kShVEmpty + s), ((i / kShStages) & 1) ^ 1);
                    if (!ok) break;
                    store(base + L.vst + (uint32_t)s * L.blk_bytes, vv, vs);
                    fence_proxy_async_smem();
                    mbar_arrive(bar(kShVFull + s));
                    if (more) load(p.v_pool, true, (k + 1) & 7, vv, vs);
                }
            }
        } else if (warp >= kShMmaWarp) {
            // ---------------------------------------------------------------- MMA issuers
            // A warp for each tile; the whole warp walks the tile's blocks and waits, one lane issues.
            const uint32_t lead = elect_lane();
            constexpr uint32_t idesc_s = tc_idesc(128, 64, 0), idesc_o = tc_idesc(128, D, 1);
            const uint32_t t = __reduce_or_sync(0xffffffffu, (uint32_t)(warp - kShMmaWarp));
            const uint32_t qd = desc_lo(smem_u32(base + L.q), 16u) +
                                (alt ? 0u : t * (128u * 128u >> 4));
            const uint32_t kd = desc_lo(smem_u32(base + L.kst), 16u);
            const uint32_t vd = desc_lo(smem_u32(base + L.vst), kHalf);
            const uint32_t tb = __reduce_or_sync(0xffffffffu, tbase);
            const uint32_t oc = tb + 128u * t, sc = tb + 256u + 128u * t;
            const int32_t nl = alt ? (n + 1 - (int32_t)t) / 2 : n;
            const uint32_t t0 = t ? tdone1 : tdone0;
            // a stage is given back by both warps, or twice by the one that read it
            auto release = [&](uint32_t b) {
                pb_commit(lead, b);
                if (alt) pb_commit(lead, b);
            };
            bool ok = true;
            for (int32_t jl = 0; jl <= nl && ok; ++jl) {
                if (jl < nl) {
                    const uint32_t i = done + (alt ? 2 * jl + t : jl), s = i % kShStages;
                    ok = wait(bar(kShKFull + s), (i / kShStages) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    // into buffer j % 2, whose P V (of the tile's block j - 2) was issued before
                    const uint32_t j = t0 + jl, to = sc + 64u * (j & 1u);
                    const uint32_t k_lo = kd + s * (64u * D * 2u >> 4);
                    pb_mma_ss<false>(lead, to, qd, k_lo, idesc_s);
#pragma unroll
                    for (int kk = 1; kk < D / 16; ++kk)
                        pb_mma_ss<true>(lead, to,
                                        qd + (((kk >> 2) * (kShRows * 128u) + (kk & 3) * 32u) >> 4),
                                        k_lo + (((kk >> 2) * kHalf + (kk & 3) * 32u) >> 4), idesc_s);
                    pb_commit(lead, bar(kShS) + 16u * t + 8u * (j & 1u));
                    release(bar(kShKEmpty + s));
                }
                if (jl > 0) {
                    const uint32_t i = done + (alt ? 2 * (jl - 1) + t : jl - 1), s = i % kShStages;
                    const uint32_t j = t0 + jl - 1;
                    ok = wait(bar(kShVFull + s), (i / kShStages) & 1) &&
                         wait(bar(kShP) + 16u * t + 8u * (j & 1u), (j >> 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t v_lo = vd + s * (64u * D * 2u >> 4), from = sc + 64u * (j & 1u);
                    const uint32_t more = (uint32_t)(jl - 1) & (kShEmpty - 1u);  // 0: a new sum
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            pb_mma_ts(lead, oc, from + 32u * part + 8u * kk, v_lo + (kk * 2048u >> 4),
                                      idesc_o, (part > 0 || kk > 0) ? 1u : more);
                    }
                    pb_commit(lead, bar(kShPv) + 8u * t);
                    release(bar(kShVEmpty + s));
                }
            }
            // every product is done: the epilogue's signal, and nothing of this warp's may still run on
            // the tensor cores when the CTA goes on
            pb_commit(lead, bar(kShDrain) + 8u * t);
            wait(bar(kShDrain) + 8u * t, piece & 1);
        } else if (warp < 8) {
            // ---------------------------------------------------------------- softmax threads
            const int t = warp >> 2, r = tid & 127;
            const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t ocol = tbase + lanes + 128u * t;
            const int32_t nl = alt ? (n + 1 - t) / 2 : n;
            const uint32_t t0 = t ? tdone1 : tdone0;
            const int32_t rid = alt ? r : 128 * t + r;  // the row of the segment
            const bool rowok = rid < pc.rows;
            int32_t lim = 0;  // the row sees the prefix's keys below lim
            if (rowok) {
                const int32_t rr = pc.row0 + rid, b = first + rr / tg, tok = (rr % tg) / p.g;
                const int32_t len = min(max(__ldcg(p.seq_lens + b), 0), p.max_pages * p.P);
                lim = min(prefix, len - p.T + tok + 1);
            }
            const int64_t slot = pc.slot + (alt ? t * pc.rows : 0) + rid;
            float* to = p.slots + slot * D;
            // |scale| log2(e), at least 1e-30 so that a masked key (-inf) never meets a zero factor
            const float sl2a = fmaxf(fabsf(p.sl2), 1e-30f);
            constexpr int32_t kFull = 16 | (16 << 5) | (16 << 10) | (16 << 15);
            float m_used = kPfNegInf, m_true = kPfNegInf, l = 0.f;  // l and O are relative to m_used
            float ref = kPfNegInf;              // and what the slot holds of earlier sums to ref
            bool ok = true;
            for (int32_t jl = 0; jl < nl; ++jl) {
                const uint32_t i = done + (alt ? 2 * jl + t : jl), j = t0 + jl;
                ok = wait(bar(kShMetaFull + i % kShMeta), (i / kShMeta) & 1) &&
                     wait(bar(kShS + 2 * t) + 8u * (j & 1u), (j >> 1) & 1u);
                if (!ok) break;
                tc_fence_after();
                const int2 mt = meta[i % kShMeta];
                const uint32_t sbuf = tbase + lanes + 256u + 128u * t + 64u * (j & 1u);
                if (jl > 0 && (jl & (kShEmpty - 1)) == 0) {
                    // the sum so far moves to the slot
                    ok = wait(bar(kShPv) + 8u * t, (j - 1) & 1u);
                    if (!ok) break;
                    tc_fence_after();
                    const float down = ref == kPfNegInf ? 0.f : exp2f(ref - m_used);
#pragma unroll 1
                    for (int cc = 0; cc < D / 16; ++cc) {
                        __syncwarp();
                        float v[16];
                        tc_ld16(ocol + 16u * cc, v);
                        tc_wait_ld();
                        if (rowok) {
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                float4* at = reinterpret_cast<float4*>(to + 16 * cc + e);
                                float4 o = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                                if (jl > kShEmpty) {
                                    const float4 a = *at;
                                    o = make_float4(fmaf(a.x, down, o.x), fmaf(a.y, down, o.y),
                                                    fmaf(a.z, down, o.z), fmaf(a.w, down, o.w));
                                }
                                *at = o;
                            }
                        }
                    }
                    __syncwarp();
                    tc_fence_before();
                    ref = m_used;
                }
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
                const int32_t cut = lim - mt.x * kPfBlock;
                if (!__all_sync(0xffffffffu, cut >= kPfBlock && mt.y == kFull)) {
                    int32_t lims[kPfTiles];
#pragma unroll
                    for (int u = 0; u < kPfTiles; ++u)
                        lims[u] = min(16 * u + ((mt.y >> (5 * u)) & 31), cut);
#pragma unroll
                    for (int e = 0; e < 64; ++e) xs[e] = e < lims[e >> 4] ? xs[e] : kPfNegInf;
                }
                const float mx = row_max64(xs) * sl2a;  // log2 units; -inf stays -inf
                m_true = fmaxf(m_true, mx);
                const bool need = mx > m_used + kTcRescale || (m_used == kPfNegInf && mx != kPfNegInf);
                const float f = need && m_used != kPfNegInf ? exp2f(m_used - mx) : 1.f;
                if (__any_sync(0xffffffffu, f != 1.f) && (jl & (kShEmpty - 1)) != 0) {
                    // O holds the blocks before this one: wait for them, then scale it
                    ok = wait(bar(kShPv) + 8u * t, (j - 1) & 1u);
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
                // p = 2^(x |scale| log2(e) - mu) in pairs; a masked key gives +0. P goes to the score
                // buffer as two bf16 terms: p cut to its upper 16 bits, and the exact rest, rounded.
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
                    // V rows past the prefix in a short tile hold other tokens or nothing: zeros, so that
                    // a zero weight cannot meet a NaN (P V of this block waits for this warp)
                    bool short_tile = false;
#pragma unroll
                    for (int u = 0; u < kPfTiles; ++u) {
                        const int32_t hi = (mt.y >> (5 * u)) & 31;
                        short_tile = short_tile || (hi > 0 && hi < 16);
                    }
                    if (short_tile && wait(bar(kShVFull + i % kShStages), (i / kShStages) & 1)) {
                        uint8_t* vst = base + L.vst + (i % kShStages) * L.blk_bytes;
                        for (int idx = r; idx < 64 * KH * 8; idx += 128) {
                            const int kr = idx / (KH * 8), rem = idx - kr * (KH * 8);
                            const int hh = rem >> 3, ch = rem & 7;
                            const int32_t hi = (mt.y >> (5 * (kr >> 4))) & 31;
                            if (hi > 0 && (kr & 15) >= hi)
                                *reinterpret_cast<uint4*>(vst + hh * kHalf + kr * 128 + ch * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                }
                __syncwarp();
                tc_fence_before();
                mbar_arrive(bar(kShP + 2 * t) + 8u * (j & 1u));
            }
            // ---- this row's sum and weight, relative to its maximum -----------------------------
            ok = wait(bar(kShDrain) + 8u * t, piece & 1) && ok;
            tc_fence_after();
            const bool some = nl > 0 && ok;
            const float fac = m_true == kPfNegInf ? 0.f : exp2f(m_used - m_true);
            const float down = ref == kPfNegInf ? 0.f : exp2f(ref - m_true);
#pragma unroll 1
            for (int cc = 0; cc < D / 16; ++cc) {
                __syncwarp();
                float v[16];
                if (some) {
                    tc_ld16(ocol + 16u * cc, v);
                    tc_wait_ld();
                }
                if (rowok && some) {
#pragma unroll
                    for (int e = 0; e < 16; e += 4) {
                        float4* at = reinterpret_cast<float4*>(to + 16 * cc + e);
                        float4 o = make_float4(v[e] * fac, v[e + 1] * fac, v[e + 2] * fac,
                                               v[e + 3] * fac);
                        if (nl > kShEmpty) {
                            const float4 a = *at;
                            o = make_float4(fmaf(a.x, down, o.x), fmaf(a.y, down, o.y),
                                            fmaf(a.z, down, o.z), fmaf(a.w, down, o.w));
                        }
                        *at = o;
                    }
                }
            }
            if (rowok)
                p.slot_me[slot] = make_float2(some ? m_true : kPfNegInf, some ? l * fac : 0.f);
            tc_fence_before();
        }
        done += n;
        tdone0 += alt ? (n + 1) / 2 : n;
        tdone1 += alt ? n / 2 : n;
        __syncthreads();  // the query rows and the accumulators are free
        tc_fence_after();
        if (*abort_p) break;
    }
    // ---- teardown: the allocating warp frees the tensor memory ----------------------------------
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tc_dealloc(tbase, 512u);
    }
    // the merge waits for this kernel alone, and so this one for the engine
    grid_dependency_wait();
}

struct ShMerge {
    int32_t B, T, Hq, Hkv, g, groups;
    const int32_t* group_indptr;
    const float* slots;
    const float2* slot_me;
    const int32_t* plan;
    const float* own;    // [B][T][Hq][D] MA of the own tokens
    const float* own_m;  // [B][T][Hq], log2 units
    const float* own_e;
    float* out;
    int32_t out_bf16;
    float* m_g;
    float* e_g;
};

constexpr int kShMergeThreads = 128;

// D/4 lanes join the pieces of a row: (m, e, MA) of its own tokens and of every run of its prefix.
template <int D>
__global__ void __launch_bounds__(kShMergeThreads)
shared_merge_kernel(const __grid_constant__ ShMerge p) {
    constexpr int LPR = D / 4, kBatch = 8;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = (int64_t)blockIdx.x * (kShMergeThreads / LPR) + threadIdx.x / LPR;
    const int d = 4 * (threadIdx.x % LPR);
    if (row >= (int64_t)p.B * p.T * p.Hq) return;
    const int32_t h = (int32_t)(row % p.Hq);
    const int32_t bt = (int32_t)(row / p.Hq), b = bt / p.T, t = bt - b * p.T;
    const int32_t W = __ldcg(p.plan);
    const int32_t i = W > 0 ? shared_group(p.group_indptr, p.groups, b) : -1;
    // the row's place in its segment, the runs' rows: the q'th at first + q step (+ rows: a second half)
    int64_t first = 0;
    int32_t runs = 0, second = 0;
    if (i >= 0) {
        const int32_t Gw = __ldcg(p.plan + 1), prefix = __ldcg(p.plan + 3 + p.groups + i);
        const int32_t c0 = __ldcg(p.group_indptr + i);
        const int32_t rows = (__ldcg(p.group_indptr + i + 1) - c0) * p.T * p.g;
        const int32_t pairs = (rows + kShRows - 1) / kShRows;
        const int32_t blocks = (prefix + kPfBlock - 1) / kPfBlock;
        if (blocks > 0) {
            const int32_t kvh = h / p.g, rr = ((b - c0) * p.T + t) * p.g + (h - kvh * p.g);
            const int32_t pair = rr / kShRows, rid = rr - pair * kShRows;
            const int32_t seg_rows = min(kShRows, rows - pair * kShRows);
            const int64_t cs = __ldcg(p.plan + 2 + i) +
                               (int64_t)(kvh * pairs + pair) * (blocks + kShSegCost);
            const int32_t cf = split_owner(cs, W, Gw), cl = split_owner(cs + blocks - 1, W, Gw);
            first = 2 * ((int64_t)c0 * p.T * p.Hq + (int64_t)kvh * rows + pair * kShRows) +
                    (int64_t)kShRows * cf + rid;
            second = seg_rows <= 128 ? seg_rows : 0;
            runs = (cl - cf + 1) * (second > 0 ? 2 : 1);
        }
    }
    float m = __ldcg(p.own_m + row), e = __ldcg(p.own_e + row);
    float4 acc = __ldcg(reinterpret_cast<const float4*>(p.own + row * D + d));
    for (int32_t q0 = 0; q0 < runs; q0 += kBatch) {
        float2 me[kBatch];
        float4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int32_t q = q0 + k;
            const int64_t at = second > 0 ? first + (int64_t)kShRows * (q >> 1) + (q & 1) * second
                                          : first + (int64_t)kShRows * q;
            me[k] = make_float2(kPfNegInf, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (q < runs) {
                me[k] = __ldcg(p.slot_me + at);
                v[k] = __ldcg(reinterpret_cast<const float4*>(p.slots + at * D + d));
            }
        }
        float mx = m;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) mx = fmaxf(mx, me[k].x);
        if (mx == kPfNegInf) continue;  // nothing is seen so far
        const float f = m == kPfNegInf ? 0.f : exp2f(m - mx);
        e *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (me[k].x == kPfNegInf) continue;  // (the run's row may never have been written)
            const float w = exp2f(me[k].x - mx);
            e = fmaf(me[k].y, w, e);
            acc = make_float4(fmaf(v[k].x, w, acc.x), fmaf(v[k].y, w, acc.y), fmaf(v[k].z, w, acc.z),
                              fmaf(v[k].w, w, acc.w));
        }
        m = mx;
    }
    const float inv = e > 0.f ? 1.f / e : 0.f;
    acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (p.out_bf16 != 0)
        *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + row * D + d) =
            make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    else
        *reinterpret_cast<float4*>(p.out + row * D + d) = acc;
    if (d == 0) {
        if (p.m_g) p.m_g[row] = m == kPfNegInf ? kPfNegInf : m * kLn2;
        if (p.e_g) p.e_g[row] = e;
    }
}

// The workspace: the engine's, then the partials of the own tokens, the pieces' rows and the plan.
struct ShWorkspace {
    size_t own, own_m, own_e, slots, slot_me, plan, total;
};
ShWorkspace shared_workspace(int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D) {
    const int64_t rows = (int64_t)B * T * Hq;
    const int64_t slots = shared_slot_rows(rows, sm_count_current());
    ShWorkspace w;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += (bytes + 255) & ~(size_t)255;
        return at;
    };
    take(attn_workspace_bytes(B * Hkv, Hq / Hkv * T, D, sm_count_current() * kMaxCtasPerSm));
    w.own = take((size_t)rows * D * 4);
    w.own_m = take((size_t)rows * 4);
    w.own_e = take((size_t)rows * 4);
    w.slots = take((size_t)slots * D * 4);
    w.slot_me = take((size_t)slots * 8);
    w.plan = take((size_t)(2 * (B < kShMaxGroups ? B : kShMaxGroups) + 3) * 4);
    w.total = o;
    return w;
}

std::mutex g_sh_mutex;

template <int D, int FMT>
dattn_status_t launch_prefix(const ShParams& p, const void* k_pool, const void* v_pool,
                             cudaStream_t stream) {
    const ShSmem L = sh_smem_layout(D, p.groups);
    {
        static int set[kMaxDevices] = {};  // a function attribute belongs to a device
        std::lock_guard<std::mutex> lock(g_sh_mutex);
        int& mine = set[device_index()];
        if ((int)L.total > mine) {
            if (cudaFuncSetAttribute(shared_prefix_kernel<D, FMT>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)L.total) != cudaSuccess)
                return DATTN_ERR_CUDA;
            mine = (int)L.total;
        }
    }
    alignas(64) CUtensorMap tk{};
    alignas(64) CUtensorMap tv{};
    if (FMT == DATTN_KV_BF16) {
        const int64_t rows = (int64_t)p.num_pages * p.Hkv * p.P;
        dattn_status_t st;
        if ((st = make_half_tensor_map(&tk, k_pool, rows, D)) != DATTN_OK) return st;
        if ((st = make_half_tensor_map(&tv, v_pool, rows, D)) != DATTN_OK) return st;
    }
    return launch_pdl(shared_prefix_kernel<D, FMT>, dim3((unsigned)sm_count_current()),
                      dim3(kShThreads), L.total, stream, p, tk, tv) == cudaSuccess
               ? DATTN_OK
               : DATTN_ERR_CUDA;
}

}  // namespace
}  // namespace dattn

using namespace dattn;

extern "C" {

size_t dattn_shared_workspace_size(int32_t B, int32_t T, int32_t Hq, int32_t Hkv,
                                   int32_t head_dim) {
    if (B < 0 || B > kMaxItems || T < 1 || Hq <= 0 || Hkv <= 0 || Hkv > kMaxKvHeads ||
        Hq % Hkv != 0 || Hq / Hkv * (int64_t)T > kMaxGroup)
        return 0;
    if (head_dim != 64 && head_dim != 128) return 0;
    return shared_workspace(B, T, Hq, Hkv, head_dim).total;
}

dattn_status_t dattn_decode_shared(const dattn_kv_layout* layout, const void* k_pool,
                                   const void* v_pool, const dattn_bf16* q, int32_t B, int32_t T,
                                   int32_t Hq, float scale, const int32_t* seq_lens,
                                   int32_t num_groups, const int32_t* group_indptr,
                                   const int32_t* prefix_lens, void* ws, size_t ws_bytes, void* out,
                                   int32_t out_bf16, float* m_g, float* e_g, int32_t* dev_err,
                                   void* stream) {
    dattn_status_t st = check_layout(layout);
    if (st != DATTN_OK) return st;
    if ((st = check_heads(layout, B, Hq)) != DATTN_OK) return st;
    if (T < 1 || num_groups < 0 || num_groups > B || (out_bf16 & ~1)) return DATTN_ERR_INVALID_ARG;
    if (layout->kv_format != DATTN_KV_BF16 && layout->kv_format != DATTN_KV_FP8_BLOCK)
        return DATTN_ERR_UNSUPPORTED;
    const int32_t g = Hq / layout->num_kv_heads, D = layout->head_dim;
    if (g * (int64_t)T > kMaxGroup || num_groups > kShMaxGroups) return DATTN_ERR_UNSUPPORTED;
    if (B == 0) return DATTN_OK;
    if (!k_pool || !v_pool || !q || !seq_lens || !out ||
        (num_groups > 0 && (!group_indptr || !prefix_lens)))
        return DATTN_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(q) || !aligned16(out))
        return DATTN_ERR_INVALID_ARG;
    const int64_t tokens = (int64_t)layout->max_pages_per_req * layout->page_size;
    const int64_t bound = (int64_t)B * layout->num_kv_heads *
                          (tokens / 16 + seg_cost(layout->kv_format, g * T));
    const int64_t segments =
        (int64_t)layout->num_kv_heads * ((int64_t)B * T * g / kShRows + num_groups);
    if (bound >= (1ll << 31) || segments * (tokens / kPfBlock + 1 + kShSegCost) >= (1ll << 31))
        return DATTN_ERR_UNSUPPORTED;
    const ShWorkspace w = shared_workspace(B, T, Hq, layout->num_kv_heads, D);
    if (ws == nullptr || ws_bytes < w.total || (reinterpret_cast<uintptr_t>(ws) & 255))
        return DATTN_ERR_WORKSPACE;
    uint8_t* wb = static_cast<uint8_t*>(ws);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool shared = num_groups > 0;
    // the own tokens: with groups as partials in the workspace
    AttnParams a{};
    a.mode = MODE_WINDOW;
    a.num_pages = layout->num_pages;
    a.Hkv = layout->num_kv_heads;
    a.P = layout->page_size;
    a.max_pages = layout->max_pages_per_req;
    a.block_table = layout->block_table;
    a.q = q;
    a.B = B;
    a.Hq = Hq;
    a.g = g;
    a.T = T;
    a.gq = g * T;
    a.sl2 = scale * kLog2e;
    a.seq_lens = seq_lens;
    a.window = 1 << 30;
    a.groups = num_groups;
    a.group_indptr = group_indptr;
    a.prefix_lens = prefix_lens;
    a.normalise = shared ? 0 : 1;
    a.out = shared ? reinterpret_cast<float*>(wb + w.own) : static_cast<float*>(out);
    a.out_bf16 = shared ? 0 : out_bf16;
    a.m_out = shared ? reinterpret_cast<float*>(wb + w.own_m) : m_g;
    a.e_out = shared ? reinterpret_cast<float*>(wb + w.own_e) : e_g;
    a.nseg = B * a.Hkv;
    a.nitems = B;
    a.dev_err = dev_err;
    a.fmt = layout->kv_format;
    a.kv_scale = layout->kv_scale;
    if ((st = launch_attention_window(a, k_pool, v_pool, D, 0, ws, w.own, s, bound)) != DATTN_OK)
        return st;
    if (!shared) return DATTN_OK;
    ShParams p{};
    p.num_pages = a.num_pages;
    p.Hkv = a.Hkv;
    p.P = a.P;
    p.max_pages = a.max_pages;
    p.block_table = a.block_table;
    p.q = q;
    p.B = B;
    p.T = T;
    p.Hq = Hq;
    p.g = g;
    p.sl2 = a.sl2;
    p.seq_lens = seq_lens;
    p.groups = num_groups;
    p.group_indptr = group_indptr;
    p.prefix_lens = prefix_lens;
    p.k_pool = static_cast<const uint8_t*>(k_pool);
    p.v_pool = static_cast<const uint8_t*>(v_pool);
    p.scale = reinterpret_cast<const float2*>(layout->kv_scale);
    p.slots = reinterpret_cast<float*>(wb + w.slots);
    p.slot_me = reinterpret_cast<float2*>(wb + w.slot_me);
    p.plan = reinterpret_cast<int32_t*>(wb + w.plan);
    p.dev_err = dev_err;
    const bool blk = layout->kv_format == DATTN_KV_FP8_BLOCK;
    auto launch = D == 64 ? (blk ? launch_prefix<64, DATTN_KV_FP8_BLOCK>
                                 : launch_prefix<64, DATTN_KV_BF16>)
                          : (blk ? launch_prefix<128, DATTN_KV_FP8_BLOCK>
                                 : launch_prefix<128, DATTN_KV_BF16>);
    if ((st = launch(p, k_pool, v_pool, s)) != DATTN_OK) return st;
    ShMerge m{};
    m.B = B;
    m.T = T;
    m.Hq = Hq;
    m.Hkv = a.Hkv;
    m.g = g;
    m.groups = num_groups;
    m.group_indptr = group_indptr;
    m.slots = p.slots;
    m.slot_me = p.slot_me;
    m.plan = p.plan;
    m.own = a.out;
    m.own_m = a.m_out;
    m.own_e = a.e_out;
    m.out = static_cast<float*>(out);
    m.out_bf16 = out_bf16;
    m.m_g = m_g;
    m.e_g = e_g;
    const int64_t rows = (int64_t)B * T * Hq;
    const int64_t per = kShMergeThreads / (D / 4);
    const dim3 grid((unsigned)((rows + per - 1) / per)), block(kShMergeThreads);
    const cudaError_t err = D == 64 ? launch_pdl(shared_merge_kernel<64>, grid, block, 0, s, m)
                                    : launch_pdl(shared_merge_kernel<128>, grid, block, 0, s, m);
    return err == cudaSuccess ? DATTN_OK : DATTN_ERR_CUDA;
}

}  // extern "C"
