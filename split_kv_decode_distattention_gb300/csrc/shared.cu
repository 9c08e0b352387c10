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
//   2. tile_attention.cuh's kernel over the prefixes, which needs nothing of 1 and starts as its CTAs
//      leave. A segment is a (group, KV head, up to 256 rows: a pair of tiles, or one tile); the 64-key
//      blocks of all segments are laid end to end and cut into equal runs, one per CTA, which leaves the
//      unnormalised sum, maximum and weight of a segment's rows in the workspace for every piece of it in
//      its run;
//   3. shared_merge_kernel, which joins the pieces.
// What bounds 2: from 128 rows on the tensor cores (1.1 us for a block of 256 rows on an SM), below the tiles'
// latency (0.8 us a block; block-scaled pool: the widening, 1.3 us). Measured on a GB300, 32 / 8 heads of 128: 64
// requests behind 16384 tokens with 100-2000 of their own 69 us (engine 34, prefix 22, merge 7); 4 requests behind
// 1808 tokens 18 us; 4 and 64 requests of 10 tokens behind 65536 tokens 65 and 97 us (268 MB of prefix).
#include "shared.cuh"
#include "tile_attention.cuh"

namespace dattn {

namespace {

// Key blocks of a tile whose sum stays in tensor memory, where the tensor cores add rounding towards
// zero: 8 products a block, each losing up to 2^-24 of the sum. A longer piece is joined in the
// workspace in fp32.
constexpr int32_t kShEmpty = 64;
constexpr int32_t kShSegCost = 4;    // a piece's fixed cost in blocks
constexpr int32_t kShMinCost = 5;    // blocks (and fixed costs) of a CTA at least: 4 requests behind 1808 tokens
                                     // 21.6 us with 2, 19.0 with 4, 17.6 with 5, 19.1 with 8
constexpr int32_t kShMaxGroups = kTaThreads;  // (a thread for each)

struct SharedParams {
    int32_t B, T;
    const int32_t* seq_lens;
    int32_t groups;
    const int32_t* group_indptr;
    const int32_t* prefix_lens;
    // the workspace: the pieces' rows, and (m in log2 units, e) of each; the plan: per group its first
    // request, its requests, its prefix and its first cost unit; then W and the CTAs with work, and per
    // request its group (-1: none)
    float* slots;
    float2* slot_me;
    int4* plan;
};

// The rows of pieces in the workspace: a piece of segment s in CTA c begins at rowbase(s) + 256 c, where
// rowbase counts the rows of earlier segments, and has up to 256 rows: the pieces of a CTA, and of a
// segment, are apart. A tile's R rows of D channels lie as [D/4][R] float4, so that the threads of a warp,
// a row each, write whole lines.
__host__ __device__ inline int64_t shared_slot_rows(int64_t rows, int32_t ctas) {
    return rows + 256ll * ctas;
}

// A group's geometry: its query tokens, its segments of a KV head and the cost of one.
struct SharedGroup {
    int32_t tokens, pairs, blocks, cost;
    __device__ SharedGroup(int32_t requests, int32_t T, int32_t tok, int32_t prefix) {
        tokens = requests * T;
        pairs = (tokens + 2 * tok - 1) / (2 * tok);
        blocks = (prefix + kPfBlock - 1) / kPfBlock;
        cost = blocks > 0 ? blocks + kShSegCost : 0;
    }
};

__host__ __device__ __forceinline__ int32_t shared_ctas(int32_t W, int32_t grid) {
    const int32_t c = W / kShMinCost;
    return c < 1 ? 1 : c < grid ? c : grid;
}

// The plan in shared memory: 8 bytes per group, two arrays of groups + 1 integers, and the scan's 16
inline uint32_t shared_job_bytes(int32_t groups) { return (uint32_t)groups * 16u + 8u + 64u; }

template <int D>
struct SharedJob {
    using Params = SharedParams;
    const TaParams& p;
    const Params& w;
    // per group: (prefix, the request whose pages hold it); its first cost unit; its first request
    const int2* info;
    const int32_t* start;
    const int32_t* ind;
    int32_t x, X1;      // cost units that are still to come
    int32_t j, j1;      // the blocks that are left of the piece
    int32_t acc;        // the slot holds earlier blocks of the piece
    int64_t slot;       // the piece's first row in the workspace
    // this thread's row
    int64_t me_at;
    float4* to;
    int32_t rows;
    float fn, fo, max_, sum_;

    __device__ SharedJob(const TaParams& p_, const Params& w_, uint8_t* smem) : p(p_), w(w_) {
        // No dependency wait here: the kernel before on the stream is the engine's launch of the same
        // call, whose results this one does not read, and whose CTAs let this kernel start only after
        // their own wait: what this call reads is there, in L2, and is read from L2 (an SM's L1 may be
        // older).
        grid_launch_dependents();
        unsigned long long* key = reinterpret_cast<unsigned long long*>(smem);
        int2* inf = reinterpret_cast<int2*>(smem);
        int32_t* st = reinterpret_cast<int32_t*>(smem + 8 * w.groups);
        int32_t* id = st + w.groups + 1;
        int32_t* scan = id + w.groups + 1;
        info = inf;
        start = st;
        ind = id;
        const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
        const int32_t cap = p.max_pages * p.P;
        // a thread per group; its bounds, its prefix and the lengths are all asked for at once
        int32_t prefix = 0, len = tid < w.B ? __ldcg(w.seq_lens + tid) : 0;
        if (tid < w.groups) {
            key[tid] = 0ull;
            id[tid] = __ldcg(w.group_indptr + tid);
            prefix = __ldcg(w.prefix_lens + tid);
        }
        if (tid == 0) id[w.groups] = __ldcg(w.group_indptr + w.groups);
        __syncthreads();
        bool order = true;
        if (tid < w.groups) order = id[tid] >= 0 && id[tid] <= id[tid + 1] && id[tid + 1] <= w.B;
        order = __syncthreads_and(order) != 0;
        int32_t W = 0;
        if (order) {  // (else the engine attends everything)
            // the longest request of a group has all pages of its prefix; the first of several
            for (int32_t i = tid; i < w.B; i += kTaThreads) {
                if (i != tid) len = __ldcg(w.seq_lens + i);
                int32_t lo = 0, hi = w.groups;  // the groups that end at or before i
                while (lo < hi) {
                    const int32_t mid = (lo + hi) >> 1;
                    if (id[mid + 1] <= i) lo = mid + 1; else hi = mid;
                }
                const bool in = lo < w.groups && id[lo] <= i;
                if (in)
                    atomicMax(key + lo,
                              ((unsigned long long)min(max(len, 0), cap) << 32) | (uint32_t)~i);
                if (blockIdx.x == 0) reinterpret_cast<int32_t*>(w.plan + w.groups + 1)[i] = in ? lo : -1;
            }
            __syncthreads();
            int32_t cost = 0;
            if (tid < w.groups) {
                const unsigned long long k = key[tid];
                prefix = min(max(prefix, 0), (int32_t)(k >> 32));
                inf[tid] = make_int2(prefix, (int32_t)~(uint32_t)k);
                const SharedGroup G(id[tid + 1] - id[tid], w.T, p.tok, prefix);
                cost = p.Hkv * G.pairs * G.cost;
            }
            int32_t incl = cost;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int32_t v = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += v;
            }
            if (lane == 31) scan[warp] = incl;
            __syncthreads();
            int32_t run = incl - cost;
            for (int v = 0; v < kTaThreads / 32; ++v) {
                if (v < warp) run += scan[v];
                W += scan[v];
            }
            if (tid < w.groups) st[tid] = run;
            __syncthreads();
        }
        const int32_t cta = blockIdx.x, Gw = shared_ctas(W, gridDim.x);
        if (cta == 0) {  // for the merge
            if (tid < w.groups && W > 0)
                w.plan[tid] = make_int4(id[tid], id[tid + 1] - id[tid], inf[tid].x, st[tid]);
            if (tid == 0) w.plan[w.groups] = make_int4(W, Gw, 0, 0);
        }
        x = X1 = 0;
        j = j1 = 0;
        if (cta < Gw && W > 0) {
            x = (int32_t)split_begin(W, Gw, cta);
            X1 = (int32_t)split_begin(W, Gw, cta + 1);
        }
    }
    __device__ static void skip() {
        grid_launch_dependents();
        grid_dependency_wait();
    }
    // the merge waits for this kernel alone, and so this one for the engine
    __device__ void end() { grid_dependency_wait(); }

    __device__ bool next(TaItem& it) {
        acc = 1;
        while (j >= j1) {  // the next piece
            if (x >= X1) return false;
            int32_t lo = 0, hi = w.groups - 1;  // the last group with start <= x
            while (lo < hi) {
                const int32_t mid = (lo + hi + 1) >> 1;
                if (start[mid] <= x) lo = mid; else hi = mid - 1;
            }
            const SharedGroup G(ind[lo + 1] - ind[lo], w.T, p.tok, info[lo].x);
            const int32_t seg = (x - start[lo]) / G.cost, cs = start[lo] + seg * G.cost;
            it.kvh = seg / G.pairs;
            const int32_t tok0 = (seg - it.kvh * G.pairs) * 2 * p.tok, left = G.tokens - tok0;
            j = x - cs;
            j1 = min(X1 - cs, G.blocks);
            x = cs + G.cost;
            slot = (int64_t)ind[lo] * w.T * p.Hq + (int64_t)it.kvh * G.tokens * p.g + tok0 * p.g +
                   256ll * blockIdx.x;
            acc = 0;
            it.tok[0] = min(p.tok, left);
            it.tok[1] = min(p.tok, max(left - p.tok, 0));
            it.alt = it.tok[1] == 0 ? 1 : 0;
            it.n0 = ind[lo] * w.T + tok0;
            it.trow = info[lo].y;
            it.kmax = info[lo].x;
            it.first = it.low = it.sinks = 0;
        }
        it.from = j;
        it.count = min(j1 - j, it.alt ? 2 * kShEmpty : kShEmpty);
        j += it.count;
        const int32_t c = it.count - 1;
        it.last[0] = it.alt ? c - (c & 1) : c;
        it.last[1] = it.alt ? c - 1 + (c & 1) : c;
        return true;
    }
    __device__ bool keeps(const TaItem&, int, int32_t) const { return true; }
    __device__ void row(const TaItem& it, int t, int r, TaRow& out) {
        if (it.alt) t = 0;
        const int32_t tok = r / p.g, n = it.n0 + t * p.tok + tok;
        out.ok = tok < it.tok[t];
        out.low = 0;
        out.sinks = 0;
        // (rows of no query compute on what the copy brought, and see all of it)
        out.lim = 0x7fffffff;
        if (out.ok) {
            const int32_t b = n / w.T;
            const int32_t len = min(max(__ldcg(w.seq_lens + b), 0), p.max_pages * p.P);
            out.lim = min(it.kmax, len - w.T + (n - b * w.T) + 1);
        }
        rows = it.tok[t] * p.g;
        const int64_t first = slot + t * p.tok * p.g;
        me_at = first + r;
        to = reinterpret_cast<float4*>(w.slots + first * D) + r;
    }
    __device__ void begin_row(bool ok, float m, float sum) {
        max_ = m;
        sum_ = sum;
        fn = 1.f;
        fo = 0.f;
        if (acc && ok) {
            const float2 old = __ldcg(w.slot_me + me_at);
            max_ = fmaxf(m, old.x);
            fn = m == kPfNegInf ? 0.f : exp2f(m - max_);
            fo = old.x == kPfNegInf ? 0.f : exp2f(old.x - max_);
            sum_ = sum * fn + old.y * fo;
        }
    }
    __device__ void write16(int c, const float (&v)[16]) const {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float4* at = to + (int64_t)(c / 4 + e) * rows;
            float4 o = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            if (acc) {
                const float4 a = __ldcg(at);
                o = make_float4(fmaf(a.x, fo, o.x * fn), fmaf(a.y, fo, o.y * fn),
                                fmaf(a.z, fo, o.z * fn), fmaf(a.w, fo, o.w * fn));
            }
            __stcg(at, o);
        }
    }
    __device__ void finish_row() const { __stcg(w.slot_me + me_at, make_float2(max_, sum_)); }
};

struct MergeParams {
    int32_t B, T, Hq, g, tok, groups;
    const float* slots;
    const float2* slot_me;
    const int4* plan;
    const float* own;    // [B][T][Hq][D] MA of the own tokens
    const float* own_m;  // [B][T][Hq], log2 units
    const float* own_e;
    float* out;
    int32_t out_bf16;
    float* m_g;
    float* e_g;
};

constexpr int kMergeThreads = 128;

// Joins the pieces of a row, (m, e, MA) of its own tokens and of every run of its prefix. A block takes
// 512 / D rows, in the order of the segments' rows (KV head, token, query head of the KV head), a thread
// four channels of one; neighbouring threads take neighbouring rows, as the pieces lie. Bound by latency: what
// a row needs to know takes two loads in turn, and the runs of most rows are asked for in one go (64
// requests of 32 heads, 20 runs: 8.5 us with four loads in turn and eight runs at a time).
template <int D>
__global__ void __launch_bounds__(kMergeThreads)
shared_merge_kernel(const __grid_constant__ MergeParams p) {
    constexpr int RB = 512 / D, kBatch = 24;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t n = (int64_t)blockIdx.x * RB + threadIdx.x % RB;
    const int c4 = threadIdx.x / RB;
    const int32_t N = p.B * p.T;
    if (n >= (int64_t)N * p.Hq) return;
    const int32_t kvh = (int32_t)(n / ((int64_t)N * p.g));
    const int32_t k = (int32_t)(n - (int64_t)kvh * N * p.g);
    const int32_t bt = k / p.g, b = bt / p.T;  // the query token and its request
    const int64_t row = (int64_t)bt * p.Hq + kvh * p.g + (k - bt * p.g);
    float m = __ldcg(p.own_m + row), e = __ldcg(p.own_e + row);
    float4 acc = __ldcg(reinterpret_cast<const float4*>(p.own + row * D) + c4);
    const int4 head = __ldcg(p.plan + p.groups);
    const int32_t i = head.x > 0 ? __ldcg(reinterpret_cast<const int32_t*>(p.plan + p.groups + 1) + b) : -1;
    // the q'th run's rows begin at first + 256 q; this thread's is the r'th of `rows`
    int64_t first = 0;
    int32_t runs = 0, rows = 0, r = 0;
    if (i >= 0) {
        const int4 group = __ldcg(p.plan + i);
        const SharedGroup G(group.y, p.T, p.tok, group.z);
        if (G.blocks > 0) {
            const int32_t tk = bt - group.x * p.T, pair = tk / (2 * p.tok), in = tk - pair * 2 * p.tok;
            const int32_t t = in / p.tok, left = G.tokens - pair * 2 * p.tok - t * p.tok;
            const int64_t cs = group.w + (int64_t)(kvh * G.pairs + pair) * G.cost;
            const int32_t cf = split_owner(cs, head.x, head.y);
            runs = split_owner(cs + G.blocks - 1, head.x, head.y) - cf + 1;
            rows = min(p.tok, left) * p.g;
            r = (in - t * p.tok) * p.g + (k - bt * p.g);
            first = (int64_t)group.x * p.T * p.Hq + (int64_t)kvh * G.tokens * p.g +
                    (pair * 2 + t) * p.tok * p.g + 256ll * cf;
        }
    }
    for (int32_t q0 = 0; q0 < runs; q0 += kBatch) {
        float2 me[kBatch];
        float4 v[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const int64_t at = first + 256ll * (q0 + x);
            me[x] = make_float2(kPfNegInf, 0.f);
            v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (q0 + x < runs) {
                me[x] = __ldcg(p.slot_me + at + r);
                v[x] = __ldcg(reinterpret_cast<const float4*>(p.slots + at * D) + (int64_t)c4 * rows + r);
            }
        }
        float mx = m;
#pragma unroll
        for (int x = 0; x < kBatch; ++x) mx = fmaxf(mx, me[x].x);
        if (mx == kPfNegInf) continue;  // nothing is seen so far
        const float f = m == kPfNegInf ? 0.f : exp2f(m - mx);
        e *= f;
        acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const float u = me[x].x == kPfNegInf ? 0.f : exp2f(me[x].x - mx);
            e = fmaf(me[x].y, u, e);
            acc = make_float4(fmaf(v[x].x, u, acc.x), fmaf(v[x].y, u, acc.y), fmaf(v[x].z, u, acc.z),
                              fmaf(v[x].w, u, acc.w));
        }
        m = mx;
    }
    const float inv = e > 0.f ? 1.f / e : 0.f;
    acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (p.out_bf16 != 0)
        reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p.out) + row * D)[c4] =
            make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    else
        reinterpret_cast<float4*>(p.out + row * D)[c4] = acc;
    if (c4 == 0) {
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
    w.plan = take((size_t)((B < kShMaxGroups ? B : kShMaxGroups) + 1) * 16 + (size_t)B * 4);
    w.total = o;
    return w;
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
        (int64_t)layout->num_kv_heads * ((int64_t)B * T * g / 128 + num_groups);
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
    TaParams p{};
    p.num_pages = a.num_pages;
    p.Hkv = a.Hkv;
    p.P = a.P;
    p.max_pages = a.max_pages;
    p.block_table = a.block_table;
    p.Hq = Hq;
    p.g = g;
    p.tok = 128 / g;
    p.sl2 = a.sl2;
    p.scale = reinterpret_cast<const float2*>(layout->kv_scale);
    p.dev_err = dev_err;
    SharedParams sp{};
    sp.B = B;
    sp.T = T;
    sp.seq_lens = seq_lens;
    sp.groups = num_groups;
    sp.group_indptr = group_indptr;
    sp.prefix_lens = prefix_lens;
    sp.slots = reinterpret_cast<float*>(wb + w.slots);
    sp.slot_me = reinterpret_cast<float2*>(wb + w.slot_me);
    sp.plan = reinterpret_cast<int4*>(wb + w.plan);
    const bool blk = layout->kv_format == DATTN_KV_FP8_BLOCK;
    auto launch = D == 64 ? (blk ? launch_tiles<SharedJob<64>, 64, DATTN_KV_FP8_BLOCK>
                                 : launch_tiles<SharedJob<64>, 64, DATTN_KV_BF16>)
                          : (blk ? launch_tiles<SharedJob<128>, 128, DATTN_KV_FP8_BLOCK>
                                 : launch_tiles<SharedJob<128>, 128, DATTN_KV_BF16>);
    if ((st = launch(p, sp, q, (int64_t)B * T, k_pool, v_pool, sm_count_current(),
                     shared_job_bytes(num_groups), s)) != DATTN_OK)
        return st;
    MergeParams m{};
    m.B = B;
    m.T = T;
    m.Hq = Hq;
    m.g = g;
    m.tok = p.tok;
    m.groups = num_groups;
    m.slots = sp.slots;
    m.slot_me = sp.slot_me;
    m.plan = sp.plan;
    m.own = a.out;
    m.own_m = a.m_out;
    m.own_e = a.e_out;
    m.out = static_cast<float*>(out);
    m.out_bf16 = out_bf16;
    m.m_g = m_g;
    m.e_g = e_g;
    const int64_t rows = (int64_t)B * T * Hq, per = 512 / D;
    const dim3 grid((unsigned)((rows + per - 1) / per)), block(kMergeThreads);
    const cudaError_t err = D == 64 ? launch_pdl(shared_merge_kernel<64>, grid, block, 0, s, m)
                                    : launch_pdl(shared_merge_kernel<128>, grid, block, 0, s, m);
    return err == cudaSuccess ? DATTN_OK : DATTN_ERR_CUDA;
}

}  // extern "C"
