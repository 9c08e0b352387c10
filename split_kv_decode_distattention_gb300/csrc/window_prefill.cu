// dattn_prefill_window: a chunk of Tq new tokens per request attends the paged cache through a sliding
// window with first tokens that stay visible. The query at position p sees the keys i <= p with
// i > p - window or i < sinks ("LLM长序列服务优化：LServe的块稀疏注意力技术" §2.1.2 keeps whole 64-token
// blocks of this pattern; here it is exact).
//
// The kernel is tile_attention.cuh's. An item is 2 * 128 / g neighbouring query tokens of one request
// under one KV head (or half of them, see below) over the key blocks that their windows and the first
// tokens touch, found without a list: the blocks of the first tokens, then those from the first query's
// window on. A tile skips the blocks that only the other one sees, and masks rows in the blocks at the
// windows' edges. Items run from a chunk's last tokens to its first, the KV heads side by side. Where the
// last round of items would fill at most half of the SMs (and so for few items), each becomes two of one
// tile, whose blocks the CTA's two tiles share.
//
// What bounds it: the tensor cores, three products of 128 x 64 x d for two that count, and the softmax
// (with a short window an item's first scores and its epilogue; over the block-scaled pool the widening).
// Measured on a GB300, 32 / 8 heads of 128: a prompt of 16K tokens, bf16 pool, through a window of 64, 1024, 4096
// and without one 130, 354, 1001 and 2275 us (967 TFLOP/s counted); 4096 tokens after 28K through 4096,
// block-scaled pool, 362 us (772 TFLOP/s).
#include "tile_attention.cuh"

namespace dattn {

namespace {

struct WindowParams {
    int32_t B, Tq;
    const int32_t* seq_lens;
    int32_t window, sinks;
    int32_t pairs;         // pairs of tiles of a request and KV head
    int32_t whole, items;  // items [0, whole) are pairs, the others single tiles
    void* out;
    int32_t out_bf16;
    float* m;
    float* e;
};

template <int D>
struct WindowJob {
    using Params = WindowParams;
    const TaParams& p;
    const Params& w;
    int32_t at, pos;  // pos: the position of the item's first token
    int64_t row_at;   // this thread's row of the output
    float inv, max_, sum_;

    __device__ WindowJob(const TaParams& p_, const Params& w_, uint8_t*) : p(p_), w(w_), at(blockIdx.x) {
        grid_dependency_wait();  // the lengths, the queries and the pool may come from the previous kernel
        grid_launch_dependents();
    }
    __device__ static void skip() {}
    __device__ void end() {}

    __device__ bool next(TaItem& it) {
        while (at < w.items) {
            int32_t x = at;
            at += gridDim.x;
            it.alt = x >= w.whole ? 1 : 0;
            const int32_t half = it.alt ? (x - w.whole) & 1 : 0;
            if (it.alt) x = w.whole + ((x - w.whole) >> 1);
            it.kvh = x % p.Hkv;
            x /= p.Hkv;
            const int32_t pair = w.pairs - 1 - x % w.pairs, b = x / w.pairs;
            const int32_t L = __ldg(w.seq_lens + b);
            if (L < w.Tq || L > p.max_pages * p.P) {
                if (threadIdx.x == 0) set_err(p.dev_err, DATTN_DEVERR_LEN_OOB);
                continue;
            }
            const int32_t t0 = (2 * pair + half) * p.tok, left = w.Tq - t0;
            if (left <= 0) continue;
            it.tok[0] = min(p.tok, left);
            it.tok[1] = it.alt ? 0 : min(p.tok, max(left - p.tok, 0));
            it.n0 = b * w.Tq + t0;
            it.trow = b;
            it.kmax = L;
            pos = L - w.Tq + t0;
            it.low = pos - w.window + 1;
            it.sinks = w.sinks;
            const int32_t last0 = (pos + it.tok[0] - 1) / kPfBlock;
            const int32_t last1 = (pos + it.tok[0] + it.tok[1] - 1) / kPfBlock;
            it.from = max(pos - w.window + 1, 0) / kPfBlock;
            it.first = min((w.sinks + kPfBlock - 1) / kPfBlock, it.from);
            it.count = it.first + last1 - it.from + 1;
            const int32_t c = it.count - 1;
            it.last[0] = it.alt ? c - (c & 1) : it.first + last0 - it.from;
            it.last[1] = it.alt ? c - 1 + (c & 1) : it.tok[1] > 0 ? c : -1;
            return true;
        }
        return false;
    }
    // Whether tile t has a row that sees a key of block kb.
    __device__ bool keeps(const TaItem& it, int t, int32_t kb) const {
        const int32_t first = pos + t * p.tok, k0 = kb * kPfBlock;
        return it.tok[t] > 0 && k0 < first + it.tok[t] &&
               (k0 < w.sinks || k0 + kPfBlock > first - w.window + 1);
    }
    __device__ void row(const TaItem& it, int t, int r, TaRow& out) {
        if (it.alt) t = 0;
        const int32_t tok = r / p.g, at_ = t * p.tok + tok;
        out.ok = tok < it.tok[t];
        // (rows of no query compute on what the copy brought, and see all of it)
        out.lim = out.ok ? pos + at_ + 1 : 0x7fffffff;
        out.low = out.ok ? pos + at_ - w.window + 1 : 0;
        out.sinks = w.sinks;
        row_at = (int64_t)(it.n0 + at_) * p.Hq + it.kvh * p.g + (r - tok * p.g);
    }
    __device__ void begin_row(bool, float m, float sum) {
        max_ = m;
        sum_ = sum;
        inv = sum > 0.f ? 1.f / sum : 0.f;
    }
    __device__ void write16(int c, const float (&v)[16]) const {
        if (w.out_bf16 != 0) {
            uint16_t* to = static_cast<uint16_t*>(w.out) + row_at * D + c;
#pragma unroll
            for (int e = 0; e < 16; e += 8)
                *reinterpret_cast<uint4*>(to + e) = make_uint4(
                    pack_bf16(v[e] * inv, v[e + 1] * inv), pack_bf16(v[e + 2] * inv, v[e + 3] * inv),
                    pack_bf16(v[e + 4] * inv, v[e + 5] * inv),
                    pack_bf16(v[e + 6] * inv, v[e + 7] * inv));
        } else {
            float* to = static_cast<float*>(w.out) + row_at * D + c;
#pragma unroll
            for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<float4*>(to + e) =
                    make_float4(v[e] * inv, v[e + 1] * inv, v[e + 2] * inv, v[e + 3] * inv);
        }
    }
    __device__ void finish_row() const {
        if (w.m) w.m[row_at] = max_ == kPfNegInf ? kPfNegInf : max_ * kLn2;
        if (w.e) w.e[row_at] = sum_;
    }
};

}  // namespace
}  // namespace dattn

using namespace dattn;

extern "C" dattn_status_t dattn_prefill_window(
    const dattn_kv_layout* layout, const void* k_pool, const void* v_pool, const dattn_bf16* q,
    int32_t B, int32_t Tq, int32_t Hq, float scale, const int32_t* seq_lens, int32_t window,
    int32_t sinks, void* out, int32_t out_bf16, float* m, float* e, int32_t* dev_err,
    void* stream) {
    dattn_status_t st = check_layout(layout);
    if (st != DATTN_OK) return st;
    if (layout->kv_format != DATTN_KV_BF16 && layout->kv_format != DATTN_KV_FP8_BLOCK)
        return DATTN_ERR_UNSUPPORTED;
    if ((st = check_heads(layout, B, Hq)) != DATTN_OK) return st;
    if (Tq < 0 || window < 1 || sinks < 0 || (out_bf16 & ~1)) return DATTN_ERR_INVALID_ARG;
    if (B == 0 || Tq == 0) return DATTN_OK;
    if (!k_pool || !v_pool || !q || !seq_lens || !out) return DATTN_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(q) || !aligned16(out))
        return DATTN_ERR_INVALID_ARG;
    if ((int64_t)Tq > (int64_t)layout->max_pages_per_req * layout->page_size)
        return DATTN_ERR_INVALID_ARG;
    const int32_t Hkv = layout->num_kv_heads, g = Hq / Hkv, sms = sm_count_current();
    WindowParams w{};
    w.B = B;
    w.Tq = Tq;
    w.seq_lens = seq_lens;
    // (no length reaches 2^30, so that a window or sinks beyond it see the same)
    w.window = window < (1 << 30) ? window : 1 << 30;
    w.sinks = sinks < (1 << 30) ? sinks : 1 << 30;
    w.out = out;
    w.out_bf16 = out_bf16;
    w.m = m;
    w.e = e;
    TaParams p{};
    p.num_pages = layout->num_pages;
    p.Hkv = Hkv;
    p.P = layout->page_size;
    p.max_pages = layout->max_pages_per_req;
    p.block_table = layout->block_table;
    p.Hq = Hq;
    p.g = g;
    p.tok = 128 / g;
    p.sl2 = scale * kLog2e;
    p.scale = reinterpret_cast<const float2*>(layout->kv_scale);
    p.dev_err = dev_err;
    w.pairs = (Tq + 2 * p.tok - 1) / (2 * p.tok);
    const int64_t all = (int64_t)B * Hkv * w.pairs, tokens = (int64_t)B * Tq;
    if (2 * all + sms >= (1ll << 31) || tokens >= (1ll << 31)) return DATTN_ERR_UNSUPPORTED;
    const int32_t rest = (int32_t)(all % sms);
    w.whole = (int32_t)(2 * rest <= sms ? all - rest : all);
    w.items = (int32_t)(w.whole + 2 * (all - w.whole));
    const int32_t grid = w.items < sms ? w.items : sms;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool blk = layout->kv_format == DATTN_KV_FP8_BLOCK;
    auto launch = layout->head_dim == 64
                      ? (blk ? launch_tiles<WindowJob<64>, 64, DATTN_KV_FP8_BLOCK>
                             : launch_tiles<WindowJob<64>, 64, DATTN_KV_BF16>)
                      : (blk ? launch_tiles<WindowJob<128>, 128, DATTN_KV_FP8_BLOCK>
                             : launch_tiles<WindowJob<128>, 128, DATTN_KV_BF16>);
    return launch(p, w, q, tokens, k_pool, v_pool, grid, 0u, s);
}
