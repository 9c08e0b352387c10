// dattn_decode_window: a step of T query tokens per request through a sliding window with first
// tokens that stay visible, in the windowed mode of the split-KV attention engine (attention.cuh).
//
// Query token t of request b, at position p = L_b - T + t, sees the keys i <= p with i < sinks or
// i > p - window. A request's tokens are read once for all its query tokens and the query heads of
// a KV head: the tiles of the sinks, then those from the first key of token 0's window on; a tile
// at a window's edge is masked row by row for each query token.
//
// What bounds it: the memory, and for small batches the latency of one wave of tiles and its merge. Measured on a
// GB300: 64 requests of 2 tokens through a window of 4096, 32 / 8 heads of 128, 8-bit pool, 82 us (5.58 TB/s,
// 0.82 of copy bandwidth); 2 requests of 4 tokens through 512, 16 / 8 heads, bf16, 12.3 us.
#include "attention.cuh"

namespace dattn {

dattn_status_t launch_attention_window(const AttnParams& p, const void* k_pool, const void* v_pool,
                                       int D, int32_t num_splits, void* ws, size_t ws_bytes,
                                       cudaStream_t stream, int64_t tiles_bound) {
    const bool pk = p.gq == 2 || p.gq == 4;  // as in launch_attention
#define DATTN_LAUNCH(FMT_, PK_)                                                           \
    (D == 64 ? launch_d<64, FMT_, false, PK_, true> : launch_d<128, FMT_, false, PK_, true>)
    auto launch = p.fmt == DATTN_KV_FP8_BLOCK  ? DATTN_LAUNCH(DATTN_KV_FP8_BLOCK, false)
                  : p.fmt == DATTN_KV_MIXED    ? DATTN_LAUNCH(DATTN_KV_MIXED, false)
                  : p.fmt == DATTN_KV_FP8_E4M3 ? DATTN_LAUNCH(DATTN_KV_FP8_E4M3, false)
                  : p.fmt == DATTN_KV_BF16     ? DATTN_LAUNCH(DATTN_KV_BF16, false)
                  : pk                         ? DATTN_LAUNCH(DATTN_KV_INT4, true)
                                               : DATTN_LAUNCH(DATTN_KV_INT4, false);
#undef DATTN_LAUNCH
    return launch(p, k_pool, v_pool, num_splits, ws, ws_bytes, stream, tiles_bound);
}

}  // namespace dattn

using namespace dattn;

extern "C" dattn_status_t dattn_decode_window(
    const dattn_kv_layout* layout, const void* k_pool, const void* v_pool, const dattn_bf16* q,
    int32_t B, int32_t T, int32_t Hq, float scale, const int32_t* seq_lens, int32_t window,
    int32_t sinks, int32_t num_splits, void* ws, size_t ws_bytes, void* out, int32_t out_bf16,
    float* m_g, float* e_g, int32_t* dev_err, void* stream) {
    dattn_status_t st = check_layout(layout);
    if (st != DATTN_OK) return st;
    if ((st = check_heads(layout, B, Hq)) != DATTN_OK) return st;
    if (num_splits < 0 || T < 1 || window < 1 || sinks < 0 || (out_bf16 & ~1))
        return DATTN_ERR_INVALID_ARG;
    const int32_t g = Hq / layout->num_kv_heads;
    if (g * (int64_t)T > kMaxGroup) return DATTN_ERR_UNSUPPORTED;
    if (B == 0) return DATTN_OK;
    if (!k_pool || !v_pool || !q || !seq_lens || !out) return DATTN_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(q) || !aligned16(out))
        return DATTN_ERR_INVALID_ARG;
    // (no length reaches 2^30, so that a window or sinks beyond it see the same)
    window = window < (1 << 30) ? window : 1 << 30;
    sinks = sinks < (1 << 30) ? sinks : 1 << 30;
    const int64_t all = (int64_t)layout->max_pages_per_req * (layout->page_size / 16);
    int64_t per_head = (sinks + 15ll) / 16 + (window + T + 29ll) / 16;
    if (per_head > all + 1) per_head = all + 1;  // (the tile where the sinks end may come twice)
    const int64_t bound =
        (int64_t)B * layout->num_kv_heads * (per_head + seg_cost(layout->kv_format, g * T));
    if (bound >= (1ll << 31)) return DATTN_ERR_UNSUPPORTED;
    AttnParams p{};
    p.mode = MODE_WINDOW;
    p.num_pages = layout->num_pages;
    p.Hkv = layout->num_kv_heads;
    p.P = layout->page_size;
    p.max_pages = layout->max_pages_per_req;
    p.block_table = layout->block_table;
    p.q = q;
    p.B = B;
    p.Hq = Hq;
    p.g = g;
    p.T = T;
    p.gq = g * T;
    p.sl2 = scale * kLog2e;
    p.seq_lens = seq_lens;
    p.window = window;
    p.sinks = sinks;
    p.normalise = 1;
    p.out = static_cast<float*>(out);
    p.out_bf16 = out_bf16;
    p.m_out = m_g;
    p.e_out = e_g;
    p.nseg = B * p.Hkv;
    p.nitems = B;
    p.dev_err = dev_err;
    p.fmt = layout->kv_format;
    p.kv_scale = layout->kv_scale;
    head_formats(*layout, p.hf);  // checked with the layout
    return launch_attention_window(p, k_pool, v_pool, layout->head_dim, num_splits, ws, ws_bytes,
                                   static_cast<cudaStream_t>(stream), bound);
}
