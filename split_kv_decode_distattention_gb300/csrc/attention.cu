// The launches of the split-KV attention engine (attention.cuh) in its dense, block-sparse and
// partial modes: dattn_decode, dattn_decode_multi, dattn_append_decode and dattn_partial.
#include "attention.cuh"

namespace dattn {

size_t attn_workspace_bytes(int32_t nseg, int32_t g, int32_t D, int32_t G) {
    return attn_counter_bytes(nseg) + (size_t)(G + nseg) * slot_floats(g, D) * 4;
}

dattn_status_t launch_attention(const AttnParams& p, const void* k_pool, const void* v_pool,
                                int D, int32_t num_splits, void* ws, size_t ws_bytes,
                                cudaStream_t stream, int64_t tiles_bound) {
    if (D != 64 && D != 128) return DATTN_ERR_UNSUPPORTED;
    // 2 or 4 query columns over the 4-bit pool: the packed-column consumers. (The mixed pool's
    // 4-bit heads keep two products per m-tile: a packed instance of the mixed kernel slowed
    // its 8-bit tiles, 27.0 against 25.1 µs per sparse-512k launch.)
    const bool pk = p.fmt == DATTN_KV_INT4 && (p.gq == 2 || p.gq == 4);
    if (p.fmt == DATTN_KV_FP8_BLOCK) {
        if (p.append != 0) return DATTN_ERR_UNSUPPORTED;  // refused at the entry
        return D == 64 ? launch_d<64, DATTN_KV_FP8_BLOCK, false, false, false>(
                             p, k_pool, v_pool, num_splits, ws, ws_bytes, stream, tiles_bound)
                       : launch_d<128, DATTN_KV_FP8_BLOCK, false, false, false>(
                             p, k_pool, v_pool, num_splits, ws, ws_bytes, stream, tiles_bound);
    }
    auto pick = [&](auto bf16, auto f8, auto i4, auto mix, auto i4p) {
        return p.fmt == DATTN_KV_MIXED    ? mix
             : p.fmt == DATTN_KV_INT4     ? (pk ? i4p : i4)
             : p.fmt == DATTN_KV_FP8_E4M3 ? f8
                                          : bf16;
    };
#define DATTN_LAUNCHES(D_, APP_)                                                              \
    pick(launch_d<D_, DATTN_KV_BF16, APP_, false, false>,                                     \
         launch_d<D_, DATTN_KV_FP8_E4M3, APP_, false, false>,                                 \
         launch_d<D_, DATTN_KV_INT4, APP_, false, false>,                                     \
         launch_d<D_, DATTN_KV_MIXED, APP_, false, false>,                                    \
         launch_d<D_, DATTN_KV_INT4, APP_, true, false>)
    auto launch = p.append != 0 ? (D == 64 ? DATTN_LAUNCHES(64, true) : DATTN_LAUNCHES(128, true))
                                : (D == 64 ? DATTN_LAUNCHES(64, false) : DATTN_LAUNCHES(128, false));
#undef DATTN_LAUNCHES
    return launch(p, k_pool, v_pool, num_splits, ws, ws_bytes, stream, tiles_bound);
}

}  // namespace dattn
