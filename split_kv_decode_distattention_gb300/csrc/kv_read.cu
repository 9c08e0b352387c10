// dattn_kv_read: tokens of the paged cache read back into dense rows, bf16 or fp32, taken back from
// codes where the pool is quantized: value = code * scale, the inverse of the append's
// code = round(x / scale) ("LLM长序列服务优化：LServe的块稀疏注意力技术" §3.2.1 keeps the cache
// quantized in pages).
//
// Bound by memory: every code (and scale) is read once and every value written once. A block takes 32
// consecutive output rows: a thread per row finds the row's request, token and page once for all KV
// heads; then a warp takes 16 of the rows of one KV head at a time, 8 channels of a row to a lane,
// so that its loads (4, 8 or 16 bytes a lane) and its stores (16 or 32 bytes) are both contiguous, and
// all loads of K and V are on their way before the first conversion. Measured on a GB300: eight requests of
// 4000-12000 tokens, 8 heads of 128, block-scaled pool to bf16, 57.5 us (6.22 TB/s, 0.92 of copy bandwidth).
#include "common.cuh"
#include "internal.h"

namespace dattn {

namespace {

constexpr int kReadRows = 32;     // output rows of a block
constexpr int kReadStep = 16;     // rows of a warp's step
constexpr int kReadThreads = 256;

struct ReadParams {
    int32_t num_pages, Hkv, P, max_pages;
    const int32_t* block_table;
    const uint8_t* k_pool;
    const uint8_t* v_pool;
    const float* kv_scale;
    KvHeadFormats hf;
    int32_t B, N;
    const int32_t* out_indptr;  // [B + 1]
    const int32_t* starts;      // [B], nullable
    const int32_t* seq_lens;    // [B]
    void* k_out;                // nullable
    void* v_out;                // nullable
    int64_t k_stride, v_stride; // elements between tokens
    int32_t* dev_err;
};

// 8 channels of a stored row: bf16 values, 8-bit codes or 4-bit codes
template <int FMT>
struct Chunk {
    uint32_t w[FMT == DATTN_KV_BF16 ? 4 : FMT == DATTN_KV_INT4 ? 1 : 2];
};

// 8 bytes of codes (i4: 4 bytes) at `at`, or 16 bytes of values
template <int FMT>
__device__ __forceinline__ void load_chunk(Chunk<FMT>& c, const uint8_t* at, bool i4) {
    if constexpr (FMT == DATTN_KV_BF16) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(at));
        c.w[0] = v.x; c.w[1] = v.y; c.w[2] = v.z; c.w[3] = v.w;
    } else if constexpr (FMT == DATTN_KV_INT4) {
        c.w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
    } else if (FMT == DATTN_KV_MIXED && i4) {
        c.w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
        c.w[0] = v.x; c.w[1] = v.y;
    }
}

// The chunk's 8 values: code * scale in fp32 (rounded once; an 8-bit block's scale is a power of two)
template <int FMT>
__device__ __forceinline__ void chunk_values(const Chunk<FMT>& c, float scale, bool i4, float (&x)[8]) {
    if constexpr (FMT == DATTN_KV_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(c.w[i]);
            x[2 * i + 1] = bf16_hi(c.w[i]);
        }
    } else if (FMT == DATTN_KV_INT4 || (FMT == DATTN_KV_MIXED && i4)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = (float)((int)((c.w[0] >> (4 * i)) & 15u) - 8) * scale;
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t lo, hi;
            e4m3x4_to_f16(c.w[FMT == DATTN_KV_INT4 ? 0 : i], lo, hi);
            x[4 * i] = f16_lo(lo) * scale;
            x[4 * i + 1] = f16_hi(lo) * scale;
            x[4 * i + 2] = f16_lo(hi) * scale;
            x[4 * i + 3] = f16_hi(hi) * scale;
        }
    }
}

// By a whole warp; `some`: this lane's row is read. In fp32 two neighbouring lanes (of one row) write
// their 64 bytes in two stores of 32 bytes each, the lanes' halves exchanged, so that a store fills
// whole sectors (three requests of 4-bit and 8-bit heads: 22.9 us without).
template <int FMT, bool F32>
__device__ __forceinline__ void store_chunk(void* out, int64_t at, const Chunk<FMT>& c, float scale,
                                            bool i4, bool some) {
    if constexpr (FMT == DATTN_KV_BF16 && !F32) {  // the values as they are
        if (some)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
                make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
        return;
    }
    float x[8];
    chunk_values<FMT>(c, scale, i4, x);
    if constexpr (F32) {
        const bool odd = threadIdx.x & 1;
        float y[4];  // the other lane's: an even lane gets the first half, an odd one the second
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = __shfl_xor_sync(0xffffffffu, odd ? x[i] : x[4 + i], 1);
        if (!some) return;
        float4* to = reinterpret_cast<float4*>(static_cast<float*>(out) + at) - (odd ? 2 : 0);
        to[odd] = odd ? make_float4(y[0], y[1], y[2], y[3]) : make_float4(x[0], x[1], x[2], x[3]);
        to[2 + odd] = odd ? make_float4(x[4], x[5], x[6], x[7]) : make_float4(y[0], y[1], y[2], y[3]);
    } else if (some) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) =
            make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                       pack_bf16(x[6], x[7]));
    }
}

template <int D, int FMT, bool F32>
__global__ void __launch_bounds__(kReadThreads)
kv_read_kernel(const __grid_constant__ ReadParams p) {
    constexpr int LPR = D / 8;                         // lanes of a row
    constexpr int RPA = 32 / LPR;                      // rows of a warp's access
    constexpr int NA = kReadStep / RPA;                // accesses of a step
    // each row's page and slot in it, -1 where nothing is read
    __shared__ int32_t pages[kReadRows], slots[kReadRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int32_t row0 = blockIdx.x * kReadRows;
    grid_dependency_wait();
    grid_launch_dependents();
    if (tid < kReadRows) {
        const int32_t i = row0 + tid;
        int32_t page = -1, slot = 0;
        if (i < p.N) {
            int32_t lo = 0, hi = p.B;  // the number of requests whose rows end at or before i
            while (lo < hi) {
                const int32_t mid = (lo + hi) >> 1;
                if (__ldg(p.out_indptr + mid + 1) <= i) lo = mid + 1; else hi = mid;
            }
            const int32_t b = min(lo, p.B - 1);
            const int32_t first = __ldg(p.out_indptr + b);
            if (lo < p.B && first <= i) {
                const int64_t t = (int64_t)(p.starts ? __ldg(p.starts + b) : 0) + (i - first);
                const int64_t L = min((int64_t)__ldg(p.seq_lens + b), (int64_t)p.max_pages * p.P);
                if (first < 0 || t < i - (int64_t)first || t >= L) {
                    set_err(p.dev_err, first < 0 ? DATTN_DEVERR_CHUNK_OOB : DATTN_DEVERR_LEN_OOB);
                } else {
                    const int32_t lp = (int32_t)t / p.P;
                    slot = (int32_t)t - lp * p.P;
                    page = __ldg(p.block_table + (int64_t)b * p.max_pages + lp);
                    if (page < 0) {
                        set_err(p.dev_err, DATTN_DEVERR_UNMAPPED_PAGE);
                    } else if (page >= p.num_pages) {
                        set_err(p.dev_err, DATTN_DEVERR_PAGE_OOB);
                        page = -1;
                    }
                }
            } else if (i >= __ldg(p.out_indptr) && i < __ldg(p.out_indptr + p.B)) {
                set_err(p.dev_err, DATTN_DEVERR_CHUNK_OOB);  // the bounds do not ascend
            }
        }
        pages[tid] = page;
        slots[tid] = slot;
    }
    __syncthreads();
    const int c8 = lane % LPR, rr = lane / LPR;
    constexpr int kSteps = kReadRows / kReadStep;
    for (int32_t it = warp; it < p.Hkv * kSteps; it += kReadThreads / 32) {
        const int32_t h = it / kSteps, r0 = (it - h * kSteps) * kReadStep;
        bool i4 = FMT == DATTN_KV_INT4;
        const uint8_t *kp = p.k_pool, *vp = p.v_pool;
        int32_t heads = p.Hkv, hc = h;  // the heads of the region, and this head's place in it
        if constexpr (FMT == DATTN_KV_MIXED) {
            i4 = head_is_i4(p.hf, h);
            hc = head_class_index(p.hf, h, i4);
            heads = i4 ? p.hf.h4 : p.Hkv - p.hf.h4;
            if (i4) {
                const int64_t region8 = (int64_t)p.num_pages * (p.Hkv - p.hf.h4) * p.P * D;
                kp += region8;
                vp += region8;
            }
        }
        const int64_t row_bytes = FMT == DATTN_KV_BF16 ? 2 * D : i4 ? D / 2 : D;
        const int at_bytes = FMT == DATTN_KV_BF16 ? 16 * c8 : i4 ? 4 * c8 : 8 * c8;
        Chunk<FMT> k[NA], v[NA];
        float ks[NA], vs[NA];
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int r = r0 + a * RPA + rr;
            const int32_t page = pages[r], slot = slots[r];
            ks[a] = vs[a] = 1.f;
            k[a] = v[a] = Chunk<FMT>{};
            if (page < 0) continue;
            const int64_t at = (((int64_t)page * heads + hc) * p.P + slot) * row_bytes + at_bytes;
            if (p.k_out) load_chunk<FMT>(k[a], kp + at, i4);
            if (p.v_out) load_chunk<FMT>(v[a], vp + at, i4);
            const int64_t row = ((int64_t)page * p.Hkv + h) * p.P + slot;
            if constexpr (FMT == DATTN_KV_FP8_BLOCK) {
                const float2 s = __ldg(reinterpret_cast<const float2*>(p.kv_scale) + (row >> 4));
                ks[a] = s.x;
                vs[a] = s.y;
            } else if constexpr (FMT != DATTN_KV_BF16) {
                const float* s = p.kv_scale + (row >> 4) * 32 + (row & 15);
                ks[a] = __ldg(s);
                vs[a] = __ldg(s + 16);
            }
        }
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int r = r0 + a * RPA + rr;
            const bool some = pages[r] >= 0;
            const int64_t n = row0 + r, c = (int64_t)h * D + 8 * c8;
            if (p.k_out) store_chunk<FMT, F32>(p.k_out, n * p.k_stride + c, k[a], ks[a], i4, some);
            if (p.v_out) store_chunk<FMT, F32>(p.v_out, n * p.v_stride + c, v[a], vs[a], i4, some);
        }
    }
}

template <int FMT>
dattn_status_t launch_read(const ReadParams& p, int D, bool f32, cudaStream_t stream) {
    auto kern = D == 64 ? (f32 ? kv_read_kernel<64, FMT, true> : kv_read_kernel<64, FMT, false>)
                        : (f32 ? kv_read_kernel<128, FMT, true> : kv_read_kernel<128, FMT, false>);
    const unsigned blocks = (unsigned)(((int64_t)p.N + kReadRows - 1) / kReadRows);
    return launch_pdl(kern, dim3(blocks), dim3(kReadThreads), 0, stream, p) == cudaSuccess
               ? DATTN_OK
               : DATTN_ERR_CUDA;
}

}  // namespace
}  // namespace dattn

using namespace dattn;

extern "C" dattn_status_t dattn_kv_read(const dattn_kv_layout* layout, const void* k_pool,
                                        const void* v_pool, int32_t B, const int32_t* out_indptr,
                                        const int32_t* starts, const int32_t* seq_lens, int32_t N,
                                        void* k_out, int64_t k_stride, void* v_out,
                                        int64_t v_stride, int32_t out_f32, int32_t* dev_err,
                                        void* stream) {
    const dattn_status_t st = check_layout(layout);
    if (st != DATTN_OK) return st;
    if (B < 0 || N < 0 || (out_f32 & ~1)) return DATTN_ERR_INVALID_ARG;
    if (B > kMaxItems || N > (1 << 30)) return DATTN_ERR_UNSUPPORTED;
    if (B == 0 || N == 0) return DATTN_OK;
    if (!k_out && !v_out) return DATTN_ERR_INVALID_ARG;
    if (!k_pool || !v_pool || !out_indptr || !seq_lens) return DATTN_ERR_INVALID_ARG;
    const int64_t row = (int64_t)layout->num_kv_heads * layout->head_dim, align = out_f32 ? 4 : 8;
    if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_out) || !aligned16(v_out) ||
        (k_out && k_stride % align != 0) || (v_out && v_stride % align != 0))
        return DATTN_ERR_INVALID_ARG;
    if (N > 1 && ((k_out && k_stride < row) || (v_out && v_stride < row)))
        return DATTN_ERR_INVALID_ARG;
    ReadParams p{};
    p.num_pages = layout->num_pages;
    p.Hkv = layout->num_kv_heads;
    p.P = layout->page_size;
    p.max_pages = layout->max_pages_per_req;
    p.block_table = layout->block_table;
    p.k_pool = static_cast<const uint8_t*>(k_pool);
    p.v_pool = static_cast<const uint8_t*>(v_pool);
    p.kv_scale = layout->kv_scale;
    head_formats(*layout, p.hf);  // checked with the layout
    p.B = B;
    p.N = N;
    p.out_indptr = out_indptr;
    p.starts = starts;
    p.seq_lens = seq_lens;
    p.k_out = k_out;
    p.v_out = v_out;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.dev_err = dev_err;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int D = layout->head_dim;
    const bool f32 = out_f32 != 0;
    switch (layout->kv_format) {
        case DATTN_KV_BF16: return launch_read<DATTN_KV_BF16>(p, D, f32, s);
        case DATTN_KV_FP8_E4M3: return launch_read<DATTN_KV_FP8_E4M3>(p, D, f32, s);
        case DATTN_KV_INT4: return launch_read<DATTN_KV_INT4>(p, D, f32, s);
        case DATTN_KV_MIXED: return launch_read<DATTN_KV_MIXED>(p, D, f32, s);
        default: return launch_read<DATTN_KV_FP8_BLOCK>(p, D, f32, s);
    }
}
