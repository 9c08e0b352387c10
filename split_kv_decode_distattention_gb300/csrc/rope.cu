// Rotary positions (dattn_rope) and the paged append that rotates on the way
// (dattn_rope_append, and dattn_kv_append for the block-scaled pool).
//
// The rotation turns channel pair k of a row at position p by the angle p f_k:
//     y_a = A (x_a cos - x_b sin),  y_b = A (x_b cos + x_a sin),
// the pair being channels (k, k + r/2) or (2k, 2k + 1) of the first r. Its transpose (the angle
// negated) is the gradient.
//
// Angles: a frequency is kept as the fraction of a turn per position in units of 2^-64, so the
// 64-bit integer product p * f_k wraps at whole turns and its upper 32 bits are the angle to
// 2^-32 of a turn at any position, without a 64-bit floating-point operation; fp32 products lose
// 0.06 rad at position 10^6. Sine and cosine of that fraction come from sincospif.
//
// Both kernels move bytes: 2 reads and writes of 16 bytes against some 30 instructions. What
// costs beside the bytes is the sine and cosine, so a CTA computes them once for 16 tokens
// (16 x r/2 pairs into shared memory) and uses them for all its heads. A warp takes one head of
// the 16 tokens: D/16 lanes to a row, each with the two 8-channel chunks that are paired in
// the half layout (chunks l and l + r/16; the unrotated chunks come in neighbouring pairs), so
// that a lane holds both members of every pair in either layout and no value changes lanes.
// The 16-token windows of the append are logical pages (positions 16j .. 16j + 15 of the
// request), so one warp owns all that the append changes of a (logical page, KV head): its
// rows, its scales and its statistics; nothing is shared between CTAs and the results do not
// depend on any order.
//
// The block-scaled pool (DATTN_KV_FP8_BLOCK): one scale for the 16 tokens, K and V apart, the
// smallest power of two s with max |x| <= 448 s. Scaling by a power of two is exact, so a row is
// rounded once, to E4M3, and raising the scale of a page that already holds tokens re-rounds
// only the codes that become subnormal (below 2^-6).
#include "common.cuh"
#include "internal.h"

namespace dattn {

namespace {

constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = kRopeWarps * 32;
constexpr int kWin = 16;  // tokens of a CTA: a logical page

// Lane geometry of a [16 rows][D] tile: LPR lanes to a row, RPP rows in a pass, NP passes; the
// rows of a lane are consecutive (rg * NP + i), so that a logical page's statistics fold in
// token order.
template <int D>
struct Tile {
    static constexpr int LPR = D / 16, RPP = 32 / LPR, NP = kWin / RPP;
};

// cos and sin tables of 16 tokens in shared memory. A lane l of a row reads two runs of four
// pairs, at 4l and off2 + 4l: conflict-free. Half layout: its pairs 8l .. 8l + 7, stored as two
// halves; interleaved: its two chunks' pairs.
template <int D>
struct RopeTable {
    float c[kWin][D / 2], s[kWin][D / 2];
};

struct RotArgs {
    int32_t rot_dim, interleaved;
    float amplitude;
    uint64_t turns[kMaxHeadDim / 2];
};

template <int D>
__device__ __forceinline__ int32_t table_off2(const RotArgs& r) {
    return r.interleaved ? r.rot_dim / 4 : D / 4;
}

// Fills the table rows [r0, r1): row r at position pos_of(r). All threads of the CTA.
template <int D, typename F>
__device__ __forceinline__ void fill_table(RopeTable<D>& tab, const RotArgs& rot, bool inverse,
                                           int r0, int r1, F pos_of) {
    const int n = rot.rot_dim >> 1;
    for (int i = threadIdx.x; i < (r1 - r0) * n; i += kRopeThreads) {
        const int r = r0 + i / n, k = i - (i / n) * n;
        // the position times the turns per position, mod one turn: the upper 32 bits as a
        // signed fraction in [-1/2, 1/2) turn, in units of half a turn for sincospi
        const uint64_t phase = (uint64_t)(int64_t)pos_of(r) * rot.turns[k];
        const float x = (float)(int32_t)(phase >> 32) * 4.656612873077393e-10f;  // 2^-31
        float sn, cs;
        sincospif(x, &sn, &cs);
        const int at = rot.interleaved ? k : ((k >> 2) & 1) * (D / 4) + (k >> 3) * 4 + (k & 3);
        tab.c[r][at] = cs * rot.amplitude;
        tab.s[r][at] = (inverse ? -sn : sn) * rot.amplitude;
    }
}

// Rotates a lane's two chunks (8 channels each) of row r; l is the lane's place in the row.
template <int D>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const RopeTable<D>& tab, int r,
                                       int l, const RotArgs& rot) {
    if (16 * l >= rot.rot_dim) return;  // unrotated channels
    const int off2 = table_off2<D>(rot);
    const float4 c0 = *reinterpret_cast<const float4*>(&tab.c[r][4 * l]);
    const float4 c1 = *reinterpret_cast<const float4*>(&tab.c[r][off2 + 4 * l]);
    const float4 s0 = *reinterpret_cast<const float4*>(&tab.s[r][4 * l]);
    const float4 s1 = *reinterpret_cast<const float4*>(&tab.s[r][off2 + 4 * l]);
    const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    if (rot.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = a[2 * j], y = a[2 * j + 1], u = b[2 * j], v = b[2 * j + 1];
            a[2 * j] = fmaf(x, c[j], -(y * s[j]));
            a[2 * j + 1] = fmaf(y, c[j], x * s[j]);
            b[2 * j] = fmaf(u, c[4 + j], -(v * s[4 + j]));
            b[2 * j + 1] = fmaf(v, c[4 + j], u * s[4 + j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = a[j], y = b[j];
            a[j] = fmaf(x, c[j], -(y * s[j]));
            b[j] = fmaf(y, c[j], x * s[j]);
        }
    }
}

// The first channels of a lane's two chunks.
__device__ __forceinline__ void lane_chunks(int l, int32_t rot_dim, int& ca, int& cb) {
    const bool in = 16 * l < rot_dim;
    ca = in ? 8 * l : 16 * l;
    cb = in ? 8 * l + (rot_dim >> 1) : 16 * l + 8;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
}

// ------------------------------------------------------------------ dattn_rope

struct RopeParams {
    const void* x;
    void* out;
    int64_t x_stride, out_stride;  // elements between tokens
    int32_t N, H, slices, inverse;
    const int32_t* positions;
    RotArgs rot;
};

template <int D, bool F32>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    using TL = Tile<D>;
    __shared__ __align__(16) RopeTable<D> tab;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % TL::LPR, rg = lane / TL::LPR;
    const int32_t win = blockIdx.x / p.slices, slice = blockIdx.x - win * p.slices;
    const int32_t t0 = win * kWin, n = min(kWin, p.N - t0);
    int ca, cb;
    lane_chunks(l, p.rot.rot_dim, ca, cb);
    grid_dependency_wait();
    grid_launch_dependents();
    fill_table<D>(tab, p.rot, p.inverse != 0, 0, n,
                  [&](int r) { return __ldg(p.positions + t0 + r); });
    __syncthreads();
    for (int32_t h = slice * kRopeWarps + warp; h < p.H; h += p.slices * kRopeWarps) {
        if constexpr (F32) {
            const float* x = static_cast<const float*>(p.x) + (int64_t)h * D;
            float* out = static_cast<float*>(p.out) + (int64_t)h * D;
#pragma unroll
            for (int i = 0; i < TL::NP; ++i) {
                const int r = rg * TL::NP + i;
                if (r >= n) break;
                const float* row = x + (t0 + r) * p.x_stride;
                float a[8], b[8];
                *reinterpret_cast<float4*>(a) = *reinterpret_cast<const float4*>(row + ca);
                *reinterpret_cast<float4*>(a + 4) = *reinterpret_cast<const float4*>(row + ca + 4);
                *reinterpret_cast<float4*>(b) = *reinterpret_cast<const float4*>(row + cb);
                *reinterpret_cast<float4*>(b + 4) = *reinterpret_cast<const float4*>(row + cb + 4);
                rotate<D>(a, b, tab, r, l, p.rot);
                float* dst = out + (t0 + r) * p.out_stride;
                *reinterpret_cast<float4*>(dst + ca) = *reinterpret_cast<float4*>(a);
                *reinterpret_cast<float4*>(dst + ca + 4) = *reinterpret_cast<float4*>(a + 4);
                *reinterpret_cast<float4*>(dst + cb) = *reinterpret_cast<float4*>(b);
                *reinterpret_cast<float4*>(dst + cb + 4) = *reinterpret_cast<float4*>(b + 4);
            }
        } else {
            const uint16_t* x = static_cast<const uint16_t*>(p.x) + (int64_t)h * D;
            uint16_t* out = static_cast<uint16_t*>(p.out) + (int64_t)h * D;
            uint4 va[TL::NP], vb[TL::NP];
#pragma unroll
            for (int i = 0; i < TL::NP; ++i) {
                const int r = rg * TL::NP + i;
                if (r < n) {
                    const uint16_t* row = x + (t0 + r) * p.x_stride;
                    va[i] = *reinterpret_cast<const uint4*>(row + ca);
                    vb[i] = *reinterpret_cast<const uint4*>(row + cb);
                }
            }
#pragma unroll
            for (int i = 0; i < TL::NP; ++i) {
                const int r = rg * TL::NP + i;
                if (r < n) {
                    float a[8], b[8];
                    unpack8(va[i], a);
                    unpack8(vb[i], b);
                    rotate<D>(a, b, tab, r, l, p.rot);
                    uint16_t* dst = out + (t0 + r) * p.out_stride;
                    *reinterpret_cast<uint4*>(dst + ca) = pack8(a);
                    *reinterpret_cast<uint4*>(dst + cb) = pack8(b);
                }
            }
        }
    }
}

// ------------------------------------------------------------------ dattn_rope_append

struct RopeAppendParams {
    dattn_kv_layout L;
    KvHeadFormats hf;
    uint8_t* k_pool;
    uint8_t* v_pool;
    uint16_t* stats;
    const uint16_t* q;
    const uint16_t* k_new;
    const uint16_t* v_new;
    uint16_t* q_out;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    int32_t T, Hq, slices;
    int32_t* seq_lens;
    const int32_t* positions;  // nullable: seq_lens[b] + t
    const int32_t* new_lens;   // nullable: T
    int32_t advance;           // 1: this launch advances seq_lens (one cluster per request)
    int32_t* dev_err;
    RotArgs rot;
};

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// New tokens of request b: new_lens[b] inside [0, T]; another value is flagged and clamped.
__device__ __forceinline__ int32_t new_count(const int32_t* new_lens, int32_t b, int32_t T,
                                             int32_t* dev_err) {
    if (new_lens == nullptr) return T;
    const int32_t n = new_lens[b];
    if (n < 0 || n > T) set_err(dev_err, DATTN_DEVERR_LEN_OOB);
    return min(max(n, 0), T);
}

// The smallest power of two s with m <= 448 s (448 = 1.75 * 2^8), clamped to [2^-126, 2^119];
// 0 for m = 0. Beyond the upper clamp (m > 448 * 2^119, infinity) the codes saturate.
__device__ __forceinline__ float block_scale(float m) {
    const int32_t bits = __float_as_int(m);
    const int32_t k = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
    return m > 0.f ? __int_as_float((min(119, max(-126, k)) + 127) << 23) : 0.f;
}

// 2^-k of a scale 2^k in [2^-126, 2^119] (0 for 0, which makes every code +0 or -0).
__device__ __forceinline__ float pow2_inverse(float s) {
    return s > 0.f ? __int_as_float((254 << 23) - __float_as_int(s)) : 0.f;
}

// E4M3 codes of 8 bf16 values times f (a power of two: exact), rounded to nearest even.
__device__ __forceinline__ uint2 codes8(const uint4& v, float f) {
    float x[8];
    unpack8(v, x);
    return make_uint2(f32x4_to_e4m3(x[0] * f, x[1] * f, x[2] * f, x[3] * f),
                      f32x4_to_e4m3(x[4] * f, x[5] * f, x[6] * f, x[7] * f));
}

// Four E4M3 codes times f (a power of two), rounded again.
__device__ __forceinline__ uint32_t recode4(uint32_t c, float f) {
    uint32_t lo, hi;
    e4m3x4_to_f16(c, lo, hi);
    return f32x4_to_e4m3(f16_lo(lo) * f, f16_hi(lo) * f, f16_lo(hi) * f, f16_hi(hi) * f);
}

// Writes a warp's rows of K or V (chunks va, vb of the rows in [r0, r1)) to the slots of the
// logical page at pool row `row0` (over all heads), in the pool's format. `crow0` is the codes'
// row and `pool` the codes' region (they differ in a mixed pool), `kv` 0 for K and 1 for V.
template <int D, int FMT>
__device__ __forceinline__ void write_rows(const RopeAppendParams& p, uint8_t* pool, int64_t row0,
                                           int64_t crow0, int kv, bool i4, const uint4* va,
                                           const uint4* vb, int r0, int r1, bool extends, int l,
                                           int rg, int ca, int cb) {
    using TL = Tile<D>;
    if constexpr (FMT == DATTN_KV_FP8_BLOCK) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < TL::NP; ++i) {
            const int r = rg * TL::NP + i;
            if (r >= r0 && r < r1) m = fmaxf(m, fmaxf(absmax8(va[i]), absmax8(vb[i])));
        }
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
        float* sc = p.L.kv_scale + (row0 >> 4) * 2 + kv;
        const float was = extends ? *sc : 0.f;
        const float s = fmaxf(was, block_scale(m)), inv = pow2_inverse(s);
        if (s > was && was > 0.f) {  // earlier rows of the page move to the larger scale
            const float f = was * inv;
#pragma unroll
            for (int i = 0; i < TL::NP; ++i) {
                const int r = rg * TL::NP + i;
                if (r < r0) {
                    uint2* a = reinterpret_cast<uint2*>(pool + (crow0 + r) * D + ca);
                    uint2* b = reinterpret_cast<uint2*>(pool + (crow0 + r) * D + cb);
                    const uint2 x = *a, y = *b;
                    *a = make_uint2(recode4(x.x, f), recode4(x.y, f));
                    *b = make_uint2(recode4(y.x, f), recode4(y.y, f));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < TL::NP; ++i) {
            const int r = rg * TL::NP + i;
            if (r >= r0 && r < r1) {
                *reinterpret_cast<uint2*>(pool + (crow0 + r) * D + ca) = codes8(va[i], inv);
                *reinterpret_cast<uint2*>(pool + (crow0 + r) * D + cb) = codes8(vb[i], inv);
            }
        }
        __syncwarp();  // every lane has read the old scale
        if (l == 0 && rg == 0) *sc = s;
    } else {
#pragma unroll
        for (int i = 0; i < TL::NP; ++i) {
            const int r = rg * TL::NP + i;
            const bool in = r >= r0 && r < r1;
            if constexpr (FMT == DATTN_KV_BF16) {
                if (in) {
                    uint16_t* dst = reinterpret_cast<uint16_t*>(pool) + (crow0 + r) * D;
                    *reinterpret_cast<uint4*>(dst + ca) = va[i];
                    *reinterpret_cast<uint4*>(dst + cb) = vb[i];
                }
            } else {  // a scale per row, over the row's LPR lanes
                float m = in ? fmaxf(absmax8(va[i]), absmax8(vb[i])) : 0.f;
#pragma unroll
                for (int off = 1; off < TL::LPR; off <<= 1)
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                if (in) {
                    float s;
                    if (i4) {
                        uint8_t* dst = pool + (crow0 + r) * (D / 2);
                        *reinterpret_cast<uint32_t*>(dst + ca / 2) = quant4_chunk(va[i], m, s);
                        *reinterpret_cast<uint32_t*>(dst + cb / 2) = quant4_chunk(vb[i], m, s);
                    } else {
                        uint8_t* dst = pool + (crow0 + r) * D;
                        *reinterpret_cast<uint2*>(dst + ca) = quant8_chunk(va[i], m, s);
                        *reinterpret_cast<uint2*>(dst + cb) = quant8_chunk(vb[i], m, s);
                    }
                    if (l == 0) p.L.kv_scale[(row0 >> 4) * 32 + 16 * kv + r] = s;
                }
            }
        }
    }
}

// Folds the keys of rows [r0, r1) into the logical page's k_max / k_min, in token order: a lane
// group folds its consecutive rows, then the groups are folded in order (on a tie the earlier
// value stays; the first row of a page that this call opens is taken as it is).
template <int D>
__device__ __forceinline__ void fold_stats(uint16_t* st, const uint4* v, int r0, int r1, int rg,
                                           int c) {
    using TL = Tile<D>;
    uint4 mx = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);  // -inf
    uint4 mn = make_uint4(0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u);
    if (rg == 0) {
        if (r0 == 0) {
            mx = mn = v[0];
        } else {
            mx = *reinterpret_cast<const uint4*>(st + c);
            mn = *reinterpret_cast<const uint4*>(st + D + c);
        }
    }
#pragma unroll
    for (int i = 0; i < TL::NP; ++i) {
        const int r = rg * TL::NP + i;
        if (r >= r0 && r < r1) bf16_fold8(v[i], mx, mn);
    }
#pragma unroll
    for (int off = TL::LPR; off < 32; off <<= 1) {
        const bool up = (rg * TL::LPR) & off;  // this group comes after its partner
        uint4 ox, on;
        ox.x = __shfl_xor_sync(0xffffffffu, mx.x, off);
        ox.y = __shfl_xor_sync(0xffffffffu, mx.y, off);
        ox.z = __shfl_xor_sync(0xffffffffu, mx.z, off);
        ox.w = __shfl_xor_sync(0xffffffffu, mx.w, off);
        on.x = __shfl_xor_sync(0xffffffffu, mn.x, off);
        on.y = __shfl_xor_sync(0xffffffffu, mn.y, off);
        on.z = __shfl_xor_sync(0xffffffffu, mn.z, off);
        on.w = __shfl_xor_sync(0xffffffffu, mn.w, off);
        uint4 fx = up ? ox : mx, fn = up ? on : mn;  // the earlier group's, then the later's
        const uint4 lx = up ? mx : ox, ln = up ? mn : on;
        uint4 unused_x = fx, unused_n = fn;
        bf16_fold8(lx, fx, unused_n);
        bf16_fold8(ln, unused_x, fn);
        mx = fx;
        mn = fn;
    }
    if (rg == 0) {
        *reinterpret_cast<uint4*>(st + c) = mx;
        *reinterpret_cast<uint4*>(st + D + c) = mn;
    }
}

// Grid: (windows * slices, B). CTA (window, slice) of request b takes the new tokens of the
// window'th logical page from the one that holds position seq_lens[b], for every slices'th
// group of eight heads: the KV heads (K and V together), then the query heads.
template <int D, int FMT>
__global__ void __launch_bounds__(kRopeThreads)
rope_append_kernel(const __grid_constant__ RopeAppendParams p) {
    using TL = Tile<D>;
    __shared__ __align__(16) RopeTable<D> tab;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane % TL::LPR, rg = lane / TL::LPR;
    const int32_t b = blockIdx.y;
    const int32_t win = blockIdx.x / p.slices, slice = blockIdx.x - win * p.slices;
    const int32_t Hkv = p.L.num_kv_heads, P = p.L.page_size;
    int ca, cb;
    lane_chunks(l, p.rot.rot_dim, ca, cb);
    grid_dependency_wait();  // the previous kernel may still read the pool or write the rows
    grid_launch_dependents();
    const int32_t pos0 = p.seq_lens[b];
    const int32_t n = new_count(p.new_lens, b, p.T, blockIdx.x == 0 && threadIdx.x == 0
                                                        ? p.dev_err : nullptr);
    if (p.advance) {
        __syncwarp();
        cluster_arrive();  // this thread has read the length
    }
    // positions stay below 2^31: a layout holds fewer than 2^30 tokens, a call brings fewer than 2^28
    const bool bad = pos0 < 0 || pos0 >= (1 << 30);
    const int32_t base = ((bad ? 0 : pos0) & ~15) + win * kWin;  // the window's first position
    const int r0 = max(pos0 - base, 0), r1 = min(kWin, pos0 + n - base);
    if (bad) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_err(p.dev_err, DATTN_DEVERR_LEN_OOB);
    } else if (r0 < r1) {
        const int64_t tok0 = (int64_t)b * p.T + (base - pos0);  // the new-token row of row 0
        fill_table<D>(tab, p.rot, false, r0, r1, [&](int r) {
            return p.positions ? __ldg(p.positions + tok0 + r) : base + r;
        });
        // the logical page's place in the pool
        int32_t page = -1;
        const int32_t lp = base / P;
        if (lp >= p.L.max_pages_per_req) {
            if (threadIdx.x == 0) set_err(p.dev_err, DATTN_DEVERR_LEN_OOB);
        } else {
            const int32_t pg = __ldg(p.L.block_table + (int64_t)b * p.L.max_pages_per_req + lp);
            if (pg < 0) set_err(threadIdx.x == 0 ? p.dev_err : nullptr, DATTN_DEVERR_UNMAPPED_PAGE);
            else if (pg >= p.L.num_pages)
                set_err(threadIdx.x == 0 ? p.dev_err : nullptr, DATTN_DEVERR_PAGE_OOB);
            else page = pg;
        }
        const int32_t slot0 = base - lp * P;
        __syncthreads();
        const int32_t units = Hkv + p.Hq;
        for (int32_t u = slice * kRopeWarps + warp; u < units; u += p.slices * kRopeWarps) {
            const bool isq = u >= Hkv;
            if (!isq && page < 0) continue;
            const int32_t h = isq ? u - Hkv : u;
            uint4 va[TL::NP], vb[TL::NP];
            auto load = [&](const uint16_t* x, int64_t stride) {
#pragma unroll
                for (int i = 0; i < TL::NP; ++i) {
                    const int r = rg * TL::NP + i;
                    va[i] = vb[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (r >= r0 && r < r1) {
                        const uint16_t* row = x + (tok0 + r) * stride + (int64_t)h * D;
                        va[i] = *reinterpret_cast<const uint4*>(row + ca);
                        vb[i] = *reinterpret_cast<const uint4*>(row + cb);
                    }
                }
            };
            load(isq ? p.q : p.k_new, isq ? p.q_stride : p.k_stride);
#pragma unroll
            for (int i = 0; i < TL::NP; ++i) {
                const int r = rg * TL::NP + i;
                if (r >= r0 && r < r1) {
                    float a[8], c[8];
                    unpack8(va[i], a);
                    unpack8(vb[i], c);
                    rotate<D>(a, c, tab, r, l, p.rot);
                    va[i] = pack8(a);
                    vb[i] = pack8(c);
                    if (isq) {
                        uint16_t* dst = p.q_out + ((tok0 + r) * p.Hq + h) * D;
                        *reinterpret_cast<uint4*>(dst + ca) = va[i];
                        *reinterpret_cast<uint4*>(dst + cb) = vb[i];
                    }
                }
            }
            if (isq) continue;
            const int64_t row0 = ((int64_t)page * Hkv + h) * P + slot0;
            int64_t crow0 = row0;
            uint8_t *kd = p.k_pool, *vd = p.v_pool;
            bool i4 = FMT == DATTN_KV_INT4;
            if constexpr (FMT == DATTN_KV_MIXED) {  // each format in its own region
                i4 = head_is_i4(p.hf, h);
                const int32_t h4 = p.hf.h4, h8 = Hkv - h4;
                crow0 = ((int64_t)page * (i4 ? h4 : h8) + head_class_index(p.hf, h, i4)) * P + slot0;
                if (i4) {
                    const int64_t region8 = (int64_t)p.L.num_pages * h8 * P * D;
                    kd += region8;
                    vd += region8;
                }
            }
            const bool extends = r0 > 0;  // the page already holds tokens of this request
            write_rows<D, FMT>(p, kd, row0, crow0, 0, i4, va, vb, r0, r1, extends, l, rg, ca, cb);
            if (p.stats != nullptr) {
                uint16_t* st = p.stats + (row0 >> 4) * 2 * D;
                fold_stats<D>(st, va, r0, r1, rg, ca);
                fold_stats<D>(st, vb, r0, r1, rg, cb);
            }
            load(p.v_new, p.v_stride);
            write_rows<D, FMT>(p, vd, row0, crow0, 1, i4, va, vb, r0, r1, extends, l, rg, ca, cb);
        }
    }
    if (p.advance) {
        __syncwarp();
        cluster_wait();  // every thread of the request's CTAs has read the length
        if (blockIdx.x == 0 && threadIdx.x == 0 && !bad) p.seq_lens[b] = pos0 + n;
    }
}

__global__ void rope_advance_kernel(int32_t* seq_lens, const int32_t* new_lens, int32_t B,
                                    int32_t T) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t b = blockIdx.x * blockDim.x + threadIdx.x;
    if (b < B && seq_lens[b] >= 0 && seq_lens[b] < (1 << 30)) seq_lens[b] += new_count(new_lens, b, T, nullptr);
}

RotArgs rot_args(const dattn_rotation* rot) {
    RotArgs r{};
    r.amplitude = 1.f;
    if (rot == nullptr) return r;
    r.rot_dim = rot->rot_dim;
    r.interleaved = rot->interleaved;
    r.amplitude = rot->amplitude;
    for (int i = 0; i < rot->rot_dim / 2; ++i) r.turns[i] = rot->turns[i];
    return r;
}

// CTAs that share the heads of a window: about two CTAs per SM in all, at least one head each.
int32_t head_slices(int64_t windows, int32_t heads) {
    const int64_t want = (2 * (int64_t)sm_count_current() + windows - 1) / windows;
    const int64_t most = (heads + kRopeWarps - 1) / kRopeWarps;
    return (int32_t)(want < 1 ? 1 : want > most ? most : want);
}

}  // namespace

dattn_status_t launch_rope(const dattn_rotation* rot, const void* x, int64_t x_stride, void* out,
                           int64_t out_stride, int32_t N, int32_t H, int32_t D, bool f32,
                           const int32_t* positions, bool inverse, cudaStream_t stream) {
    RopeParams p{x, out, x_stride, out_stride, N, H, 1, inverse ? 1 : 0, positions, rot_args(rot)};
    const int64_t windows = ((int64_t)N + kWin - 1) / kWin;
    p.slices = head_slices(windows, H);
    if (windows * p.slices >= (1ll << 31)) return DATTN_ERR_UNSUPPORTED;
    auto kern = D == 64 ? (f32 ? rope_kernel<64, true> : rope_kernel<64, false>)
                        : (f32 ? rope_kernel<128, true> : rope_kernel<128, false>);
    return launch_pdl(kern, dim3((unsigned)(windows * p.slices)), dim3(kRopeThreads), 0, stream,
                      p) == cudaSuccess
               ? DATTN_OK
               : DATTN_ERR_CUDA;
}

dattn_status_t launch_rope_append(const dattn_kv_layout& L, void* k_pool, void* v_pool,
                                  uint16_t* stats, const dattn_rotation* rot, const uint16_t* q,
                                  int64_t q_stride, const uint16_t* k_new, int64_t k_stride,
                                  const uint16_t* v_new, int64_t v_stride, int32_t B, int32_t T,
                                  int32_t Hq, uint16_t* q_out, int32_t* seq_lens,
                                  const int32_t* positions, const int32_t* new_lens, bool advance,
                                  int32_t* dev_err, cudaStream_t stream) {
    RopeAppendParams p{};
    p.L = L;
    p.L.head_format = nullptr;  // a host array: the kernel reads hf
    if (head_formats(L, p.hf) != DATTN_OK) return DATTN_ERR_INVALID_ARG;
    p.k_pool = static_cast<uint8_t*>(k_pool);
    p.v_pool = static_cast<uint8_t*>(v_pool);
    p.stats = stats;
    p.q = q;
    p.k_new = k_new;
    p.v_new = v_new;
    p.q_out = q_out;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.T = T;
    p.Hq = Hq;
    p.seq_lens = seq_lens;
    p.positions = positions;
    p.new_lens = new_lens;
    p.dev_err = dev_err;
    p.rot = rot_args(rot);
    // T tokens from any position touch at most this many logical pages
    const int64_t windows = T == 1 ? 1 : ((int64_t)T + 30) / kWin;
    int32_t slices = head_slices(windows * B, L.num_kv_heads + Hq);
    // A request's CTAs that fit one cluster (8) advance its length themselves, behind a cluster
    // barrier; beyond that a second small kernel does.
    const bool inside = advance && windows <= 8;
    if (inside && windows * slices > 8) slices = (int32_t)(8 / windows);
    p.slices = slices;
    p.advance = inside ? 1 : 0;
    if (windows * slices >= (1ll << 31)) return DATTN_ERR_UNSUPPORTED;
    auto pick = [&](auto bf16, auto f8, auto i4, auto mix, auto blk) {
        return L.kv_format == DATTN_KV_MIXED     ? mix
             : L.kv_format == DATTN_KV_INT4      ? i4
             : L.kv_format == DATTN_KV_FP8_E4M3  ? f8
             : L.kv_format == DATTN_KV_FP8_BLOCK ? blk
                                                 : bf16;
    };
#define DATTN_ROPE_KERNELS(D_)                                                              \
    pick(rope_append_kernel<D_, DATTN_KV_BF16>, rope_append_kernel<D_, DATTN_KV_FP8_E4M3>,  \
         rope_append_kernel<D_, DATTN_KV_INT4>, rope_append_kernel<D_, DATTN_KV_MIXED>,     \
         rope_append_kernel<D_, DATTN_KV_FP8_BLOCK>)
    auto kern = L.head_dim == 64 ? DATTN_ROPE_KERNELS(64) : DATTN_ROPE_KERNELS(128);
#undef DATTN_ROPE_KERNELS
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(windows * slices), (unsigned)B);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)(windows * slices), 1u, 1u};
    cfg.attrs = attr;
    cfg.numAttrs = inside ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return DATTN_ERR_CUDA;
    if (advance && !inside &&
        launch_pdl(rope_advance_kernel, dim3((B + 255) / 256), dim3(256), 0, stream, seq_lens,
                   new_lens, B, T) != cudaSuccess)
        return DATTN_ERR_CUDA;
    return DATTN_OK;
}

}  // namespace dattn
