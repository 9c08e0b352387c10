// Rotary positions (dattn_rope) and the paged append that rotates on the way
// (dattn_rope_append, and dattn_kv_append for the block-scaled pool).
//
// The rotation turns channel pair k of a row at position p by the angle p f_k:
//     y_a = A (x_a cos - x_b sin),  y_b = A (x_b cos + x_a sin),
// the pair being channels (k, k + r/2) or (2k, 2k + 1) of the first r. Its transpose (the angle
// negated) is the gradient.
//
// Angles: a frequency is kept as the fraction of a turn per position in units of 2^-64 (rounded to
// nearest), so the 64-bit integer product p * f_k wraps at whole turns, is within 2^-34 of a turn at
// any int32 position, and its upper 32 bits are the angle to 2^-32 of a turn, without a 64-bit
// floating-point operation; fp32 products lose 0.06 rad at position 10^6. Sine and cosine of that
// fraction: sincos_turn.
//
// The kernels are bound by the bytes they move for long inputs (dattn_rope of 16384 tokens of 32
// heads of 128 out of a fused projection: 41 us, 0.96 of the copy bandwidth) and by latency for
// short ones. What costs beside the bytes is the sine and cosine, so a CTA computes them once for
// 16 tokens (16 x r/2 pairs into shared memory) and uses them for all its heads. A warp takes one head of
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
template <int D, int ROWS = kWin>
struct RopeTable {
    float c[ROWS][D / 2], s[ROWS][D / 2];
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

// sin and cos of `phase` / 2^32 of a turn. The nearest quarter turn is taken off in integers; the
// rest, at most pi/4, goes into Taylor polynomials of degree 9 and 8 (their first omitted terms,
// t^11 / 11! and t^10 / 10!, are below 2e-9 and 3e-8).
__device__ __forceinline__ void sincos_turn(uint32_t phase, float& sn, float& cs) {
    const uint32_t quarter = (phase + 0x20000000u) >> 30;
    const float t = (float)(int32_t)(phase - (quarter << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
    const float z = t * t;
    float a = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
    a = fmaf(z, a, 8.3333333e-3f);
    a = fmaf(z, a, -1.6666667e-1f);
    a = fmaf(t * z, a, t);
    float b = fmaf(z, 2.4801587e-5f, -1.3888889e-3f);
    b = fmaf(z, b, 4.1666667e-2f);
    b = fmaf(z, b, -0.5f);
    b = fmaf(z, b, 1.f);
    const bool odd = quarter & 1u;
    sn = odd ? b : a;
    cs = odd ? a : b;
    // quarters 2, 3 negate the sine, 1, 2 the cosine
    sn = __uint_as_float(__float_as_uint(sn) ^ ((quarter & 2u) << 30));
    cs = __uint_as_float(__float_as_uint(cs) ^ (((quarter + 1u) & 2u) << 30));
}

// Fills the table rows [r0, r1): row r at position pos_of(r). All threads of the CTA; a thread
// keeps one frequency (an indexed kernel parameter costs a cycle per lane) and takes every
// kRopeThreads / n'th row.
template <int D, int ROWS, typename F>
__device__ __forceinline__ void fill_table(RopeTable<D, ROWS>& tab, const RotArgs& rot, bool inverse,
                                           int r0, int r1, F pos_of) {
    const int n = rot.rot_dim >> 1;
    if (n == 0) return;
    const int first = threadIdx.x / n, k = threadIdx.x - first * n, step = kRopeThreads / n;
    if (first >= step || r0 + first >= r1) return;
    const uint64_t turns = rot.turns[k];
    const int at = rot.interleaved ? k : ((k >> 2) & 1) * (D / 4) + (k >> 3) * 4 + (k & 3);
    const float amp_s = inverse ? -rot.amplitude : rot.amplitude;
    for (int r = r0 + first; r < r1; r += step) {
        // the position times the turns per position, mod one turn: the upper 32 bits
        float sn, cs;
        sincos_turn((uint32_t)(((uint64_t)(int64_t)pos_of(r) * turns) >> 32), sn, cs);
        tab.c[r][at] = cs * rot.amplitude;
        tab.s[r][at] = sn * amp_s;
    }
}

// Rotates a lane's two chunks (8 channels each) of row r; l is the lane's place in the row. (Packed
// fp32 pairs need fewer operations but more moves between registers: 35.3 us for 33.7 in an append
// of 2 x 4093 tokens.)
template <int D, int ROWS>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const RopeTable<D, ROWS>& tab,
                                       int r, int l, const RotArgs& rot) {
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
__device__ __forceinline__ void unpack8f(const uint4 (&v)[2], float (&x)[8]) {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
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

// A lane's rows of one head: loaded together, so that NP * 2 (fp32: NP * 4) 16-byte loads are in
// flight.
template <int D, bool F32>
struct RopeRows {
    static constexpr int W = F32 ? 2 : 1;  // 16-byte words of 8 channels
    uint4 a[Tile<D>::NP][W], b[Tile<D>::NP][W];

    __device__ __forceinline__ void load(const RopeParams& p, int32_t t0, int32_t n, int32_t h,
                                         int rg, int ca, int cb) {
        constexpr int E = F32 ? 4 : 2;
        const uint8_t* x = static_cast<const uint8_t*>(p.x) + (int64_t)h * D * E;
#pragma unroll
        for (int i = 0; i < Tile<D>::NP; ++i) {
            const int r = rg * Tile<D>::NP + i;
            if (r < n) {
                const uint8_t* row = x + (t0 + r) * p.x_stride * E;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    a[i][w] = *reinterpret_cast<const uint4*>(row + ca * E + 16 * w);
                    b[i][w] = *reinterpret_cast<const uint4*>(row + cb * E + 16 * w);
                }
            }
        }
    }
    __device__ __forceinline__ void turn_and_store(const RopeParams& p, const RopeTable<D>& tab,
                                                   int32_t t0, int32_t n, int32_t h, int l, int rg,
                                                   int ca, int cb) {
        constexpr int E = F32 ? 4 : 2;
        uint8_t* out = static_cast<uint8_t*>(p.out) + (int64_t)h * D * E;
#pragma unroll
        for (int i = 0; i < Tile<D>::NP; ++i) {
            const int r = rg * Tile<D>::NP + i;
            if (r < n) {
                float x[8], y[8];
                if constexpr (F32) {
                    unpack8f(a[i], x);
                    unpack8f(b[i], y);
                } else {
                    unpack8(a[i][0], x);
                    unpack8(b[i][0], y);
                }
                rotate(x, y, tab, r, l, p.rot);
                uint8_t* dst = out + (t0 + r) * p.out_stride * E;
                if constexpr (F32) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        *reinterpret_cast<float4*>(dst + ca * E + 16 * w) =
                            make_float4(x[4 * w], x[4 * w + 1], x[4 * w + 2], x[4 * w + 3]);
                        *reinterpret_cast<float4*>(dst + cb * E + 16 * w) =
                            make_float4(y[4 * w], y[4 * w + 1], y[4 * w + 2], y[4 * w + 3]);
                    }
                } else {
                    *reinterpret_cast<uint4*>(dst + ca * E) = pack8(x);
                    *reinterpret_cast<uint4*>(dst + cb * E) = pack8(y);
                }
            }
        }
    }
};

template <int D, bool F32>
__global__ void __launch_bounds__(kRopeThreads, F32 ? 2 : 3)
rope_kernel(const __grid_constant__ RopeParams p) {
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
    // the first head's rows are on their way while the table is made
    RopeRows<D, F32> rows;
    int32_t h = slice * kRopeWarps + warp;
    if (h < p.H) rows.load(p, t0, n, h, rg, ca, cb);
    fill_table<D>(tab, p.rot, p.inverse != 0, 0, n,
                  [&](int r) { return __ldg(p.positions + t0 + r); });
    __syncthreads();
    while (h < p.H) {
        rows.turn_and_store(p, tab, t0, n, h, l, rg, ca, cb);
        h += p.slices * kRopeWarps;
        if (h < p.H) rows.load(p, t0, n, h, rg, ca, cb);
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

// Folds |x| of 8 bf16 values into a running pair of maxima (NaN is passed over, as by fmaxf).
__device__ __forceinline__ void fold_abs(const uint4& v, __nv_bfloat162& m) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t a = w[i] & 0x7fff7fffu;
        m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&a));
    }
}

// E4M3 codes of 8 bf16 values times f, rounded to nearest even. The product with a power of two
// is exact in bf16 for every result that is not far below E4M3's smallest, 2^-9.
__device__ __forceinline__ uint2 codes8(const uint4& v, __nv_bfloat162 f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), f);
        const uint32_t z = *reinterpret_cast<const uint32_t*>(&y);
        x[2 * i] = bf16_lo(z);
        x[2 * i + 1] = bf16_hi(z);
    }
    return make_uint2(f32x4_to_e4m3(x[0], x[1], x[2], x[3]), f32x4_to_e4m3(x[4], x[5], x[6], x[7]));
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
        float* sc = p.L.kv_scale + (row0 >> 4) * 2 + kv;
        const float was = extends ? *sc : 0.f;
        __nv_bfloat162 m2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < TL::NP; ++i) {  // (rows outside [r0, r1) were loaded as zeros)
            fold_abs(va[i], m2);
            fold_abs(vb[i], m2);
        }
        // magnitudes order as their bits do
        const float m = __uint_as_float(__reduce_max_sync(
            0xffffffffu, __float_as_uint(fmaxf(__low2float(m2), __high2float(m2)))));
        const float s = fmaxf(was, block_scale(m)), inv = pow2_inverse(s);
        const __nv_bfloat162 inv2 = __float2bfloat162_rn(inv);  // a power of two: exact
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
                *reinterpret_cast<uint2*>(pool + (crow0 + r) * D + ca) = codes8(va[i], inv2);
                *reinterpret_cast<uint2*>(pool + (crow0 + r) * D + cb) = codes8(vb[i], inv2);
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

// Folds the keys of rows [r0, r1) (chunks va, vb) into the logical page's k_max / k_min, in token
// order: a lane group folds its consecutive rows, then the groups are folded in order (on a tie
// the earlier value stays; the first row of a page that this call opens is taken as it is).
template <int D>
__device__ __forceinline__ void fold_stats(uint16_t* st, const uint4* va, const uint4* vb, int r0,
                                           int r1, int rg, int ca, int cb) {
    using TL = Tile<D>;
    constexpr uint32_t kLow = 0xff80ff80u, kHigh = 0x7f807f80u;  // -inf, +inf
    uint4 mx[2], mn[2];
    mx[0] = mx[1] = make_uint4(kLow, kLow, kLow, kLow);
    mn[0] = mn[1] = make_uint4(kHigh, kHigh, kHigh, kHigh);
    if (rg == 0) {
        if (r0 == 0) {
            mx[0] = mn[0] = va[0];
            mx[1] = mn[1] = vb[0];
        } else {
            mx[0] = *reinterpret_cast<const uint4*>(st + ca);
            mx[1] = *reinterpret_cast<const uint4*>(st + cb);
            mn[0] = *reinterpret_cast<const uint4*>(st + D + ca);
            mn[1] = *reinterpret_cast<const uint4*>(st + D + cb);
        }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint4* v = c == 0 ? va : vb;
#pragma unroll
        for (int i = 0; i < TL::NP; ++i) {
            const int r = rg * TL::NP + i;
            if (r >= r0 && r < r1) bf16_fold8(v[i], mx[c], mn[c]);
        }
#pragma unroll
        for (int off = TL::LPR; off < 32; off <<= 1) {
            const bool up = (rg * TL::LPR) & off;  // this group comes after its partner
            uint4 ox, on;
            ox.x = __shfl_xor_sync(0xffffffffu, mx[c].x, off);
            ox.y = __shfl_xor_sync(0xffffffffu, mx[c].y, off);
            ox.z = __shfl_xor_sync(0xffffffffu, mx[c].z, off);
            ox.w = __shfl_xor_sync(0xffffffffu, mx[c].w, off);
            on.x = __shfl_xor_sync(0xffffffffu, mn[c].x, off);
            on.y = __shfl_xor_sync(0xffffffffu, mn[c].y, off);
            on.z = __shfl_xor_sync(0xffffffffu, mn[c].z, off);
            on.w = __shfl_xor_sync(0xffffffffu, mn[c].w, off);
            uint4 fx = up ? ox : mx[c], fn = up ? on : mn[c];  // the earlier group's
            const uint4 lx = up ? mx[c] : ox, ln = up ? mn[c] : on;  // the later group's
            uint4 unused_x = fx, unused_n = fn;
            bf16_fold8(lx, fx, unused_n);
            bf16_fold8(ln, unused_x, fn);
            mx[c] = fx;
            mn[c] = fn;
        }
    }
    if (rg == 0) {
        *reinterpret_cast<uint4*>(st + ca) = mx[0];
        *reinterpret_cast<uint4*>(st + cb) = mx[1];
        *reinterpret_cast<uint4*>(st + D + ca) = mn[0];
        *reinterpret_cast<uint4*>(st + D + cb) = mn[1];
    }
}

// Grid: (windows * slices, B). CTA (window, slice) of request b takes the new tokens of the
// window'th logical page from the one that holds position seq_lens[b], for every slices'th
// group of eight units: the KV heads' K, their V, then the query heads.
template <int D, int FMT>
__global__ void __launch_bounds__(kRopeThreads, 3)
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
        // a warp's unit u is one head's K, V or query rows; its rows are loaded together, the
        // first unit's while the table is made
        const int32_t units = 2 * Hkv + p.Hq;
        int32_t u = slice * kRopeWarps + warp;
        uint4 va[TL::NP], vb[TL::NP];
        auto load = [&]() {
            if (u >= units) return;
            const int kind = u < Hkv ? 0 : u < 2 * Hkv ? 1 : 2;
            const uint16_t* x = kind == 0 ? p.k_new : kind == 1 ? p.v_new : p.q;
            const int64_t stride = kind == 0 ? p.k_stride : kind == 1 ? p.v_stride : p.q_stride;
            x += tok0 * stride + (int64_t)(u - kind * Hkv) * D;
#pragma unroll
            for (int i = 0; i < TL::NP; ++i) {
                const int r = rg * TL::NP + i;
                va[i] = vb[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r >= r0 && r < r1) {
                    va[i] = *reinterpret_cast<const uint4*>(x + r * stride + ca);
                    vb[i] = *reinterpret_cast<const uint4*>(x + r * stride + cb);
                }
            }
        };
        load();
        // the logical page's place in the pool: looked up here, checked after the table
        const int32_t lp = base / P;
        const bool within = lp < p.L.max_pages_per_req;
        int32_t page = within ? __ldg(p.L.block_table + (int64_t)b * p.L.max_pages_per_req + lp) : -1;
        fill_table<D>(tab, p.rot, false, r0, r1, [&](int r) {
            return p.positions ? __ldg(p.positions + tok0 + r) : base + r;
        });
        if (page < 0 || page >= p.L.num_pages) {
            if (threadIdx.x == 0)
                set_err(p.dev_err, !within    ? DATTN_DEVERR_LEN_OOB
                                   : page < 0 ? DATTN_DEVERR_UNMAPPED_PAGE
                                              : DATTN_DEVERR_PAGE_OOB);
            page = -1;
        }
        const int32_t slot0 = base - lp * P;
        __syncthreads();
        while (u < units) {
            const int kind = u < Hkv ? 0 : u < 2 * Hkv ? 1 : 2;
            const int32_t h = u - kind * Hkv;
            if (kind != 1) {
#pragma unroll
                for (int i = 0; i < TL::NP; ++i) {
                    const int r = rg * TL::NP + i;
                    if (r >= r0 && r < r1) {
                        float x[8], y[8];
                        unpack8(va[i], x);
                        unpack8(vb[i], y);
                        rotate(x, y, tab, r, l, p.rot);
                        va[i] = pack8(x);
                        vb[i] = pack8(y);
                        if (kind == 2) {
                            uint16_t* dst = p.q_out + ((tok0 + r) * p.Hq + h) * D;
                            *reinterpret_cast<uint4*>(dst + ca) = va[i];
                            *reinterpret_cast<uint4*>(dst + cb) = vb[i];
                        }
                    }
                }
            }
            if (kind != 2 && page >= 0) {
                const int64_t row0 = ((int64_t)page * Hkv + h) * P + slot0;
                int64_t crow0 = row0;
                uint8_t* pool = kind == 0 ? p.k_pool : p.v_pool;
                bool i4 = FMT == DATTN_KV_INT4;
                if constexpr (FMT == DATTN_KV_MIXED) {  // each format in its own region
                    i4 = head_is_i4(p.hf, h);
                    const int32_t h4 = p.hf.h4, h8 = Hkv - h4;
                    crow0 =
                        ((int64_t)page * (i4 ? h4 : h8) + head_class_index(p.hf, h, i4)) * P + slot0;
                    if (i4) pool += (int64_t)p.L.num_pages * h8 * P * D;
                }
                // r0 > 0: the page already holds tokens of this request
                write_rows<D, FMT>(p, pool, row0, crow0, kind, i4, va, vb, r0, r1, r0 > 0, l, rg, ca,
                                   cb);
                if (kind == 0 && p.stats != nullptr) {
                    uint16_t* st = p.stats + (row0 >> 4) * 2 * D;
                    fold_stats<D>(st, va, vb, r0, r1, rg, ca, cb);
                }
            }
            u += p.slices * kRopeWarps;
            load();
        }
    }
    if (p.advance) {
        __syncwarp();
        cluster_wait();  // every thread of the request's CTAs has read the length
        if (blockIdx.x == 0 && threadIdx.x == 0 && !bad) p.seq_lens[b] = pos0 + n;
    }
}

// One new token per request (T = 1, a decode step), where latency counts. Grid (slices, B). A lane
// group of D/16 lanes takes one unit's row (a KV head's K or V, or a query head), so a warp has
// 32 / (D/16) units in hand with one row each, and whatever a unit's logical page holds already (its
// scale, its statistics) is read before the rotation. Measured on 32 + 2 x 8 heads of 128 (block-
// scaled pool with statistics, calls back to back in a graph): 64 requests 2.7 us, 6.2 us by the
// window kernel, whose warps walk 16 rows for the one; one request into a bf16 pool 2.3 and 2.7.
template <int D, int FMT>
__global__ void __launch_bounds__(kRopeThreads)
rope_append_token_kernel(const __grid_constant__ RopeAppendParams p) {
    using TL = Tile<D>;
    __shared__ __align__(16) RopeTable<D, 1> tab;
    const int lane = threadIdx.x & 31;
    const int l = lane % TL::LPR, group = threadIdx.x / TL::LPR;
    constexpr int kGroups = kRopeThreads / TL::LPR;
    const int32_t b = blockIdx.y, Hkv = p.L.num_kv_heads, P = p.L.page_size;
    int ca, cb;
    lane_chunks(l, p.rot.rot_dim, ca, cb);
    grid_dependency_wait();
    grid_launch_dependents();
    const int32_t pos0 = p.seq_lens[b];
    const int32_t n = new_count(p.new_lens, b, 1, blockIdx.x == 0 && threadIdx.x == 0
                                                      ? p.dev_err : nullptr);
    const int32_t units = 2 * Hkv + p.Hq;
    int32_t u = blockIdx.x * kGroups + group;
    uint4 va, vb;
    auto load = [&]() {
        va = vb = make_uint4(0u, 0u, 0u, 0u);
        if (u >= units) return;
        const int kind = u < Hkv ? 0 : u < 2 * Hkv ? 1 : 2;
        const uint16_t* x = kind == 0 ? p.k_new : kind == 1 ? p.v_new : p.q;
        x += b * (kind == 0 ? p.k_stride : kind == 1 ? p.v_stride : p.q_stride) +
             (int64_t)(u - kind * Hkv) * D;
        va = *reinterpret_cast<const uint4*>(x + ca);
        vb = *reinterpret_cast<const uint4*>(x + cb);
    };
    load();  // the row does not depend on the length
    if (p.advance) {
        __syncwarp();
        cluster_arrive();  // this thread has read the length
    }
    const bool bad = pos0 < 0 || pos0 >= (1 << 30);
    if (bad) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_err(p.dev_err, DATTN_DEVERR_LEN_OOB);
    } else if (n > 0) {
        const int32_t lp = pos0 / P;
        const bool within = lp < p.L.max_pages_per_req;
        int32_t page = within ? __ldg(p.L.block_table + (int64_t)b * p.L.max_pages_per_req + lp) : -1;
        fill_table<D>(tab, p.rot, false, 0, 1,
                      [&](int) { return p.positions ? __ldg(p.positions + b) : pos0; });
        if (page < 0 || page >= p.L.num_pages) {
            if (threadIdx.x == 0)
                set_err(p.dev_err, !within    ? DATTN_DEVERR_LEN_OOB
                                   : page < 0 ? DATTN_DEVERR_UNMAPPED_PAGE
                                              : DATTN_DEVERR_PAGE_OOB);
            page = -1;
        }
        const int32_t slot = pos0 - lp * P, r0 = pos0 & 15;
        __syncthreads();
        // the warp's groups stay together: a group past the last unit computes on zeros
        for (int32_t u0 = u - group % TL::RPP; u0 < units; u0 += gridDim.x * kGroups) {
            const int kind = u < Hkv ? 0 : u < 2 * Hkv ? 1 : 2;
            const int32_t h = u - kind * Hkv;
            const bool write = u < units && kind != 2 && page >= 0;
            const int64_t row = ((int64_t)page * Hkv + h) * P + slot;
            const bool stats = write && kind == 0 && p.stats != nullptr;
            uint16_t* st = p.stats + (row >> 4) * 2 * D;
            uint4 xa, xb, na, nb;  // the page's k_max and k_min
            float was = 0.f;
            if (r0 > 0) {
                if (FMT == DATTN_KV_FP8_BLOCK && write)
                    was = p.L.kv_scale[(row >> 4) * 2 + kind];
                if (stats) {
                    xa = *reinterpret_cast<const uint4*>(st + ca);
                    xb = *reinterpret_cast<const uint4*>(st + cb);
                    na = *reinterpret_cast<const uint4*>(st + D + ca);
                    nb = *reinterpret_cast<const uint4*>(st + D + cb);
                }
            }
            if (kind != 1) {
                float x[8], y[8];
                unpack8(va, x);
                unpack8(vb, y);
                rotate(x, y, tab, 0, l, p.rot);
                va = pack8(x);
                vb = pack8(y);
                if (kind == 2 && u < units) {
                    uint16_t* dst = p.q_out + ((int64_t)b * p.Hq + h) * D;
                    *reinterpret_cast<uint4*>(dst + ca) = va;
                    *reinterpret_cast<uint4*>(dst + cb) = vb;
                }
            }
            float m = 0.f;  // the row's largest magnitude
            if constexpr (FMT != DATTN_KV_BF16) {
                m = fmaxf(absmax8(va), absmax8(vb));
#pragma unroll
                for (int off = 1; off < TL::LPR; off <<= 1)
                    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
            }
            if (write) {
                int64_t crow = row;
                uint8_t* pool = kind == 0 ? p.k_pool : p.v_pool;
                bool i4 = FMT == DATTN_KV_INT4;
                if constexpr (FMT == DATTN_KV_MIXED) {  // each format in its own region
                    i4 = head_is_i4(p.hf, h);
                    const int32_t h4 = p.hf.h4, h8 = Hkv - h4;
                    crow = ((int64_t)page * (i4 ? h4 : h8) + head_class_index(p.hf, h, i4)) * P + slot;
                    if (i4) pool += (int64_t)p.L.num_pages * h8 * P * D;
                }
                if constexpr (FMT == DATTN_KV_BF16) {
                    uint16_t* dst = reinterpret_cast<uint16_t*>(pool) + crow * D;
                    *reinterpret_cast<uint4*>(dst + ca) = va;
                    *reinterpret_cast<uint4*>(dst + cb) = vb;
                } else if constexpr (FMT == DATTN_KV_FP8_BLOCK) {
                    const float s = fmaxf(was, block_scale(m)), inv = pow2_inverse(s);
                    const __nv_bfloat162 inv2 = __float2bfloat162_rn(inv);  // exact
                    if (s > was && was > 0.f) {  // earlier rows move to the larger scale
                        const float f = was * inv;
                        for (int32_t r = 1; r <= r0; ++r) {
                            uint2* a = reinterpret_cast<uint2*>(pool + (crow - r) * D + ca);
                            uint2* c = reinterpret_cast<uint2*>(pool + (crow - r) * D + cb);
                            const uint2 x = *a, y = *c;
                            *a = make_uint2(recode4(x.x, f), recode4(x.y, f));
                            *c = make_uint2(recode4(y.x, f), recode4(y.y, f));
                        }
                    }
                    *reinterpret_cast<uint2*>(pool + crow * D + ca) = codes8(va, inv2);
                    *reinterpret_cast<uint2*>(pool + crow * D + cb) = codes8(vb, inv2);
                    if (l == 0) p.L.kv_scale[(row >> 4) * 2 + kind] = s;
                } else {
                    float s;
                    if (i4) {
                        uint8_t* dst = pool + crow * (D / 2);
                        *reinterpret_cast<uint32_t*>(dst + ca / 2) = quant4_chunk(va, m, s);
                        *reinterpret_cast<uint32_t*>(dst + cb / 2) = quant4_chunk(vb, m, s);
                    } else {
                        uint8_t* dst = pool + crow * D;
                        *reinterpret_cast<uint2*>(dst + ca) = quant8_chunk(va, m, s);
                        *reinterpret_cast<uint2*>(dst + cb) = quant8_chunk(vb, m, s);
                    }
                    if (l == 0) p.L.kv_scale[(row >> 4) * 32 + 16 * kind + r0] = s;
                }
                if (stats) {
                    if (r0 == 0) {  // this token opens the page
                        xa = na = va;
                        xb = nb = vb;
                    } else {
                        bf16_fold8(va, xa, na);
                        bf16_fold8(vb, xb, nb);
                    }
                    *reinterpret_cast<uint4*>(st + ca) = xa;
                    *reinterpret_cast<uint4*>(st + cb) = xb;
                    *reinterpret_cast<uint4*>(st + D + ca) = na;
                    *reinterpret_cast<uint4*>(st + D + cb) = nb;
                }
            }
            u += gridDim.x * kGroups;
            load();
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

// CTAs that share the heads of a window: about eight CTAs per SM in all (near three waves), a head
// each at least. 2, 4, 8 and 12 per SM measured: 42.9, 42.9, 41.5 and 41.5 us for 16384 tokens of 32
// heads; 39.0, 34.6, 33.9 and 35.5 us for an append of 2 x 4093 tokens, where a window makes its
// table once per slice.
int32_t head_slices(int64_t windows, int32_t heads) {
    const int64_t want = (8 * (int64_t)sm_count_current() + windows - 1) / windows;
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
    // T tokens from any position touch at most this many logical pages. A single token has a
    // kernel of its own.
    const int64_t windows = T == 1 ? 1 : ((int64_t)T + 30) / kWin;
    const int32_t units = 2 * L.num_kv_heads + Hq;
    const int32_t groups = kRopeThreads / (L.head_dim / 16);  // rows a CTA of that kernel has in hand
    int32_t slices = T == 1 ? (units + groups - 1) / groups : head_slices(windows * B, units);
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
#define DATTN_ROPE_KERNELS(K_, D_)                                                      \
    pick(K_<D_, DATTN_KV_BF16>, K_<D_, DATTN_KV_FP8_E4M3>, K_<D_, DATTN_KV_INT4>,       \
         K_<D_, DATTN_KV_MIXED>, K_<D_, DATTN_KV_FP8_BLOCK>)
    auto kern = T == 1 ? (L.head_dim == 64 ? DATTN_ROPE_KERNELS(rope_append_token_kernel, 64)
                                           : DATTN_ROPE_KERNELS(rope_append_token_kernel, 128))
                       : (L.head_dim == 64 ? DATTN_ROPE_KERNELS(rope_append_kernel, 64)
                                           : DATTN_ROPE_KERNELS(rope_append_kernel, 128));
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
