// Shared parts of the paged attention (csa2_paged_attn_fp8): arguments, the
// requests' rows and keys, the line of work that CTAs share out, and the output
// of a row.
#pragma once

#include "common.cuh"

namespace csa2 {

// A unit that a CTA began and did not finish, for the kernel that joins the parts:
// CTA c's part is slot 2 c + 1, those of the CTAs after it, to the last, slots 2 c'.
struct JoinUnit {
    int64_t row0;                   // first row of the request
    int h, r0, rows, last;          // KV head, first row of the unit, rows of the request, last CTA (-1: no such unit)
    int pad[2];
};

struct PagedAttnArgs {
    int B, Hq, Hkv, G, S, M, window;
    int64_t T, n_blocks, table_stride, q_token_stride, q_head_stride;
    const uint16_t *q;
    const uint8_t *k_codes, *v_codes;
    const float *k_scale, *v_scale;
    const int32_t *table, *kv_len, *cu_len;
    float logit_scale;              // sm_scale * log2(e)
    uint16_t *out;
    float *lse;
    uint32_t *err_flag;
    int split_rows;                 // requests of more rows than this are the tile kernel's
    JoinUnit *join, *join_tc;       // one per CTA of the split and of the tile kernel
    float *partial;                 // split kernel's [2 * CTAs][8 NT rows][D + 4]: o, m, mv, l
    float *partial_tc;              // tile kernel's [2 * CTAs][256 rows][D + 4]
};

// The weights of the values go to f16 with 2^kUp above the reference Mv, the largest
// of a row's z + log2(v_scale): f16 has 2^15 above 1 and 2^-14 (2^-24 with subnormals)
// below.  Weights down to 2^-22 of all weights' sum keep their 11 bits; smaller ones are off
// by 2^-33 of it at most, which a long tail of n keys adds up to n 2^-33 (2^-16 at 131k).
// More room below leaves less above, by which scores may exceed the references before these
// have to move: 3 prompts of up to 4096 tokens on up to 8192 took 841 us with 8 (803 with
// 0, 820 with 4, 871 with 10), the windows of paged_attn.cu 36.5 (35.0 with 0), 64 requests of
// up to 16k tokens the same with any.
constexpr int kUp = 8;
constexpr float kUpFactor = 1 << kUp, kDownFactor = 1.0f / kUpFactor;
constexpr float kMostWeight = 0x1p118f;      // bound of v_scale 2^(M - Mv): finite times 2^kUp, for scales of keys that no row sees

__device__ __forceinline__ void cp_async16(uint32_t smem, const void *gmem, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Byte offset of 16-byte chunk c of row r in a tile of D-byte rows, swizzled so
// that the fragment loads below meet every bank once.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// log2 of 2^kUp v_scale for the common case of both kernels, whose factors 2^(Mv - M) and
// 1 / v_scale stay normal fp32 numbers for scales within 2^+-40; -inf for others (and 0),
// which take the way with maxima.
__device__ __forceinline__ float log_scale(float vs) {
    return vs >= 0x1p-40f && vs <= 0x1p40f ? lg2(vs) + kUp : __int_as_float(0xff800000);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <bool HALF>
__device__ __forceinline__ float2 unpack_in(uint32_t w) {
    if (HALF) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool HALF>
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
    if (HALF) return pack_f16(lo, hi);
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Request b's rows and keys, clamped to what the tensors hold.
struct Request {
    int64_t row0;
    int n, kv;
};
__device__ __forceinline__ Request request_of(const PagedAttnArgs &a, int b) {
    const int64_t c0 = a.cu_len[b], c1 = a.cu_len[b + 1], cap = (int64_t)a.M * a.S, k = a.kv_len[b];
    Request r;
    r.row0 = c0 < 0 ? 0 : (c0 > a.T ? a.T : c0);
    const int64_t e = c1 < r.row0 ? r.row0 : (c1 > a.T ? a.T : c1);
    r.n = (int)(e - r.row0);
    r.kv = (int)(k < 0 ? 0 : (k > cap ? cap : k));
    return r;
}

// A request's work is a number of units (KV head, tile of query rows), each a
// number of key tiles.  The units' key tiles, in the order of requests, heads
// and row tiles, are one long line that the CTAs cut into equal shares: a ragged
// batch loads every SM alike, and a long context is split over as many CTAs as
// it is worth.  A CTA's piece of a unit is a segment; only its first and its
// last segment can be parts of a unit.  A segment's fixed cost (its rows of Q, the
// first loads, its output) counts too: a unit stands in the line with so many
// places more, before its tiles, which nobody works on.
struct Plan {
    int64_t share;                  // key tiles per CTA, a multiple of `round`
    int b;                          // request that holds the CTA's first tile (if there is one)
    int64_t base;                   // that request's first tile in the line
    int64_t total;
};

// Every thread of the block takes a run of requests; a prefix sum over the
// threads finds the total and the thread that holds the CTA's first tile.
template <typename Work>
__device__ __forceinline__ Plan plan_of(const PagedAttnArgs &a, int cta, int ctas, int round, int64_t *s_sum,
                                        int64_t *s_found) {
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.B + nt - 1) / nt, b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += Work::tiles(a, request_of(a, b));
    int64_t s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += y;
    }
    if (lane == 31) s_sum[warp] = s;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < nt / 32; ++w) {
        if (w < warp) before += s_sum[w];
        total += s_sum[w];
    }
    Plan p;
    p.total = total;
    const int64_t even = (total + ctas - 1) / ctas;
    p.share = (even + round - 1) / round * round;
    const int64_t t0 = cta * p.share;
    int64_t at = before + s - mine;
    if (t0 >= at && t0 < at + mine) {
        for (int b = b0; b < b1; ++b) {
            const int64_t w = Work::tiles(a, request_of(a, b));
            if (t0 < at + w) {
                s_found[0] = b;
                s_found[1] = at;
                break;
            }
            at += w;
        }
    }
    __syncthreads();
    p.b = (int)s_found[0];
    p.base = s_found[1];
    return p;
}

// Where in a unit a place of the line is.
struct Place {
    int h, r0, tile, tiles;         // KV head, first row, place in the unit, the unit's places
};

// The split kernel's work: units of R = 8 NT rows, key tiles of K keys (4 KB of
// keys); every row tile of a request has the same tiles, at least one so that each row gets its
// output, and counts as a whole number of rounds of the CTA's warps, so that short
// units go to CTAs of their own.
// kSplitCost: 64 requests of up to 16k tokens (8 heads of 128) 185 us with 16, 186 with
// 8, 192 with 0; 48 of up to 9k in a window of 4096 (5 heads of 64) 35.0, 36.0 and
// (before the segments' first loads were reordered) 42.0 against 36.7; 35.6 with 20.
constexpr int kSplitWarps = 4, kSplitCost = 16;
static_assert(kSplitCost % kSplitWarps == 0, "segments begin at whole rounds of the warps");
template <int R, int K>
struct SplitWork {
    static __device__ __forceinline__ int low_key(const PagedAttnArgs &a, const Request &r) {       // of the first row's window
        const int64_t p = (int64_t)r.kv - r.n - a.window + 1;
        return a.window > 0 && p > 0 ? (int)p : 0;
    }
    static __device__ __forceinline__ int first_key(const PagedAttnArgs &a, const Request &r) { return low_key(a, r) & ~(K - 1); }
    static __device__ __forceinline__ int real_tiles(const PagedAttnArgs &a, const Request &r) {
        const int keys = r.kv - first_key(a, r);
        return keys > 0 ? (keys + K - 1) / K : 1;
    }
    static __device__ __forceinline__ int unit_places(const PagedAttnArgs &a, const Request &r) {
        return kSplitCost + (real_tiles(a, r) + kSplitWarps - 1) / kSplitWarps * kSplitWarps;
    }
    static __device__ __forceinline__ int64_t tiles(const PagedAttnArgs &a, const Request &r) {
        const int rows = r.n * a.G;
        return rows > a.split_rows ? 0 : (int64_t)((rows + R - 1) / R) * a.Hkv * unit_places(a, r);
    }
    static __device__ __forceinline__ Place place(const PagedAttnArgs &a, const Request &r, int64_t off) {
        const int row_tiles = (r.n * a.G + R - 1) / R, per = unit_places(a, r);
        const int unit = (int)(off / per);
        Place p;
        p.h = unit / row_tiles;
        p.r0 = (unit - p.h * row_tiles) * R;
        p.tile = (int)(off - (int64_t)unit * per);
        p.tiles = per;
        return p;
    }
};

// The tile kernel's work: units of 256 rows, key tiles of 128, for each row tile
// those that its first to last row see.
// kTcCost, when it was chosen: 3 prompts of up to 4096 tokens on up to 8192 (32 heads of
// 128) 794 us, 801 with 3, 796 with 7; before, 905 with 0, 854 with 4 and with 6, 872 with 10.
constexpr int kTcRows = 256, kTcKeys = 128, kTcCost = 5;
struct TcWork {
    // A walk over the row tiles of a request, without a division per step.
    struct Rows {
        int G, q256, m256, q255, m255;
        int r0, tok, rem;                 // first row = tok * G + rem
        __device__ __forceinline__ Rows(int g) : G(g), q256(kTcRows / g), m256(kTcRows % g), q255((kTcRows - 1) / g),
                                                 m255((kTcRows - 1) % g), r0(0), tok(0), rem(0) {}
        __device__ __forceinline__ void next() {
            r0 += kTcRows;
            tok += q256;
            rem += m256;
            if (rem >= G) ++tok, rem -= G;
        }
        __device__ __forceinline__ int last_tok() const { return tok + q255 + (rem + m255 >= G); }
    };
    static __device__ __forceinline__ int low_key(const PagedAttnArgs &a, const Request &r, const Rows &w) {
        const int64_t p = (int64_t)r.kv - r.n + w.tok - a.window + 1;
        return a.window > 0 && p > 0 ? (int)p : 0;
    }
    static __device__ __forceinline__ int first_key(const PagedAttnArgs &a, const Request &r, const Rows &w) {
        return low_key(a, r, w) & ~(kTcKeys - 1);
    }
    static __device__ __forceinline__ int unit_places(const PagedAttnArgs &a, const Request &r, const Rows &w) {
        const int last = min(w.last_tok(), r.n - 1);
        const int keys = min(r.kv, r.kv - r.n + last + 1) - first_key(a, r, w);
        return kTcCost + (keys > 0 ? (keys + kTcKeys - 1) / kTcKeys : 1);
    }
    static __device__ __forceinline__ bool mine(const PagedAttnArgs &a, const Request &r) { return r.n * a.G > a.split_rows; }
    static __device__ __forceinline__ int64_t head_tiles(const PagedAttnArgs &a, const Request &r) {
        int64_t n = 0;
        for (Rows w(a.G); w.r0 < r.n * a.G; w.next()) n += unit_places(a, r, w);
        return n;
    }
    static __device__ __forceinline__ int64_t tiles(const PagedAttnArgs &a, const Request &r) {
        return mine(a, r) ? head_tiles(a, r) * a.Hkv : 0;
    }
    // The unit of place `off` of the request's tiles; `w` is left at its row tile.
    static __device__ __forceinline__ Place place(const PagedAttnArgs &a, const Request &r, int64_t off, Rows &w) {
        const int64_t per = head_tiles(a, r);
        Place p;
        p.h = (int)(off / per);
        int64_t left = off - p.h * per;
        for (;; w.next()) {
            p.tiles = unit_places(a, r, w);
            if (left < p.tiles) break;
            left -= p.tiles;
        }
        p.r0 = w.r0;
        p.tile = (int)left;
        return p;
    }
};

// P threads per row, D / P channels each: o = x / (2^kUp l) f in the output's type (f = 2^(Mv - M)), lse.
template <int D, bool HALF, int P>
__device__ __forceinline__ void store_row(const PagedAttnArgs &a, int64_t o_row, int part, const float *x, float f, float M, float l) {
    const float inv = l > 0.0f ? kDownFactor / l : (l == 0.0f ? 0.0f : l);
    constexpr int W = D / P / 2;
    uint32_t w[W];
#pragma unroll
    for (int c = 0; c < W; ++c) w[c] = pack_out<HALF>(x[2 * c] * inv * f, x[2 * c + 1] * inv * f);
    uint16_t *dst = a.out + o_row * D + part * (D / P);
    if constexpr (W == 2) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int c = 0; c < W; c += 4) *reinterpret_cast<uint4 *>(dst + 2 * c) = make_uint4(w[c], w[c + 1], w[c + 2], w[c + 3]);
    }
    if (a.lse && part == 0) a.lse[o_row] = l > 0.0f || l != l ? (M + log2f(l)) * 0.69314718055994531f : __int_as_float(0xff800000);
}

// The tile kernel (paged_attn_tc.cu): one CTA per SM.
int paged_attn_tc_ctas();
cudaError_t launch_paged_attn_tc(const PagedAttnArgs &a, int D, bool half, cudaStream_t stream);

}  // namespace csa2
