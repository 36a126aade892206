// csa2_quantize_kv_fp4_paged and csa2_dequantize_kv_fp4_paged: bf16 / fp16 key and
// value rows -> E2M1 codes and E4M3 scales (one per 16 channels) in the blocks of the
// paged 4-bit cache, the keys rotated on the way if asked, and back.
//
// A row's codes depend on that row alone, so tokens go to the threads freely: a thread
// takes the 16 channels of one scale, for several heads of a token, whose cosines and
// sines (keys) it loads once.  No exchange between threads.
//
// Exact rounding without a division: let s be the scale (4 significant bits) and x a
// value of 8 (bf16) or 11 (fp16).  A tie of |x| / s on the E2M1 grid, or of amax / 6 on
// the E4M3 grid, happens only where the quotient is exactly a midpoint, of at most 5
// significant bits; x and midpoint times s have at most 11 bits, so any other quotient
// is 2^-12 or more (relative) away from every midpoint.  The quotient is formed by a
// multiplication (relative error below 2^-21) and rounded to 16 bits, which brings exact
// midpoints back and carries no other value across one.
//
// Bound by memory and, in the append, nearly as much by issue (0.56 instructions per cycle).  16384
// tokens, 8 heads of 128, keys rotated, with the stored values (152 MB): 27.6 us, 5.5 TB/s of a
// copy's 6.8 (40000 tokens 59.9, 6.2 TB/s); a decode step's 64 tokens 2.1 us in a graph.  28.5, 61.8 and 2.3 with
// a row's loads behind those of its place.
#include "fp4.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 64;         // of a block (16384 tokens as above: 128 0.9 us slower)

struct Rope4 {
    const int32_t *pos;
    const float *table;              // NULL: no rotation
    int64_t n_pos;
    int pairs, first;
    bool split;
};

struct Quant4Args {
    const uint16_t *x[2];            // k, v
    int64_t token_stride[2], head_stride[2];
    uint8_t *codes[2], *scales[2];
    uint16_t *values[2];             // what the codes stand for [T, H, D], or NULL
    const int64_t *slots;
    int64_t T, n_slots;
    int H, S, shift, per;
    uint32_t chunks;                 // heads per thread, threads' shares of a token's heads
    Rope4 rope;
    uint32_t *err_flag;
};

// fp32 to 16 significant bits, nearest (not for infinities and NaN).
__device__ __forceinline__ float round16(float v) { return __uint_as_float((__float_as_uint(v) + 0x80u) & 0xFFFFFF00u); }

__device__ __forceinline__ float rcp_of(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// fp32 -> E4M3 byte, nearest even, saturating.
__device__ __forceinline__ uint32_t to_e4m3(float v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xFFu;
}

// The keys' or the values' member of a pair among a kernel's arguments.  A select: an index
// would have every thread copy the arguments to local memory first (65536 tokens read back, 8
// heads of 128: 79 us).
template <typename X>
__device__ __forceinline__ X of(const X (&pair)[2], bool is_v) { return is_v ? pair[1] : pair[0]; }

// The values of eight codes, of either 16-bit type.
template <bool HALF>
__device__ __forceinline__ uint4 values8(uint32_t codes, uint32_t scale2) {
    uint32_t r[4];
    e2m1x8_to_f16(codes, scale2, r);
    if (!HALF)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 z = unpack16<true>(r[k]);
            r[k] = pack16<false>(z.x, z.y);
        }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// The rotation of 8 channels of a key: their cosines and sines, and the channels that
// are their partners.
struct Turn {
    float2 cs[8];                    // split: of each channel; interleaved: of the four pairs
    int partner;                     // split: channels from here to the partners, 0: not rotated
    bool on, low;                    // rotated at all; split: the partners come behind
};

template <bool HALF>
__device__ __forceinline__ void turn8(uint4 &x, const uint4 &y, const Turn &t, bool split) {
    uint32_t *w = reinterpret_cast<uint32_t *>(&x);
    const uint32_t *z = reinterpret_cast<const uint32_t *>(&y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = unpack16<HALF>(w[i]);
        if (split) {
            const float2 p = unpack16<HALF>(z[i]), c0 = t.cs[2 * i], c1 = t.cs[2 * i + 1];
            const float a = t.low ? rotate(v.x, p.x, c0.x, c0.y).x : rotate(p.x, v.x, c0.x, c0.y).y;
            const float b = t.low ? rotate(v.y, p.y, c1.x, c1.y).x : rotate(p.y, v.y, c1.x, c1.y).y;
            w[i] = pack16<HALF>(a, b);
        } else {
            const float2 r = rotate(v.x, v.y, t.cs[i].x, t.cs[i].y);
            w[i] = pack16<HALF>(r.x, r.y);
        }
    }
}

// 16 values w of row (t, h), a group g of its channels: their codes, scale and, if asked
// for, the values that these stand for.
template <bool HALF>
__device__ __forceinline__ void store_group(const Quant4Args &a, bool is_v, int D, int64_t t, int h, int64_t row, int g, uint32_t (&w)[8]) {
    constexpr uint32_t INF = HALF ? 0x7C00u : 0x7F80u, ABS2 = 0x7FFF7FFFu;
    uint32_t m2 = 0;                 // largest sign-less patterns of the even and odd channels
#pragma unroll
    for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & ABS2);
    uint32_t top = max(m2 & 0xFFFFu, m2 >> 16);
    if (top >= INF) {                // infinities and NaN do not count: the one becomes the largest value, the other 0
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t both = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t u = (w[i] >> (16 * k)) & 0xFFFFu;
                const uint32_t mag = u & 0x7FFFu;
                if (mag < INF) top = max(top, mag);
                else u = mag > INF ? 0u : u - 1;
                both |= u << (16 * k);
            }
            w[i] = both;
        }
        flag_error(a.err_flag, CSA2_FLAG_NONFINITE);
    }
    const uint32_t s8 = to_e4m3(round16(unpack16<HALF>(top).x * (1.0f / 6.0f)));
    const uint32_t s2 = e4m3x2_to_f16x2(s8 | s8 << 8);
    const float inv = s8 ? rcp_of(__half2float(__ushort_as_half((unsigned short)(s2 & 0xFFFFu)))) : 0.0f;
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 z = unpack16<HALF>(w[4 * i + k]);
            f[2 * k] = round16(z.x * inv), f[2 * k + 1] = round16(z.y * inv);
        }
        c[i] = to_e2m1x8(f);
    }
    *reinterpret_cast<uint2 *>(of(a.codes, is_v) + row * (D / 2) + 8 * g) = make_uint2(c[0], c[1]);
    of(a.scales, is_v)[row * (D / 16) + g] = (uint8_t)s8;
    if (of(a.values, is_v)) {
        uint4 *dst = reinterpret_cast<uint4 *>(of(a.values, is_v) + (t * a.H + h) * D + 16 * g);
        dst[0] = values8<HALF>(c[0], s2);
        dst[1] = values8<HALF>(c[1], s2);
    }
}

// Where a token's row goes: false, and a flag if that is an error, if it is not stored.
__device__ __forceinline__ bool place_of(const Quant4Args &a, int64_t t, bool first_thread, int64_t &row0, int64_t &p) {
    const int64_t slot = a.slots[t];
    p = a.rope.table ? a.rope.pos[t] : 0;                // on its way beside the slot
    if (slot < 0 || slot >= a.n_slots) {
        if (slot != -1 && first_thread) flag_error(a.err_flag, CSA2_FLAG_BAD_SLOT);
        return false;
    }
    if (a.rope.table) {              // a token without a position is not stored
        if (p < 0 || p >= a.rope.n_pos) {
            if (first_thread) flag_error(a.err_flag, CSA2_FLAG_BAD_INDEX);
            return false;
        }
    }
    row0 = (slot >> a.shift) * a.H * a.S + (slot & (a.S - 1));       // of head 0; the others S rows apart
    return true;
}

// Any rotation: a thread takes one group of a row and reads its partners beside it.  16384 tokens,
// 8 heads of 128: 33.7 us with pairs side by side, 34.1 with halves of 64 channels (4.5 TB/s; issue 0.49 a cycle,
// and loads that it waits for: none are under way while a row is stored, and partners are asked for twice).
template <bool HALF>
__global__ void __launch_bounds__(kThreads) quantize_fp4_paged_any_kernel(Quant4Args a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= a.T) return;
    const int g = threadIdx.x, D = blockDim.x * 16;
    const bool is_v = blockIdx.y >= a.chunks;
    const int chunk = is_v ? blockIdx.y - a.chunks : blockIdx.y;
    int64_t row0, p;
    if (!place_of(a, t, g == 0 && blockIdx.y == 0, row0, p)) return;
    Turn turn[2];
    turn[0].on = turn[1].on = false;
    if (!is_v) {
        const float *row = a.rope.table + 2 * p * a.rope.pairs;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = 16 * g + 8 * i - a.rope.first;             // of the rotated channels
            Turn &u = turn[i];
            if (c < 0 || c >= 2 * a.rope.pairs) continue;
            u.on = true;
            u.low = c < a.rope.pairs;
            u.partner = u.low ? a.rope.pairs : -a.rope.pairs;
            const float4 *src = reinterpret_cast<const float4 *>(row + (a.rope.split ? 2 * (u.low ? c : c - a.rope.pairs) : c));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k >= 2 && !a.rope.split) continue;
                const float4 v = src[k];
                u.cs[2 * k] = make_float2(v.x, v.y), u.cs[2 * k + 1] = make_float2(v.z, v.w);
            }
        }
    }
    const int64_t hs = of(a.head_stride, is_v);
    const uint16_t *x = of(a.x, is_v) + t * of(a.token_stride, is_v) + 16 * g;
    const int h0 = chunk * a.per, h1 = min(a.H, h0 + a.per);
    for (int h = h0; h < h1; ++h) {
        uint4 v[2], y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            y[i] = v[i] = *reinterpret_cast<const uint4 *>(x + h * hs + 8 * i);
            if (turn[i].on && a.rope.split) y[i] = *reinterpret_cast<const uint4 *>(x + h * hs + 8 * i + turn[i].partner);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (turn[i].on) turn8<HALF>(v[i], y[i], turn[i], a.rope.split);
        uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        store_group<HALF>(a, is_v, D, t, h, row0 + (int64_t)h * a.S, g, w);
    }
}

// No rotation, or one of halves over the whole head: a thread takes a group and the one
// half a row behind it, which are each other's partners, so nothing is read or turned twice: 27.6 us
// where the kernel above takes 34.  The next head's loads are on their way
// meanwhile (34.5 otherwise).
template <bool HALF>
__global__ void __launch_bounds__(kThreads) quantize_fp4_paged_kernel(Quant4Args a) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= a.T) return;
    const int g = threadIdx.x, far = blockDim.x, D = far * 32;
    const bool is_v = blockIdx.y >= a.chunks, turns = a.rope.table && !is_v;
    const int chunk = is_v ? blockIdx.y - a.chunks : blockIdx.y;
    const int64_t hs = of(a.head_stride, is_v);
    const uint16_t *x = of(a.x, is_v) + t * of(a.token_stride, is_v) + 16 * g;
    const int h0 = chunk * a.per, h1 = min(a.H, h0 + a.per);
    uint4 next[4];
    auto load = [&](int h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) next[i] = *reinterpret_cast<const uint4 *>(x + h * hs + (i >> 1) * (D / 2) + (i & 1) * 8);
    };
    load(h0);                        // beside the chain of slot, position and table row
    int64_t row0, p;
    if (!place_of(a, t, g == 0 && blockIdx.y == 0, row0, p)) return;
    float2 cs[16];
    if (turns) {
        const float4 *src = reinterpret_cast<const float4 *>(a.rope.table + p * D + 32 * g);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float4 v = src[k];
            cs[2 * k] = make_float2(v.x, v.y), cs[2 * k + 1] = make_float2(v.z, v.w);
        }
    }
    for (int h = h0; h < h1; ++h) {
        uint32_t w[2][8] = {{next[0].x, next[0].y, next[0].z, next[0].w, next[1].x, next[1].y, next[1].z, next[1].w},
                            {next[2].x, next[2].y, next[2].z, next[2].w, next[3].x, next[3].y, next[3].z, next[3].w}};
        if (h + 1 < h1) load(h + 1);
        if (turns) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 u = unpack16<HALF>(w[0][i]), v = unpack16<HALF>(w[1][i]);
                const float2 r0 = rotate(u.x, v.x, cs[2 * i].x, cs[2 * i].y), r1 = rotate(u.y, v.y, cs[2 * i + 1].x, cs[2 * i + 1].y);
                w[0][i] = pack16<HALF>(r0.x, r1.x), w[1][i] = pack16<HALF>(r0.y, r1.y);
            }
        }
        const int64_t row = row0 + (int64_t)h * a.S;
        store_group<HALF>(a, is_v, D, t, h, row, g, w[0]);
        store_group<HALF>(a, is_v, D, t, h, row, g + far, w[1]);
    }
}

struct Read4Args {
    const uint8_t *codes[2], *scales[2];
    uint16_t *x[2];
    int64_t token_stride[2], head_stride[2];
    const int64_t *slots;
    int64_t T, n_slots;
    int H, S, shift;
    uint32_t *err_flag;
};

// A thread writes 16 bytes of every head of a token, so that a warp's store fills whole sectors
// and the row's place is worked out once.  65536 tokens, 8 heads of 128, to bf16 (344 MB): 55 us,
// 6.3 TB/s of a copy's 6.8; 57.4 with the loads of four heads on their way together in place
// of eight, 60 with the heads dealt out to two threads, 67 with a thread per row.
constexpr int kReadThreads = 64, kReadBatch = 8;         // heads whose loads are on their way together

template <int D, bool HALF>
__global__ void __launch_bounds__(kReadThreads) dequantize_fp4_paged_kernel(Read4Args a) {
    constexpr int TOKENS = kReadThreads / (D / 8);
    pdl_wait();
    pdl_launch_dependents();
    const bool is_v = blockIdx.x & 1;                    // side by side, as the two read the same slots
    const int64_t t = (int64_t)(blockIdx.x >> 1) * TOKENS + threadIdx.x / (D / 8);
    if (t >= a.T) return;
    const int c = threadIdx.x % (D / 8);                 // 8 channels
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) {
        if (slot != -1 && !is_v && c == 0) flag_error(a.err_flag, CSA2_FLAG_BAD_SLOT);
        return;
    }
    const int64_t row = (slot >> a.shift) * a.H * a.S + (slot & (a.S - 1)), hs = of(a.head_stride, is_v);    // of head 0; the others S rows apart
    const uint8_t *codes = of(a.codes, is_v) + row * (D / 2) + 4 * c, *scales = of(a.scales, is_v) + row * (D / 16) + (c >> 1);
    uint16_t *x = of(a.x, is_v) + t * of(a.token_stride, is_v) + 8 * c;
    for (int h = 0; h < a.H; h += kReadBatch) {
        uint32_t w[kReadBatch], s8[kReadBatch];
#pragma unroll
        for (int k = 0; k < kReadBatch; ++k) {
            if (h + k < a.H) {
                w[k] = *reinterpret_cast<const uint32_t *>(codes);
                s8[k] = *scales;
            }
            codes += (int64_t)a.S * (D / 2), scales += (int64_t)a.S * (D / 16);
        }
#pragma unroll
        for (int k = 0; k < kReadBatch; ++k) {
            if (h + k < a.H) *reinterpret_cast<uint4 *>(x) = values8<HALF>(w[k], e4m3x2_to_f16x2(s8[k] | s8[k] << 8));
            x += hs;
        }
    }
}

// Threads of a block, blocks, and heads per thread: as many heads (loads that share a
// token's slot, position and table row) as leave every SM 8 blocks.
struct Shape4 {
    dim3 grid, block;
    int per, chunks;
};
Shape4 shape_of(int64_t T, int H, int groups) {
    const int rows = kThreads / groups;
    const int64_t blocks = (T + rows - 1) / rows;
    int per = 1;
    while (per < 8 && per < H && blocks * 2 * ((H + 2 * per - 1) / (2 * per)) >= (int64_t)num_sms() * 8) per *= 2;
    const int chunks = (H + per - 1) / per;
    return {dim3((unsigned)blocks, 2 * chunks), dim3(groups, rows), per, chunks};
}

csa2_status check4(const char *who, csa2_dtype dt, int64_t T, int H, int D, int64_t n_blocks, int S, const void *k,
                   const void *v, const int64_t *stride, const int64_t *slots, const void *k_codes, const void *v_codes,
                   const void *k_scales, const void *v_scales, const void *err_flag) {
    CSA2_REQUIRE(dt == CSA2_BF16 || dt == CSA2_FP16, "%s: rows must be bf16 or fp16", who);
    CSA2_REQUIRE(T >= 0 && T <= (1ll << 30), "%s: T=%lld not in [0, 2^30]", who, (long long)T);
    CSA2_REQUIRE(H >= 1 && H <= 32767, "%s: Hkv=%d not in [1, 32767]", who, H);
    CSA2_REQUIRE(n_blocks >= 0 && n_blocks < (1ll << 31), "%s: n_blocks=%lld", who, (long long)n_blocks);
    CSA2_REQUIRE(S == 16 || S == 32 || S == 64 || S == 128, "%s: S=%d not in {16, 32, 64, 128}", who, S);
    for (int i = 0; i < 4; ++i)
        CSA2_REQUIRE(stride[i] >= 0 && stride[i] % 8 == 0 && stride[i] < (1ll << 31),
                     "%s: strides must be multiples of 8 in [0, 2^31)", who);
    if (D != 64 && D != 128) {
        set_error("%s: D=%d not in {64, 128}", who, D);
        return CSA2_ERR_UNSUPPORTED;
    }
    if (T == 0) return CSA2_OK;
    CSA2_REQUIRE(k && v && slots, "%s: null pointer", who);
    CSA2_REQUIRE((k_codes && v_codes && k_scales && v_scales) || n_blocks == 0, "%s: null pointer", who);
    CSA2_REQUIRE(aligned(k, 16) && aligned(v, 16), "%s: k and v must be 16-byte aligned", who);
    CSA2_REQUIRE(aligned(k_codes, 16) && aligned(v_codes, 16) && aligned(k_scales, 16) && aligned(v_scales, 16),
                 "%s: codes and scales must be 16-byte aligned", who);
    CSA2_REQUIRE(aligned(slots, 8) && aligned(err_flag, 4), "%s: misaligned slots / flag (8- and 4-byte aligned)", who);
    return CSA2_OK;
}

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" csa2_status csa2_quantize_kv_fp4_paged(const void *k, const void *v, csa2_dtype dt, int64_t T, int Hkv, int D,
                                                  int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                                                  int64_t v_head_stride, const int64_t *slots, int64_t n_blocks, int S,
                                                  uint8_t *k_codes, uint8_t *v_codes, uint8_t *k_scales, uint8_t *v_scales,
                                                  const int32_t *pos, const float *cos_sin, int64_t n_pos, int rope_dim,
                                                  int first, csa2_rope_layout layout, void *k_values, void *v_values,
                                                  uint32_t *err_flag, csa2_stream_t stream) {
    clear_error();
    const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
    const csa2_status st = check4("quantize_fp4_paged", dt, T, Hkv, D, n_blocks, S, k, v, strides, slots, k_codes, v_codes,
                                  k_scales, v_scales, err_flag);
    if (st != CSA2_OK) return st;
    if (cos_sin) {
        CSA2_REQUIRE(rope_dim >= 16 && rope_dim <= D && rope_dim % 16 == 0,
                     "quantize_fp4_paged: rope_dim=%d must be a multiple of 16 in [16, D]", rope_dim);
        CSA2_REQUIRE(first >= 0 && first % 8 == 0 && first + rope_dim <= D,
                     "quantize_fp4_paged: first=%d must be a multiple of 8 in [0, D - rope_dim]", first);
        CSA2_REQUIRE(layout == CSA2_ROPE_INTERLEAVED || layout == CSA2_ROPE_HALF, "quantize_fp4_paged: layout=%d", (int)layout);
        CSA2_REQUIRE(n_pos >= 1 && n_pos <= (1ll << 31), "quantize_fp4_paged: n_pos=%lld not in [1, 2^31]", (long long)n_pos);
    }
    if (T == 0) return CSA2_OK;
    CSA2_REQUIRE((pos != nullptr) == (cos_sin != nullptr), "quantize_fp4_paged: pos and cos_sin go together");
    CSA2_REQUIRE(aligned(pos, 4) && aligned(cos_sin, 16), "quantize_fp4_paged: pos must be 4-byte, cos_sin 16-byte aligned");
    CSA2_REQUIRE(aligned(k_values, 16) && aligned(v_values, 16), "quantize_fp4_paged: values must be 16-byte aligned");
    const Rows in[2] = {{k, T, Hkv, D, k_token_stride, k_head_stride}, {v, T, Hkv, D, v_token_stride, v_head_stride}};
    const int64_t dense = 2 * T * Hkv * D, plane = n_blocks * Hkv * S * (D / 2);
    const struct {
        const void *p;
        int64_t bytes;
    } outs[6] = {{k_codes, plane}, {v_codes, plane}, {k_scales, plane / 8}, {v_scales, plane / 8}, {k_values, k_values ? dense : 0},
                 {v_values, v_values ? dense : 0}},
      ins[6] = {{k, in[0].bytes()}, {v, in[1].bytes()}, {slots, 8 * T}, {pos, pos ? 4 * T : 0},
                {cos_sin, cos_sin ? 4 * n_pos * rope_dim : 0}, {err_flag, err_flag ? 4 : 0}};
    for (int i = 0; i < 6; ++i) {
        bool over = false;
        for (const auto &x : ins) over = over || meet(outs[i].p, outs[i].bytes, x.p, x.bytes);
        for (int j = 0; j < i; ++j) over = over || meet(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes);
        CSA2_REQUIRE(!over, "quantize_fp4_paged: an output (codes, scales or values) overlaps another argument");
    }
    const bool any = cos_sin && (layout != CSA2_ROPE_HALF || rope_dim != D);
    const Shape4 sh = shape_of(T, Hkv, any ? D / 16 : D / 32);
    Quant4Args a = {};
    a.x[0] = (const uint16_t *)k, a.x[1] = (const uint16_t *)v;
    a.token_stride[0] = k_token_stride, a.token_stride[1] = v_token_stride;
    a.head_stride[0] = k_head_stride, a.head_stride[1] = v_head_stride;
    a.codes[0] = k_codes, a.codes[1] = v_codes, a.scales[0] = k_scales, a.scales[1] = v_scales;
    a.values[0] = (uint16_t *)k_values, a.values[1] = (uint16_t *)v_values;
    a.slots = slots, a.T = T, a.n_slots = n_blocks * S, a.H = Hkv, a.S = S, a.err_flag = err_flag;
    a.shift = S == 16 ? 4 : (S == 32 ? 5 : (S == 64 ? 6 : 7));
    a.per = sh.per, a.chunks = sh.chunks;
    a.rope = {pos, cos_sin, n_pos, rope_dim / 2, first, layout == CSA2_ROPE_HALF};
    const bool half = dt == CSA2_FP16;
    void (*kern)(Quant4Args) = any ? (half ? quantize_fp4_paged_any_kernel<true> : quantize_fp4_paged_any_kernel<false>)
                                   : (half ? quantize_fp4_paged_kernel<true> : quantize_fp4_paged_kernel<false>);
    CSA2_CUDA_CALL(launch_pdl(kern, sh.grid, sh.block, 0, stream_of(stream), a), "quantize_fp4_paged_kernel launch");
    CSA2_LAUNCH_CHECK("quantize_fp4_paged_kernel");
    return CSA2_OK;
}

extern "C" csa2_status csa2_dequantize_kv_fp4_paged(const int64_t *slots, int64_t T, int64_t n_blocks, int Hkv, int S, int D,
                                                    const uint8_t *k_codes, const uint8_t *v_codes, const uint8_t *k_scales,
                                                    const uint8_t *v_scales, csa2_dtype dt, void *k, void *v,
                                                    int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                                                    int64_t v_head_stride, uint32_t *err_flag, csa2_stream_t stream) {
    clear_error();
    const int64_t strides[4] = {k_token_stride, k_head_stride, v_token_stride, v_head_stride};
    const csa2_status st = check4("dequantize_fp4_paged", dt, T, Hkv, D, n_blocks, S, k, v, strides, slots, k_codes, v_codes,
                                  k_scales, v_scales, err_flag);
    if (st != CSA2_OK) return st;
    if (T == 0) return CSA2_OK;
    const Rows out[2] = {{k, T, Hkv, D, k_token_stride, k_head_stride}, {v, T, Hkv, D, v_token_stride, v_head_stride}};
    const int64_t plane = n_blocks * Hkv * S * (D / 2);
    for (const Rows &r : out) {
        CSA2_REQUIRE(r.apart(), "dequantize_fp4_paged: rows of an output share elements");
        bool over = meet(r.p, r.bytes(), slots, 8 * T) || meet(r.p, r.bytes(), err_flag, err_flag ? 4 : 0);
        for (const uint8_t *p : {k_codes, v_codes}) over = over || meet(r.p, r.bytes(), p, plane);
        for (const uint8_t *p : {k_scales, v_scales}) over = over || meet(r.p, r.bytes(), p, plane / 8);
        CSA2_REQUIRE(!over, "dequantize_fp4_paged: an output overlaps another argument");
    }
    CSA2_REQUIRE(!share(out[0], out[1]), "dequantize_fp4_paged: k and v share elements");
    const int tokens = kReadThreads / (D / 8);
    const int64_t blocks = (T + tokens - 1) / tokens * 2;           // T <= 2^30, tokens >= 4
    Read4Args a = {};
    a.codes[0] = k_codes, a.codes[1] = v_codes, a.scales[0] = k_scales, a.scales[1] = v_scales;
    a.x[0] = (uint16_t *)k, a.x[1] = (uint16_t *)v;
    a.token_stride[0] = k_token_stride, a.token_stride[1] = v_token_stride;
    a.head_stride[0] = k_head_stride, a.head_stride[1] = v_head_stride;
    a.slots = slots, a.T = T, a.n_slots = n_blocks * S, a.H = Hkv, a.S = S, a.err_flag = err_flag;
    a.shift = S == 16 ? 4 : (S == 32 ? 5 : (S == 64 ? 6 : 7));
    const bool half = dt == CSA2_FP16;
    void (*kern)(Read4Args) = D == 64 ? (half ? dequantize_fp4_paged_kernel<64, true> : dequantize_fp4_paged_kernel<64, false>)
                                      : (half ? dequantize_fp4_paged_kernel<128, true> : dequantize_fp4_paged_kernel<128, false>);
    CSA2_CUDA_CALL(launch_pdl(kern, dim3((unsigned)blocks), dim3(kReadThreads), 0, stream_of(stream), a),
                   "dequantize_fp4_paged_kernel launch");
    CSA2_LAUNCH_CHECK("dequantize_fp4_paged_kernel");
    return CSA2_OK;
}
