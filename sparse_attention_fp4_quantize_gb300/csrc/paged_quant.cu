// csa2_quantize_kv_fp8_paged: bf16 / fp16 key and value rows -> E4M3 codes in
// the blocks of the paged cache, one power-of-two scale per (block, head).
//
// A run is the rows that the call brings to one block.  The scale of the block
// is the least power of two s with amax <= 448 s, not below the block's scale
// if it holds earlier rows.  Powers of two, because E4M3 is a floating-point
// format: x / s then only shifts the exponent, so a finer scale would move where
// values are rounded but not how finely (3 mantissa bits either way), and when a
// later row makes s grow by 2^k the stored codes are re-encoded exactly except
// for bits that fall below the subnormal step 2^-9 s.  Errors do not pile up
// over the S appends that a decoding request makes to a block.
//
// A CTA of four warps looks at a window of up to 64 rows for one head of K or V,
// with two loads per lane: a run begins where the block changes, and its length
// comes from ballots over the slots behind it.  Few runs (prompts) the warps take
// together, up to eight loads in flight per lane, whose values stay in registers
// from the maximum to the codes; many (decoding) they share out.  The largest
// magnitude is an integer maximum of the sign-less bit patterns (order-preserving
// for both formats).  A row's D codes are contiguous, a run's rows too, so loads
// and stores are 16 and 8 bytes per lane of full lines.
//
// Bound by memory for prompts, by latency (slots, old scale, rows) and the launch
// for decoding.  16384 tokens, 8 heads of 128, blocks of 64, K and V (94.5 MB):
// 22.0 us, 4.3 TB/s, where a copy takes 13.9; 25 us with a warp per run, which has to
// read its rows twice, 22.2 and 22.8 us with 8 and 6 CTAs per SM.  64 decoding
// requests 6 us, 1501 tokens of 37 requests (5 heads of 64, blocks of 16) 11 us, both
// less than the host takes for the call.
#include "common.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 4, kMostWindow = 64;

struct PagedQuantArgs {
    const uint16_t *x[2];            // k, v
    int64_t token_stride[2], head_stride[2];
    uint8_t *codes[2];
    float *scale[2];
    const int64_t *slots;
    int64_t T, n_slots;
    int H, S, shift, window;       // S = 1 << shift; rows per window
    uint32_t *err_flag;
};

__device__ __forceinline__ float2 unpack2(uint32_t w, bool half_type) {
    if (half_type) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Two fp32 -> two E4M3 bytes (lo in the low byte), nearest even, saturating.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Least power of two s >= 2^-126 with amax <= 448 s: 448 = 1.75 * 2^8, so its
// exponent is that of amax less 8, one more if amax's significand exceeds 1.75.
__device__ __forceinline__ float scale_of(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // biased exponent of s
    e = e < 1 ? 1 : e;
    return __uint_as_float((uint32_t)e << 23);
}

template <int D, bool HALF>
__global__ void __launch_bounds__(kWarps * 32, 7) quantize_fp8_paged_kernel(PagedQuantArgs a) {
    constexpr int LPR = D / 8;            // lanes per row: 8 channels each
    constexpr int RPW = 32 / LPR;         // rows per warp load
    constexpr uint32_t INF = HALF ? 0x7C00u : 0x7F80u;
    constexpr uint32_t ABS2 = 0x7FFF7FFFu, ALL = 0xFFFFFFFFu;
    __shared__ uint32_t s_top[2][2][kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x % (2 * a.H);          // (head, K or V)
    pdl_wait();
    pdl_launch_dependents();
    const int h = unit >> 1;
    const bool is_v = unit & 1;
    const uint16_t *x = (is_v ? a.x[1] : a.x[0]) + h * (is_v ? a.head_stride[1] : a.head_stride[0]) + (lane % LPR) * 8;
    const int64_t ts = is_v ? a.token_stride[1] : a.token_stride[0];
    uint8_t *codes = is_v ? a.codes[1] : a.codes[0];
    float *scales = is_v ? a.scale[1] : a.scale[0];
    const int64_t w0 = (int64_t)(blockIdx.x / (2 * a.H)) * a.window;

    // lane = rows lane, lane + 32 of the window: the slot, the one before it
    int64_t slot[2];
    uint64_t leads = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int64_t mine = w0 + 32 * k + lane;
        const bool in = 32 * k + lane < a.window && mine < a.T;
        slot[k] = in ? a.slots[mine] : -1;
        const int64_t prev = in && mine > 0 ? a.slots[mine - 1] : -1;
        const bool valid = slot[k] >= 0 && slot[k] < a.n_slots;
        const bool goes_on = valid && prev >= 0 && prev < a.n_slots && prev >> a.shift == slot[k] >> a.shift;
        if (unit == 0 && warp == 0 && ((slot[k] != -1 && !valid) || (goes_on && prev != slot[k] - 1)))
            flag_error(a.err_flag, CSA2_FLAG_BAD_SLOT);
        leads |= (uint64_t)__ballot_sync(ALL, valid && !goes_on) << (32 * k);
    }
    const bool together = __popcll(leads) < kWarps;
    const int parts = together ? kWarps : 1, part = together ? warp : 0;
    const int row0 = part * RPW + lane / LPR, step = parts * RPW;    // this lane's first row of a run, and on from there
    for (int turn = 0; leads; leads &= leads - 1, ++turn) {
        if (!together && turn % kWarps != warp) continue;
        const int lead = __ffsll(leads) - 1;
        const int64_t i = w0 + lead, s0 = __shfl_sync(ALL, lead < 32 ? slot[0] : slot[1], lead & 31), block = s0 >> a.shift;
        const int start = (int)(s0 & (a.S - 1));
        float *scale = scales + block * a.H + h;
        const float old = start > 0 ? *scale : 0.0f;
        int n = 0;                        // rows of the run
        for (const int most = a.S - start; n < most;) {
            const int k = n + lane;
            const bool same = k < most && i + k < a.T && a.slots[i + k] == s0 + k;
            const uint32_t ok = __ballot_sync(ALL, same);
            n += ok == ALL ? 32 : __ffs(~ok) - 1;
            if (ok != ALL) break;
        }
        // the warps' maximum
        auto of_all = [&](uint32_t v, int which) {
            v = __reduce_max_sync(ALL, v);
            if (together) {
                uint32_t (&t)[kWarps] = s_top[turn & 1][which];
                if (lane == 0) t[warp] = v;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < kWarps; ++w) v = max(v, t[w]);
            }
            return v;
        };
        uint4 v[8];
        auto load = [&](int r) {          // rows r, r + step, ...
#pragma unroll
            for (int q = 0; q < 8; ++q)
                v[q] = r + q * step < n ? *reinterpret_cast<const uint4 *>(x + (i + r + q * step) * ts) : make_uint4(0, 0, 0, 0);
        };
        uint32_t m2 = 0;                  // largest sign-less patterns of the even and odd channels
        for (int r = row0; r < n; r += 8 * step) {
            load(r);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                m2 = __vmaxu2(__vmaxu2(m2, __vmaxu2(v[q].x & ABS2, v[q].y & ABS2)), __vmaxu2(v[q].z & ABS2, v[q].w & ABS2));
        }
        uint32_t top = of_all(max(m2 & 0xFFFFu, m2 >> 16), 0);
        const bool bad = top >= INF;
        if (bad) {                        // infinities and NaN do not count
            uint32_t t = 0;
            for (int r = row0; r < n; r += step)
                for (int c = 0; c < 8; ++c) {
                    const uint32_t u = x[(i + r) * ts + c] & 0x7FFFu;
                    if (u < INF) t = max(t, u);
                }
            top = of_all(t, 1);
            if (lane == 0) flag_error(a.err_flag, CSA2_FLAG_NONFINITE);
        }
        const float need = scale_of(unpack2(top, HALF).x);
        uint8_t *dst = codes + ((block * a.H + h) * a.S + start) * (int64_t)D + (lane % LPR) * 8;
        float s = need;
        if (start > 0) {
            s = fmaxf(old, need);
            if (s != old) {               // re-encode the rows stored before
                const float ratio = old > 0.0f ? old / s : 0.0f;
                for (int r = row0 - start; r < 0; r += step) {
                    uint2 *p = reinterpret_cast<uint2 *>(dst + (int64_t)r * D);
                    uint2 c = *p;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t lo, hi;
                        e4m3x4_to_f16x2x2(q ? c.y : c.x, lo, hi);
                        const float2 f0 = unpack2(lo, true), f1 = unpack2(hi, true);
                        (q ? c.y : c.x) = to_e4m3x2(f0.x * ratio, f0.y * ratio) |
                                          (to_e4m3x2(f1.x * ratio, f1.y * ratio) << 16);
                    }
                    *p = c;
                }
            }
        }
        __syncwarp();                     // every lane, and behind of_all's barrier every warp, has read the old scale
        if (lane == 0 && part == 0) *scale = s;
        const float inv = 1.0f / s;       // exact: a power of two
        for (int r = row0; r < n; r += 8 * step) {
            if (n > 8 * step) load(r);    // else the values are at hand
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
                uint32_t c[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float2 f = unpack2(w[k], HALF);
                    if (bad) {
                        if (f.x != f.x) f.x = 0.0f;
                        if (f.y != f.y) f.y = 0.0f;
                    }
                    c[k] = to_e4m3x2(f.x * inv, f.y * inv);
                }
                if (r + q * step < n)
                    *reinterpret_cast<uint2 *>(dst + (int64_t)(r + q * step) * D) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
            }
        }
        __syncwarp();
    }
}

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" csa2_status csa2_quantize_kv_fp8_paged(const void *k, const void *v, csa2_dtype dt, int64_t T, int Hkv,
                                                  int D, int64_t k_token_stride, int64_t k_head_stride,
                                                  int64_t v_token_stride, int64_t v_head_stride, const int64_t *slots,
                                                  int64_t n_blocks, int S, uint8_t *k_codes, uint8_t *v_codes,
                                                  float *k_scale, float *v_scale, uint32_t *err_flag,
                                                  csa2_stream_t stream) {
    clear_error();
    CSA2_REQUIRE(dt == CSA2_BF16 || dt == CSA2_FP16, "quantize_paged: rows must be bf16 or fp16");
    CSA2_REQUIRE(T >= 0 && T <= (1ll << 30), "quantize_paged: T=%lld not in [0, 2^30]", (long long)T);
    CSA2_REQUIRE(Hkv >= 1 && Hkv <= 65536, "quantize_paged: Hkv=%d not in [1, 65536]", Hkv);
    CSA2_REQUIRE(n_blocks >= 0 && n_blocks < (1ll << 31), "quantize_paged: n_blocks=%lld", (long long)n_blocks);
    CSA2_REQUIRE(S == 16 || S == 32 || S == 64 || S == 128, "quantize_paged: S=%d not in {16, 32, 64, 128}", S);
    CSA2_REQUIRE(k_token_stride % 8 == 0 && k_head_stride % 8 == 0 && v_token_stride % 8 == 0 &&
                     v_head_stride % 8 == 0 && k_token_stride >= 0 && k_head_stride >= 0 && v_token_stride >= 0 &&
                     v_head_stride >= 0,
                 "quantize_paged: strides must be multiples of 8, not negative");
    if (D != 64 && D != 128) {
        set_error("quantize_paged: D=%d not in {64, 128}", D);
        return CSA2_ERR_UNSUPPORTED;
    }
    if (T == 0) return CSA2_OK;
    CSA2_REQUIRE(k && v && slots, "quantize_paged: null pointer");
    CSA2_REQUIRE((k_codes && v_codes && k_scale && v_scale) || n_blocks == 0, "quantize_paged: null pointer");
    CSA2_REQUIRE(aligned(k, 16) && aligned(v, 16), "quantize_paged: k and v must be 16-byte aligned");
    CSA2_REQUIRE(aligned(k_codes, 16) && aligned(v_codes, 16), "quantize_paged: codes must be 16-byte aligned");
    CSA2_REQUIRE(aligned(k_scale, 4) && aligned(v_scale, 4) && aligned(slots, 8) && aligned(err_flag, 4),
                 "quantize_paged: misaligned scales / slots / flag (4-, 8- and 4-byte aligned)");
    PagedQuantArgs a = {};
    a.x[0] = (const uint16_t *)k, a.x[1] = (const uint16_t *)v;
    a.token_stride[0] = k_token_stride, a.token_stride[1] = v_token_stride;
    a.head_stride[0] = k_head_stride, a.head_stride[1] = v_head_stride;
    a.codes[0] = k_codes, a.codes[1] = v_codes;
    a.scale[0] = k_scale, a.scale[1] = v_scale;
    a.slots = slots, a.T = T, a.n_slots = n_blocks * S, a.H = Hkv, a.S = S, a.err_flag = err_flag;
    a.shift = S == 16 ? 4 : (S == 32 ? 5 : (S == 64 ? 6 : 7));
    // as many CTAs as run at once (7 per SM), each with at least one row to look at
    const int64_t at_once = (int64_t)num_sms() * 7;
    const int64_t window = (T * 2 * Hkv + at_once - 1) / at_once;
    a.window = (int)(window < 1 ? 1 : (window > kMostWindow ? kMostWindow : window));
    const int64_t ctas = (T + a.window - 1) / a.window * 2 * Hkv;
    CSA2_REQUIRE(ctas < (1ll << 31), "quantize_paged: T * Hkv = %lld rows", (long long)(T * Hkv));
    void (*kern)(PagedQuantArgs);
    if (dt == CSA2_FP16) kern = D == 64 ? quantize_fp8_paged_kernel<64, true> : quantize_fp8_paged_kernel<128, true>;
    else kern = D == 64 ? quantize_fp8_paged_kernel<64, false> : quantize_fp8_paged_kernel<128, false>;
    CSA2_CUDA_CALL(launch_pdl(kern, dim3((unsigned)ctas), dim3(kWarps * 32), 0, stream_of(stream), a),
                   "quantize_fp8_paged_kernel launch");
    CSA2_LAUNCH_CHECK("quantize_fp8_paged_kernel");
    return CSA2_OK;
}
