// csa2_rope_table and csa2_rope: rotary positions, the table of cosines and sines
// from (scaled) frequencies, and the rotation of query and key rows by it.
#include "fp4.cuh"

namespace csa2 {
namespace {

// ---- the table.  The angle of position p and pair i is p f_i radians.  At far
// positions it is many turns, of which only the fraction counts: f_i becomes a
// fraction of a turn in 64-bit fixed point once per thread, and its product with p
// wraps at whole turns by itself, with an error below p 2^-65 turns.  What is left of
// the nearest quarter turn becomes an fp32 angle of at most pi / 4 with all its leading
// bits, and the Taylor series around 0 end with its 9th and 10th power (the next terms
// are 2^-28 and 2^-31 of the results).
//
// Bound by the stores.  262144 positions of 64 pairs (134 MB): 20.0 us, a copy's rate (6.7 TB/s).  It is
// near what can be issued, too: 24.6 with the frequency converted in fp64, 21.9 with 64-bit arithmetic
// for the quarter and the rest, 21.4 with two positions in place of four in flight; 67 as fp64 angles
// through sinpi and cospi.  A thread keeps its pair, whose frequency it converts once, and steps over
// positions: four CTAs to an SM (8: 20.3 us) and four positions per thread at least: 4096 positions
// of 32 pairs 1.7 us in a graph (2.4 with one, 1.8 with eight; 5.5 in fp64).
constexpr uint64_t kTurnHigh = 0x28BE60DB9391054Aull, kTurnLow = 0x7F09D5F47D4D3770ull;      // 2^128 / (2 pi)
constexpr int kMostExp = 1023 + 20, kLeastExp = 1023 - 30;   // biased exponents: 2^20 radians per position, 2^-30

struct TableArgs {
    const double *freq;
    float2 *table;
    int64_t start, n_pos;
    int half;
    float amplitude;
};

// Turns of f radians modulo 1, in 2^-64, nearest, for kLeastExp <= exponent and |f| <= 2^20: its 53 bits
// times 128 of 1 / (2 pi), in integers (fp64 has a 64th of their rate).
__device__ __forceinline__ uint64_t turns_of(uint64_t bits) {
    const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | 1ull << 52;
    const int s = 1139 - (int)(bits >> 52 & 0x7FF);              // 96 .. 146: the product's bits below 2^-64 turns
    const uint64_t b0 = m * kTurnHigh, p1 = __umul64hi(m, kTurnLow) + b0, p2 = __umul64hi(m, kTurnHigh) + (p1 < b0);
    const uint64_t at = s < 128 ? p2 << (128 - s) | p1 >> (s - 64) : p2 >> (s - 128);
    const uint64_t half = s <= 128 ? p1 >> (s - 65) : p2 >> (s - 129);
    const uint64_t turns = at + (half & 1);
    return bits >> 63 ? 0 - turns : turns;
}

// Cosine and sine of phase 2^-64 turns.
__device__ __forceinline__ float2 cos_sin_of(uint64_t phase) {
    const uint32_t high = (uint32_t)(phase >> 32) + (1u << 29);  // its two leading bits: the nearest quarter
    const int32_t hi = (int32_t)((high & 0x3FFFFFFFu) - (1u << 29));                    // of the rest
    constexpr float UNIT = 3.14159265358979f * 0x1p-31f;         // radians of 2^-32 turns
    const float x = fmaf((float)hi, UNIT, (float)(uint32_t)phase * (UNIT * 0x1p-32f)), y = x * x;
    float s = fmaf(y, fmaf(y, fmaf(y, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6);
    float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f);
    s = fmaf(x * y, s, x);
    c = fmaf(y, c, 1.0f);
    const bool odd = high & 0x40000000u;
    const uint32_t u = __float_as_uint(odd ? s : c), v = __float_as_uint(odd ? c : s);
    return make_float2(__uint_as_float(u ^ ((high + 0x40000000u) & 0x80000000u)), __uint_as_float(v ^ (high & 0x80000000u)));
}

__global__ void __launch_bounds__(512) rope_table_kernel(TableArgs a) {
    pdl_wait();
    pdl_launch_dependents();
    const int i = threadIdx.x;
    const double f = a.freq[i];
    const uint64_t bits = (uint64_t)__double_as_longlong(f);
    const bool fine = (bits & 0x7FFFFFFFFFFFFFFFull) <= (uint64_t)kMostExp << 52;     // no NaN either
    const float amp = fine ? a.amplitude : __int_as_float(0x7FC00000);
    const int64_t n0 = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, ahead = (int64_t)gridDim.x * blockDim.y;
    float2 *out = a.table + n0 * a.half + i;
    if ((int)(bits >> 52 & 0x7FF) < kLeastExp) {                 // fixed point would cost it leading bits; its angles fit fp64
        for (int64_t n = n0; n < a.n_pos; n += ahead, out += ahead * a.half) {
            const double x = f * 0.3183098861837907 * (double)(a.start + n);
            *out = make_float2(amp * (float)cospi(x), amp * (float)sinpi(x));
        }
        return;
    }
    const uint64_t step = fine ? turns_of(bits) : 0;
    uint64_t phase = step * (uint64_t)(a.start + n0);
    const uint64_t phases = step * (uint64_t)ahead;
    const int64_t out_step = ahead * a.half;
#pragma unroll 4
    for (uint32_t n = (uint32_t)n0; n < (uint32_t)a.n_pos; n += (uint32_t)ahead, out += out_step, phase += phases) {      // n_pos <= 2^31
        const float2 v = cos_sin_of(phase);
        *out = make_float2(amp * v.x, amp * v.y);
    }
}

// ---- the rotation.  A thread takes 8 channels of a head (with the 8 that are their
// partners, in the layout of halves), holds their cosines and sines and walks over heads.
// Bound by memory: 16384 tokens of 32 + 8 heads of 128 (344 MB with the table's rows) take 52.6 us, 97 %
// of a copy's rate; in place only the rotated channels are touched.  55.6 with pairs side by side, whose threads have
// 8 channels of a head on their way where those of halves have 16; with 64 of the 128 channels rotated 58.5 in halves,
// where threads that only copy 8 walk beside those that turn 16, 55.0 side by side.
struct RotateArgs {
    const uint16_t *in[2];                   // q, k
    uint16_t *out[2];
    int64_t in_token[2], in_head[2], out_token[2], out_head[2];
    int heads[2], per;                       // heads; heads per thread
    int64_t T, n_pos;
    const int32_t *pos;
    const float *table;
    int pairs, first, turned;                // rotated pairs and first rotated channel of a head; units that rotate
    uint32_t shares;                         // threads' shares of a token's heads
    uint32_t *err_flag;
};

constexpr int kBatch = 2;                    // heads whose loads are in flight together (52.6 us as above; 1: 56.2, 4: slower too)

template <bool HALF, bool SPLIT>
__global__ void __launch_bounds__(128) rope_kernel(RotateArgs a) {
    constexpr int P = SPLIT ? 8 : 4;         // pairs of a thread
    pdl_wait();
    pdl_launch_dependents();
    // the blocks that share the heads of some tokens stand side by side, so that the table's rows are read once
    const uint32_t tokens = blockIdx.x / a.shares, share = blockIdx.x - tokens * a.shares;
    const int64_t t = (int64_t)tokens * blockDim.y + threadIdx.y;
    if (t >= a.T) return;
    const int64_t p = a.pos[t];
    if (p < 0 || p >= a.n_pos) {             // -1: a row without a token
        if (p != -1 && threadIdx.x == 0 && share == 0) flag_error(a.err_flag, CSA2_FLAG_BAD_INDEX);
        return;
    }
    const int u = threadIdx.x, H = a.heads[0] + a.heads[1];
    const bool turns = u < a.turned;
    int c0 = a.first + 8 * u, c1 = c0 + a.pairs;
    float2 cs[P];
    if (turns) {
        const float4 *row = reinterpret_cast<const float4 *>(a.table + 2 * (p * a.pairs + P * u));
#pragma unroll
        for (int i = 0; i < P / 2; ++i) {
            const float4 v = row[i];
            cs[2 * i] = make_float2(v.x, v.y), cs[2 * i + 1] = make_float2(v.z, v.w);
        }
    } else {                                 // a piece that is copied as it is
        c0 = 8 * (u - a.turned);
        if (c0 >= a.first) c0 += 2 * a.pairs;
        c1 = c0;
    }
    const int end = min(H, (int)(share + 1) * a.per);
    for (int h0 = share * a.per; h0 < end; h0 += kBatch) {
        uint4 x[kBatch], y[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int h = h0 + k, w = h >= a.heads[0];
            if (h >= end) continue;
            const uint16_t *src = (w ? a.in[1] : a.in[0]) + t * (w ? a.in_token[1] : a.in_token[0]) +
                                  (w ? h - a.heads[0] : h) * (w ? a.in_head[1] : a.in_head[0]);
            x[k] = *reinterpret_cast<const uint4 *>(src + c0);
            if (SPLIT && turns) y[k] = *reinterpret_cast<const uint4 *>(src + c1);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int h = h0 + k, w = h >= a.heads[0];
            if (h >= end) continue;
            uint16_t *dst = (w ? a.out[1] : a.out[0]) + t * (w ? a.out_token[1] : a.out_token[0]) +
                            (w ? h - a.heads[0] : h) * (w ? a.out_head[1] : a.out_head[0]);
            if (turns) {
                uint32_t *xw = reinterpret_cast<uint32_t *>(&x[k]), *yw = reinterpret_cast<uint32_t *>(&y[k]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = unpack16<HALF>(xw[i]);
                    if (SPLIT) {
                        const float2 z = unpack16<HALF>(yw[i]), r0 = rotate(v.x, z.x, cs[2 * i].x, cs[2 * i].y),
                                     r1 = rotate(v.y, z.y, cs[(2 * i + 1) % P].x, cs[(2 * i + 1) % P].y);
                        xw[i] = pack16<HALF>(r0.x, r1.x), yw[i] = pack16<HALF>(r0.y, r1.y);
                    } else {
                        const float2 r = rotate(v.x, v.y, cs[i].x, cs[i].y);
                        xw[i] = pack16<HALF>(r.x, r.y);
                    }
                }
                if (SPLIT) *reinterpret_cast<uint4 *>(dst + c1) = y[k];
            }
            *reinterpret_cast<uint4 *>(dst + c0) = x[k];
        }
    }
}

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" csa2_status csa2_rope_table(const double *inv_freq, int half, int64_t start, int64_t n_pos, float amplitude,
                                       float *cos_sin, csa2_stream_t stream) {
    clear_error();
    CSA2_REQUIRE(half >= 1 && half <= 512, "rope_table: half=%d not in [1, 512]", half);
    CSA2_REQUIRE(n_pos >= 0 && n_pos <= (1ll << 31), "rope_table: n_pos=%lld not in [0, 2^31]", (long long)n_pos);
    CSA2_REQUIRE(start >= 0 && start <= (1ll << 31), "rope_table: start=%lld not in [0, 2^31]", (long long)start);
    if (n_pos == 0) return CSA2_OK;
    CSA2_REQUIRE(inv_freq && cos_sin, "rope_table: null pointer");
    CSA2_REQUIRE(aligned(inv_freq, 8) && aligned(cos_sin, 8), "rope_table: inv_freq and cos_sin must be 8-byte aligned");
    const uintptr_t f0 = (uintptr_t)inv_freq, t0 = (uintptr_t)cos_sin;
    CSA2_REQUIRE(f0 + 8 * half <= t0 || t0 + 8 * n_pos * half <= f0, "rope_table: cos_sin overlaps inv_freq");
    const int rows = half >= 256 ? 1 : 256 / half;
    const int64_t want = (n_pos + 4 * rows - 1) / (4 * rows), most = (int64_t)num_sms() * 4;     // 4 positions per thread or more
    const TableArgs a = {inv_freq, (float2 *)cos_sin, start, n_pos, half, amplitude};
    CSA2_CUDA_CALL(launch_pdl(rope_table_kernel, dim3((unsigned)(want < most ? want : most)), dim3(half, rows), 0,
                              stream_of(stream), a),
                   "rope_table_kernel launch");
    CSA2_LAUNCH_CHECK("rope_table_kernel");
    return CSA2_OK;
}

extern "C" csa2_status csa2_rope(const void *q, void *q_out, int Hq, int64_t q_token_stride, int64_t q_head_stride,
                                 int64_t qo_token_stride, int64_t qo_head_stride, const void *k, void *k_out, int Hk,
                                 int64_t k_token_stride, int64_t k_head_stride, int64_t ko_token_stride,
                                 int64_t ko_head_stride, csa2_dtype dt, int64_t T, int D, const int32_t *pos,
                                 const float *cos_sin, int64_t n_pos, int rope_dim, int first, csa2_rope_layout layout,
                                 uint32_t *err_flag, csa2_stream_t stream) {
    clear_error();
    CSA2_REQUIRE(dt == CSA2_BF16 || dt == CSA2_FP16, "rope: rows must be bf16 or fp16");
    CSA2_REQUIRE(T >= 0 && T <= (1ll << 30), "rope: T=%lld not in [0, 2^30]", (long long)T);
    CSA2_REQUIRE(Hq >= 0 && Hk >= 0 && Hq <= 32768 && Hk <= 32767, "rope: Hq=%d, Hk=%d not in [0, 32768], [0, 32767]", Hq, Hk);
    CSA2_REQUIRE(D >= 16 && D <= 1024 && D % 8 == 0, "rope: D=%d must be a multiple of 8 in [16, 1024]", D);
    CSA2_REQUIRE(layout == CSA2_ROPE_INTERLEAVED || layout == CSA2_ROPE_HALF, "rope: layout=%d", (int)layout);
    CSA2_REQUIRE(rope_dim >= 16 && rope_dim <= D && rope_dim % 16 == 0, "rope: rope_dim=%d must be a multiple of 16 in [16, D]",
                 rope_dim);
    CSA2_REQUIRE(first >= 0 && first % 8 == 0 && first + rope_dim <= D, "rope: first=%d must be a multiple of 8 in [0, D - rope_dim]",
                 first);
    CSA2_REQUIRE(n_pos >= 1 && n_pos <= (1ll << 31), "rope: n_pos=%lld not in [1, 2^31]", (long long)n_pos);
    if (T == 0 || Hq + Hk == 0) return CSA2_OK;
    CSA2_REQUIRE(pos && cos_sin && (Hq == 0 || (q && q_out)) && (Hk == 0 || (k && k_out)), "rope: null pointer");
    CSA2_REQUIRE(aligned(pos, 4) && aligned(err_flag, 4) && aligned(cos_sin, 16),
                 "rope: pos and flag must be 4-byte aligned, cos_sin 16-byte");
    RotateArgs a = {{(const uint16_t *)q, (const uint16_t *)k}, {(uint16_t *)q_out, (uint16_t *)k_out},
                    {q_token_stride, k_token_stride}, {q_head_stride, k_head_stride}, {qo_token_stride, ko_token_stride},
                    {qo_head_stride, ko_head_stride}, {Hq, Hk}, 1, T, n_pos, pos, cos_sin, rope_dim / 2, first, 0, 1, err_flag};
    bool in_place = true;
    Rows in[2] = {}, out[2] = {};
    for (int i = 0; i < 2; ++i) {
        if (a.heads[i] == 0) continue;
        in[i] = {a.in[i], T, a.heads[i], D, a.in_token[i], a.in_head[i]};
        out[i] = {a.out[i], T, a.heads[i], D, a.out_token[i], a.out_head[i]};
        for (int64_t s : {a.in_token[i], a.in_head[i], a.out_token[i], a.out_head[i]})
            CSA2_REQUIRE(s >= 0 && s % 8 == 0 && s < (1ll << 31), "rope: strides must be multiples of 8 in [0, 2^31)");
        CSA2_REQUIRE(aligned(a.in[i], 16) && aligned(a.out[i], 16), "rope: rows must be 16-byte aligned");
        CSA2_REQUIRE(out[i].apart(), "rope: rows of an output share elements");
        const bool same = a.in[i] == a.out[i] && (T == 1 || a.in_token[i] == a.out_token[i]) &&
                          (a.heads[i] == 1 || a.in_head[i] == a.out_head[i]);
        CSA2_REQUIRE(same || !share(out[i], in[i]), "rope: an output overlaps its input");
        CSA2_REQUIRE(!meet(out[i].p, out[i].bytes(), pos, 4 * T) && !meet(out[i].p, out[i].bytes(), cos_sin, 4 * n_pos * rope_dim) &&
                         !meet(out[i].p, out[i].bytes(), err_flag, err_flag ? 4 : 0),
                     "rope: an output overlaps pos, cos_sin or the flag");
        in_place = in_place && same;
    }
    CSA2_REQUIRE(!share(out[0], out[1]), "rope: q_out and k_out share elements");
    CSA2_REQUIRE(!share(out[0], in[1]) && !share(out[1], in[0]), "rope: an output overlaps the other input");
    const int vectors = D / 8, turned = layout == CSA2_ROPE_HALF ? rope_dim / 16 : rope_dim / 8;
    const int units = in_place ? turned : turned + vectors - rope_dim / 8;
    a.turned = turned;
    const int rows = 128 / units, H = Hq + Hk;
    const int64_t blocks = (T + rows - 1) / rows;
    // Cosines and sines are loaded once for all heads of a thread, as many as leave work for every SM: 32
    // blocks each (16384 tokens as above 53.2 us; with 16 blocks 55.6, 8: 59.6, 64: 53.7, 128: 60.1).  Few
    // tokens, such as a decode step's, want every head on a thread of its own.
    int per = kBatch;
    while (per < H && blocks * ((H + 2 * per - 1) / (2 * per)) >= (int64_t)num_sms() * 32) per *= 2;
    if (blocks * ((H + per - 1) / per) < (int64_t)num_sms() * 4) per = 1;
    a.per = per;
    a.shares = (H + per - 1) / per;
    CSA2_REQUIRE(blocks * a.shares < (1ll << 31), "rope: T * (Hq + Hk) = %lld rows", (long long)(T * H));
    const bool half_type = dt == CSA2_FP16;
    void (*kern)(RotateArgs) = layout == CSA2_ROPE_HALF ? (half_type ? rope_kernel<true, true> : rope_kernel<false, true>)
                                                        : (half_type ? rope_kernel<true, false> : rope_kernel<false, false>);
    CSA2_CUDA_CALL(launch_pdl(kern, dim3((unsigned)(blocks * a.shares)), dim3(units, rows), 0, stream_of(stream), a), "rope_kernel launch");
    CSA2_LAUNCH_CHECK("rope_kernel");
    return CSA2_OK;
}
