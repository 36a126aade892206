// csa2_paged_attn_fp8: causal attention of a ragged batch over the paged 8-bit
// cache (E4M3 codes, one fp32 scale per block and KV head).
//
// The rows of a (request, KV head) are its new tokens times the G = Hq / Hkv
// query heads that share the KV head: row r is token r / G, head r % G, so a
// key read once serves all of them.  z_j = sm_scale * k_scale * (q . code_j)
// and out = sum_j P_j v_scale code_j / sum_j P_j with an online softmax in the
// log2 domain.
//
// Both products run on the warp tensor cores in f16 with fp32 accumulation.
// E4M3 codes are f16 values; q is scaled per row by a power of two into the
// f16 range.  The weight of a value is P_j * v_scale: v_scale differs from
// block to block, so each row keeps two references, the running maximum M of
// z and the running maximum Mv of z + log2(v_scale) (its exponent), and feeds
// P_j v_scale 2^(M - Mv) <= 2 to the product: no weight that matters is lost to
// f16's range, whatever the ratio of the scales.
#include "common.cuh"

namespace csa2 {
namespace {

constexpr int kAttnWarps = 4;

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
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
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

// A warp's share of the softmax over keys for 16 rows: lane (g, t) = (lane / 4,
// lane % 4) holds rows g and g + 8.  Fragment layouts are chosen so that every
// load of codes is contiguous: in q . k, lane t's part of the contraction is
// channels [t D/4, (t+1) D/4); in P v, lane g's output columns of the B operand
// are channels [g D/8, (g+1) D/8), so the accumulators of lane t are channels
// [t D/4, (t+1) D/4) of its two rows.
template <int D>
struct Tile {
    static constexpr int KS = D / 16;                // k-steps of q . k
    static constexpr int NT = D / 8;                 // n-tiles of P v
    uint32_t q[KS][4];
    float o[NT][4];
    float m[2], mv[2], l[2];                         // running maxima (log2), sum of P of this lane's keys

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        m[0] = m[1] = mv[0] = mv[1] = __int_as_float(0xff800000);
        l[0] = l[1] = 0.0f;
    }

    // 16 keys of one block: kc, vc point at their first code rows.  zf: logit
    // factor per row (with the block's k_scale); vis0..1: keys [lo, hi) of the
    // 16 that rows g, g + 8 see; stored: how many of the 16 are stored rows.
    __device__ __forceinline__ void keys16(const uint8_t *kc, const uint8_t *vc, const float (&zf)[2], float vs,
                                           const int (&lo)[2], const int (&hi)[2], int stored) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        constexpr int KW = D / 16;                   // words of a key row per lane
        uint32_t kw[2][KW];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int c = 0; c < KW / 4; ++c) {
                const uint4 v = *reinterpret_cast<const uint4 *>(kc + (8 * i + g) * D + t * (D / 4) + 16 * c);
                kw[i][4 * c] = v.x, kw[i][4 * c + 1] = v.y, kw[i][4 * c + 2] = v.z, kw[i][4 * c + 3] = v.w;
            }
        constexpr int VW = D / 32;                   // words of a value row per lane
        uint32_t vw[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int key = 2 * t + (i & 1) + 8 * (i >> 1);
            const uint8_t *p = vc + key * D + g * (D / 8);
            if constexpr (VW == 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(p);
                vw[i][0] = v.x, vw[i][1] = v.y, vw[i][2] = v.z, vw[i][3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                vw[i][0] = v.x, vw[i][1] = v.y;
            }
            if (key >= stored) {                     // not a stored row: whatever is there must not meet a zero weight
#pragma unroll
                for (int w = 0; w < VW; ++w) vw[i][w] = 0u;
            }
        }
        float s[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t b0, b1;
                e4m3x4_to_f16x2x2(kw[i][k], b0, b1);
                mma_f16_16816(s[i], q[k][0], q[k][1], q[k][2], q[k][3], b0, b1);
            }
        }
        const float NEG_INF = __int_as_float(0xff800000);
        const float ve = (float)((int)((__float_as_uint(vs) >> 23) & 0xFFu) - 127);
        uint32_t p[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float z[4], top = NEG_INF;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int key = 8 * i + 2 * t + c;
                    const float v = s[i][2 * r + c] * zf[r];
                    z[2 * i + c] = key >= lo[r] && key < hi[r] ? v : NEG_INF;
                    top = fmaxf(top, z[2 * i + c]);
                }
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const float m1 = fmaxf(m[r], top), mv1 = fmaxf(mv[r], top + ve);
            const float ref = m1 == NEG_INF ? 0.0f : m1, refv = mv1 == NEG_INF ? 0.0f : mv1;
            l[r] *= ex2(m[r] - ref);
            const float grow = ex2(mv[r] - refv);
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                o[j][2 * r] *= grow;
                o[j][2 * r + 1] *= grow;
            }
            m[r] = m1, mv[r] = mv1;
            const float f = fminf(vs * ex2(ref - refv), 1e38f);
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = ex2(z[i] - ref);
                l[r] += e;
                w[i] = z[i] == NEG_INF ? 0.0f : e * f;
            }
            p[0][r] = pack_f16(w[0], w[1]);
            p[1][r] = pack_f16(w[2], w[3]);
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
            // bytes of keys (2t, 2t+1) and (2t+8, 2t+9) interleaved: pairs along the keys
            const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), a1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
            const uint32_t c0 = __byte_perm(vw[2][w], vw[3][w], 0x5140), c1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
            uint32_t b0[4], b1[4];
            e4m3x4_to_f16x2x2(a0, b0[0], b0[1]);
            e4m3x4_to_f16x2x2(a1, b0[2], b0[3]);
            e4m3x4_to_f16x2x2(c0, b1[0], b1[1]);
            e4m3x4_to_f16x2x2(c1, b1[2], b1[3]);
#pragma unroll
            for (int x = 0; x < 4; ++x) mma_f16_16816(o[4 * w + x], p[0][0], p[0][1], p[1][0], p[1][1], b0[x], b1[x]);
        }
    }
};

template <int D, bool HALF>
__global__ void __launch_bounds__(kAttnWarps * 32) paged_attn_kernel(PagedAttnArgs a) {
    __shared__ float s_o[kAttnWarps][16][D + 4];
    __shared__ float s_st[kAttnWarps][16][3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int h = blockIdx.y;
    const float NEG_INF = __int_as_float(0xff800000);
    pdl_wait();
    pdl_launch_dependents();
    for (int b = blockIdx.z; b < a.B; b += gridDim.z) {
        const Request rq = request_of(a, b);
        const int rows = rq.n * a.G;
        for (int r0 = blockIdx.x * 16; r0 < rows; r0 += gridDim.x * 16) {
            Tile<D> tile;
            tile.clear();
            int pos[2], first[2];
            float zf[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = r0 + g + 8 * r;
                const bool real = row < rows;
                const int tok = real ? row / a.G : 0, hq = h * a.G + (real ? row - tok * a.G : 0);
                pos[r] = real ? rq.kv - rq.n + tok : -1;
                first[r] = a.window > 0 ? max(0, pos[r] - a.window + 1) : 0;
                const uint16_t *src = a.q + (rq.row0 + tok) * a.q_token_stride + hq * a.q_head_stride + t * (D / 4);
                uint32_t w[D / 8];
                float top = 0.0f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (real) v = *reinterpret_cast<const uint4 *>(src + 8 * c);
                    w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
                }
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const float2 f = unpack_in<HALF>(w[c]);
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                // largest magnitude to [2^14, 2^15); a row below 2^-100 keeps its factor's limit
                const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
                const float mul = HALF ? 1.0f : __uint_as_float((uint32_t)(127 + 14 - e) << 23);
                zf[r] = a.logit_scale / mul;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const float2 f0 = unpack_in<HALF>(w[2 * k]), f1 = unpack_in<HALF>(w[2 * k + 1]);
                    tile.q[k][r] = pack_f16(f0.x * mul, f0.y * mul);
                    tile.q[k][2 + r] = pack_f16(f1.x * mul, f1.y * mul);
                }
            }
            // keys that some row of the tile sees
            const int last_tok = (min(r0 + 16, rows) - 1) / a.G, first_tok = r0 / a.G;
            const int end = min(rq.kv, rq.kv - rq.n + last_tok + 1);
            int begin = 0;
            if (a.window > 0) begin = max(0, rq.kv - rq.n + first_tok - a.window + 1) & ~15;
            for (int j = begin + 16 * warp; j < end; j += 16 * kAttnWarps) {
                const int32_t block = a.table[b * a.table_stride + j / a.S];
                if (block < 0 || block >= a.n_blocks) {
                    if (lane == 0) flag_error(a.err_flag, CSA2_FLAG_BAD_INDEX);
                    continue;
                }
                const int64_t bh = (int64_t)block * a.Hkv + h;
                const float ks = a.k_scale[bh], vs = a.v_scale[bh];
                const int64_t at = (bh * a.S + j % a.S) * D;
                const float z[2] = {zf[0] * ks, zf[1] * ks};
                const int lo[2] = {first[0] - j, first[1] - j}, hi[2] = {pos[0] + 1 - j, pos[1] + 1 - j};
                tile.keys16(a.k_codes + at, a.v_codes + at, z, vs, lo, hi, rq.kv - j);
            }
            // the warps' shares meet in shared memory
            __syncthreads();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float l = tile.l[r];
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
                l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
                if (t == 0) {
                    s_st[warp][g + 8 * r][0] = tile.m[r];
                    s_st[warp][g + 8 * r][1] = tile.mv[r];
                    s_st[warp][g + 8 * r][2] = l;
                }
#pragma unroll
                for (int j = 0; j < D / 8; ++j) {
                    s_o[warp][g + 8 * r][t * (D / 4) + j] = tile.o[j][2 * r];
                    s_o[warp][g + 8 * r][t * (D / 4) + D / 8 + j] = tile.o[j][2 * r + 1];
                }
            }
            __syncthreads();
            const int row = r0 + tid / 8, part = tid % 8;   // 8 threads per row, D / 8 channels each
            if (row < rows) {
                float M = NEG_INF, l = 0.0f, f[kAttnWarps];
                for (int w = 0; w < kAttnWarps; ++w) M = fmaxf(M, s_st[w][tid / 8][0]);
                const float ref = M == NEG_INF ? 0.0f : M;
                for (int w = 0; w < kAttnWarps; ++w) {
                    l += s_st[w][tid / 8][2] * ex2(s_st[w][tid / 8][0] - ref);
                    f[w] = s_st[w][tid / 8][1] == NEG_INF ? 0.0f : exp2f(s_st[w][tid / 8][1] - ref);
                }
                const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
                const int tok = row / a.G, hq = h * a.G + row - tok * a.G;
                const int64_t o_row = (rq.row0 + tok) * a.Hq + hq;
                uint32_t w32[D / 16];
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    float x[2] = {0.0f, 0.0f};
                    for (int w = 0; w < kAttnWarps; ++w) {
                        x[0] += f[w] * s_o[w][tid / 8][part * (D / 8) + 2 * c];
                        x[1] += f[w] * s_o[w][tid / 8][part * (D / 8) + 2 * c + 1];
                    }
                    w32[c] = pack_out<HALF>(x[0] * inv, x[1] * inv);
                }
                uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + o_row * D + part * (D / 8));
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    reinterpret_cast<uint4 *>(dst)[c] = make_uint4(w32[4 * c], w32[4 * c + 1], w32[4 * c + 2], w32[4 * c + 3]);
                if (a.lse && part == 0)
                    a.lse[o_row] = l > 0.0f || l != l ? (M + log2f(l)) * 0.69314718055994531f : NEG_INF;
            }
        }
    }
}

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_paged_attn_workspace_bytes(int B, int64_t T, int Hq, int Hkv, int D, int max_new) {
    (void)B, (void)T, (void)Hq, (void)Hkv, (void)D, (void)max_new;
    return 0;
}

extern "C" csa2_status csa2_paged_attn_fp8(int B, int64_t T, int Hq, int Hkv, int D, csa2_dtype dt, const void *q,
                                           int64_t q_token_stride, int64_t q_head_stride, const uint8_t *k_codes,
                                           const uint8_t *v_codes, const float *k_scale, const float *v_scale,
                                           int64_t n_blocks, int S, const int32_t *block_table, int M,
                                           int64_t table_stride, const int32_t *kv_len, const int32_t *cu_len,
                                           int max_new, int window, float sm_scale, void *out, float *lse,
                                           uint32_t *err_flag, void *workspace, size_t ws_bytes,
                                           csa2_stream_t stream) {
    clear_error();
    CSA2_REQUIRE(dt == CSA2_BF16 || dt == CSA2_FP16, "paged_attn: q must be bf16 or fp16");
    CSA2_REQUIRE(B >= 0 && B <= 65536, "paged_attn: B=%d not in [0, 65536]", B);
    CSA2_REQUIRE(T >= 0 && T <= (1ll << 30), "paged_attn: T=%lld not in [0, 2^30]", (long long)T);
    CSA2_REQUIRE(Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && Hq <= 65536, "paged_attn: Hq=%d, Hkv=%d", Hq, Hkv);
    CSA2_REQUIRE(T * (Hq / Hkv) < (1ll << 31), "paged_attn: T * Hq / Hkv = %lld rows", (long long)(T * (Hq / Hkv)));
    CSA2_REQUIRE(S == 16 || S == 32 || S == 64 || S == 128, "paged_attn: S=%d not in {16, 32, 64, 128}", S);
    CSA2_REQUIRE(M >= 1 && (int64_t)M * S < (1ll << 31), "paged_attn: M=%d: need 1 <= M, M * S < 2^31", M);
    CSA2_REQUIRE(table_stride >= M, "paged_attn: table_stride=%lld < M=%d", (long long)table_stride, M);
    CSA2_REQUIRE(n_blocks >= 0 && n_blocks < (1ll << 31), "paged_attn: n_blocks=%lld", (long long)n_blocks);
    CSA2_REQUIRE(max_new >= 1, "paged_attn: max_new=%d < 1", max_new);
    CSA2_REQUIRE(window >= 0, "paged_attn: window=%d < 0", window);
    CSA2_REQUIRE(q_token_stride >= 0 && q_head_stride >= 0 && q_token_stride % 8 == 0 && q_head_stride % 8 == 0,
                 "paged_attn: q strides must be multiples of 8, not negative");
    if (D != 64 && D != 128) {
        set_error("paged_attn: D=%d not in {64, 128}", D);
        return CSA2_ERR_UNSUPPORTED;
    }
    if (B == 0 || T == 0) return CSA2_OK;
    CSA2_REQUIRE(q && out && block_table && kv_len && cu_len, "paged_attn: null pointer");
    CSA2_REQUIRE((k_codes && v_codes && k_scale && v_scale) || n_blocks == 0, "paged_attn: null pointer");
    CSA2_REQUIRE(aligned(q, 16) && aligned(out, 16) && aligned(k_codes, 16) && aligned(v_codes, 16),
                 "paged_attn: q, out and codes must be 16-byte aligned");
    const size_t need = csa2_paged_attn_workspace_bytes(B, T, Hq, Hkv, D, max_new);
    if (need > 0 && (!workspace || ws_bytes < need || !aligned(workspace, 16))) {
        set_error("paged_attn: workspace of %zu bytes (16-byte aligned) needed, %zu given", need, ws_bytes);
        return CSA2_ERR_WORKSPACE;
    }
    const PagedAttnArgs a = {B, Hq, Hkv, Hq / Hkv, S, M, window, T, n_blocks, table_stride, q_token_stride,
                             q_head_stride, (const uint16_t *)q, k_codes, v_codes, k_scale, v_scale, block_table,
                             kv_len, cu_len, sm_scale * 1.4426950408889634f, (uint16_t *)out, lse, err_flag};
    const int64_t tiles = ((int64_t)max_new * a.G + 15) / 16;
    const dim3 grid((unsigned)(tiles < (1 << 20) ? tiles : (1 << 20)), (unsigned)Hkv, (unsigned)(B < 65535 ? B : 65535));
    void (*kern)(PagedAttnArgs);
    if (dt == CSA2_FP16) kern = D == 64 ? paged_attn_kernel<64, true> : paged_attn_kernel<128, true>;
    else kern = D == 64 ? paged_attn_kernel<64, false> : paged_attn_kernel<128, false>;
    CSA2_CUDA_CALL(launch_pdl(kern, grid, dim3(kAttnWarps * 32), 0, stream_of(stream), a), "paged_attn_kernel launch");
    CSA2_LAUNCH_CHECK("paged_attn_kernel");
    return CSA2_OK;
}
