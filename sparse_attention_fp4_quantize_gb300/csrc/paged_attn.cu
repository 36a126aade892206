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
#include "paged_attn.cuh"

namespace csa2 {
namespace {

constexpr int kAttnWarps = 4;
constexpr int kTileKeys = kSplitKeys;   // keys per warp tile
constexpr int kStages = 2;          // tiles in flight per warp

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

struct StageMeta {
    float ks[2], vs[2];             // scales of the two 16-key halves
    int stored[2];                  // keys of each half that are there
};

// A warp's share of the softmax over keys for 16 MT rows: lane (g, t) =
// (lane / 4, lane % 4) holds rows g and g + 8 of each 16.  Fragment layouts are
// chosen so that every load of codes is contiguous: in q . k, lane t's part of
// the contraction is channels [t D/4, (t+1) D/4); in P v, lane g's output
// columns of the B operand are channels [g D/8, (g+1) D/8), so the accumulators
// of lane t are channels [t D/4, (t+1) D/4) of its rows.
template <int D, int MT>
struct Tile {
    static constexpr int KS = D / 16;                // k-steps of q . k
    static constexpr int NT = D / 8;                 // n-tiles of P v
    uint32_t q[MT][KS][4];
    float o[MT][NT][4];
    float m[2 * MT], mv[2 * MT], l[2 * MT];          // running maxima (log2), sum of P of this lane's keys

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.0f;
#pragma unroll
        for (int r = 0; r < 2 * MT; ++r) {
            m[r] = mv[r] = __int_as_float(0xff800000);
            l[r] = 0.0f;
        }
    }

    // 32 keys from shared memory (codes at kb, vb).  zf: logit factor per row; a
    // row sees keys [lo, hi) of the 32, as far as they are stored.
    __device__ __forceinline__ void keys32(uint32_t kb, uint32_t vb, const StageMeta &meta, const float (&zf)[2 * MT],
                                           const int (&lo)[2 * MT], const int (&hi)[2 * MT]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        constexpr uint32_t ALL = 0xFFFFFFFFu;
        const float NEG_INF = __int_as_float(0xff800000);
        float s[MT][4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t kw[D / 16];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const uint4 v = lds128(kb + chunk_at<D>(8 * i + g, t * (D / 64) + c));
                kw[4 * c] = v.x, kw[4 * c + 1] = v.y, kw[4 * c + 2] = v.z, kw[4 * c + 3] = v.w;
            }
#pragma unroll
            for (int x = 0; x < MT; ++x) s[x][i][0] = s[x][i][1] = s[x][i][2] = s[x][i][3] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t b0, b1;
                e4m3x4_to_f16x2x2(kw[k], b0, b1);
#pragma unroll
                for (int x = 0; x < MT; ++x)
                    mma_f16_16816(s[x][i], q[x][k][0], q[x][k][1], q[x][k][2], q[x][k][3], b0, b1);
            }
        }
        const float ve[2] = {(float)((int)((__float_as_uint(meta.vs[0]) >> 23) & 0xFFu) - 127),
                             (float)((int)((__float_as_uint(meta.vs[1]) >> 23) & 0xFFu) - 127)};
        uint32_t p[MT][4][2];
        float grow[2 * MT];
        bool grew = false;
#pragma unroll
        for (int r = 0; r < 2 * MT; ++r) {
            float z[8], top[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float f = zf[r] * meta.ks[u];
                const int end = min(hi[r], 16 * u + meta.stored[u]);
                top[u] = NEG_INF;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int key = 16 * u + 8 * i + 2 * t + c;
                        const float v = s[r / 2][2 * u + i][2 * (r & 1) + c] * f;
                        z[4 * u + 2 * i + c] = key >= lo[r] && key < end ? v : NEG_INF;
                        top[u] = fmaxf(top[u], z[4 * u + 2 * i + c]);
                    }
                top[u] = fmaxf(top[u], __shfl_xor_sync(ALL, top[u], 1));
                top[u] = fmaxf(top[u], __shfl_xor_sync(ALL, top[u], 2));
            }
            const float m1 = fmaxf(m[r], fmaxf(top[0], top[1]));
            const float mv1 = fmaxf(mv[r], fmaxf(top[0] + ve[0], top[1] + ve[1]));
            const float ref = m1 == NEG_INF ? 0.0f : m1, refv = mv1 == NEG_INF ? 0.0f : mv1;
            l[r] *= ex2(m[r] - ref);
            grow[r] = ex2(mv[r] - refv);
            grew |= mv1 != mv[r];
            m[r] = m1, mv[r] = mv1;
            const float g2 = ex2(ref - refv);
            float w[8];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float f = fminf(meta.vs[u] * g2, 1e38f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = ex2(z[4 * u + i] - ref);
                    l[r] += e;
                    w[4 * u + i] = z[4 * u + i] == NEG_INF ? 0.0f : e * f;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) p[r / 2][i][r & 1] = pack_f16(w[2 * i], w[2 * i + 1]);
        }
        if (__any_sync(ALL, grew)) {
#pragma unroll
            for (int x = 0; x < MT; ++x)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[x][j][0] *= grow[2 * x], o[x][j][1] *= grow[2 * x];
                    o[x][j][2] *= grow[2 * x + 1], o[x][j][3] *= grow[2 * x + 1];
                }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            constexpr int VW = D / 32;               // words of a value row per lane
            uint32_t vw[4][VW];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (D == 128) {
                    const uint4 v = lds128(vb + chunk_at<D>(16 * u + 2 * t + (i & 1) + 8 * (i >> 1), g));
                    vw[i][0] = v.x, vw[i][1] = v.y, vw[i][2] = v.z, vw[i][3] = v.w;
                } else {
                    // odd t reads its second key first: even and odd rows share a 128-byte line
                    const int key = 16 * u + 2 * t + ((i ^ t) & 1) + 8 * (i >> 1);
                    const uint2 v = lds64(vb + chunk_at<D>(key, g >> 1) + 8 * (g & 1));
                    vw[i][0] = v.x, vw[i][1] = v.y;
                }
            }
            if constexpr (D == 64) {
#pragma unroll
                for (int i = 0; i < 4; i += 2)
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        const uint32_t x = vw[i][w], y = vw[i + 1][w];
                        vw[i][w] = t & 1 ? y : x;
                        vw[i + 1][w] = t & 1 ? x : y;
                    }
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
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int x = 0; x < MT; ++x)
                        mma_f16_16816(o[x][4 * w + c], p[x][2 * u][0], p[x][2 * u][1], p[x][2 * u + 1][0],
                                      p[x][2 * u + 1][1], b0[c], b1[c]);
            }
        }
    }
};

template <int D, int MT>
constexpr int attn_smem() {
    constexpr int ring = kAttnWarps * kStages * 2 * kTileKeys * D, merge = kAttnWarps * 16 * (D + 4) * 4;
    return ring > merge ? ring : merge;
}

template <int D, int MT, bool HALF>
__global__ void __launch_bounds__(kAttnWarps * 32, MT == 1 ? 3 : 2) paged_attn_split_kernel(PagedAttnArgs a) {
    constexpr int R = 16 * MT;
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_st[kAttnWarps][16][3];
    __shared__ StageMeta s_meta[kAttnWarps][kStages];
    __shared__ int64_t s_sum[kAttnWarps], s_found[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const float NEG_INF = __int_as_float(0xff800000);
    pdl_wait();
    pdl_launch_dependents();
    using Work = SplitWork<R>;
    const Plan plan = plan_of<Work>(a, blockIdx.x, gridDim.x, kAttnWarps, s_sum, s_found);
    int64_t at = blockIdx.x * plan.share;
    const int64_t stop = min(plan.total, at + plan.share);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (kStages * 2 * kTileKeys * D);
    int64_t base = plan.base;
    for (int b = plan.b; at < stop && b < a.B; ++b) {
        const Request rq = request_of(a, b);
        const int64_t end = base + Work::tiles(a, rq);
        const int key0 = Work::first_key(a, rq), rows = rq.n * a.G;
        while (at < stop && at < end) {
            // segment: tiles [ta, tb) of one unit
            const Place pl = Work::place(a, rq, at - base);
            const int h = pl.h, r0 = pl.r0, ta = pl.tile, tb = (int)min((int64_t)pl.tiles, ta + (stop - at));
            at += tb - ta;

            Tile<D, MT> tile;
            tile.clear();
            int pos[2 * MT], first[2 * MT];
            float zf[2 * MT];
            // this warp's tiles are ta + warp + 4 i; lane holds (tile lane / 2, half lane % 2) of 16 of them
            const int count = tb - ta > warp ? (tb - ta - warp + kAttnWarps - 1) / kAttnWarps : 0;
            const int32_t *table = a.table + b * a.table_stride;
            auto entry = [&](int i) -> int32_t {     // block of this lane's half of the 16 tiles from i on
                const int key = key0 + (ta + warp + (i + (lane >> 1)) * kAttnWarps) * kTileKeys + 16 * (lane & 1);
                return i + (lane >> 1) < count && key < rq.kv ? table[key / a.S] : -1;
            };
            int32_t block = entry(0), block_next = entry(16);
            float ks = 0.0f, vs = 0.0f;
            auto scales = [&]() {
                const bool ok = block >= 0 && block < a.n_blocks;
                ks = ok ? a.k_scale[(int64_t)block * a.Hkv + h] : 0.0f;
                vs = ok ? a.v_scale[(int64_t)block * a.Hkv + h] : 0.0f;
            };
            scales();
            auto issue = [&](int i) {                // start the copy of this warp's tile i
                if (i < count) {
                    if (i && (i & 15) == 0) {
                        block = block_next;
                        block_next = entry(i + 16);
                        scales();
                    }
                    const int key = key0 + (ta + warp + i * kAttnWarps) * kTileKeys;
                    const uint32_t dst = ring + (i % kStages) * (2 * kTileKeys * D);
                    constexpr int CPR = D / 16, RPI = 32 / CPR;      // chunks per row, rows per instruction
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int who = 2 * (i & 15) + u;
                        const int32_t bl = __shfl_sync(ALL, block, who);
                        int stored = min(16, rq.kv - key - 16 * u);
                        if (bl < 0 || bl >= a.n_blocks) {
                            if (stored > 0 && lane == 0) flag_error(a.err_flag, CSA2_FLAG_BAD_INDEX);
                            stored = 0;
                        }
                        stored = max(stored, 0);
                        if (lane == who) {
                            StageMeta &m = s_meta[warp][i % kStages];
                            m.ks[u] = ks, m.vs[u] = vs, m.stored[u] = stored;
                        }
                        const int64_t off = stored ? (((int64_t)bl * a.Hkv + h) * a.S + (key + 16 * u) % a.S) * D : 0;
                        const int c = lane % CPR;
#pragma unroll
                        for (int x = 0; x < 16 / RPI; ++x) {
                            const int r = x * RPI + lane / CPR;
                            const uint32_t n = r < stored ? 16 : 0;          // rows that are not there read as zero
                            const int64_t src = off + (n ? r * D + c * 16 : 0);
                            const uint32_t to = dst + chunk_at<D>(16 * u + r, c);
                            cp_async16(to, a.k_codes + src, n);
                            cp_async16(to + kTileKeys * D, a.v_codes + src, n);
                        }
                    }
                }
                cp_async_commit();
            };
#pragma unroll
            for (int i = 0; i < kStages - 1; ++i) issue(i);

#pragma unroll
            for (int r = 0; r < 2 * MT; ++r) {
                const int row = r0 + 16 * (r / 2) + g + 8 * (r & 1);
                const bool real = row < rows;
                const int tok = real ? row / a.G : 0, hq = h * a.G + (real ? row - tok * a.G : 0);
                pos[r] = real ? max(-1, rq.kv - rq.n + tok) : -1;
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
                top = fmaxf(top, __shfl_xor_sync(ALL, top, 1));
                top = fmaxf(top, __shfl_xor_sync(ALL, top, 2));
                // largest magnitude to [2^14, 2^15); a row below 2^-100 keeps that factor
                const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
                const float mul = HALF ? 1.0f : __uint_as_float((uint32_t)(127 + 14 - e) << 23);
                zf[r] = a.logit_scale / mul;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const float2 f0 = unpack_in<HALF>(w[2 * k]), f1 = unpack_in<HALF>(w[2 * k + 1]);
                    tile.q[r / 2][k][r & 1] = pack_f16(f0.x * mul, f0.y * mul);
                    tile.q[r / 2][k][2 + (r & 1)] = pack_f16(f1.x * mul, f1.y * mul);
                }
            }
            for (int i = 0; i < count; ++i) {
                issue(i + kStages - 1);
                cp_async_wait<kStages - 1>();
                __syncwarp();
                const int key = key0 + (ta + warp + i * kAttnWarps) * kTileKeys;
                int lo[2 * MT], hi[2 * MT];
#pragma unroll
                for (int r = 0; r < 2 * MT; ++r) lo[r] = first[r] - key, hi[r] = pos[r] + 1 - key;
                const uint32_t kb = ring + (i % kStages) * (2 * kTileKeys * D);
                tile.keys32(kb, kb + kTileKeys * D, s_meta[warp][i % kStages], zf, lo, hi);
                __syncwarp();
            }
            cp_async_wait<0>();

            // the warps' shares meet in shared memory, 16 rows at a time
            const bool whole = ta == 0 && tb == pl.tiles;
            float *s_o = reinterpret_cast<float *>(smem);
            constexpr int LD = D + 4;
#pragma unroll
            for (int x = 0; x < MT; ++x) {
                __syncthreads();
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int r = 2 * x + y;
                    float l = tile.l[r];
                    l += __shfl_xor_sync(ALL, l, 1);
                    l += __shfl_xor_sync(ALL, l, 2);
                    if (t == 0) {
                        s_st[warp][g + 8 * y][0] = tile.m[r];
                        s_st[warp][g + 8 * y][1] = tile.mv[r];
                        s_st[warp][g + 8 * y][2] = l;
                    }
                    float *dst = s_o + (warp * 16 + g + 8 * y) * LD + t * (D / 4);
#pragma unroll
                    for (int j = 0; j < D / 8; j += 4) {
                        *reinterpret_cast<float4 *>(dst + j) = make_float4(tile.o[x][j][2 * y], tile.o[x][j + 1][2 * y],
                                                                           tile.o[x][j + 2][2 * y], tile.o[x][j + 3][2 * y]);
                        *reinterpret_cast<float4 *>(dst + D / 8 + j) =
                            make_float4(tile.o[x][j][2 * y + 1], tile.o[x][j + 1][2 * y + 1], tile.o[x][j + 2][2 * y + 1],
                                        tile.o[x][j + 3][2 * y + 1]);
                    }
                }
                __syncthreads();
                const int y = tid / 8, part = tid % 8, row = r0 + 16 * x + y;
                if (row < rows) {
                    float M = NEG_INF, MV = NEG_INF, l = 0.0f, o[D / 8];
#pragma unroll
                    for (int w = 0; w < kAttnWarps; ++w) {
                        M = fmaxf(M, s_st[w][y][0]);
                        MV = fmaxf(MV, s_st[w][y][1]);
                    }
                    const float ref = M == NEG_INF ? 0.0f : M, refv = MV == NEG_INF ? 0.0f : MV;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) o[c] = 0.0f;
#pragma unroll
                    for (int w = 0; w < kAttnWarps; ++w) {
                        l += s_st[w][y][2] * ex2(s_st[w][y][0] - ref);
                        const float f = ex2(s_st[w][y][1] - refv);
                        const float *src = s_o + (w * 16 + y) * LD + part * (D / 8);
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) o[c] += f * src[c];
                    }
                    if (whole) {
                        const float f = exp2f(refv - ref);
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) o[c] *= f;
                        const int tok = row / a.G;
                        store_row<D, HALF>(a, (rq.row0 + tok) * a.Hq + h * a.G + row - tok * a.G, part, o, M, l);
                    } else {
                        float *dst = a.partial + ((2 * (int64_t)blockIdx.x + (ta == 0)) * R + 16 * x + y) * LD;
#pragma unroll
                        for (int c = 0; c < D / 8; c += 4)
                            *reinterpret_cast<float4 *>(dst + part * (D / 8) + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                        if (part == 0) *reinterpret_cast<float4 *>(dst + D) = make_float4(M, MV, l, 0.0f);
                    }
                }
            }
            __syncthreads();
        }
        base = end;
    }
}

// Joins the partial results of a unit that several CTAs share: the unit that
// CTA c began and did not finish.  CTA c's part is slot 2 c + 1, those of the
// CTAs after it slots 2 c'.  A block takes JR rows of the unit; each of its four
// warps joins every fourth part of them, then the warps' results meet.
template <int D, bool HALF, typename Work, int JR>
__device__ __forceinline__ void join_unit(const PagedAttnArgs &a, const float *partial, int c, int ctas, int round, int y0,
                                          float (*s_o)[16][D + 4], int64_t *s_sum, int64_t *s_found) {
    constexpr int R = Work::ROWS, LD = D + 4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float NEG_INF = __int_as_float(0xff800000);
    const Plan plan = plan_of<Work>(a, c, ctas, round, s_sum, s_found);
    const int64_t t0 = c * plan.share, last = min(plan.total, t0 + plan.share) - 1;
    if (t0 >= plan.total || last + 1 == plan.total) return;
    int64_t base = plan.base;
    for (int b = plan.b; b < a.B; ++b) {             // the request of the CTA's last tile
        const Request rq = request_of(a, b);
        const int64_t end = base + Work::tiles(a, rq);
        if (last >= end) {
            base = end;
            continue;
        }
        const Place pl = Work::place(a, rq, last - base);
        const int64_t u0 = last - pl.tile, u1 = u0 + pl.tiles;
        if (u0 < t0 || u1 <= last + 1) return;       // begun by an earlier CTA, or finished by this one
        const int64_t c1 = (u1 - 1) / plan.share;    // the CTA with the unit's last tile
        const int rows = rq.n * a.G;
        constexpr int TPR = 32 / JR, CH = D / TPR;   // threads per row in a warp, channels per thread
        const int rr = lane / TPR, x0 = (lane % TPR) * CH, in_unit = y0 + rr;
        float M = NEG_INF, MV = NEG_INF, l = 0.0f, o[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) o[i] = 0.0f;
        if (pl.r0 + in_unit < rows) {
            for (int64_t x = c + warp; x <= c1; x += 4) {
                const float *src = partial + ((x == c ? 2 * x + 1 : 2 * x) * R + in_unit) * LD;
                const float4 st = *reinterpret_cast<const float4 *>(src + D);
                const float M1 = fmaxf(M, st.x), MV1 = fmaxf(MV, st.y);
                const float ref = M1 == NEG_INF ? 0.0f : M1, refv = MV1 == NEG_INF ? 0.0f : MV1;
                l = l * ex2(M - ref) + st.z * ex2(st.x - ref);
                const float f0 = ex2(MV - refv), f1 = ex2(st.y - refv);
#pragma unroll
                for (int i = 0; i < CH; i += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(src + x0 + i);
                    o[i] = o[i] * f0 + v.x * f1, o[i + 1] = o[i + 1] * f0 + v.y * f1;
                    o[i + 2] = o[i + 2] * f0 + v.z * f1, o[i + 3] = o[i + 3] * f0 + v.w * f1;
                }
                M = M1, MV = MV1;
            }
        }
#pragma unroll
        for (int i = 0; i < CH; ++i) s_o[warp][rr][x0 + i] = o[i];
        if (x0 == 0) s_o[warp][rr][D] = M, s_o[warp][rr][D + 1] = MV, s_o[warp][rr][D + 2] = l;
        __syncthreads();
        if (tid < JR * 8) {
            const int y = tid / 8, part = tid % 8, row = pl.r0 + y0 + y;
            if (row < rows) {
                float Ma = NEG_INF, MVa = NEG_INF, la = 0.0f, acc[D / 8];
                for (int w = 0; w < 4; ++w) Ma = fmaxf(Ma, s_o[w][y][D]), MVa = fmaxf(MVa, s_o[w][y][D + 1]);
                const float ref = Ma == NEG_INF ? 0.0f : Ma, refv = MVa == NEG_INF ? 0.0f : MVa;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) acc[i] = 0.0f;
                for (int w = 0; w < 4; ++w) {
                    la += s_o[w][y][D + 2] * ex2(s_o[w][y][D] - ref);
                    const float f = ex2(s_o[w][y][D + 1] - refv);
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) acc[i] += f * s_o[w][y][part * (D / 8) + i];
                }
                const float f = exp2f(refv - ref);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) acc[i] *= f;
                const int tok = row / a.G;
                store_row<D, HALF>(a, (rq.row0 + tok) * a.Hq + pl.h * a.G + row - tok * a.G, part, acc, Ma, la);
            }
        }
        return;
    }
}

// Blocks [0, 4 split_ctas) join the split kernel's units of 16 MT rows, 4 MT rows
// each; the others the tile kernel's of 256 rows, 16 rows each.
template <int D, int MT, bool HALF>
__global__ void __launch_bounds__(128) paged_attn_join_kernel(PagedAttnArgs a, int split_ctas, int tc_ctas) {
    __shared__ int64_t s_sum[4], s_found[2];
    __shared__ float s_o[4][16][D + 4];
    pdl_wait();
    pdl_launch_dependents();
    const int x = blockIdx.x, n = 4 * split_ctas;
    if (x < n)
        join_unit<D, HALF, SplitWork<16 * MT>, 4 * MT>(a, a.partial, x / 4, split_ctas, kAttnWarps, x % 4 * 4 * MT, s_o, s_sum,
                                                       s_found);
    else
        join_unit<D, HALF, TcWork, 16>(a, a.partial_tc, (x - n) / 16, tc_ctas, kTcRound, (x - n) % 16 * 16, s_o, s_sum,
                                       s_found);
}

template <int D, int MT, bool HALF>
cudaError_t launch_attn(const PagedAttnArgs &a, int split_ctas, int tc_ctas, cudaStream_t stream) {
    static bool done[64];
    constexpr int smem = attn_smem<D, MT>();
    cudaError_t e = cudaSuccess;
    if (split_ctas) {
        e = ensure_smem_limit((const void *)paged_attn_split_kernel<D, MT, HALF>, smem, done);
        if (e != cudaSuccess) return e;
        e = launch_pdl(paged_attn_split_kernel<D, MT, HALF>, dim3(split_ctas), dim3(kAttnWarps * 32), smem, stream, a);
        if (e != cudaSuccess) return e;
    }
    if (tc_ctas) {
        e = launch_paged_attn_tc(a, D, HALF, stream);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(paged_attn_join_kernel<D, MT, HALF>, dim3(4 * split_ctas + 16 * tc_ctas), dim3(128), 0, stream, a,
                      split_ctas, tc_ctas);
}

// Which kernels a call launches.  Rows of one request that share a KV head are
// G * max_new at most.  Up to 32 of them the split kernel takes every request (a
// row tile of 16, or of 32 that reads the keys once for all).  Beyond, requests
// of more than 16 rows go to the tile kernel; the split kernel then runs for
// the others, unless there is but one request.
struct Choice {
    int MT, split_ctas, tc_ctas, split_rows;
};
inline Choice choose(int B, int G, int max_new) {
    const int64_t rows = (int64_t)G * max_new;
    Choice c = {1, num_sms() * 3, 0, 0x7FFFFFFF};    // CTAs that run at once: three per SM, two with 32 rows
    if (rows > 32) {
        c.tc_ctas = paged_attn_tc_ctas();
        c.split_rows = B > 1 ? 16 : 0;
        if (B == 1) c.split_ctas = 0;
    } else if (rows > 16) {
        c.MT = 2;
        c.split_ctas = num_sms() * 2;
    }
    return c;
}
inline size_t split_partial_floats(const Choice &c, int D) { return (size_t)2 * c.split_ctas * 16 * c.MT * (D + 4); }

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_paged_attn_workspace_bytes(int B, int64_t T, int Hq, int Hkv, int D, int max_new) {
    if (B <= 0 || T <= 0 || Hkv <= 0 || Hq < Hkv || D <= 0 || max_new <= 0) return 0;
    const Choice c = choose(B, Hq / Hkv, max_new);
    return (split_partial_floats(c, D) + (size_t)2 * c.tc_ctas * kTcRows * (D + 4)) * sizeof(float);
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
    CSA2_REQUIRE(T * (Hq / Hkv) <= (1ll << 30), "paged_attn: T * Hq / Hkv = %lld rows", (long long)(T * (Hq / Hkv)));
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
    const Choice c = choose(B, Hq / Hkv, max_new);
    float *partial = (float *)workspace;
    const PagedAttnArgs a = {B, Hq, Hkv, Hq / Hkv, S, M, window < M * S ? window : 0, T, n_blocks, table_stride,
                             q_token_stride, q_head_stride, (const uint16_t *)q, k_codes, v_codes, k_scale, v_scale,
                             block_table, kv_len, cu_len, sm_scale * 1.4426950408889634f, (uint16_t *)out, lse, err_flag,
                             c.split_rows, partial, partial + split_partial_floats(c, D)};
    cudaError_t (*go)(const PagedAttnArgs &, int, int, cudaStream_t);
    if (dt == CSA2_FP16)
        go = D == 64 ? (c.MT == 1 ? launch_attn<64, 1, true> : launch_attn<64, 2, true>)
                     : (c.MT == 1 ? launch_attn<128, 1, true> : launch_attn<128, 2, true>);
    else
        go = D == 64 ? (c.MT == 1 ? launch_attn<64, 1, false> : launch_attn<64, 2, false>)
                     : (c.MT == 1 ? launch_attn<128, 1, false> : launch_attn<128, 2, false>);
    CSA2_CUDA_CALL(go(a, c.split_ctas, c.tc_ctas, stream_of(stream)), "paged_attn launch");
    CSA2_LAUNCH_CHECK("paged_attn kernels");
    return CSA2_OK;
}
