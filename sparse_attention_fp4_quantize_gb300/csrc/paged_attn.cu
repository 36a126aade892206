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
// P_j v_scale 2^(M - Mv) to the product, times 2^kUp (paged_attn.cuh) so that the many
// small weights of a long tail are not lost to f16's range.  Both references may lag
// behind the maxima as long as the weights stay below 65000, f16's end.  The weights are
// rounded to f16's 11 bits because the products' other operand, a code, has 4: sums and
// statistics stay in 32.
//
// Three kernels.  The split kernel (this file) takes rows as few as a decode step's,
// 8 or 16 to a tile, whose time is the reading of the cache; the tile kernel
// (paged_attn_tc.cu) prompts, whose time is the products; the join kernel adds up the
// parts of units that several CTAs shared.
//
// The split kernel, 64 requests of up to 16k tokens, 64 heads of 128 over 8 (1212 MB):
// 184 us with the join, 6.6 TB/s, a copy's rate 6.8.  3 of up to 131k (257 MB): 52 us,
// of which 10 are the launch, the first loads and the join.  48 with 5 new tokens in
// a window of 4096, 15 heads of 64 over 5 (108 MB): 36.5 us, of which 8 go by before the
// first tile (lengths, table, codes, each after the other), then latency: 1.8 warps per
// scheduler issue 0.35 instructions a cycle, and a key takes as many as with 128 channels
// but brings half the bytes.  One request of 1000 tokens: 8 us and 4.6 for the join.
#include "paged_attn.cuh"

namespace csa2 {
namespace {

constexpr int kAttnWarps = kSplitWarps;
constexpr int kHalf = 4096;             // bytes of a warp tile's keys, and of its values
template <int D>
constexpr int kTileKeys = kHalf / D;
constexpr int kStages = 2;              // tiles in flight per warp
// CTAs that an SM holds at once: two of 255 registers stream faster than three of
// 168 (64 requests of up to 16k tokens, 8 heads of 128: 192 against 202 us; 16 rows
// per tile, 19 of up to 32k: 60 against 88; 64 channels: 42 against 44.6), and two tiles
// in flight per warp faster than three (195 against 204).
constexpr int kSplitPerSm = 2;

__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

template <int D>
struct StageMeta {
    static constexpr int U = kTileKeys<D> / 16;
    float ks[U], vs[U], lg[U], rv[U];   // scales of the 16-key groups; log2 of 2^kUp v's, its reciprocal
    int stored[U];                  // keys of each group that are there
};

// 8 x 8 halves, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// A warp's share of the softmax over keys for 8 NT rows.  Both products are
// computed transposed, S^T = K . Q^T and O^T = V^T . P^T, with the keys and the
// channels on the 16 rows of an MMA and the query rows on its 8 columns: a decode
// step's rows (the heads of a group) are few, and 8 fill what 16 would leave half
// empty.  Lane (g, t) = (lane / 4, lane % 4).  The fragments are chosen so that
// every load of codes is contiguous:
//   S^T  A: keys g, g + 8; lane t's part of the contraction is channels
//        [t D/4, (t+1) D/4).  B: the same channels of query row g.
//        C: keys g, g + 8 of query rows 2 t, 2 t + 1.
//   P^T  C transposed 8 x 8 at a time (keys 2 t, 2 t + 1 of query row g).
//   O^T  A: channels of lane g are [g D/8, (g+1) D/8), interleaved by keys; C: those
//        channels of query rows 2 t, 2 t + 1.
template <int D, int NT>
struct Tile {
    static constexpr int KS = D / 16;                // k-steps of q . k
    static constexpr int MO = D / 16;                // 16-channel tiles of O^T
    static constexpr int U = kTileKeys<D> / 16;      // 16-key groups of a tile
    uint32_t q[NT][KS][2];
    float o[NT][MO][4];
    float m[NT][2], mv[NT][2], l[NT][2];             // rows 2 t, 2 t + 1: references (log2), sum of P of this lane's keys
    float back[NT][2], dmin, dmax;                   // 2^(mv - m); least and largest m - mv (-inf: a row without keys so far)

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int j = 0; j < MO; ++j) o[x][j][0] = o[x][j][1] = o[x][j][2] = o[x][j][3] = 0.0f;
            m[x][0] = m[x][1] = mv[x][0] = mv[x][1] = __int_as_float(0xff800000);
            l[x][0] = l[x][1] = back[x][0] = back[x][1] = 0.0f;
        }
        dmin = dmax = __int_as_float(0xff800000);
    }

    // Weights of a tile whose keys every row sees, with the references as they are:
    // one exponential per score and no maximum, P = 2^(s f + log2(2^kUp vs) - mv), and l
    // gains sum P / (2^kUp vs) 2^(mv - m).  False if a row's P may leave f16 or a scale is so
    // far from the others that P would not carry its keys' part of l.
    __device__ __forceinline__ bool weights(const float (&s)[NT][U][4], const StageMeta<D> &meta, const float (&zf)[NT][2],
                                            uint32_t (&p)[NT][U][2]) {
        float least = meta.lg[0], most = meta.lg[0];
#pragma unroll
        for (int u = 1; u < U; ++u) least = fminf(least, meta.lg[u]), most = fmaxf(most, meta.lg[u]);
        bool ok = dmin + least > -64.0f && dmax + most < 64.0f;
        if (!__all_sync(0xFFFFFFFFu, ok)) return false;
        float gain[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            float total[2] = {0.0f, 0.0f};
            gain[x][0] = gain[x][1] = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float e[2][2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float f = zf[x][r] * meta.ks[u], c = meta.lg[u] - mv[x][r];
                    e[r][0] = ex2(fmaf(s[x][u][r], f, c)), e[r][1] = ex2(fmaf(s[x][u][2 + r], f, c));
                    const float sum = e[r][0] + e[r][1];
                    total[r] += sum;
                    gain[x][r] = fmaf(sum, meta.rv[u], gain[x][r]);
                }
                p[x][u][0] = transpose8x8(pack_f16(e[0][0], e[1][0]));
                p[x][u][1] = transpose8x8(pack_f16(e[0][1], e[1][1]));
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                gain[x][r] *= back[x][r];
                ok = ok && total[r] < 65000.0f && gain[x][r] < 1e30f;        // (f16 ends at 65504)
            }
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) return false;
#pragma unroll
        for (int x = 0; x < NT; ++x) l[x][0] += gain[x][0], l[x][1] += gain[x][1];
        return true;
    }

    // A tile of keys from shared memory (codes at kb, vb), the first of them `key0`.  zf:
    // logit factor per row.  If masked, a row sees keys [seen.x, seen.y] as far as
    // they are stored; else all of them.
    __device__ __forceinline__ void keys(uint32_t kb, uint32_t vb, const StageMeta<D> &meta, const float (&zf)[NT][2], bool masked,
                                           int key0, const int2 *seen) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        constexpr uint32_t ALL = 0xFFFFFFFFu;
        const float NEG_INF = __int_as_float(0xff800000);
        float s[NT][U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t kw[2][D / 16];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const uint4 v = lds128(kb + chunk_at<D>(16 * u + 8 * h + g, t * (D / 64) + c));
                    kw[h][4 * c] = v.x, kw[h][4 * c + 1] = v.y, kw[h][4 * c + 2] = v.z, kw[h][4 * c + 3] = v.w;
                }
#pragma unroll
            for (int x = 0; x < NT; ++x) s[x][u][0] = s[x][u][1] = s[x][u][2] = s[x][u][3] = 0.0f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16x2x2(kw[0][k], a0, a2);
                e4m3x4_to_f16x2x2(kw[1][k], a1, a3);
#pragma unroll
                for (int x = 0; x < NT; ++x) mma_f16_16816(s[x][u], a0, a1, a2, a3, q[x][k][0], q[x][k][1]);
            }
        }
        uint32_t p[NT][U][2];
        if (masked || !weights(s, meta, zf, p)) {
            float grow[NT][2];
            bool grew = false;
            dmin = __int_as_float(0x7f800000), dmax = NEG_INF;
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                float w[2][2 * U];                       // [row][16 u + 8 h + g at 2 u + h]
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int2 sees = seen[8 * x + 2 * t + r];
                    float z[2 * U], tz = NEG_INF, tv = NEG_INF;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float f = zf[x][r] * meta.ks[u];
                        const float ve = (float)((int)((__float_as_uint(meta.vs[u]) >> 23) & 0xFFu) - 127);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int key = 16 * u + 8 * h + g;
                            float v = s[x][u][2 * h + r] * f;
                            if (masked && !(key0 + key >= sees.x && key0 + key <= sees.y && 8 * h + g < meta.stored[u])) v = NEG_INF;
                            z[2 * u + h] = v;
                            tz = fmaxf(tz, v);
                            tv = fmaxf(tv, v + ve);
                        }
                    }
                    // the row's keys are spread over the 8 lanes of equal t
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        tz = fmaxf(tz, __shfl_xor_sync(ALL, tz, d));
                        tv = fmaxf(tv, __shfl_xor_sync(ALL, tv, d));
                    }
                    const float m1 = fmaxf(m[x][r], tz), mv1 = fmaxf(mv[x][r], tv);
                    const float ref = m1 == NEG_INF ? 0.0f : m1, refv = mv1 == NEG_INF ? 0.0f : mv1;
                    float sum = l[x][r] * ex2(m[x][r] - ref);
                    grow[x][r] = ex2(mv[x][r] - refv);
                    grew |= mv1 != mv[x][r];
                    m[x][r] = m1, mv[x][r] = mv1;
                    const float g2 = ex2(0.5f * (ref - refv));          // 2^(m - mv) in two steps: it need not be an fp32 number
                    back[x][r] = ex2(refv - ref);
                    dmin = fminf(dmin, m1 == NEG_INF || mv1 == NEG_INF ? NEG_INF : m1 - mv1);
                    dmax = fmaxf(dmax, ref - refv);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float f = fminf(meta.vs[u] * g2 * g2, kMostWeight) * kUpFactor;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float e = ex2(z[2 * u + h] - ref);
                            sum += e;
                            w[r][2 * u + h] = z[2 * u + h] == NEG_INF ? 0.0f : e * f;
                        }
                    }
                    l[x][r] = sum;
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) p[x][u][h] = transpose8x8(pack_f16(w[0][2 * u + h], w[1][2 * u + h]));
            }
            if (__any_sync(ALL, grew)) {
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int j = 0; j < MO; ++j) {
                        o[x][j][0] *= grow[x][0], o[x][j][1] *= grow[x][1];
                        o[x][j][2] *= grow[x][0], o[x][j][3] *= grow[x][1];
                    }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
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
                        const uint32_t a = vw[i][w], b = vw[i + 1][w];
                        vw[i][w] = t & 1 ? b : a;
                        vw[i + 1][w] = t & 1 ? a : b;
                    }
            }
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                // bytes of keys (2t, 2t+1) and (2t+8, 2t+9) interleaved: pairs along the keys
                const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), a1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
                const uint32_t c0 = __byte_perm(vw[2][w], vw[3][w], 0x5140), c1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
                uint32_t lo4[4], hi4[4];             // channels 4 w .. 4 w + 3: the low keys, the high keys
                e4m3x4_to_f16x2x2(a0, lo4[0], lo4[1]);
                e4m3x4_to_f16x2x2(a1, lo4[2], lo4[3]);
                e4m3x4_to_f16x2x2(c0, hi4[0], hi4[1]);
                e4m3x4_to_f16x2x2(c1, hi4[2], hi4[3]);
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int x = 0; x < NT; ++x)
                        mma_f16_16816(o[x][2 * w + c], lo4[2 * c], lo4[2 * c + 1], hi4[2 * c], hi4[2 * c + 1], p[x][u][0], p[x][u][1]);
            }
        }
    }
};

template <int D, int NT>
constexpr int attn_smem() {
    constexpr int ring = kAttnWarps * kStages * 2 * kHalf, merge = kAttnWarps * 8 * (D + 4) * 4;
    return ring > merge ? ring : merge;
}

template <int D, int NT, bool HALF>
__global__ void __launch_bounds__(kAttnWarps * 32, kSplitPerSm) paged_attn_split_kernel(PagedAttnArgs a) {
    constexpr int R = 8 * NT;
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_st[kAttnWarps][8][3];
    __shared__ int2 s_seen[kAttnWarps][R];
    __shared__ StageMeta<D> s_meta[kAttnWarps][kStages];
    __shared__ int64_t s_sum[kAttnWarps], s_found[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const float NEG_INF = __int_as_float(0xff800000);
    pdl_wait();
    pdl_launch_dependents();
    using Work = SplitWork<R, kTileKeys<D>>;
    const Plan plan = plan_of<Work>(a, blockIdx.x, gridDim.x, kAttnWarps, s_sum, s_found);
    int64_t at = blockIdx.x * plan.share;
    const int64_t stop = min(plan.total, at + plan.share);
    if (tid == 0) a.join[blockIdx.x].last = -1;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (kStages * 2 * kHalf);
    int64_t base = plan.base;
    for (int b = plan.b; at < stop && b < a.B; ++b) {
        const Request rq = request_of(a, b);
        const int64_t end = base + Work::tiles(a, rq);
        const int low = Work::low_key(a, rq), key0 = Work::first_key(a, rq), rows = rq.n * a.G;
        while (at < stop && at < end) {
            // segment: tiles [ta, tb) of one unit
            const Place pl = Work::place(a, rq, at - base);
            const int64_t unit = at - pl.tile;       // its first place
            at = min(stop, unit + pl.tiles);
            const int h = pl.h, r0 = pl.r0, ta = max(0, pl.tile - kSplitCost), tb = (int)(at - unit) - kSplitCost;
            if (tb <= 0) continue;
            const bool first_part = ta == 0, whole = first_part && at == unit + pl.tiles;
            if (tid == 0 && first_part && !whole)
                a.join[blockIdx.x] = {rq.row0, h, r0, rows, (int)((unit + pl.tiles - 1) / plan.share), {0, 0}};

            // this warp's tiles are ta + warp + 4 i; lane holds (tile lane / U, 16-key group lane % U) of 32 / U of them
            constexpr int U = kTileKeys<D> / 16, BT = 32 / U;
            const int todo = min(tb, Work::real_tiles(a, rq)) - ta;
            const int count = todo > warp ? (todo - warp + kAttnWarps - 1) / kAttnWarps : 0;
            const int32_t *table = a.table + b * a.table_stride;
            auto key_of = [&](int i) { return key0 + (ta + warp + (i + lane / U) * kAttnWarps) * kTileKeys<D> + 16 * (lane % U); };
            // groups that end before every row's window are not read: their blocks may be another request's by now
            auto there = [&](int i) { return i + lane / U < count && key_of(i) < rq.kv && key_of(i) + 16 > low; };
            auto entry = [&](int i) -> int32_t { return there(i) ? table[key_of(i) / a.S] : -1; };   // block of this lane's group
            int32_t block = entry(0), block_next = entry(BT);
            // Q travels beside the chain of loads to the first codes: for a B operand row g,
            // channels [t D/4, (t+1) D/4)
            uint4 qv[NT][D / 32];
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                const int row = r0 + 8 * x + g;
                const bool real = row < rows;
                const int tok = real ? row / a.G : 0, hq = h * a.G + (real ? row - tok * a.G : 0);
                const uint16_t *src = a.q + (rq.row0 + tok) * a.q_token_stride + hq * a.q_head_stride + t * (D / 4);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) qv[x][c] = real ? *reinterpret_cast<const uint4 *>(src + 8 * c) : make_uint4(0, 0, 0, 0);
            }
            float ks = 0.0f, vs = 0.0f;
            int64_t off = -1;                        // code offset of the group's first row, -1: not there
            auto scales = [&](int i) {
                const bool ok = there(i) && block >= 0 && block < a.n_blocks;
                if (there(i) && !ok) flag_error(a.err_flag, CSA2_FLAG_BAD_INDEX);
                const int64_t bh = ok ? (int64_t)block * a.Hkv + h : 0;
                ks = ok ? a.k_scale[bh] : 0.0f;
                vs = ok ? a.v_scale[bh] : 0.0f;
                off = ok ? (bh * a.S + (key_of(i) & (a.S - 1))) * D : -1;
            };
            scales(0);
            auto issue = [&](int i) {                // start the copy of this warp's tile i
                if (i < count) {
                    if (i && i % BT == 0) {
                        block = block_next;
                        block_next = entry(i + BT);
                        scales(i);
                    }
                    const int key = key0 + (ta + warp + i * kAttnWarps) * kTileKeys<D>;
                    const uint32_t dst = ring + (i % kStages) * (2 * kHalf);
                    constexpr int CPR = D / 16, RPI = 32 / CPR;      // chunks per row, rows per instruction
                    const int c = lane % CPR, r1 = lane / CPR;
                    const uint32_t who = U * (i % BT);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int64_t from = __shfl_sync(ALL, off, who + u);
                        const int stored = from < 0 ? 0 : rq.kv - key - 16 * u;
                        const int64_t lane_at = (from < 0 ? 0 : from) + r1 * D + 16 * c;
                        const uint8_t *ksrc = a.k_codes + lane_at, *vsrc = a.v_codes + lane_at;
                        if (stored >= 16) {
#pragma unroll
                            for (int x = 0; x < 16 / RPI; ++x) {
                                const uint32_t to = dst + chunk_at<D>(16 * u + x * RPI + r1, c);
                                cp_async16(to, ksrc + x * RPI * D, 16);
                                cp_async16(to + kHalf, vsrc + x * RPI * D, 16);
                            }
                        } else {                     // rows that are not there read as zero
#pragma unroll
                            for (int x = 0; x < 16 / RPI; ++x) {
                                const bool there = x * RPI + r1 < stored;
                                const uint32_t to = dst + chunk_at<D>(16 * u + x * RPI + r1, c);
                                cp_async16(to, there ? (const void *)(ksrc + x * RPI * D) : a.q, there ? 16 : 0);
                                cp_async16(to + kHalf, there ? (const void *)(vsrc + x * RPI * D) : a.q, there ? 16 : 0);
                            }
                        }
                    }
                }
                cp_async_commit();
            };
            // The scales of tile i, a tile after they were asked for: the codes' copies do not wait for them.
            auto scales_of = [&](int i) {
                if (lane / U == i % BT) {
                    StageMeta<D> &m = s_meta[warp][i % kStages];
                    const int u = lane % U, key = key0 + (ta + warp + i * kAttnWarps) * kTileKeys<D>;
                    m.ks[u] = ks, m.vs[u] = vs, m.lg[u] = log_scale(vs), m.rv[u] = rcp(vs) * kDownFactor;
                    m.stored[u] = off < 0 ? 0 : min(16, rq.kv - key - 16 * u);
                }
            };
            static_assert(kStages == 2, "a tile's scales are kept until the next tile is asked for");
            issue(0);

            Tile<D, NT> tile;
            tile.clear();
            float zf[NT][2];
            int all_lo = 0, all_hi = 0x7FFFFFFF;     // keys that every real row of this lane sees
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                {
                    uint32_t w[D / 8];
                    float top = 0.0f;
#pragma unroll
                    for (int c = 0; c < D / 32; ++c)
                        w[4 * c] = qv[x][c].x, w[4 * c + 1] = qv[x][c].y, w[4 * c + 2] = qv[x][c].z, w[4 * c + 3] = qv[x][c].w;
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
                    const float f = a.logit_scale / mul;
                    zf[x][0] = __shfl_sync(ALL, f, 8 * t);
                    zf[x][1] = __shfl_sync(ALL, f, 8 * t + 4);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const float2 f0 = unpack_in<HALF>(w[2 * k]), f1 = unpack_in<HALF>(w[2 * k + 1]);
                        tile.q[x][k][0] = pack_f16(f0.x * mul, f0.y * mul);
                        tile.q[x][k][1] = pack_f16(f1.x * mul, f1.y * mul);
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {        // the lane's rows of S^T and O^T
                    const int row = r0 + 8 * x + 2 * t + r;
                    const bool real = row < rows;
                    // a row that is not there sees everything: it holds no other back, and is not stored
                    const int pos = real ? max(-1, rq.kv - rq.n + row / a.G) : 0x7FFFFFF0;
                    const int first = real && a.window > 0 ? max(0, pos - a.window + 1) : 0;
                    if (g == 0) s_seen[warp][8 * x + 2 * t + r] = make_int2(first, pos);
                    if (real) all_lo = max(all_lo, first), all_hi = min(all_hi, pos + 1);
                }
            }
            for (int i = 0; i < count; ++i) {
                scales_of(i);
                issue(i + 1);
                cp_async_wait<1>();
                __syncwarp();
                const int key = key0 + (ta + warp + i * kAttnWarps) * kTileKeys<D>;
                const uint32_t kb = ring + (i % kStages) * (2 * kHalf);
                const StageMeta<D> &meta = s_meta[warp][i % kStages];
                bool plain = key >= all_lo && key + kTileKeys<D> <= all_hi;
#pragma unroll
                for (int u = 0; u < U; ++u) plain = plain && meta.stored[u] == 16;
                tile.keys(kb, kb + kHalf, meta, zf, !__all_sync(ALL, plain), key, s_seen[warp]);
                __syncwarp();
            }
            cp_async_wait<0>();

            // the warps' shares meet in shared memory, 8 rows at a time
            float *s_o = reinterpret_cast<float *>(smem);
            constexpr int LD = D + 4;
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                __syncthreads();
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float l = tile.l[x][r];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(ALL, l, d);
                    if (g == 0) {
                        s_st[warp][2 * t + r][0] = tile.m[x][r];
                        s_st[warp][2 * t + r][1] = tile.mv[x][r];
                        s_st[warp][2 * t + r][2] = l;
                    }
                    float *dst = s_o + (warp * 8 + 2 * t + r) * LD + g * (D / 8);
#pragma unroll
                    for (int j = 0; j < D / 16; j += 2)
                        *reinterpret_cast<float4 *>(dst + 2 * j) = make_float4(tile.o[x][j][r], tile.o[x][j][2 + r],
                                                                               tile.o[x][j + 1][r], tile.o[x][j + 1][2 + r]);
                }
                __syncthreads();
                const int y = tid / 16, part = tid % 16, row = r0 + 8 * x + y;   // 16 threads per row, D / 16 channels each
                if (row < rows) {
                    float M = NEG_INF, MV = NEG_INF, l = 0.0f, o[D / 16];
#pragma unroll
                    for (int w = 0; w < kAttnWarps; ++w) {
                        M = fmaxf(M, s_st[w][y][0]);
                        MV = fmaxf(MV, s_st[w][y][1]);
                    }
                    const float ref = M == NEG_INF ? 0.0f : M, refv = MV == NEG_INF ? 0.0f : MV;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) o[c] = 0.0f;
#pragma unroll
                    for (int w = 0; w < kAttnWarps; ++w) {
                        l += s_st[w][y][2] * ex2(s_st[w][y][0] - ref);
                        const float f = ex2(s_st[w][y][1] - refv);
                        const float *src = s_o + (w * 8 + y) * LD + part * (D / 16);
#pragma unroll
                        for (int c = 0; c < D / 16; c += 4) {
                            const float4 v = *reinterpret_cast<const float4 *>(src + c);
                            o[c] += f * v.x, o[c + 1] += f * v.y, o[c + 2] += f * v.z, o[c + 3] += f * v.w;
                        }
                    }
                    if (whole) {
                        const int tok = row / a.G;
                        store_row<D, HALF, 16>(a, (rq.row0 + tok) * a.Hq + h * a.G + row - tok * a.G, part, o, exp2f(refv - ref), M, l);
                    } else {
                        float *dst = a.partial + ((2 * (int64_t)blockIdx.x + first_part) * R + 8 * x + y) * LD;
#pragma unroll
                        for (int c = 0; c < D / 16; c += 4)
                            *reinterpret_cast<float4 *>(dst + part * (D / 16) + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                        if (part == 0) *reinterpret_cast<float4 *>(dst + D) = make_float4(M, MV, l, 0.0f);
                    }
                }
            }
            __syncthreads();
        }
        base = end;
    }
}

// Joins the parts of the unit that CTA c began and did not finish.  A block takes
// 4 JR rows of the unit from y0 on if ROWS (few parts: each warp JR rows and all
// parts), else JR rows (many parts: each warp every fourth part, then the warps'
// results meet).  Four parts are loaded at a time.
template <int D, bool HALF, int R, int JR, bool ROWS>
__device__ __forceinline__ void join_unit(const PagedAttnArgs &a, const JoinUnit &unit, const float *partial, int c, int y0,
                                          float (*s_o)[JR][D + 4]) {
    constexpr int LD = D + 4, STEP = ROWS ? 1 : 4;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float NEG_INF = __int_as_float(0xff800000);
    const int c1 = unit.last, rows = unit.rows, r0 = unit.r0;
    if (c1 < 0 || r0 + y0 >= rows) return;
    constexpr int TPR = 32 / JR, CH = D / TPR;       // threads per row in a warp, channels per thread: 4 of every 4 TPR
    const int rr = lane / TPR, x0 = (lane % TPR) * 4, in_unit = y0 + (ROWS ? warp * JR : 0) + rr;
    float M = NEG_INF, MV = NEG_INF, l = 0.0f, o[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) o[i] = 0.0f;
    if (r0 + in_unit < rows) {
        for (int x = c + (ROWS ? 0 : warp); x <= c1; x += 4 * STEP) {
            float4 st[4], v[4][CH / 4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int y = x + k * STEP;
                const float *src = partial + ((int64_t)(y == c ? 2 * y + 1 : 2 * y) * R + in_unit) * LD;
                st[k] = y <= c1 ? *reinterpret_cast<const float4 *>(src + D) : make_float4(NEG_INF, NEG_INF, 0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < CH / 4; ++i)
                    v[k][i] = y <= c1 ? *reinterpret_cast<const float4 *>(src + x0 + 4 * TPR * i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            const float M1 = fmaxf(fmaxf(fmaxf(M, st[0].x), fmaxf(st[1].x, st[2].x)), st[3].x);
            const float MV1 = fmaxf(fmaxf(fmaxf(MV, st[0].y), fmaxf(st[1].y, st[2].y)), st[3].y);
            const float ref = M1 == NEG_INF ? 0.0f : M1, refv = MV1 == NEG_INF ? 0.0f : MV1, f0 = ex2(MV - refv);
            l *= ex2(M - ref);
#pragma unroll
            for (int i = 0; i < CH; ++i) o[i] *= f0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                l += st[k].z * ex2(st[k].x - ref);
                const float f = ex2(st[k].y - refv);
#pragma unroll
                for (int i = 0; i < CH / 4; ++i) {
                    o[4 * i] += v[k][i].x * f, o[4 * i + 1] += v[k][i].y * f;
                    o[4 * i + 2] += v[k][i].z * f, o[4 * i + 3] += v[k][i].w * f;
                }
            }
            M = M1, MV = MV1;
        }
    }
    // the rows, whole, through shared memory: of all warps, or of this one
#pragma unroll
    for (int i = 0; i < CH / 4; ++i)
        *reinterpret_cast<float4 *>(&s_o[warp][rr][x0 + 4 * TPR * i]) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    if (x0 == 0) s_o[warp][rr][D] = M, s_o[warp][rr][D + 1] = MV, s_o[warp][rr][D + 2] = l;
    __syncthreads();
    constexpr int N = ROWS ? 4 * JR : JR;            // rows of the block, 8 threads each
    for (int u = tid; u < N * 8; u += 128) {
        const int y = u / 8, part = u % 8, row = r0 + y0 + y;
        if (row >= rows) continue;
        float Ma = NEG_INF, MVa = NEG_INF, la = 0.0f, acc[D / 8];
        constexpr int W = ROWS ? 1 : 4;
        const int w0 = ROWS ? y / JR : 0, yy = ROWS ? y % JR : y;
#pragma unroll
        for (int w = 0; w < W; ++w) Ma = fmaxf(Ma, s_o[w0 + w][yy][D]), MVa = fmaxf(MVa, s_o[w0 + w][yy][D + 1]);
        const float ref = Ma == NEG_INF ? 0.0f : Ma, refv = MVa == NEG_INF ? 0.0f : MVa;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            la += s_o[w0 + w][yy][D + 2] * ex2(s_o[w0 + w][yy][D] - ref);
            const float f = ex2(s_o[w0 + w][yy][D + 1] - refv);
#pragma unroll
            for (int i = 0; i < D / 8; ++i) acc[i] += f * s_o[w0 + w][yy][part * (D / 8) + i];
        }
        const int tok = row / a.G;
        store_row<D, HALF, 8>(a, (unit.row0 + tok) * a.Hq + unit.h * a.G + row - tok * a.G, part, acc, exp2f(refv - ref), Ma, la);
    }
}

// The first blocks join the split kernel's units of 8 NT rows, 4 rows each; the
// others the tile kernel's of 256 rows, 16 rows each.
template <int D, int NT, bool HALF>
__global__ void __launch_bounds__(128) paged_attn_join_kernel(PagedAttnArgs a, int split_ctas, int tc_ctas) {
    constexpr int JR = 4, JB = 8 * NT / JR;                    // rows per block, blocks per unit
    __shared__ float s_o[4][4][D + 4];
    pdl_wait();
    pdl_launch_dependents();
    const int x = blockIdx.x, n = JB * split_ctas;
    if (x < n)
        join_unit<D, HALF, 8 * NT, JR, false>(a, a.join[x / JB], a.partial, x / JB, x % JB * JR,
                                              reinterpret_cast<float (*)[JR][D + 4]>(s_o));
    else
        join_unit<D, HALF, kTcRows, 4, true>(a, a.join_tc[(x - n) / 16], a.partial_tc, (x - n) / 16, (x - n) % 16 * 16,
                                             reinterpret_cast<float (*)[4][D + 4]>(s_o));
}

template <int D, int NT, bool HALF>
cudaError_t launch_attn(const PagedAttnArgs &a, int split_ctas, int tc_ctas, cudaStream_t stream) {
    static bool done[64];
    constexpr int smem = attn_smem<D, NT>();
    cudaError_t e = cudaSuccess;
    // Neither kernel uses the other's results, but each waits for the one before it: what
    // was written before both is visible to a grid only once it has waited itself.  The
    // split kernel first: a mixed batch of 17 took 217 us, 221 the other way round.
    if (split_ctas) {
        e = ensure_smem_limit((const void *)paged_attn_split_kernel<D, NT, HALF>, smem, done);
        if (e != cudaSuccess) return e;
        e = launch_pdl(paged_attn_split_kernel<D, NT, HALF>, dim3(split_ctas), dim3(kAttnWarps * 32), smem, stream, a);
        if (e != cudaSuccess) return e;
    }
    if (tc_ctas) {
        e = launch_paged_attn_tc(a, D, HALF, stream);
        if (e != cudaSuccess) return e;
    }
    constexpr int JB = 2 * NT;
    return launch_pdl(paged_attn_join_kernel<D, NT, HALF>, dim3(JB * split_ctas + 16 * tc_ctas), dim3(128), 0, stream, a,
                      split_ctas, tc_ctas);
}

template <int D, bool HALF>
cudaError_t launch_attn_nt(int NT, const PagedAttnArgs &a, int split_ctas, int tc_ctas, cudaStream_t stream) {
    return NT == 1 ? launch_attn<D, 1, HALF>(a, split_ctas, tc_ctas, stream)
                   : launch_attn<D, 2, HALF>(a, split_ctas, tc_ctas, stream);
}

// Which kernels a call launches.  Rows of one request that share a KV head are
// G * max_new at most.  Up to 32 of them the split kernel takes every request, in
// row tiles of 8 or 16 that each read the keys.  Beyond, requests with more rows
// than a single token needs (8, or 32 if that is more than 8) go to the tile kernel;
// the split kernel then runs for the others, if there can be any.  24 requests of up
// to 16000 tokens, 8 KV heads of 128 (of 64), split kernel and tile kernel: 16 rows
// 87 and 181 us (54 and 163), 32 rows 149 and 182 (94 and 163), 64 rows 282 and 185
// (175 and 164); of up to 2000 tokens 28 and 48, 40 and 50, 64 and 51.
constexpr int kSplitRows = 32;
struct Choice {
    int NT, split_ctas, tc_ctas, split_rows;
};
inline Choice choose(int B, int G, int max_new) {
    const int64_t rows = (int64_t)G * max_new;
    Choice c = {(rows <= kSplitRows ? rows : G) <= 8 ? 1 : 2, 0, 0, 0x7FFFFFFF};
    if (rows > kSplitRows) {
        c.tc_ctas = paged_attn_tc_ctas();
        c.split_rows = B == 1 || G > kSplitRows ? 0 : (c.NT == 1 ? 8 : kSplitRows);
    }
    if (c.split_rows) c.split_ctas = num_sms() * kSplitPerSm;
    return c;
}
inline size_t split_partial_floats(const Choice &c, int D) { return (size_t)2 * c.split_ctas * 8 * c.NT * (D + 4); }

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_paged_attn_workspace_bytes(int B, int64_t T, int Hq, int Hkv, int D, int max_new) {
    if (B <= 0 || T <= 0 || Hkv <= 0 || Hq < Hkv || D <= 0 || max_new <= 0) return 0;
    const Choice c = choose(B, Hq / Hkv, max_new);
    return (c.split_ctas + c.tc_ctas) * sizeof(JoinUnit) +
           (split_partial_floats(c, D) + (size_t)2 * c.tc_ctas * kTcRows * (D + 4)) * sizeof(float);
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
    CSA2_REQUIRE(M >= 1 && (int64_t)M * S <= (1ll << 30), "paged_attn: M=%d: need 1 <= M, M * S <= 2^30", M);
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
    CSA2_REQUIRE(aligned(k_scale, 4) && aligned(v_scale, 4) && aligned(block_table, 4) && aligned(kv_len, 4) &&
                     aligned(cu_len, 4) && aligned(lse, 4) && aligned(err_flag, 4),
                 "paged_attn: scales, table, lengths, lse and flag must be 4-byte aligned");
    const size_t need = csa2_paged_attn_workspace_bytes(B, T, Hq, Hkv, D, max_new);
    if (need > 0 && (!workspace || ws_bytes < need || !aligned(workspace, 16))) {
        set_error("paged_attn: workspace of %zu bytes (16-byte aligned) needed, %zu given", need, ws_bytes);
        return CSA2_ERR_WORKSPACE;
    }
    const Choice c = choose(B, Hq / Hkv, max_new);
    JoinUnit *join = (JoinUnit *)workspace;
    float *partial = (float *)(join + c.split_ctas + c.tc_ctas);
    const PagedAttnArgs a = {B, Hq, Hkv, Hq / Hkv, S, M, window < M * S ? window : 0, T, n_blocks, table_stride,
                             q_token_stride, q_head_stride, (const uint16_t *)q, k_codes, v_codes, k_scale, v_scale,
                             block_table, kv_len, cu_len, sm_scale * 1.4426950408889634f, (uint16_t *)out, lse, err_flag,
                             c.split_rows, join, join + c.split_ctas, partial, partial + split_partial_floats(c, D)};
    auto go = dt == CSA2_FP16 ? (D == 64 ? launch_attn_nt<64, true> : launch_attn_nt<128, true>)
                              : (D == 64 ? launch_attn_nt<64, false> : launch_attn_nt<128, false>);
    CSA2_CUDA_CALL(go(c.NT, a, c.split_ctas, c.tc_ctas, stream_of(stream)), "paged_attn launch");
    CSA2_LAUNCH_CHECK("paged_attn kernels");
    return CSA2_OK;
}
