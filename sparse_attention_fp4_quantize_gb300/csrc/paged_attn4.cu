// csa2_paged_attn_fp4: causal attention of a ragged batch over the paged 4-bit
// cache (E2M1 codes, one E4M3 scale per token, KV head and 16 channels).
//
// Rows, units, the line of work and the join are those of the 8-bit cache
// (paged_attn.cu).  A key or value is code * scale, a number of at most 6 significant
// bits between 2^-10 and 2688, so exact in f16: both products run on the warp tensor
// cores in f16 with fp32 accumulation, and unlike there no scale is left for the scores
// or the weights.  One reference M per row, the running maximum of its scores in the
// log2 domain; weights P = 2^(z - M + kUp), rounded to f16's 11 bits for the product,
// their sum in fp32 before that.  M may lag behind the maximum as long as the weights
// stay below f16's end.
//
// The split kernel (this file) has a warp walk over tiles of 64 keys (few_keys4: or 32).  64 requests of up to
// 16k tokens, 64 heads of 128 over 8 (687 MB): 127 us with the join, 5.4 TB/s, a copy's rate
// 6.8; with its loads alone 110.  What it lacks are instructions' slots: of the 289 that a warp
// issues per 16 keys 128 turn codes into f16 and apply the scales, the schedulers issue 0.6 a cycle
// with 3 warps each, the codes' pipe is busy for 54 % and the tensor cores for 27.  CTAs of an SM end
// 7 us apart, but shares that make up for it (5 to 15 % more for the first) only slow the last ones'
// keys down: 131 to 141 us.  48 requests with 5 new tokens in a window of 4096, 15 heads of 64
// over 5 (61 MB): 33 us, of which 5 go by before the first tile (lengths, table, codes, each after
// the other) and 3 in the join; the loads alone take 20.  One request of 1000 tokens: 8.2 us in a
// graph.
#include "fp4.cuh"
#include "paged_attn.cuh"

namespace csa2 {
namespace {

constexpr int kWarps4 = kSplitWarps;
// CTAs that an SM holds at once: 16 rows of 128 channels need the registers of two (24
// requests of up to 16k tokens, 8 heads, 16 rows each: 77 us, 84 with three), others run
// fastest with three (8 rows of 128 channels, 64 requests: 130 us, 141 with two, 148 with four;
// of 64 channels 82, 91 with two).
constexpr int per_sm4(int D, int NT) { return D == 128 && NT == 2 ? 2 : 3; }
// Tiles that a unit's fixed cost counts as (64 requests as above 136 us, 137 with 4, 141 with 16; in a
// window 38.7, 39.3 and 41.2, as measured then).
constexpr int kCost4 = 8;
template <int D, int LGK>
struct Stage4 {                         // a tile in shared memory: codes and scales of its keys and of its values
    static constexpr int KEYS = 1 << LGK;                    // of a warp's tile
    static constexpr int CODES = KEYS * D / 2, SCALES = KEYS * D / 16;
    static constexpr int K = 0, V = CODES, KS = 2 * CODES, VS = KS + SCALES, BYTES = VS + SCALES;
    static constexpr int N = 2;                              // of them per warp
};
constexpr float kMostP4 = 65000.0f;     // bound of a row's weights in a tile (f16 ends at 65504)
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
// 8 x 8 halves, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Row i of S^T, which is place i of P V's contraction, is key key_at(i) of its 16: the
// four keys that the lanes of a quarter read together lie next to one another, so that
// with the staged chunks' order (chunk4_at) every load of codes meets a bank once.
__device__ __forceinline__ int key_at(int i) { return (i & 8) + (i & 1 ? 7 - ((i & 7) >> 1) : (i & 7) >> 1); }

// Byte offset of 16-byte chunk c of row r of codes in a staged tile.
template <int D>
__device__ __forceinline__ uint32_t chunk4_at(int r, int c) { return D == 128 ? r * 64 + ((c ^ (r & 2)) << 4) : r * 32 + (c << 4); }

// A warp's share of the softmax over keys for 8 NT rows, transposed as in paged_attn.cu:
// keys and channels on the 16 rows of an MMA, query rows on its 8 columns.  Lane
// (g, t) = (lane / 4, lane % 4).
//   S^T  A: rows g, g + 8; lane t's channels are [t D/4, (t+1) D/4).  B: the same channels of
//        query row g.  C: rows g, g + 8 of query rows 2 t, 2 t + 1.
//   P^T  C transposed 8 x 8 at a time.
//   O^T  A: lane g's channels are [g D/8, (g+1) D/8), of which 2 j, 2 j + 1 are rows g and
//        g + 8 of MMA j; C: those channels of query rows 2 t, 2 t + 1.
template <int D, int NT, int LGK>
struct Tile4 {
    using St = Stage4<D, LGK>;
    static constexpr int KS = D / 16, MO = D / 16, ROW = D / 2, SROW = D / 16;
    // Keys whose scores a warp holds together: all of a tile, of 8 rows (64 requests of up to 16k tokens 128.6 us, 134.3 with
    // 32); of 16 rows half, as more would spill (48 in a window 33.1 us, 33.5 with 64).
    static constexpr int AT_ONCE = NT == 2 || LGK == 5 ? 32 : 64, U = AT_ONCE / 16;
    uint32_t q[NT][KS][2];
    float o[NT][MO][4];
    float m[NT][2], l[NT][2];                // rows 2 t, 2 t + 1: reference (log2), sum of P of this lane's keys

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int j = 0; j < MO; ++j) o[x][j][0] = o[x][j][1] = o[x][j][2] = o[x][j][3] = 0.0f;
            m[x][0] = m[x][1] = __int_as_float(0xff800000);
            l[x][0] = l[x][1] = 0.0f;
        }
    }

    // Weights of a tile whose keys every row sees, with the references as they are: no
    // maximum.  False if a row's may leave f16 (or it has no reference yet).
    __device__ __forceinline__ bool weights(const float (&s)[NT][U][4], const float (&zf)[NT][2], uint32_t (&p)[NT][U][2]) {
        float total[NT][2];
        bool ok = true;
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            total[x][0] = total[x][1] = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float e[2][2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float c = kUp - m[x][r];
                    e[r][0] = ex2(fmaf(s[x][u][r], zf[x][r], c)), e[r][1] = ex2(fmaf(s[x][u][2 + r], zf[x][r], c));
                    total[x][r] += e[r][0] + e[r][1];
                }
                p[x][u][0] = transpose8(pack_f16(e[0][0], e[1][0]));
                p[x][u][1] = transpose8(pack_f16(e[0][1], e[1][1]));
            }
            ok = ok && total[x][0] < kMostP4 && total[x][1] < kMostP4;
        }
        if (!__all_sync(0xFFFFFFFFu, ok)) return false;
#pragma unroll
        for (int x = 0; x < NT; ++x) l[x][0] += total[x][0], l[x][1] += total[x][1];
        return true;
    }

    // Keys [first, first + 16 U) of a tile in shared memory, whose own first is `key0`.  zf:
    // logit factor per row.  If masked, a row sees the keys [seen.x, seen.y] of the first
    // `stored` of the tile in its 16-key groups of `there`; else all of them.
    __device__ __forceinline__ void keys(uint32_t kb, int first, const float (&zf)[NT][2], bool masked, int key0, int stored,
                                         uint32_t there, const int2 *seen) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        constexpr uint32_t ALL = 0xFFFFFFFFu;
        const float NEG_INF = __int_as_float(0xff800000);
        const uint32_t vb = kb + St::V + first * ROW, ksb = kb + St::KS + first * SROW, vsb = kb + St::VS + first * SROW;
        kb += first * ROW, key0 += first, stored -= first, there >>= first / 16;
        const int kg = key_at(g);
        float s[NT][U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            constexpr int W = D / 32;                // words of 8 channels per lane and key
            uint32_t c[2][W], sc[2][W];              // codes and scale (both halves) of each
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = 16 * u + 8 * h + kg;
                if constexpr (D == 128) {
                    const uint4 v = lds128(kb + chunk4_at<D>(row, t));
                    c[h][0] = v.x, c[h][1] = v.y, c[h][2] = v.z, c[h][3] = v.w;
                    const uint32_t two = e4m3x2_to_f16x2(lds16(ksb + row * SROW + 2 * t));
                    sc[h][0] = sc[h][1] = __byte_perm(two, 0, 0x1010);
                    sc[h][2] = sc[h][3] = __byte_perm(two, 0, 0x3232);
                } else {
                    const uint2 v = lds64(kb + row * ROW + 8 * t);
                    c[h][0] = v.x, c[h][1] = v.y;
                    const uint32_t one = lds8(ksb + row * SROW + t);
                    sc[h][0] = sc[h][1] = e4m3x2_to_f16x2(one | one << 8);
                }
            }
#pragma unroll
            for (int x = 0; x < NT; ++x) s[x][u][0] = s[x][u][1] = s[x][u][2] = s[x][u][3] = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                uint32_t a[4], b[4];
                e2m1x8_to_f16(c[0][w], sc[0][w], a);
                e2m1x8_to_f16(c[1][w], sc[1][w], b);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int x = 0; x < NT; ++x)
                        mma_f16_16816(s[x][u], a[2 * k], b[2 * k], a[2 * k + 1], b[2 * k + 1], q[x][2 * w + k][0], q[x][2 * w + k][1]);
            }
        }
        uint32_t p[NT][U][2];
        if (masked || !weights(s, zf, p)) {
            bool grew = false;
            float grow[NT][2];
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                float w[2][2 * U];                   // [row][16 u + 8 h + key_at(g) at 2 u + h]
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int2 sees = seen[8 * x + 2 * t + r];
                    float z[2 * U], tz = NEG_INF;
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int key = 16 * u + 8 * h + kg;
                            float v = __fmul_rn(s[x][u][2 * h + r], zf[x][r]);
                            if (masked && !(key0 + key >= sees.x && key0 + key <= sees.y && key < stored && ((there >> u) & 1))) v = NEG_INF;
                            z[2 * u + h] = v;
                            tz = fmaxf(tz, v);
                        }
                    // the row's keys are spread over the 8 lanes of equal t
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) tz = fmaxf(tz, __shfl_xor_sync(ALL, tz, d));
                    const float m1 = fmaxf(m[x][r], tz), ref = m1 == NEG_INF ? 0.0f : m1;
                    grow[x][r] = ex2(m[x][r] - ref);
                    grew |= m1 != m[x][r];
                    m[x][r] = m1;
                    float sum = l[x][r] * grow[x][r];
#pragma unroll
                    for (int i = 0; i < 2 * U; ++i) {
                        const float e = ex2(__fadd_rn(z[i], -ref) + kUp);
                        sum += e;
                        w[r][i] = e;
                    }
                    l[x][r] = sum;
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) p[x][u][h] = transpose8(pack_f16(w[0][2 * u + h], w[1][2 * u + h]));
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
            constexpr int W = D / 64;                // words of 8 channels per lane and key
            uint32_t v[4][W], sc[4];                 // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of the contraction
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 16 * u + 8 * (i >> 1) + (i & 1 ? 7 - t : t);
                if constexpr (D == 128) {
                    const uint2 x = lds64(vb + chunk4_at<D>(row, g >> 1) + 8 * (g & 1));
                    v[i][0] = x.x, v[i][1] = x.y;
                    sc[i] = lds8(vsb + row * SROW + g);
                } else {
                    v[i][0] = lds32(vb + row * ROW + 4 * g);
                    sc[i] = lds8(vsb + row * SROW + (g >> 1));
                }
                // what is not stored has a weight of 0, but its scale may be NaN
                if (masked && !(row < stored && ((there >> u) & 1))) sc[i] = 0;
            }
            const uint32_t sa = e4m3x2_to_f16x2(sc[0] | sc[1] << 8), sb = e4m3x2_to_f16x2(sc[2] | sc[3] << 8);
            constexpr uint32_t LOW = 0x0F0F0F0Fu;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                // nibbles of two keys side by side: even channels, odd channels
                uint32_t ea[4], oa[4], eb[4], ob[4];
                e2m1x8_to_f16((v[0][w] & LOW) | ((v[1][w] << 4) & ~LOW), sa, ea);
                e2m1x8_to_f16(((v[0][w] >> 4) & LOW) | (v[1][w] & ~LOW), sa, oa);
                e2m1x8_to_f16((v[2][w] & LOW) | ((v[3][w] << 4) & ~LOW), sb, eb);
                e2m1x8_to_f16(((v[2][w] >> 4) & LOW) | (v[3][w] & ~LOW), sb, ob);
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int x = 0; x < NT; ++x)
                        mma_f16_16816(o[x][4 * w + b], ea[b], oa[b], eb[b], ob[b], p[x][u][0], p[x][u][1]);
            }
        }
    }
};

template <int D, int LGK>
constexpr int split4_smem() {
    constexpr int ring = kWarps4 * Stage4<D, LGK>::N * Stage4<D, LGK>::BYTES, merge = kWarps4 * 8 * (D + 4) * 4;
    return ring > merge ? ring : merge;
}

template <int D, int NT, bool HALF, int LGK>
__global__ void __launch_bounds__(kWarps4 * 32, per_sm4(D, NT)) paged_attn4_split_kernel(PagedAttnArgs a) {
    using St = Stage4<D, LGK>;
    constexpr int R = 8 * NT, K = St::KEYS, ROW = D / 2, SROW = D / 16, N = St::N;
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_st[kWarps4][8][2];
    __shared__ int2 s_seen[kWarps4][R];
    __shared__ uint32_t s_info[kWarps4][N];
    __shared__ int64_t s_sum[kWarps4];
    __shared__ Found s_found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const float NEG_INF = __int_as_float(0xff800000);
    // A tile's rows of one block are a piece: GR rows, GU pieces to a tile.
    const int lgGR = 31 - __clz(min(a.S, K)), lgGU = LGK - lgGR, GU = 1 << lgGU, GR = 1 << lgGR;
    static_assert(LGK >= 5 && LGK <= 7, "pieces of a tile: blocks are 16, 32, 64 or 128 tokens");
    pdl_wait();
    pdl_launch_dependents();
    using Work = SplitWork<R, K, kCost4>;
    const Plan plan = plan_of<Work>(a, blockIdx.x, gridDim.x, kWarps4, s_sum, &s_found);
    int64_t at = blockIdx.x * plan.share;
    const int64_t stop = min(plan.total, at + plan.share);
    if (tid == 0) a.join[blockIdx.x].last = -1;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (N * St::BYTES);
    // this lane's chunk of a copy by the warp, 512 bytes: 8 or 16 rows
    constexpr int CPR = D / 32, RPC = 32 / CPR;
    const uint32_t lane_to = chunk4_at<D>(lane / CPR, lane % CPR);
    constexpr int SC = St::SCALES / 16;              // chunks of a plane's scales
    constexpr bool BOTH = SC <= 16;                  // one copy takes the keys' and the values'
    static_assert(BOTH || SC == 32, "a lane's chunk of each plane's scales, or of one's");
    const bool scales = !BOTH || lane < 2 * SC, of_v = BOTH && lane >= SC;
    const int sc_at = BOTH ? lane & (SC - 1) : lane;
    static_assert(RPC % 4 == 0 && RPC <= 16, "the order of a row's chunks goes by its number modulo 4");
    int64_t base = plan.base;
    for (int b = plan.b; at < stop && b < a.B; ++b) {
        const Request rq = b == plan.b ? plan.rq : request_of(a, b);
        const int64_t end = base + Work::tiles(a, rq);
        const int low = Work::low_key(a, rq), key0 = Work::first_key(a, rq), rows = rq.n * a.G;
        while (at < stop && at < end) {
            // segment: tiles [ta, tb) of one unit
            const Place pl = Work::place(a, rq, at - base);
            const int64_t unit = at - pl.tile;       // its first place
            at = min(stop, unit + pl.tiles);
            const int h = pl.h, r0 = pl.r0, ta = max(0, pl.tile - kCost4), tb = (int)(at - unit) - kCost4;
            if (tb <= 0) continue;
            const bool first_part = ta == 0, whole = first_part && at == unit + pl.tiles;
            if (tid == 0 && first_part && !whole)
                a.join[blockIdx.x] = {rq.row0, h, r0, rows, (int)((unit + pl.tiles - 1) / plan.share), {0, 0}};

            // this warp's tiles are ta + warp + 4 i; lane holds (tile lane / GU, piece lane % GU) of BT of them
            const int BT = 32 >> lgGU, my_tile = lane >> lgGU, my_piece = lane & (GU - 1);
            const int todo = min(tb, Work::real_tiles(a, rq)) - ta;
            const int count = todo > warp ? (todo - warp + kWarps4 - 1) / kWarps4 : 0;
            const int32_t *table = a.table + b * a.table_stride;
            auto key_of = [&](int i) { return key0 + (ta + warp + (i + my_tile) * kWarps4) * K + GR * my_piece; };
            // rows that end before every row's window are not read: their blocks may be another request's by now
            auto asked = [&](int i) { return i + my_tile < count && key_of(i) < rq.kv && key_of(i) + GR > low; };
            auto entry = [&](int i) -> int32_t { return asked(i) ? table[key_of(i) / a.S] : -1; };
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
            int64_t off = -1;                        // first row of this lane's piece among the cache's, -1: not there
            uint32_t have = 0, whole_rows = 0;       // lanes whose piece is there; whose rows all are keys
            auto locate = [&](int i) {
                const bool ok = asked(i) && block >= 0 && block < a.n_blocks;
                if (asked(i) && !ok) flag_error(a.err_flag, CSA2_FLAG_BAD_INDEX);
                off = ok ? ((int64_t)block * a.Hkv + h) * a.S + (key_of(i) & (a.S - 1)) : -1;
                have = __ballot_sync(ALL, ok);
                whole_rows = __ballot_sync(ALL, ok && key_of(i) + GR <= rq.kv);
            };
            locate(0);
            uint32_t fill = 0, take = 0;             // next stages
            auto issue = [&](int i) {                // start the copies of this warp's tile i
                if (i < count) {
                    const int in = i & (BT - 1), who = in << lgGU;               // its place in the batch, its first lane
                    if (i && in == 0) {
                        block = block_next;
                        block_next = entry(i + BT);
                        locate(i);
                    }
                    const uint32_t dst = ring + fill * St::BYTES, mine = (1u << GU) - 1;
                    if (lane == 0) s_info[warp][fill] = ((have >> who) & mine) | (((whole_rows >> who) & mine) << 8);
                    if (lgGU == 0) {                 // all rows from one place
                        const int64_t row = __shfl_sync(ALL, off, who);
                        if (row >= 0) {
                            const uint8_t *kc = a.k_codes + row * ROW + 16 * lane, *vc = a.v_codes + row * ROW + 16 * lane;
#pragma unroll
                            for (int x = 0; x < K / RPC; ++x) {
                                cp_async16(dst + St::K + lane_to + 512 * x, kc + 512 * x, 16);
                                cp_async16(dst + St::V + lane_to + 512 * x, vc + 512 * x, 16);
                            }
                            if (scales) cp_async16(dst + St::KS + 16 * lane, (of_v ? a.v_scale4 : a.k_scale4) + row * SROW + 16 * sc_at, 16);
                            if (!BOTH) cp_async16(dst + St::VS + 16 * lane, a.v_scale4 + row * SROW + 16 * lane, 16);
                        }
                    } else {
#pragma unroll
                        for (int x = 0; x < K / RPC; ++x) {
                            const int64_t row = __shfl_sync(ALL, off, who + ((x * RPC + lane / CPR) >> lgGR));
                            if (row >= 0) {
                                const int64_t at = row * ROW + ((x * RPC + lane / CPR) & (GR - 1)) * ROW + 16 * (lane % CPR);
                                cp_async16(dst + St::K + lane_to + 512 * x, a.k_codes + at, 16);
                                cp_async16(dst + St::V + lane_to + 512 * x, a.v_codes + at, 16);
                            }
                        }
                        const int r = sc_at * (16 / SROW);                   // first row of this lane's scales
                        const int64_t row = __shfl_sync(ALL, off, who + (r >> lgGR)), at = (row + (r & (GR - 1))) * SROW;
                        if (row >= 0 && scales) {
                            cp_async16(dst + St::KS + 16 * lane, (of_v ? a.v_scale4 : a.k_scale4) + at, 16);
                            if (!BOTH) cp_async16(dst + St::VS + 16 * lane, a.v_scale4 + at, 16);
                        }
                    }
                    if (++fill == N) fill = 0;
                }
                cp_async_commit();
            };
#pragma unroll 1
            for (int i = 0; i < N - 1; ++i) issue(i);

            Tile4<D, NT, LGK> tile;
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
            __syncwarp();
            for (int i = 0; i < count; ++i) {
                issue(i + N - 1);
                cp_async_wait<N - 1>();
                __syncwarp();
                const uint32_t stage = take;
                if (++take == N) take = 0;
                const int key = key0 + (ta + warp + i * kWarps4) * K;
                const uint32_t info = s_info[warp][stage], full = (1u << GU) - 1;
                const bool masked = !__all_sync(ALL, key >= all_lo && key + K <= all_hi && (info >> 8) == full);
                uint32_t there = 0;
                if (masked)
                    for (int u = 0; u < GU; ++u)
                        if ((info >> u) & 1) there |= ((1u << (GR / 16)) - 1) << (u * (GR / 16));
#pragma unroll 1
                for (int first = 0; first < K; first += Tile4<D, NT, LGK>::AT_ONCE)
                    tile.keys(ring + stage * St::BYTES, first, zf, masked, key, rq.kv - key, there, s_seen[warp]);
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
                        s_st[warp][2 * t + r][1] = l * kDownFactor;
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
                    float M = NEG_INF, l = 0.0f, o[D / 16];
#pragma unroll
                    for (int w = 0; w < kWarps4; ++w) M = fmaxf(M, s_st[w][y][0]);
                    const float ref = M == NEG_INF ? 0.0f : M;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) o[c] = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWarps4; ++w) {
                        const float f = ex2(s_st[w][y][0] - ref);
                        l += s_st[w][y][1] * f;
                        const float *src = s_o + (w * 8 + y) * LD + part * (D / 16);
#pragma unroll
                        for (int c = 0; c < D / 16; c += 4) {
                            const float4 v = *reinterpret_cast<const float4 *>(src + c);
                            o[c] += f * v.x, o[c + 1] += f * v.y, o[c + 2] += f * v.z, o[c + 3] += f * v.w;
                        }
                    }
                    if (whole) {
                        const int tok = row / a.G;
                        store_row<D, HALF, 16>(a, (rq.row0 + tok) * a.Hq + h * a.G + row - tok * a.G, part, o, 1.0f, M, l);
                    } else {
                        float *dst = a.partial + ((2 * (int64_t)blockIdx.x + first_part) * R + 8 * x + y) * LD;
#pragma unroll
                        for (int c = 0; c < D / 16; c += 4)
                            *reinterpret_cast<float4 *>(dst + part * (D / 16) + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                        if (part == 0) *reinterpret_cast<float4 *>(dst + D) = make_float4(M, M, l, 0.0f);
                    }
                }
            }
            __syncthreads();
        }
        base = end;
    }
}

template <int D, int NT, bool HALF, int LGK = 6>
cudaError_t launch_split4(const PagedAttnArgs &a, int ctas, cudaStream_t stream) {
    static bool done[64];
    cudaError_t e = ensure_smem_limit((const void *)paged_attn4_split_kernel<D, NT, HALF, LGK>, split4_smem<D, LGK>(), done);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attn4_split_kernel<D, NT, HALF, LGK>, dim3(ctas), dim3(kWarps4 * 32), split4_smem<D, LGK>(), stream, a);
}
// Warps' tiles of 32 keys in place of 64, for 8 rows: a tile is done sooner, and where a CTA has few of
// them that is what counts.  8 KV heads, tiles of 64 and of 32: 1 request of up to 1000 tokens 8.8
// and 8.2 us, 64 of up to 1000 24.9 and 22.0, of up to 4000 47.3 and 45.6, of up to 8000 72.0 and 75.4,
// of up to 16k 127.7 and 136.3; 8 of up to 32k 40.3 and 39.8.  Of 64 channels 1 of up to 1000 7.4 and 7.0, 64 of up
// to 1000 16.9 and 15.6, of up to 2000 21.8 and 22.7, 8 of up to 8000 12.9 and 13.2.  The lengths are the
// GPU's: the rule goes by what the tables (or the windows) could hold, at most so many tiles of 64 keys per CTA.
// It is wrong where that says little: short contexts behind tables that could hold long ones get the long tiles (64 of up to
// 1000 tokens with room for 131072: 24.9 in place of 22.0), and of 64 channels the two sides are not parted by it, 64 of up
// to 1000 (18 tiles per CTA) want the short tiles and get the long ones, 1.3 us, as 8 of up to 8000 (17.5) want them.
constexpr int few4(int D) { return D == 128 ? 96 : 16; }
inline bool few_keys4(const PagedAttnArgs &a, int D, int max_new, int ctas) {
    const int64_t most = (int64_t)a.M * a.S, keys = a.window > 0 && a.window + (int64_t)max_new < most ? a.window + (int64_t)max_new : most;
    return (int64_t)a.B * a.Hkv * ((keys + 63) / 64) <= (int64_t)few4(D) * ctas;
}

// Requests of more rows per KV head than this are the tile kernel's.  24 requests of up to 16k tokens,
// 8 KV heads of 128 (of 64) channels, split and tile kernel: 16 rows 78 and 168 us (51, 135), 32 rows
// 140 and 169 (87, 136), 64 rows 263 and 173 (160, 137); of up to 2000 tokens 27 and 46 (19, 38), 38
// and 46 (27, 38), 62 and 48 (43, 39).
constexpr int kSplitRows4 = 32;
struct Choice4 {
    int NT, split_ctas, tc_ctas, split_rows;
};
inline Choice4 choose4(int B, int G, int D, int max_new) {
    const int64_t rows = (int64_t)G * max_new;
    Choice4 c = {(rows <= kSplitRows4 ? rows : G) <= 8 ? 1 : 2, 0, 0, 0x7FFFFFFF};
    if (rows > kSplitRows4) {               // a batch may hold requests of fewer rows, which the split kernel takes beside the other
        c.tc_ctas = paged_attn_tc_ctas();
        c.split_rows = B == 1 || G > kSplitRows4 ? 0 : (c.NT == 1 ? 8 : kSplitRows4);
    }
    if (c.split_rows) c.split_ctas = num_sms() * per_sm4(D, c.NT);
    return c;
}
inline size_t partial4_floats(const Choice4 &c, int D) { return (size_t)2 * c.split_ctas * 8 * c.NT * (D + 4); }

}  // namespace
}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_paged_attn_fp4_workspace_bytes(int B, int64_t T, int Hq, int Hkv, int D, int max_new) {
    if (B <= 0 || T <= 0 || Hkv <= 0 || Hq < Hkv || D <= 0 || max_new <= 0) return 0;
    const Choice4 c = choose4(B, Hq / Hkv, D, max_new);
    return (c.split_ctas + c.tc_ctas) * sizeof(JoinUnit) +
           (partial4_floats(c, D) + (size_t)2 * c.tc_ctas * kTcRows * (D + 4)) * sizeof(float);
}

extern "C" csa2_status csa2_paged_attn_fp4(int B, int64_t T, int Hq, int Hkv, int D, csa2_dtype dt, const void *q,
                                           int64_t q_token_stride, int64_t q_head_stride, const uint8_t *k_codes,
                                           const uint8_t *v_codes, const uint8_t *k_scales, const uint8_t *v_scales,
                                           int64_t n_blocks, int S, const int32_t *block_table, int M, int64_t table_stride,
                                           const int32_t *kv_len, const int32_t *cu_len, int max_new, int window,
                                           float sm_scale, void *out, float *lse, uint32_t *err_flag, void *workspace,
                                           size_t ws_bytes, csa2_stream_t stream) {
    clear_error();
    const csa2_status st = check_paged_attn(B, T, Hq, Hkv, D, dt, q_token_stride, q_head_stride, n_blocks, S, M, table_stride,
                                            max_new, window);
    if (st != CSA2_OK) return st;
    if (B == 0 || T == 0) return CSA2_OK;
    CSA2_REQUIRE(q && out && block_table && kv_len && cu_len, "paged_attn: null pointer");
    CSA2_REQUIRE((k_codes && v_codes && k_scales && v_scales) || n_blocks == 0, "paged_attn: null pointer");
    CSA2_REQUIRE(aligned(q, 16) && aligned(out, 16) && aligned(k_codes, 16) && aligned(v_codes, 16) && aligned(k_scales, 16) &&
                     aligned(v_scales, 16),
                 "paged_attn: q, out, codes and scales must be 16-byte aligned");
    CSA2_REQUIRE(aligned(block_table, 4) && aligned(kv_len, 4) && aligned(cu_len, 4) && aligned(lse, 4) && aligned(err_flag, 4),
                 "paged_attn: table, lengths, lse and flag must be 4-byte aligned");
    const size_t need = csa2_paged_attn_fp4_workspace_bytes(B, T, Hq, Hkv, D, max_new);
    if (need > 0 && (!workspace || ws_bytes < need || !aligned(workspace, 16))) {
        set_error("paged_attn: workspace of %zu bytes (16-byte aligned) needed, %zu given", need, ws_bytes);
        return CSA2_ERR_WORKSPACE;
    }
    const Choice4 c = choose4(B, Hq / Hkv, D, max_new);
    JoinUnit *join = (JoinUnit *)workspace;
    float *partial = (float *)(join + c.split_ctas + c.tc_ctas);
    const PagedAttnArgs a = {B, Hq, Hkv, Hq / Hkv, S, M, window < M * S ? window : 0, T, n_blocks, table_stride,
                             q_token_stride, q_head_stride, (const uint16_t *)q, k_codes, v_codes, nullptr, nullptr, k_scales,
                             v_scales, block_table, kv_len, cu_len, sm_scale * 1.4426950408889634f, (uint16_t *)out, lse,
                             err_flag, c.split_rows, join, join + c.split_ctas, partial, partial + partial4_floats(c, D)};
    const bool half = dt == CSA2_FP16;
    auto go = D == 64 ? (c.NT == 1 ? (few_keys4(a, D, max_new, c.split_ctas)
                                          ? (half ? launch_split4<64, 1, true, 5> : launch_split4<64, 1, false, 5>)
                                          : (half ? launch_split4<64, 1, true> : launch_split4<64, 1, false>))
                                   : (half ? launch_split4<64, 2, true> : launch_split4<64, 2, false>))
                      : (c.NT == 1 ? (few_keys4(a, D, max_new, c.split_ctas)
                                          ? (half ? launch_split4<128, 1, true, 5> : launch_split4<128, 1, false, 5>)
                                          : (half ? launch_split4<128, 1, true> : launch_split4<128, 1, false>))
                                   : (half ? launch_split4<128, 2, true> : launch_split4<128, 2, false>));
    if (c.split_ctas) CSA2_CUDA_CALL(go(a, c.split_ctas, stream_of(stream)), "paged_attn launch");
    if (c.tc_ctas) CSA2_CUDA_CALL(launch_paged_attn_tc(a, D, half, true, stream_of(stream)), "paged_attn tile launch");
    CSA2_CUDA_CALL(launch_paged_attn_join(a, D, c.NT, half, c.split_ctas, c.tc_ctas, stream_of(stream)), "paged_attn join launch");
    CSA2_LAUNCH_CHECK("paged_attn kernels");
    return CSA2_OK;
}
