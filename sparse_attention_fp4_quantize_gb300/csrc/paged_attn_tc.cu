// The tile kernel of csa2_paged_attn_fp8: prompts, and whatever else brings more
// rows per KV head than the split kernel's row tiles hold.
//
// A unit is 256 rows of one (request, KV head), two sub-tiles of 128, against
// tiles of 128 keys: 2 x 2 x 128 x 128 x D MACs per key tile on tcgen05 in f16
// with fp32 accumulators in TMEM.  Per key tile and sub-tile
//   S = Q . K^T      (M = 128 rows, N = 128 keys; Q and K tiles in shared memory)
//   P = f16 of the softmax weights, written over S in TMEM
//   O += P . V       (M = 128 rows, N = D; A = P from TMEM, V tile in shared memory)
// The E4M3 codes become f16 once per CTA and key tile; both sub-tiles use them.
// K is read K-major and V MN-major from the same core-matrix layout, so one
// conversion serves both.  Roles (13 warps):
//   warps 0-3, 4-7   softmax of sub-tile 0, 1: thread = row (TMEM lane), so the
//                    row's maximum and sum need no exchange; also load Q and
//                    store the output
//   warps 8-11       load codes (a key tile ahead, in registers), convert, store
//   warp 12          issues every MMA
// While one sub-tile's softmax runs, the tensor cores have the other's products.
// The running references M, Mv (paged_attn.cu) move only when a tile exceeds them
// by more than 2^8, so O in TMEM is rescaled rarely; the weights stay below 2^9.
#include "paged_attn.cuh"
#include "tc.cuh"

namespace csa2 {
namespace {

constexpr int kSoftWarps = 8, kConvWarps = 4, kMmaWarp = kSoftWarps + kConvWarps;
constexpr int kTcThreads = (kMmaWarp + 1) * 32;
constexpr uint32_t kPolls = 1u << 22;
constexpr float kSlack = 8.0f;               // log2: how far a tile may exceed a reference
constexpr int kMetas = 4;                    // key tiles whose scales are kept

struct TileMeta {
    float ks[8], vs[8];                      // scales of the 16-key groups
    uint32_t missing[4];                     // per converting warp: its groups that are not stored (a bit each)
};

template <int D>
struct Lay {
    static constexpr uint32_t GROUP = D * 16;            // core matrices of 8 rows: D / 8 x 128 bytes
    static constexpr uint32_t Q = 128 * D * 2, KV = kTcKeys * D * 2;
    static constexpr uint32_t OFF_Q = 0, OFF_K = 2 * Q, OFF_V = OFF_K + 2 * KV, OFF_META = OFF_V + 2 * KV,
                              OFF_BAR = OFF_META + kMetas * sizeof(TileMeta);
    static constexpr int BARS = 21;
    static constexpr uint32_t USED = OFF_BAR + BARS * 8 + 8;
    static constexpr uint32_t SMEM = USED + 128 > 120 * 1024 ? USED + 128 : 120 * 1024;   // one CTA per SM (TMEM)
    static constexpr uint32_t COL_S = 0, COL_O = 256;    // TMEM columns: S0, S1 (P over them), O0, O1
};

__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ uint64_t f2u(uint32_t lo, uint32_t hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ float2 un2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bounded wait of a whole warp (every lane gets the same answer) that also gives
// up once another warp has raised the abort word.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_word) {
    uint32_t ok = 0;
    for (uint32_t i = 0; i < kPolls && !ok; ++i) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (!ok && (i & 63) == 63 && *abort_word) break;
    }
    if (__all_sync(0xFFFFFFFFu, ok)) return true;
    *abort_word = 1;
    return false;
}

// The CTA's segments in order; every role walks them by itself.
struct Segment {
    Request rq;
    Place pl;
    int b, tb;                    // request, end of its key tiles [pl.tile, tb)
    int rows, key0;               // rows of the request and KV head; key of the unit's first tile
};
struct Walk {
    int64_t at, stop, base;
    int b;
    __device__ __forceinline__ bool next(const PagedAttnArgs &a, Segment &s) {
        for (; at < stop && b < a.B; ++b) {
            s.rq = request_of(a, b);
            const int64_t end = base + TcWork::tiles(a, s.rq);
            if (at < end) {
                s.pl = TcWork::place(a, s.rq, at - base);
                s.b = b;
                s.tb = (int)min((int64_t)s.pl.tiles, s.pl.tile + (stop - at));
                s.rows = s.rq.n * a.G;
                s.key0 = TcWork::first_key(a, s.rq, s.pl.r0);
                at += s.tb - s.pl.tile;
                return true;
            }
            base = end;
        }
        return false;
    }
};

template <int D, bool HALF>
__global__ void __launch_bounds__(kTcThreads, 1) paged_attn_tc_kernel(PagedAttnArgs a) {
    using L = Lay<D>;
    constexpr uint32_t ALL = 0xFFFFFFFFu;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((128u - (tc::smem_u32(smem_raw) & 127u)) & 127u);
    __shared__ int64_t s_sum[kTcThreads / 32], s_found[2];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sb = tc::smem_u32(smem);
    TileMeta *metas = reinterpret_cast<TileMeta *>(smem + L::OFF_META);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::OFF_BAR + L::BARS * 8);
    volatile int *abort_word = reinterpret_cast<volatile int *>(smem + L::OFF_BAR + L::BARS * 8 + 4);
    const uint32_t bar0 = sb + L::OFF_BAR;
    auto kfull = [&](int i) { return bar0 + 8u * i; };
    auto kempty = [&](int i) { return bar0 + 8u * (2 + i); };
    auto vfull = [&](int i) { return bar0 + 8u * (4 + i); };
    auto vempty = [&](int i) { return bar0 + 8u * (6 + i); };
    auto qfull = [&](int i) { return bar0 + 8u * (8 + i); };
    auto sfull = [&](int i) { return bar0 + 8u * (10 + i); };
    auto pfull = [&](int i) { return bar0 + 8u * (12 + i); };
    auto ofull = [&](int i) { return bar0 + 8u * (14 + i); };
    auto mfull = [&](int i) { return bar0 + 8u * (16 + i); };
    const uint32_t drain = bar0 + 8u * 20;
    const float NEG_INF = __int_as_float(0xff800000);

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(kfull(i), kConvWarps);
            tc::mbar_init(kempty(i), 1);
            tc::mbar_init(vfull(i), kConvWarps);
            tc::mbar_init(vempty(i), 1);
            tc::mbar_init(qfull(i), 4);
            tc::mbar_init(sfull(i), 1);
            tc::mbar_init(pfull(i), 4);
            tc::mbar_init(ofull(i), 1);
        }
        for (int i = 0; i < kMetas; ++i) tc::mbar_init(mfull(i), kConvWarps);
        tc::mbar_init(drain, 1);
        *abort_word = 0;
        tc::mbar_init_fence();
    }
    if (warp == 0) tc::tmem_alloc(tmem_slot, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();
    const Plan plan = plan_of<TcWork>(a, blockIdx.x, gridDim.x, kTcRound, s_sum, s_found);
    Walk walk;
    walk.at = blockIdx.x * plan.share;
    walk.stop = min(plan.total, walk.at + plan.share);
    walk.base = plan.base;
    walk.b = plan.b;
    bool run = true;

    if (warp == kMmaWarp) {
        // ---- every MMA: S of the next key tile goes out behind P V of this one
        constexpr uint32_t idesc_s = tc::idesc_f16_f32(128, kTcKeys, false, false);
        constexpr uint32_t idesc_o = tc::idesc_f16_f32(128, D, false, true);
        const uint64_t dq = tc::desc_noswizzle(sb + L::OFF_Q, 128, L::GROUP);
        const uint64_t dk = tc::desc_noswizzle(sb + L::OFF_K, 128, L::GROUP);
        const uint64_t dv = tc::desc_noswizzle(sb + L::OFF_V, L::GROUP, 128);
        uint32_t nk = 0, segs[2] = {0, 0}, np[2] = {0, 0};   // key tiles, segments and P tiles so far
        auto issue_s = [&](int sub, uint32_t tile, bool first) -> bool {
            if (first && !wait_bar(qfull(sub), segs[sub]++ & 1, abort_word)) return false;
            if (!wait_bar(kfull(tile & 1), (tile >> 1) & 1, abort_word)) return false;
            tc::fence_after();
            if (lane == 0) {
                const uint64_t q = tc::desc_at(dq, sub * L::Q), k = tc::desc_at(dk, (tile & 1) * L::KV);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc::mma_f16(tmem + L::COL_S + sub * 128, tc::desc_at(q, ks * 256), tc::desc_at(k, ks * 256), idesc_s,
                                ks > 0);
                tc::commit(sfull(sub));
            }
            __syncwarp();
            return true;
        };
        auto issue_o = [&](int sub, uint32_t tile, bool first) -> bool {
            if (!wait_bar(pfull(sub), np[sub]++ & 1, abort_word)) return false;
            if (!wait_bar(vfull(tile & 1), (tile >> 1) & 1, abort_word)) return false;
            tc::fence_after();
            if (lane == 0) {
                const uint64_t v = tc::desc_at(dv, (tile & 1) * L::KV);
#pragma unroll
                for (int ks = 0; ks < kTcKeys / 16; ++ks)
                    tc::mma_f16_ta(tmem + L::COL_O + sub * D, tmem + L::COL_S + sub * 128 + ks * 8,
                                   tc::desc_at(v, ks * 2 * L::GROUP), idesc_o, !first || ks > 0);
                tc::commit(ofull(sub));
            }
            __syncwarp();
            return true;
        };
        auto release = [&](uint32_t bar) {
            if (lane == 0) tc::commit(bar);
            __syncwarp();
        };
        Segment seg;
        bool more = walk.next(a, seg);
        int active = 0;
        if (more) {
            active = seg.rows - seg.pl.r0 > 128 ? 2 : 1;
            for (int sub = 0; run && sub < active; ++sub) run = issue_s(sub, nk, true);
            release(kempty(0));
        }
        while (run && more) {
            const int n = seg.tb - seg.pl.tile, subs = active;
            for (int j = 0; run && j < n; ++j, ++nk) {
                const bool last = j == n - 1;
                if (!last) {
                    for (int sub = 0; run && sub < subs; ++sub)
                        run = issue_o(sub, nk, j == 0) && issue_s(sub, nk + 1, false);
                    release(vempty(nk & 1));
                    release(kempty((nk + 1) & 1));
                } else {
                    for (int sub = 0; run && sub < subs; ++sub) run = issue_o(sub, nk, j == 0);
                    release(vempty(nk & 1));
                    more = walk.next(a, seg);
                    if (run && more) {
                        active = seg.rows - seg.pl.r0 > 128 ? 2 : 1;
                        for (int sub = 0; run && sub < active; ++sub) run = issue_s(sub, nk + 1, true);
                        release(kempty((nk + 1) & 1));
                    }
                }
            }
        }
    } else if (warp >= kSoftWarps) {
        // ---- codes -> f16 tiles.  A warp takes 32 keys of a tile; lane = (row of
        // 8, 16-byte chunk), so a quarter-warp's stores fill a core matrix.
        // Scales go to a ring of kMetas: tile j + 4's are written once V of tile j + 3
        // is, for which P V of tile j + 1 had to be done, so both softmaxes are past
        // tile j and its slot is free.
        constexpr int CH = D / 64, N = 4 * CH;           // 64-byte column groups, loads per thread and operand
        const int cw = warp - kSoftWarps, row = lane & 7, chunk = lane >> 3;
        uint32_t nt = 0;
        Segment ahead;
        uint4 kc[N], vc[N];
        float sc[2][2] = {};
        uint32_t miss = 0;
        int tile_ahead = 0;
        bool have = walk.next(a, ahead);
        int32_t blk[2];
        auto blocks = [&]() {                            // block ids of this warp's two 16-key groups of the tile ahead
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int key = ahead.key0 + tile_ahead * kTcKeys + 32 * cw + 16 * u;
                blk[u] = key < ahead.rq.kv ? a.table[ahead.b * a.table_stride + key / a.S] : -1;
            }
        };
        int64_t off[2];
        auto offsets = [&]() {
            miss = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int key = ahead.key0 + tile_ahead * kTcKeys + 32 * cw + 16 * u;
                const bool there = key < ahead.rq.kv, ok = there && blk[u] >= 0 && blk[u] < a.n_blocks;
                if (there && !ok && lane == 0) flag_error(a.err_flag, CSA2_FLAG_BAD_INDEX);
                if (!ok) miss |= 1u << (2 * cw + u);
                const int64_t bh = ok ? (int64_t)blk[u] * a.Hkv + ahead.pl.h : 0;
                sc[u][0] = ok ? a.k_scale[bh] : 0.0f;
                sc[u][1] = ok ? a.v_scale[bh] : 0.0f;
                off[u] = ok ? (bh * a.S + key % a.S) * D : -1;
            }
        };
        auto fetch = [&](const uint8_t *codes, uint4 (&c)[N]) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int g = i / CH, r = 8 * (g & 1) + row;                 // 8-key group of the warp's 32, row of its 16
                const int key = ahead.key0 + tile_ahead * kTcKeys + 32 * cw + 16 * (g >> 1) + r;
                c[i] = make_uint4(0, 0, 0, 0);                               // rows that are not there read as zero
                if (off[g >> 1] >= 0 && key < ahead.rq.kv)
                    c[i] = *reinterpret_cast<const uint4 *>(codes + off[g >> 1] + r * D + 64 * (i % CH) + 16 * chunk);
            }
        };
        auto store = [&](uint32_t dst, const uint4 (&c)[N]) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int g = i / CH;
                const uint32_t to = dst + (4 * cw + g) * L::GROUP + (8 * (i % CH) + 2 * chunk) * 128 + row * 16;
                uint32_t h[8];
                e4m3x4_to_f16x2x2(c[i].x, h[0], h[1]);
                e4m3x4_to_f16x2x2(c[i].y, h[2], h[3]);
                e4m3x4_to_f16x2x2(c[i].z, h[4], h[5]);
                e4m3x4_to_f16x2x2(c[i].w, h[6], h[7]);
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to + 128), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7]) : "memory");
            }
        };
        auto step = [&]() {                              // the tile after the one ahead
            if (++tile_ahead >= ahead.tb) {
                have = walk.next(a, ahead);
                tile_ahead = ahead.pl.tile;
            }
        };
        if (have) {
            tile_ahead = ahead.pl.tile;
            blocks();
            offsets();
            fetch(a.k_codes, kc);
            fetch(a.v_codes, vc);
        }
        while (run && have) {
            const int buf = nt & 1;
            const uint32_t par = ((nt >> 1) & 1) ^ 1;
            if (!wait_bar(kempty(buf), par, abort_word)) break;
            TileMeta &m = metas[nt % kMetas];
            if (lane == 0) {
#pragma unroll
                for (int u = 0; u < 2; ++u) m.ks[2 * cw + u] = sc[u][0], m.vs[2 * cw + u] = sc[u][1];
                m.missing[cw] = miss;
                arrive(mfull(nt % kMetas));
            }
            store(sb + L::OFF_K + buf * L::KV, kc);
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive(kfull(buf));
            step();
            if (have) {
                blocks();
                offsets();
                fetch(a.k_codes, kc);
            }
            if (!wait_bar(vempty(buf), par, abort_word)) break;
            store(sb + L::OFF_V + buf * L::KV, vc);
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive(vfull(buf));
            if (have) fetch(a.v_codes, vc);
            ++nt;
        }
    } else {
        // ---- softmax: thread = row
        const int sub = warp >> 2, rr = 32 * (warp & 3) + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + lanes + L::COL_S + sub * 128, to = tmem + lanes + L::COL_O + sub * D;
        uint32_t nt = 0, ns = 0;                         // key tiles of the CTA so far; of this sub-tile
        Segment seg, nxt;
        bool more = walk.next(a, seg);
        float zf = 0.0f, zf_next = 0.0f;
        auto load_q = [&](const Segment &s) {            // this thread's row of Q into shared memory, its logit factor
            const int row = s.pl.r0 + 128 * sub + rr;
            const bool real = row < s.rows;
            const int tok = real ? row / a.G : 0, hq = s.pl.h * a.G + (real ? row - tok * a.G : 0);
            const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (s.rq.row0 + tok) * a.q_token_stride + hq * a.q_head_stride);
            float top = 0.0f;
            if (!HALF) {                                 // read twice, the second time from L1: registers are scarce
#pragma unroll 4
                for (int i = 0; i < D / 8; ++i) {
                    const uint4 v = real ? src[i] : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const float2 f = unpack_in<HALF>(w[c]);
                        top = max3(top, fabsf(f.x), fabsf(f.y));
                    }
                }
            }
            const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
            const float mul = HALF ? 1.0f : __uint_as_float((uint32_t)(127 + 14 - e) << 23);
            zf_next = fabsf(a.logit_scale) / mul;
            const uint32_t flip = a.logit_scale < 0.0f ? 0x80008000u : 0u;   // the sign goes to q: factors are not negative
            const uint32_t dst = sb + L::OFF_Q + sub * L::Q + (rr >> 3) * L::GROUP + (rr & 7) * 16;
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                const uint4 v = real ? src[i] : make_uint4(0, 0, 0, 0);
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (!HALF) {
                        const float2 f = unpack_in<HALF>(w[c]);
                        w[c] = pack_f16(f.x * mul, f.y * mul);
                    }
                    w[c] ^= flip;
                }
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst + i * 128), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive(qfull(sub));
        };
        auto takes = [&](const Segment &s) { return sub == 0 || s.rows - s.pl.r0 > 128; };
        if (more && takes(seg)) load_q(seg);
        while (run && more) {
            const int n = seg.tb - seg.pl.tile;
            bool nxt_more = false;
            if (!takes(seg)) {
                nt += n;
                nxt_more = walk.next(a, nxt);
                if (nxt_more && takes(nxt)) load_q(nxt);
            } else {
                zf = zf_next;
                const int row = seg.pl.r0 + 128 * sub + rr;
                const bool real = row < seg.rows;
                const int tok = real ? row / a.G : 0, hq = seg.pl.h * a.G + (real ? row - tok * a.G : 0);
                // rows that are not there see everything: they hold no warp back, and are not stored
                const int pos = real ? max(-1, seg.rq.kv - seg.rq.n + tok) : 0x7FFFFFF0;
                const int first = real && a.window > 0 ? max(0, pos - a.window + 1) : 0;
                float M = NEG_INF, MV = NEG_INF, l = 0.0f;
                for (int j = 0; j < n; ++j, ++nt, ++ns) {
                    if (!wait_bar(mfull(nt % kMetas), (nt / kMetas) & 1, abort_word) ||
                        !wait_bar(sfull(sub), ns & 1, abort_word)) {
                        run = false;
                        break;
                    }
                    tc::fence_after();
                    const TileMeta &m = metas[nt % kMetas];
                    const int key0 = seg.key0 + (seg.pl.tile + j) * kTcKeys;
                    const uint32_t missing = m.missing[0] | m.missing[1] | m.missing[2] | m.missing[3];
                    const int lo = max(first - key0, 0), hi = min(pos + 1 - key0, kTcKeys);
                    const bool masked = __any_sync(ALL, lo > 0 || hi < kTcKeys || missing != 0);
                    // does the row see key k of the tile
                    auto sees = [&](int k) { return k >= lo && k < hi && !((missing >> (k >> 4)) & 1); };
                    float tz = NEG_INF, tv = NEG_INF;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32];
                        tc::tmem_ld32(ts + 32 * c, r);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const float vs = m.vs[2 * c + g], f = zf * m.ks[2 * c + g];
                            float t = NEG_INF;
                            if (masked) {
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    if (sees(32 * c + 16 * g + i)) t = fmaxf(t, __uint_as_float(r[16 * g + i]));
                            } else {
#pragma unroll
                                for (int i = 0; i < 16; i += 2)
                                    t = max3(t, __uint_as_float(r[16 * g + i]), __uint_as_float(r[16 * g + i + 1]));
                            }
                            t = t == NEG_INF ? t : t * f;
                            tz = fmaxf(tz, t);
                            tv = fmaxf(tv, t + (float)((int)((__float_as_uint(vs) >> 23) & 0xFFu) - 127));
                        }
                    }
                    if (tz > M + kSlack || (M == NEG_INF && tz > M)) {
                        l *= ex2(M - tz);
                        M = tz;
                    }
                    const bool move = tv > MV + kSlack || (MV == NEG_INF && tv > MV);
                    const float grow = move ? ex2(MV - tv) : 1.0f;
                    if (move) MV = tv;
                    if (j > 0 && __any_sync(ALL, move)) {            // O so far to the new reference, once P V is done
                        if (!wait_bar(ofull(sub), (ns - 1) & 1, abort_word)) {
                            run = false;
                            break;
                        }
                        tc::fence_after();
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t r[32];
                            tc::tmem_ld32(to + 32 * c, r);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * grow);
                            tc::tmem_st32(to + 32 * c, r);
                        }
                    }
                    const float ref = M == NEG_INF ? 0.0f : M, refv = MV == NEG_INF ? 0.0f : MV;
                    const float g2 = ex2(ref - refv);
                    const uint64_t nref = f2(-ref, -ref);
                    uint64_t sum = f2(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t r[32], p[16];
                        tc::tmem_ld32(ts + 32 * c, r);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            const float f = zf * m.ks[2 * c + g], w = fminf(m.vs[2 * c + g] * g2, 1e38f);
                            const uint64_t ff = f2(f, f), ww = f2(w, w);
#pragma unroll
                            for (int i = 0; i < 16; i += 2) {
                                const float2 z = un2(fma2(f2u(r[16 * g + i], r[16 * g + i + 1]), ff, nref));
                                float e0 = ex2(z.x), e1 = ex2(z.y);
                                if (masked) {
                                    if (!sees(32 * c + 16 * g + i)) e0 = 0.0f;
                                    if (!sees(32 * c + 16 * g + i + 1)) e1 = 0.0f;
                                }
                                const uint64_t e = f2(e0, e1);
                                sum = add2(sum, e);
                                const float2 x = un2(mul2(e, ww));
                                p[8 * g + i / 2] = pack_f16(x.x, x.y);
                            }
                        }
                        tc::tmem_st16(ts + 16 * c, p);
                    }
                    const float2 s2 = un2(sum);
                    l += s2.x + s2.y;
                    tc::tmem_st_wait();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) arrive(pfull(sub));
                }
                if (!run) break;
                nxt_more = walk.next(a, nxt);
                if (nxt_more && takes(nxt)) load_q(nxt);             // Q is free: S of the last tile is done
                if (!wait_bar(ofull(sub), (ns - 1) & 1, abort_word)) break;
                tc::fence_after();
                const bool whole = seg.pl.tile == 0 && seg.tb == seg.pl.tiles;
                const float ref = M == NEG_INF ? 0.0f : M, refv = MV == NEG_INF ? 0.0f : MV;
                const float scale = exp2f(refv - ref), inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
                const int64_t o_row = (seg.rq.row0 + tok) * a.Hq + hq;
                float *part = a.partial_tc + ((2 * (int64_t)blockIdx.x + (seg.pl.tile == 0)) * kTcRows + 128 * sub + rr) * (D + 4);
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t r[32];
                    tc::tmem_ld32(to + 32 * c, r);
                    tc::tmem_ld_wait();
                    if (!real) continue;
                    if (whole) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = pack_out<HALF>(__uint_as_float(r[2 * i]) * scale * inv, __uint_as_float(r[2 * i + 1]) * scale * inv);
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out + o_row * D + 32 * c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(part + 32 * c + 4 * i) = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                    }
                }
                tc::fence_before();
                if (real && whole && a.lse)
                    a.lse[o_row] = l > 0.0f || l != l ? (M + log2f(l)) * 0.69314718055994531f : NEG_INF;
                if (real && !whole) *reinterpret_cast<float4 *>(part + D) = make_float4(M, MV, l, 0.0f);
            }
            seg = nxt;
            more = nxt_more;
        }
    }
    if (*abort_word && warp == kMmaWarp) {
        // MMAs still in flight end before the tensor memory is given back (bounded)
        if (lane == 0) tc::commit(drain);
        tc::mbar_wait(drain, 0, kPolls);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (tid == 0 && *abort_word) flag_error(a.err_flag, CSA2_FLAG_TIMEOUT);
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

template <int D, bool HALF>
cudaError_t go(const PagedAttnArgs &a, cudaStream_t stream) {
    static bool done[64];
    cudaError_t e = ensure_smem_limit((const void *)paged_attn_tc_kernel<D, HALF>, Lay<D>::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attn_tc_kernel<D, HALF>, dim3(paged_attn_tc_ctas()), dim3(kTcThreads), Lay<D>::SMEM, stream, a);
}

}  // namespace

int paged_attn_tc_ctas() { return num_sms(); }

cudaError_t launch_paged_attn_tc(const PagedAttnArgs &a, int D, bool half, cudaStream_t stream) {
    if (half) return D == 64 ? go<64, true>(a, stream) : go<128, true>(a, stream);
    return D == 64 ? go<64, false>(a, stream) : go<128, false>(a, stream);
}

}  // namespace csa2
